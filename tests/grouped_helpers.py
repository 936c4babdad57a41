"""Shared helpers of the grouped-product tests: integer-valued inputs, for which every fp32 partial
sum is exact, and the operators in plain 64-bit torch on the CPU."""
import numpy as np
import torch

TORCH_DT = {"f32": torch.float32, "f16": torch.float16, "bf16": torch.bfloat16}
SENTINEL = 77.0        # exact in every type; marks elements that must stay untouched


def offsets_of(counts, start=0):
    return np.concatenate([[start], start + np.cumsum(counts)]).astype(np.int32)


def ints(g, shape, lo, hi, dtype):
    return torch.from_numpy(g.integers(lo, hi + 1, size=shape).astype(np.float32)).to(dtype)


def rounded(x, dtype):
    """A 64-bit result in the output type (one rounding to nearest even; the values here are
    integers below 2^24, which float32 holds, so the step through it adds none)."""
    return x.to(torch.float32).to(dtype)


def rows_reference(A, B, C, D0, offs, op_b, bias, alpha, beta, epilogue):
    """D of a rows plan in 64 bits, starting from D0 (the rows outside the ranges)."""
    D = D0.double().clone()
    for e, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        if lo == hi:
            continue
        b = B[e if B.shape[0] > 1 else 0].double()
        d = alpha * (A[lo:hi].double() @ (b if op_b == "N" else b.t()))
        if epilogue == "gate":
            d = torch.where(C[lo:hi].double() > 0, d, torch.zeros_like(d))
        elif beta:
            d = d + beta * C[lo:hi].double()
        if "bias" in epilogue:
            d = d + bias[e].double()
        if "relu" in epilogue:
            d = torch.clamp(d, min=0)
        D[lo:hi] = d
    return D


def grad_reference(A, B, C, offs, alpha, beta):
    """(D, bias_grad) of a gradient plan in 64 bits."""
    D, sums = [], []
    for e, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        d = alpha * (A[lo:hi].double().t() @ B[lo:hi].double())
        D.append(d + beta * C[e].double() if beta else d)
        sums.append(B[lo:hi].double().sum(0))
    return torch.stack(D), torch.stack(sums)
