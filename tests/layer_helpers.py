"""Shared helpers of the tests of a layer's products: the activations and their slopes in 64 bits, and
bounds of the kernels' errors counted in roundings."""
import math

import torch

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]
U = 2.0 ** -24                                  # half a step of fp32, relative
A, B = 2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715
# relative error of the fitted share of the normal distribution's far side, by output type
FIT = {torch.float16: 8.3e-6, torch.bfloat16: 8.3e-6, torch.float32: 8.4e-8}


def phi64(z):
    """The normal distribution function (torch.special.ndtr is off by 1e-5 of it at -7, where 64-bit erfc has
    all its digits)."""
    return torch.erfc(z * -math.sqrt(0.5)) / 2


def act64(name, z):
    if name == "relu":
        return torch.where(z < 0, torch.zeros_like(z), z)
    if name == "gelu":
        return z * phi64(z)
    if name == "gelu_tanh":
        return z * torch.sigmoid(z * (A + B * z * z))
    if name == "silu":
        return z * torch.sigmoid(z)
    return z


def slope64(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).double()
    if name == "gelu":
        return phi64(z) + z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)
    w, dw = (z, torch.ones_like(z)) if name == "silu" else (z * (A + B * z * z), A + 3 * B * z * z)
    s = torch.sigmoid(w)
    return s + z * dw * s * torch.sigmoid(-w)


def act_bound(name, z, dtype):
    """Bound of |act computed - act64| for an exact z.  Logistic ones: the exponent -w log2(e) has up to
    four roundings, |w| 4 U in e^-w, the exponential one step (2 U), 1 + e^-w one rounding, the
    reciprocal one step, the product one.  gelu: the exponent -z^2 / 2 has two roundings (z^2 U), the
    exponential one step, the polynomial's argument (a rounding and one step) moves its value by at
    most four times its own error, and its terms (of both signs, 2.3 times the sum in size at most) add
    up with one rounding each: 6 + 12 + 5 roundings and the product.  Results below 2^-126 may become 0."""
    v = act64(name, z).abs()
    if name in ("silu", "gelu_tanh"):
        w = z.abs() if name == "silu" else (z * (A + B * z * z)).abs()
        return v * (4 * w + 8) * U + 1e-37
    if name == "gelu":
        return v * ((z * z + 26) * U + FIT[dtype]) + 1e-37
    return torch.zeros_like(z)


def slope_bound(name, z, dtype):
    """The same for the slope; its two terms have their own errors: s as above, and u s (e^-w s), whose
    factors have up to three roundings more than twice s's."""
    if name == "gelu":
        p = phi64(z)
        q = (z * torch.exp(-z * z / 2) / math.sqrt(2 * math.pi)).abs()
        return p * ((z * z + 26) * U + FIT[dtype]) + q * (z * z + 6) * U + 1e-37
    if name in ("silu", "gelu_tanh"):
        w, dw = (z, torch.ones_like(z)) if name == "silu" else (z * (A + B * z * z), A + 3 * B * z * z)
        s, t = torch.sigmoid(w), torch.sigmoid(-w)
        return s * (4 * w.abs() + 8) * U + (z * dw * s * t).abs() * (12 * w.abs() + 24) * U + 1e-28
    return torch.zeros_like(z)


def rounding(x, dtype):
    """Half a step of the output type at x, at most (the smallest normal's below it)."""
    f = torch.finfo(dtype)
    return x.abs().clamp(min=f.tiny) * f.eps / 2


def close(got, want, bound, what=""):
    got, want = got.double().cpu(), want.double().cpu()
    bad = ~((got - want).abs() <= bound)
    if bad.any():
        i = tuple(bad.nonzero()[0].tolist())
        raise AssertionError(f"{what}: {int(bad.sum())} of {bad.numel()} too far, first {i}: {got[i]:.9g} for "
                             f"{want[i]:.9g}, bound {float(bound[i]):.3g}")
