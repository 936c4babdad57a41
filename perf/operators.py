"""Products of a mixture-of-experts layer, case by case: the plain form of each operator in
elementary torch operations, and the framework's own kernels on the same inputs.

  rows   products grouped by expert over ragged row ranges, with the fused epilogue (a layer's
         forward pass, its gradient towards the input, and single tokens)
  grad   the weight gradients of such a layer, summed over ragged row ranges, with the bias's
  quant  products with 4-bit weights and a scale (and zero point) per block of K, for one
         weight matrix or one per expert

`own` selects the framework's kernels; otherwise run() computes the plain form in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}


# ---- cases -------------------------------------------------------------------------------------
# rows: rows of the token buffer, the last `pad` of them behind the last expert's range (a buffer
# is allocated for the largest batch); experts: number of weight matrices; K x N: each of them
# (op_b T: stored N x K, the layout of a linear layer's weight); epi: the fused epilogue
# (gate: a ReLU's gradient, D = product where C > 0); skew: spread of the router's logits.

def listed():
    return [
        # one small model's expert layer for a single request: launch latency counts
        {"name": "rows_decode_small", "op": "rows", "rows": 8, "pad": 0, "experts": 16, "K": 2048,
         "N": 1024, "op_b": "T", "ab": "f16", "cd": "f16", "epi": "none", "skew": 0.5},
        # a batch of 8 requests, 8 experts each: every chosen expert's weights are read once
        {"name": "rows_decode", "op": "rows", "rows": 64, "pad": 0, "experts": 64, "K": 4096,
         "N": 2048, "op_b": "T", "ab": "bf16", "cd": "bf16", "epi": "none", "skew": 0.5},
        # a short prompt over many experts, a few tens of rows each
        {"name": "rows_mid", "op": "rows", "rows": 2100, "pad": 37, "experts": 32, "K": 2048,
         "N": 1408, "op_b": "N", "ab": "f16", "cd": "f16", "epi": "bias_relu", "skew": 1.0},
        # training's forward pass: few wide experts, thousands of rows each
        {"name": "rows_train", "op": "rows", "rows": 32768, "pad": 0, "experts": 8, "K": 4096,
         "N": 14336, "op_b": "T", "ab": "bf16", "cd": "bf16", "epi": "bias_relu", "skew": 0.5},
        # the gradient towards the hidden activations, through the ReLU between the two layers
        {"name": "rows_dgrad", "op": "rows", "rows": 16384, "pad": 500, "experts": 16, "K": 2048,
         "N": 8192, "op_b": "T", "ab": "bf16", "cd": "bf16", "epi": "gate", "skew": 0.5},
        # odd everything: no row starts on a 16-byte boundary
        {"name": "rows_odd", "op": "rows", "rows": 3001, "pad": 13, "experts": 7, "K": 1001,
         "N": 777, "op_b": "N", "ab": "f16", "cd": "f32", "epi": "bias", "skew": 1.0},
        # training's weight gradients with the bias's, kept in 32 bits
        {"name": "grad_train", "op": "grad", "rows": 16384, "pad": 0, "experts": 16, "M": 4096,
         "N": 2048, "ab": "bf16", "cd": "f32", "bias": True, "skew": 0.5},
        # a small layer's weight gradients in the weights' own type, ragged ends
        {"name": "grad_small", "op": "grad", "rows": 1003, "pad": 3, "experts": 8, "M": 1024,
         "N": 704, "ab": "f16", "cd": "f16", "bias": False, "skew": 1.0},
        # one token through one layer: a matrix-vector product
        {"name": "quant_token", "op": "quant", "rows": 1, "pad": 0, "experts": 1, "K": 4096,
         "N": 4096, "block": 128, "zeros": False, "ab": "bf16", "cd": "bf16", "epi": "none",
         "skew": 0.0},
        # a batch of single tokens through a wide layer, zero points and a fine block
        {"name": "quant_batch", "op": "quant", "rows": 16, "pad": 0, "experts": 1, "K": 4096,
         "N": 16384, "block": 64, "zeros": True, "ab": "f16", "cd": "f16", "epi": "bias_relu",
         "skew": 0.0},
        # the experts of a served layer in 4 bits, a batch of 8 requests, 4 experts each
        {"name": "quant_experts", "op": "quant", "rows": 32, "pad": 0, "experts": 32, "K": 4096,
         "N": 2048, "block": 128, "zeros": False, "ab": "bf16", "cd": "bf16", "epi": "none",
         "skew": 0.5},
        # a prompt through the same 4-bit layer
        {"name": "quant_prompt", "op": "quant", "rows": 2000, "pad": 0, "experts": 1, "K": 4096,
         "N": 4096, "block": 128, "zeros": True, "ab": "bf16", "cd": "bf16", "epi": "bias",
         "skew": 0.0},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over its logarithm: whole 16-byte chunks three times out of four, else any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["rows", "grad", "quant"])
    while True:
        c = {"op": op, "rows": _log(rng, 1, 32768), "experts": _log(rng, 1, 64)}
        c["pad"] = rng.randrange(0, max(1, c["rows"] // 16)) if rng.random() < 0.5 else 0
        c["skew"] = rng.choice([0.0, 0.5, 1.0])
        c["ab"] = rng.choice(["f16", "bf16"])
        c["cd"] = rng.choice([c["ab"], "f32"])
        if op == "rows":
            c.update(K=_size(rng, 64, 8192), N=_size(rng, 64, 16384), op_b=rng.choice("NT"),
                     epi=rng.choice(["none", "bias", "bias_relu", "gate"]))
            k, n = c["K"], c["N"]
        elif op == "grad":
            c.update(M=_size(rng, 64, 8192), N=_size(rng, 64, 8192),
                     bias=rng.random() < 0.5)
            k, n = c["M"], c["N"]
        else:
            c["rows"] = _log(rng, 1, 4096)
            c["pad"] = 0
            if rng.random() < 0.5:
                c["experts"] = 1
            c["block"] = rng.choice([32, 64, 128])
            c.update(K=c["block"] * _log(rng, 2, 8192 // c["block"]), N=_size(rng, 64, 16384),
                     zeros=rng.random() < 0.5, epi=rng.choice(["none", "bias", "bias_relu"]))
            k, n = c["K"], c["N"]
        # no more than the largest listed case: products, weights, and a buffer's padding
        if (c["rows"] * k * n <= 32768 * 4096 * 14336 and c["experts"] * k * n <= 64 * 4096 * 4096
                and c["experts"] * c["rows"] * (k + n) <= 1 << 31):
            return c


# ---- inputs ------------------------------------------------------------------------------------

def _counts(case, seed):
    """Rows of every expert, from a router's skewed probabilities."""
    g = np.random.default_rng([seed, 1])
    e, used = case["experts"], case["rows"] - case["pad"]
    p = np.exp(case["skew"] * g.standard_normal(e))
    return g.multinomial(used, p / p.sum())


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    E, T = case["experts"], case["rows"]
    ab, cd = TORCH[case["ab"]], TORCH[case["cd"]]
    counts = _counts(case, seed)
    ends = np.concatenate([[0], np.cumsum(counts)])

    def normal(*shape, scale=1.0, dtype=ab):
        out = torch.empty(shape, dtype=dtype, device=DEV)
        # in slices along the first axis: a stack of weights has several GB in 32 bits
        for i in range(shape[0]) if len(shape) == 3 else [slice(None)]:
            out[i] = torch.randn(out[i].shape, generator=g, device=DEV) * scale
        return out

    s = {"case": dict(case), "used": int(ends[-1]), "most": int(counts.max()),
         "offsets": torch.tensor(ends, dtype=torch.int32, device=DEV)}
    N = case["N"]
    if case["op"] == "grad":
        M = case["M"]
        s["A"], s["B"] = normal(T, M), normal(T, N, scale=1 / 8)
        s["D"] = torch.zeros(E, M, N, dtype=cd, device=DEV)
        s["bias"] = torch.zeros(E, N, dtype=torch.float32, device=DEV) if case["bias"] else None
    else:
        K = case["K"]
        s["A"] = normal(T, K)
        s["bias"] = (normal(E, N, scale=0.5, dtype=torch.float32) if "bias" in case["epi"] else None)
        s["D"] = torch.zeros(T, N, dtype=cd, device=DEV)
        if case["op"] == "rows":
            s["B"] = normal(E, *((K, N) if case["op_b"] == "N" else (N, K)), scale=K ** -0.5)
            s["C"] = normal(T, N, dtype=cd) if case["epi"] == "gate" else None
        else:
            nb = K // case["block"]
            s["Q"] = torch.randint(0, 256, (E, N, K // 2), generator=g, dtype=torch.uint8, device=DEV)
            # scales of weights with a spread of about 1 / sqrt(K)
            s["scales"] = ((torch.rand(E, N, nb, generator=g, device=DEV) + 0.5)
                           * (K ** -0.5 / 4.6)).to(ab)
            s["zeros"] = (torch.randint(5, 12, (E, N, nb), generator=g, dtype=torch.uint8, device=DEV)
                          if case["zeros"] else None)
    if own:
        s["plan"] = _plan(case)
    return s


def _plan(c):
    import tiled_gemm_epilogues_amd as tge
    if c["op"] == "rows":
        return tge.GroupedPlan(c["rows"], c["N"], c["K"], c["experts"], c["op_b"], ab=c["ab"],
                               cd=c["cd"], epilogue=c["epi"])
    if c["op"] == "grad":
        return tge.GroupedGradPlan(c["rows"], c["M"], c["N"], c["experts"], ab=c["ab"], cd=c["cd"])
    return tge.QuantPlan(c["rows"], c["N"], c["K"], c["block"], c["experts"], zeros=c["zeros"],
                         ab=c["ab"], cd=c["cd"], epilogue=c["epi"])


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    if own:
        if c["op"] == "rows":
            s["plan"].run(s["A"], s["B"], s["C"], s["D"], s["offsets"], s["bias"])
        elif c["op"] == "grad":
            s["plan"].run(s["A"], s["B"], None, s["D"], s["offsets"], s["bias"])
        else:
            s["plan"].run(s["A"], s["Q"], s["scales"], s["zeros"], None, s["D"],
                          s["offsets"] if c["experts"] > 1 else None, s["bias"])
        return [s["D"], s["bias"]] if c["op"] == "grad" and c["bias"] else s["D"]
    return _plain_grad(s) if c["op"] == "grad" else _plain_rows(s)


def _places(s):
    """(expert, position within it) of every used row."""
    r = torch.arange(s["used"], device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    return e, r - s["offsets"].long()[e]


def _padded(s, x, e, pos):
    """The used rows of x in 32 bits, expert by expert, each filled up with zeros to the longest."""
    out = torch.zeros(s["case"]["experts"], s["most"], x.shape[1], device=DEV)
    out[e, pos] = x[:s["used"]].float()
    return out


def _plain_rows(s):
    c = s["case"]
    if c["op"] == "quant":
        q = torch.stack([s["Q"] & 15, s["Q"] >> 4], dim=-1).reshape(c["experts"], c["N"], -1, c["block"]).float()
        z = s["zeros"].float() if c["zeros"] else torch.full_like(s["scales"], 8.0, dtype=torch.float32)
        b = (q - z[..., None]) * s["scales"].float()[..., None]
        b = b.reshape(c["experts"], c["N"], c["K"]).transpose(1, 2).contiguous()
    else:
        b = s["B"].float()
        b = b if c["op_b"] == "N" else b.transpose(1, 2).contiguous()
    if c["experts"] == 1:
        used = slice(0, s["used"])
        d, e = s["A"][used].float() @ b[0], torch.zeros(s["used"], dtype=torch.long, device=DEV)
    else:
        e, pos = _places(s)
        d = torch.bmm(_padded(s, s["A"], e, pos), b)[e, pos]
    if c["epi"] == "gate":
        d = torch.where(s["C"][:s["used"]] > 0, d, 0.0)
    if s["bias"] is not None:
        d = d + s["bias"][e]
    if c["epi"] == "bias_relu":
        d = torch.clamp(d, min=0.0)
    out = torch.zeros_like(s["D"])
    out[:s["used"]] = d.to(out.dtype)
    return out


def _plain_grad(s):
    e, pos = _places(s)
    a, b = _padded(s, s["A"], e, pos), _padded(s, s["B"], e, pos)
    d = torch.bmm(a.transpose(1, 2).contiguous(), b).to(s["D"].dtype)
    return [d, b.sum(dim=1)] if s["bias"] is not None else d


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    E, T, N = case["experts"], case["rows"] - case["pad"], case["N"]
    a, d = BYTES[case["ab"]], BYTES[case["cd"]]
    if case["op"] == "grad":
        M = case["M"]
        return {"bytes": T * (M + N) * a + E * M * N * d + (E * N * 4 if case["bias"] else 0),
                "flops": 2 * T * M * N}
    K = case["K"]
    active = E * (1 - (1 - 1 / E) ** T) if E > 1 else 1   # experts with a row, on average
    weight = (K * N * a if case["op"] == "rows" else
              N * K / 2 + N * K / case["block"] * (a + (1 if case["zeros"] else 0)))
    return {"bytes": T * K * a + active * (weight + (4 * N if "bias" in case["epi"] else 0))
            + T * N * d * (2 if case["epi"] == "gate" else 1),
            "flops": 2 * T * K * N}


# ---- the definition in 64 bits -----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    offs = s["offsets"].tolist()
    D = s["D"].double()
    sums = torch.zeros(case["experts"], case["N"], dtype=torch.float64, device=DEV)
    for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
        if lo == hi:
            continue
        a = s["A"][lo:hi].double()
        if case["op"] == "grad":
            g = s["B"][lo:hi].double()
            D[e] = a.t().contiguous() @ g
            sums[e] = g.sum(0)
            continue
        if case["op"] == "rows":
            w = s["B"][e].double()
            w = w if case["op_b"] == "N" else w.t().contiguous()
        else:
            w = torch.empty(case["N"], case["K"], dtype=torch.float64, device=DEV)
            w[:, 0::2] = (s["Q"][e] % 16).double()
            w[:, 1::2] = torch.div(s["Q"][e], 16, rounding_mode="floor").double()
            near = torch.arange(case["K"], device=DEV) // case["block"]
            w -= s["zeros"][e].double()[:, near] if case["zeros"] else 8
            w = (w * s["scales"][e].double()[:, near]).t().contiguous()
        d = a @ w
        if s["bias"] is not None:
            d += s["bias"][e].double()
        if case["epi"] == "bias_relu":
            d = d * (d > 0)
        if case["epi"] == "gate":
            d = d * (s["C"][lo:hi] > 0)
        D[lo:hi] = d
    return [D, sums] if case["op"] == "grad" and case["bias"] else D
