"""What stands around the products of a feed-forward layer, case by case: the plain form of each
operator in elementary torch operations, and the framework's own kernels on the same inputs.

  layer  products with bias, activation and residual in their epilogue, the activation's argument
         kept for training, and the product that carries a gradient back through the activation;
         with one weight matrix or one per expert
  norm   layer norm in front of the products, and its gradients towards rows, weight and bias
  route  the routing of rows to experts: their choice and weights, the per-expert counts (as the
         offsets that the products grouped by expert read) with the rows' order, the balance loss,
         and the gradient of weights and loss towards the router's logits

`own` selects the framework's kernels; otherwise run() computes the plain form in 32 bits.
"""
import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TORCH = {"f16": torch.float16, "bf16": torch.bfloat16, "f32": torch.float32}
BYTES = {"f16": 2, "bf16": 2, "f32": 4}
EPS = 1e-5


# ---- cases -------------------------------------------------------------------------------------
# layer: rows of the token buffer, the last `pad` of them behind the last expert's range; K x N:
# each expert's weights (op_b T: stored N x K); way "forward": D = act(A B + bias) + C, the
# activation's argument Z = A B + bias kept where `pre`; way "grad": D = (A B) act'(Z).
# norm: rows of N values; way "forward" (stats: mean and 1 / deviation kept) or "grad" (residual:
# the gradient that goes round the layer is added to that of the rows).
# route: rows of logits over `experts`, the `k` largest chosen, their probabilities divided by
# their sum where `normalize`; the last `pad` rows are padding, left out by the mask; loss: with the
# balance loss (training).

def listed():
    return [
        # three requests' next tokens through a small layer: launch latency counts
        {"name": "layer_token", "op": "layer", "way": "forward", "rows": 3, "pad": 0, "experts": 1,
         "K": 2048, "N": 2048, "op_b": "T", "ab": "bf16", "cd": "bf16", "act": "silu", "bias": False,
         "residual": False, "pre": False, "skew": 0.0},
        # a served batch through a wide layer's second product, back into the residual stream
        {"name": "layer_batch", "op": "layer", "way": "forward", "rows": 64, "pad": 0, "experts": 1,
         "K": 16384, "N": 4096, "op_b": "T", "ab": "f16", "cd": "f16", "act": "none", "bias": True,
         "residual": True, "pre": False, "skew": 0.0},
        # training: the first product of a wide layer, its activation's argument kept
        {"name": "layer_train", "op": "layer", "way": "forward", "rows": 8192, "pad": 0, "experts": 1,
         "K": 4096, "N": 16384, "op_b": "T", "ab": "bf16", "cd": "bf16", "act": "gelu", "bias": True,
         "residual": False, "pre": True, "skew": 0.0},
        # training: the gradient of the layer's output carried back through the activation
        {"name": "layer_grad", "op": "layer", "way": "grad", "rows": 8192, "pad": 0, "experts": 1,
         "K": 4096, "N": 16384, "op_b": "N", "ab": "bf16", "cd": "bf16", "act": "gelu_tanh",
         "bias": False, "residual": False, "pre": True, "skew": 0.0},
        # experts with odd everything: no row starts on a 16-byte boundary
        {"name": "layer_experts_odd", "op": "layer", "way": "forward", "rows": 3001, "pad": 13,
         "experts": 7, "K": 1001, "N": 777, "op_b": "N", "ab": "f16", "cd": "f32", "act": "silu",
         "bias": True, "residual": True, "pre": True, "skew": 1.0},
        # seven requests' next tokens in front of a layer
        {"name": "norm_token", "op": "norm", "way": "forward", "rows": 7, "N": 4096, "type": "bf16",
         "stats": False, "residual": False},
        # training's forward pass over a batch of long rows
        {"name": "norm_train", "op": "norm", "way": "forward", "rows": 16384, "N": 8192, "type": "bf16",
         "stats": True, "residual": False},
        # its gradients, the residual stream's added
        {"name": "norm_grad", "op": "norm", "way": "grad", "rows": 16384, "N": 4096, "type": "bf16",
         "stats": True, "residual": True},
        # odd rows of a small model
        {"name": "norm_grad_odd", "op": "norm", "way": "grad", "rows": 5003, "N": 1001, "type": "f16",
         "stats": True, "residual": False},
        # a served batch of single tokens
        {"name": "route_token", "op": "route", "way": "forward", "rows": 16, "pad": 0, "experts": 64,
         "k": 8, "type": "f32", "normalize": True, "loss": False, "skew": 0.5},
        # a training batch with padded sequences
        {"name": "route_train", "op": "route", "way": "forward", "rows": 65536, "pad": 1500,
         "experts": 128, "k": 8, "type": "f32", "normalize": True, "loss": True, "skew": 0.5},
        # and its gradient towards the logits
        {"name": "route_grad", "op": "route", "way": "grad", "rows": 65536, "pad": 1500,
         "experts": 128, "k": 8, "type": "f32", "normalize": True, "loss": True, "skew": 0.5},
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def _size(rng, lo, hi):
    """A size spread over its logarithm: whole 16-byte chunks three times out of four, else any."""
    n = _log(rng, lo, hi)
    return n if rng.random() < 0.25 else max(8, n // 8 * 8)


def draw(rng):
    op = rng.choice(["layer", "layer", "norm", "route"])
    way = rng.choice(["forward", "grad"])
    while True:
        if op == "layer":
            ab = rng.choice(["f16", "bf16", "bf16", "f32"])
            c = {"op": op, "way": way, "rows": _log(rng, 1, 16384), "pad": 0,
                 "experts": _log(rng, 2, 64) if rng.random() < 0.4 else 1, "K": _size(rng, 64, 16384),
                 "N": _size(rng, 64, 16384), "op_b": rng.choice("NT"), "ab": ab,
                 "cd": rng.choice([ab, "f32"]),
                 "act": rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu"]),
                 "bias": way == "forward" and rng.random() < 0.5,
                 "residual": way == "forward" and rng.random() < 0.5,
                 "pre": way == "grad" or rng.random() < 0.5, "skew": rng.choice([0.0, 0.5, 1.0])}
            if c["experts"] > 1 and rng.random() < 0.5:
                c["pad"] = rng.randrange(0, max(1, c["rows"] // 16))
            # no more than the largest listed case: products (in 32 bits a tenth), weights, padding
            most = 8192 * 4096 * 16384 // (10 if ab == "f32" else 1)
            if (c["rows"] * c["K"] * c["N"] <= most and c["experts"] * c["K"] * c["N"] <= 1 << 29
                    and c["experts"] * c["rows"] * (c["K"] + c["N"]) <= 1 << 29):
                return c
        elif op == "norm":
            c = {"op": op, "way": way, "rows": _log(rng, 1, 65536), "N": _size(rng, 32, 16384),
                 "type": rng.choice(["f16", "bf16", "f32"]), "stats": way == "grad" or rng.random() < 0.5,
                 "residual": way == "grad" and rng.random() < 0.5}
            if c["rows"] * c["N"] * BYTES[c["type"]] <= 16384 * 8192 * 2:
                return c
        else:
            e = rng.choice([_log(rng, 2, 512), 8, 64, 256])
            c = {"op": op, "way": way, "rows": _log(rng, 1, 131072), "pad": 0, "experts": e,
                 "k": rng.randrange(1, min(e, 10) + 1), "type": rng.choice(["f32", "f32", "bf16", "f16"]),
                 "normalize": rng.random() < 0.5, "loss": way == "grad" or rng.random() < 0.7,
                 "skew": rng.choice([0.0, 0.5, 1.0])}
            if rng.random() < 0.5:
                c["pad"] = rng.randrange(0, max(1, c["rows"] // 16))
            if c["rows"] * e <= 65536 * 128 and c["rows"] * c["k"] <= 65536 * 8:
                return c


# ---- inputs ------------------------------------------------------------------------------------

def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    out = torch.empty(shape, dtype=dtype, device=DEV)
    # in slices along the first axis of a stack, whose 32-bit form would be large
    for i in range(shape[0]) if len(shape) == 3 else [slice(None)]:
        out[i] = (torch.randn(out[i].shape, generator=g, device=DEV) * scale).to(dtype)
    return out


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(int(seed))
    s = {"case": dict(case)}
    {"layer": _prepare_layer, "norm": _prepare_norm, "route": _prepare_route}[case["op"]](case, seed, g, s)
    if own:
        s["plan"] = _plan(case)
        if getattr(s["plan"], "workspace_bytes", 0):
            s["workspace"] = torch.empty(s["plan"].workspace_bytes, dtype=torch.uint8, device=DEV)
    return s


def _prepare_layer(c, seed, g, s):
    E, T, K, N = c["experts"], c["rows"], c["K"], c["N"]
    ab, cd = TORCH[c["ab"]], TORCH[c["cd"]]
    h = np.random.default_rng([seed, 1])
    p = np.exp(c["skew"] * h.standard_normal(E))
    counts = h.multinomial(T - c["pad"], p / p.sum())          # a router's skewed choice
    ends = np.concatenate([[0], np.cumsum(counts)])
    s["used"], s["most"] = int(ends[-1]), int(counts.max())
    s["offsets"] = torch.tensor(ends, dtype=torch.int32, device=DEV)
    # a gradient's rows are smaller than a layer's normed input
    s["A"] = _normal(g, T, K, scale=1.0 if c["way"] == "forward" else 1 / 8, dtype=ab)
    s["B"] = _normal(g, E, *((K, N) if c["op_b"] == "N" else (N, K)), scale=K ** -0.5, dtype=ab)
    s["bias"] = _normal(g, E, N, scale=0.5) if c["bias"] else None
    s["C"] = _normal(g, T, N, dtype=cd) if c["residual"] else None
    s["D"] = torch.zeros(T, N, dtype=cd, device=DEV)
    # an activation's arguments have a spread of about 1.5
    s["Z"] = (None if not c["pre"] else _normal(g, T, N, scale=1.5, dtype=cd) if c["way"] == "grad"
              else torch.zeros(T, N, dtype=cd, device=DEV))


def _prepare_norm(c, seed, g, s):
    T, N, t = c["rows"], c["N"], TORCH[c["type"]]
    # a residual stream: rows of different size, a shifted mean, a few large channels
    size = torch.exp(0.3 * torch.randn(T, 1, generator=g, device=DEV))
    channel = torch.exp(0.5 * torch.randn(N, generator=g, device=DEV))
    s["X"] = torch.empty(T, N, dtype=t, device=DEV)
    for i in range(0, T, 8192):
        s["X"][i:i + 8192] = ((torch.randn(s["X"][i:i + 8192].shape, generator=g, device=DEV) * channel + 0.3)
                              * size[i:i + 8192]).to(t)
    s["weight"] = 1 + 0.2 * torch.randn(N, generator=g, device=DEV)
    s["bias"] = 0.2 * torch.randn(N, generator=g, device=DEV)
    if c["stats"]:
        s["mean"] = torch.zeros(T, device=DEV)
        s["rstd"] = torch.zeros(T, device=DEV)
    if c["way"] == "forward":
        s["Y"] = torch.empty(T, N, dtype=t, device=DEV)
        return
    s["dY"] = _normal(g, T, N, scale=0.1, dtype=t)
    s["C"] = _normal(g, T, N, scale=0.1, dtype=t) if c["residual"] else None
    s["dX"] = torch.empty(T, N, dtype=t, device=DEV)
    s["dweight"] = torch.empty(N, device=DEV)
    s["dbias"] = torch.empty(N, device=DEV)
    for i in range(0, T, 8192):                # what the forward pass kept
        x = s["X"][i:i + 8192].double()
        m = x.mean(1)
        s["mean"][i:i + 8192] = m.float()
        s["rstd"][i:i + 8192] = (((x - m[:, None]) ** 2).mean(1) + EPS).rsqrt().float()


def _prepare_route(c, seed, g, s):
    T, E, k = c["rows"], c["experts"], c["k"]
    s["logits"] = (torch.randn(T, E, generator=g, device=DEV)
                   + c["skew"] * torch.randn(E, generator=g, device=DEV)).to(TORCH[c["type"]])
    s["mask"] = None
    if c["pad"]:
        s["mask"] = torch.ones(T, dtype=torch.uint8, device=DEV)
        s["mask"][T - c["pad"]:] = 0
    i32 = dict(dtype=torch.int32, device=DEV)
    s["index"] = torch.zeros(T, k, **i32)
    s["slope"] = torch.zeros(E, device=DEV) if c["loss"] else None
    if c["way"] == "forward":
        s["weight"] = torch.zeros(T, k, device=DEV)
        s["order"], s["place"] = torch.zeros(T * k, **i32), torch.zeros(T, k, **i32)
        s["offsets"] = torch.zeros(E + 1, **i32)
        s["loss"] = torch.zeros(1, device=DEV) if c["loss"] else None
        return
    index, _, _, counts = _choose(s)           # what the forward pass kept
    s["index"].copy_(index)
    used = T - c["pad"]
    s["slope"].copy_(counts.double() * E / k / used / used)
    s["dweight"] = 0.1 * torch.randn(T, k, generator=g, device=DEV) / T
    s["dloss"] = torch.full((1,), 0.01, device=DEV)
    s["dlogits"] = torch.empty_like(s["logits"])


def _plan(c):
    import tiled_gemm_epilogues_amd as tge
    if c["op"] == "layer":
        return tge.LayerPlan(c["rows"], c["N"], c["K"], c["experts"], c["op_b"], ab=c["ab"], cd=c["cd"],
                             act=c["act"])
    if c["op"] == "norm":
        return tge.NormPlan(c["rows"], c["N"], type=c["type"], eps=EPS)
    return tge.RoutePlan(c["rows"], c["experts"], c["k"], type=c["type"], normalize=c["normalize"])


# ---- one pass ----------------------------------------------------------------------------------

def run(s):
    c = s["case"]
    return (_own if own else _plain)[c["op"], c["way"]](s)


def _own_layer(s):
    offsets = s["offsets"] if s["case"]["experts"] > 1 else None
    s["plan"].run(s["A"], s["B"], s["C"], s["D"], offsets, s["bias"], s["Z"],
                  beta=1.0 if s["C"] is not None else 0.0)
    return [s["D"], s["Z"]] if s["Z"] is not None else s["D"]


def _own_layer_grad(s):
    s["plan"].run_grad(s["A"], s["B"], s["Z"], s["D"], s["offsets"] if s["case"]["experts"] > 1 else None)
    return s["D"]


def _own_norm(s):
    s["plan"].run(s["X"], s["weight"], s["bias"], s["Y"], s.get("mean"), s.get("rstd"))
    return [s["Y"], s["mean"], s["rstd"]] if s["case"]["stats"] else s["Y"]


def _own_norm_grad(s):
    s["plan"].run_grad(s["dY"], s["X"], s["weight"], s["mean"], s["rstd"], s["dX"], s["dweight"], s["dbias"],
                       s["C"], beta=1.0 if s["C"] is not None else 0.0, workspace=s.get("workspace"))
    return [s["dX"], s["dweight"], s["dbias"]]


def _own_route(s):
    s["plan"].run(s["logits"], s["index"], s["weight"], s["order"], s["place"], s["offsets"], s["slope"],
                  s["loss"], s["mask"], workspace=s.get("workspace"))
    out = [s["index"], s["weight"], s["order"], s["place"], s["offsets"]]
    return out + [s["slope"], s["loss"]] if s["case"]["loss"] else out


def _own_route_grad(s):
    s["plan"].run_grad(s["logits"], s["index"], s["dweight"], s["slope"], s["dloss"], s["dlogits"], s["mask"])
    return s["dlogits"]


def _product(s):
    """A times each expert's weights, in 32 bits, for the rows in use; and each row's expert."""
    c, used = s["case"], s["used"]
    b = s["B"].float()
    b = b if c["op_b"] == "N" else b.transpose(1, 2).contiguous()
    if c["experts"] == 1:
        return s["A"][:used].float() @ b[0], torch.zeros(used, dtype=torch.long, device=DEV)
    r = torch.arange(used, device=DEV)
    e = torch.searchsorted(s["offsets"][1:].long(), r, right=True)
    pos = r - s["offsets"].long()[e]
    # expert by expert, each filled up with zeros to the longest
    a = torch.zeros(c["experts"], s["most"], c["K"], device=DEV)
    a[e, pos] = s["A"][:used].float()
    return torch.bmm(a, b)[e, pos], e


def _phi(z):
    """The normal distribution function; through the complement, exact in the negative tail."""
    return 0.5 * torch.erfc(z * -math.sqrt(0.5))


def _sigmoid(w):
    return 1 / (1 + torch.exp(-w))


TANH_A, TANH_B = 2 * math.sqrt(2 / math.pi), 2 * math.sqrt(2 / math.pi) * 0.044715


def _act(name, z):
    if name == "none":
        return z
    if name == "relu":
        return torch.clamp(z, min=0)
    if name == "gelu":
        return z * _phi(z)
    # (1 + tanh u) / 2 is the logistic function of 2 u
    return z * _sigmoid(z if name == "silu" else z * (TANH_A + TANH_B * z * z))


def _act_slope(name, z):
    if name == "none":
        return torch.ones_like(z)
    if name == "relu":
        return (z > 0).to(z.dtype)
    if name == "gelu":
        return _phi(z) + z * torch.exp(-0.5 * z * z) / math.sqrt(2 * math.pi)
    if name == "silu":
        s = _sigmoid(z)
        return s + z * s * (1 - s)
    s = _sigmoid(z * (TANH_A + TANH_B * z * z))
    return s + z * s * (1 - s) * (TANH_A + 3 * TANH_B * z * z)


def _plain_layer(s):
    c, used = s["case"], s["used"]
    z, e = _product(s)
    if s["bias"] is not None:
        z = z + s["bias"][e]
    d = _act(c["act"], z)
    if s["C"] is not None:
        d = d + s["C"][:used].float()
    out = []
    for x in [d, z] if c["pre"] else [d]:
        full = torch.zeros_like(s["D"])
        full[:used] = x.to(full.dtype)
        out.append(full)
    return out if c["pre"] else out[0]


def _plain_layer_grad(s):
    used = s["used"]
    out = torch.zeros_like(s["D"])
    out[:used] = (_product(s)[0] * _act_slope(s["case"]["act"], s["Z"][:used].float())).to(out.dtype)
    return out


def _plain_norm(s):
    c, x = s["case"], s["X"].float()
    mean = x.mean(1)
    d = x - mean[:, None]
    rstd = ((d * d).mean(1) + EPS).rsqrt()
    y = (d * rstd[:, None] * s["weight"] + s["bias"]).to(s["X"].dtype)
    return [y, mean, rstd] if c["stats"] else y


def _plain_norm_grad(s):
    xhat = (s["X"].float() - s["mean"][:, None]) * s["rstd"][:, None]
    dy = s["dY"].float()
    g = dy * s["weight"]
    dx = s["rstd"][:, None] * (g - g.mean(1)[:, None] - xhat * (g * xhat).mean(1)[:, None])
    if s["C"] is not None:
        dx = dx + s["C"].float()
    return [dx.to(s["X"].dtype), (dy * xhat).sum(0), dy.sum(0)]


def _choose(s):
    """(index, order, place, counts): the k largest logits of every row in use, ties to the lowest
    expert, and the choices in the order of their experts."""
    c = s["case"]
    T, E, k = c["rows"], c["experts"], c["k"]
    used = T - c["pad"]
    index = torch.full((T, k), -1, dtype=torch.int64, device=DEV)
    index[:used] = torch.sort(s["logits"][:used].float(), dim=1, descending=True, stable=True)[1][:, :k]
    flat = index[:used].reshape(-1)
    order = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
    order[:used * k] = torch.sort(flat, stable=True)[1]
    place = torch.full((T * k,), -1, dtype=torch.int64, device=DEV)
    place[order[:used * k]] = torch.arange(used * k, device=DEV)
    return index, order, place.reshape(T, k), torch.bincount(flat, minlength=E)


def _softmax(x):
    e = torch.exp(x - x.max(1)[0][:, None])
    return e / e.sum(1)[:, None]


def _plain_route(s):
    c = s["case"]
    T, E, k = c["rows"], c["experts"], c["k"]
    used = T - c["pad"]
    index, order, place, counts = _choose(s)
    p = _softmax(s["logits"][:used].float())
    weight = torch.zeros(T, k, device=DEV)
    w = torch.gather(p, 1, index[:used])
    weight[:used] = w / w.sum(1)[:, None] if c["normalize"] else w
    offsets = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = torch.cumsum(counts, 0)
    out = [index.int(), weight, order.int(), place.int(), offsets]
    if not c["loss"]:
        return out
    slope = counts.float() * (E / k / used / used)
    return out + [slope, (slope * p.sum(0)).sum().reshape(1)]


def _plain_route_grad(s):
    c = s["case"]
    used = c["rows"] - c["pad"]
    p = _softmax(s["logits"][:used].float())
    index, dw = s["index"][:used].long(), s["dweight"][:used]
    w = torch.gather(p, 1, index)
    d = s["dloss"] * p * (s["slope"] - (p * s["slope"]).sum(1)[:, None])
    if c["normalize"]:
        w = w / w.sum(1)[:, None]
        d.scatter_add_(1, index, w * (dw - (w * dw).sum(1)[:, None]))
    else:
        d.scatter_add_(1, index, w * dw)
        d = d - p * (w * dw).sum(1)[:, None]
    out = torch.zeros_like(s["dlogits"])
    out[:used] = d.to(out.dtype)
    return out


_own = {("layer", "forward"): _own_layer, ("layer", "grad"): _own_layer_grad, ("norm", "forward"): _own_norm,
        ("norm", "grad"): _own_norm_grad, ("route", "forward"): _own_route, ("route", "grad"): _own_route_grad}
_plain = {("layer", "forward"): _plain_layer, ("layer", "grad"): _plain_layer_grad,
          ("norm", "forward"): _plain_norm, ("norm", "grad"): _plain_norm_grad,
          ("route", "forward"): _plain_route, ("route", "grad"): _plain_route_grad}


# ---- what a pass cannot do without -------------------------------------------------------------

def work(case):
    if case["op"] == "layer":
        E, T, K, N = case["experts"], case["rows"] - case["pad"], case["K"], case["N"]
        a, d = BYTES[case["ab"]], BYTES[case["cd"]]
        active = E * (1 - (1 - 1 / E) ** T) if E > 1 else 1    # experts with a row, on average
        return {"bytes": T * K * a + active * (K * N * a + (4 * N if case["bias"] else 0))
                + T * N * d * (1 + case["residual"] + case["pre"]),
                "flops": 2 * T * K * N}
    if case["op"] == "norm":
        T, N, t = case["rows"], case["N"], BYTES[case["type"]]
        if case["way"] == "forward":
            return {"bytes": 2 * T * N * t + 8 * N + (8 * T if case["stats"] else 0), "flops": 8 * T * N}
        return {"bytes": T * N * t * (3 + case["residual"]) + 8 * T + 12 * N, "flops": 16 * T * N}
    T, E, k = case["rows"], case["experts"], case["k"]
    used, t = T - case["pad"], BYTES[case["type"]]
    mask = T if case["pad"] else 0
    if case["way"] == "forward":
        return {"bytes": used * E * t + mask + 16 * T * k + 4 * (E + 1) + (4 * E + 4 if case["loss"] else 0),
                "flops": used * E * (6 + k)}
    return {"bytes": used * (E * t + 8 * k) + mask + T * E * t + 4 * E + 4, "flops": 10 * used * E}


# ---- the definitions in 64 bits ----------------------------------------------------------------

def exact(case, seed):
    s = prepare(case, seed)
    return {"layer": _exact_layer, "norm": _exact_norm, "route": _exact_route}[case["op"]](case, s)


def _define_act(name, z):
    return {"none": lambda: z, "relu": lambda: z * (z > 0),
            "gelu": lambda: z / 2 * torch.erfc(z * -math.sqrt(0.5)),
            "gelu_tanh": lambda: z / 2 * (1 + torch.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))),
            "silu": lambda: z * torch.sigmoid(z)}[name]()


def _exact_layer(c, s):
    offs = s["offsets"].tolist()
    D = s["D"].double()
    Z = torch.zeros_like(D)
    for e, (lo, hi) in enumerate(zip(offs, offs[1:])):
        if lo == hi:
            continue
        w = s["B"][e].double()
        z = s["A"][lo:hi].double() @ (w if c["op_b"] == "N" else w.t().contiguous())
        if c["way"] == "grad":
            x = s["Z"][lo:hi].double().requires_grad_()
            D[lo:hi] = torch.autograd.grad(_define_act(c["act"], x).sum(), x)[0] * z
            continue
        if s["bias"] is not None:
            z = z + s["bias"][e].double()
        Z[lo:hi] = z
        D[lo:hi] = _define_act(c["act"], z)
        if s["C"] is not None:
            D[lo:hi] += s["C"][lo:hi].double()
    return [D, Z] if c["way"] == "forward" and c["pre"] else D


def _exact_norm(c, s):
    weight, bias = s["weight"].double(), s["bias"].double()
    T, N = s["X"].shape
    out = torch.empty(T, N, dtype=torch.float64, device=DEV)
    means, rstds = torch.empty(T, dtype=torch.float64, device=DEV), torch.empty(T, dtype=torch.float64, device=DEV)
    dweight, dbias = torch.zeros_like(weight), torch.zeros_like(bias)
    for i in range(0, T, 4096):
        rows = slice(i, min(i + 4096, T))
        x = s["X"][rows].double()
        if c["way"] == "forward":
            var, m = torch.var_mean(x, dim=1, unbiased=False)
            means[rows], rstds[rows] = m, 1 / torch.sqrt(var + EPS)
            out[rows] = (x - m[:, None]) / torch.sqrt(var + EPS)[:, None] * weight + bias
            continue
        r = s["rstd"][rows].double()[:, None]
        xhat, dy = (x - s["mean"][rows].double()[:, None]) * r, s["dY"][rows].double()
        dweight += torch.einsum("ij,ij->j", dy, xhat)
        dbias += dy.sum(0)
        a = (dy @ weight)[:, None] / N
        b = ((dy * xhat) @ weight)[:, None] / N
        out[rows] = r * (dy * weight - a - b * xhat)
        if s["C"] is not None:
            out[rows] += s["C"][rows].double()
    if c["way"] == "grad":
        return [out, dweight, dbias]
    return [out, means, rstds] if c["stats"] else out


def _exact_route(c, s):
    T, E, k = c["rows"], c["experts"], c["k"]
    used = T - c["pad"]
    x = s["logits"][:used].double().requires_grad_()
    p = torch.softmax(x, 1)
    if c["way"] == "grad":
        w = torch.gather(p, 1, s["index"][:used].long())
        w = w / w.sum(1, keepdim=True) if c["normalize"] else w
        total = (w * s["dweight"][:used].double()).sum() + (p.sum(0) * s["slope"].double()).sum() * s["dloss"].double()[0]
        out = torch.zeros(T, E, dtype=torch.float64, device=DEV)
        out[:used] = torch.autograd.grad(total, x)[0]
        return out
    p = p.detach()
    # one expert after another, the lowest of the largest logits each time
    left = s["logits"][:used].double().clone()
    index = torch.full((T, k), -1, dtype=torch.int32, device=DEV)
    w = torch.zeros(T, k, dtype=torch.float64, device=DEV)
    number = torch.arange(E, device=DEV)
    for j in range(k):
        best = torch.where(left == left.max(1, keepdim=True)[0], number, E).min(1)[0]
        index[:used, j] = best.int()
        w[:used, j] = p[torch.arange(used, device=DEV), best]
        left[torch.arange(used, device=DEV), best] = -math.inf
    if c["normalize"]:
        w[:used] /= w[:used].sum(1, keepdim=True)
    host = index.cpu().numpy().reshape(-1)
    order, place = np.full(T * k, -1, np.int32), np.full(T * k, -1, np.int32)
    chosen = np.nonzero(host >= 0)[0]
    sorted_ = chosen[np.argsort(host[chosen], kind="stable")]
    order[:len(sorted_)] = sorted_
    place[sorted_] = np.arange(len(sorted_))
    counts = np.bincount(host[chosen], minlength=E)
    offsets = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    put = lambda a: torch.from_numpy(a).to(DEV)
    out = [index, w, put(order), put(place.reshape(T, k)), put(offsets)]
    if not c["loss"]:
        return out
    f = put(counts).double() / (k * used)
    return out + [E * f / used, (E * f * p.mean(0)).sum().reshape(1)]
