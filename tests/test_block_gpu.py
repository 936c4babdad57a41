"""The block of a mixture-of-experts model made of the plans, as it would be used: layer norm, the router's
product, routing, the experts' two products with an activation between them, the weighted sum with the
residual, and the way back to every parameter with the balance loss.

The block is written once, over an object that has its operators.  With plain formulas in 64 bits its
gradients are those of autograd (on the CPU); with the plans every operator's result is compared with
the formula on the inputs that it had; and captured in graphs the plans give what they give eagerly."""
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import TORCH_DT
from layer_helpers import U, act64, act_bound, close, rounding, slope64, slope_bound

DEV = "cuda:0"
EPS = 1e-5


@pytest.fixture
def gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Block:
    """Y = X + sum over j of weight_j (act(N W1_e + b1_e) W2_e + b2_e), N = layer norm of X, e and weight by
    the router's logits N Wr^T; the loss is sum(Y dY) + dloss * balance."""

    def __init__(self, ops, k, act):
        self.ops, self.k, self.act = ops, k, act

    def forward(self, X, P, mask=None):
        o, k = self.ops, self.k
        N, mean, rstd = o.norm(X, P["g"], P["b"])
        logits = o.layer(N, P["Wr"], "T", out="wide")[0]
        index, weight, order, place, offs, slope, loss = o.route(logits, mask, k)
        rows = order.clamp(min=0).long() // k                       # (what is behind the last range is not read)
        S = N.index_select(0, rows)
        H, Z = o.layer(S, P["W1"], "N", offs, P["b1"], act=self.act, keep=True)
        O = o.layer(H, P["W2"], "N", offs, P["b2"])[0]
        Y = X.to(weight.dtype)
        for j in range(k):
            Y = Y + self.of(O, place, j).to(weight.dtype) * weight[:, j:j + 1]
        self.saved = (X, N, mean, rstd, logits, index, weight, order, place, offs, slope, rows, S, H, Z, O, mask)
        return Y.to(X.dtype), loss

    @staticmethod
    def of(O, place, j):
        """The j-th chosen expert's row for every row; 0 where there is none."""
        got = O.index_select(0, place[:, j].clamp(min=0).long())
        return torch.where(place[:, j:j + 1] >= 0, got, torch.zeros_like(got))

    def backward(self, dY, dloss, P):
        o, k = self.ops, self.k
        X, N, mean, rstd, logits, index, weight, order, place, offs, slope, rows, S, H, Z, O, mask = self.saved
        G = {}
        dO = (dY.index_select(0, rows).to(weight.dtype) * weight.reshape(-1).index_select(0, order.clamp(min=0).long())[:, None]).to(X.dtype)
        dw = torch.cat([(dY.to(weight.dtype) * self.of(O, place, j).to(weight.dtype)).sum(1, keepdim=True) for j in range(k)], 1)
        dZ = o.layer_grad(dO, P["W2"], "T", offs, self.act, Z)
        G["W2"], G["b2"] = o.weights(H, dO, offs)
        dS = o.layer(dZ, P["W1"], "T", offs)[0]
        G["W1"], G["b1"] = o.weights(S, dZ, offs)
        dl = o.route_grad(logits, mask, index, dw, slope, dloss).to(X.dtype)
        dN = self.of(dS, place, 0)
        for j in range(1, k):
            dN = dN + self.of(dS, place, j)
        dN = o.layer(dl, P["Wr"], "N", C=dN)[0]
        G["Wr"] = o.weights(dl, N, None)[0]
        G["X"], G["g"], G["b"] = o.norm_grad(dN, X, P["g"], mean, rstd, dY)
        return G


class Plain:
    """The operators' formulas in 64 bits on the host."""

    def norm(self, X, g, b):
        m = X.mean(1, keepdim=True)
        r = 1 / torch.sqrt(((X - m) ** 2).mean(1, keepdim=True) + EPS)
        return (X - m) * r * g + b, m[:, 0], r[:, 0]

    def norm_grad(self, dY, X, g, mean, rstd, C):
        h, w = (X - mean[:, None]) * rstd[:, None], dY * g
        dX = rstd[:, None] * (w - w.mean(1, keepdim=True) - h * (w * h).mean(1, keepdim=True)) + C
        return dX, (dY * h).sum(0), dY.sum(0)

    def ranges(self, B, offs, rows):
        if offs is None:
            return [(B, 0, rows, 0)]
        at = offs.tolist()
        return [(B[e], at[e], at[e + 1], e) for e in range(len(at) - 1)]

    def product(self, A, B, op_b, offs, bias=None):
        first = B if offs is None else B[0]
        out = torch.zeros(A.shape[0], first.shape[1 if op_b == "N" else 0], dtype=A.dtype)
        for b, lo, hi, e in self.ranges(B, offs, A.shape[0]):
            out[lo:hi] = A[lo:hi] @ (b if op_b == "N" else b.t()) + (0 if bias is None else bias[e])
        return out

    def layer(self, A, B, op_b, offs=None, bias=None, act="none", C=None, keep=False, out=None):
        Z = self.product(A, B, op_b, offs, bias)
        return act64(act, Z) + (0 if C is None else C), Z

    def layer_grad(self, A, B, op_b, offs, act, Z):
        return self.product(A, B, op_b, offs) * slope64(act, Z)

    def weights(self, A, B, offs):
        at = [0, A.shape[0]] if offs is None else offs.tolist()
        parts = [(A[lo:hi].t() @ B[lo:hi], B[lo:hi].sum(0)) for lo, hi in zip(at[:-1], at[1:])]
        return (torch.stack([p[0] for p in parts]), torch.stack([p[1] for p in parts])) if offs is not None else parts[0]

    def choose(self, logits, mask, k):
        T, E = logits.shape
        on = torch.ones(T, dtype=torch.bool) if mask is None else mask != 0
        index = torch.sort(logits, dim=1, descending=True, stable=True)[1][:, :k]
        index = torch.where(on[:, None], index, -torch.ones_like(index))
        flat = index.reshape(-1)
        chosen = (flat >= 0).nonzero()[:, 0]
        srt = chosen[torch.sort(flat[chosen], stable=True)[1]]
        order, place = torch.full((T * k,), -1), torch.full((T * k,), -1)
        order[:len(srt)] = srt
        place[srt] = torch.arange(len(srt))
        counts = torch.bincount(flat[chosen], minlength=E)
        offs = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)])
        return index, order, place.reshape(T, k), offs, counts, on

    def route(self, logits, mask, k):
        index, order, place, offs, counts, on = self.choose(logits, mask, k)
        p = torch.softmax(logits, 1) * on[:, None]
        w = torch.gather(p, 1, index.clamp(min=0)) * (index >= 0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        n = int(on.sum())
        slope = counts.to(logits.dtype) * logits.shape[1] / k / n / n
        return index, w, order, place, offs, slope, (slope * p.sum(0)).sum()

    def route_grad(self, logits, mask, index, dweight, slope, dloss):
        on = torch.ones(len(logits), dtype=torch.bool) if mask is None else mask != 0
        p = torch.softmax(logits, 1) * on[:, None]
        w = torch.gather(p, 1, index.long().clamp(min=0)) * (index >= 0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        h = dloss * slope
        d = p * (h - (p * h).sum(1, keepdim=True))
        return d.scatter_add(1, index.long().clamp(min=0), w * (dweight - (w * dweight).sum(1, keepdim=True)) * (index >= 0))


class Plans:
    """The operators by the plans; `type` is that of X, the weights and what is between them."""

    def __init__(self, type):
        self.type, self.dt, self.made = type, TORCH_DT[type], {}

    def plan(self, cls, *args, **kw):
        key = (cls, args, tuple(sorted(kw.items())))
        if key not in self.made:
            self.made[key] = cls(*args, **kw)
        return self.made[key]

    def new(self, *shape, dtype=None):
        return torch.empty(*shape, dtype=dtype or self.dt, device=DEV)

    def norm(self, X, g, b):
        T, h = X.shape
        Y, mean, rstd = self.new(T, h), self.new(T, dtype=torch.float32), self.new(T, dtype=torch.float32)
        self.plan(tge.NormPlan, T, h, type=self.type, eps=EPS).run(X, g, b, Y, mean, rstd)
        return Y, mean, rstd

    def norm_grad(self, dY, X, g, mean, rstd, C):
        T, h = X.shape
        dX, dg, db = self.new(T, h), self.new(h, dtype=torch.float32), self.new(h, dtype=torch.float32)
        self.plan(tge.NormPlan, T, h, type=self.type, eps=EPS).run_grad(dY, X, g, mean, rstd, dX, dg, db, C, 1.0)
        return dX, dg, db

    def layer_plan(self, A, B, op_b, offs, act, cd):
        b = B if offs is None else B[0]
        N = b.shape[1 if op_b == "N" else 0]
        return N, self.plan(tge.LayerPlan, A.shape[0], N, A.shape[1], 1 if offs is None else len(B), op_b,
                            ab=self.type, cd=cd, act=act)

    def layer(self, A, B, op_b, offs=None, bias=None, act="none", C=None, keep=False, out=None):
        cd = "f32" if out == "wide" else self.type
        N, plan = self.layer_plan(A, B, op_b, offs, act, cd)
        D = self.new(A.shape[0], N, dtype=TORCH_DT[cd])
        Z = torch.empty_like(D) if keep else None
        plan.run(A, B, C, D, offs, bias, Z, beta=0.0 if C is None else 1.0)
        return D, Z

    def layer_grad(self, A, B, op_b, offs, act, Z):
        N, plan = self.layer_plan(A, B, op_b, offs, act, self.type)
        D = self.new(A.shape[0], N)
        plan.run_grad(A, B, Z, D, offs)
        return D

    def weights(self, A, B, offs):
        E = 1 if offs is None else len(offs) - 1
        M, N = A.shape[1], B.shape[1]
        if offs is None:
            offs = torch.arange(2, dtype=torch.int32, device=DEV) * len(A)
        dW, db = self.new(E, M, N, dtype=torch.float32), self.new(E, N, dtype=torch.float32)
        self.plan(tge.GroupedGradPlan, A.shape[0], M, N, E, ab=self.type, cd="f32").run(A, B, None, dW, offs, db)
        return dW, db

    def route(self, logits, mask, k):
        T, E = logits.shape
        i = lambda *s: self.new(*s, dtype=torch.int32)
        f = lambda *s: self.new(*s, dtype=torch.float32)
        out = i(T, k), f(T, k), i(T * k), i(T, k), i(E + 1), f(E), f(1)
        self.plan(tge.RoutePlan, T, E, k, normalize=True).run(logits, *out, mask=mask)
        return out

    def route_grad(self, logits, mask, index, dweight, slope, dloss):
        d = torch.empty_like(logits)
        self.plan(tge.RoutePlan, *logits.shape, index.shape[1], normalize=True).run_grad(
            logits, index, dweight.contiguous(), slope, dloss, d, mask)
        return d


def host(x):
    return x.detach().double().cpu() if x.is_floating_point() else x.detach().cpu().long()


class Checked(Plans):
    """Every result against the formula on the same inputs.  Products of K terms in fp32 are off by (K + 4)
    roundings of the sum of their sizes at most, and their activation by 1.13 times that (its steepest
    slope) and its own error; then one rounding to the type."""
    plain = Plain()

    def norm(self, X, g, b):
        import test_norm_gpu
        Y, mean, rstd = super().norm(X, g, b)
        test_norm_gpu.check_forward(X.cpu(), g.cpu(), b.cpu(), Y, mean, rstd, self.type, EPS)
        return Y, mean, rstd

    def norm_grad(self, dY, X, g, mean, rstd, C):
        import test_norm_gpu
        out = super().norm_grad(dY, X, g, mean, rstd, C)
        test_norm_gpu.check_grad(*(t.cpu() for t in (dY, X, g, mean, rstd, C)), 1.0, *out, self.type)
        return out

    def sums(self, A, B, op_b, offs, bias=None):
        a, b, at = host(A), host(B), None if offs is None else host(offs)
        z = self.plain.product(a, b, op_b, at, None if bias is None else host(bias))
        off = (A.shape[1] + 4) * U * (self.plain.product(a.abs(), b.abs(), op_b, at, None if bias is None else host(bias).abs()))
        used = torch.arange(len(z)) < (len(z) if at is None else int(at[-1]))
        return z, off, used

    def layer(self, A, B, op_b, offs=None, bias=None, act="none", C=None, keep=False, out=None):
        D, Z = super().layer(A, B, op_b, offs, bias, act, C, keep, out)
        z, off, used = self.sums(A, B, op_b, offs, bias)
        want, bound = act64(act, z), 1.13 * off + act_bound(act, z, D.dtype)
        if C is not None:
            want = want + host(C)
            bound = bound + U * (want.abs() + bound)
        bound = bound + rounding(want.abs() + bound, D.dtype) * 1.0001
        close(D.cpu()[used], want[used], bound[used], f"{act} product")
        if keep:
            close(Z.cpu()[used], z[used], (off + rounding(z.abs() + off, D.dtype))[used] * 1.0001, "argument")
        return D, Z

    def layer_grad(self, A, B, op_b, offs, act, Z):
        D = super().layer_grad(A, B, op_b, offs, act, Z)
        p, off, used = self.sums(A, B, op_b, offs)
        z = host(Z)
        want = p * slope64(act, z)
        bound = 1.13 * off + (p.abs() + off) * slope_bound(act, z, D.dtype) + U * want.abs()
        bound = bound + rounding(want.abs() + bound, D.dtype) * 1.0001
        close(D.cpu()[used], want[used], bound[used], f"{act} gradient")
        return D

    def weights(self, A, B, offs):
        dW, db = super().weights(A, B, offs)
        a, b, at = host(A), host(B), host(offs) if offs is not None else None
        w, s = self.plain.weights(a, b, at)
        aw, as_ = self.plain.weights(a.abs(), b.abs(), at)
        n = (len(A) + 4) * U
        close(dW.reshape(w.shape), w, n * aw + 1e-37, "weights' gradient")
        close(db.reshape(s.shape), s, n * as_ + 1e-37, "biases' gradient")
        return dW, db

    def route(self, logits, mask, k):
        out = super().route(logits, mask, k)
        x, m = host(logits), None if mask is None else mask.cpu()
        index, w, order, place, offs, slope, loss = self.plain.route(x, m, k)
        for got, want in zip((out[0], out[2], out[3], out[4]), (index, order, place, offs)):
            assert torch.equal(got.cpu().long(), want)
        # a probability: its exponent (6 times the largest logit in roundings), and 48 more, for the weights twice
        off = (6 * x.abs().max() + 48) * U
        close(out[1], w, 2 * off * w + 1e-37, "weight")
        close(out[5], slope, 2 * U * slope, "slope")
        close(out[6], loss.reshape(1), ((off + (min(len(x), 4096) + 64) * U) * loss).reshape(1), "loss")
        return out

    def route_grad(self, logits, mask, index, dweight, slope, dloss):
        d = super().route_grad(logits, mask, index, dweight, slope, dloss)
        x, m, i, dw, s = host(logits), None if mask is None else mask.cpu(), host(index), host(dweight), host(slope)
        want = self.plain.route_grad(x, m, i, dw, s, float(dloss))
        # the sum of the sizes of the formula's terms
        p = torch.softmax(x, 1)
        w = torch.gather(p, 1, i.clamp(min=0)) * (i >= 0)
        w = w / w.sum(1, keepdim=True).clamp(min=1e-300)
        h = abs(float(dloss)) * s
        size = (p * (h + (p * h).sum(1, keepdim=True))).scatter_add(
            1, i.clamp(min=0), w * (dw.abs() + (w * dw.abs()).sum(1, keepdim=True)))
        close(d, want, size * (6 * x.abs().max() + 48) * U * 4 + 1e-37, "router's gradient")
        return d


def parameters(seed, T, h, f, E, dtype, device):
    g = torch.Generator().manual_seed(seed)
    r = lambda *s, scale=1.0: torch.randn(*s, generator=g, dtype=torch.float64) * scale
    P = {"Wr": r(E, h, scale=2 * h ** -0.5), "W1": r(E, h, f, scale=h ** -0.5), "W2": r(E, f, h, scale=f ** -0.5)}
    P = {n: t.to(dtype).to(device) for n, t in P.items()}
    wide = torch.promote_types(dtype, torch.float32)
    P |= {n: t.to(wide).to(device) for n, t in (("g", 1 + r(h, scale=0.2)), ("b", r(h, scale=0.2)), ("b1", r(E, f, scale=0.3)),
                                                 ("b2", r(E, h, scale=0.3)))}
    return r(T, h).to(dtype).to(device), r(T, h).to(dtype).to(device), P


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("masked", [False, True])
def test_formulas_are_autograds(act, masked):
    T, h, f, E, k = 23, 10, 14, 6, 3
    X, dY, P = parameters(1, T, h, f, E, torch.float64, "cpu")
    mask = (torch.arange(T) % 5 != 2).to(torch.uint8) if masked else None
    block = Block(Plain(), k, act)
    Y, loss = block.forward(X, P, mask)
    G = block.backward(dY, 0.7, P)
    index, slope = block.saved[5], block.saved[10]
    leaves = {n: t.clone().requires_grad_() for n, t in {**P, "X": X}.items()}
    L = leaves
    m = L["X"].mean(1, keepdim=True)
    N = (L["X"] - m) / torch.sqrt(((L["X"] - m) ** 2).mean(1, keepdim=True) + EPS) * L["g"] + L["b"]
    p = torch.softmax(N @ L["Wr"].t(), 1)
    out = []
    for t in range(T):
        y = L["X"][t]
        if mask is None or mask[t]:
            total = p[t, index[t]].sum()
            for e in index[t].tolist():
                z = N[t] @ L["W1"][e] + L["b1"][e]
                a = {"none": lambda v: v, "relu": torch.relu, "gelu": torch.nn.functional.gelu, "silu": torch.nn.functional.silu,
                     "gelu_tanh": lambda v: torch.nn.functional.gelu(v, approximate="tanh")}[act](z)
                y = y + p[t, e] / total * (a @ L["W2"][e] + L["b2"][e])
        out.append(y)
    want = torch.stack(out)
    on = torch.ones(T, dtype=torch.float64) if mask is None else mask.double()
    n = on.sum()
    share = torch.bincount(index[index >= 0], minlength=E) / (k * n)          # constant, as the choice is
    balance = E * (share * (p * on[:, None]).sum(0) / n).sum()
    assert torch.allclose(Y, want.detach(), rtol=1e-10, atol=1e-10) and torch.allclose(loss, balance.detach(), rtol=1e-10)
    assert torch.allclose(slope, E * share / n, rtol=1e-12)
    grads = torch.autograd.grad((want * dY).sum() + 0.7 * balance, list(leaves.values()))
    for name, g in zip(leaves, grads):
        assert torch.allclose(G[name], g, rtol=1e-9, atol=1e-10), name


SIZES = [(1, 64, 96, 8, 2), (3, 72, 40, 5, 5), (70, 65, 97, 7, 2), (300, 128, 200, 24, 6), (2000, 256, 96, 16, 2),
         (1500, 64, 136, 130, 8)]


@pytest.mark.gpu
@pytest.mark.parametrize("type", ["f32", "f16", "bf16"])
@pytest.mark.parametrize("T,h,f,E,k", SIZES)
def test_every_step(T, h, f, E, k, type, gpu):
    acts = ["gelu", "silu", "gelu_tanh", "relu"]
    for masked in (False, True):
        X, dY, P = parameters(T + masked, T, h, f, E, TORCH_DT[type], DEV)
        mask = (torch.arange(T, device=DEV) % 4 != 1).to(torch.uint8) if masked else None
        block = Block(Checked(type), k, acts[(T + masked) % 4])
        Y, loss = block.forward(X, P, mask)
        G = block.backward(dY, torch.full((1,), 0.5, device=DEV), P)
        for t in (Y, loss, *G.values()):
            assert t.isfinite().all()


def everything(block, X, dY, dl, P, mask):
    Y, loss = block.forward(X, P, mask)
    G = block.backward(dY, dl, P)
    return [Y, loss, *block.saved[5:8], *(G[n] for n in sorted(G))]


@pytest.mark.gpu
@pytest.mark.parametrize("T,h,f,E,k,type", [(2, 64, 96, 8, 2, "bf16"), (400, 64, 96, 12, 3, "bf16"), (3000, 64, 72, 20, 2, "f32")])
def test_two_graphs_follow_their_inputs(T, h, f, E, k, type, gpu):
    # two graphs over the same plans, replayed on two streams, with eager work in between; every replay
    # has other inputs, and other routes
    ops = Plans(type)
    dl = torch.full((1,), 0.5, device=DEV)
    sets = [parameters(s, T, h, f, E, TORCH_DT[type], DEV) for s in range(3)]
    runs = []
    for s in range(2):
        X, dY, P = parameters(50, T, h, f, E, TORCH_DT[type], DEV)
        mask = torch.ones(T, dtype=torch.uint8, device=DEV)
        everything(Block(ops, k, "gelu"), X, dY, dl, P, mask)
        torch.cuda.synchronize()
        graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
        with torch.cuda.graph(graph, stream=stream):
            outs = everything(Block(ops, k, "gelu"), X, dY, dl, P, mask)
        runs.append((graph, stream, outs, X, dY, P, mask))
    for turn in range(4):
        for r, (graph, stream, outs, X, dY, P, mask) in enumerate(runs):
            x, dy, p = sets[(turn + r) % 3]
            X.copy_(x)
            dY.copy_(dy)
            for n in P:
                P[n].copy_(p[n])
            mask.copy_((torch.arange(T, device=DEV) + turn) % 5 != 0)
            for t in outs:
                t.fill_(7)
        torch.cuda.synchronize()
        for graph, stream, *_ in runs:
            with torch.cuda.stream(stream):
                graph.replay()
        torch.cuda.synchronize()
        for graph, stream, outs, X, dY, P, mask in runs:
            want = everything(Block(ops, k, "gelu"), X, dY, dl, P, mask)
            torch.cuda.synchronize()
            for got, w in zip(outs, want):
                assert torch.equal(got, w)
