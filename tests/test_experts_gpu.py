"""A mixture-of-experts layer made of the grouped plans, as it would be used: the forward pass of two
expert layers with a ReLU between them, every gradient (against the formulas in 64 bits and against
differences of the forward pass), gradients added over two batches, the same weights served in 4
bits, and all of it captured in graphs whose offsets change between replays, on other streams, and
from two graphs at once."""
import numpy as np
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import SENTINEL, TORCH_DT, ints, offsets_of

pytestmark = pytest.mark.gpu
DEV = "cuda:0"


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


class Layer:
    """Y = relu(X W1_e + b1_e) W2_e + b2_e over row ranges, with its gradients; buffers made once."""

    def __init__(self, T, E, h, f, ab, cd):
        self.T, self.E, self.h, self.f = T, E, h, f
        tab, tcd = TORCH_DT[ab], TORCH_DT[cd]
        P, G = tge.GroupedPlan, tge.GroupedGradPlan
        self.p1 = P(T, f, h, E, "N", ab=ab, cd=ab, epilogue="bias_relu")
        self.p2 = P(T, h, f, E, "N", ab=ab, cd=cd, epilogue="bias")
        self.d2 = P(T, f, h, E, "T", ab=ab, cd=ab, epilogue="gate")     # W2 is f x h: dY W2^T
        self.d1 = P(T, h, f, E, "T", ab=ab, cd=cd)
        self.g1 = G(T, h, f, E, ab=ab, cd="f32")
        self.g2 = G(T, f, h, E, ab=ab, cd="f32")
        z = lambda *s, dtype: torch.zeros(*s, dtype=dtype, device=DEV)
        self.H, self.Y = z(T, f, dtype=tab), z(T, h, dtype=tcd)
        self.dH, self.dX = z(T, f, dtype=tab), z(T, h, dtype=tcd)
        self.dW1, self.dW2 = z(E, h, f, dtype=torch.float32), z(E, f, h, dtype=torch.float32)
        self.db1, self.db2 = z(E, f, dtype=torch.float32), z(E, h, dtype=torch.float32)

    def forward(self, X, W1, b1, W2, b2, offs, stream=None):
        self.p1.run(X, W1, None, self.H, offs, b1, stream=stream)
        self.p2.run(self.H, W2, None, self.Y, offs, b2, stream=stream)

    def backward(self, X, W1, W2, dY, offs, beta=0.0, stream=None):
        self.d2.run(dY, W2, self.H, self.dH, offs, stream=stream)
        self.g2.run(self.H, dY, self.dW2, self.dW2, offs, self.db2, beta=beta, stream=stream)
        self.d1.run(self.dH, W1, None, self.dX, offs, stream=stream)
        self.g1.run(X, self.dH, self.dW1, self.dW1, offs, self.db1, beta=beta, stream=stream)

    def outputs(self):
        return [x.clone() for x in (self.Y, self.dX, self.dW1, self.dW2, self.db1, self.db2)]


def data(seed, T, E, h, f, ab):
    """Integers small enough that every intermediate is exact in fp16 and bf16 alike (below 256)."""
    g = np.random.default_rng(seed)
    t = TORCH_DT[ab]
    sparse = lambda *s: ints(g, s, -1, 1, torch.float32) * ints(g, s, 0, 3, torch.float32).eq(0)
    X = sparse(T, h).to(t)
    W1, W2 = sparse(E, h, f).to(t), sparse(E, f, h).to(t)
    b1, b2 = ints(g, (E, f), -2, 2, torch.float32), ints(g, (E, h), -2, 2, torch.float32)
    dY = sparse(T, h).to(t)
    return [x.to(DEV) for x in (X, W1, b1, W2, b2, dY)]


def reference(X, W1, b1, W2, b2, dY, offs):
    """(Y, dX, dW1, dW2, db1, db2) in 64 bits by autograd; rows outside the ranges zero."""
    X, W1, b1, W2, b2, dY = (x.detach().double().cpu() for x in (X, W1, b1, W2, b2, dY))
    leaves = [x.requires_grad_() for x in (X, W1, b1, W2, b2)]
    Y = torch.zeros(X.shape[0], W2.shape[2], dtype=torch.float64)
    parts = []
    for e, (lo, hi) in enumerate(zip(offs[:-1], offs[1:])):
        parts.append((lo, hi, torch.relu(X[lo:hi] @ W1[e] + b1[e]) @ W2[e] + b2[e]))
    loss = sum((y * dY[lo:hi]).sum() for lo, hi, y in parts)
    for lo, hi, y in parts:
        Y[lo:hi] = y.detach()
    dX, dW1, db1, dW2, db2 = torch.autograd.grad(loss, leaves)
    return [Y, dX, dW1, dW2, db1, db2]


def check(got, want):
    for name, a, b in zip(("Y", "dX", "dW1", "dW2", "db1", "db2"), got, want):
        assert torch.equal(a.cpu().double(), b), f"{name}: {int((a.cpu().double() != b).sum())} differ"


SHAPES = [(37, 5, 24, 40, "f32", "f32"), (300, 6, 64, 96, "f16", "f32"), (300, 6, 65, 97, "bf16", "f32"),
          (1500, 9, 128, 64, "bf16", "f32")]


@pytest.mark.parametrize("T,E,h,f,ab,cd", SHAPES)
def test_layer_and_its_gradients(T, E, h, f, ab, cd):
    x = data(1, T, E, h, f, ab)
    counts = np.random.default_rng(2).multinomial(T - 3, np.ones(E) / E)
    counts[1] += counts[2]
    counts[2] = 0                                   # an expert without rows
    offs = offsets_of(counts, 1)
    d = torch.from_numpy(offs).to(DEV)
    layer = Layer(T, E, h, f, ab, cd)
    layer.forward(*x[:5], d)
    layer.backward(x[0], x[1], x[3], x[5], d)
    want = reference(*x, offs)
    check(layer.outputs(), want)
    # a second batch added to the weights' gradients (bias gradients are written)
    layer.backward(x[0], x[1], x[3], x[5], d, beta=1.0)
    assert torch.equal(layer.dW1.cpu().double(), 2 * want[2])
    assert torch.equal(layer.dW2.cpu().double(), 2 * want[3])
    assert torch.equal(layer.db1.cpu().double(), want[4])


def test_gradients_against_differences():
    # in fp32, integers: the layer is linear in each parameter while no ReLU switches, so that
    # (L(p + 1/4) - L(p - 1/4)) * 2 is the gradient exactly; the biases keep every ReLU's argument at
    # least 1/2 away from 0 and the steps move it by 1/4 at most
    T, E, h, f = 19, 3, 7, 9
    x = data(3, T, E, h, f, "f32")
    x[2] = torch.where(x[2] >= 0, x[2] + 0.5, x[2] - 0.5)
    offs = offsets_of([8, 0, 10], 1)
    d = torch.from_numpy(offs).to(DEV)
    layer = Layer(T, E, h, f, "f32", "f32")
    layer.forward(*x[:5], d)
    layer.backward(x[0], x[1], x[3], x[5], d)
    X, dX, dW1, dW2, db1, db2 = (v.cpu() for v in layer.outputs())

    def loss():
        layer.forward(*x[:5], d)
        return float((layer.Y.double() * x[5].double())[offs[0]:offs[-1]].sum())

    g = np.random.default_rng(4)
    for p, grad in ((0, dX), (1, dW1), (2, db1), (3, dW2), (4, db2)):
        flat = x[p].view(-1)
        for i in g.choice(flat.numel(), min(25, flat.numel()), replace=False):
            flat[i] += 0.25
            up = loss()
            flat[i] -= 0.5
            down = loss()
            flat[i] += 0.25
            assert 2 * (up - down) == float(grad.view(-1)[i]), (p, i)


def test_captured_layer_follows_the_offsets():
    # one graph of a training step; the routing changes between replays, with eager work between
    T, E, h, f = 300, 6, 64, 96
    x = data(5, T, E, h, f, "bf16")
    layer, eager = Layer(T, E, h, f, "bf16", "f32"), Layer(T, E, h, f, "bf16", "f32")
    d = torch.zeros(E + 1, dtype=torch.int32, device=DEV)
    layer.forward(*x[:5], d)
    torch.cuda.synchronize()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        layer.forward(*x[:5], d)
        layer.backward(x[0], x[1], x[3], x[5], d)
    for seed in range(4):
        counts = np.random.default_rng(seed).multinomial(T - 40 * seed, np.ones(E) / E)
        offs = offsets_of(counts, 7 * seed)
        d.copy_(torch.from_numpy(offs))
        for t in (layer.Y, layer.dX, layer.H, layer.dH):
            t.zero_()
        g.replay()
        torch.cuda.synchronize()
        check(layer.outputs(), reference(*x, offs))
        eager.forward(*x[:5], d)
        eager.backward(x[0], x[1], x[3], x[5], d)
        torch.cuda.synchronize()
        assert torch.equal(eager.dW1, layer.dW1)


def test_two_graphs_and_streams_share_the_plans():
    # the plans hold no memory: two graphs over the same plans, replayed at once on two streams, and
    # an eager run on a third
    T, E, h, f = 300, 6, 64, 96
    offs = offsets_of(np.random.default_rng(6).multinomial(T, np.ones(E) / E))
    d = torch.from_numpy(offs).to(DEV)
    runs = []
    plans = Layer(T, E, h, f, "f16", "f32")
    for seed in (7, 8, 9):
        layer = Layer(T, E, h, f, "f16", "f32")
        layer.p1, layer.p2, layer.d1, layer.d2, layer.g1, layer.g2 = (
            plans.p1, plans.p2, plans.d1, plans.d2, plans.g1, plans.g2)
        runs.append((layer, data(seed, T, E, h, f, "f16"), torch.cuda.Stream()))
    torch.cuda.synchronize()
    graphs = []
    for layer, x, s in runs[:2]:
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g, stream=s):
            layer.forward(*x[:5], d)
            layer.backward(x[0], x[1], x[3], x[5], d)
        graphs.append(g)
    torch.cuda.synchronize()
    for _ in range(3):
        for g, (_, _, s) in zip(graphs, runs):
            with torch.cuda.stream(s):
                g.replay()
        layer, x, s = runs[2]
        layer.forward(*x[:5], d, stream=s)                       # a stream object
        layer.backward(x[0], x[1], x[3], x[5], d, stream=s.cuda_stream)   # a raw handle
        torch.cuda.synchronize()
        for layer, x, _ in runs:
            check(layer.outputs(), reference(*x, offs))
            for t in (layer.Y, layer.dX, layer.dW1, layer.dW2, layer.db1, layer.db2):
                t.fill_(SENTINEL if t is layer.dW1 else 0)
    with torch.cuda.stream(runs[0][2]):                           # the current stream is the default
        runs[0][0].forward(*runs[0][1][:5], d)
        runs[0][2].synchronize()
    assert torch.equal(runs[0][0].Y.cpu().double(), reference(*runs[0][1], offs)[0])


def test_served_in_16_and_in_4_bits():
    # weights whose 4-bit form is exact: both plans give the same integers, for a prompt's rows and
    # for single tokens, eagerly and from a graph
    E, h, f, block = 5, 128, 72, 64
    g = np.random.default_rng(10)
    codes = g.integers(0, 16, (E, f, h))
    zeros = g.integers(6, 10, (E, f, h // block)).astype(np.uint8)
    scales = 2.0 ** g.integers(-1, 2, (E, f, h // block))
    W = ((codes - np.repeat(zeros, block, 2)) * np.repeat(scales, block, 2)).astype(np.float32)
    Q = torch.from_numpy((codes[..., 0::2] | codes[..., 1::2] << 4).astype(np.uint8)).to(DEV)
    z, s = torch.from_numpy(zeros).to(DEV), torch.from_numpy(scales).to(torch.bfloat16).to(DEV)
    W = torch.from_numpy(W).to(torch.bfloat16).to(DEV)
    bias = ints(g, (E, f), -3, 3, torch.float32).to(DEV)
    for counts in ([1, 0, 0, 2, 1], [200, 3, 0, 64, 1]):
        T = sum(counts)
        offs = torch.from_numpy(offsets_of(counts)).to(DEV)
        A = ints(g, (T, h), -2, 2, torch.bfloat16).to(DEV)
        D16 = torch.zeros(T, f, dtype=torch.float32, device=DEV)
        D4, Dg = torch.zeros_like(D16), torch.zeros_like(D16)
        p16 = tge.GroupedPlan(T, f, h, E, "T", ab="bf16", cd="f32", epilogue="bias_relu")
        p4 = tge.QuantPlan(T, f, h, block, E, zeros=True, ab="bf16", cd="f32", epilogue="bias_relu")
        p16.run(A, W, None, D16, offs, bias)
        p4.run(A, Q, s, z, None, D4, offs, bias)
        assert torch.equal(D16, D4) and (D16 > 0).any()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            p4.run(A, Q, s, z, None, Dg, offs, bias)
        for _ in range(3):
            Dg.zero_()
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(Dg, D16)
            p16.run(A, W, None, D4, offs, bias)


def test_runs_are_deterministic():
    g = torch.Generator(device=DEV).manual_seed(11)
    r = lambda *s: torch.randn(*s, generator=g, device=DEV).to(torch.bfloat16)
    offs = torch.from_numpy(offsets_of([700, 5, 0, 300])).to(DEV)
    A, B, G = r(1005, 512), r(4, 512, 264), r(1005, 264)
    outs = []
    for _ in range(3):
        D = torch.empty(1005, 264, dtype=torch.bfloat16, device=DEV)
        W, b = torch.empty(4, 512, 264, device=DEV), torch.empty(4, 264, device=DEV)
        tge.GroupedPlan(1005, 264, 512, 4, ab="bf16", cd="bf16").run(A, B, None, D, offs)
        tge.GroupedGradPlan(1005, 512, 264, 4, ab="bf16").run(A, G, None, W, offs, b)
        outs.append((D, W, b))
    for o in outs[1:]:
        assert all(torch.equal(x, y) for x, y in zip(o, outs[0]))


def test_tensors_of_another_device_are_refused():
    p = tge.GroupedPlan(8, 16, 16, 2)
    offs = torch.tensor([0, 4, 8], dtype=torch.int32, device=DEV)
    A, B = torch.zeros(8, 16).half(), torch.zeros(2, 16, 16).half()
    D = torch.zeros(8, 16, device=DEV).half()
    with pytest.raises(ValueError, match="A must be a device tensor"):
        p.run(A, B.to(DEV), None, D, offs)
    with pytest.raises(ValueError, match="offsets must be a device tensor"):
        p.run(A.to(DEV), B.to(DEV), None, D, offs.cpu())
    with pytest.raises(TypeError, match="D must be"):
        p.run(A.to(DEV), B.to(DEV), None, D.float(), offs)
    with pytest.raises(ValueError, match="B holds"):
        p.run(A.to(DEV), B[:1].to(DEV), None, D, offs)
    with pytest.raises(tge.GemmError, match="INVALID_VALUE"):
        p.run(A.to(DEV), B.to(DEV), None, D, None)
