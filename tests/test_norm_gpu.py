"""Layer norm and its gradients against 64 bits: every shape of team, type, odd and short rows, strides,
missing weights, residual gradients, values that cancel, NaN and infinities, graphs and streams."""
import pytest
import torch

import tiled_gemm_epilogues_amd as tge
from grouped_helpers import SENTINEL, TORCH_DT
from layer_helpers import U, close, rounding

pytestmark = pytest.mark.gpu
DEV = "cuda:0"
NAN = float("nan")
EPS = 1e-5
# rows of 1, 2, 3, 4, ... KiB in 16 bits: every team's shape, whole and ragged; and rows below a chunk
WIDTHS = [1, 2, 3, 7, 8, 9, 63, 64, 511, 512, 513, 1000, 1024, 1025, 1536, 2048, 2500, 3000, 4096, 4097, 5120, 6144,
          8191, 8192, 10240, 12288, 12289, 16384, 20001, 24576, 32768]


@pytest.fixture(autouse=True)
def _need_gpu():
    if not torch.cuda.is_available():
        pytest.skip("no GPU")


def inputs(seed, rows, N, type, shift=0.5):
    g = torch.Generator().manual_seed(seed)
    t = TORCH_DT[type]
    X = (torch.randn(rows, N, generator=g) * (0.5 + torch.rand(N, generator=g)) + shift).to(t)
    weight, bias = 1 + 0.3 * torch.randn(N, generator=g), 0.3 * torch.randn(N, generator=g)
    dY, C = torch.randn(rows, N, generator=g).to(t), torch.randn(rows, N, generator=g).to(t)
    return X, weight, bias, dY, C


def forward64(X, weight, bias, eps=EPS):
    x = X.double()
    m = x.mean(1, keepdim=True)
    r = 1 / torch.sqrt(((x - m) ** 2).mean(1, keepdim=True) + eps)
    return (x - m) * r * weight.double() + bias.double(), m[:, 0], r[:, 0]


def depth(N):
    """Additions on the way of one term of a sum of N: up to 32 in a lane, 6 between lanes, 16 between
    waves, and the joining of parts."""
    return min(N, 32) + 6 + 16 + 4


def stats_bounds(X, eps=EPS):
    """(bound of |mean|'s error, relative bound of rstd's): every addition rounds by at most U of the sum of
    the sizes; the squared deviations are taken from a part's own mean, whose error adds its square."""
    x = X.double()
    N = x.shape[1]
    d = depth(N) + 2
    em = d * U * x.abs().mean(1)
    m = x.mean(1, keepdim=True)
    var = ((x - m) ** 2).mean(1)
    # deviations: each has one rounding of itself and the error of its part's mean (em, of which the sum of
    # the deviations is 0 but for roundings)
    ev = (2 * d + 6) * U * var + 4 * em * em + 4 * U * em * (x - m).abs().mean(1)
    rel = 0.5 * ev / (var + eps) + 4 * U
    return em, rel


def check_forward(X, weight, bias, Y, mean, rstd, type, eps=EPS):
    want, m, r = forward64(X, weight, bias, eps)
    em, rel = stats_bounds(X, eps)
    close(mean, m, em, "mean")
    close(rstd, r, r * rel, "rstd")
    h = ((X.double() - m[:, None]) * r[:, None]).abs()
    bound = weight.double().abs() * ((em * r)[:, None] + h * (rel + 2 * U)[:, None]) + 2 * U * want.abs() \
        + U * bias.double().abs()
    close(Y, want, bound + rounding(want.abs() + bound, TORCH_DT[type]) * 1.0001, "Y")


def grad64(dY, X, weight, mean, rstd, C=None, beta=0.0):
    dy, h, w = dY.double(), (X.double() - mean.double()[:, None]) * rstd.double()[:, None], weight.double()
    g = dy * w
    dx = rstd.double()[:, None] * (g - g.mean(1, keepdim=True) - h * (g * h).mean(1, keepdim=True))
    if C is not None:
        dx = dx + beta * C.double()
    return dx, (dy * h).sum(0), dy.sum(0)


def check_grad(dY, X, weight, mean, rstd, C, beta, dX, dw, db, type):
    want, ww, wb = grad64(dY, X, weight, mean, rstd, C if beta else None, beta)
    N, rows = X.shape[1], X.shape[0]
    dy, r = dY.double().abs(), rstd.double()[:, None]
    x0 = X.double() - mean.double()[:, None]
    h = (x0 * r).abs()
    g = dy * weight.double().abs()
    d = depth(N) + 4
    # h has two roundings, each product one more, each sum d; the result's differences one each
    a, b = g.mean(1, keepdim=True), (g * h).mean(1, keepdim=True)
    bound = r * (4 * U * g + (d + 4) * U * a + h * (d + 8) * U * b) + 3 * U * want.abs()
    if beta:
        bound = bound + U * (beta * C.double()).abs()
    if dX is not None:
        close(dX, want, bound + rounding(want.abs() + bound, TORCH_DT[type]) * 1.0001, "dX")
    # column sums: rows additions at most, each of at most U of the sum of the sizes
    if dw is not None:
        close(dw, ww, (min(rows, 4096) + 8) * U * (dy * h).sum(0) + 1e-37, "dweight")
    if db is not None:
        close(db, wb, (min(rows, 4096) + 8) * U * dy.sum(0) + 1e-37, "dbias")


def run_all(rows, N, type, seed=0, pad=0, beta=0.0, shift=0.5):
    X, weight, bias, dY, C = inputs(seed, rows, N, type, shift)
    t = TORCH_DT[type]
    plan = tge.NormPlan(rows, N, type=type, eps=EPS, ldx=N + pad, ldy=N + 2 * pad)

    def wide(x, extra):
        out = torch.full((rows, N + extra), SENTINEL, dtype=t, device=DEV)
        out[:, :N] = x.to(DEV)
        return out
    Xd, Y = wide(X, pad), torch.full((rows, N + 2 * pad), SENTINEL, dtype=t, device=DEV)
    mean, rstd = torch.full((rows,), NAN, device=DEV), torch.full((rows,), NAN, device=DEV)
    plan.run(Xd, weight.to(DEV), bias.to(DEV), Y, mean, rstd)
    check_forward(X, weight, bias, Y[:, :N], mean, rstd, type)
    dX = torch.full((rows, N + pad), SENTINEL, dtype=t, device=DEV)
    dw, db = torch.full((N,), NAN, device=DEV), torch.full((N,), NAN, device=DEV)
    plan.run_grad(wide(dY, 2 * pad), Xd, weight.to(DEV), mean, rstd, dX, dw, db, wide(C, pad) if beta else None, beta)
    check_grad(dY, X, weight, mean.cpu(), rstd.cpu(), C, beta, dX[:, :N], dw, db, type)
    assert (Y[:, N:] == SENTINEL).all() and (dX[:, N:] == SENTINEL).all()


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N", WIDTHS)
def test_widths(N, type):
    if type == "f32" and N > 16384:
        N //= 2
    run_all(37, N, type, seed=N)
    run_all(5, N, type, seed=N + 1, pad=3, beta=0.5)


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("rows", [1, 2, 3, 8, 9, 255, 1000, 5003])
def test_rows(rows, type):
    for N in (24, 200, 1001, 2304):
        run_all(rows, N, type, seed=rows, beta=1.0)


@pytest.mark.parametrize("type", ["f16", "bf16", "f32"])
@pytest.mark.parametrize("N", [1, 3, 8, 9, 31, 32, 33, 64, 65, 100, 128, 129, 200, 256, 257])
def test_short_rows(N, type):
    # rows that share a wave, all of them there and not
    for rows in (1, 2, 5, 31, 33, 65, 517, 9001):
        run_all(rows, N, type, seed=rows, pad=rows % 3, beta=0.5 * (rows % 2))


@pytest.mark.parametrize("type", ["bf16", "f32"])
@pytest.mark.parametrize("off", [1, 2, 5])
def test_pointers_off_the_16_byte_grid(off, type):
    rows, N, t = 20, 700, TORCH_DT[type]
    X, weight, bias, dY, C = inputs(3, rows, N, type)
    plan = tge.NormPlan(rows, N, type=type, eps=EPS)

    def moved(x):
        buf = torch.full((x.numel() + off + 8,), SENTINEL, dtype=x.dtype, device=DEV)
        buf[off:off + x.numel()] = x.reshape(-1).to(DEV)
        return buf, buf[off:off + x.numel()].view(x.shape)
    _, Xd = moved(X)
    full, Y = moved(torch.zeros(rows, N, dtype=t))
    _, w = moved(weight)
    _, b = moved(bias)
    mean, rstd = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
    plan.run(Xd, w, b, Y, mean, rstd)
    check_forward(X, weight, bias, Y, mean, rstd, type)
    assert (full[:off] == SENTINEL).all() and (full[off + rows * N:] == SENTINEL).all()
    _, dYd = moved(dY)
    _, Cd = moved(C)
    fullx, dX = moved(torch.zeros(rows, N, dtype=t))
    fullw, dw = moved(torch.zeros(N))
    _, db = moved(torch.zeros(N))
    plan.run_grad(dYd, Xd, w, mean, rstd, dX, dw, db, Cd, 1.0)
    check_grad(dY, X, weight, mean.cpu(), rstd.cpu(), C, 1.0, dX, dw, db, type)
    assert (fullx[:off] == SENTINEL).all() and (fullx[off + rows * N:] == SENTINEL).all()
    assert (fullw[:off] == SENTINEL).all() and (fullw[off + N:] == SENTINEL).all()


def test_optional_operands():
    rows, N = 33, 520
    X, weight, bias, dY, C = inputs(4, rows, N, "f32")
    one, zero = torch.ones(N), torch.zeros(N)
    plan = tge.NormPlan(rows, N, type="f32", eps=EPS)
    mean, rstd, Y = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV), torch.zeros(rows, N, device=DEV)
    plan.run(X.to(DEV), None, None, Y, mean, rstd)
    check_forward(X, one, zero, Y, mean, rstd, "f32")
    Y2 = torch.zeros(rows, N, device=DEV)
    plan.run(X.to(DEV), None, None, Y2)
    assert torch.equal(Y, Y2)
    args = (dY.to(DEV), X.to(DEV), None, mean, rstd)
    dX, dw, db = torch.zeros(rows, N, device=DEV), torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)
    plan.run_grad(*args, dX)
    check_grad(dY, X, one, mean.cpu(), rstd.cpu(), C, 0.0, dX, None, None, "f32")
    plan.run_grad(*args, dX, dw)
    plan.run_grad(*args, dX, None, db)
    check_grad(dY, X, one, mean.cpu(), rstd.cpu(), C, 0.0, dX, dw, db, "f32")


def test_in_place():
    rows, N = 70, 1500
    X, weight, bias, dY, C = (t.to(DEV) for t in inputs(5, rows, N, "bf16"))
    plan = tge.NormPlan(rows, N, type="bf16", eps=EPS)
    Y, Y2, mean, rstd = torch.zeros_like(X), X.clone(), torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
    plan.run(X, weight, bias, Y, mean, rstd)
    plan.run(Y2, weight, bias, Y2)
    assert torch.equal(Y, Y2)
    dX, dX2, dX3 = torch.zeros_like(X), C.clone(), dY.clone()
    plan.run_grad(dY, X, weight, mean, rstd, dX, C=C, beta=1.0)
    plan.run_grad(dY, X, weight, mean, rstd, dX2, C=dX2, beta=1.0)
    plan.run_grad(dX3, X, weight, mean, rstd, dX3, C=C, beta=1.0)
    assert torch.equal(dX, dX2) and torch.equal(dX, dX3)


@pytest.mark.parametrize("type,N", [("f32", 8449), ("f32", 12290), ("bf16", 17925), ("bf16", 25609), ("f16", 4099), ("f32", 259)])
def test_gradient_added_in_place_where_waves_share_columns(type, N):
    # the row's last chunk is that of a wave's first lane, and shares columns with the wave before
    rows = 600
    X, weight, bias, dY, C = (t.to(DEV) for t in inputs(N, rows, N, type))
    plan = tge.NormPlan(rows, N, type=type, eps=EPS)
    Y, mean, rstd = torch.empty_like(X), torch.empty(rows, device=DEV), torch.empty(rows, device=DEV)
    plan.run(X, weight, bias, Y, mean, rstd)
    apart, inside = torch.empty_like(X), C.clone()
    sums = [torch.empty(N, device=DEV) for _ in range(4)]
    plan.run_grad(dY, X, weight, mean, rstd, apart, sums[0], sums[1], C, 0.5)
    for turn in range(5):
        inside.copy_(C)
        plan.run_grad(dY, X, weight, mean, rstd, inside, sums[2], sums[3], inside, 0.5)
        assert torch.equal(inside, apart) and torch.equal(sums[0], sums[2]) and torch.equal(sums[1], sums[3])
    same = X.clone()                                # the forward pass over its own input
    plan.run(same, weight, bias, same)
    assert torch.equal(same, Y)
    own = dY.clone()                                # and the gradient over the one that comes in
    plan.run_grad(own, X, weight, mean, rstd, own, sums[2], sums[3], C, 0.5)
    assert torch.equal(own, apart)
    check_grad(*(t.cpu() for t in (dY, X, weight, mean, rstd, C)), 0.5, apart, sums[0], sums[1], type)
    # without a weight
    plan.run_grad(dY, X, None, mean, rstd, apart)
    one = torch.ones(N, device=DEV)
    plan.run_grad(dY, X, one, mean, rstd, inside)
    assert torch.equal(apart, inside)
    plan.run(X, None, None, Y)
    plan.run(X, one, torch.zeros(N, device=DEV), same)
    assert torch.equal(Y, same)


def test_refusals_name_the_operand():
    plan = tge.NormPlan(8, 16, type="f32")
    X, v, r = torch.zeros(8, 16, device=DEV), torch.zeros(16, device=DEV), torch.zeros(8, device=DEV)
    for args, err in (((X.cpu(), v, v, X), "X must be a device tensor"), ((X, v[:15], v, X), "weight holds"),
                      ((X, v, v, X[:7]), "Y holds")):
        with pytest.raises(ValueError, match=err):
            plan.run(*args)
    short = torch.zeros(plan.workspace_bytes - 1, dtype=torch.uint8, device=DEV)
    with pytest.raises(ValueError, match="workspace holds"):
        plan.run_grad(X, X, v, r, r, X.clone(), v.clone(), None, workspace=short)
    with pytest.raises(ValueError, match="needs a workspace"):
        plan.run_grad(X, X, v, r, r, X.clone(), v.clone(), None, stream=torch.cuda.Stream())
    with pytest.raises(tge.GemmError, match="INVALID_VALUE"):
        plan.run_grad(X, X, v, r, r, X.clone(), beta=1.0)


def test_means_far_from_zero_do_not_cancel():
    # deviations of 1 around 1000: the squares of the values would leave no digits of the variance
    for N in (300, 2048, 9000):
        X, weight, bias, _, _ = inputs(6, 12, N, "f32", shift=1000.0)
        plan = tge.NormPlan(12, N, type="f32", eps=EPS)
        Y, mean, rstd = torch.zeros(12, N, device=DEV), torch.zeros(12, device=DEV), torch.zeros(12, device=DEV)
        plan.run(X.to(DEV), weight.to(DEV), bias.to(DEV), Y, mean, rstd)
        check_forward(X, weight, bias, Y, mean, rstd, "f32")
        # and in figures: 3e-3 of the deviation's scale, where an error of 1e6 U in the variance is 6e-2
        r = forward64(X, weight, bias)[2]
        assert ((rstd.cpu().double() / r - 1).abs() < 1e-4).all()


def test_constant_rows_and_one_column():
    for N in (1, 5, 1024, 4100):
        X = torch.full((6, N), 2.5, dtype=torch.float32, device=DEV)
        plan = tge.NormPlan(6, N, type="f32", eps=0.25)
        bias = torch.arange(N, dtype=torch.float32, device=DEV)
        Y, mean, rstd = torch.zeros(6, N, device=DEV), torch.zeros(6, device=DEV), torch.zeros(6, device=DEV)
        plan.run(X, None, bias, Y, mean, rstd)
        # the mean of a constant is off by its roundings at most
        assert ((mean - 2.5).abs() <= 2.5 * 64 * U).all() and ((rstd - 2).abs() <= 2 * 8 * U).all()
        assert ((Y - bias).abs() <= (2.5 * 64 * 2 + bias) * 2 * U).all()


def test_nan_and_infinities_keep_to_their_rows():
    rows, N = 30, 1100
    X, weight, bias, dY, _ = inputs(7, rows, N, "f16")
    plan = tge.NormPlan(rows, N, type="f16", eps=EPS)
    X[3, 1099], X[17, 0] = NAN, float("inf")
    Y, mean, rstd = (torch.zeros(rows, N, dtype=torch.float16, device=DEV), torch.zeros(rows, device=DEV),
                     torch.zeros(rows, device=DEV))
    plan.run(X.to(DEV), weight.to(DEV), bias.to(DEV), Y, mean, rstd)
    ok = torch.ones(rows, dtype=torch.bool)
    ok[[3, 17]] = False
    assert Y.cpu()[3].isnan().all()
    check_forward(X[ok], weight, bias, Y[ok.to(DEV)], mean[ok.to(DEV)], rstd[ok.to(DEV)], "f16")


def test_no_rows_and_no_columns():
    plan = tge.NormPlan(0, 40, type="f16")
    e = torch.zeros(0, 40, dtype=torch.float16, device=DEV)
    none = torch.zeros(0, device=DEV)
    dw, db = torch.full((40,), NAN, device=DEV), torch.full((40,), NAN, device=DEV)
    plan.run(e, None, None, e, none, none)
    plan.run_grad(e, e, None, none, none, e, dw, db)
    assert (dw == 0).all() and (db == 0).all()
    plan = tge.NormPlan(4, 0, type="f16")
    e = torch.zeros(4, 0, dtype=torch.float16, device=DEV)
    plan.run(e, None, None, e)
    plan.run_grad(e, e, None, torch.zeros(4, device=DEV), torch.zeros(4, device=DEV), e, none, none)


def test_runs_repeat_in_graphs_and_on_streams():
    rows, N = 700, 1600
    X, weight, bias, dY, C = (t.to(DEV) for t in inputs(8, rows, N, "bf16"))
    plan = tge.NormPlan(rows, N, type="bf16", eps=EPS)
    out = lambda: [torch.zeros_like(X), torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV), torch.zeros_like(X),
                   torch.zeros(N, device=DEV), torch.zeros(N, device=DEV)]

    def step(o, ws=None, stream=None):
        plan.run(X, weight, bias, o[0], o[1], o[2], stream=stream)
        plan.run_grad(dY, X, weight, o[1], o[2], o[3], o[4], o[5], C, 1.0, workspace=ws, stream=stream)
    want = out()
    step(want)
    # two graphs, one that takes its workspace from the allocator, one with the caller's, replayed in turn
    a, b = out(), out()
    ws = torch.empty(plan.workspace_bytes, dtype=torch.uint8, device=DEV)
    graphs = []
    torch.cuda.synchronize()
    for o, w in ((a, None), (b, ws)):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            step(o, w)
        graphs.append(g)
    for turn in range(4):
        for o in (a, b):
            for t in o:
                t.fill_(NAN)
        for g in graphs:
            g.replay()
        scratch = out()
        step(scratch)                               # eager work between the replays
        torch.cuda.synchronize()
        for o in (a, b, scratch):
            for x, y in zip(o, want):
                assert torch.equal(x, y)
    # two streams, a workspace each
    streams = [torch.cuda.Stream() for _ in range(2)]
    outs, wss = [out() for _ in streams], [torch.empty_like(ws) for _ in streams]
    torch.cuda.synchronize()
    for _ in range(3):
        for s, o, w in zip(streams, outs, wss):
            step(o, w, s)
    torch.cuda.synchronize()
    for o in outs:
        for x, y in zip(o, want):
            assert torch.equal(x, y)


def test_gradient_against_differences():
    # fp32: the loss sum(dY Y) at X + h v and X - h v in 64 bits from the kernel's Y; its slope along v is
    # sum(dX v) up to h^2 of the third derivative and the roundings of Y over 2h
    rows, N = 6, 200
    X, weight, bias, dY, _ = inputs(9, rows, N, "f32")
    v = torch.randn(rows, N, generator=torch.Generator().manual_seed(1))
    plan = tge.NormPlan(rows, N, type="f32", eps=EPS)
    w, b = weight.to(DEV), bias.to(DEV)
    Y, mean, rstd = torch.zeros(rows, N, device=DEV), torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)

    def loss(x):
        plan.run(x.to(DEV), w, b, Y, mean, rstd)
        return (Y.cpu().double() * dY.double()).sum(1)
    h = 2.0 ** -7
    slope = (loss(X + h * v) - loss(X - h * v)) / (2 * h)
    loss(X)
    dX = torch.zeros(rows, N, device=DEV)
    plan.run_grad(dY.to(DEV), X.to(DEV), w, mean, rstd, dX)
    got = (dX.cpu().double() * v.double()).sum(1)
    scale = (dY.double().abs().sum(1) * 3)
    assert ((got - slope).abs() <= scale * (h * h * 4 + 64 * U / h)).all()


def test_rows_beyond_32_bits():
    # more than 2^32 bytes: the last rows are where they belong
    rows, N = 600000, 4096
    X = torch.zeros(rows, N, dtype=torch.bfloat16, device=DEV)
    X[:, ::2] = 1
    X[-1] *= 3
    Y = torch.full((rows, N), SENTINEL, dtype=torch.bfloat16, device=DEV)
    mean, rstd = torch.zeros(rows, device=DEV), torch.zeros(rows, device=DEV)
    plan = tge.NormPlan(rows, N, type="bf16", eps=0.0)
    plan.run(X, None, None, Y, mean, rstd)
    for r in (0, 1, 299999, 524289, rows - 1):
        assert (Y[r, ::2] == 1).all() and (Y[r, 1::2] == -1).all()
    assert float(mean[-1]) == 1.5 and float(mean[0]) == 0.5
