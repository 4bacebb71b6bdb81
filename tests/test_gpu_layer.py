"""The layer operators on a GPU against their float64 forms (layer_ref.py):
every output element within the bound that the kernels' arithmetic gives."""

import pytest
import torch

import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0, dt=BF16, ld=None, offset=0):
    """A seeded matrix or vector; with `ld` a view with that row stride that
    starts `offset` elements into its buffer."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    v = (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)
    if ld is None:
        return v
    buf = torch.full((shape[0] * ld + offset,), float("nan"), dtype=dt, device=DEV)
    view = buf[offset:].view(shape[0], ld)[:, :shape[1]]
    view.copy_(v)
    return view


def blank(rows, cols, dt=BF16, ld=None, offset=0):
    """An output full of NaN inside a buffer of sevens, and the check that
    nothing but the output was written."""
    ld = cols if ld is None else ld
    buf = torch.full((rows * ld + offset + 16,), 7.0, dtype=dt, device=DEV)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.fill_(float("nan"))

    def guarded():
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
        assert bool((buf[mask] == 7).all()), "written outside the output"

    return view, guarded


def check(name, got, want, limit=1.0):
    w = ref.worst(got, want)
    assert w <= limit, f"{name}: {w:.3g} times the bound"


# ---- linear -------------------------------------------------------------------

LINEAR = [
    # rows, k, n, dtype, act, bias, residual
    (1, 64, 64, BF16, "none", False, False),
    (1, 7168, 896, BF16, "none", False, True),
    (7, 3584, 7168, BF16, "none", False, True),
    (20, 896, 448, FP16, "gelu", True, True),
    (33, 1001, 517, BF16, "gelu_tanh", True, True),
    (64, 200, 1000, BF16, "relu", True, False),
    (128, 512, 2048, BF16, "silu", False, False),
    (129, 65, 129, FP16, "sigmoid", True, True),
    (256, 256, 256, BF16, "none", True, False),
    (257, 320, 264, BF16, "silu", True, True),
    (300, 1, 1, BF16, "none", True, True),
    (515, 8, 7, FP16, "relu", True, False),
    (1024, 640, 1536, BF16, "gelu", True, True),
    (2050, 896, 1792, FP16, "none", False, True),
    (1, 13, 4096, BF16, "none", True, False),
    (4099, 128, 72, BF16, "gelu", False, False),
]


@pytest.mark.parametrize("rows,k,n,dt,act,bias,residual", LINEAR)
def test_linear_forward_and_backward(rows, k, n, dt, act, bias, residual):
    x, W = normal(1, rows, k, dt=dt), normal(2, k, n, scale=k ** -0.5, dt=dt)
    b = normal(3, n, dt=dt) if bias else None
    res = normal(4, rows, n, dt=dt) if residual else None
    dout = normal(5, rows, n, dt=dt)
    with route.LinearPlan(rows, k, n, dt, act=act, train=True) as plan:
        saved = plan.new_saved()
        out, guard = blank(rows, n, dt)
        route.linear_forward(plan, x, W, out, bias=b, residual=res, saved=saved)
        dx, guard_dx = blank(rows, k, dt)
        dW, guard_dW = blank(k, n, dt)
        dbias = torch.full((n,), float("nan"), dtype=dt, device=DEV)
        route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW, dbias=dbias)
        plan.status()
        again = torch.full_like(out, float("nan"))
        route.linear_forward(plan, x, W, again, bias=b, residual=res)
        plan.status()
        assert torch.equal(again, out)  # the inference call is the same product
    want, z = ref.linear(x, W, b, res, act, dt)
    check("out", out, want)
    grads = ref.linear_grads(x, W, z, dout, act, dt)
    check("dx", dx, grads["dx"])
    check("dW", dW, grads["dW"])
    check("dbias", dbias, grads["dbias"])
    for g in (guard, guard_dx, guard_dW):
        g()


@pytest.mark.parametrize("rows", [1, 5, 40, 300])
def test_linear_strided_views_in_place_residual_and_fp32_out(rows):
    k, n, dt = 136, 200, BF16
    x = normal(1, rows, k, dt=dt, ld=k + 24, offset=8)
    W = normal(2, k, n, scale=k ** -0.5, dt=dt, ld=n + 8, offset=16)
    res = normal(3, rows, n, dt=FP32, ld=n + 3, offset=1)
    want, _ = ref.linear(x, W, None, res, "none", dt, FP32)
    out, guard = blank(rows, n, FP32, ld=n + 5, offset=3)
    with route.LinearPlan(2 * rows, k, n, dt, out_dtype=FP32) as plan:
        route.linear_forward(plan, x, W, out, residual=res)
        check("out", out, want)
        guard()
        route.linear_forward(plan, x, W, res, residual=res)  # in place
        plan.status()
        assert torch.equal(res, out)


@pytest.mark.parametrize("rows,k,n", [(9, 77, 131), (260, 131, 77)])
def test_linear_odd_strides_and_offsets(rows, k, n):
    """Widths that are no multiple of 8: any alignment of rows and bases."""
    dt = BF16
    x = normal(1, rows, k, dt=dt, ld=k + 2, offset=1)
    W = normal(2, k, n, scale=k ** -0.5, dt=dt, ld=n + 4, offset=3)
    b = normal(3, n, dt=dt)
    dout = normal(4, rows, n, dt=dt, ld=n + 1, offset=5)
    out, g0 = blank(rows, n, dt, ld=n + 1, offset=1)
    dx, g1 = blank(rows, k, dt, ld=k + 3, offset=1)
    dW, g2 = blank(k, n, dt, ld=n + 2, offset=7)
    with route.LinearPlan(rows, k, n, dt, act="silu", train=True) as plan:
        saved = plan.new_saved()
        route.linear_forward(plan, x, W, out, bias=b, saved=saved)
        route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW)
        plan.status()
    want, z = ref.linear(x, W, b, None, "silu", dt)
    grads = ref.linear_grads(x, W, z, dout, "silu", dt)
    for name, got, w in (("out", out, want), ("dx", dx, grads["dx"]), ("dW", dW, grads["dW"])):
        check(name, got, w)
    for g in (g0, g1, g2):
        g()


# ---- gated --------------------------------------------------------------------

GATED = [
    # rows, k, f, n, dtype, act, residual
    (1, 7168, 512, 7168, BF16, "silu", True),
    (8, 896, 1024, 896, BF16, "silu", False),
    (20, 256, 130, 64, FP16, "gelu", True),
    (33, 100, 51, 77, BF16, "gelu_tanh", True),
    (130, 512, 640, 512, BF16, "silu", False),
    (257, 264, 200, 328, FP16, "sigmoid", True),
    (700, 1000, 702, 1000, BF16, "relu", False),
    (1030, 448, 896, 448, BF16, "silu", True),
    (2, 1, 1, 1, BF16, "silu", True),
    (512, 64, 17, 9, FP16, "none", False),
]


@pytest.mark.parametrize("rows,k,f,n,dt,act,residual", GATED)
def test_gated_forward_and_backward(rows, k, f, n, dt, act, residual):
    x = normal(1, rows, k, dt=dt)
    Wg, Wu = normal(2, k, f, scale=k ** -0.5, dt=dt), normal(3, k, f, scale=k ** -0.5, dt=dt)
    Wd = normal(4, f, n, scale=f ** -0.5, dt=dt)
    res = normal(5, rows, n, dt=dt) if residual else None
    dout = normal(6, rows, n, dt=dt)
    with route.GatedPlan(rows, k, f, n, dt, act=act, train=True) as plan:
        saved = plan.new_saved()
        out, g0 = blank(rows, n, dt)
        route.gated_forward(plan, x, Wg, Wu, Wd, out, residual=res, saved=saved)
        dx, g1 = blank(rows, k, dt)
        dWg, g2 = blank(k, f, dt)
        dWu, g3 = blank(k, f, dt)
        dWd, g4 = blank(f, n, dt)
        route.gated_backward(plan, dout, x, Wg, Wu, Wd, saved, dx=dx, dW_gate=dWg, dW_up=dWu,
                             dW_down=dWd)
        again = torch.full_like(out, float("nan"))
        route.gated_forward(plan, x, Wg, Wu, Wd, again, residual=res)
        only, g5 = blank(f, n, dt)
        route.gated_backward(plan, dout, x, Wg, Wu, Wd, saved, dW_down=only)
        plan.status()
        assert torch.equal(again, out) and torch.equal(only, dWd)
    want, kept = ref.gated(x, Wg, Wu, Wd, res, act, dt)
    check("out", out, want)
    grads = ref.gated_grads(x, Wg, Wu, Wd, kept, dout, act, dt)
    for name, got in (("dx", dx), ("dW_gate", dWg), ("dW_up", dWu), ("dW_down", dWd)):
        check(name, got, grads[name])
    for g in (g0, g1, g2, g3, g4, g5):
        g()


# ---- norm ---------------------------------------------------------------------

def norm_ref(x, gamma, beta, eps, dt):
    v = x.double()
    n = v.shape[1]
    mean = v.mean(1, keepdim=True)
    d = v - mean
    var = (d * d).mean(1, keepdim=True)
    r = (var + eps) ** -0.5
    g = gamma.double() if gamma is not None else torch.ones(n, device=DEV, dtype=torch.float64)
    b = beta.double() if beta is not None else torch.zeros(n, device=DEV, dtype=torch.float64)
    y = d * r * g + b
    # FP32 sums over blocks of at most 64 in sequence: the mean within
    # 2^-18 of the mean magnitude, and through it each deviation; the
    # variance within 2^-18 of itself and the squared error of the mean
    em = 2.0 ** -18 * v.abs().mean(1, keepdim=True)
    er = r * (2.0 ** -18 + 0.5 * r * r * em * em)
    e = (em * r + d.abs() * er + ref.F32 * d.abs() * r) * g.abs() + ref.F32 * (y.abs() + b.abs())
    return ref.rounded((y, e), dt), mean, r


NORM = [(1, 7168, BF16), (3, 1, BF16), (5, 8, FP32), (9, 64, FP16), (33, 1000, BF16),
        (64, 1001, FP32), (130, 1024, BF16), (17, 1032, FP16), (300, 3584, BF16),
        (40, 4097, BF16), (70, 8192, FP32), (11, 9000, FP16), (6, 16384, BF16), (2, 16383, FP32),
        (2000, 96, BF16)]


@pytest.mark.parametrize("rows,dim,dt", NORM)
def test_norm_forward_and_backward(rows, dim, dt):
    x = normal(1, rows, dim, dt=dt) * 3 + normal(2, rows, 1, dt=dt)
    x = x.to(dt)
    gamma, beta = (1 + normal(3, dim, dt=dt) * 0.3).to(dt), normal(4, dim, dt=dt)
    dy = normal(5, rows, dim, dt=dt)
    y, g0 = blank(rows, dim, dt)
    dx, g1 = blank(rows, dim, dt)
    stats = torch.full((rows, 2), float("nan"), device=DEV)
    dgamma, dbeta = (torch.full((dim,), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    with route.NormPlan(rows, dim, dt) as plan:
        route.norm_forward(plan, x, gamma, beta, y, stats=stats)
        route.norm_backward(plan, dy, x, gamma, stats, dx=dx, dgamma=dgamma, dbeta=dbeta)
        plan.status()
    want, mean, r = norm_ref(x, gamma, beta, 1e-5, dt)
    check("y", y, want)
    em = 2.0 ** -18 * x.double().abs().mean(1, keepdim=True)
    check("mean", stats[:, :1], (mean, em + 1e-30))
    # the backward pass with the statistics that it was given
    m, s = stats[:, :1].double(), stats[:, 1:].double()
    xh = (x.double() - m) * s
    exh = ref.F32 * (x.double().abs() + m.abs()) * s
    g = dy.double() * gamma.double()
    a, b = g.mean(1, keepdim=True), (g * xh).mean(1, keepdim=True)
    ea = 2.0 ** -18 * g.abs().mean(1, keepdim=True)
    eb = 2.0 ** -18 * (g * xh).abs().mean(1, keepdim=True) + (g.abs() * exh).mean(1, keepdim=True)
    v = s * (g - a - xh * b)
    e = s * (ref.F32 * (g.abs() + a.abs() + (xh * b).abs()) + ea + xh.abs() * eb + exh * b.abs())
    check("dx", dx, ref.rounded((v, e), dt))
    terms = dy.double() * xh
    eg = dy.double().abs() * exh + ref.F32 * terms.abs()
    check("dgamma", dgamma, ref.rounded(ref.column_sum((terms, eg)), dt))
    check("dbeta", dbeta, ref.rounded(ref.column_sum(ref.exact(dy)), dt))
    g0()
    g1()


def test_norm_views_partial_gradients_and_in_place():
    rows, dim, dt = 37, 333, BF16
    x = normal(1, rows, dim, dt=dt, ld=dim + 2, offset=1)
    dy = normal(2, rows, dim, dt=dt, ld=dim + 1, offset=3)
    gamma = normal(3, dim, dt=dt)
    y, g0 = blank(rows, dim, dt, ld=dim + 4, offset=1)
    stats = torch.empty((rows, 2), device=DEV)
    with route.NormPlan(64, dim, dt) as plan:
        route.norm_forward(plan, x, gamma, None, y, stats=stats, eps=0.5)
        check("y", y, norm_ref(x, gamma, None, 0.5, dt)[0])
        full = [torch.empty((rows, dim), dtype=dt, device=DEV)] + \
               [torch.empty((dim,), dtype=dt, device=DEV) for _ in range(2)]
        route.norm_backward(plan, dy, x, gamma, stats, dx=full[0], dgamma=full[1], dbeta=full[2])
        for i, name in enumerate(("dx", "dgamma", "dbeta")):
            one = torch.empty_like(full[i])
            route.norm_backward(plan, dy, x, gamma, stats, **{name: one})
            assert torch.equal(one, full[i]), name
        want = full[0].clone()
        route.norm_backward(plan, dy, x, gamma, stats, dx=dy)  # over its own input
        assert torch.equal(dy, want)
        route.norm_forward(plan, x, None, None, x, eps=0.5)
        plan.status()
    g0()


def test_norm_constant_rows_and_large_offsets():
    """A constant row's variance is zero; a row far from zero keeps the
    variance of its deviations."""
    dim = 1024
    x = torch.full((3, dim), 2.5, device=DEV)
    x[1] = 4096.0 + torch.arange(dim, device=DEV) % 4
    x[2] = 0
    y = torch.empty_like(x)
    with route.NormPlan(3, dim, FP32) as plan:
        route.norm_forward(plan, x, None, None, y)
        plan.status()
    want = (x - x.mean(1, keepdim=True)).double()
    want = want / (want.square().mean(1, keepdim=True) + 1e-5).sqrt()
    assert torch.equal(y[0], torch.zeros_like(y[0])) and torch.equal(y[2], torch.zeros_like(y[2]))
    assert (y - want).abs().max() < 1e-5


# ---- common behaviour -----------------------------------------------------------

def test_zero_rows():
    k, f, n = 72, 48, 40
    e = lambda *s: torch.empty(s, dtype=BF16, device=DEV)  # noqa: E731
    nan = lambda *s: torch.full(s, float("nan"), dtype=BF16, device=DEV)  # noqa: E731
    with route.LinearPlan(4, k, n, BF16, act="silu", train=True) as lin, \
            route.GatedPlan(4, k, f, n, BF16, train=True) as gated, \
            route.NormPlan(4, k, BF16) as norm:
        dW, db = nan(k, n), nan(n)
        route.linear_forward(lin, e(0, k), e(k, n), e(0, n))
        route.linear_backward(lin, e(0, n), e(0, k), e(k, n), dx=e(0, k), dW=dW, dbias=db)
        ws = nan(k, f), nan(k, f), nan(f, n)
        route.gated_forward(gated, e(0, k), e(k, f), e(k, f), e(f, n), e(0, n))
        route.gated_backward(gated, e(0, n), e(0, k), e(k, f), e(k, f), e(f, n), None, dx=e(0, k),
                             dW_gate=ws[0], dW_up=ws[1], dW_down=ws[2])
        dg = nan(k)
        route.norm_forward(norm, e(0, k), None, None, e(0, k))
        route.norm_backward(norm, e(0, k), e(0, k), None, torch.empty((0, 2), device=DEV),
                            dx=e(0, k), dgamma=dg)
        for p in (lin, gated, norm):
            p.status()
        for t in (dW, db, *ws, dg):
            assert bool((t == 0).all())


@pytest.mark.parametrize("rows", [6, 300])
def test_special_values_stay_in_their_rows(rows):
    """NaN and infinities of a row reach that row's results and no other's."""
    k, f, n = 128, 96, 136
    x = normal(1, rows, k)
    Wg, Wu, Wd = normal(2, k, f), normal(3, k, f), normal(4, f, n)
    clean, dirty = (torch.empty((rows, n), dtype=BF16, device=DEV) for _ in range(2))
    bad = x.clone()
    bad[2, 5] = float("nan")
    bad[4, 0] = float("inf")
    keep = [i for i in range(rows) if i not in (2, 4)]
    with route.GatedPlan(rows, k, f, n, BF16) as plan:
        route.gated_forward(plan, x, Wg, Wu, Wd, clean)
        route.gated_forward(plan, bad, Wg, Wu, Wd, dirty)
        plan.status()
    assert torch.equal(clean[keep], dirty[keep])
    assert bool(torch.isnan(dirty[2]).all()) and not bool(torch.isfinite(dirty[4]).any())
    for act in route.ACTIVATIONS:
        with route.LinearPlan(rows, k, n, BF16, act=act) as plan:
            route.linear_forward(plan, bad, Wg[:, :1].repeat(1, n).contiguous(), dirty)
            plan.status()
        assert bool(torch.isnan(dirty[2]).all()) and bool(torch.isfinite(dirty[keep]).all()), act


def test_other_stream_and_graph_replay():
    rows, k, f, n = 70, 320, 192, 320
    x = normal(1, rows, k)
    w = normal(2, k, f, scale=0.05), normal(3, k, f, scale=0.05), normal(4, f, n, scale=0.05)
    want, got = (torch.empty((rows, n), dtype=BF16, device=DEV) for _ in range(2))
    y = torch.empty_like(x)
    with route.GatedPlan(rows, k, f, n, BF16) as plan, route.NormPlan(rows, k, BF16) as norm:
        def step(out):
            route.norm_forward(norm, x, None, None, y)
            route.gated_forward(plan, y, *w, out, residual=x)
        step(want)
        torch.cuda.synchronize()
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            step(got)
        s.synchronize()
        assert torch.equal(want, got)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            step(got)
        for seed in (11, 12):
            x.copy_(normal(seed, rows, k))
            step(want)
            got.fill_(float("nan"))
            graph.replay()
            torch.cuda.synchronize()
            assert torch.equal(want, got)
        plan.status()


def test_stalled_product_reports_a_timeout_and_recovers():
    rows, k, n = 300, 512, 512
    x, W = normal(1, rows, k), normal(2, k, n)
    out, want = (torch.empty((rows, n), dtype=BF16, device=DEV) for _ in range(2))
    with route.LinearPlan(rows, k, n, BF16) as plan:
        route.linear_forward(plan, x, W, want)
        plan.status()
        assert route.lib().route_layer_test_stall(plan.handle, 1, 2_000_000) == 0
        route.linear_forward(plan, x, W, out)
        with pytest.raises(route.RouteError, match="TIMEOUT"):
            plan.status()
        assert route.lib().route_layer_test_stall(plan.handle, 0, 0) == 0
        route.linear_forward(plan, x, W, out)
        plan.status()
        assert torch.equal(out, want)


def test_refusals_of_tensors():
    k, n = 64, 32
    x, W = normal(1, 4, k), normal(2, k, n)
    out = torch.empty((4, n), dtype=BF16, device=DEV)
    with route.LinearPlan(4, k, n, BF16) as plan:
        with pytest.raises(TypeError, match="dtype"):
            route.linear_forward(plan, x.half(), W, out)
        with pytest.raises(ValueError, match="shape"):
            route.linear_forward(plan, x, W.t(), out)
        with pytest.raises(ValueError, match="unit stride"):
            route.linear_forward(plan, x, normal(2, n, k).t(), out)
        with pytest.raises(ValueError, match="cuda:0"):
            route.linear_forward(plan, x.cpu(), W, out)
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ROWS"):
            route.linear_forward(plan, normal(1, 5, k), W, torch.empty((5, n), dtype=BF16, device=DEV))
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ALIGN"):
            route.linear_forward(plan, normal(1, 4, k, ld=k + 1), W, out)
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ALIGN"):
            route.linear_forward(plan, normal(1, 4, k, ld=k, offset=1), W, out)
        with pytest.raises(route.RouteError, match="without train"):
            route.linear_backward(plan, out, x, W, dx=torch.empty_like(x))
        with pytest.raises(route.RouteError, match="ROUTE_ERR_PLAN"):
            route.linear_forward(plan, x[:1].expand(4, k), W, out)
    with route.LinearPlan(4, k, n, BF16, act="gelu", train=True) as plan:
        with pytest.raises(ValueError, match="saved holds"):
            route.linear_forward(plan, x, W, out, saved=torch.empty((8,), dtype=torch.uint8, device=DEV))
        with pytest.raises(route.RouteError, match="ROUTE_ERR_NULL"):
            route.linear_backward(plan, out, x, W, dx=torch.empty_like(x))
    with pytest.raises(route.RouteError, match="closed"):
        route.linear_forward(plan, x, W, out)


# ---- the ways products are cut ----------------------------------------------------

def _random_shapes(seed, count, odd):
    import random
    r = random.Random(seed)

    def width():
        w = int(2 ** r.uniform(2, 10.4))
        return (w | 1) if odd else max(8, w // 8 * 8)
    return [(int(2 ** r.uniform(0, 11)), width(), width(), width()) for _ in range(count)]


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_linear_over_many_shapes(dt, odd):
    """Shapes over the ranges where tile, split and launch choices change."""
    for i, (rows, k, n, _) in enumerate(_random_shapes(3 + odd, 24, odd)):
        act = route.ACTIVATIONS[i % len(route.ACTIVATIONS)]
        x, W = normal(i, rows, k, dt=dt), normal(i + 1, k, n, scale=k ** -0.5, dt=dt)
        b, res, dout = normal(i + 2, n, dt=dt), normal(i + 3, rows, n, dt=dt), normal(i + 4, rows, n, dt=dt)
        with route.LinearPlan(rows, k, n, dt, act=act, train=True) as plan:
            saved = plan.new_saved()
            out, g0 = blank(rows, n, dt)
            dx, g1 = blank(rows, k, dt)
            dW, g2 = blank(k, n, dt)
            db = torch.full((n,), float("nan"), dtype=dt, device=DEV)
            route.linear_forward(plan, x, W, out, bias=b, residual=res, saved=saved)
            route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW, dbias=db)
            plan.status()
        want, z = ref.linear(x, W, b, res, act, dt)
        grads = ref.linear_grads(x, W, z, dout, act, dt)
        for name, got, w in (("out", out, want), ("dx", dx, grads["dx"]), ("dW", dW, grads["dW"]),
                             ("dbias", db, grads["dbias"])):
            check(f"{name} of {rows}x{k}x{n} {act}", got, w)
        for g in (g0, g1, g2):
            g()


@pytest.mark.parametrize("odd", [False, True])
def test_gated_over_many_shapes(odd):
    dt = BF16
    for i, (rows, k, f, n) in enumerate(_random_shapes(7 + odd, 16, odd)):
        act = route.ACTIVATIONS[i % len(route.ACTIVATIONS)]
        x = normal(i, rows, k, dt=dt)
        Wg, Wu = (normal(i + j, k, f, scale=k ** -0.5, dt=dt) for j in (1, 2))
        Wd, dout = normal(i + 3, f, n, scale=f ** -0.5, dt=dt), normal(i + 4, rows, n, dt=dt)
        with route.GatedPlan(rows, k, f, n, dt, act=act, train=True) as plan:
            saved = plan.new_saved()
            out, g0 = blank(rows, n, dt)
            outs = {"dx": blank(rows, k, dt), "dW_gate": blank(k, f, dt), "dW_up": blank(k, f, dt),
                    "dW_down": blank(f, n, dt)}
            route.gated_forward(plan, x, Wg, Wu, Wd, out, saved=saved)
            route.gated_backward(plan, dout, x, Wg, Wu, Wd, saved, **{m: v[0] for m, v in outs.items()})
            plan.status()
        want, kept = ref.gated(x, Wg, Wu, Wd, None, act, dt)
        check(f"out of {rows}x{k}x{f}x{n} {act}", out, want)
        grads = ref.gated_grads(x, Wg, Wu, Wd, kept, dout, act, dt)
        for m, (got, guard) in outs.items():
            check(f"{m} of {rows}x{k}x{f}x{n} {act}", got, grads[m])
            guard()
        g0()


def test_fewer_rows_than_the_plan_and_choices_by_row_count():
    """One plan, calls of many row counts in turn: each as on its own plan."""
    k, n, dt = 264, 520, BF16
    W = normal(1, k, n, scale=k ** -0.5)
    with route.LinearPlan(3000, k, n, dt, act="silu", train=True) as plan:
        for rows in (3000, 1, 700, 17, 3000, 129, 1):
            x, dout = normal(rows, rows, k), normal(rows + 1, rows, n)
            outs = []
            for p in (plan, route.LinearPlan(rows, k, n, dt, act="silu", train=True)):
                saved = p.new_saved(rows)
                o = [torch.full(s, float("nan"), dtype=dt, device=DEV) for s in ((rows, n), (rows, k), (k, n))]
                route.linear_forward(p, x, W, o[0], saved=saved)
                route.linear_backward(p, dout, x, W, saved=saved, dx=o[1], dW=o[2])
                p.status()
                outs.append(o)
            assert all(torch.equal(a, b) for a, b in zip(*outs))


def test_results_do_not_depend_on_what_else_is_asked_for_or_ran():
    """Bits of each gradient alone and with the others, and of repeated calls."""
    for rows, k, n in ((6, 896, 448), (300, 200, 1032), (2050, 128, 904), (5000, 72, 40)):
        x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
        dout = normal(3, rows, n)
        with route.LinearPlan(rows, k, n, BF16, train=True) as plan:
            dx, dW = torch.empty_like(x), torch.empty_like(W)
            route.linear_backward(plan, dout, x, W, dx=dx, dW=dW)
            for _ in range(2):
                a, b = torch.empty_like(x), torch.empty_like(W)
                route.linear_backward(plan, dout, None, W, dx=a)
                route.linear_backward(plan, dout, x, None, dW=b)
                plan.status()
                assert torch.equal(a, dx) and torch.equal(b, dW)


def test_offsets_past_32_bits():
    """A result of more than 2^31 elements (5.2 GB): its last rows."""
    rows, k, n = 65536, 64, 40000
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    out = torch.full((rows, n), float("nan"), dtype=BF16, device=DEV)
    with route.LinearPlan(rows, k, n, BF16) as plan:
        route.linear_forward(plan, x, W, out)
        plan.status()
    for at in (0, 53686, rows - 40):
        want, _ = ref.linear(x[at:at + 40], W, None, None, "none", BF16)
        check(f"rows {at}", out[at:at + 40], want)
    assert not bool(torch.isnan(out[:, ::4999]).any())


def test_operands_that_share_memory():
    """The same tensor as two weights, and weights that start at one address
    with other shapes."""
    rows, k = 40, 128
    x, W = normal(1, rows, k), normal(2, k, k, scale=k ** -0.5)
    out = torch.empty((rows, k), dtype=BF16, device=DEV)
    with route.GatedPlan(rows, k, k, k, BF16, train=True) as plan:
        saved = plan.new_saved()
        route.gated_forward(plan, x, W, W, W, out, saved=saved)
        dx = torch.empty_like(x)
        dW = [torch.empty_like(W) for _ in range(3)]
        route.gated_backward(plan, x, x, W, W, W, saved, dx=dx, dW_gate=dW[0], dW_up=dW[1], dW_down=dW[2])
        plan.status()
    want, kept = ref.gated(x, W, W, W, None, "silu", BF16)
    check("out", out, want)
    grads = ref.gated_grads(x, W, W, W, kept, x, "silu", BF16)
    for got, name in zip((dx, *dW), ("dx", "dW_gate", "dW_up", "dW_down")):
        check(name, got, grads[name])
    # W_gate [128, 64] and W_down [64, 128] are views of one buffer's start
    f = 64
    buf = normal(5, k * k, 1, scale=k ** -0.5).view(-1)
    Wg, Wd = buf[:k * f].view(k, f), buf[:f * k].view(f, k)
    Wu = normal(6, k, f, scale=k ** -0.5)
    with route.GatedPlan(rows, k, f, k, BF16, train=True) as plan:
        saved = plan.new_saved()
        route.gated_forward(plan, x, Wg, Wu, Wd, out, saved=saved)
        route.gated_backward(plan, x, x, Wg, Wu, Wd, saved, dx=dx)
        plan.status()
    want, kept = ref.gated(x, Wg, Wu, Wd, None, "silu", BF16)
    check("out", out, want)
    check("dx", dx, ref.gated_grads(x, Wg, Wu, Wd, kept, x, "silu", BF16)["dx"])


@pytest.mark.parametrize("rows,dim,dt", [(70, 200, BF16), (70, 201, FP32)])
def test_norm_gradients_against_differences(rows, dim, dt):
    """The kernels' gradients in a direction against central differences of
    the FP64 loss: the differences' own error is h^2 of third derivatives
    (h = 1e-4: under 1e-6 of the sum of magnitudes), the gradients' that of
    their elements' rounding, 2^-8 or 2^-20 of each."""
    x, dy = normal(1, rows, dim, dt=dt), normal(2, rows, dim, dt=dt)
    gamma, beta = normal(3, dim, dt=dt), normal(4, dim, dt=dt)
    y, dx = torch.empty_like(x), torch.empty_like(x)
    stats = torch.empty((rows, 2), device=DEV)
    dg, db = torch.empty_like(gamma), torch.empty_like(beta)
    with route.NormPlan(rows, dim, dt) as plan:
        route.norm_forward(plan, x, gamma, beta, y, stats=stats)
        route.norm_backward(plan, dy, x, gamma, stats, dx=dx, dgamma=dg, dbeta=db)
        plan.status()

    def loss(x, g, b):
        d = x - x.mean(1, keepdim=True)
        return float((dy.double() * (d * (d.square().mean(1, keepdim=True) + 1e-5) ** -0.5 * g + b)).sum())

    p = [x.double(), gamma.double(), beta.double()]
    rel = {BF16: 2.0 ** -8, FP32: 2.0 ** -20}[dt]
    for i, grad in enumerate((dx, dg, db)):
        v = normal(9 + i, *p[i].shape, dt=FP32).double()
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-4 * v, p[i] - 1e-4 * v
        diff = (loss(*hi) - loss(*lo)) / 2e-4
        got = grad.double() * v
        assert abs(diff - float(got.sum())) <= (rel + 1e-6) * float(got.abs().sum()) + 1e-6


# ---- rows of the result at every alignment, in the products' large tiles ---------

@pytest.mark.parametrize("dt,act", [(BF16, "none"), (FP16, "silu")])
@pytest.mark.parametrize("k", [72, 1608])  # a short contraction, and one past every rule on lengths
@pytest.mark.parametrize("pad,offset", [(0, 0), (8, 8), (4, 4), (1, 3)])
def test_large_tiles_with_rows_of_any_alignment(dt, act, k, pad, offset):
    rows, n = 1097, 3528  # no tile's multiples
    x, W = normal(61, rows, k, dt=dt), normal(62, k, n, scale=k ** -0.5, dt=dt)
    b = normal(63, 1, n, dt=dt, ld=n, offset=offset)[0]
    res = normal(64, rows, n, dt=dt, ld=n + pad, offset=offset)
    with route.LinearPlan(rows, k, n, dt, act=act) as plan:
        for residual in (None, res):
            out, guard = blank(rows, n, dt, ld=n + pad, offset=offset)
            route.linear_forward(plan, x, W, out, bias=b, residual=residual)
            plan.status()
            want, _ = ref.linear(x, W, b, residual, act, dt)
            check("out", out, want)
            guard()
        # in place of the residual
        inplace, guard = blank(rows, n, dt, ld=n + pad, offset=offset)
        inplace.copy_(res)
        route.linear_forward(plan, x, W, inplace, bias=b, residual=inplace)
        plan.status()
        assert torch.equal(inplace, out)
        guard()


@pytest.mark.parametrize("rows", [1, 15, 128, 129, 700, 2300])
@pytest.mark.parametrize("act", ["none", "gelu"])
@pytest.mark.parametrize("offset", [0, 3])
def test_bias_gradient_alone_and_beside_the_products(rows, act, offset):
    # with an offset the rows start at any alignment, and the products copy them
    k, n, dt = 200, 521 if offset else 520, BF16
    x = normal(71, rows, k, dt=dt)
    W = normal(72, k, n, scale=k ** -0.5, dt=dt)
    dout = normal(73, rows, n, dt=dt, ld=n + 2, offset=offset) if offset else normal(73, rows, n, dt=dt)
    with route.LinearPlan(rows, k, n, dt, act=act, train=True) as plan:
        saved = plan.new_saved()
        out = torch.empty(rows, n, dtype=dt, device=DEV)
        route.linear_forward(plan, x, W, out, saved=saved)
        got = []
        for what in ((), ("dx",), ("dx", "dW"), ("dW",), ()):
            dbias = torch.full((n,), float("nan"), dtype=dt, device=DEV)
            bufs = {"dx": torch.empty_like(x), "dW": torch.empty_like(W)}
            route.linear_backward(plan, dout, x, W, saved=saved, dbias=dbias, **{w: bufs[w] for w in what})
            got.append(dbias)
        plan.status()
    z = ref.linear(x, W, None, None, act, dt)[1]
    check("dbias", got[0], ref.linear_grads(x, W, z, dout, act, dt)["dbias"])
    for g in got[1:]:
        assert torch.equal(g, got[0])


def test_calls_by_either_way_are_the_same():
    """The compiled way of a call (taken here) and the checks in Python (taken
    with a stream given) reach the same entry points with the same arguments."""
    rows, k, f, n, dt = 70, 200, 136, 264, BF16
    s = torch.cuda.current_stream()
    x = normal(81, rows, k, dt=dt, ld=k + 8)
    Wg, Wu, Wd = (normal(82 + i, a, b, scale=a ** -0.5, dt=dt) for i, (a, b) in
                  enumerate(((k, f), (k, f), (f, n))))
    W, b, res = normal(85, k, n, scale=k ** -0.5, dt=dt), normal(86, n, dt=dt), normal(87, rows, n, dt=dt)
    dout, dk = normal(88, rows, n, dt=dt), normal(89, rows, k, dt=dt)
    gamma = torch.nn.Parameter(normal(90, k, dt=dt))  # a subclass, and one that autograd watches
    got = []
    with route.NormPlan(rows, k, dt) as np, route.LinearPlan(rows, k, n, dt, act="gelu", train=True) as lp, \
            route.GatedPlan(rows, k, f, n, dt, train=True) as gp:
        for stream in (None, s, s.cuda_stream):
            e = lambda *shape, d=dt: torch.full(shape, float("nan"), dtype=d, device=DEV)  # noqa: E731
            o = [e(rows, k), e(rows, 2, d=FP32), e(rows, k), e(k), e(k), e(rows, n), e(rows, k), e(k, n), e(n),
                 e(rows, n), e(rows, k), e(k, f), e(k, f), e(f, n)]
            ls, gs = lp.new_saved(), gp.new_saved()
            route.norm_forward(np, x, gamma, None, o[0], stats=o[1], eps=0.5, stream=stream)
            route.norm_backward(np, dk, x, gamma, o[1], dx=o[2], dgamma=o[3], dbeta=o[4], stream=stream)
            route.linear_forward(lp, x, W, o[5], bias=b, residual=res, saved=ls, stream=stream)
            route.linear_backward(lp, dout, x, W, saved=ls, dx=o[6], dW=o[7], dbias=o[8], stream=stream)
            route.gated_forward(gp, x, Wg, Wu, Wd, o[9], residual=res, saved=gs, stream=stream)
            route.gated_backward(gp, dout, x, Wg, Wu, Wd, gs, dx=o[10], dW_gate=o[11], dW_up=o[12],
                                 dW_down=o[13], stream=stream)
            for p in (np, lp, gp):
                p.status()
            got.append(o)
        # an integer eps goes through the checks
        y = torch.empty_like(got[0][0])
        route.norm_forward(np, x, gamma, None, y, eps=0)
        z = torch.empty_like(y)
        route.norm_forward(np, x, gamma, None, z, eps=0.0)
        assert torch.equal(y, z)
    for others in got[1:]:
        for a, c in zip(got[0], others):
            assert not bool(torch.isnan(a).any()) and torch.equal(a, c)
    with pytest.raises(route.RouteError):
        route.norm_forward(np, x, gamma, None, y)  # closed


@pytest.mark.parametrize("dt,act", [(BF16, "none"), (FP16, "gelu")])
@pytest.mark.parametrize("pad,offset", [(0, 0), (0, 1), (1, 1), (2, 3), (4, 2)])
@pytest.mark.parametrize("rows,n", [(1097, 3527), (1281, 3529), (2050, 449)])
def test_large_tiles_of_odd_rows(rows, n, dt, act, pad, offset):
    """No residual, an aligned bias: rows of the result at every alignment, and
    the gradients dx and dW of odd widths."""
    k = 73
    x, W = normal(91, rows, k, dt=dt), normal(92, k, n, scale=k ** -0.5, dt=dt)
    b, dout = normal(93, n, dt=dt), normal(94, rows, n, dt=dt)
    with route.LinearPlan(rows, k, n, dt, act=act, train=True) as plan:
        out, guard = blank(rows, n, dt, ld=n + pad, offset=offset)
        route.linear_forward(plan, x, W, out, bias=b)
        saved = plan.new_saved()
        kept = torch.empty(rows, n, dtype=dt, device=DEV)
        route.linear_forward(plan, x, W, kept, bias=b, saved=saved)
        dx, guard_dx = blank(rows, k, dt, ld=k + pad, offset=offset)
        dW, guard_dW = blank(k, n, dt, ld=n + pad, offset=offset)
        route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW)
        plan.status()
    want, z = ref.linear(x, W, b, None, act, dt)
    check("out", out, want)
    assert torch.equal(kept, out)
    grads = ref.linear_grads(x, W, z, dout, act, dt)
    check("dx", dx, grads["dx"])
    check("dW", dW, grads["dW"])
    for g in (guard, guard_dx, guard_dW):
        g()
