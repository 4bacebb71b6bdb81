"""The routed experts' operators and dropout on a GPU against their plain forms
(experts_ref.py, layer_ref.py): whole numbers equal, every other value within
the bound that the kernels' arithmetic gives."""

import numpy as np
import pytest
import torch

import experts_ref
import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0, dt=BF16, ld=None, offset=0):
    """A seeded matrix; with `ld` a view with that row stride, `offset` into its buffer."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    v = (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)
    if ld is None:
        return v
    buf = torch.full((shape[0] * ld + offset,), float("nan"), dtype=dt, device=DEV)
    view = buf[offset:].view(shape[0], ld)[:, :shape[1]]
    view.copy_(v)
    return view


def sevens(rows, cols, dt=BF16, ld=None, offset=0):
    """An output full of sevens, and the buffer around it."""
    ld = cols if ld is None else ld
    buf = torch.full((rows * ld + offset + 16,), 7.0, dtype=dt, device=DEV)
    return buf[offset:offset + rows * ld].view(rows, ld)[:, :cols], buf


def written(view, buf, rows):
    """Nothing but `rows` (a slice) of the view was written in its buffer."""
    rest = buf.clone()
    lo = (view.data_ptr() - buf.data_ptr()) // buf.element_size()
    sub = rest[lo:lo + view.shape[0] * view.stride(0)].view(view.shape[0], view.stride(0)) \
        if view.shape[0] else rest[:0].view(0, 1)
    sub[rows, :view.shape[1]] = 7
    assert bool((rest == 7).all()), "written outside the output"


def check(name, got, want, limit=1.0):
    w = ref.worst(got, want)
    assert w <= limit, f"{name}: {w:.3g} times the bound"


def some_ids(seed, rows, topk, total, repeat=False):
    rng = np.random.default_rng(seed)
    if repeat:
        return rng.integers(0, total, (rows, topk)).astype(np.int32)
    return np.stack([rng.permutation(total)[:topk] for _ in range(rows)]).astype(np.int32) \
        if rows else np.zeros((0, topk), np.int32)


def to_gpu(a):
    return torch.from_numpy(np.ascontiguousarray(a)).to(DEV)


# ---- sort -----------------------------------------------------------------------

SORT = [
    # rows, topk, total, experts, first, what
    (0, 16, 896, 896, 0, "plain"),
    (1, 1, 1, 1, 0, "plain"),
    (1, 16, 896, 896, 0, "plain"),
    (8, 16, 896, 112, 224, "plain"),
    (20, 16, 896, 896, 0, "plain"),
    (33, 2, 8, 8, 0, "plain"),
    (300, 6, 64, 64, 0, "padding"),
    (1000, 32, 1024, 1024, 0, "plain"),
    (2049, 4, 64, 16, 48, "plain"),
    (4096, 16, 896, 896, 0, "plain"),
    (5000, 3, 5, 5, 0, "repeat"),
    (777, 8, 256, 256, 0, "one"),
    (513, 7, 256, 32, 100, "none"),
    (9001, 31, 1024, 1000, 3, "repeat"),
    (65536, 16, 896, 896, 0, "repeat"),
]


@pytest.mark.parametrize("rows,topk,total,experts,first,what", SORT)
def test_sort(rows, topk, total, experts, first, what):
    ids = some_ids(rows, rows, topk, total, what == "repeat" or rows > 5000)
    if what == "padding":
        ids[::3] = -1
        ids[1, :] = np.array([-2147483648, 2147483647, 64, 63, 0, -1])
    elif what == "one":
        ids[:] = 200
    elif what == "none":
        ids[:] = 5
    wide = torch.full((rows, topk + 3), 1, dtype=I32, device=DEV)
    wide[:, :topk] = to_gpu(ids)
    offsets = torch.full((experts + 1,), -9, dtype=I32, device=DEV)
    place = torch.full((rows, topk), -9, dtype=I32, device=DEV)
    source = torch.full((rows * topk,), -9, dtype=I32, device=DEV)
    with route.DispatchPlan(max(rows, 1), 8, BF16, experts=experts, topk=topk, first=first) as plan:
        route.dispatch_sort(plan, wide[:, :topk], offsets, place, source=source)
        again = torch.empty_like(place)
        route.dispatch_sort(plan, wide[:, :topk].contiguous(), torch.empty_like(offsets), again)
        plan.status()
    o, p, pairs = experts_ref.sort(ids, experts, first)
    assert np.array_equal(offsets.cpu().numpy(), o)
    assert np.array_equal(place.cpu().numpy(), p)
    want = np.full(rows * topk, -9)
    want[:len(pairs)] = pairs
    assert np.array_equal(source.cpu().numpy(), want)
    assert torch.equal(again, place)


# ---- gather and combine -----------------------------------------------------------

MOVES = [
    # rows, dim, topk, total, experts, first, dtype
    (1, 3584, 16, 896, 896, 0, BF16),
    (8, 3584, 16, 896, 112, 224, BF16),
    (5, 1, 2, 8, 8, 0, FP32),
    (37, 333, 4, 64, 32, 32, FP16),
    (64, 1001, 4, 64, 64, 0, FP32),
    (129, 896, 6, 64, 64, 0, FP16),
    (300, 4096, 2, 8, 4, 4, FP32),
    (513, 72, 32, 64, 64, 0, BF16),
    (700, 2056, 8, 256, 64, 64, BF16),
    (20, 7168, 16, 896, 896, 0, BF16),
    (9, 16392, 3, 5, 5, 0, BF16),
]


@pytest.mark.parametrize("rows,dim,topk,total,experts,first,dt", MOVES)
def test_gather_and_combine_with_gradients(rows, dim, topk, total, experts, first, dt):
    ids = some_ids(3, rows, topk, total)
    if rows > 4:
        ids[rows // 2] = -1
    offsets, place, pairs = experts_ref.sort(ids, experts, first)
    n = len(pairs)
    P = rows * topk
    at = to_gpu(place).to(I32)
    w = torch.rand((rows, topk), device=DEV) + 0.1
    w[at < 0] = float("nan")  # weights of nobody's pairs
    x, y = normal(1, rows, dim, dt=dt), normal(2, P, dim, dt=dt)
    y[n:] = float("nan")
    res, dout = normal(4, rows, dim, dt=dt), normal(5, rows, dim, dt=dt)
    with route.DispatchPlan(rows, dim, dt, experts=experts, topk=topk, first=first) as plan:
        xs, buf = sevens(P, dim, dt)
        route.dispatch_gather(plan, x, at, xs)
        assert torch.equal(xs[:n], x[to_gpu(pairs // topk)])
        written(xs, buf, slice(n))
        dx, buf = sevens(rows, dim, dt)
        route.dispatch_gather_backward(plan, y, at, dx)
        check("dx", dx, experts_ref.combine(y, at, None, None, dt))
        written(dx, buf, slice(None))
        for r in (None, res):
            out, buf = sevens(rows, dim, dt)
            route.dispatch_combine(plan, y, at, w, out, residual=r)
            check("out", out, experts_ref.combine(y, at, w, r, dt))
            written(out, buf, slice(None))
        inplace = res.clone()
        route.dispatch_combine(plan, y, at, w, inplace, residual=inplace)
        assert torch.equal(inplace, out)
        dy, buf = sevens(P, dim, dt)
        dw = torch.full((rows, topk), float("nan"), device=DEV)
        route.dispatch_combine_backward(plan, dout, y, at, w, dy=dy, dweights=dw)
        i, want_dy, want_dw = experts_ref.combine_grads(dout, y, at, w, dt, P)
        check("dy", dy[i], want_dy)
        check("dw", dw, want_dw)
        written(dy, buf, slice(n))
        only_dy, only_dw = torch.full_like(dy, 7.0), torch.empty_like(dw)
        route.dispatch_combine_backward(plan, dout, None, at, w, dy=only_dy)
        route.dispatch_combine_backward(plan, dout, y, at, w, dweights=only_dw)
        plan.status()
        assert torch.equal(only_dy, dy) and torch.equal(only_dw, dw)


@pytest.mark.parametrize("dim,dt", [(77, BF16), (80, FP16), (45, FP32), (256, BF16)])
def test_moves_of_strided_views(dim, dt):
    """Any row stride and offset; only what lies in the views is touched."""
    rows, topk, P = 19, 3, 50
    rng = np.random.default_rng(1)
    place = np.full(rows * topk, -1)
    place[:P] = rng.permutation(P)
    at = to_gpu(rng.permutation(place).reshape(rows, topk)).to(I32)
    w = torch.rand((rows, topk), device=DEV)
    x, y = normal(1, rows, dim, dt=dt, ld=dim + 3, offset=1), normal(2, P, dim, dt=dt, ld=dim + 5, offset=3)
    res = normal(3, rows, dim, dt=dt, ld=dim + 1, offset=5)
    with route.DispatchPlan(64, dim, dt, experts=4, topk=topk) as plan:
        xs, b0 = sevens(P, dim, dt, ld=dim + 7, offset=3)
        route.dispatch_gather(plan, x, at, xs)
        r, j = torch.nonzero(at >= 0, as_tuple=True)
        assert torch.equal(xs[at[r, j].long()], x[r])
        written(xs, b0, slice(None))
        out, b1 = sevens(rows, dim, dt, ld=dim + 2, offset=1)
        route.dispatch_combine(plan, y, at, w, out, residual=res)
        check("out", out, experts_ref.combine(y, at, w, res, dt))
        written(out, b1, slice(None))
        dy, b2 = sevens(P, dim, dt, ld=dim + 4, offset=7)
        dw = torch.empty((rows, topk), device=DEV)
        route.dispatch_combine_backward(plan, res, y, at, w, dy=dy, dweights=dw)
        plan.status()
        i, want_dy, want_dw = experts_ref.combine_grads(res, y, at, w, dt, P)
        check("dy", dy[i], want_dy)
        check("dw", dw, want_dw)
        written(dy, b2, slice(None))


@pytest.mark.parametrize("dim", [1, 2, 7, 8, 9, 15, 16, 23, 40, 259, 2051])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_moves_at_every_alignment(dim, dt):
    """Rows that begin anywhere in 16 bytes, tight and apart, NaN around them: what
    is read beside a row counts for nothing, and nothing is written there."""
    rows, topk, P = 9, 2, 16
    rng = np.random.default_rng(dim)
    place = np.full(rows * topk, -1)
    place[:P] = rng.permutation(P)
    at = to_gpu(rng.permutation(place).reshape(rows, topk)).to(I32)
    r, j = torch.nonzero(at >= 0, as_tuple=True)
    w = torch.rand((rows, topk), device=DEV)
    dw, dw_only = torch.empty((2, rows, topk), device=DEV)
    with route.DispatchPlan(rows, dim, dt, experts=4, topk=topk) as plan:
        for o in range(8):
            x = normal(o, rows, dim, dt=dt, ld=dim + o, offset=o)
            y = normal(o + 8, P, dim, dt=dt, ld=dim + (5 * o) % 8, offset=(3 * o + 1) % 8)
            xs, b0 = sevens(P, dim, dt, ld=dim + (o + 4) % 8, offset=(5 * o + 2) % 8)
            route.dispatch_gather(plan, x, at, xs)
            assert torch.equal(xs[at[r, j].long()], x[r])
            written(xs, b0, slice(None))
            out, b1 = sevens(rows, dim, dt, ld=dim + (3 * o) % 8, offset=(7 * o) % 8)
            route.dispatch_combine(plan, y, at, w, out, residual=x)
            check("out", out, experts_ref.combine(y, at, w, x, dt))
            written(out, b1, slice(None))
            dx, b2 = sevens(rows, dim, dt, ld=dim + o // 2, offset=7 - o)
            route.dispatch_gather_backward(plan, y, at, dx)
            check("dx", dx, experts_ref.combine(y, at, None, None, dt))
            written(dx, b2, slice(None))
            dy, b3 = sevens(P, dim, dt, ld=dim + (7 * o + 3) % 8, offset=(o + 5) % 8)
            route.dispatch_combine_backward(plan, x, y, at, w, dy=dy, dweights=dw)
            i, want_dy, want_dw = experts_ref.combine_grads(x, y, at, w, dt, P)
            check("dy", dy[i], want_dy)
            check("dw", dw, want_dw)
            written(dy, b3, slice(None))
            route.dispatch_combine_backward(plan, x, y, at, w, dweights=dw_only)
            check("dw alone", dw_only, want_dw)
            # in place: the residual is the result
            before = out.clone()
            route.dispatch_combine(plan, y, at, w, out, residual=out)
            check("in place", out, experts_ref.combine(y, at, w, before, dt))
            written(out, b1, slice(None))
        plan.status()


def test_places_outside_the_rows_are_none():
    rows, topk, dim, P = 40, 4, 64, 30
    at = torch.randint(-5, 40, (rows, topk), device=DEV, dtype=I32)
    at[0] = torch.tensor([-2147483648, 2147483647, 30, 29], dtype=I32)
    y, w = normal(1, P, dim), torch.rand((rows, topk), device=DEV)
    out, dw = torch.empty((rows, dim), dtype=BF16, device=DEV), torch.empty((rows, topk), device=DEV)
    with route.DispatchPlan(rows, dim, BF16, experts=4, topk=topk) as plan:
        route.dispatch_combine(plan, y, at, w, out)
        check("out", out, experts_ref.combine(y, at, w, None, BF16))
        xs, buf = sevens(P, dim)
        route.dispatch_gather(plan, out, at, xs)
        written(xs, buf, slice(None))
        route.dispatch_combine_backward(plan, out, y, at, w, dy=xs, dweights=dw)
        plan.status()
        check("dw", dw, experts_ref.combine_grads(out, y, at, w, BF16, P)[2])
        written(xs, buf, slice(None))
        # no rows of the experts at all: the residual alone
        route.dispatch_combine(plan, y[:0], at, w, out, residual=out.clone())
        route.dispatch_gather(plan, out, at, y[:0])
        route.dispatch_combine_backward(plan, out, y[:0], at, w, dy=y[:0], dweights=dw)
        plan.status()
        assert float(dw.abs().max()) == 0


# ---- the experts' products --------------------------------------------------------

def sizes(*counts):
    return np.concatenate([[0], np.cumsum(counts)])


EXPERTS = [
    # k, f, n, offsets, rows behind the last, dtype, act
    (64, 64, 64, sizes(1), 0, BF16, "silu"),
    (8, 8, 8, sizes(0, 1, 0, 2), 3, BF16, "silu"),
    (3584, 256, 3584, sizes(1, 0, 2, 0, 0, 1, 4), 40, BF16, "silu"),
    (896, 448, 896, sizes(0, 0, 17, 0, 33, 1), 0, FP16, "gelu"),
    (264, 200, 328, sizes(64, 128, 63, 65, 1, 0), 5, BF16, "gelu_tanh"),
    (512, 640, 512, sizes(256, 257, 255, 0, 31, 32), 0, BF16, "silu"),
    (128, 72, 1000, sizes(513, 0, 700), 100, FP16, "relu"),
    (1000, 1400, 1000, sizes(90, 300, 5), 7, FP16, "gelu"),
    (320, 136, 264, sizes(0, 0, 0), 4, BF16, "silu"),
    (64, 17 * 8, 72, sizes(1030), 0, BF16, "sigmoid"),
    (72, 96, 40, np.array([3, 10, 10, 75]), 2, BF16, "silu"),  # rows before the first, too
]


def stack(seed, E, rows, cols, dt, scale):
    return torch.stack([normal(seed + 100 * e, rows, cols, dt=dt, scale=scale) for e in range(E)])


@pytest.mark.parametrize("k,f,n,offsets,behind,dt,act", EXPERTS)
def test_experts_forward_and_backward(k, f, n, offsets, behind, dt, act):
    E, T = len(offsets) - 1, int(offsets[-1])
    R = T + behind
    x, dout = normal(1, max(R, 1), k, dt=dt), normal(2, max(R, 1), n, dt=dt, scale=0.5)
    for t in (x, dout):  # nobody's rows
        t[T:] = float("nan")
        t[:offsets[0]] = float("inf")
    Wg, Wu = stack(3, E, k, f, dt, k ** -0.5), stack(4, E, k, f, dt, k ** -0.5)
    Wd = stack(5, E, f, n, dt, f ** -0.5)
    o = to_gpu(offsets).to(I32)
    mine = slice(int(offsets[0]), T)
    with route.ExpertsPlan(len(x), k, f, n, E, dt, act=act, train=True) as plan:
        saved = plan.new_saved()
        out, buf = sevens(len(x), n, dt)
        route.experts_forward(plan, x, o, Wg, Wu, Wd, out, saved=saved)
        dx, bufx = sevens(len(x), k, dt)
        grads = [torch.full_like(w, float("nan")) for w in (Wg, Wu, Wd)]
        route.experts_backward(plan, dout, x, o, Wg, Wu, Wd, saved, dx=dx, dW_gate=grads[0],
                               dW_up=grads[1], dW_down=grads[2])
        again = torch.full_like(out, 7.0)
        route.experts_forward(plan, x, o, Wg, Wu, Wd, again)  # inference: the same products
        only = torch.full_like(Wd, float("nan"))
        route.experts_backward(plan, dout, None, o, Wg, Wu, Wd, saved, dW_down=only)
        up = torch.full_like(Wu, float("nan"))
        route.experts_backward(plan, dout, x, o, Wg, Wu, Wd, saved, dW_up=up)
        plan.status()
    assert torch.equal(again, out) and torch.equal(only, grads[2]) and torch.equal(up, grads[1])
    written(out, buf, mine)
    written(dx, bufx, mine)
    for e, (lo, hi) in enumerate(experts_ref.runs_of(offsets, R)):
        if lo == hi:
            assert all(float(g[e].abs().max()) == 0 for g in grads)
            continue
        want, kept = ref.gated(x[lo:hi], Wg[e], Wu[e], Wd[e], None, act, dt)
        check(f"out of {e}", out[lo:hi], want)
        w = ref.gated_grads(x[lo:hi], Wg[e], Wu[e], Wd[e], kept, dout[lo:hi], act, dt)
        for name, got in (("dx", dx[lo:hi]), ("dW_gate", grads[0][e]), ("dW_up", grads[1][e]),
                          ("dW_down", grads[2][e])):
            check(f"{name} of {e}", got, w[name])


def test_experts_keep_infinities_and_nan_to_themselves():
    """An expert whose rows are not finite changes nothing of its neighbours',
    whose last blocks reach into its rows."""
    k, f, n, dt = 128, 64, 136, BF16
    offsets = sizes(30, 40, 70, 1)
    o = to_gpu(offsets).to(I32)
    E, R = 4, int(offsets[-1])
    x, dout = normal(1, R, k, dt=dt), normal(2, R, n, dt=dt)
    W = stack(3, E, k, f, dt, 0.1), stack(4, E, k, f, dt, 0.1), stack(5, E, f, n, dt, 0.1)

    def run(x, dout):
        with route.ExpertsPlan(R, k, f, n, E, dt, train=True) as plan:
            saved, out, dx = plan.new_saved(), torch.empty_like(dout), torch.empty_like(x)
            g = [torch.empty_like(w) for w in W]
            route.experts_forward(plan, x, o, *W, out, saved=saved)
            route.experts_backward(plan, dout, x, o, *W, saved, dx=dx, dW_gate=g[0], dW_up=g[1], dW_down=g[2])
            plan.status()
        return out, dx, g

    clean = run(x, dout)
    bad_x, bad_dout = x.clone(), dout.clone()
    bad_x[30:70], bad_dout[30:70] = float("inf"), float("nan")
    bad = run(bad_x, bad_dout)
    for a, b in zip(clean[:2], bad[:2]):
        assert torch.equal(a[:30], b[:30]) and torch.equal(a[70:], b[70:])
    for a, b in zip(clean[2], bad[2]):
        assert all(torch.equal(a[e], b[e]) for e in (0, 2, 3))
        assert not bool(torch.isfinite(b[1]).any())


def test_experts_strided_operands_and_results():
    """Rows and experts any multiple of 8 apart, experts inside a row too."""
    k, f, n, E, dt = 72, 80, 48, 3, BF16
    offsets = sizes(20, 0, 45)
    o = to_gpu(offsets).to(I32)
    R = 65
    x, dout = normal(1, R, k, dt=dt, ld=k + 8, offset=8), normal(2, R, n, dt=dt, ld=n + 16, offset=24)
    Wg = stack(3, E, k, f, dt, 0.1).transpose(0, 1).contiguous().transpose(0, 1)  # [k][E][f]
    Wu = torch.full((E, k + 1, f + 8), float("nan"), dtype=dt, device=DEV)[:, :k, :f]
    Wu.copy_(stack(4, E, k, f, dt, 0.1))
    Wd = torch.full((2 * E, f, n), float("nan"), dtype=dt, device=DEV)[::2]
    Wd.copy_(stack(5, E, f, n, dt, 0.1))
    out, b0 = sevens(R, n, dt, ld=n + 8, offset=8)
    dx, b1 = sevens(R, k, dt, ld=k + 24, offset=16)
    dWg = torch.full((k, E, f), 7.0, dtype=dt, device=DEV).transpose(0, 1)
    buf = torch.full((E, k + 2, f + 8), 7.0, dtype=dt, device=DEV)
    dWu = buf[:, :k, :f]
    dWd = torch.full((E, f, n), 7.0, dtype=dt, device=DEV)
    with route.ExpertsPlan(100, k, f, n, E, dt, train=True) as plan:
        saved = plan.new_saved(R)
        route.experts_forward(plan, x, o, Wg, Wu, Wd, out, saved=saved)
        route.experts_backward(plan, dout, x, o, Wg, Wu, Wd, saved, dx=dx, dW_gate=dWg, dW_up=dWu, dW_down=dWd)
        plan.status()
    for e, (lo, hi) in enumerate(experts_ref.runs_of(offsets, R)):
        if lo == hi:
            continue
        want, kept = ref.gated(x[lo:hi], Wg[e], Wu[e], Wd[e], None, "silu", dt)
        check("out", out[lo:hi], want)
        w = ref.gated_grads(x[lo:hi], Wg[e], Wu[e], Wd[e], kept, dout[lo:hi], "silu", dt)
        for name, got in (("dx", dx[lo:hi]), ("dW_gate", dWg[e]), ("dW_up", dWu[e]), ("dW_down", dWd[e])):
            check(name, got, w[name])
    written(out, b0, slice(None))
    written(dx, b1, slice(None))
    buf[:, :k, :f] = 7
    assert bool((buf == 7).all())


def test_experts_no_rows():
    k, f, n, E = 64, 48, 40, 3
    e = lambda *s: torch.empty(s, dtype=BF16, device=DEV)  # noqa: E731
    W = e(E, k, f), e(E, k, f), e(E, f, n)
    o = torch.zeros(E + 1, dtype=I32, device=DEV)
    g = [torch.full_like(w, float("nan")) for w in W]
    wide = torch.full((E, k, f + 8), 7.0, dtype=BF16, device=DEV)
    with route.ExpertsPlan(4, k, f, n, E, BF16, train=True) as plan:
        route.experts_forward(plan, e(0, k), o, *W, e(0, n))
        route.experts_backward(plan, e(0, n), e(0, k), o, *W, None, dx=e(0, k), dW_gate=g[0], dW_up=g[1],
                               dW_down=g[2])
        route.experts_backward(plan, e(0, n), e(0, k), o, *W, None, dW_up=wide[:, :, :f])
        plan.status()
    assert all(float(w.abs().max()) == 0 for w in g)
    assert float(wide[:, :, :f].abs().max()) == 0 and bool((wide[:, :, f:] == 7).all())


def test_experts_offsets_that_are_no_runs():
    """Offsets past the rows, negative or descending: cut, nothing outside touched."""
    k, f, n, E, R = 64, 64, 64, 5, 40
    o = torch.tensor([-5, 10, 4, 30, 2147483647, 35], dtype=I32, device=DEV)
    x = normal(1, R, k)
    W = stack(3, E, k, f, BF16, 0.1), stack(4, E, k, f, BF16, 0.1), stack(5, E, f, n, BF16, 0.1)
    out, buf = sevens(R, n)
    with route.ExpertsPlan(R, k, f, n, E, BF16, train=True) as plan:
        saved = plan.new_saved()
        route.experts_forward(plan, x, o, *W, out, saved=saved)
        g = [torch.empty_like(w) for w in W]
        route.experts_backward(plan, x, x, o, *W, saved, dW_gate=g[0], dW_up=g[1], dW_down=g[2])
        plan.status()
    written(out, buf, slice(None))


def test_experts_reports_a_wait_that_expired():
    k, f, n, E = 64, 64, 64, 2
    o = to_gpu(sizes(5, 70)).to(I32)
    x = normal(1, 75, k)
    W = stack(3, E, k, f, BF16, 0.1), stack(4, E, k, f, BF16, 0.1), stack(5, E, f, n, BF16, 0.1)
    out, want = torch.empty((75, n), dtype=BF16, device=DEV), torch.empty((75, n), dtype=BF16, device=DEV)
    L = route.lib()
    with route.ExpertsPlan(75, k, f, n, E, BF16, train=True) as plan:
        saved = plan.new_saved()
        route.experts_forward(plan, x, o, *W, want, saved=saved)
        plan.status()
        L.route_layer_test_stall(plan.handle, 1, 20_000_000)
        route.experts_forward(plan, x, o, *W, out)
        with pytest.raises(route.RouteError, match="TIMEOUT"):
            plan.status()
        g = torch.empty_like(W[2])
        route.experts_backward(plan, x, None, o, *W, saved, dW_down=g)
        with pytest.raises(route.RouteError, match="TIMEOUT"):
            plan.status()
        L.route_layer_test_stall(plan.handle, 0, 0)
        route.experts_forward(plan, x, o, *W, out)
        plan.status()
    assert torch.equal(out, want)


FEW = [
    # k, f, n, offsets, dtype, act: so few tiles that each is split over a cluster
    (64, 64, 128, sizes(1), BF16, "silu"),
    (8, 8, 8, sizes(0, 3, 0), FP16, "relu"),
    (200, 72, 264, sizes(0, 5, 0, 0, 1), BF16, "gelu"),
    (3584, 192, 520, sizes(0, 0, 17, 2), BF16, "silu"),
    (896, 448, 896, sizes(1, 0, 0, 1), FP16, "gelu_tanh"),
    (7168, 64, 128, sizes(32), BF16, "sigmoid"),
    (512, 1024, 72, sizes(*[0] * 1023, 2), BF16, "silu"),
]


@pytest.mark.parametrize("k,f,n,offsets,dt,act", FEW)
def test_experts_of_few_rows_and_tiles(k, f, n, offsets, dt, act):
    E, T = len(offsets) - 1, int(offsets[-1])
    x = normal(1, T + 1, k, dt=dt)
    x[T:] = float("nan")
    W = stack(3, E, k, f, dt, k ** -0.5) if E < 100 else normal(3, E, k, f, dt=dt, scale=k ** -0.5), \
        normal(4, E, k, f, dt=dt, scale=k ** -0.5), normal(5, E, f, n, dt=dt, scale=f ** -0.5)
    o = to_gpu(offsets).to(I32)
    out, buf = sevens(T + 1, n, dt)
    L = route.lib()
    with route.ExpertsPlan(64, k, f, n, E, dt, act=act, train=True) as plan:
        saved = plan.new_saved(T)
        for _ in range(3):
            route.experts_forward(plan, x[:T], o, *W, out[:T], saved=saved)
        dx = torch.empty((T, k), dtype=dt, device=DEV)
        route.experts_backward(plan, out[:T], None, o, *W, saved, dx=dx)  # what it saved
        plan.status()
        L.route_layer_test_stall(plan.handle, 1, 20_000_000)
        again = torch.full_like(out, 7.0)
        route.experts_forward(plan, x[:T], o, *W, again[:T])
        with pytest.raises(route.RouteError, match="TIMEOUT"):
            plan.status()
        L.route_layer_test_stall(plan.handle, 0, 0)
        route.experts_forward(plan, x[:T], o, *W, again[:T])
        plan.status()
    assert torch.equal(again, out)
    written(out, buf, slice(int(offsets[0]), T))
    for e, (lo, hi) in enumerate(experts_ref.runs_of(offsets, T)):
        if lo < hi:
            w = [t[e] for t in W]
            want, kept = ref.gated(x[lo:hi], *w, None, act, dt)
            check(f"out of {e}", out[lo:hi], want)
            check(f"dx of {e}", dx[lo:hi], ref.gated_grads(x[lo:hi], *w, kept, out[lo:hi], act, dt)["dx"])


# ---- dropout ------------------------------------------------------------------------

DROPOUT = [
    # rows, dim, dtype, p, residual
    (1, 7168, BF16, 0.1, True),
    (20, 7168, BF16, 0.1, False),
    (33, 1001, FP32, 0.5, True),
    (7, 1, BF16, 0.2, True),
    (100, 77, FP16, 0.05, True),
    (64, 520, FP16, 0.9, False),
    (3000, 96, BF16, 0.1, True),
    (5, 64, FP32, 0.0, True),
    (5, 72, BF16, 1.0, True),
    (5, 72, BF16, 1e-6, False),
]


@pytest.mark.parametrize("rows,dim,dt,p,residual", DROPOUT)
def test_dropout(rows, dim, dt, p, residual):
    x, dout = normal(1, rows, dim, dt=dt), normal(2, rows, dim, dt=dt)
    res = normal(3, rows, dim, dt=dt) if residual else None
    seed, offset = 0xFEDCBA9876543210, 2 ** 33 + 5
    out, b0 = sevens(rows, dim, dt)
    dx, b1 = sevens(rows, dim, dt)
    with route.DropoutPlan(rows, dim, dt) as plan:
        route.dropout_forward(plan, x, p, seed, out, offset=offset, residual=res)
        route.dropout_backward(plan, dout, p, seed, dx, offset=offset)
        plan.status()
        want, keep = experts_ref.dropout(x, p, seed, offset, res, dt)
        check("out", out, want)
        check("dx", dx, experts_ref.dropout(dout, p, seed, offset, None, dt)[0])
        assert bool((dx[~keep] == 0).all())
        written(out, b0, slice(None))
        written(dx, b1, slice(None))
        # what is dropped is gone, whatever it was; and in place
        bad = torch.where(keep, x, torch.full_like(x, float("nan")))
        route.dropout_forward(plan, bad, p, seed, bad, offset=offset, residual=res)
        assert torch.equal(bad, out)
        if residual:
            over = res.clone()
            route.dropout_forward(plan, x, p, seed, over, offset=offset, residual=over)
            assert torch.equal(over, out)
        plan.status()


@pytest.mark.parametrize("dim", [1, 7, 8, 9, 63, 247, 248, 249, 256, 500])
@pytest.mark.parametrize("dt", [BF16, FP16, FP32])
def test_dropout_at_every_alignment(dim, dt):
    """The lots are the places', wherever rows begin; NaN around them, and nothing
    written there."""
    rows, p, seed = 9, 0.3, 77
    with route.DropoutPlan(rows, dim, dt) as plan:
        for o in range(8):
            x = normal(o, rows, dim, dt=dt, ld=dim + o, offset=o)
            res = normal(o + 8, rows, dim, dt=dt, ld=dim + (5 * o) % 8, offset=(3 * o + 1) % 8)
            out, buf = sevens(rows, dim, dt, ld=dim + (3 * o) % 8, offset=(7 * o) % 8)
            route.dropout_forward(plan, x, p, seed, out, offset=o, residual=res)
            want, keep = experts_ref.dropout(x, p, seed, o, res, dt)
            check("out", out, want)
            written(out, buf, slice(None))
            route.dropout_backward(plan, x, p, seed, out, offset=o)
            check("dx", out, experts_ref.dropout(x, p, seed, o, None, dt)[0])
            written(out, buf, slice(None))
            # in place
            route.dropout_forward(plan, x, p, seed, res, offset=o, residual=res)
            check("in place", res, want)
        plan.status()


def test_dropout_views_rows_and_offsets():
    """Lots go by the place in the matrix, not by strides or the number of rows."""
    rows, dim, dt = 29, 75, BF16
    x = normal(1, rows, dim, dt=dt, ld=dim + 6, offset=3)
    res = normal(2, rows, dim, dt=dt, ld=dim + 1, offset=1)
    out, b0 = sevens(rows, dim, dt, ld=dim + 2, offset=5)
    with route.DropoutPlan(64, dim, dt) as plan:
        route.dropout_forward(plan, x, 0.3, 11, out, residual=res)
        flat = torch.empty((rows, dim), dtype=dt, device=DEV)
        route.dropout_forward(plan, x.contiguous(), 0.3, 11, flat, residual=res.contiguous())
        assert torch.equal(out, flat)
        tail = torch.empty((9, dim), dtype=dt, device=DEV)
        route.dropout_forward(plan, x[20:], 0.3, 11, tail, offset=plan.draws(20), residual=res[20:])
        assert torch.equal(tail, flat[20:])
        step = torch.tensor([plan.draws(20) - 7], dtype=torch.int64, device=DEV)
        route.dropout_forward(plan, x[20:], 0.3, 11, tail.zero_(), offset=7, residual=res[20:], step=step)
        assert torch.equal(tail, flat[20:])
        wrap = torch.empty((2, dim), dtype=dt, device=DEV)
        route.dropout_forward(plan, x[:2], 0.3, 11, wrap, offset=2 ** 64 - 3)
        check("wrap", wrap, experts_ref.dropout(x[:2], 0.3, 11, 2 ** 64 - 3, None, dt)[0])
        route.dropout_forward(plan, x[:0], 0.3, 11, out[:0])
        plan.status()
    written(out, b0, slice(None))


def test_dropout_in_a_replayed_graph_draws_new_lots():
    rows, dim = 16, 640
    x = normal(1, rows, dim)
    out = torch.empty_like(x)
    with route.DropoutPlan(rows, dim, BF16) as plan:
        step = torch.zeros(1, dtype=torch.int64, device=DEV)
        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            route.dropout_forward(plan, x, 0.5, 3, out, step=step)
        torch.cuda.current_stream().wait_stream(s)
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            route.dropout_forward(plan, x, 0.5, 3, out, step=step)
            step += plan.draws()
        for i in range(3):
            g.replay()
            torch.cuda.synchronize()
            check("out", out, experts_ref.dropout(x, 0.5, 3, i * plan.draws(), None, BF16)[0])


# ---- refusals -----------------------------------------------------------------------

def test_calls_refuse():
    e = lambda *s, dt=BF16: torch.empty(s, dtype=dt, device=DEV)  # noqa: E731
    i = lambda *s: torch.zeros(s, dtype=I32, device=DEV)  # noqa: E731
    with route.DispatchPlan(4, 64, BF16, experts=8, topk=2) as plan:
        with pytest.raises(TypeError, match="ids has dtype"):
            route.dispatch_sort(plan, i(4, 2).long(), i(9), i(4, 2))
        with pytest.raises(ValueError, match="offsets has shape"):
            route.dispatch_sort(plan, i(4, 2), i(8), i(4, 2))
        with pytest.raises(ValueError, match="place must be contiguous"):
            route.dispatch_sort(plan, i(4, 2), i(9), i(4, 3)[:, :2])
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ROWS"):
            route.dispatch_sort(plan, i(5, 2), i(9), i(5, 2))
        with pytest.raises(route.RouteError, match="pairs 9"):
            route.dispatch_gather(plan, e(4, 64), i(4, 2), e(9, 64))
        with pytest.raises(route.RouteError, match="row stride"):
            route.dispatch_gather(plan, e(4, 64), i(4, 2), e(64).expand(8, 64))
        with pytest.raises(TypeError, match="weights has dtype"):
            route.dispatch_combine(plan, e(8, 64), i(4, 2), e(4, 2), e(4, 64))
        with pytest.raises(TypeError, match="y must be"):
            route.dispatch_combine_backward(plan, e(4, 64), None, i(4, 2), None, dweights=e(4, 2, dt=FP32))
        with pytest.raises(route.RouteError, match="another operator"):
            route.dropout_forward(plan, e(4, 64), 0.1, 0, e(4, 64))
    with route.ExpertsPlan(8, 64, 32, 64, 2, BF16) as plan:
        W = e(2, 64, 32), e(2, 64, 32), e(2, 32, 64)
        with pytest.raises(route.RouteError, match="without train"):
            route.experts_backward(plan, e(8, 64), e(8, 64), i(3), *W, None, dx=e(8, 64))
        with pytest.raises(route.RouteError, match="16 bytes"):
            route.experts_forward(plan, e(8 * 64 + 1)[1:].view(8, 64), i(3), *W, e(8, 64))
        with pytest.raises(route.RouteError, match="multiple of 8"):
            route.experts_forward(plan, e(8, 64), i(3), e(2, 64, 36)[:, :, :32], W[1], W[2], e(8, 64))
        with pytest.raises(route.RouteError, match="experts' stride"):
            route.experts_forward(plan, e(8, 64), i(3), e(1, 64, 32).expand(2, 64, 32), W[1], W[2], e(8, 64))
        with pytest.raises(ValueError, match="W_down has shape"):
            route.experts_forward(plan, e(8, 64), i(3), W[0], W[1], W[0], e(8, 64))
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ROWS"):
            route.experts_forward(plan, e(9, 64), i(3), *W, e(9, 64))
    with route.DropoutPlan(4, 64, BF16) as plan:
        for p in (-0.1, 1.1, float("nan")):
            with pytest.raises(route.RouteError, match="p must be"):
                route.dropout_forward(plan, e(4, 64), p, 0, e(4, 64))
        with pytest.raises(ValueError, match="64 bits"):
            route.dropout_forward(plan, e(4, 64), 0.1, -1, e(4, 64))
        with pytest.raises(TypeError, match="step has dtype"):
            route.dropout_forward(plan, e(4, 64), 0.1, 1, e(4, 64), step=i(1))
    with pytest.raises(route.RouteError, match="closed"):
        route.dropout_forward(plan, e(4, 64), 0.1, 0, e(4, 64))
