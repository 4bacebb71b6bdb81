"""Kernels of the layer operators that leave while others start: products whose
blocks read each other's shared memory, again and again with other kernels
right behind them.  What a late access could break is a bit of some result, so
every call's results are compared with the first one's bits, and those with the
float64 forms."""

import pytest
import torch

import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
TIMES = 40


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0, dt=BF16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def outputs(*shapes, dt=BF16):
    return [[torch.full(s, float("nan"), dtype=dt, device=DEV) for s in shapes] for _ in range(TIMES)]


def same(sets):
    for other in sets[1:]:
        assert all(torch.equal(a, b) for a, b in zip(sets[0], other))


@pytest.mark.parametrize("rows,k,n", [
    # few rows and a long contraction: a tile's sums meet over a cluster, and
    # the last tile has columns that do not exist
    (1, 3584, 130), (7, 2048, 200), (20, 7168, 452), (96, 1792, 264),
    # the same a column a thread
    (5, 3584, 129), (64, 1408, 387), (20, 7167, 451),
])
@pytest.mark.parametrize("dt", [BF16, FP16])
def test_linear_columns_that_do_not_exist(rows, k, n, dt):
    x, W = normal(1, rows, k, dt=dt), normal(2, k, n, scale=k ** -0.5, dt=dt)
    dout, b = normal(3, rows, n, dt=dt), normal(4, n, dt=dt)
    outs = outputs((rows, n), (rows, k), (k, n), dt=dt)
    with route.LinearPlan(rows, k, n, dt, act="silu", train=True) as plan, \
            route.NormPlan(rows, k, dt) as norm:
        saved, y = plan.new_saved(), torch.empty_like(x)
        for out, dx, dW in outs:
            route.linear_forward(plan, x, W, out, bias=b, saved=saved)
            route.norm_forward(norm, x, None, None, y)
            route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW)
        plan.status()
    same(outs)
    want, z = ref.linear(x, W, b, None, "silu", dt)
    grads = ref.linear_grads(x, W, z, dout, "silu", dt)
    for got, w in zip(outs[0], (want, grads["dx"], grads["dW"])):
        assert ref.worst(got, w) <= 1


@pytest.mark.parametrize("rows,k,f,n", [(1, 2048, 72, 1032), (20, 3584, 200, 136), (33, 1001, 77, 515)])
def test_gated_columns_that_do_not_exist(rows, k, f, n):
    x = normal(1, rows, k)
    Wg, Wu, Wd = (normal(i, a, b, scale=a ** -0.5) for i, a, b in ((2, k, f), (3, k, f), (4, f, n)))
    dout = normal(5, rows, n)
    outs = outputs((rows, n), (rows, k), (k, f), (k, f), (f, n))
    with route.GatedPlan(rows, k, f, n, BF16, train=True) as plan:
        saved = plan.new_saved()
        for out, dx, dWg, dWu, dWd in outs:
            route.gated_forward(plan, x, Wg, Wu, Wd, out, saved=saved)
            route.gated_backward(plan, dout, x, Wg, Wu, Wd, saved, dx=dx, dW_gate=dWg, dW_up=dWu,
                                 dW_down=dWd)
        plan.status()
    same(outs)
    want, kept = ref.gated(x, Wg, Wu, Wd, None, "silu", BF16)
    grads = ref.gated_grads(x, Wg, Wu, Wd, kept, dout, "silu", BF16)
    for got, w in zip(outs[0], (want, grads["dx"], grads["dW_gate"], grads["dW_up"], grads["dW_down"])):
        assert ref.worst(got, w) <= 1


# ---- tiles of a pair of SMs: the last tiles of each pair, and what starts behind them

@pytest.mark.parametrize("rows,k,n", [
    (2050, 64, 3584),    # tiles whose epilogue is their whole time
    (4096, 896, 2432),   # more tiles than pairs, an odd number of them a pair
    (700, 2048, 1032),   # fewer tiles than pairs
])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_pair_tiles_with_calls_right_behind(rows, k, n, act):
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    dout = normal(3, rows, n)
    outs = outputs((rows, n), (rows, k), (k, n))
    with route.LinearPlan(rows, k, n, BF16, act=act, train=True) as plan, \
            route.NormPlan(rows, k, BF16) as norm:
        saved, y = plan.new_saved(), torch.empty_like(x)
        for out, dx, dW in outs:
            route.linear_forward(plan, x, W, out, saved=saved)
            route.norm_forward(norm, x, None, None, y)
            route.linear_backward(plan, dout, x, W, saved=saved, dx=dx, dW=dW)
        plan.status()
    same(outs)
    want, z = ref.linear(x, W, None, None, act, BF16)
    grads = ref.linear_grads(x, W, z, dout, act, BF16)
    for got, w in zip(outs[0], (want, grads["dx"], grads["dW"])):
        assert ref.worst(got, w) <= 1


@pytest.mark.parametrize("rows,k,n", [
    (300, 512, 512),      # small tiles, one block of the contraction a CTA
    (16, 16384, 256),     # small tiles, more blocks than stages a CTA
    (4096, 512, 2048),    # pair tiles, one or two a pair
    (16384, 192, 2048),   # pair tiles, many a pair
    (139, 3520, 4536),    # pair tiles, split
])
@pytest.mark.parametrize("act", ["none", "silu"])
def test_expired_waits_leave_the_next_call_right(rows, k, n, act):
    """Copies that never come (the hook of test_stalled_product..): every wait
    gives up, the kernels return, and the call after that is right."""
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    dout = normal(3, rows, n)
    e = lambda *s: torch.full(s, float("nan"), dtype=BF16, device=DEV)  # noqa: E731
    with route.LinearPlan(rows, k, n, BF16, act=act, train=True) as plan:
        saved = plan.new_saved()

        def step():
            o = e(rows, n), e(rows, k), e(k, n)
            route.linear_forward(plan, x, W, o[0], saved=saved)
            route.linear_backward(plan, dout, x, W, saved=saved, dx=o[1], dW=o[2])
            return o

        want = step()
        plan.status()
        assert route.lib().route_layer_test_stall(plan.handle, 1, 2_000_000) == 0
        step()
        with pytest.raises(route.RouteError, match="TIMEOUT"):
            plan.status()
        assert route.lib().route_layer_test_stall(plan.handle, 0, 0) == 0
        got = step()
        plan.status()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
