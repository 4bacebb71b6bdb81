"""The routed experts' operators as they run in programs: again and again with
other kernels behind them, from several threads and streams, in graphs whose
inputs change, and with sizes past 32 bits."""

import threading

import numpy as np
import pytest
import torch

import experts_ref
import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, FP16 = torch.bfloat16, torch.float16
I32 = torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0, dt=BF16):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


def offsets_of(counts):
    return torch.from_numpy(np.concatenate([[0], np.cumsum(counts)])).to(I32).to(DEV)


def nan_like(t):
    return torch.full_like(t, float("nan"))


@pytest.mark.parametrize("k,f,n,most,experts,dt", [
    (256, 128, 264, 70, 300, BF16),    # more experts than pairs of SMs, all with ends inside a block
    (1024, 520, 256, 9, 40, FP16),
    (320, 256, 320, 900, 12, BF16),
    (2048, 1024, 2048, 130, 30, BF16),
])
def test_many_runs_give_the_same_bits(k, f, n, most, experts, dt):
    """What a wait that is missing could break is a bit of some result."""
    rng = np.random.default_rng(k)
    counts = rng.integers(0, most, experts)
    counts[::7] = 0
    o = offsets_of(counts)
    R = int(o[-1])
    x, dout = normal(1, R, k, dt=dt), normal(2, R, n, dt=dt)
    W = (normal(3, experts, k, f, scale=k ** -0.5, dt=dt), normal(4, experts, k, f, scale=k ** -0.5, dt=dt),
         normal(5, experts, f, n, scale=f ** -0.5, dt=dt))
    first = None
    with route.ExpertsPlan(R, k, f, n, experts, dt, train=True) as plan, route.NormPlan(R, k, dt) as norm:
        saved = plan.new_saved()
        y = torch.empty_like(x)
        for _ in range(25):
            got = [nan_like(dout), nan_like(x)] + [nan_like(w) for w in W]
            route.experts_forward(plan, x, o, *W, got[0], saved=saved)
            route.norm_forward(norm, x, None, None, y)
            route.experts_backward(plan, dout, x, o, *W, saved, dx=got[1], dW_gate=got[2], dW_up=got[3],
                                   dW_down=got[4])
            if first is None:
                first = got
            else:
                assert all(torch.equal(a, b) for a, b in zip(first, got))
        plan.status()
    for e in rng.permutation(experts)[:20]:
        lo, hi = int(o[e]), int(o[e + 1])
        if lo == hi:
            assert all(float(g[e].abs().max()) == 0 for g in first[2:])
            continue
        want, kept = ref.gated(x[lo:hi], W[0][e], W[1][e], W[2][e], None, "silu", dt)
        assert ref.worst(first[0][lo:hi], want) <= 1
        g = ref.gated_grads(x[lo:hi], W[0][e], W[1][e], W[2][e], kept, dout[lo:hi], "silu", dt)
        for name, t in (("dx", first[1][lo:hi]), ("dW_gate", first[2][e]), ("dW_up", first[3][e]),
                        ("dW_down", first[4][e])):
            assert ref.worst(t, g[name]) <= 1, name


def test_a_graph_of_the_whole_follows_its_inputs():
    """Sort, gather, experts, combine and dropout captured once: replays with
    other ids, rows and lots, from none of the experts to all rows at one."""
    rows, dim, f, E, topk = 40, 256, 128, 24, 4
    dt = BF16
    W = (normal(3, E, dim, f, scale=dim ** -0.5), normal(4, E, dim, f, scale=dim ** -0.5),
         normal(5, E, f, dim, scale=f ** -0.5))
    x, w, ids = normal(1, rows, dim), torch.rand((rows, topk), device=DEV), torch.zeros((rows, topk), dtype=I32, device=DEV)
    offsets = torch.empty(E + 1, dtype=I32, device=DEV)
    place = torch.empty((rows, topk), dtype=I32, device=DEV)
    xs, ys, out, step = (normal(9, rows * topk, dim), normal(9, rows * topk, dim), torch.empty_like(x),
                         torch.zeros(1, dtype=torch.int64, device=DEV))
    with route.DispatchPlan(rows, dim, dt, experts=E, topk=topk) as d, \
            route.ExpertsPlan(rows * topk, dim, f, dim, E, dt) as e, route.DropoutPlan(rows, dim, dt) as drop:
        def run():
            route.dispatch_sort(d, ids, offsets, place)
            route.dispatch_gather(d, x, place, xs)
            route.experts_forward(e, xs, offsets, *W, ys)
            route.dispatch_combine(d, ys, place, w, out, residual=x)
            route.dropout_forward(drop, out, 0.25, 5, out, step=step)

        s = torch.cuda.Stream()
        s.wait_stream(torch.cuda.current_stream())
        with torch.cuda.stream(s):
            run()
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run()
        rng = np.random.default_rng(2)
        for i, fill in enumerate(("random", "one", "none", "random", "padding")):
            a = rng.integers(0, E, (rows, topk)).astype(np.int32)
            if fill == "one":
                a[:] = 3
            elif fill == "none":
                a[:] = -1
            elif fill == "padding":
                a[::2] = -1
            ids.copy_(torch.from_numpy(a))
            x.copy_(normal(20 + i, rows, dim))
            step.fill_(1000 * i)
            g.replay()
            torch.cuda.synchronize()
            o, p, pairs = experts_ref.sort(a, E, 0)
            assert offsets.tolist() == o.tolist() and (place.cpu().numpy() == p).all()
            for q, (lo, hi) in enumerate(experts_ref.runs_of(o, rows * topk)):
                if lo < hi:
                    assert ref.worst(ys[lo:hi], ref.gated(xs[lo:hi], W[0][q], W[1][q], W[2][q], None, "silu", dt)[0]) <= 1
            mixed = torch.empty_like(x)
            route.dispatch_combine(d, ys, place, w, mixed, residual=x)
            assert ref.worst(mixed, experts_ref.combine(ys, place, w, x, dt)) <= 1
            assert ref.worst(out, experts_ref.dropout(mixed, 0.25, 5, 1000 * i, None, dt)[0]) <= 1
        e.status()


def test_a_training_step_in_a_graph():
    k, f, n, E = 192, 136, 200, 10
    o = offsets_of([0, 5, 70, 64, 0, 130, 1, 0, 33, 16])
    R = int(o[-1])
    x, dout = normal(1, R, k), normal(2, R, n)
    W = normal(3, E, k, f, scale=0.1), normal(4, E, k, f, scale=0.1), normal(5, E, f, n, scale=0.1)
    with route.ExpertsPlan(R, k, f, n, E, BF16, train=True) as plan:
        saved = plan.new_saved()

        def run(out, dx, *g):
            route.experts_forward(plan, x, o, *W, out, saved=saved)
            route.experts_backward(plan, dout, x, o, *W, saved, dx=dx, dW_gate=g[0], dW_up=g[1], dW_down=g[2])

        eager = [nan_like(t) for t in (dout, x, *W)]
        run(*eager)
        graphed = [nan_like(t) for t in (dout, x, *W)]
        torch.cuda.synchronize()
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            run(*graphed)
        for _ in range(3):
            for t in graphed:
                t.fill_(float("nan"))
            g.replay()
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(eager, graphed))
        plan.status()


def test_streams_and_both_ways_of_a_call():
    """By ctypes (a stream is given) and by the compiled way, the same bits; a
    dispatch and a dropout plan on two streams at the same time."""
    rows, dim, topk, E = 700, 520, 4, 16
    x = normal(1, rows, dim)
    ids = torch.randint(-1, E, (rows, topk), device=DEV, dtype=I32)
    w = torch.rand((rows, topk), device=DEV)
    streams = [torch.cuda.Stream() for _ in range(2)]
    with route.DispatchPlan(rows, dim, BF16, experts=E, topk=topk) as d, route.DropoutPlan(rows, dim, BF16) as drop, \
            route.ExpertsPlan(rows * topk, dim, 64, dim, E, BF16) as e:
        W = normal(3, E, dim, 64, scale=0.05), normal(4, E, dim, 64, scale=0.05), normal(5, E, 64, dim, scale=0.1)

        def run(stream):
            offsets, place = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty((rows, topk), dtype=I32, device=DEV)
            source = torch.full((rows * topk,), -7, dtype=I32, device=DEV)
            xs, out = torch.zeros((rows * topk, dim), dtype=BF16, device=DEV), torch.empty_like(x)
            dy, dw = torch.zeros_like(xs), torch.empty_like(w)
            dx, dropped = torch.empty_like(x), torch.empty_like(x)
            route.dispatch_sort(d, ids, offsets, place, source=source, stream=stream)
            route.dispatch_gather(d, x, place, xs, stream=stream)
            route.dispatch_combine(d, xs, place, w, out, residual=x, stream=stream)
            route.dispatch_combine_backward(d, out, xs, place, w, dy=dy, dweights=dw, stream=stream)
            route.dispatch_gather_backward(d, dy, place, dx, stream=stream)
            route.dropout_forward(drop, out, 0.1, 3, dropped, residual=x, stream=stream)
            route.dropout_backward(drop, dropped, 0.1, 3, dx, stream=stream)
            return [offsets, place, source, xs, out, dy, dw, dx, dropped]

        want = run(None)
        torch.cuda.synchronize()
        for stream in (torch.cuda.current_stream(), torch.cuda.current_stream().cuda_stream):
            got = run(stream)
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(want, got))
        for _ in range(10):
            sets = []
            for s in streams:
                s.wait_stream(torch.cuda.current_stream())
                with torch.cuda.stream(s):
                    sets.append(run(None))
            torch.cuda.synchronize()
            for got in sets:
                assert all(torch.equal(a, b) for a, b in zip(want, got))
        outs = [torch.zeros_like(want[3]) for _ in range(2)]
        route.experts_forward(e, want[3], want[0], *W, outs[0])
        route.experts_forward(e, want[3], want[0], *W, outs[1], stream=torch.cuda.current_stream())
        e.status()
        assert torch.equal(*outs)


def test_threads_share_an_experts_plan():
    k, f, n, E, times = 264, 256, 328, 8, 60
    W = normal(1, E, k, f, scale=0.06), normal(2, E, k, f, scale=0.06), normal(3, E, f, n, scale=0.06)
    jobs, errors = [], []
    stream = torch.cuda.current_stream()
    with route.ExpertsPlan(3000, k, f, n, E, BF16, train=True) as plan:
        for rows in (8, 3000, 100, 700):
            o = offsets_of([rows // E] * E)
            R = int(o[-1])
            x, dout = normal(rows, R, k), normal(rows + 1, R, n)

            def step(out, dx, dWd, saved, x=x, dout=dout, o=o):
                route.experts_forward(plan, x, o, *W, out, saved=saved)
                route.experts_backward(plan, dout, x, o, *W, saved, dx=dx, dW_down=dWd)

            sets = [[nan_like(dout), nan_like(x), nan_like(W[2])] for _ in range(2)]
            saved = [plan.new_saved(R) for _ in range(2)]
            step(*sets[0], saved[0])
            jobs.append((step, sets, saved))
        torch.cuda.synchronize()

        def work(step, out, saved):
            try:
                with torch.cuda.stream(stream):
                    for _ in range(times):
                        step(*out, saved)
            except Exception as e:  # shown by the assertion below
                errors.append(e)

        threads = [threading.Thread(target=work, args=(step, sets[1], saved[1])) for step, sets, saved in jobs]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        plan.status()
        assert not errors
        for _, sets, _ in jobs:
            assert all(torch.equal(a, b) for a, b in zip(*sets))


def test_moves_past_32_bits():
    """More than 2^31 values of the experts' rows."""
    rows, dim, topk = 65536, 2112, 16
    place = torch.arange(rows * topk, dtype=I32, device=DEV).view(rows, topk)
    x = normal(1, rows, dim)
    w = torch.zeros((rows, topk), device=DEV)
    w[:, -1] = 1
    with route.DispatchPlan(rows, dim, BF16, experts=4, topk=topk) as plan:
        xs = torch.zeros((rows * topk, dim), dtype=BF16, device=DEV)
        assert xs.numel() > 2 ** 31
        route.dispatch_gather(plan, x, place, xs)
        for r in (0, 1, 63550, 65535):
            assert torch.equal(xs[r * topk:(r + 1) * topk], x[r:r + 1].expand(topk, dim))
        out = torch.empty_like(x)
        route.dispatch_combine(plan, xs, place, w, out)
        assert torch.equal(out, x)
        dw = torch.empty_like(w)
        route.dispatch_combine_backward(plan, x, xs, place, w, dy=xs, dweights=None)
        route.dispatch_combine_backward(plan, x, xs, place, w, dweights=dw)
        plan.status()
        assert torch.equal(xs[topk - 1::topk], x) and float(xs[::topk].abs().max()) == 0
        assert float(dw[:, :-1].abs().max()) == 0


def test_experts_past_32_bits():
    R, k, f, n, E = 640000, 3584, 64, 3584, 3
    x = torch.zeros((R, k), dtype=BF16, device=DEV)
    o = torch.tensor([0, 10, R - 600, R - 3], dtype=I32, device=DEV)
    tail = normal(1, 700, k)
    x[R - 700:] = tail
    W = normal(3, E, k, f, scale=k ** -0.5), normal(4, E, k, f, scale=k ** -0.5), normal(5, E, f, n, scale=f ** -0.5)
    out = torch.full((R, n), 7.0, dtype=BF16, device=DEV)
    assert out.numel() > 2 ** 31
    with route.ExpertsPlan(R, k, f, n, E, BF16) as plan:
        route.experts_forward(plan, x, o, *W, out)
        plan.status()
    assert bool((out[R - 3:] == 7).all()) and float(out[:R - 700].abs().max()) == 0
    want = ref.gated(x[R - 600:R - 3], W[0][2], W[1][2], W[2][2], None, "silu", BF16)[0]
    assert ref.worst(out[R - 600:R - 3], want) <= 1
    want = ref.gated(x[R - 700:R - 600], W[0][1], W[1][1], W[2][1], None, "silu", BF16)[0]
    assert ref.worst(out[R - 700:R - 600], want) <= 1


def test_many_experts_and_places():
    """The most experts and ids a row."""
    rows, E, topk, k = 50, 1024, 32, 64
    ids = torch.rand((rows, E), device=DEV).topk(topk, dim=1).indices.to(I32)
    x, w = normal(1, rows, k), torch.rand((rows, topk), device=DEV)
    W = normal(3, E, k, 64, scale=0.1), normal(4, E, k, 64, scale=0.1), normal(5, E, 64, k, scale=0.1)
    offsets, place = torch.empty(E + 1, dtype=I32, device=DEV), torch.empty((rows, topk), dtype=I32, device=DEV)
    xs = torch.empty((rows * topk, k), dtype=BF16, device=DEV)
    ys, out = nan_like(xs), nan_like(x)
    with route.DispatchPlan(rows, k, BF16, experts=E, topk=topk) as d, \
            route.ExpertsPlan(rows * topk, k, 64, k, E, BF16) as e:
        route.dispatch_sort(d, ids, offsets, place)
        route.dispatch_gather(d, x, place, xs)
        route.experts_forward(e, xs, offsets, *W, ys)
        route.dispatch_combine(d, ys, place, w, out)
        e.status()
    r = torch.arange(rows, device=DEV)[:, None].expand(rows, topk)
    t, q = x[r].double(), ids.long()
    gate = torch.einsum("rjk,rjkf->rjf", t, W[0][q].double())
    up = torch.einsum("rjk,rjkf->rjf", t, W[1][q].double())
    y = torch.einsum("rjf,rjfn->rjn", torch.nn.functional.silu(gate) * up, W[2][q].double())
    want = (y * w[..., None].double()).sum(1)
    # h, the results and their sum are rounded, half a step of BF16 each
    assert float((out.double() - want).norm() / want.norm()) <= 3 * 2.0 ** -8
