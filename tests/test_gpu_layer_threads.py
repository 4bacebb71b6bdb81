"""Host threads and the ways of a layer operator's call.  Threads that share a
plan and stream: each call's kernels stay together, and each is cut for its own
number of rows."""

import threading

import pytest
import torch

import latent_projection_top_gb300 as route
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


@pytest.mark.parametrize("by_stream", [True, False])
def test_threads_share_a_plan(by_stream):
    """By ctypes (a stream is given) and by the compiled way."""
    k, f, n, times = 264, 1000, 520, 200
    w = normal(1, k, f, scale=k ** -0.5), normal(2, k, f, scale=k ** -0.5), normal(3, f, n, scale=f ** -0.5)
    stream = torch.cuda.current_stream()
    jobs = []
    with route.GatedPlan(3000, k, f, n, BF16, train=True) as plan:
        for rows in (1, 3000, 17, 700):
            x, dout = normal(rows, rows, k), normal(rows + 1, rows, n)

            def step(out, dx, dWd, saved, x=x, dout=dout):
                s = stream if by_stream else None
                route.gated_forward(plan, x, *w, out, saved=saved, stream=s)
                route.gated_backward(plan, dout, x, *w, saved, dx=dx, dW_down=dWd, stream=s)

            sets = [(torch.full((rows, n), float("nan"), dtype=BF16, device=DEV),
                     torch.full((rows, k), float("nan"), dtype=BF16, device=DEV),
                     torch.full((f, n), float("nan"), dtype=BF16, device=DEV)) for _ in range(2)]
            saved = [plan.new_saved(rows) for _ in range(2)]
            step(*sets[0], saved[0])
            jobs.append((step, sets, saved))
        plan.status()
        torch.cuda.synchronize()
        errors = []

        def work(step, out, saved):
            try:
                with torch.cuda.stream(stream):
                    for _ in range(times):
                        step(*out, saved)
            except Exception as e:  # shown by the assertion below
                errors.append(e)

        threads = [threading.Thread(target=work, args=(step, sets[1], saved[1]))
                   for step, sets, saved in jobs]
        for t in threads:
            t.start()
        for t in threads:
            t.join()
        plan.status()
    assert not errors
    for _, (want, got), _ in jobs:
        assert all(torch.equal(a, b) for a, b in zip(want, got))


@pytest.mark.parametrize("by_stream", [True, False])
def test_first_cuda_call_of_a_thread(by_stream):
    """A host thread needs no CUDA context of its own making before a call."""
    rows, k, n = 40, 264, 520
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    want, got = (torch.empty((rows, n), dtype=BF16, device=DEV) for _ in range(2))
    stream = torch.cuda.current_stream() if by_stream else None
    with route.LinearPlan(rows, k, n, BF16) as plan:
        route.linear_forward(plan, x, W, want)
        t = threading.Thread(target=lambda: route.linear_forward(plan, x, W, got, stream=stream))
        torch.cuda.synchronize()
        t.start()
        t.join()
        plan.status()
    assert torch.equal(want, got)


def test_other_threads_run_during_a_call():
    """While an entry point waits (here one that only sleeps takes its place),
    other Python threads go on."""
    import ctypes
    import time

    from latent_projection_top_gb300 import layer
    short = layer._short_way()
    x = normal(1, 4, 64)
    names = ("norm_forward", "norm_backward", "linear_forward", "linear_backward", "gated_forward",
             "gated_backward")
    address = lambda f: ctypes.cast(f, ctypes.c_void_p).value  # noqa: E731
    ticks, stop = [], threading.Event()

    def tick():
        while not stop.wait(0.005):
            ticks.append(time.perf_counter())

    t = threading.Thread(target=tick)
    t.start()
    try:
        # usleep's only argument is the first one, a plan's handle
        short.bind(*[address(ctypes.CDLL(None).usleep)] * 6)
        start = time.perf_counter()
        assert short.norm_forward((400000, 0, 0, 0, 64, 0, 0, 0), x, None, None, x, None, 1e-5, 0) == 0
        end = time.perf_counter()
    finally:
        short.bind(*(address(getattr(route.lib(), f"route_{n}")) for n in names))
        stop.set()
        t.join()
    assert end - start >= 0.4
    assert sum(start + 0.1 < at < end - 0.1 for at in ticks) >= 5


def test_calls_without_the_compiled_module(monkeypatch):
    from latent_projection_top_gb300 import layer
    rows, k, n = 40, 264, 520
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    want, got = (torch.empty((rows, n), dtype=BF16, device=DEV) for _ in range(2))
    with route.LinearPlan(rows, k, n, BF16) as plan:
        route.linear_forward(plan, x, W, want)
    monkeypatch.setattr(layer, "_short", None)
    monkeypatch.setattr(layer, "_without", True)
    with route.LinearPlan(rows, k, n, BF16) as plan:
        route.linear_forward(plan, x, W, got)
        plan.status()
    assert torch.equal(want, got)
