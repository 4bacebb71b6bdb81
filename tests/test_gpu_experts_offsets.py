"""The experts' products with offsets that a sort does not make, in both kernels
(40 rows: CTA pairs; 32 and fewer: clusters): offsets past the rows are cut to
them, descending and overlapping runs reach nothing outside the results."""

import pytest
import torch

import experts_ref
import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32
MOST, LEAST = 2 ** 31 - 1, -2 ** 31
k, f, n = 72, 64, 80


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


class Margins:
    """A result with sevens all around it: 64 before the first value, 24 behind
    every row, 64 behind the last."""

    def __init__(self, *shape):
        *outer, cols = shape
        rows = torch.Size(outer).numel()
        self.buf = torch.full((64 + rows * (cols + 24) + 64,), 7.0, dtype=BF16, device=DEV)
        self.view = self.buf[64:-64].view(*outer, cols + 24)[..., :cols]

    def untouched(self):
        rest = self.buf.clone()
        cols = self.view.shape[-1]
        rest[64:-64].view(-1, cols + 24)[:, :cols] = 7
        return bool((rest == 7).all())


def run(R, offsets):
    """Forward and backward on R rows; the tensors, and the results in their margins."""
    E = len(offsets) - 1
    o = torch.tensor(offsets, dtype=I32, device=DEV)
    x, dout = normal(1, R, k), normal(2, R, n)
    W = normal(3, E, k, f, scale=0.1), normal(4, E, k, f, scale=0.1), normal(5, E, f, n, scale=0.1)
    got = [Margins(*s) for s in ((R, n), (R, k), (E, k, f), (E, k, f), (E, f, n))]
    out, dx, *g = (m.view for m in got)
    with route.ExpertsPlan(R, k, f, n, E, BF16, train=True) as plan:
        guard = torch.full((plan.saved_bytes() + 256,), 7, dtype=torch.uint8, device=DEV)
        saved = guard[:plan.saved_bytes()]
        saved.zero_()  # of rows that are nobody's: finite
        route.experts_forward(plan, x, o, *W, out, saved=saved)
        route.experts_backward(plan, dout, x, o, *W, saved, dx=dx, dW_gate=g[0], dW_up=g[1], dW_down=g[2])
        plan.status()
    assert bool((guard[plan.saved_row * R:] == 7).all())
    assert all(m.untouched() for m in got)
    return x, dout, W, out, dx, g


@pytest.mark.parametrize("R", [1, 24, 32, 40])
def test_offsets_past_the_rows_are_cut(R):
    """Ascending after the cut: runs like any others."""
    a, b = R // 4, R // 2
    offsets = [LEAST, -5, a, a, b, R + 9, MOST]
    x, dout, W, out, dx, g = run(R, offsets)
    for e, (lo, hi) in enumerate(experts_ref.runs_of(offsets, R)):
        if lo == hi:
            assert all(float(t[e].abs().max()) == 0 for t in g)
            continue
        w = [t[e] for t in W]
        want, kept = ref.gated(x[lo:hi], *w, None, "silu", BF16)
        grads = ref.gated_grads(x[lo:hi], *w, kept, dout[lo:hi], "silu", BF16)
        for name, t, v in (("out", out[lo:hi], want), ("dx", dx[lo:hi], grads["dx"]),
                           ("dW_gate", g[0][e], grads["dW_gate"]), ("dW_up", g[1][e], grads["dW_up"]),
                           ("dW_down", g[2][e], grads["dW_down"])):
            assert ref.worst(t, v) <= 1, (name, e)


@pytest.mark.parametrize("R", [3, 24, 40])
@pytest.mark.parametrize("offsets", [
    [-5, 10, 4, 30, MOST, 35],                 # descending, and past both ends
    [0, MOST, 0, MOST, 0, MOST, 0, MOST, 0, MOST],  # all rows five times: more runs than three rows
    [MOST, 20, 10, 5, 0, LEAST],               # descending throughout: no runs
    [2, 24, 1, 23, 0, 22],
])
def test_descending_and_overlapping_runs_stay_inside(R, offsets):
    x, dout, W, out, dx, g = run(R, offsets)
    for e, (lo, hi) in enumerate(experts_ref.runs_of(offsets, R)):
        if lo == hi:
            assert all(float(t[e].abs().max()) == 0 for t in g)
