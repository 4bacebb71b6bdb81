"""Accuracy of the layer operators where a step of the arithmetic could lose it:
rows far from zero, and activations' tails.  Tolerances are the FP32 steps of
the formulas, not of a rearrangement of them."""

import pytest
import torch

import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, FP16, FP32 = torch.bfloat16, torch.float16, torch.float32
U = 2.0 ** -24  # FP32's unit roundoff


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def normal(seed, *shape, scale=1.0, dt=FP32):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)


@pytest.mark.parametrize("dim", [1024, 1001, 96, 4096, 9000])
@pytest.mark.parametrize("offset", [0.3, 10.0, 100.0, 4096.0])
@pytest.mark.parametrize("dt", [FP32, FP16])
def test_norm_gradients_of_rows_far_from_zero(dim, offset, dt):
    """xh = (x - mean) rstd, with the statistics given, is within 2 U of its own
    size (one rounding each), whatever the row's offset and alignment."""
    rows = 64
    x = (normal(1, rows, dim) + offset).to(dt)
    dy, gamma = normal(2, rows, dim, dt=dt), (1 + 0.3 * normal(3, dim)).to(dt)
    v = x.double()
    stats = torch.stack([v.mean(1), (v.var(1, unbiased=False) + 1e-5) ** -0.5], 1).float().contiguous()
    dx, dgamma, dbeta = torch.empty_like(x), torch.empty_like(gamma), torch.empty_like(gamma)
    with route.NormPlan(rows, dim, dt) as plan:
        route.norm_backward(plan, dy, x, gamma, stats, dx=dx, dgamma=dgamma, dbeta=dbeta)
        plan.status()
    m, s = stats[:, :1].double(), stats[:, 1:].double()
    xh = (v - m) * s
    exh = 2.1 * U * xh.abs()
    g, d = dy.double() * gamma.double(), dy.double()
    # a sum of n terms in any order: n U of the sum of magnitudes
    a, ea = g.mean(1, keepdim=True), (dim + 3) * U * g.abs().mean(1, keepdim=True)
    gx = g * xh
    b = gx.mean(1, keepdim=True)
    eb = (dim + 3) * U * gx.abs().mean(1, keepdim=True) + (g.abs() * exh).mean(1, keepdim=True)
    want = s * (g - a - xh * b)
    e = s * (6 * U * (g.abs() + a.abs() + (xh * b).abs()) + ea + xh.abs() * eb + exh * b.abs())
    assert ref.worst(dx, ref.rounded((want, e), dt)) <= 1
    terms = d * xh
    e = (d.abs() * exh + U * terms.abs()).sum(0) + rows * U * terms.abs().sum(0)
    assert ref.worst(dgamma, ref.rounded((terms.sum(0), e), dt)) <= 1
    assert ref.worst(dbeta, ref.rounded((d.sum(0), rows * U * d.abs().sum(0)), dt)) <= 1
