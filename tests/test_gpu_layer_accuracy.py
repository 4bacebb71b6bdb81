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


def every_bf16(least, most):
    """All BF16 values of both signs whose magnitude is in [least, most]."""
    v = torch.arange(0, 1 << 15, device=DEV, dtype=torch.int32).to(torch.int16).view(BF16)
    v = v[(v.float() >= least) & (v.float() <= most)]
    return torch.cat([v, -v])


def activated(act, z, bias=None):
    """act(z) in FP32 of each value: a product with the 64 x 64 identity."""
    n = 64
    rows = (z.numel() + n - 1) // n
    x = torch.zeros(rows * n, device=DEV, dtype=BF16)
    x[:z.numel()] = z
    W, out = torch.eye(n, device=DEV, dtype=BF16), torch.empty((rows, n), device=DEV)
    with route.LinearPlan(rows, n, n, BF16, act=act, out_dtype=FP32) as plan:
        route.linear_forward(plan, x.view(rows, n), W, out, bias=bias)
        plan.status()
    return out.view(-1)[:z.numel()]


@pytest.mark.parametrize("act", route.ACTIVATIONS)
def test_activations_in_fp32(act):
    """Within layer_ref's bound for the activations' own evaluation (z exact)."""
    z = every_bf16(2.0 ** -20, 40.0)
    got = activated(act, z)
    want = ref.rounded(ref.act(act, ref.exact(z))[0], FP32)
    assert ref.worst(got, want) <= 1


def test_gelu_tail():
    """gelu of negative z relative to itself.  The tail's exponent z^2 / 2 has
    three roundings, each of which moves the tail by z^2 / 2 times U; the rest
    (t: 3 U, the polynomial and its fit: 4 U, the exponential: 4 U, products: 3 U)
    is within 16 U."""
    z = every_bf16(2.0 ** -8, 8.0)
    z = z[z < 0]
    v = z.double()
    want = v * torch.erfc(-v / 2 ** 0.5) / 2
    e = (1.5 * v * v + 16) * U * want.abs()
    assert ref.worst(activated("gelu", z), (want, e)) <= 1
