"""The example layer (norm, route step, latent projection, shared expert)
against the float64 forms: a decode batch, a prompt chunk, a training step."""

import os
import sys

import pytest
import torch

import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rows_of(seed, rows, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn((rows, route.K_HIDDEN), generator=g, device=DEV) * scale).bfloat16()


def expert(layer, n, residual):
    return ref.gated(n, layer.W_gate, layer.W_up, layer.W_down, residual, "silu", torch.bfloat16)


@pytest.mark.parametrize("rows", [1, 8, 150])
def test_serving_step(rows):
    """Each call against its float64 form on the inputs that it was given."""
    from shared_expert_layer import SharedExpertLayer
    layer = SharedExpertLayer(rows, expert_width=512)
    x = rows_of(1, rows)
    whole = x.clone()
    layer.step(whole)
    n = layer.normed
    v = x.double()
    want = (v - v.mean(1, keepdim=True)) * (v.var(1, unbiased=False, keepdim=True) + 1e-5) ** -0.5
    assert ref.worst(n, ref.rounded((want, 2.0 ** -18 * (1 + want.abs())), torch.bfloat16)) <= 1
    latent = ref.rounded(ref.matmul(ref.exact(n), ref.exact(layer.W_latent)), torch.bfloat16)
    assert ref.worst(layer.latent, latent) <= 1
    middle = torch.empty_like(x)
    route.linear_forward(layer.out, layer.latent, layer.W_out, middle, residual=x)
    assert ref.worst(middle, ref.linear(layer.latent, layer.W_out, None, x, "none", torch.bfloat16)[0]) <= 1
    assert ref.worst(whole, expert(layer, n, middle)[0]) <= 1
    for plan in (layer.norm, layer.out, layer.expert):
        plan.status()
    route.route_device_status(layer.route)
    layer.close()


def test_training_step():
    from shared_expert_layer import SharedExpertLayer
    rows = 70
    layer = SharedExpertLayer(rows, expert_width=256, train=True)
    x, dy = rows_of(1, rows), rows_of(2, rows, 0.1)
    y, dx, grads = layer.forward_backward(x, dy)
    n = layer.normed
    want, kept = expert(layer, n, x)
    assert ref.worst(y, want) <= 1
    g = ref.gated_grads(n, layer.W_gate, layer.W_up, layer.W_down, kept, dy, "silu", torch.bfloat16)
    for name in ("W_gate", "W_up", "W_down"):
        assert ref.worst(grads[name], g["d" + name]) <= 1, name
    # dbeta is the column sum of the rounded dn: within its rounding and dn's
    # bounds; dx as a whole within a few percent of dy and dn's size
    dn, dn_err = g["dx"]
    sum_err = dn_err.sum(0) + 2.0 ** -20 * dn.abs().sum(0)
    assert ref.worst(grads["beta"], ref.rounded((dn.sum(0), sum_err), torch.bfloat16)) <= 1
    v = x.double().requires_grad_()
    norm = (v - v.mean(1, keepdim=True)) * (v.var(1, unbiased=False, keepdim=True) + 1e-5) ** -0.5
    (norm * dn).sum().backward()
    total = v.grad + dy.double()
    # two roundings to BF16 (dx, then the sum) and dn's: 2^-8 each of what they round
    assert (dx.double() - total).norm() <= 3 * 2.0 ** -8 * (total.norm() + v.grad.norm())
    layer.close()


@pytest.mark.parametrize("producer", ["norm", "norm_grad", "linear", "gated", "input_grad"])
def test_results_feed_an_overlapped_route_step(producer):
    """With route_set_overlap a decode step reads its hidden rows as soon as
    the work before it lets it launch: a layer operator's call must not let
    it before its result is complete."""
    rows, K, dt = 8, route.K_HIDDEN, torch.bfloat16
    x, dy = rows_of(1, 4096), rows_of(2, 4096)
    big, W = rows_of(3, rows), (torch.randn((K, K), device=DEV) * K ** -0.5).to(dt)
    f = 4096
    w = [(torch.randn(s, device=DEV) * s[0] ** -0.5).to(dt) for s in ((K, f), (K, f), (f, K))]
    wl, wr = (torch.randn((K, n), device=DEV).to(dt) * K ** -0.5 for n in (route.N_LATENT, route.N_EXPERTS))
    stats = torch.tensor([[0.0, 1.0]], device=DEV).repeat(4096, 1).contiguous()
    hidden = torch.empty((4096, K), dtype=dt, device=DEV)
    with route.NormPlan(4096, K, dt) as norm, route.LinearPlan(rows, K, K, dt, train=True) as lin, \
            route.GatedPlan(rows, K, f, K, dt) as gated, route.Plan(route.DECODE, rows) as plan:
        def produce():
            if producer == "norm":
                route.norm_forward(norm, x, None, None, hidden)
                return hidden[-rows:]
            if producer == "norm_grad":
                route.norm_backward(norm, dy, x, None, stats, dx=hidden)
                return hidden[-rows:]
            if producer == "linear":
                route.linear_forward(lin, big, W, hidden[:rows])
            elif producer == "gated":
                route.gated_forward(gated, big, *w, hidden[:rows])
            else:
                route.linear_backward(lin, big, None, W, dx=hidden[:rows])
            return hidden[:rows]

        def step(h):
            lat = torch.full((rows, route.N_LATENT), float("nan"), dtype=dt, device=DEV)
            lg = torch.full((rows, route.N_EXPERTS), float("nan"), device=DEV)
            ids = torch.empty((rows, route.TOPK), dtype=torch.int32, device=DEV)
            wt = torch.empty((rows, route.TOPK), device=DEV)
            route.route_step(plan, h, wl, wr, lat, lg, ids, wt)
            return lat, lg, ids, wt

        h = produce()
        torch.cuda.synchronize()
        want = step(h)
        torch.cuda.synchronize()
        route.route_set_overlap(plan, True)
        for _ in range(5):
            hidden.zero_()
            got = step(produce())
            torch.cuda.synchronize()
            assert all(torch.equal(a, b) for a, b in zip(got, want))
        route.route_device_status(plan)
