"""The example layer of the routed experts: each call against its float64 form on
the inputs that it was given, and the whole against float64 autograd."""

import os
import sys

import pytest
import torch

import experts_ref
import latent_projection_top_gb300 as route
import layer_ref as ref
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16 = torch.bfloat16
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def rows_of(seed, *shape, scale=1.0):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


def runs(layer):
    return experts_ref.runs_of(layer.offsets.tolist(), layer.sorted.shape[0])


@pytest.mark.parametrize("rows,experts,first", [(1, 896, 0), (8, 896, 0), (8, 112, 448), (150, 112, 0)])
def test_serving_step(rows, experts, first):
    from routed_experts_layer import RoutedExpertsLayer
    layer = RoutedExpertsLayer(rows, experts=experts, first=first)
    x = rows_of(1, rows, route.K_HIDDEN)
    whole = x.clone()
    layer.step(whole)
    offsets, place, pairs = experts_ref.sort(layer.ids.cpu().numpy(), experts, first)
    assert layer.offsets.tolist() == offsets.tolist()
    assert (layer.place.cpu().numpy() == place).all()
    n = len(pairs)
    source = torch.from_numpy(pairs // route.TOPK).to(DEV)
    assert torch.equal(layer.sorted[:n], layer.latent[source])
    for e, (lo, hi) in enumerate(runs(layer)):
        if lo < hi:
            want, _ = ref.gated(layer.sorted[lo:hi], layer.W_gate[e], layer.W_up[e], layer.W_down[e], None,
                                "silu", BF16)
            assert ref.worst(layer.results[lo:hi], want) <= 1, e
    assert ref.worst(layer.mixed, experts_ref.combine(layer.results, layer.place, layer.weights, None, BF16)) <= 1
    assert ref.worst(whole, ref.linear(layer.mixed, layer.W_out, None, x, "none", BF16)[0]) <= 1
    for plan in (layer.norm, layer.dispatch, layer.experts, layer.out):
        plan.status()
    layer.close()


def test_shards_add_up_to_the_layer():
    """The shards' sums of a layer with the same weights: each rounds its part."""
    from routed_experts_layer import RoutedExpertsLayer
    rows, L = 30, route.N_LATENT
    whole = RoutedExpertsLayer(rows, expert_width=32)
    latent = rows_of(1, rows, L)
    ids = torch.rand((rows, 896), device=DEV).topk(16, dim=1).indices.to(torch.int32)
    ids[7] = -1
    weights = torch.rand((rows, 16), device=DEV) / 8
    whole.mix(latent, ids, weights)
    total = torch.zeros((rows, L), dtype=torch.float64, device=DEV)
    mag = torch.zeros_like(total)
    for first in range(0, 896, 224):
        shard = RoutedExpertsLayer(rows, experts=224, first=first, expert_width=32)
        for name in ("W_gate", "W_up", "W_down"):
            setattr(shard, name, getattr(whole, name)[first:first + 224])
        shard.mix(latent, ids, weights)
        total += shard.mixed.double()
        mag += shard.mixed.double().abs()
        shard.close()
    assert float(whole.mixed[7].abs().max()) == 0
    # one rounding of the whole and one of each part; the FP32 sums are the same terms
    bound = 2.0 ** -8 * 1.02 * (total.abs() + mag)
    assert bool(((whole.mixed.double() - total).abs() <= bound + 1e-6).all())
    whole.close()


def test_training_step():
    from routed_experts_layer import RoutedExpertsLayer
    rows, E, F, L, p, seed = 96, 64, 128, route.N_LATENT, 0.25, 77
    layer = RoutedExpertsLayer(rows, experts=E, first=32, expert_width=F, train=True)
    latent, residual, dy = rows_of(1, rows, L), rows_of(2, rows, L), rows_of(3, rows, L, scale=0.1)
    ids = torch.rand((rows, 128), device=DEV).topk(16, dim=1).indices.to(torch.int32)
    weights = torch.rand((rows, 16), device=DEV) / 8
    y, dlatent, dweights, grads = layer.forward_backward(latent, ids, weights, residual, dy, p=p, seed=seed, step=3)
    offset = 3 * layer.dropout.draws()
    want, keep = experts_ref.dropout(layer.mixed, p, seed, offset, residual, BF16)
    assert ref.worst(y, want) <= 1
    dmixed = experts_ref.dropout(dy, p, seed, offset, None, BF16)[0]
    P = rows * 16
    # the gradient calls one by one, from what the one before gave
    given = torch.empty_like(dy)
    route.dropout_backward(layer.dropout, dy, p, seed, given, offset=offset)
    assert ref.worst(given, dmixed) <= 1
    at, want_dy, want_dw = experts_ref.combine_grads(given, layer.results, layer.place, weights, BF16, P)
    assert ref.worst(layer.dresults[at], want_dy) <= 1 and ref.worst(dweights, want_dw) <= 1
    for e, (lo, hi) in enumerate(runs(layer)):
        if lo == hi:
            continue
        x, w = layer.sorted[lo:hi], (layer.W_gate[e], layer.W_up[e], layer.W_down[e])
        kept = ref.gated(x, *w, None, "silu", BF16)[1]
        g = ref.gated_grads(x, *w, kept, layer.dresults[lo:hi], "silu", BF16)
        assert ref.worst(layer.dsorted[lo:hi], g["dx"]) <= 1, e
        for name in grads:
            assert ref.worst(grads[name][e], g["d" + name]) <= 1, (name, e)
    assert ref.worst(dlatent, experts_ref.combine(layer.dsorted, layer.place, None, None, BF16)) <= 1

    # the whole in float64, by autograd
    v = {n: getattr(layer, n).double().requires_grad_() for n in grads}
    lat, wts = latent.double().requires_grad_(), weights.double().requires_grad_()
    here = (ids >= 32) & (ids < 32 + E)
    mixed = torch.zeros((rows, L), dtype=torch.float64, device=DEV)
    for e in range(E):
        r, j = torch.nonzero(here & (ids - 32 == e), as_tuple=True)
        if len(r):
            t = lat[r]
            h = torch.nn.functional.silu(t @ v["W_gate"][e]) * (t @ v["W_up"][e])
            mixed = mixed.index_add(0, r, wts[r, j, None] * (h @ v["W_down"][e]))
    t = int(p * 65536 + 0.5)
    out = residual.double() + torch.where(keep, mixed, torch.zeros_like(mixed)) * (65536 / (65536 - t))
    out.backward(dy.double())
    # roundings to BF16, half a step (2^-8) each, on the way of each: h, the result,
    # mixed and y; backwards dmixed, dresults, dgate or dup (h), and the gradient
    for name, got, want in [("y", y, out.detach()), ("dlatent", dlatent, lat.grad), ("dweights", dweights, wts.grad)] + \
            [(n, grads[n], v[n].grad) for n in grads]:
        err = float((got.double() - want).norm() / want.norm())
        assert err <= 5 * 2.0 ** -8, (name, err)
    layer.close()


def test_main_runs(capsys):
    import routed_experts_layer
    routed_experts_layer.main(4)
    assert "experts at work" in capsys.readouterr().out
