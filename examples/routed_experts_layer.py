"""One MoE layer's routed experts, as a serving program and a trainer run them.

Serving, for a batch of residual-stream rows x:

    n = norm(x)                                    route.norm_forward
    latent, logits, ids, weights = route(n)        route.route_step
    offsets, place = sort(ids)                     route.dispatch_sort
    sorted = latent at its places                  route.dispatch_gather
    results = experts(sorted)                      route.experts_forward
    mixed = sum of weights * results               route.dispatch_combine
    x = x + mixed W_out                            route.linear_forward (in place)

A rank that holds a shard of the experts (first .. first + experts) runs the same
calls: pairs of other ranks' experts have no place, and the ranks' `mixed` add
up to the layer's.

Training, for the routed experts alone, in the latent width (what the route step
made is given, and it has no gradient): y = residual + dropout(mixed), then the
gradients of the latent rows, of the routing weights and of every expert's weights.
A layer that is trained whole has its dropout behind W_out, in the hidden width, with
route.linear_forward and linear_backward between it and `mixed`.

    python examples/routed_experts_layer.py [rows]
"""

from __future__ import annotations

import os
import sys

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))

import torch  # noqa: E402

import latent_projection_top_gb300 as route  # noqa: E402

DEV = "cuda:0"
BF16 = torch.bfloat16


def _weights(seed: int, *shape, scale: float):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return (torch.randn(shape, generator=g, device=DEV) * scale).to(BF16)


class RoutedExpertsLayer:
    """Plans, weights and buffers of one layer for up to `rows` rows."""

    def __init__(self, rows: int, experts: int = route.N_EXPERTS, first: int = 0,
                 expert_width: int = 64, train: bool = False, seed: int = 0):
        K, L, F, topk = route.K_HIDDEN, route.N_LATENT, expert_width, route.TOPK
        self.rows, pairs = rows, rows * topk
        mode = route.DECODE if rows <= route.DECODE_MAX_ROWS else route.PREFILL
        self.route = route.Plan(mode, rows)
        self.norm = route.NormPlan(rows, K, BF16)
        self.dispatch = route.DispatchPlan(rows, L, BF16, experts=experts, topk=topk, first=first)
        self.experts = route.ExpertsPlan(pairs, L, F, L, experts, BF16, act="silu", train=train)
        self.out = route.LinearPlan(rows, L, K, BF16)
        self.dropout = route.DropoutPlan(rows, L, BF16)
        self.W_latent = _weights(seed, K, L, scale=K ** -0.5)
        self.W_router = _weights(seed + 1, K, route.N_EXPERTS, scale=K ** -0.5)
        self.W_out = _weights(seed + 2, L, K, scale=L ** -0.5)
        self.W_gate = _weights(seed + 3, experts, L, F, scale=L ** -0.5)
        self.W_up = _weights(seed + 4, experts, L, F, scale=L ** -0.5)
        self.W_down = _weights(seed + 5, experts, F, L, scale=F ** -0.5)
        e = lambda r, n, dt=BF16: torch.empty((r, n), dtype=dt, device=DEV)  # noqa: E731
        self.normed, self.latent, self.mixed = e(rows, K), e(rows, L), e(rows, L)
        self.logits = e(rows, route.N_EXPERTS, torch.float32)
        self.ids, self.weights = e(rows, topk, torch.int32), e(rows, topk, torch.float32)
        self.offsets = torch.empty(experts + 1, dtype=torch.int32, device=DEV)
        self.place = e(rows, topk, torch.int32)
        self.sorted, self.results = e(pairs, L), e(pairs, L)
        if train:
            self.saved = self.experts.new_saved()
            self.dresults, self.dsorted = e(pairs, L), e(pairs, L)

    def mix(self, latent, ids, weights, saved=None) -> None:
        """`mixed` from the latent rows and the routing."""
        route.dispatch_sort(self.dispatch, ids, self.offsets, self.place)
        route.dispatch_gather(self.dispatch, latent, self.place, self.sorted)
        route.experts_forward(self.experts, self.sorted, self.offsets, self.W_gate, self.W_up,
                              self.W_down, self.results, saved=saved)
        route.dispatch_combine(self.dispatch, self.results, self.place, weights, self.mixed)

    def step(self, x) -> None:
        """Serving: `x` [rows, 7168] in place."""
        route.norm_forward(self.norm, x, None, None, self.normed)
        route.route_step(self.route, self.normed, self.W_latent, self.W_router, self.latent,
                         self.logits, self.ids, self.weights)
        self.mix(self.latent, self.ids, self.weights)
        route.linear_forward(self.out, self.mixed, self.W_out, x, residual=x)

    def forward_backward(self, latent, ids, weights, residual, dy, p: float = 0.1, seed: int = 0,
                         step: int = 0):
        """Training: y = residual + dropout(mixed); returns y and the gradients
        for dy.  Every `step` drops other values."""
        offset = step * self.dropout.draws()
        y, dmixed, dlatent = (torch.empty_like(latent) for _ in range(3))
        dweights = torch.empty_like(weights)
        grads = {n: torch.empty_like(getattr(self, n)) for n in ("W_gate", "W_up", "W_down")}
        self.mix(latent, ids, weights, saved=self.saved)
        route.dropout_forward(self.dropout, self.mixed, p, seed, y, offset=offset, residual=residual)
        route.dropout_backward(self.dropout, dy, p, seed, dmixed, offset=offset)
        route.dispatch_combine_backward(self.dispatch, dmixed, self.results, self.place, weights,
                                        dy=self.dresults, dweights=dweights)
        route.experts_backward(self.experts, self.dresults, self.sorted, self.offsets, self.W_gate,
                               self.W_up, self.W_down, self.saved, dx=self.dsorted,
                               dW_gate=grads["W_gate"], dW_up=grads["W_up"], dW_down=grads["W_down"])
        route.dispatch_gather_backward(self.dispatch, self.dsorted, self.place, dlatent)
        return y, dlatent, dweights, grads

    def close(self) -> None:
        for plan in (self.route, self.norm, self.dispatch, self.experts, self.out, self.dropout):
            plan.close()


def main(rows: int = 8) -> None:
    layer = RoutedExpertsLayer(rows, train=True)
    x = _weights(9, rows, route.K_HIDDEN, scale=1.0)
    layer.step(x)
    print(f"{rows} rows: {int((layer.offsets.diff() > 0).sum())} experts at work, "
          f"|mixed| = {float(layer.mixed.float().norm()):.4f}")
    y, dlatent, dweights, grads = layer.forward_backward(
        layer.latent, layer.ids, layer.weights, _weights(10, rows, route.N_LATENT, scale=1.0),
        _weights(11, rows, route.N_LATENT, scale=0.1))
    print(f"|dlatent| = {float(dlatent.float().norm()):.4f}, |dweights| = {float(dweights.norm()):.4f}, "
          + ", ".join(f"|d{n}| = {float(g.float().norm()):.4f}" for n, g in grads.items()))
    layer.close()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
