"""One MoE layer around the route step, as a serving program and a trainer run it.

Serving, for a batch of residual-stream rows x:

    n = norm(x)                                  route.norm_forward
    latent, logits, ids, weights = route(n)      route.route_step
    x = x + latent W_out                         route.linear_forward (in place)
    x = x + shared expert(n)                     route.gated_forward  (in place)

(the routed experts, which would turn `latent` into their weighted sum before
its projection back to the hidden width, are the caller's).

Training, for the norm and the shared expert of the same layer:

    y = x + gated(norm(x)),  then the gradients of every weight and of x

    python examples/shared_expert_layer.py [rows]
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


class SharedExpertLayer:
    """Plans, weights and buffers of one layer for up to `rows` rows."""

    def __init__(self, rows: int, expert_width: int = 2048, train: bool = False, seed: int = 0):
        K, L, F = route.K_HIDDEN, route.N_LATENT, expert_width
        self.rows = rows
        mode = route.DECODE if rows <= route.DECODE_MAX_ROWS else route.PREFILL
        self.route = route.Plan(mode, rows)
        self.norm = route.NormPlan(rows, K, BF16)
        self.out = route.LinearPlan(rows, L, K, BF16)
        self.expert = route.GatedPlan(rows, K, F, K, BF16, act="silu", train=train)
        self.gamma = torch.ones((K,), dtype=BF16, device=DEV)
        self.beta = torch.zeros((K,), dtype=BF16, device=DEV)
        self.W_latent = _weights(seed, K, L, scale=K ** -0.5)
        self.W_router = _weights(seed + 1, K, route.N_EXPERTS, scale=K ** -0.5)
        self.W_out = _weights(seed + 2, L, K, scale=L ** -0.5)
        self.W_gate, self.W_up = (_weights(seed + s, K, F, scale=K ** -0.5) for s in (3, 4))
        self.W_down = _weights(seed + 5, F, K, scale=F ** -0.5)
        e = lambda n, dt=BF16: torch.empty((rows, n), dtype=dt, device=DEV)  # noqa: E731
        self.normed, self.latent = e(K), e(L)
        self.logits = e(route.N_EXPERTS, torch.float32)
        self.ids, self.weights = e(route.TOPK, torch.int32), e(route.TOPK, torch.float32)
        self.stats = e(2, torch.float32)
        self.saved = self.expert.new_saved() if train else None

    def step(self, x) -> None:
        """Serving: `x` [rows, 7168] in place; ids and weights name the routed experts."""
        route.norm_forward(self.norm, x, self.gamma, self.beta, self.normed)
        route.route_step(self.route, self.normed, self.W_latent, self.W_router, self.latent,
                         self.logits, self.ids, self.weights)
        route.linear_forward(self.out, self.latent, self.W_out, x, residual=x)
        route.gated_forward(self.expert, self.normed, self.W_gate, self.W_up, self.W_down, x,
                            residual=x)

    def forward_backward(self, x, dy):
        """Training: y = x + expert(norm(x)); returns y and the gradients for dy."""
        w = (self.W_gate, self.W_up, self.W_down)
        y, dn, dx = torch.empty_like(x), torch.empty_like(x), torch.empty_like(x)
        grads = {name: torch.empty_like(t) for name, t in
                 zip(("gamma", "beta", "W_gate", "W_up", "W_down"), (self.gamma, self.beta, *w))}
        route.norm_forward(self.norm, x, self.gamma, self.beta, self.normed, stats=self.stats)
        route.gated_forward(self.expert, self.normed, *w, y, residual=x, saved=self.saved)
        route.gated_backward(self.expert, dy, self.normed, *w, self.saved, dx=dn,
                             dW_gate=grads["W_gate"], dW_up=grads["W_up"],
                             dW_down=grads["W_down"])
        route.norm_backward(self.norm, dn, x, self.gamma, self.stats, dx=dx,
                            dgamma=grads["gamma"], dbeta=grads["beta"])
        dx += dy  # the residual's own gradient
        return y, dx, grads

    def close(self) -> None:
        for plan in (self.route, self.norm, self.out, self.expert):
            plan.close()


def main(rows: int = 8) -> None:
    layer = SharedExpertLayer(rows, train=True)
    x = _weights(9, rows, route.K_HIDDEN, scale=1.0)
    stream = x.clone()
    layer.step(stream)
    print(f"{rows} rows: experts of row 0: {layer.ids[0].tolist()}")
    _, dx, grads = layer.forward_backward(x, _weights(10, rows, route.K_HIDDEN, scale=0.1))
    print(f"|dx| = {float(dx.float().norm()):.4f}, " + ", ".join(
        f"|d{name}| = {float(g.float().norm()):.4f}" for name, g in grads.items()))
    layer.close()


if __name__ == "__main__":
    main(int(sys.argv[1]) if len(sys.argv) > 1 else 8)
