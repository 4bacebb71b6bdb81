"""The layer operators that stand around the route step, as measured work.

Three operators, each in the directions a user runs it:

* ``norm``   -- layer norm of token rows: forward, and the backward pass with
  the reduction of the gain's and the offset's gradients over the rows;
* ``linear`` -- a projection with bias, activation and residual in its
  epilogue: forward, and a training step (forward and backward);
* ``gated``  -- a gated feed-forward block, ``(act(x W_gate) * (x W_up)) W_down``
  with an optional residual: forward, and a training step.

``run`` computes them in plain torch operations in FP32 (``own`` false) or by
the calls a user makes of this package (``own`` true); ``exact`` computes them
in FP64 from their definitions.  Weights are stored [K, N], N contiguous.
"""

import math

import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}
EPS = 1e-5


def _case(op, rows, k, n=0, f=0, dtype="bf16", act="none", bias=False, residual=False, name=None):
    c = {"op": op, "rows": rows, "k": k, "n": n, "f": f, "dtype": dtype, "act": act, "bias": bias,
         "residual": residual}
    if name is not None:
        c["name"] = name
    return c


def listed():
    return [
        # the norm before the route step of one decoded token: latency
        _case("norm_fwd", 1, 7168, name="norm fwd 1x7168"),
        # the same over a long prompt's hidden rows: bandwidth
        _case("norm_fwd", 16384, 7168, name="norm fwd 16384x7168"),
        # its backward pass over a training micro-batch of hidden rows
        _case("norm_bwd", 8192, 7168, name="norm bwd 8192x7168"),
        # an FP32 model of odd width, a ragged batch
        _case("norm_bwd", 1037, 1001, dtype="fp32", name="norm bwd 1037x1001 fp32"),
        # latent up projection of a decode batch, added to the residual stream
        _case("linear_fwd", 8, 3584, 7168, residual=True, name="linear fwd 8x3584x7168"),
        # the same for a prompt chunk
        _case("linear_fwd", 4096, 3584, 7168, residual=True, name="linear fwd 4096x3584x7168"),
        # a projection with bias and activation, trained; a row count of no tile's multiple
        _case("linear_train", 2050, 896, 3584, dtype="fp16", act="gelu", bias=True,
              name="linear train 2050x896x3584"),
        # widths that are odd: rows of x, W and the output start at every alignment
        _case("linear_fwd", 333, 1001, 517, act="gelu_tanh", bias=True, residual=True,
              name="linear fwd 333x1001x517"),
        # the shared expert's block for one decoded token
        _case("gated_fwd", 1, 7168, 7168, 2048, act="silu", name="gated fwd 1x7168x2048"),
        # the same for a prompt chunk, added to the residual stream
        _case("gated_fwd", 4096, 7168, 7168, 2048, act="silu", residual=True,
              name="gated fwd 4096x7168x2048"),
        # a block at the latent's width, one training step of a micro-batch
        _case("gated_train", 8192, 3584, 3584, 3584, act="silu",
              name="gated train 8192x3584x3584"),
        # a small ragged FP16 block, trained
        _case("gated_train", 1531, 1000, 1000, 1404, dtype="fp16", act="gelu",
              name="gated train 1531x1000x1404"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo=64, hi=7168):
        w = log(lo, hi)
        kind = rng.random()
        if kind < 0.6:  # most models' widths
            return max(64, w // 64 * 64)
        if kind < 0.8:
            return max(8, w // 8 * 8)
        return w | 1

    op = rng.choice(["norm_fwd", "norm_bwd", "linear_fwd", "linear_train", "gated_fwd",
                     "gated_train"])
    if op.startswith("norm"):
        return _case(op, log(1, 16384), width(64, 7168), dtype=rng.choice(["bf16", "fp16", "fp32"]))
    rows = log(1, 8192)
    dtype = rng.choice(["bf16", "bf16", "fp16"])
    bias, residual = rng.random() < 0.5, rng.random() < 0.5
    if op.startswith("linear"):
        act = rng.choice(["none", "relu", "gelu", "gelu_tanh", "silu", "sigmoid"])
        k, n = width(), width()
        rows = min(rows, 3 * 8192 * 3584 ** 2 // (k * n))
        return _case(op, rows, k, n, dtype=dtype, act=act, bias=bias, residual=residual)
    act = rng.choice(["silu", "gelu", "gelu_tanh", "relu", "sigmoid"])
    k, f = width(), width(64, 3584)
    rows = min(rows, 8192 * 3584 ** 2 // (k * f))
    return _case(op, rows, k, k, f, dtype=dtype, act=act, residual=residual)


def prepare(case, seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    dt = TYPES[case["dtype"]]
    op, R, K, N, F = case["op"], case["rows"], case["k"], case["n"], case["f"]

    def normal(*shape, scale=1.0, dtype=dt):
        return (torch.randn(shape, generator=g, device=DEV) * scale).to(dtype)

    s = {"case": case}
    # hidden rows: a scale and an offset of each row's own, a few channels that stand out
    x = torch.randn((R, K), generator=g, device=DEV)
    if op.startswith("norm"):
        x *= 1 + 19 * (torch.rand((1, K), generator=g, device=DEV) < 0.002)
        x *= torch.rand((R, 1), generator=g, device=DEV) * 3 + 0.25
        x += torch.randn((R, 1), generator=g, device=DEV) * 0.3
    s["x"] = x.to(dt)
    del x
    if op.startswith("norm"):
        s["gamma"] = (1 + 0.2 * torch.randn((K,), generator=g, device=DEV)).to(dt)
        s["beta"] = normal(K, scale=0.1)
        if op == "norm_bwd":
            s["dy"] = normal(R, K, scale=0.1)
            xf = s["x"].float()  # the statistics that the forward pass kept
            mean = xf.mean(1)
            var = (xf - mean[:, None]).square().mean(1)
            s["stats"] = torch.stack([mean, torch.rsqrt(var + EPS)], 1).contiguous()
            del xf
    elif op.startswith("linear"):
        s["W"] = normal(K, N, scale=K ** -0.5)
        s["bias"] = normal(N, scale=0.2) if case["bias"] else None
        s["residual"] = normal(R, N) if case["residual"] else None
    else:
        s["W_gate"] = normal(K, F, scale=K ** -0.5)
        s["W_up"] = normal(K, F, scale=K ** -0.5)
        s["W_down"] = normal(F, N, scale=F ** -0.5)
        s["residual"] = normal(R, N) if case["residual"] else None
    if op.endswith("train"):
        s["dy"] = normal(R, N, scale=0.1)

    if own:
        import latent_projection_top_gb300 as route

        def like(t):
            return None if t is None else torch.empty_like(t)

        train = op.endswith("train")
        if op.startswith("norm"):
            s["plan"] = route.NormPlan(R, K, dt)
            s["y"], s["dgamma"], s["dbeta"] = like(s["x"]), like(s["gamma"]), like(s["beta"])
        else:
            s["y"] = torch.empty((R, N), dtype=dt, device=DEV)
            if op.startswith("linear"):
                s["plan"] = route.LinearPlan(R, K, N, dt, act=case["act"], train=train)
            else:
                s["plan"] = route.GatedPlan(R, K, F, N, dt, act=case["act"], train=train)
            if train:
                s["saved"] = s["plan"].new_saved()
                for w in ("x", "W", "bias", "W_gate", "W_up", "W_down"):
                    s["d" + w] = like(s.get(w))
    return s


# ---- the plain form: FP32 throughout, rounded once at the end ------------------

def _act(a, v):
    """act(v) and its derivative."""
    if a == "none":
        return v, torch.ones_like(v)
    if a == "relu":
        return v.clamp(min=0), (v > 0).to(v.dtype)
    if a == "sigmoid":
        s = 1 / (1 + torch.exp(-v))
        return s, s * (1 - s)
    if a == "silu":
        s = 1 / (1 + torch.exp(-v))
        return v * s, s * (1 + v * (1 - s))
    if a == "gelu":
        c = 0.5 * (1 + torch.erf(v * 0.5 ** 0.5))
        return v * c, c + v * torch.exp(-0.5 * v * v) * (2 * math.pi) ** -0.5
    u = (2 / math.pi) ** 0.5 * (v + 0.044715 * v * v * v)
    t = torch.tanh(u)
    du = (2 / math.pi) ** 0.5 * (1 + 3 * 0.044715 * v * v)
    return 0.5 * v * (1 + t), 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * du


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    x = s["x"].float()
    if op == "norm_fwd":
        d = x - x.mean(1, keepdim=True)
        r = torch.rsqrt((d * d).mean(1, keepdim=True) + EPS)
        return {"y": (d * r * s["gamma"].float() + s["beta"].float()).to(dt)}
    if op == "norm_bwd":
        dy, mean, r = s["dy"].float(), s["stats"][:, :1], s["stats"][:, 1:]
        xh = (x - mean) * r
        gdy = dy * s["gamma"].float()
        dx = r * (gdy - gdy.mean(1, keepdim=True) - xh * (gdy * xh).mean(1, keepdim=True))
        return {"dx": dx.to(dt), "dgamma": (dy * xh).sum(0).to(dt), "dbeta": dy.sum(0).to(dt)}
    res = s["residual"]
    if op.startswith("linear"):
        W = s["W"].float()
        z = x @ W
        if s["bias"] is not None:
            z = z + s["bias"].float()
        y, d = _act(c["act"], z)
        out = {"y": (y if res is None else y + res.float()).to(dt)}
        if op == "linear_train":
            dz = s["dy"].float() * d
            out["dx"] = (dz @ W.t()).to(dt)
            out["dW"] = (x.t() @ dz).to(dt)
            if s["bias"] is not None:
                out["dbias"] = dz.sum(0).to(dt)
        return out
    Wg, Wu, Wd = s["W_gate"].float(), s["W_up"].float(), s["W_down"].float()
    u = x @ Wu
    a, d = _act(c["act"], x @ Wg)
    h = a * u
    y = h @ Wd
    out = {"y": (y if res is None else y + res.float()).to(dt)}
    if op == "gated_train":
        dy = s["dy"].float()
        dh = dy @ Wd.t()
        dg, du = dh * u * d, dh * a
        out["dx"] = (dg @ Wg.t() + du @ Wu.t()).to(dt)
        out["dW_gate"] = (x.t() @ dg).to(dt)
        out["dW_up"] = (x.t() @ du).to(dt)
        out["dW_down"] = (h.t() @ dy).to(dt)
    return out


def run(s):
    if not own:
        return _plain(s)
    import latent_projection_top_gb300 as route
    c = s["case"]
    op, plan = c["op"], s["plan"]
    if op == "norm_fwd":
        route.norm_forward(plan, s["x"], s["gamma"], s["beta"], s["y"], eps=EPS)
        return {"y": s["y"]}
    if op == "norm_bwd":
        route.norm_backward(plan, s["dy"], s["x"], s["gamma"], s["stats"], dx=s["y"],
                            dgamma=s["dgamma"], dbeta=s["dbeta"])
        return {"dx": s["y"], "dgamma": s["dgamma"], "dbeta": s["dbeta"]}
    if op == "linear_fwd":
        route.linear_forward(plan, s["x"], s["W"], s["y"], bias=s["bias"], residual=s["residual"])
        return {"y": s["y"]}
    if op == "linear_train":
        route.linear_forward(plan, s["x"], s["W"], s["y"], bias=s["bias"], residual=s["residual"],
                             saved=s["saved"])
        route.linear_backward(plan, s["dy"], s["x"], s["W"], saved=s["saved"], dx=s["dx"],
                              dW=s["dW"], dbias=s["dbias"])
        out = {"y": s["y"], "dx": s["dx"], "dW": s["dW"]}
        if s["bias"] is not None:
            out["dbias"] = s["dbias"]
        return out
    w = (s["W_gate"], s["W_up"], s["W_down"])
    if op == "gated_fwd":
        route.gated_forward(plan, s["x"], *w, s["y"], residual=s["residual"])
        return {"y": s["y"]}
    route.gated_forward(plan, s["x"], *w, s["y"], residual=s["residual"], saved=s["saved"])
    route.gated_backward(plan, s["dy"], s["x"], *w, s["saved"], dx=s["dx"], dW_gate=s["dW_gate"],
                         dW_up=s["dW_up"], dW_down=s["dW_down"])
    return {"y": s["y"], "dx": s["dx"], "dW_gate": s["dW_gate"], "dW_up": s["dW_up"],
            "dW_down": s["dW_down"]}


def work(case):
    op, R, K, N, F = case["op"], case["rows"], case["k"], case["n"], case["f"]
    e = 4 if case["dtype"] == "fp32" else 2
    if op == "norm_fwd":
        return {"bytes": e * (2 * R * K + 2 * K), "flops": 8 * R * K}
    if op == "norm_bwd":
        return {"bytes": e * (3 * R * K + 3 * K) + 8 * R, "flops": 14 * R * K}
    res = R * N if case["residual"] else 0
    if op.startswith("linear"):
        b = N if case["bias"] else 0
        fwd, mm = R * K + K * N + R * N + b + res, 2 * R * K * N
        if op == "linear_fwd":
            return {"bytes": e * fwd, "flops": mm}
        return {"bytes": e * (fwd + R * N + R * K + K * N + b), "flops": 3 * mm}
    fwd = R * K + 2 * K * F + F * N + R * N + res
    mm = 2 * R * (2 * K * F + F * N)
    if op == "gated_fwd":
        return {"bytes": e * fwd, "flops": mm}
    return {"bytes": e * (fwd + R * N + R * K + 2 * K * F + F * N), "flops": 3 * mm}


# ---- the definitions in FP64, written on their own ---------------------------------

_SLOPE = {
    "none": (lambda v: v, lambda v: v * 0 + 1),
    "relu": (lambda v: torch.where(v > 0, v, v * 0), lambda v: (v > 0).double()),
    "sigmoid": (lambda v: torch.reciprocal(1 + torch.exp(-v)),
                lambda v: torch.reciprocal(2 + torch.exp(v) + torch.exp(-v))),
    "silu": (lambda v: v / (1 + torch.exp(-v)),
             lambda v: (1 + torch.exp(-v) * (1 + v)) / (1 + torch.exp(-v)) ** 2),
    "gelu": (lambda v: v * torch.erfc(-v / math.sqrt(2)) / 2,
             lambda v: torch.erfc(-v / math.sqrt(2)) / 2
             + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)),
    # 0.5 v (1 + tanh u) = v / (1 + exp(-2 u))
    "gelu_tanh": (lambda v: v / (1 + torch.exp(-2 * _cubic(v))),
                  lambda v: torch.reciprocal(1 + torch.exp(-2 * _cubic(v)))
                  + v * math.sqrt(2 / math.pi) * (1 + 0.134145 * v * v)
                  / (2 * torch.cosh(_cubic(v)) ** 2)),
}


def _cubic(v):
    return math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)


def exact(case, seed):
    s = prepare(case, seed)
    t = {k: v.double() for k, v in s.items() if isinstance(v, torch.Tensor)}
    op, R, K = case["op"], case["rows"], case["k"]
    x = t["x"]
    if op == "norm_fwd":
        mu = x.sum(1, keepdim=True) / K
        var = ((x - mu) ** 2).sum(1, keepdim=True) / K
        return {"y": (x - mu) / torch.sqrt(var + EPS) * t["gamma"] + t["beta"]}
    if op == "norm_bwd":
        # with the kept statistics as given: dx_j = r (g_j - sum_i g_i (1 + xh_i xh_j) / K)
        r = t["stats"][:, 1:2]
        xh = (x - t["stats"][:, 0:1]) * r
        g = t["dy"] * t["gamma"]
        dx = r * (g - (g.sum(1, keepdim=True) + xh * (g * xh).sum(1, keepdim=True)) / K)
        return {"dx": dx, "dgamma": torch.einsum("rk,rk->k", t["dy"], xh),
                "dbeta": t["dy"].sum(0)}
    f, df = _SLOPE[case["act"]]
    add = t["residual"] if case["residual"] else 0
    if op.startswith("linear"):
        z = torch.matmul(x, t["W"]) + (t["bias"] if case["bias"] else 0)
        out = {"y": f(z) + add}
        if op == "linear_train":
            dz = df(z).mul_(t["dy"])
            out["dx"] = torch.matmul(dz, t["W"].T)
            out["dW"] = torch.matmul(x.T, dz)
            if case["bias"]:
                out["dbias"] = dz.sum(0)
        return out
    gate, up = torch.matmul(x, t["W_gate"]), torch.matmul(x, t["W_up"])
    h = f(gate) * up
    out = {"y": torch.matmul(h, t["W_down"]) + add}
    if op == "gated_train":
        out["dW_down"] = torch.matmul(h.T, t["dy"])
        dh = torch.matmul(t["dy"], t["W_down"].T)
        dgate, dup = dh * up * df(gate), dh * f(gate)
        out["dW_gate"] = torch.matmul(x.T, dgate)
        out["dW_up"] = torch.matmul(x.T, dup)
        out["dx"] = torch.matmul(dgate, t["W_gate"].T) + torch.matmul(dup, t["W_up"].T)
    return out
