"""The routed experts' operators, and dropout, as measured work.

What a layer runs between the route step's ids and weights and the residual
stream:

* ``dispatch``     -- token rows sorted by expert: the sort of the (row, expert)
  pairs and the rows copied to their places; ``dispatch_bwd`` is the copies'
  gradient, each row the sum of its places;
* ``combine``      -- rows back in their order, each the weighted sum of its
  experts' results, added to a residual; ``combine_bwd`` gives the gradients
  of the experts' results and of the weights;
* ``experts``      -- the gated feed-forward block of every expert on its own
  run of the sorted rows: forward, and a training step;
* ``dropout``      -- from a counter-based generator (Philox 4x32 of ten rounds,
  Salmon et al., SC 2011), added to a residual; ``dropout_train`` is forward
  and backward.  No mask is stored.

``run`` computes them in plain torch operations in FP32 (``own`` false) or by
the calls a user makes of this package (``own`` true); ``exact`` computes them
in FP64 from their definitions.  Experts' weights are stored [experts, K, N],
N contiguous.

Ids name experts of the whole layer (``total``); a program that holds a shard
of them (``first`` .. ``first + experts``) leaves the other pairs out.
"""

import math

import numpy as np
import torch

own = False

DEV = "cuda:0"
TYPES = {"bf16": torch.bfloat16, "fp16": torch.float16, "fp32": torch.float32}


def _routed(op, rows, dim, total, topk, experts=None, first=0, dtype="bf16", residual=False, name=None):
    c = {"op": op, "rows": rows, "dim": dim, "total": total, "topk": topk,
         "experts": total if experts is None else experts, "first": first, "dtype": dtype,
         "residual": residual}
    return c if name is None else {**c, "name": name}


def _experts(op, rows, k, f, n, total, topk, experts=None, first=0, dtype="bf16", act="silu", name=None):
    c = {"op": op, "rows": rows, "k": k, "f": f, "n": n, "total": total, "topk": topk,
         "experts": total if experts is None else experts, "first": first, "dtype": dtype, "act": act}
    return c if name is None else {**c, "name": name}


def _dropout(op, rows, dim, p, dtype="bf16", residual=False, name=None):
    c = {"op": op, "rows": rows, "dim": dim, "p": p, "dtype": dtype, "residual": residual}
    return c if name is None else {**c, "name": name}


def listed():
    return [
        # a decode batch's latent rows to all of the layer's experts: latency
        _routed("dispatch", 8, 3584, 896, 16, name="dispatch 8x3584"),
        # a prompt chunk's: bandwidth
        _routed("dispatch", 4096, 3584, 896, 16, name="dispatch 4096x3584"),
        # gradient of the copies, an FP32 model of odd width with few experts
        _routed("dispatch_bwd", 2049, 1001, 64, 4, dtype="fp32", name="dispatch bwd 2049x1001 fp32"),
        # a decode batch's results back to their rows, one of eight shards of the experts
        _routed("combine", 8, 3584, 896, 16, experts=112, first=224, residual=True,
                name="combine 8x3584 shard"),
        # gradients of a training micro-batch's results and weights
        _routed("combine_bwd", 4096, 3584, 896, 16, name="combine bwd 4096x3584"),
        # one token through a small layer, two of 64 experts: latency
        _experts("experts_fwd", 1, 896, 448, 896, 64, 2, name="experts fwd 1 row 896x448"),
        # a decode batch on one of eight shards: each expert's weights are read for a row or two
        _experts("experts_fwd", 8, 3584, 2048, 3584, 896, 16, experts=112, first=448,
                 name="experts fwd 8 rows 3584x2048 shard"),
        # a prompt on few experts, about a thousand rows each: the tensor cores' rate
        _experts("experts_fwd", 8192, 3584, 2048, 3584, 64, 8, experts=16, first=16,
                 name="experts fwd 8192 rows 3584x2048 shard"),
        # a training micro-batch on a shard of narrow experts, about 73 rows each
        _experts("experts_train", 4096, 3584, 1024, 3584, 896, 16, experts=28, first=56,
                 name="experts train 4096 rows 3584x1024 shard"),
        # a small FP16 layer, trained: two of eight experts, ragged
        _experts("experts_train", 1531, 1000, 1400, 1000, 8, 2, dtype="fp16", act="gelu",
                 name="experts train 1531 rows 1000x1400 fp16"),
        # residual dropout of a few rows: latency
        _dropout("dropout_fwd", 20, 7168, 0.1, residual=True, name="dropout fwd 20x7168"),
        # of a training micro-batch, forward and backward
        _dropout("dropout_train", 8192, 7168, 0.1, residual=True, name="dropout train 8192x7168"),
    ]


def draw(rng):
    def log(lo, hi):
        return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))

    def width(lo, hi):
        w = log(lo, hi)
        return max(64, w // 64 * 64) if rng.random() < 0.7 else max(8, w // 8 * 8)

    op = rng.choice(["dispatch", "dispatch_bwd", "combine", "combine_bwd", "experts_fwd",
                     "experts_fwd", "experts_train", "experts_train", "dropout_fwd",
                     "dropout_train"])
    if op.startswith("dropout"):
        d = log(64, 7168)
        return _dropout(op, log(1, 8192), d if rng.random() < 0.3 else max(8, d // 8 * 8),
                        rng.choice([0.05, 0.1, 0.2, 0.5]), dtype=rng.choice(["bf16", "fp16", "fp32"]),
                        residual=rng.random() < 0.5)
    total, topk = rng.choice([(896, 16), (896, 16), (256, 8), (64, 6), (64, 4), (8, 2), (5, 3)])
    shard = rng.choice([1, 1, 2, 4, 8])
    experts = max(1, total // shard)
    first = rng.randrange(shard) * experts
    if not op.startswith("experts"):
        d = log(64, 4096)
        d = d | 1 if rng.random() < 0.2 else max(8, d // 8 * 8)
        return _routed(op, min(log(1, 8192), 4096 * 16 // topk), d, total, topk, experts, first,
                       dtype=rng.choice(["bf16", "bf16", "fp16", "fp32"]),
                       residual=op == "combine" and rng.random() < 0.5)
    k, f = width(64, 3584), width(64, 2048)
    n = k if rng.random() < 0.7 else width(64, 3584)
    # no more weights and no more products than the largest listed cases'
    room = 740_000_000 if op == "experts_train" else 2_200_000_000
    experts = max(1, min(experts, room // (2 * f * (2 * k + n))))
    if first + experts > total:
        first = 0
    most = 16384 * 2048 * 3 * 3584 * total // (f * (2 * k + n) * experts * topk)
    rows = max(1, min(log(1, 8192), most // (3 if op == "experts_train" else 1)))
    return _experts(op, rows, k, f, n, total, topk, experts, first, dtype=rng.choice(["bf16", "bf16", "fp16"]),
                    act=rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"]))


# ---- inputs ----------------------------------------------------------------------

def _generator(seed):
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    return g


def _routing(case, g):
    """A router's choice: some experts are wanted more than others.  Rows pick
    without repetition; a batch's last rows are padding now and then (id -1)."""
    R, E, topk = case["rows"], case["total"], case["topk"]
    liking = torch.randn((1, E), generator=g, device=DEV) * 0.5
    logits = torch.randn((R, E), generator=g, device=DEV) + liking
    top = logits.topk(topk, dim=1)
    ids = top.indices.to(torch.int32)
    if R > 8:
        ids[R - R // 64 - 1:] = -1
    w = torch.sigmoid(top.values)
    return ids, w / w.sum(1, keepdim=True)


def _sorted_pairs(ids, first, experts):
    """offsets [experts + 1], place [rows, topk] (-1: not here), and the pairs
    in their sorted order (stable), of which the first offsets[-1] are here."""
    flat = ids.reshape(-1).long() - first
    here = (flat >= 0) & (flat < experts)
    key = torch.where(here, flat, torch.full_like(flat, experts))
    order = torch.sort(key, stable=True).indices
    counts = (key[:, None] == torch.arange(experts, device=DEV)[None]).sum(0) if key.numel() * experts < 1 << 22 \
        else torch.zeros(experts + 1, dtype=torch.long, device=DEV).index_add_(0, key, torch.ones_like(key))[:experts]
    offsets = torch.zeros(experts + 1, dtype=torch.int32, device=DEV)
    offsets[1:] = counts.cumsum(0)
    place = torch.empty_like(flat)
    place[order] = torch.arange(flat.numel(), device=DEV)
    place = torch.where(here, place, torch.full_like(place, -1)).to(torch.int32)
    return offsets, place.reshape(ids.shape), order


def prepare(case, seed):
    g = _generator(seed)
    dt = TYPES[case["dtype"]]
    op, R = case["op"], case["rows"]

    def normal(*shape, scale=1.0, dtype=dt):
        return torch.randn(shape, generator=g, device=DEV).mul_(scale).to(dtype)

    def weights(*shape, scale):
        w = torch.empty(shape, dtype=dt, device=DEV)
        for e in range(shape[0]):
            w[e] = torch.randn(shape[1:], generator=g, device=DEV).mul_(scale)
        return w

    s = {"case": case}
    if op.startswith("dropout"):
        D = case["dim"]
        s["x"] = normal(R, D)
        s["residual"] = normal(R, D) if case["residual"] else None
        s["seed"], s["offset"] = 0x9E3779B97F4A7C15 ^ seed, seed % 1009 << 33
        if op == "dropout_train":
            s["dy"] = normal(R, D, scale=0.1)
        if own:
            import latent_projection_top_gb300 as route
            s["plan"] = route.DropoutPlan(R, D, dt)
            s["y"], s["dx"] = torch.empty_like(s["x"]), torch.empty_like(s["x"])
        return s

    E, first, topk = case["experts"], case["first"], case["topk"]
    pairs = R * topk
    ids, w = _routing(case, g)
    offsets, place, _ = _sorted_pairs(ids, first, E)
    if op.startswith("experts"):
        k, f, n = case["k"], case["f"], case["n"]
        # sorted rows, for the pairs that could be here; those behind the last one stay unused
        s["x"], s["offsets"] = normal(pairs, k), offsets
        s["W_gate"] = weights(E, k, f, scale=k ** -0.5)
        s["W_up"] = weights(E, k, f, scale=k ** -0.5)
        s["W_down"] = weights(E, f, n, scale=f ** -0.5)
        s["y"] = torch.zeros((pairs, n), dtype=dt, device=DEV)
        if op == "experts_train":
            s["dy"] = normal(pairs, n, scale=0.1)
            s["dx"] = torch.zeros_like(s["x"])
        if own:
            import latent_projection_top_gb300 as route
            train = op == "experts_train"
            s["plan"] = route.ExpertsPlan(pairs, k, f, n, E, dt, act=case["act"], train=train)
            if train:
                s["saved"] = s["plan"].new_saved()
                for name in ("W_gate", "W_up", "W_down"):
                    s["d" + name] = torch.empty_like(s[name])
        return s

    D = case["dim"]
    if op == "dispatch":
        s["x"], s["ids"] = normal(R, D), ids
        s["xs"] = torch.zeros((pairs, D), dtype=dt, device=DEV)
        s["source"] = torch.full((pairs,), -1, dtype=torch.int32, device=DEV)
        if own:
            s["offsets"] = torch.empty(E + 1, dtype=torch.int32, device=DEV)
            s["place"] = torch.empty((R, topk), dtype=torch.int32, device=DEV)
    elif op == "dispatch_bwd":
        s["place"], s["dxs"] = place, normal(pairs, D, scale=0.1)
        s["dx"] = torch.empty((R, D), dtype=dt, device=DEV)
    else:
        s["place"], s["weights"], s["ys"] = place, w, normal(pairs, D)
        if op == "combine":
            s["residual"] = normal(R, D) if case["residual"] else None
            s["y"] = torch.empty((R, D), dtype=dt, device=DEV)
        else:
            s["dy"] = normal(R, D, scale=0.1)
            s["dys"] = torch.zeros((pairs, D), dtype=dt, device=DEV)
            s["dw"] = torch.empty((R, topk), dtype=torch.float32, device=DEV)
    if own:
        import latent_projection_top_gb300 as route
        s["plan"] = route.DispatchPlan(R, D, dt, experts=E, topk=topk, first=first)
    return s


# ---- the plain form: FP32 throughout, rounded once at the end ------------------

def _act(a, v):
    """act(v) and its derivative."""
    if a == "relu":
        return v.clamp(min=0), (v > 0).to(v.dtype)
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


def _lots(s):
    """The 16-bit lot of every element: eight of the 128 bits of a counter, a
    row's counters following one another, rows one after another."""
    R, D = s["case"]["rows"], s["case"]["dim"]
    groups = (D + 7) // 8
    m32 = 0xFFFFFFFF
    at = torch.arange(R * groups, device=DEV) + s["offset"]
    c = [at & m32, (at >> 32) & m32, torch.zeros_like(at), torch.zeros_like(at)]
    k0, k1 = s["seed"] & m32, (s["seed"] >> 32) & m32
    for _ in range(10):
        a, b = c[0] * 0xD2511F53, c[2] * 0xCD9E8D57  # of 64 bits: they wrap
        c = [((b >> 32) & m32) ^ c[1] ^ k0, b & m32, ((a >> 32) & m32) ^ c[3] ^ k1, a & m32]
        k0, k1 = (k0 + 0x9E3779B9) & m32, (k1 + 0xBB67AE85) & m32
    words = torch.stack(c, 1)
    lots = torch.stack([words & 0xFFFF, words >> 16], 2)
    return lots.reshape(R, groups * 8)[:, :D]


def _plain(s):
    c = s["case"]
    op, dt = c["op"], TYPES[c["dtype"]]
    if op.startswith("dropout"):
        t = math.floor(c["p"] * 65536 + 0.5)
        keep, scale = _lots(s) >= t, 65536 / (65536 - t)
        y = torch.where(keep, s["x"].float() * scale, torch.zeros((), device=DEV))
        y = (y if s["residual"] is None else y + s["residual"].float()).to(dt)
        if op == "dropout_fwd":
            return {"y": y}
        return {"y": y, "dx": torch.where(keep, s["dy"].float() * scale, torch.zeros((), device=DEV)).to(dt)}
    E = c["experts"]
    if op == "dispatch":
        offsets, place, order = _sorted_pairs(s["ids"], c["first"], E)
        at = torch.arange(order.numel(), device=DEV)
        here = at < offsets[-1]
        source = torch.where(here, order, torch.full_like(order, -1)).to(torch.int32)
        xs = torch.where(here[:, None], s["x"][order // c["topk"]], torch.zeros((), dtype=dt, device=DEV))
        return {"offsets": offsets, "place": place, "source": source, "xs": xs}
    if op.startswith("dispatch") or op.startswith("combine"):
        place = s["place"].long()
        here, at = place >= 0, place.clamp(min=0)
        zero = torch.zeros((), device=DEV)
        if op == "combine_bwd":
            dy, w = s["dy"].float(), s["weights"]
            dys = s["dys"].clone()
            dw = torch.zeros_like(s["dw"])
            for j in range(c["topk"]):
                p = at[:, j]
                dw[:, j] = torch.where(here[:, j], (dy * s["ys"][p].float()).sum(1), zero)
                p = torch.where(here[:, j])[0]
                dys[at[p, j]] = (w[p, j, None] * dy[p]).to(dt)
            return {"dys": dys, "dw": dw}
        src = s["dxs"] if op == "dispatch_bwd" else s["ys"]
        y = torch.zeros((c["rows"], c["dim"]), device=DEV)
        for j in range(c["topk"]):
            v = src[at[:, j]].float()
            if op == "combine":
                v = v * s["weights"][:, j, None]
            y += torch.where(here[:, j, None], v, zero)
        if op == "dispatch_bwd":
            return {"dx": y.to(dt)}
        return {"y": (y if s["residual"] is None else y + s["residual"].float()).to(dt)}
    train = op == "experts_train"
    out = {"y": s["y"].clone()}
    if train:
        out["dx"] = s["dx"].clone()
        for name in ("W_gate", "W_up", "W_down"):
            out["d" + name] = torch.zeros_like(s[name])
    at = s["offsets"].tolist()
    for e in range(E):
        lo, hi = at[e], at[e + 1]
        if lo == hi:
            continue
        x = s["x"][lo:hi].float()
        Wg, Wu, Wd = s["W_gate"][e].float(), s["W_up"][e].float(), s["W_down"][e].float()
        u = x @ Wu
        a, d = _act(c["act"], x @ Wg)
        h = a * u
        out["y"][lo:hi] = (h @ Wd).to(dt)
        if train:
            dy = s["dy"][lo:hi].float()
            dh = dy @ Wd.t()
            dg, du = dh * u * d, dh * a
            out["dx"][lo:hi] = (dg @ Wg.t() + du @ Wu.t()).to(dt)
            out["dW_gate"][e] = (x.t() @ dg).to(dt)
            out["dW_up"][e] = (x.t() @ du).to(dt)
            out["dW_down"][e] = (h.t() @ dy).to(dt)
    return out


def run(s):
    if not own:
        return _plain(s)
    import latent_projection_top_gb300 as route
    op, plan = s["case"]["op"], s["plan"]
    if op == "dispatch":
        route.dispatch_sort(plan, s["ids"], s["offsets"], s["place"], source=s["source"])
        route.dispatch_gather(plan, s["x"], s["place"], s["xs"])
        return {"offsets": s["offsets"], "place": s["place"], "source": s["source"], "xs": s["xs"]}
    if op == "dispatch_bwd":
        route.dispatch_gather_backward(plan, s["dxs"], s["place"], s["dx"])
        return {"dx": s["dx"]}
    if op == "combine":
        route.dispatch_combine(plan, s["ys"], s["place"], s["weights"], s["y"], residual=s["residual"])
        return {"y": s["y"]}
    if op == "combine_bwd":
        route.dispatch_combine_backward(plan, s["dy"], s["ys"], s["place"], s["weights"], dy=s["dys"],
                                        dweights=s["dw"])
        return {"dys": s["dys"], "dw": s["dw"]}
    if op.startswith("dropout"):
        c = s["case"]
        route.dropout_forward(plan, s["x"], c["p"], s["seed"], s["y"], offset=s["offset"],
                              residual=s["residual"])
        if op == "dropout_fwd":
            return {"y": s["y"]}
        route.dropout_backward(plan, s["dy"], c["p"], s["seed"], s["dx"], offset=s["offset"])
        return {"y": s["y"], "dx": s["dx"]}
    w = (s["W_gate"], s["W_up"], s["W_down"])
    if op == "experts_fwd":
        route.experts_forward(plan, s["x"], s["offsets"], *w, s["y"])
        return {"y": s["y"]}
    route.experts_forward(plan, s["x"], s["offsets"], *w, s["y"], saved=s["saved"])
    route.experts_backward(plan, s["dy"], s["x"], s["offsets"], *w, s["saved"], dx=s["dx"],
                           dW_gate=s["dW_gate"], dW_up=s["dW_up"], dW_down=s["dW_down"])
    return {"y": s["y"], "dx": s["dx"], "dW_gate": s["dW_gate"], "dW_up": s["dW_up"],
            "dW_down": s["dW_down"]}


def work(case):
    """Of a router that likes all experts alike: the pairs that are here, and
    the experts that any of them names."""
    op, R = case["op"], case["rows"]
    e = 4 if case["dtype"] == "fp32" else 2
    if op.startswith("dropout"):
        one = R * case["dim"]
        parts = (3 if case["residual"] else 2) + (2 if op == "dropout_train" else 0)
        return {"bytes": e * parts * one, "flops": 2 * parts * one}
    here = case["experts"] / case["total"]
    pairs = R * case["topk"]
    P = pairs * here
    rows_here = R * (1 - (1 - here) ** case["topk"])
    if op.startswith("experts"):
        k, f, n = case["k"], case["f"], case["n"]
        used = case["experts"] * (1 - (1 - case["topk"] / case["total"]) ** R)
        weights = f * (2 * k + n)
        mm = 2 * P * weights
        fwd = P * (k + n) + used * weights
        if op == "experts_fwd":
            return {"bytes": 2 * fwd, "flops": mm}
        return {"bytes": 2 * (fwd + P * (k + n) + case["experts"] * weights), "flops": 3 * mm}
    D = case["dim"]
    if op == "dispatch":
        return {"bytes": e * D * (rows_here + P) + 4 * (2 * pairs + P + case["experts"] + 1), "flops": P * D}
    if op == "dispatch_bwd":
        return {"bytes": e * D * (P + R) + 4 * pairs, "flops": P * D}
    if op == "combine":
        return {"bytes": e * D * (P + R * (2 if case["residual"] else 1)) + 8 * pairs, "flops": 2 * P * D}
    return {"bytes": e * D * (2 * P + rows_here) + 12 * pairs, "flops": 3 * P * D}


# ---- the definitions in FP64, written on their own ---------------------------------

def _logistic(v):
    return torch.reciprocal(1 + torch.exp(-v))


def _cubic(v):
    return math.sqrt(2 / math.pi) * (v + 0.044715 * v ** 3)


_SLOPE = {
    "relu": (lambda v: torch.where(v > 0, v, v * 0), lambda v: (v > 0).double()),
    "silu": (lambda v: v / (1 + torch.exp(-v)),
             lambda v: (1 + torch.exp(-v) * (1 + v)) / (1 + torch.exp(-v)) ** 2),
    "gelu": (lambda v: v * torch.erfc(-v / math.sqrt(2)) / 2,
             lambda v: torch.erfc(-v / math.sqrt(2)) / 2
             + v * torch.exp(-v * v / 2) / math.sqrt(2 * math.pi)),
    # 0.5 v (1 + tanh u) = v / (1 + exp(-2 u))
    "gelu_tanh": (lambda v: v * _logistic(2 * _cubic(v)),
                  lambda v: _logistic(2 * _cubic(v))
                  + v * math.sqrt(2 / math.pi) * (1 + 0.134145 * v * v)
                  / (2 * torch.cosh(_cubic(v)) ** 2)),
}


def _philox_keep(s):
    """Philox on the host's unsigned integers: which elements are kept."""
    c = s["case"]
    R, D = c["rows"], c["dim"]
    groups = -(-D // 8)
    counter = np.arange(R * groups, dtype=np.uint64) + np.uint64(s["offset"])
    low = np.uint64(0xFFFFFFFF)
    x0, x1 = counter & low, counter >> np.uint64(32)
    x2, x3 = np.zeros_like(x0), np.zeros_like(x0)
    key0, key1 = s["seed"] % 2 ** 32, s["seed"] // 2 ** 32 % 2 ** 32
    for _ in range(10):
        p0, p1 = x0 * np.uint64(0xD2511F53), x2 * np.uint64(0xCD9E8D57)
        x0, x1, x2, x3 = ((p1 >> np.uint64(32)) ^ x1 ^ np.uint64(key0), p1 & low,
                          (p0 >> np.uint64(32)) ^ x3 ^ np.uint64(key1), p0 & low)
        key0, key1 = (key0 + 0x9E3779B9) % 2 ** 32, (key1 + 0xBB67AE85) % 2 ** 32
    bits = np.empty((R * groups, 8), dtype=np.uint16)
    for i, word in enumerate((x0, x1, x2, x3)):
        bits[:, 2 * i] = word & np.uint64(0xFFFF)
        bits[:, 2 * i + 1] = word >> np.uint64(16)
    t = int(c["p"] * 65536 + 0.5)
    return torch.from_numpy(bits.reshape(R, groups * 8)[:, :D] >= t).to(DEV), 65536 / (65536 - t)


def exact(case, seed):
    s = prepare(case, seed)
    op, topk = case["op"], case.get("topk")
    if op.startswith("dropout"):
        keep, scale = _philox_keep(s)
        y = s["x"].double().mul_(scale).mul_(keep)
        if s["residual"] is not None:
            y += s["residual"]
        return {"y": y} if op == "dropout_fwd" else {"y": y, "dx": s["dy"].double().mul_(scale).mul_(keep)}
    if op == "dispatch":
        # every expert's pairs, one expert after another, in the pairs' order
        ids = s["ids"].cpu().numpy().reshape(-1).astype(np.int64) - case["first"]
        by = [[] for _ in range(case["experts"])]
        for pair in np.nonzero((ids >= 0) & (ids < case["experts"]))[0]:
            by[ids[pair]].append(pair)
        sorted_pairs = np.concatenate([np.asarray(b, dtype=np.int64) for b in by])
        place = np.full(ids.shape, -1, dtype=np.int32)
        place[sorted_pairs] = np.arange(len(sorted_pairs))
        source = np.full(ids.shape, -1, dtype=np.int32)
        source[:len(sorted_pairs)] = sorted_pairs
        offsets = np.concatenate([[0], np.cumsum([len(b) for b in by])]).astype(np.int32)
        xs = torch.zeros(s["xs"].shape, dtype=torch.float64, device=DEV)
        xs[:len(sorted_pairs)] = s["x"].double()[torch.from_numpy(sorted_pairs // topk).to(DEV)]
        return {"offsets": offsets, "place": place.reshape(-1, topk), "source": source, "xs": xs}
    if not op.startswith("experts"):
        # sums over the pairs that are here, as a scatter from the pairs' side
        pair = torch.nonzero(s["place"].reshape(-1) >= 0)[:, 0]
        at, row = s["place"].reshape(-1).long()[pair], pair // topk
        if op == "combine_bwd":
            w = s["weights"].double().reshape(-1)[pair]
            dys = torch.zeros(s["dys"].shape, dtype=torch.float64, device=DEV)
            dw = torch.zeros(case["rows"] * topk, dtype=torch.float64, device=DEV)
            for lo in range(0, len(pair), 8192):
                i = slice(lo, lo + 8192)
                g = s["dy"].double()[row[i]]
                dw[pair[i]] = torch.einsum("pd,pd->p", g, s["ys"][at[i]].double())
                dys[at[i]] = g * w[i, None]
            return {"dys": dys, "dw": dw.reshape(-1, topk)}
        y = torch.zeros((case["rows"], case["dim"]), dtype=torch.float64, device=DEV)
        if op == "dispatch_bwd":
            return {"dx": y.index_add_(0, row, s["dxs"][at].double())}
        y.index_add_(0, row, s["ys"][at].double() * s["weights"].double().reshape(-1)[pair][:, None])
        return {"y": y if s["residual"] is None else y + s["residual"].double()}
    f, df = _SLOPE[case["act"]]
    ends = s["offsets"].cpu().numpy()
    out = {"y": torch.zeros(s["y"].shape, dtype=torch.float64, device=DEV)}
    if op == "experts_train":
        out["dx"] = torch.zeros(s["x"].shape, dtype=torch.float64, device=DEV)
        for name in ("W_gate", "W_up", "W_down"):
            out["d" + name] = torch.zeros(s[name].shape, dtype=torch.float64, device=DEV)
    for e in np.nonzero(np.diff(ends))[0]:
        rows = slice(int(ends[e]), int(ends[e + 1]))
        x = s["x"][rows].double()
        Wg, Wu, Wd = (s[name][e].double() for name in ("W_gate", "W_up", "W_down"))
        gate, up = torch.matmul(x, Wg), torch.matmul(x, Wu)
        h = f(gate) * up
        out["y"][rows] = torch.matmul(h, Wd)
        if op == "experts_train":
            dy = s["dy"][rows].double()
            out["dW_down"][e] = torch.matmul(h.T, dy)
            dh = torch.matmul(dy, Wd.T)
            dgate, dup = dh * up * df(gate), dh * f(gate)
            out["dW_gate"][e] = torch.matmul(x.T, dgate)
            out["dW_up"][e] = torch.matmul(x.T, dup)
            out["dx"][rows] = torch.matmul(dgate, Wg.T) + torch.matmul(dup, Wu.T)
    return out
