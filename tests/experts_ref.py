"""Plain forms of the routed experts' operators and of dropout, in float64 and
whole numbers, with the bounds on what the kernels may differ (layer_ref.py).

FP32 sums of a few products: every product and addition is within 2^-24 of its
result, so a sum of n terms, each a product, is within (n + 2) 2^-24 of the sum
of magnitudes."""

import numpy as np
import torch

import layer_ref as ref


def sort(ids, experts, first):
    """offsets, place and the sorted pairs of ids [rows, topk] (numpy)."""
    flat = ids.reshape(-1).astype(np.int64) - first
    runs = [np.nonzero(flat == e)[0] for e in range(experts)]
    pairs = np.concatenate(runs) if runs else np.zeros(0, np.int64)
    offsets = np.concatenate([[0], np.cumsum([len(r) for r in runs])])
    place = np.full(flat.shape, -1, np.int64)
    place[pairs] = np.arange(len(pairs))
    return offsets, place.reshape(ids.shape), pairs


def here(place, pairs):
    return (place >= 0) & (place < pairs)


def combine(y, place, weights, residual, dt):
    """A row's sum over its places that are there."""
    ok = here(place, y.shape[0])
    rows, topk = place.shape
    v = torch.zeros((rows, y.shape[1]), dtype=torch.float64, device=y.device)
    mag = torch.zeros_like(v)
    for j in range(topk):
        t = y[place[:, j].clamp(0, max(0, y.shape[0] - 1)).long()].double() if y.shape[0] else torch.zeros_like(v)
        if weights is not None:
            t = t * weights[:, j, None].double()
        t = torch.where(ok[:, j, None], t, torch.zeros_like(t))
        v += t
        mag += t.abs()
    if residual is not None:
        v += residual.double()
        mag += residual.double().abs()
    return ref.rounded((v, (topk + 3) * 2.0 ** -24 * mag), dt)


def combine_grads(dout, y, place, weights, dt, pairs):
    """{pair: dy row} as (index, values with bounds), and dweights with bounds."""
    ok = here(place, pairs)
    r, j = torch.nonzero(ok, as_tuple=True)
    at = place[r, j].long()
    w = weights[r, j].double() if weights is not None else torch.ones(len(r), dtype=torch.float64, device=dout.device)
    dy = w[:, None] * dout[r].double()
    dy = ref.rounded((dy, 2.0 ** -24 * dy.abs()), dt)
    t = dout[r].double() * y[at].double()
    v = torch.zeros(place.shape, dtype=torch.float64, device=dout.device)
    e = torch.zeros_like(v)
    v[r, j] = t.sum(1)
    # a lane's chain of FMAs, then the lanes' sums: no more roundings than terms
    e[r, j] = (dout.shape[1] / 32 + 16) * 2.0 ** -24 * t.abs().sum(1)
    return at, dy, (v, e)


def runs_of(offsets, rows):
    """(lo, hi) of each expert, as the kernels cut what they are given."""
    o = [max(0, min(int(v), rows)) for v in offsets]
    return [(a, max(a, b)) for a, b in zip(o, o[1:])]


def philox(counter, key):
    """Philox 4x32 of ten rounds: counter [n, 4] and key (2) of 32 bits each."""
    c = [counter[:, i].astype(np.uint64) for i in range(4)]
    k = [int(key[0]), int(key[1])]
    low, s = np.uint64(0xFFFFFFFF), np.uint64(32)
    for _ in range(10):
        a, b = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(b >> s) ^ c[1] ^ np.uint64(k[0]), b & low, (a >> s) ^ c[3] ^ np.uint64(k[1]), a & low]
        k = [(k[0] + 0x9E3779B9) & 0xFFFFFFFF, (k[1] + 0xBB67AE85) & 0xFFFFFFFF]
    return np.stack(c, 1)


def lots(rows, dim, seed, offset):
    """The lot of every value, [rows, dim]."""
    groups = (dim + 7) // 8
    with np.errstate(over="ignore"):
        at = np.arange(rows * groups, dtype=np.uint64) + np.uint64(offset % 2 ** 64)
    zero = np.zeros_like(at)
    words = philox(np.stack([at & np.uint64(0xFFFFFFFF), at >> np.uint64(32), zero, zero], 1),
                   (seed & 0xFFFFFFFF, seed >> 32))
    out = np.stack([words & np.uint64(0xFFFF), words >> np.uint64(16)], 2)
    return out.reshape(rows, groups * 8)[:, :dim].astype(np.int64)


def dropout(x, p, seed, offset, residual, dt):
    t = int(np.floor(p * 65536 + 0.5))
    keep = torch.from_numpy(lots(x.shape[0], x.shape[1], seed, offset) >= t).to(x.device)
    zero = torch.zeros((), dtype=torch.float64, device=x.device)
    v = torch.where(keep, x.double() * (65536 / (65536 - t) if t < 65536 else 0.0), zero)
    mag = v.abs()
    if residual is not None:
        v = v + residual.double()
    # the scale's rounding, the product's and the sum's
    return ref.rounded((v, 2.0 ** -23 * mag * 1.01 + 2.0 ** -24 * v.abs()), dt), keep
