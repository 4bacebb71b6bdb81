"""Kernels of the layer operators that the other tests' shapes do not reach, at
shapes that do: the norms' persistent blocks past their first rows, gated tiles
of 256 columns, split tiles' finish kernel with every epilogue, FP32 results in
large tiles.  (Which way a shape goes follows from the estimates in
layer_api.cu, for 152 SMs; the comments name it.)"""

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


def normal(seed, *shape, scale=1.0, dt=BF16, pad=0, offset=0):
    """A seeded matrix; with `pad` or `offset` a view with longer rows that
    starts `offset` elements into its buffer."""
    g = torch.Generator(device=DEV)
    g.manual_seed(seed)
    v = (torch.randn(shape, generator=g, device=DEV) * scale).to(dt)
    if not pad and not offset:
        return v
    ld = shape[1] + pad
    view = torch.full((shape[0] * ld + offset,), float("nan"), dtype=dt, device=DEV)[offset:]
    view = view.view(shape[0], ld)[:, :shape[1]]
    view.copy_(v)
    return view


def blank(rows, cols, dt, pad=0, offset=0):
    """An output of NaN inside a buffer of sevens, and whether those are left."""
    ld = cols + pad
    buf = torch.full((rows * ld + offset + 16,), 7.0, dtype=dt, device=DEV)
    view = buf[offset:offset + rows * ld].view(rows, ld)[:, :cols]
    view.fill_(float("nan"))

    def kept():
        mask = torch.ones_like(buf, dtype=torch.bool)
        mask[offset:offset + rows * ld].view(rows, ld)[:, :cols] = False
        return bool((buf[mask] == 7).all())

    return view, kept


def check(name, got, want):
    w = ref.worst(got, want)
    assert w <= 1, f"{name}: {w:.3g} times the bound"


# ---- norm: ten or more rows of a block, a ring of up to six places ---------------

NORM = [
    # rows (of a block: four warps' or one), dim, type
    (20011, 64, BF16), (20011, 256, FP16), (20011, 1000, BF16), (20011, 200, FP32),
    (6203, 1032, BF16), (6203, 4096, FP16), (6203, 2048, FP32),
    (3209, 7168, BF16), (3209, 8192, FP32), (1603, 9000, FP16), (1603, 16384, BF16), (1603, 9000, FP32),
    # rows at every alignment
    (20011, 65, BF16), (20011, 1001, FP16), (20011, 129, FP32), (6203, 1033, BF16), (6203, 4095, FP32),
    (3209, 5149, FP16), (1603, 9001, BF16), (1603, 9001, FP32),
]


@pytest.mark.parametrize("rows,dim,dt", NORM)
def test_norm_of_many_rows_a_block(rows, dim, dt):
    x = (normal(1, rows, dim, dt=FP32) * 2 + normal(2, rows, 1, dt=FP32)).to(dt)
    gamma, beta = (1 + normal(3, dim, dt=dt) * 0.3).to(dt), normal(4, dim, dt=dt)
    dy = normal(5, rows, dim, dt=dt)
    (y, y_kept), (dx, dx_kept) = blank(rows, dim, dt), blank(rows, dim, dt)
    stats = torch.full((rows, 2), float("nan"), device=DEV)
    dgamma, dbeta = (torch.full((dim,), float("nan"), dtype=dt, device=DEV) for _ in range(2))
    with route.NormPlan(rows, dim, dt) as plan:
        route.norm_forward(plan, x, gamma, beta, y, stats=stats)
        route.norm_backward(plan, dy, x, gamma, stats, dx=dx, dgamma=dgamma, dbeta=dbeta)
        plan.status()
    assert y_kept() and dx_kept()
    # forward: a sum of n terms in any order is within (n + 3) U of the sum of
    # magnitudes; the variance's error is its sum's, its terms' and the mean's squared
    n3 = (dim + 3) * U
    v = x.double()
    mean = v.mean(1, keepdim=True)
    d = v - mean
    var = (d * d).mean(1, keepdim=True)
    r = (var + 1e-5) ** -0.5
    em = n3 * v.abs().mean(1, keepdim=True)
    er = r * (0.5 * (n3 + 4 * U + r * r * em * em) + 3 * U)
    check("mean", stats[:, :1], (mean, em + 1e-30))
    check("rstd", stats[:, 1:], (r, er))
    g = gamma.double()
    want = d * r * g + beta.double()
    check("y", y, ref.rounded((want, (em * r + d.abs() * er + 4 * U * d.abs() * r) * g.abs()
                               + U * (want.abs() + beta.double().abs())), dt))
    # backward, with the statistics that it was given
    m, s = stats[:, :1].double(), stats[:, 1:].double()
    del d, want
    xh = (v - m) * s
    gy = dy.double() * g
    a, ea = gy.mean(1, keepdim=True), n3 * gy.abs().mean(1, keepdim=True)
    b = (gy * xh).mean(1, keepdim=True)
    eb = (n3 + 2.1 * U) * (gy * xh).abs().mean(1, keepdim=True)
    want = s * (gy - a - xh * b)
    e = s * (6 * U * (gy.abs() + a.abs()) + (9 * U) * (xh * b).abs() + ea + xh.abs() * eb)
    check("dx", dx, ref.rounded((want, e), dt))
    terms = dy.double() * xh
    check("dgamma", dgamma, ref.rounded((terms.sum(0), (rows + 4) * U * terms.abs().sum(0)), dt))
    check("dbeta", dbeta, ref.rounded((dy.double().sum(0), rows * U * dy.double().abs().sum(0)), dt))


# ---- linear: split pair tiles and their finish kernel -----------------------------

SPLIT = [
    (139, 3520, 4536),   # 256 columns, three splits
    (137, 6600, 3120),   # 256 columns, nine splits (eight threads for four columns)
    (2843, 5056, 272),   # 128 columns, two splits
    (139, 3519, 4535),   # odd widths
    (133, 7687, 3127),
]


@pytest.mark.parametrize("rows,k,n", SPLIT)
@pytest.mark.parametrize("dt,out_dt", [(BF16, BF16), (FP16, FP16), (BF16, FP32)])
@pytest.mark.parametrize("act", ["none", "gelu"])
def test_linear_split_tiles(rows, k, n, dt, out_dt, act):
    x, W = normal(1, rows, k, dt=dt), normal(2, k, n, scale=k ** -0.5, dt=dt)
    b, res = normal(3, n, dt=dt), normal(4, rows, n, dt=out_dt)
    out, kept = blank(rows, n, out_dt)
    train = out_dt == dt
    with route.LinearPlan(rows, k, n, dt, act=act, out_dtype=out_dt, train=train) as plan:
        saved = plan.new_saved() if train else None
        route.linear_forward(plan, x, W, out, bias=b, residual=res, saved=saved)
        bare, bare_kept = blank(rows, n, out_dt)
        route.linear_forward(plan, x, W, bare)
        if train and act != "none":
            dout = normal(5, rows, n, dt=dt)
            db = torch.full((n,), float("nan"), dtype=dt, device=DEV)
            route.linear_backward(plan, dout, x, W, saved=saved, dbias=db)
        inplace = res.clone()
        route.linear_forward(plan, x, W, inplace, bias=b, residual=inplace)
        plan.status()
    assert kept() and bare_kept()
    want, z = ref.linear(x, W, b, res, act, dt, out_dt)
    check("out", out, want)
    check("bare", bare, ref.linear(x, W, None, None, act, dt, out_dt)[0])
    if train and act != "none":  # z as the finish kernel kept it
        check("dbias", db, ref.linear_grads(x, W, z, dout, act, dt)["dbias"])
    assert torch.equal(inplace, out)


# ---- FP32 results of large tiles --------------------------------------------------

@pytest.mark.parametrize("rows,k,n", [
    (266, 64, 5336), (1097, 72, 3528),   # 256 columns
    (3512, 64, 136), (2466, 64, 144),    # 128 columns
    (1097, 73, 3527), (3512, 63, 137),   # odd widths
    (20, 896, 448), (130, 1001, 517),    # small tiles
])
@pytest.mark.parametrize("act", ["none", "silu"])
@pytest.mark.parametrize("pad,offset", [(0, 0), (4, 4), (1, 3)])
def test_linear_fp32_results(rows, k, n, act, pad, offset):
    x, W = normal(1, rows, k), normal(2, k, n, scale=k ** -0.5)
    b = normal(3, n)
    res = normal(4, rows, n, dt=FP32, pad=pad, offset=offset)
    with route.LinearPlan(rows, k, n, BF16, act=act, out_dtype=FP32) as plan:
        for bias, residual in ((b, res), (None, res), (b, None), (None, None)):
            out, kept = blank(rows, n, FP32, pad, offset)
            route.linear_forward(plan, x, W, out, bias=bias, residual=residual)
            plan.status()
            check("out", out, ref.linear(x, W, bias, residual, act, BF16, FP32)[0])
            assert kept()


# ---- gated: pair tiles of both widths, whole and split ------------------------------

GATED = [
    (280, 64, 2728, 208),     # gate and up: 256 columns, whole
    (2048, 512, 4096, 512),   # the same, and d gate: 256 columns, whole; several tiles a pair
    (2053, 520, 4001, 504),
    (3589, 64, 72, 120),      # 128 columns, whole
    (131, 2984, 2312, 584),   # gate and up: 256 columns, four splits
    (139, 7392, 1568, 216),   # nine splits
    (139, 2983, 2311, 583),
    (2999, 5456, 136, 1408),  # 128 columns, two splits
    (3989, 528, 136, 4784),   # d gate: 256 columns, three splits
    (2791, 296, 264, 5696),   # d gate: 128 columns, two splits
    (3989, 527, 135, 4783),
    (527, 688, 3400, 64),     # d gate: 256 columns, whole
]


@pytest.mark.parametrize("rows,k,f,n", GATED)
@pytest.mark.parametrize("dt,act", [(BF16, "silu"), (FP16, "gelu")])
def test_gated_pair_tiles(rows, k, f, n, dt, act):
    x = normal(1, rows, k, dt=dt)
    Wg, Wu, Wd = (normal(i, a, b, scale=a ** -0.5, dt=dt) for i, a, b in ((2, k, f), (3, k, f), (4, f, n)))
    res, dout = normal(5, rows, n, dt=dt), normal(6, rows, n, scale=0.1, dt=dt)
    names = ("out", "again", "dx", "dW_gate", "dW_up", "dW_down")
    bufs = {name: blank(*shape, dt) for name, shape in zip(
        names, ((rows, n), (rows, n), (rows, k), (k, f), (k, f), (f, n)))}
    o = {name: b[0] for name, b in bufs.items()}
    with route.GatedPlan(rows, k, f, n, dt, act=act, train=True) as plan:
        saved = plan.new_saved()
        route.gated_forward(plan, x, Wg, Wu, Wd, o["out"], residual=res, saved=saved)
        route.gated_forward(plan, x, Wg, Wu, Wd, o["again"], residual=res)  # nothing kept
        route.gated_backward(plan, dout, x, Wg, Wu, Wd, saved, **{m: o[m] for m in names[2:]})
        plan.status()
    assert torch.equal(o["out"], o["again"])
    want, kept = ref.gated(x, Wg, Wu, Wd, res, act, dt)
    check("out", o["out"], want)
    grads = ref.gated_grads(x, Wg, Wu, Wd, kept, dout, act, dt)
    for m in names[2:]:
        check(m, o[m], grads[m])
    for name, (_, whole) in bufs.items():
        assert whole(), name
