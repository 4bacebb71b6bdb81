"""The layer operators' C ABI and binding on a machine without a GPU: every
declared entry point is exported and bad arguments are refused with status
codes before a device is touched.  The float64 forms that the GPU tests
compare with are checked here against differences."""

import ctypes
import os
import re

import pytest
import torch

import latent_projection_top_gb300 as route
import layer_ref as ref
from latent_projection_top_gb300 import layer

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "route_layer.h")


@pytest.fixture(scope="module")
def lib():
    route.build()
    return route.lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_declares_the_binding_exports_and_the_library_has_them(lib):
    fns = sorted(set(re.findall(r"^\s*(?:route_status|int64_t)\s+(route_\w+)\s*\(", header(), re.M)))
    assert fns == sorted(layer.EXPORTS)
    for name in fns:
        assert hasattr(lib, name), name


def test_limits_and_activations_match_the_header():
    text = header()
    for name, value in (("ROUTE_LAYER_MAX_ROWS", route.LAYER_MAX_ROWS),
                        ("ROUTE_LAYER_MAX_WIDTH", route.LAYER_MAX_WIDTH),
                        ("ROUTE_NORM_MAX_WIDTH", route.NORM_MAX_WIDTH)):
        assert int(re.search(rf"{name}\s+(\d+)", text).group(1)) == value
    acts = re.findall(r"ROUTE_ACT_(\w+)\s*=\s*(\d+)", text)
    assert [a.lower() for a, _ in sorted(acts, key=lambda x: int(x[1]))] == list(route.ACTIVATIONS)


def prepare(lib, name, *args):
    h = ctypes.c_void_p(123)
    st = getattr(lib, name)(*args, ctypes.byref(h))
    return st, h.value


@pytest.mark.parametrize("name,args,status", [
    ("route_norm_prepare", (0, 64, 0, 0), 1),           # rows
    ("route_norm_prepare", (65537, 64, 0, 0), 1),
    ("route_norm_prepare", (4, 0, 0, 0), 7),            # width
    ("route_norm_prepare", (4, 16385, 0, 0), 7),
    ("route_norm_prepare", (4, 64, 3, 0), 2),           # type
    ("route_linear_prepare", (-1, 8, 8, 0, 0, 0, 0, 0), 1),
    ("route_linear_prepare", (4, 0, 8, 0, 0, 0, 0, 0), 7),
    ("route_linear_prepare", (4, 8, 65537, 0, 0, 0, 0, 0), 7),
    ("route_linear_prepare", (4, 8, 8, 2, 2, 0, 0, 0), 2),   # FP32 operands
    ("route_linear_prepare", (4, 8, 8, 0, 1, 0, 0, 0), 2),   # BF16 in, FP16 out
    ("route_linear_prepare", (4, 8, 8, 0, 0, 6, 0, 0), 2),   # activation
    ("route_linear_prepare", (4, 8, 8, 0, 2, 0, 1, 0), 7),   # training with FP32 out
    ("route_gated_prepare", (4, 8, 0, 8, 0, 4, 0, 0), 7),
    ("route_gated_prepare", (4, 8, 8, 8, 2, 4, 0, 0), 2),
    ("route_gated_prepare", (4, 8, 8, 8, 0, -1, 0, 0), 2),
])
def test_preparation_refuses(lib, name, args, status):
    assert prepare(lib, name, *args) == (status, None)
    assert lib.route_last_error()


def test_null_plans_and_null_out(lib):
    x = ctypes.c_void_p(0x1000)
    assert lib.route_norm_prepare(4, 64, 0, 0, None) == 3
    assert lib.route_layer_destroy(None) == 0
    assert lib.route_layer_status(None) == 3
    assert lib.route_layer_saved_bytes(None, 4) == -1
    assert lib.route_layer_test_stall(None, 1, 0) == 3
    assert lib.route_norm_forward(None, 1, x, 8, x, x, 1e-5, x, 8, None, None) == 3
    assert lib.route_norm_backward(None, 1, x, 8, x, 8, x, x, x, 8, x, x, None) == 3
    assert lib.route_linear_forward(None, 1, x, 8, x, 8, x, x, 8, x, 8, None, None) == 3
    assert lib.route_linear_backward(None, 1, x, 8, x, 8, x, 8, x, x, 8, x, 8, x, None) == 3
    assert lib.route_gated_forward(None, 1, x, 8, x, 8, x, 8, x, 8, x, 8, x, 8, None, None) == 3
    assert lib.route_gated_backward(None, 1, x, 8, x, 8, x, 8, x, 8, x, 8, x, x, 8, x, 8, x, 8, x,
                                    8, None) == 3


def test_valid_request_without_gpu_fails_loudly(lib):
    if torch.cuda.is_available():
        pytest.skip("a GPU is present")
    st, h = prepare(lib, "route_linear_prepare", 4, 64, 64, 0, 0, 0, 0, 0)
    assert st in (5, 8) and h is None


def test_binding_refuses_types_and_activations():
    with pytest.raises(TypeError, match="dtype"):
        route.LinearPlan(4, 8, 8, torch.float64)
    with pytest.raises(ValueError, match="activation"):
        route.GatedPlan(4, 8, 8, 8, torch.bfloat16, act="swish")
    cpu = torch.zeros((4, 8), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cuda:0"):
        layer._mat(cpu, "x", 4, 8, torch.bfloat16, 0)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        layer._mat([1], "x", 4, 8, torch.bfloat16, 0)
    assert layer._opt_mat(None, "residual", 4, 8, torch.bfloat16, 0) == (None, 0)


# ---- the reference forms themselves -------------------------------------------

def rand(seed, *shape):
    g = torch.Generator()
    g.manual_seed(seed)
    return torch.randn(shape, generator=g, dtype=torch.float64)


@pytest.mark.parametrize("act", [a for a in route.ACTIVATIONS if a != "relu"])
def test_reference_gradients_against_differences(act):
    """Central differences of sum(dout * out): error h^2 times the third
    derivative, and 2^-52 / h of the sum's terms (h = 1e-5: about 1e-9)."""
    R, k, f, n = 5, 4, 6, 3
    x, Wg, Wu, Wd, dout = rand(1, R, k), rand(2, k, f), rand(3, k, f), rand(4, f, n), rand(5, R, n)
    dt = torch.float32

    def loss(p):
        return float((dout * ref.gated(*p, None, act, dt)[0][0]).sum())

    kept = ref.gated(x, Wg, Wu, Wd, None, act, dt)[1]
    grads = ref.gated_grads(x, Wg, Wu, Wd, kept, dout, act, dt)
    for i, name in enumerate(("dx", "dW_gate", "dW_up", "dW_down")):
        p = [x, Wg, Wu, Wd]
        v = rand(9 + i, *p[i].shape)
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-5 * v, p[i] - 1e-5 * v
        diff = (loss(hi) - loss(lo)) / 2e-5
        assert abs(diff - float((grads[name][0] * v).sum())) < 1e-6 * (1 + abs(diff)), name

    W, b = rand(6, k, n), rand(7, n)
    z = ref.linear(x, W, b, None, act, dt)[1]
    grads = ref.linear_grads(x, W, z, dout, act, dt)
    for i, name in enumerate(("dx", "dW", "dbias")):
        p = [x, W, b]
        v = rand(19 + i, *p[i].shape)
        hi, lo = list(p), list(p)
        hi[i], lo[i] = p[i] + 1e-5 * v, p[i] - 1e-5 * v
        diff = (float((dout * ref.linear(*hi, None, act, dt)[0][0]).sum())
                - float((dout * ref.linear(*lo, None, act, dt)[0][0]).sum())) / 2e-5
        assert abs(diff - float((grads[name][0] * v).sum())) < 1e-6 * (1 + abs(diff)), name


def test_reference_bound_sees_a_dropped_term():
    """A product that leaves out one of its K terms, or the bias, is outside
    the bound (the mistake is planted in the oracle)."""
    x, W = rand(1, 6, 64).bfloat16(), (rand(2, 64, 40) / 8).bfloat16()
    b = rand(3, 40).bfloat16()
    want, _ = ref.linear(x, W, b, None, "none", torch.bfloat16)
    good = want[0].bfloat16()
    assert ref.worst(good, want) <= 1
    assert ref.worst((want[0] - x[:, 9:10].double() @ W[9:10].double()).bfloat16(), want) > 1
    assert ref.worst((want[0] - b.double()).bfloat16(), want) > 1
    assert ref.worst(torch.full_like(good, float("nan")), want) == float("inf")


def test_short_way_leaves_what_is_not_plain_to_the_checks(lib):
    """The compiled module of the calls refuses with -1 and raises nothing."""
    from latent_projection_top_gb300 import layer
    short = layer._short_way()
    bf16 = torch.bfloat16
    plan = (1, 0, 0, 0, 8, 16, 8, 64)  # never passed on: no tensor here is on a GPU
    x, W = torch.zeros(4, 8, dtype=bf16), torch.zeros(8, 8, dtype=bf16)
    v, stats = torch.zeros(8, dtype=bf16), torch.zeros(4, 2)
    for call in (
        lambda: short.norm_forward(),
        lambda: short.norm_forward(plan),
        lambda: short.norm_forward(plan, x, v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward(None, x, v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward(("a",) * 8, x, v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward((0,) * 8, x, v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward(plan, None, v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward(plan, [1], v, v, "x", stats, "eps", None),
        lambda: short.norm_forward(plan, x.to_sparse(), v, v, x, stats, 1e-5, 0),
        lambda: short.norm_forward(plan, torch.empty(4, 8, dtype=bf16, device="meta"), v, v, x,
                                   stats, 1e-5, 0),
        lambda: short.norm_backward(plan, x, x, v, stats, None, None, None, 0),
        lambda: short.linear_forward(plan, x, W, x, None, None, None, 0),
        lambda: short.linear_backward(plan, x, x, W, None, None, None, None, 0),
        lambda: short.gated_forward(plan, x, W, W, W, x, None, None, 0),
        lambda: short.gated_backward(plan, x, x, W, W, W, None, None, None, None, None, 0),
    ):
        assert call() == -1
    with pytest.raises(TypeError):
        short.bind(1)
