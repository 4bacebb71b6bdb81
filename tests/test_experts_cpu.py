"""The routed experts' operators and dropout on a machine without a GPU: the
declared entry points are exported, bad arguments are refused before a device
is touched, and the plain forms that the GPU tests compare with are checked."""

import ctypes
import os
import re

import numpy as np
import pytest
import torch

import experts_ref
import latent_projection_top_gb300 as route
from latent_projection_top_gb300 import experts

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
HEADER = os.path.join(ROOT, "include", "route_experts.h")
BF16 = torch.bfloat16


@pytest.fixture(scope="module")
def lib():
    route.build()
    return route.lib()


def header():
    return re.sub(r"/\*.*?\*/", "", open(HEADER).read(), flags=re.S)


def test_header_declares_the_binding_exports_and_the_library_has_them(lib):
    fns = sorted(set(re.findall(r"^\s*route_status\s+(route_\w+)\s*\(", header(), re.M)))
    assert fns == sorted(experts.EXPORTS)
    for name in fns:
        assert hasattr(lib, name), name


def test_limits_match_the_header():
    text = header()
    for name, value in (("ROUTE_MAX_EXPERTS", route.MAX_EXPERTS), ("ROUTE_MAX_TOPK", route.MAX_TOPK),
                        ("ROUTE_EXPERTS_MAX_ROWS", route.EXPERTS_MAX_ROWS)):
        assert int(re.search(rf"{name}\s+(\d+)", text).group(1)) == value


@pytest.mark.parametrize("name,args,status", [
    # rows, dim, type, experts, first, topk, device
    ("route_dispatch_prepare", (0, 64, 0, 8, 0, 2, 0), 1),
    ("route_dispatch_prepare", (65537, 64, 0, 8, 0, 2, 0), 1),
    ("route_dispatch_prepare", (4, 0, 0, 8, 0, 2, 0), 7),
    ("route_dispatch_prepare", (4, 64, 3, 8, 0, 2, 0), 2),
    ("route_dispatch_prepare", (4, 64, 0, 0, 0, 2, 0), 7),
    ("route_dispatch_prepare", (4, 64, 0, 1025, 0, 2, 0), 7),
    ("route_dispatch_prepare", (4, 64, 0, 8, -1, 2, 0), 7),
    ("route_dispatch_prepare", (4, 64, 0, 8, 0, 0, 0), 7),
    ("route_dispatch_prepare", (4, 64, 0, 8, 0, 33, 0), 7),
    # rows, k, f, n, experts, type, act, train, device
    ("route_experts_prepare", (0, 64, 64, 64, 8, 0, 4, 0, 0), 1),
    ("route_experts_prepare", (1048577, 64, 64, 64, 8, 0, 4, 0, 0), 1),
    ("route_experts_prepare", (4, 60, 64, 64, 8, 0, 4, 0, 0), 7),
    ("route_experts_prepare", (4, 64, 65, 64, 8, 0, 4, 0, 0), 7),
    ("route_experts_prepare", (4, 64, 64, 4, 8, 0, 4, 0, 0), 7),
    ("route_experts_prepare", (4, 64, 64, 64, 0, 0, 4, 0, 0), 7),
    ("route_experts_prepare", (4, 64, 64, 64, 1025, 0, 4, 0, 0), 7),
    ("route_experts_prepare", (4, 64, 64, 64, 8, 2, 4, 0, 0), 2),
    ("route_experts_prepare", (4, 64, 64, 64, 8, 0, 6, 0, 0), 2),
    # rows, dim, type, device
    ("route_dropout_prepare", (0, 64, 0, 0), 1),
    ("route_dropout_prepare", (4, 65537, 0, 0), 7),
    ("route_dropout_prepare", (4, 64, -1, 0), 2),
])
def test_preparation_refuses(lib, name, args, status):
    h = ctypes.c_void_p(123)
    assert getattr(lib, name)(*args, ctypes.byref(h)) == status and h.value is None
    assert getattr(lib, name)(*args, None) == 3


def test_null_plans(lib):
    x = ctypes.c_void_p(0x1000)
    assert lib.route_dispatch_sort(None, 1, x, 2, x, x, x, None) == 3
    assert lib.route_dispatch_gather(None, 1, x, 8, x, 2, x, 8, None) == 3
    assert lib.route_dispatch_gather_backward(None, 1, x, 8, 2, x, x, 8, None) == 3
    assert lib.route_dispatch_combine(None, 1, x, 8, 2, x, x, x, 8, x, 8, None) == 3
    assert lib.route_dispatch_combine_backward(None, 1, x, 8, x, 8, 2, x, x, x, 8, x, None) == 3
    assert lib.route_experts_forward(None, 1, x, 8, x, *[x, 8, 64] * 3, x, 8, None, None) == 3
    assert lib.route_experts_backward(None, 1, x, 8, x, 8, x, *[x, 8, 64] * 3, x, x, 8,
                                      *[x, 8, 64] * 3, None) == 3
    assert lib.route_dropout_forward(None, 1, x, 8, 0.1, 0, 0, None, x, 8, x, 8, None) == 3
    assert lib.route_dropout_backward(None, 1, x, 8, 0.1, 0, 0, None, x, 8, None) == 3


@pytest.mark.parametrize("size", [2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8])
def test_sizes_past_32_bits_are_refused(lib, size):
    for make in (lambda: route.DispatchPlan(size, 64, BF16),
                 lambda: route.DispatchPlan(4, size, BF16),
                 lambda: route.DispatchPlan(4, 64, BF16, experts=size),
                 lambda: route.DispatchPlan(4, 64, BF16, topk=size),
                 lambda: route.ExpertsPlan(size, 64, 64, 64, 4, BF16),
                 lambda: route.ExpertsPlan(4, 64, size, 64, 4, BF16),
                 lambda: route.ExpertsPlan(4, 64, 64, 64, size, BF16),
                 lambda: route.DropoutPlan(size, 64, BF16)):
        with pytest.raises(route.RouteError, match="ROUTE_ERR_(ROWS|PLAN)"):
            make()


def test_binding_refuses_types():
    with pytest.raises(TypeError, match="dtype"):
        route.DispatchPlan(4, 8, torch.float64)
    with pytest.raises(ValueError, match="activation"):
        route.ExpertsPlan(4, 8, 8, 8, 2, BF16, act="swish")
    ids = torch.zeros((4, 2), dtype=torch.int32)
    with pytest.raises(ValueError, match="cuda:0"):
        experts._ints(ids, "place", (4, 2), 0)
    with pytest.raises(TypeError, match="must be a torch.Tensor"):
        experts._ints([1], "place", (4, 2), 0)
    with pytest.raises(ValueError, match="64 bits"):
        experts._c_u64(-1, "seed")
    with pytest.raises(ValueError, match="64 bits"):
        experts._c_u64(2 ** 64, "seed")
    assert experts._c_u64(2 ** 64 - 1, "seed") == 2 ** 64 - 1
    assert experts._opt_stack(None, "dW_up", 2, 8, 8, BF16, 0) == (None, 0, 0)


# ---- the plain forms ------------------------------------------------------------

def test_philox_known_answers():
    """The answers that the generator's authors publish with it."""
    full = 0xFFFFFFFF
    pi = (0x243F6A88, 0x85A308D3, 0x13198A2E, 0x03707344)
    for counter, key, want in (
            ((0, 0, 0, 0), (0, 0), (0x6627E8D5, 0xE169C58D, 0xBC57AC4C, 0x9B00DBD8)),
            ((full,) * 4, (full, full), (0x408F276D, 0x41C83B0E, 0xA20BC7C6, 0x6D5451FD)),
            (pi, (0xA4093822, 0x299F31D0), (0xD16CFE09, 0x94FDCCEB, 0x5001E420, 0x24126EA1))):
        got = experts_ref.philox(np.array([counter], dtype=np.uint64), key)
        assert tuple(int(v) for v in got[0]) == want


def test_lots_of_a_row_do_not_depend_on_the_others():
    a = experts_ref.lots(5, 13, 7, 100)
    b = experts_ref.lots(3, 13, 7, 104)  # rows 2.. of the first: 2 counters each
    assert np.array_equal(a[2:], b)
    wrap = experts_ref.lots(3, 8, 7, 2 ** 64 - 1)
    assert np.array_equal(wrap[1:], experts_ref.lots(2, 8, 7, 0))
    share = (experts_ref.lots(256, 1024, 3, 0) < 6554).mean()
    assert abs(share - 6554 / 65536) < 5 * (0.1 * 0.9 / 2 ** 18) ** 0.5


def test_sort_form_by_hand():
    ids = np.array([[3, 1], [5, 3], [-1, 1], [3, 3]])
    offsets, place, pairs = experts_ref.sort(ids, 3, 1)
    assert offsets.tolist() == [0, 2, 2, 6]
    assert pairs.tolist() == [1, 5, 0, 3, 6, 7]
    assert place.tolist() == [[2, 0], [-1, 3], [-1, 1], [4, 5]]


def test_combine_gradients_against_differences():
    g = torch.Generator().manual_seed(1)
    y = torch.randn((6, 5), generator=g, dtype=torch.float64)
    w = torch.rand((4, 3), generator=g)
    dout = torch.randn((4, 5), generator=g, dtype=torch.float64)
    place = torch.tensor([[0, 3, -1], [5, 1, 2], [-1, -1, -1], [4, 9, -7]], dtype=torch.int32)

    def loss(y, w):
        return float((experts_ref.combine(y, place, w, None, torch.float32)[0] * dout).sum())

    at, dy, dw = experts_ref.combine_grads(dout, y, place, w, torch.float32, 6)
    v, u = torch.randn((6, 5), generator=g, dtype=torch.float64), torch.randn((4, 3), generator=g, dtype=torch.float64)
    full = torch.zeros_like(y)
    full[at] = dy[0]
    assert abs((loss(y + v, w) - loss(y - v, w)) / 2 - float((full * v).sum())) < 1e-9
    assert abs((loss(y, w.double() + u) - loss(y, w.double() - u)) / 2 - float((dw[0] * u).sum())) < 1e-9
    assert dw[0][3, 1] == 0 and dw[0][2].abs().max() == 0
