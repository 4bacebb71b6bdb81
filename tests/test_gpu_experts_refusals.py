"""What a refused call of the routed experts' operators names is the argument that
the call has."""

import pytest
import torch

import latent_projection_top_gb300 as route
from gpu_util import DEV, require_gpu

pytestmark = pytest.mark.gpu

BF16, I32 = torch.bfloat16, torch.int32


@pytest.fixture(scope="module", autouse=True)
def _gpu():
    require_gpu()


def test_gather_gradient_names_its_own_arguments():
    rows = torch.zeros((8, 64), dtype=BF16, device=DEV)
    flat = torch.zeros((1, 64), dtype=BF16, device=DEV)
    place = torch.zeros((4, 2), dtype=I32, device=DEV)
    with route.DispatchPlan(4, 64, BF16, experts=8, topk=2) as plan:
        with pytest.raises(route.RouteError, match="dout: row stride"):
            route.dispatch_gather_backward(plan, flat.expand(8, 64), place, rows[:4])
        with pytest.raises(route.RouteError, match="dx: row stride"):
            route.dispatch_gather_backward(plan, rows, place, flat.expand(4, 64))
        with pytest.raises(route.RouteError, match=r"\by: row stride"):
            route.dispatch_combine(plan, flat.expand(8, 64), place, None, rows[:4])
        with pytest.raises(route.RouteError, match="out: row stride"):
            route.dispatch_combine(plan, rows, place, None, flat.expand(4, 64))
        lib, p, null = route.lib(), plan.handle, None
        assert lib.route_dispatch_gather_backward(p, 4, null, 64, 8, place.data_ptr(), rows.data_ptr(), 64, null) == 3
        assert route.lib().route_last_error() == b"dout must be non-NULL"
        assert lib.route_dispatch_gather_backward(p, 4, rows.data_ptr(), 64, 8, place.data_ptr(), null, 64, null) == 3
        assert route.lib().route_last_error() == b"dx must be non-NULL"
