"""Sizes that 32 bits do not hold are refused, not cut to their low bits."""

import types

import pytest
import torch

import latent_projection_top_gb300 as route
from latent_projection_top_gb300 import layer

BF16 = torch.bfloat16


@pytest.fixture(scope="module", autouse=True)
def _built():
    route.build()


@pytest.mark.parametrize("rows", [2 ** 32 + 4, 2 ** 31, -2 ** 32 + 4, 2 ** 64 + 1])
def test_rows_of_a_plan(rows):
    for make in (lambda: route.NormPlan(rows, 64, BF16),
                 lambda: route.LinearPlan(rows, 64, 64, BF16),
                 lambda: route.GatedPlan(rows, 64, 64, 64, BF16)):
        with pytest.raises(route.RouteError, match="ROUTE_ERR_ROWS"):
            make()


@pytest.mark.parametrize("width", [2 ** 32 + 8, 2 ** 31, -2 ** 32 + 8])
def test_widths_of_a_plan(width):
    for make in (lambda: route.NormPlan(4, width, BF16),
                 lambda: route.LinearPlan(4, width, 64, BF16),
                 lambda: route.LinearPlan(4, 64, width, BF16),
                 lambda: route.GatedPlan(4, width, 64, 64, BF16),
                 lambda: route.GatedPlan(4, 64, width, 64, BF16),
                 lambda: route.GatedPlan(4, 64, 64, width, BF16)):
        with pytest.raises(route.RouteError, match="ROUTE_ERR_PLAN"):
            make()


def test_rows_of_a_call(monkeypatch):
    """What reaches the library of a call of 2**32 + 4 rows is no valid number."""
    seen = []
    monkeypatch.setattr(layer._route, "_lib", types.SimpleNamespace(
        route_norm_forward=lambda handle, rows, *a: seen.append(rows) or 0))
    layer._call("route_norm_forward", types.SimpleNamespace(_p=1), 2 ** 32 + 4)
    assert seen == [2 ** 31 - 1] and seen[0] > route.LAYER_MAX_ROWS
