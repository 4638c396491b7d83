"""Options of a routing call are that call's, whatever was asked before."""
import math

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


def test_scales_that_compare_equal():
    gg_build.build()
    seen = []

    class Library:
        def cake_gg_route(self, plan, options, *rest):
            seen.append(options._obj.scale)
            return gg.CAKE_GG_OK

    import torch
    logits = torch.zeros(4, 8)
    plan, routing = gg.cake_gg_route_plan(4, 8, 2), gg.empty_routing(4, 8, 2, "cpu")
    with pytest.MonkeyPatch.context() as m:
        m.setattr(gg, "_lib", Library())
        m.setattr(gg, "_here", lambda tensor: 0)
        for scale in (0.0, -0.0, 0.0, 2.5, math.inf, math.nan):
            gg.route(logits, 2, scale=scale, plan=plan, workspace=gg.make_workspace(plan, "cpu"), out=routing, stream=1)
            assert math.copysign(1.0, seen[-1]) == math.copysign(1.0, scale)
            assert seen[-1] == scale or (math.isnan(scale) and math.isnan(seen[-1]))
