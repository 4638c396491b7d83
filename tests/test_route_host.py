"""Refusals and plans of the routing, and of the rows' way back, that need no GPU."""
import ctypes

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

INVALID, ALIGN, OVER, KIND, WORK = (gg.CAKE_GG_ERR_INVALID_ARG, gg.CAKE_GG_ERR_ALIGNMENT, gg.CAKE_GG_ERR_OVERFLOW,
                                    gg.CAKE_GG_ERR_UNSUPPORTED, gg.CAKE_GG_ERR_WORKSPACE)
AT = 1 << 20


@pytest.fixture(scope="module", autouse=True)
def lib():
    gg_build.build()
    return gg.load_library()


@pytest.mark.parametrize("sizes,code", [
    ((-1, 8, 2), INVALID), ((4, 0, 1), INVALID), ((4, 1025, 2), INVALID), ((4, 8, 0), INVALID), ((4, 8, 9), INVALID), ((4, 64, 33), INVALID),
    ((2 ** 23 + 1, 8, 1), OVER), ((2 ** 40, 8, 1), OVER),
])
def test_plan_refuses(sizes, code):
    with pytest.raises(gg.CakeGGError) as err:
        gg.cake_gg_route_plan(*sizes)
    assert err.value.code == code


def test_plans_cover_their_tokens():
    for T in list(range(0, 700)) + [1000, 4096, 16384, 155648, 155649, 2 ** 20 + 7, 2 ** 23]:
        d = gg.cake_gg_route_plan(T, 1024, 32).as_dict()
        assert d["blocks"] * d["block_tokens"] >= T and (d["blocks"] - 1) * d["block_tokens"] < max(T, 1)
        assert 1 <= d["blocks"] <= (8 if d["cluster"] else 152) and d["block_tokens"] < 2 ** 16
        assert d["workspace_bytes"] >= 256 + (0 if d["cluster"] else d["blocks"] * 1024 * 2)


def _options(**change):
    o = dict(score=0, groups=1, top_groups=1, group_score=0, renormalize=1, scale=1.0)
    o.update(change)
    return gg.CakeGGRouteOptions(*o.values())


def _route(plan, options=None, **change):
    a = dict(logits=AT, logits_dtype="fp32", row_stride=plan.E, bias=AT, expert=AT, weight=AT, offsets=AT, rows=AT, position=AT,
             workspace=AT, workspace_bytes=plan.workspace_bytes, stream=0)
    a.update(change)
    return gg.cake_gg_route(plan, options or _options(), **a)


@pytest.mark.parametrize("change,code", [
    (dict(logits=None), INVALID), (dict(expert=None), INVALID), (dict(weight=None), INVALID), (dict(offsets=None), INVALID),
    (dict(rows=None), INVALID), (dict(position=None), INVALID), (dict(workspace=None, workspace_bytes=0), INVALID),
    (dict(row_stride=63), INVALID), (dict(row_stride=2 ** 62), INVALID), (dict(logits_dtype=2), KIND), (dict(logits=AT + 2), ALIGN),
    (dict(bias=AT + 1), ALIGN), (dict(expert=AT + 2), ALIGN), (dict(offsets=AT + 1), ALIGN), (dict(workspace=AT + 8), ALIGN),
    (dict(workspace_bytes=255), WORK),
])
def test_route_refuses(change, code):
    assert _route(gg.cake_gg_route_plan(9, 64, 4), **change) == code


@pytest.mark.parametrize("change", [
    dict(score=2), dict(groups=0), dict(groups=33), dict(groups=3), dict(groups=8, top_groups=0), dict(groups=8, top_groups=9),
    dict(groups=32, top_groups=1), dict(group_score=2), dict(groups=64, group_score=1),
])
def test_options_are_refused(change):
    """64 experts, four of them chosen."""
    assert _route(gg.cake_gg_route_plan(9, 64, 4), _options(**change)) == INVALID


def test_two_largest_of_groups_of_one():
    assert _route(gg.cake_gg_route_plan(9, 16, 4), _options(groups=16, top_groups=8, group_score=1)) == INVALID


def test_route_refuses_a_changed_plan():
    plan = gg.cake_gg_route_plan(1000, 64, 4)
    for field, value in (("abi_version", 9), ("E", 0), ("T", -1), ("T", 1001), ("top_k", 65), ("blocks", 1), ("block_tokens", 3), ("cluster", 1),
                         ("workspace_bytes", 256)):
        other = gg.CakeGGRoutePlan()
        ctypes.memmove(ctypes.byref(other), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(other, field, value)
        assert _route(other, workspace_bytes=1 << 40) != gg.CAKE_GG_OK, field


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(E=0), INVALID), (dict(top_k=9), INVALID), (dict(score=3), INVALID), (dict(logits=None), INVALID),
    (dict(expert=None), INVALID), (dict(d_weight=None), INVALID), (dict(d_logits=None), INVALID), (dict(row_stride=7), INVALID),
    (dict(logits_dtype=2), KIND), (dict(d_logits=AT + 2), ALIGN), (dict(T=2 ** 23 + 1), OVER),
])
def test_route_grad_refuses(change, code):
    a = dict(T=4, E=8, top_k=2, score=0, renormalize=1, scale=1.0, logits=AT, logits_dtype="fp32", row_stride=8, expert=AT, d_weight=AT,
             d_logits=AT, stream=0)
    a.update(change)
    assert gg.cake_gg_route_grad(**a) == code


@pytest.mark.parametrize("change,code", [
    (dict(T=-1), INVALID), (dict(M=-1), INVALID), (dict(T=2 ** 31), INVALID), (dict(M=2 ** 31), INVALID), (dict(top_k=0), INVALID),
    (dict(top_k=33), INVALID), (dict(K=0), INVALID), (dict(K=12), ALIGN), (dict(K=2 ** 20 + 8), OVER), (dict(rows_dtype=2), KIND),
    (dict(out_dtype=3), KIND), (dict(rows=None), INVALID), (dict(position=None), INVALID), (dict(rows=AT + 8), ALIGN), (dict(position=AT + 2), ALIGN),
    (dict(weight=AT + 1), ALIGN),
])
def test_combine_refuses(change, code):
    a = dict(T=4, M=8, top_k=2, K=64, rows=AT, rows_dtype="bf16", position=AT, weight=AT, out=AT, out_dtype="bf16", stream=0)
    a.update(change)
    assert gg.cake_gg_combine_rows(**a) == code
    b = dict(a, d_out=AT, d_rows=AT, d_weight=AT)
    b.pop("out")
    assert gg.cake_gg_combine_grad(**b) == code


def test_combine_refuses_its_own():
    a = dict(T=4, M=8, top_k=2, K=64, rows=AT, rows_dtype="bf16", position=AT, weight=AT, stream=0)
    assert gg.cake_gg_combine_rows(**a, out=None, out_dtype="bf16") == INVALID
    assert gg.cake_gg_combine_rows(**a, out=AT + 4, out_dtype="bf16") == ALIGN
    for change in (dict(d_out=None), dict(d_rows=None), dict(rows=None)):
        b = {**a, "d_out": AT, "out_dtype": "bf16", "d_rows": AT, "d_weight": AT, **change}
        assert gg.cake_gg_combine_grad(**b) == INVALID


def test_helpers_refuse():
    import torch
    i32 = torch.int32
    l, e, w = torch.zeros(4, 8), torch.zeros((4, 2), dtype=i32), torch.zeros(4, 2)
    r = torch.zeros((8, 16), dtype=torch.bfloat16)
    routing = gg.empty_routing(4, 8, 2, "cpu")
    for err, call in [
        (TypeError, lambda: gg.route(l.half(), 2)), (ValueError, lambda: gg.route(l[0], 2)), (ValueError, lambda: gg.route(l.T, 2)),
        (ValueError, lambda: gg.route(l[:, ::2], 2)), (ValueError, lambda: gg.route(l[:1].expand(4, 8), 2)),
        (ValueError, lambda: gg.route(l, 2, score="relu")), (ValueError, lambda: gg.route(l, 2, group_score="mean")),
        (gg.CakeGGError, lambda: gg.route(l, 9)), (ValueError, lambda: gg.route(l, 2, bias=torch.zeros(7))),
        (TypeError, lambda: gg.route(l, 2, bias=torch.zeros(8).double())), (ValueError, lambda: gg.route(l, 2, plan=gg.cake_gg_route_plan(5, 8, 2))),
        (ValueError, lambda: gg.route(l, 2, out=gg.empty_routing(5, 8, 2, "cpu"))),
        (TypeError, lambda: gg.route(l, 2, out=routing._replace(weight=routing.expert))), (ValueError, lambda: gg.route(l, 2)),
        (ValueError, lambda: gg.route(l, 2, out=routing)),
        (TypeError, lambda: gg.route_grad(l, e.long(), w)), (ValueError, lambda: gg.route_grad(l, e, w[:, :1])),
        (ValueError, lambda: gg.route_grad(l, e[0], w)), (ValueError, lambda: gg.route_grad(l, e, w, score="x")),
        (TypeError, lambda: gg.route_grad(l, e, w, out=l.bfloat16())), (ValueError, lambda: gg.route_grad(l, e, w)),
        (TypeError, lambda: gg.combine_rows(r.half(), e)), (ValueError, lambda: gg.combine_rows(r[0], e)),
        (ValueError, lambda: gg.combine_rows(r.T, e)), (TypeError, lambda: gg.combine_rows(r, e.long())), (ValueError, lambda: gg.combine_rows(r, e[0])),
        (ValueError, lambda: gg.combine_rows(r, e, w[:3])), (TypeError, lambda: gg.combine_rows(r, e, w.double())),
        (TypeError, lambda: gg.combine_rows(r, e, w, out=torch.zeros(4, 16))), (ValueError, lambda: gg.combine_rows(r, e, w)),
        (ValueError, lambda: gg.combine_grad(r[:4], r, e, None)), (ValueError, lambda: gg.combine_grad(r[:3], r, e, w)),
        (ValueError, lambda: gg.combine_grad(r[:4], r[:7], e, w)), (TypeError, lambda: gg.combine_grad(r[:4].half(), r, e, w)),
        (ValueError, lambda: gg.combine_grad(r[:4], r, e, w)),
        (ValueError, lambda: gg.gather_rows(r[:3], e)), (TypeError, lambda: gg.gather_rows(r[:4].int(), e)),
        (ValueError, lambda: gg.gather_rows(r[:4], e, out=r[:7])), (ValueError, lambda: gg.gather_rows(r[:4], e)),
    ]:
        with pytest.raises(err):
            call()
