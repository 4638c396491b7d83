"""Refusals and plans of the 8-bit products that need no GPU."""
import ctypes

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


@pytest.fixture(scope="module", autouse=True)
def lib():
    gg_build.build()
    return gg.load_library()


GOOD = dict(E=4, M_max=64, T=32, N=128, K=256, x_dtype="bf16", act=None, out_dtype="bf16")


@pytest.mark.parametrize("change,code", [
    (dict(E=0), gg.CAKE_GG_ERR_INVALID_ARG), (dict(E=1025), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(M_max=-1), gg.CAKE_GG_ERR_INVALID_ARG), (dict(M_max=2 ** 31), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(T=0), gg.CAKE_GG_ERR_INVALID_ARG), (dict(T=-1), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(N=0), gg.CAKE_GG_ERR_INVALID_ARG), (dict(K=0), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(N=12), gg.CAKE_GG_ERR_ALIGNMENT), (dict(K=24), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(K=1 << 17), gg.CAKE_GG_ERR_OVERFLOW), (dict(x_dtype=3), gg.CAKE_GG_ERR_UNSUPPORTED),
    (dict(out_dtype=2), gg.CAKE_GG_ERR_UNSUPPORTED), (dict(act=2), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(x_dtype="int8", act="silu_mul"), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(max_sms=-1), gg.CAKE_GG_ERR_INVALID_ARG),
])
def test_plan_refuses(change, code):
    with pytest.raises(gg.CakeGGError) as err:
        gg.cake_gg_i8_plan(**{**GOOD, **change})
    assert err.value.code == code


def test_plan_keeps_the_problem():
    plan = gg.cake_gg_i8_plan(**GOOD)
    d = plan.as_dict()
    assert (d["E"], d["M_max"], d["T"], d["N"], d["K"]) == (4, 64, 32, 128, 256)
    assert d["workspace_bytes"] >= 256 + 4 * 32 + 32 * 256
    ready = gg.cake_gg_i8_plan(**{**GOOD, "x_dtype": "int8"})
    assert 256 <= ready.workspace_bytes <= plan.workspace_bytes


@pytest.mark.parametrize("cap", [0, 1, 7, 100])
def test_plan_does_not_follow_the_sm_cap(cap):
    a, b = gg.cake_gg_i8_plan(**GOOD).as_dict(), gg.cake_gg_i8_plan(**GOOD, max_sms=cap).as_dict()
    a.pop("max_sms"), b.pop("max_sms")
    assert a == b


def _call(plan, **change):
    """A call with made-up addresses: it has to be refused before it enqueues anything."""
    a = dict(X=1 << 20, xs=None, rows=1 << 20, W=1 << 20, ws=1 << 20, Y=1 << 20, offsets=1 << 20, workspace=1 << 20,
             workspace_bytes=plan.workspace_bytes, stream=0)
    a.update(change)
    return gg.cake_gg_i8_gemm(plan, **a)


@pytest.mark.parametrize("change,code", [
    (dict(X=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(W=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(ws=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(Y=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(workspace=None, workspace_bytes=0), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(offsets=None), gg.CAKE_GG_ERR_INVALID_ARG),            # four experts need them
    (dict(rows=None), gg.CAKE_GG_ERR_INVALID_ARG),               # 64 rows from 32 tokens
    (dict(xs=1 << 20), gg.CAKE_GG_ERR_INVALID_ARG),              # scales with BF16 tokens
    (dict(X=(1 << 20) + 8), gg.CAKE_GG_ERR_ALIGNMENT), (dict(W=(1 << 20) + 1), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(Y=(1 << 20) + 2), gg.CAKE_GG_ERR_ALIGNMENT), (dict(ws=(1 << 20) + 2), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(rows=(1 << 20) + 1), gg.CAKE_GG_ERR_ALIGNMENT), (dict(offsets=(1 << 20) + 2), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(workspace_bytes=255), gg.CAKE_GG_ERR_WORKSPACE),
])
def test_call_refuses(change, code):
    assert _call(gg.cake_gg_i8_plan(**GOOD), **change) == code


def test_call_refuses_a_changed_plan():
    plan = gg.cake_gg_i8_plan(**GOOD)
    for field, value in (("abi_version", 9), ("N", 12), ("K", 1 << 20), ("x_dtype", 7), ("path", 9), ("T", -3)):
        other = gg.CakeGGI8Plan()
        ctypes.memmove(ctypes.byref(other), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(other, field, value)
        assert _call(other) != gg.CAKE_GG_OK


def test_int8_tokens_need_scales():
    plan = gg.cake_gg_i8_plan(**{**GOOD, "x_dtype": "int8"})
    assert _call(plan) == gg.CAKE_GG_ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(X=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(Xq=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(xs=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(K=24), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(x_dtype="int8"), gg.CAKE_GG_ERR_UNSUPPORTED), (dict(X=(1 << 20) + 4), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(act=5), gg.CAKE_GG_ERR_INVALID_ARG), (dict(T=-1), gg.CAKE_GG_ERR_INVALID_ARG),
])
def test_quant_refuses(change, code):
    a = dict(X=1 << 20, x_dtype="bf16", act=None, T=4, K=64, Xq=1 << 20, xs=1 << 20, stream=0)
    a.update(change)
    assert gg.cake_gg_i8_quant(**a) == code


def test_helpers_refuse():
    import torch
    W, ws = torch.zeros((2, 16, 32), dtype=torch.int8), torch.zeros((2, 16))
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    x = torch.zeros((4, 32), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 32), dtype=torch.int8), torch.zeros(4)
    for err, args, more in [
        (TypeError, (x.half(), W, ws), dict(offsets=off)),
        (TypeError, (x, W.float(), ws), dict(offsets=off)),
        (TypeError, (x, W, ws.double()), dict(offsets=off)),
        (TypeError, (x, W, ws), dict(offsets=off.long())),
        (TypeError, (x, W, ws), dict(offsets=off, rows=torch.zeros(4, dtype=torch.int64))),
        (ValueError, (x, W, ws), dict()),
        (ValueError, (x[:, :16], W, ws), dict(offsets=off)),
        (ValueError, (x, W, ws[:1]), dict(offsets=off)),
        (ValueError, (x, W, ws), dict(offsets=off[:2])),
        (ValueError, (x, W, ws), dict(offsets=off, act="silu_mul")),
        (ValueError, (x, W, ws), dict(offsets=off, xs=s)),
        (ValueError, (x, W, ws), dict(offsets=off, act="gelu")),
        (ValueError, (q, W, ws), dict(offsets=off)),
        (ValueError, (q, W, ws), dict(offsets=off, xs=s[:3])),
        (ValueError, (x.T.contiguous().T, W, ws), dict(offsets=off)),
        (ValueError, (x, W.transpose(1, 2).contiguous().transpose(1, 2), ws), dict(offsets=off)),
        (TypeError, (x, W, ws), dict(offsets=off, out=torch.zeros((4, 16)))),
        (ValueError, (x, W, ws), dict(offsets=off, out=torch.zeros((4, 8), dtype=torch.bfloat16))),
        (ValueError, (x, W, ws), dict(offsets=off, plan=gg.cake_gg_i8_plan(2, 8, 4, 16, 32))),
    ]:
        with pytest.raises(err):
            gg.int8_gemm(*args, **more)
    for err, args, more in [(TypeError, (x.half(),), {}), (ValueError, (x[0],), {}), (ValueError, (x[:, ::2],), {}),
                            (ValueError, (x[:, :31].contiguous(),), dict(act="silu_mul")),
                            (TypeError, (x,), dict(out=x)), (ValueError, (x,), dict(scale=s[:2]))]:
        with pytest.raises(err):
            gg.quantize_rows(*args, **more)


@pytest.mark.parametrize("E", [1, 3, 30, 400, 1024])
def test_every_plan_keeps_the_converters_within_a_round(E, monkeypatch):
    """Two converter groups take alternate stages.  In an odd ring each meets a stage's barrier every
    second round, so widened tiles may run at most stages - 2 ahead of the MMAs."""
    for splits in (None, "1", "2", "3", "5", "8"):
        if splits:
            monkeypatch.setenv("CAKE_GG_I8_SPLITS", splits)
        for M in (9, 20, 40, 70, 100, 200, 500, 1500, 6000, 40000):
            for N in (8, 136, 1000, 4096, 8192):
                for K in (16, 512, 2048, 8192):
                    if splits and int(splits) > (K + 127) // 128:
                        continue
                    plan = gg.cake_gg_i8_plan(E, M, M, N, K)
                    if plan.path == 1:
                        assert plan.stages >= 2 and plan.slots >= 2
                        assert plan.slots <= (plan.stages if plan.stages % 2 == 0 else plan.stages - 2), plan.as_dict()


def test_call_refuses_a_plan_whose_converters_could_run_a_round_ahead():
    plan = gg.cake_gg_i8_plan(**{**GOOD, "M_max": 4096, "T": 4096})
    assert plan.path == 1
    plan.stages, plan.slots = 3, 3
    assert _call(plan, rows=None) == gg.CAKE_GG_ERR_INVALID_ARG


def test_more_splits_than_stages_are_refused(monkeypatch):
    monkeypatch.setenv("CAKE_GG_I8_PAIR", "1")
    monkeypatch.setenv("CAKE_GG_I8_SPLITS", "3")
    with pytest.raises(gg.CakeGGError) as err:                    # two stages of 128
        gg.cake_gg_i8_plan(1, 4096, 4096, 128, 256)
    assert err.value.code == gg.CAKE_GG_ERR_INVALID_ARG
    assert gg.cake_gg_i8_plan(1, 4096, 4096, 128, 384).splits == 3


def test_a_first_product_where_the_token_pass_is_long(monkeypatch):
    """Plans divide long calls only, by less than all their rows, and not over a split reduction."""
    for M, N, K in ((1, 8, 16), (64, 4096, 6144), (3001, 1000, 5120)):
        assert gg.cake_gg_i8_plan(1, M, M, N, K).first_rows == 0
    for M in (16384, 20001, 1 << 20, 2 ** 31 - 1):
        for E in (1, 32):
            assert 0 < gg.cake_gg_i8_plan(E, M, M, 4096, 4096, "fp32").first_rows < M
    for value, want in (("0", 0), ("77", 77), ("4096", 0)):
        monkeypatch.setenv("CAKE_GG_I8_FIRST_ROWS", value)
        assert gg.cake_gg_i8_plan(1, 4096, 4096, 4096, 4096).first_rows == want
    monkeypatch.setenv("CAKE_GG_I8_PAIR", "1")
    monkeypatch.setenv("CAKE_GG_I8_ROWS_PER_TILE", "64")
    monkeypatch.setenv("CAKE_GG_I8_SPLITS", "2")
    monkeypatch.setenv("CAKE_GG_I8_FIRST_ROWS", "77")
    plan = gg.cake_gg_i8_plan(1, 4096, 4096, 4096, 4096)
    assert plan.splits == 2 and plan.first_rows == 0


@pytest.mark.parametrize("first", [-1, 4096, 2 ** 31 - 1])
def test_call_refuses_a_first_product_of_no_or_all_rows(first):
    plan = gg.cake_gg_i8_plan(**{**GOOD, "M_max": 4096, "T": 4096})
    plan.first_rows = first
    assert _call(plan, rows=None) == gg.CAKE_GG_ERR_INVALID_ARG
