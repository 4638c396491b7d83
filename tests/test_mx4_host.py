"""Refusals and plans of the 4-bit products that need no GPU."""
import ctypes
import itertools

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
    (dict(N=12), gg.CAKE_GG_ERR_ALIGNMENT), (dict(K=48), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(K=1 << 17), gg.CAKE_GG_ERR_OVERFLOW), (dict(x_dtype="bf16", N=2 ** 31 - 8), gg.CAKE_GG_ERR_OVERFLOW),
    (dict(E=1024, N=1 << 24, K=1 << 16), gg.CAKE_GG_ERR_OVERFLOW),      # scale tiles past 2^31
    (dict(x_dtype=gg.CAKE_GG_INT8), gg.CAKE_GG_ERR_UNSUPPORTED), (dict(x_dtype=4), gg.CAKE_GG_ERR_UNSUPPORTED),
    (dict(out_dtype=2), gg.CAKE_GG_ERR_UNSUPPORTED), (dict(act=2), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(x_dtype="mx4", act="silu_mul"), gg.CAKE_GG_ERR_INVALID_ARG), (dict(max_sms=-1), gg.CAKE_GG_ERR_INVALID_ARG),
])
def test_plan_refuses(change, code):
    with pytest.raises(gg.CakeGGError) as err:
        gg.cake_gg_mx4_plan(**{**GOOD, **change})
    assert err.value.code == code


def test_every_plan_can_run():
    """Over the range of sizes the plan is one that the kernel takes, and its workspace holds what the call lays out."""
    for E, M, N, K in itertools.product((1, 2, 32, 1024), (1, 9, 64, 700, 5000, 70000, 2 ** 31 - 1), (8, 1000, 6144), (32, 544, 8192, 131040)):
        for x_dtype, routed in (("mx4", False), ("bf16", True)):
            plan = gg.cake_gg_mx4_plan(E, M, max(1, M // 2) if routed else M, N, K, x_dtype)
            d = plan.as_dict()
            assert d["pair"] in (1, 2) and 32 <= d["tile_rows"] <= 192 and d["tile_rows"] % 32 == 0
            assert 3 <= d["stages"] <= 12 and 1 <= d["splits"] <= 8 and (d["splits"] == 1 or d["pair"] == 1)
            least = 256
            if x_dtype == "bf16":
                T = max(1, M // 2)
                least += -(-T // 128) * -(-K // 128) * 512 + T * K // 2
            if d["pair"] == 2:
                least += (M // d["tile_rows"] + E) * -(-K // 128) * 512 * (2 if d["tile_rows"] > 128 else 1) + M * K // 2
            assert d["workspace_bytes"] >= least


@pytest.mark.parametrize("cap", [0, 1, 7, 100])
def test_plan_does_not_follow_the_sm_cap(cap):
    a, b = gg.cake_gg_mx4_plan(**GOOD).as_dict(), gg.cake_gg_mx4_plan(**GOOD, max_sms=cap).as_dict()
    a.pop("max_sms"), b.pop("max_sms")
    assert a == b


def test_overrides(monkeypatch):
    """Ones that the kernel cannot take change nothing or are refused."""
    plain = gg.cake_gg_mx4_plan(**GOOD).as_dict()
    for name, value in (("ROWS_PER_TILE", "224"), ("ROWS_PER_TILE", "40"), ("SPLITS", "9"), ("SPLITS", "0"), ("PAIR", "3")):
        with monkeypatch.context() as m:
            m.setenv("CAKE_GG_MX4_" + name, value)
            d = gg.cake_gg_mx4_plan(**GOOD).as_dict()
            assert d["tile_rows"] % 32 == 0 and d["tile_rows"] <= 192 and 1 <= d["splits"] <= 8 and d["pair"] in (1, 2)
    monkeypatch.setenv("CAKE_GG_MX4_SPLITS", "8")                # of one stage
    with pytest.raises(gg.CakeGGError):
        gg.cake_gg_mx4_plan(**GOOD)
    assert plain["workspace_bytes"] >= 256


def _call(plan, **change):
    """A call with made-up addresses: it has to be refused before it enqueues anything."""
    a = dict(X=1 << 20, xs=None, rows=1 << 20, W=1 << 20, ws=1 << 20, Y=1 << 20, offsets=1 << 20, workspace=1 << 20,
             workspace_bytes=plan.workspace_bytes, stream=0)
    a.update(change)
    return gg.cake_gg_mx4_gemm(plan, **a)


@pytest.mark.parametrize("change,code", [
    (dict(X=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(W=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(ws=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(Y=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(workspace=None, workspace_bytes=0), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(offsets=None), gg.CAKE_GG_ERR_INVALID_ARG),            # four experts need them
    (dict(rows=None), gg.CAKE_GG_ERR_INVALID_ARG),               # 64 rows from 32 tokens
    (dict(xs=1 << 20), gg.CAKE_GG_ERR_INVALID_ARG),              # scales with BF16 tokens
    (dict(X=(1 << 20) + 8), gg.CAKE_GG_ERR_ALIGNMENT), (dict(W=(1 << 20) + 1), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(Y=(1 << 20) + 2), gg.CAKE_GG_ERR_ALIGNMENT), (dict(ws=(1 << 20) + 4), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(rows=(1 << 20) + 1), gg.CAKE_GG_ERR_ALIGNMENT), (dict(offsets=(1 << 20) + 2), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(workspace_bytes=255), gg.CAKE_GG_ERR_WORKSPACE),
])
def test_call_refuses(change, code):
    assert _call(gg.cake_gg_mx4_plan(**GOOD), **change) == code


def test_call_refuses_a_changed_plan():
    plan = gg.cake_gg_mx4_plan(**GOOD)
    for field, value in (("abi_version", 9), ("N", 12), ("K", 1 << 20), ("x_dtype", 7), ("T", -3), ("pair", 3), ("tile_rows", 224),
                         ("tile_rows", 48), ("stages", 2), ("stages", 13), ("splits", 9), ("splits", 2), ("workspace_bytes", 256)):
        other = gg.CakeGGMx4Plan()
        ctypes.memmove(ctypes.byref(other), ctypes.byref(plan), ctypes.sizeof(plan))
        setattr(other, field, value)
        assert _call(other, workspace_bytes=1 << 40) != gg.CAKE_GG_OK, field


def test_4_bit_tokens_need_scales():
    assert _call(gg.cake_gg_mx4_plan(**{**GOOD, "x_dtype": "mx4"})) == gg.CAKE_GG_ERR_INVALID_ARG


@pytest.mark.parametrize("change,code", [
    (dict(X=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(Xq=None), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(xs=None), gg.CAKE_GG_ERR_INVALID_ARG), (dict(K=24), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(x_dtype="mx4"), gg.CAKE_GG_ERR_UNSUPPORTED), (dict(X=(1 << 20) + 4), gg.CAKE_GG_ERR_ALIGNMENT),
    (dict(act=5), gg.CAKE_GG_ERR_INVALID_ARG), (dict(R=-1), gg.CAKE_GG_ERR_INVALID_ARG), (dict(E=0), gg.CAKE_GG_ERR_INVALID_ARG),
    (dict(E=1024, R=2 ** 31 - 1), gg.CAKE_GG_ERR_OVERFLOW),
])
def test_quant_refuses(change, code):
    a = dict(X=1 << 20, x_dtype="bf16", act=None, E=1, R=4, K=64, Xq=1 << 20, xs=1 << 20, stream=0)
    a.update(change)
    assert gg.cake_gg_mx4_quant(**a) == code


def test_helpers_refuse():
    import torch
    u8 = torch.uint8
    W, ws = torch.zeros((2, 16, 32), dtype=u8), torch.zeros((2, 1, 1, 32, 4, 4), dtype=u8)
    off = torch.tensor([0, 2, 4], dtype=torch.int32)
    x = torch.zeros((4, 64), dtype=torch.bfloat16)
    q, s = torch.zeros((4, 32), dtype=u8), torch.zeros((1, 1, 32, 4, 4), dtype=u8)
    for err, args, more in [
        (TypeError, (x.half(), W, ws), dict(offsets=off)), (TypeError, (x, W.float(), ws), dict(offsets=off)),
        (TypeError, (x, W, ws.float()), dict(offsets=off)), (TypeError, (x, W, ws), dict(offsets=off.long())),
        (TypeError, (x, W, ws), dict(offsets=off, rows=torch.zeros(4, dtype=torch.int64))),
        (ValueError, (x, W, ws), dict()), (ValueError, (x[:, :32], W, ws), dict(offsets=off)),
        (ValueError, (x, W, ws[:1]), dict(offsets=off)), (ValueError, (x, W, ws), dict(offsets=off[:2])),
        (ValueError, (x, W, ws), dict(offsets=off, act="silu_mul")), (ValueError, (x, W, ws), dict(offsets=off, xs=s)),
        (ValueError, (x, W, ws), dict(offsets=off, act="gelu")), (ValueError, (q, W, ws), dict(offsets=off)),
        (ValueError, (q, W, ws), dict(offsets=off, xs=s[:, :, :3])), (ValueError, (x.T.contiguous().T, W, ws), dict(offsets=off)),
        (ValueError, (x, W.transpose(1, 2).contiguous().transpose(1, 2), ws), dict(offsets=off)),
        (TypeError, (x, W, ws), dict(offsets=off, out=torch.zeros((4, 16)))),
        (ValueError, (x, W, ws), dict(offsets=off, out=torch.zeros((4, 8), dtype=torch.bfloat16))),
        (ValueError, (x, W, ws), dict(offsets=off, plan=gg.cake_gg_mx4_plan(2, 4, 4, 16, 96))),
        (ValueError, (x, W, ws), dict(offsets=off)),             # host tensors
        (ValueError, (q, W, ws), dict(offsets=off, xs=s)),
    ]:
        with pytest.raises(err):
            gg.mx4_gemm(*args, **more)
    for err, args, more in [
        (TypeError, (x.half(),), {}), (ValueError, (x,), dict(act="gelu")), (ValueError, (x[0],), {}), (ValueError, (x[:, ::2],), {}),
        (TypeError, (x,), dict(out=q.char())), (ValueError, (x,), dict(out=q[:2])), (ValueError, (x,), dict(scale=ws)), (ValueError, (x,), {}),
    ]:
        with pytest.raises(err):
            gg.quantize_mx4(*args, **more)


def test_values_on_the_host():
    """What codes and scales stand for, element by element."""
    import torch
    g = torch.Generator().manual_seed(0)
    q = torch.randint(0, 256, (2, 130, 48), generator=g, dtype=torch.uint8)
    s = torch.randint(0, 256, (2, 2, 1, 32, 4, 4), generator=g, dtype=torch.uint8)
    s[0, 0, 0, 0, 0] = torch.tensor([0, 255, 254, 127], dtype=torch.uint8)
    v = gg.mx4_values(q, s)
    grid = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]
    for e, r, k in [(0, 0, k) for k in range(96)] + [(1, r, k) for r in (1, 31, 32, 64, 127, 128, 129) for k in (0, 1, 33, 95)]:
        byte = int(q[e, r, k // 2])
        code, scale = byte >> 4 if k % 2 else byte & 15, int(s[e, r // 128, k // 128, r % 32, r % 128 // 32, k // 32 % 4])
        want = float("nan") if scale == 255 else (-1 if code > 7 else 1) * grid[code & 7] * 2.0 ** (scale - 127)
        assert float(v[e, r, k]) == want or (want != want and v[e, r, k] != v[e, r, k]) or abs(want) > 3e38
