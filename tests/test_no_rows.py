"""Calls of an expert-parallel rank to which nothing was routed, and values of nothing."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

AT = 1 << 20


@pytest.mark.parametrize("kind", ["mx4", "i8"])
def test_no_rows_of_some_tokens_is_not_refused(kind):
    """An empty tensor has no address: the call without rows to compute does not need one."""
    gg_build.build()
    plan = getattr(gg, f"cake_gg_{kind}_plan")(4, 0, 5, 128, 256)
    a = dict(X=AT, xs=None, rows=None, W=AT, ws=AT, Y=None, offsets=AT, workspace=AT, workspace_bytes=plan.workspace_bytes, stream=0)
    call = getattr(gg, f"cake_gg_{kind}_gemm")
    assert call(plan, **a) != gg.CAKE_GG_ERR_INVALID_ARG         # (without a GPU that is what it lacks)
    # one with rows to compute does
    plan = getattr(gg, f"cake_gg_{kind}_plan")(4, 3, 5, 128, 256)
    assert call(plan, **{**a, "Y": AT, "workspace_bytes": plan.workspace_bytes}) == gg.CAKE_GG_ERR_INVALID_ARG


def test_values_of_no_rows():
    import torch
    for lead in ((), (3,)):
        q = torch.zeros((*lead, 0, 48), dtype=torch.uint8)
        scale = torch.zeros((*lead, *gg._mx4_tiles(0, 96)), dtype=torch.uint8)
        assert gg.mx4_values(q, scale).shape == (*lead, 0, 96)


@pytest.mark.gpu
def test_no_rows_of_some_tokens():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    E, N, K, T = 4, 128, 256, 5
    i32 = torch.int32
    x = torch.ones((T, K), dtype=torch.bfloat16, device="cuda")
    rows, offsets = torch.empty(0, dtype=i32, device="cuda"), torch.zeros(E + 1, dtype=i32, device="cuda")
    w = torch.ones((E, N, K), device="cuda")
    q, s = gg.quantize_mx4(w)
    assert gg.mx4_gemm(x, q, s, offsets=offsets, rows=rows).shape == (0, N)
    q, s = gg.quantize_rows(w.view(E * N, K))
    assert gg.int8_gemm(x, q.view(E, N, K), s.view(E, N), offsets=offsets, rows=rows).shape == (0, N)
