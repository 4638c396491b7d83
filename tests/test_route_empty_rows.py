"""Tokens whose mask leaves no expert, in a softmax that is not renormalised: weights and gradients are zeros, as in one that is."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("T,E,top_k", [(6, 16, 4), (300, 100, 3), (40, 600, 8), (9, 1024, 32)])
def test_rows_with_nothing_left(T, E, top_k, with_bias, dtype):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    g = torch.Generator(device="cuda").manual_seed(T)
    logits = torch.randn((T, E), generator=g, device="cuda").to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    bias = torch.randn(E, generator=g, device="cuda") if with_bias else None
    full = gg.route(logits, top_k, bias=bias, renormalize=False, scale=2.0)
    d_weight = torch.randn((T, top_k), generator=g, device="cuda")
    want = gg.route_grad(logits, full.expert, d_weight, renormalize=False, scale=2.0)
    empty = torch.zeros(T, dtype=torch.bool, device="cuda")
    empty[1::3] = True
    logits[empty] = float("-inf")
    got = gg.route(logits, top_k, bias=bias, renormalize=False, scale=2.0)
    assert not got.weight[empty].any() and torch.equal(got.weight[~empty], full.weight[~empty])
    assert torch.equal(got.expert[~empty], full.expert[~empty]) and int(got.offsets[-1]) == T * top_k
    assert torch.equal(got.expert[1].sort().values, got.expert[1].unique())
    d = gg.route_grad(logits, got.expert, d_weight, renormalize=False, scale=2.0)
    assert not d[empty].any() and torch.equal(d[~empty], want[~empty])
