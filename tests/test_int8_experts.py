"""The quantised expert layer that chains the router, the routed 8-bit product and the gated one."""
import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


def test_layer_refuses_shapes():
    import torch
    from moe_ragged_grouped_gb300.experts import Int8Experts
    z = torch.zeros
    for router, up, down, top in [(z(4, 32), z(4, 64, 32), z(4, 32, 16), 2), (z(3, 32), z(4, 64, 32), z(4, 32, 32), 2),
                                  (z(4, 32), z(4, 64, 32), z(4, 32, 32), 5), (z(4, 32), z(4, 64, 32), z(4, 32, 32), 0)]:
        with pytest.raises(ValueError):
            Int8Experts(router, up, down, top)


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 40, 333])
def test_layer_against_64_bits(T):
    """The layer's own quantised tensors multiplied in 64 bits.

    h is BF16 in the layer (relative rounding 2^-8), so the reference takes the
    layer's h and bounds each stage by itself: h within 2^-8 + 2^-20 of its
    exact value; y within the FP32 work after it (sums of top_k terms, gate and
    scale: 2^-18 of the terms' magnitudes) and one BF16 rounding.
    """
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    from moe_ragged_grouped_gb300.experts import Int8Experts
    E, K, F, top = 8, 256, 144, 3
    g = torch.Generator(device="cuda").manual_seed(T)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    layer = Int8Experts(rand(E, K) / K ** 0.5, rand(E, 2 * F, K) / K ** 0.5, rand(E, K, F) / F ** 0.5, top)
    x = rand(T, K).to(torch.bfloat16)
    y = layer(x, check=True)
    assert torch.equal(y, layer(x))                       # kept plans and workspaces
    expert, weight = layer.route(x)
    q, s = gg.quantize_rows(x)
    _, (_, _, h), _ = layer._for(T, x.device)
    order = torch.argsort(expert.reshape(-1), stable=True)
    e_of, t_of = expert.reshape(-1)[order], order // top
    want_h = torch.einsum("mk,mnk->mn", q[t_of].double(), layer.up_q[e_of].double())
    want_h *= layer.up_s[e_of].double() * s[t_of, None].double()
    assert ((h.double() - want_h).abs() <= (2.0 ** -8 + 2.0 ** -20) * want_h.abs()).all()
    hq, hs = gg.quantize_rows(h, act="silu_mul")
    rows = torch.einsum("mk,mnk->mn", hq.double(), layer.down_q[e_of].double())
    rows *= layer.down_s[e_of].double() * hs[:, None].double() * weight.reshape(-1)[order, None].double()
    want, size = torch.zeros(T, K, dtype=torch.float64, device="cuda"), torch.zeros(T, K, dtype=torch.float64, device="cuda")
    want.index_add_(0, t_of, rows)
    size.index_add_(0, t_of, rows.abs())
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all()


@pytest.mark.gpu
def test_layer_without_tokens():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    from moe_ragged_grouped_gb300.experts import Int8Experts
    rng = np.random.default_rng(0)
    t = lambda *s: torch.from_numpy(rng.standard_normal(s).astype(np.float32)).cuda()  # noqa: E731
    layer = Int8Experts(t(4, 32), t(4, 32, 32), t(4, 32, 16), 2)
    assert layer(torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")).shape == (0, 32)
