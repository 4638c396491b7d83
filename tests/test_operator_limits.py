"""Routing, rows back and 4-bit products at sizes whose offsets pass 32 bits, by a few rows each."""
import pytest

from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


def _generator(seed):
    import torch
    return torch.Generator(device="cuda").manual_seed(seed)


def test_logits_past_two_billion():
    """The last tokens of 4 million x 600 are routed, and have gradients, as they do by themselves."""
    import torch
    T, E, top_k = 2 ** 22 + 3, 600, 4
    logits = torch.empty((T, E), dtype=torch.bfloat16, device="cuda").normal_(generator=_generator(0))
    d_weight = torch.randn((T, top_k), generator=_generator(1), device="cuda")
    r = gg.route(logits, top_k, renormalize=False)
    d = gg.route_grad(logits, r.expert, d_weight, renormalize=False)
    # each expert's rows are its tokens in order
    assert torch.equal(r.offsets.diff().long(), torch.bincount(r.expert.flatten(), minlength=E))
    assert torch.equal(r.rows[r.position.long()], torch.arange(T, dtype=torch.int32, device="cuda")[:, None].expand(-1, top_k))
    for cut in (slice(T - 500, T), slice(2 ** 31 // E - 100, 2 ** 31 // E + 100)):
        alone = gg.route(logits[cut], top_k, renormalize=False)
        assert torch.equal(alone.expert, r.expert[cut]) and torch.equal(alone.weight, r.weight[cut])
        assert torch.equal(gg.route_grad(logits[cut], alone.expert, d_weight[cut], renormalize=False), d[cut])


def test_rows_past_two_billion():
    """Rows of more than 2^32 values: sums, gradients and tokens to rows."""
    import torch
    T, top_k, K = 2 ** 19 + 5, 2, 4104
    r = torch.empty((T * top_k, K), dtype=torch.bfloat16, device="cuda").normal_(generator=_generator(0))
    position = torch.randperm(T * top_k, generator=_generator(1), device="cuda").to(torch.int32).view(T, top_k)
    w = torch.rand((T, top_k), generator=_generator(2), device="cuda")
    y = gg.combine_rows(r, position, w)
    d_rows, d_weight = gg.combine_grad(y, r, position, w)
    back = gg.gather_rows(y, position)
    # (every row is named once, so the tokens at both ends meet rows of the whole range)
    for cut in (slice(0, 300), slice(T - 300, T)):
        at = position[cut].long()
        terms = r[at].double() * w[cut].double()[:, :, None]
        want = terms.sum(dim=1)
        assert bool(((y[cut].double() - want).abs() <= 2.0 ** -8 * want.abs() + top_k * 2.0 ** -24 * terms.abs().sum(dim=1)).all())
        assert torch.equal(d_rows[at], (w[cut][:, :, None] * y[cut].float()[:, None, :]).to(torch.bfloat16))
        dots = y[cut].double()[:, None, :] * r[at].double()
        assert bool(((d_weight[cut].double() - dots.sum(dim=2)).abs() <= K * 2.0 ** -24 * dots.abs().sum(dim=2)).all())
        assert torch.equal(back[at], y[cut][:, None, :].expand(-1, top_k, -1))


@pytest.mark.parametrize("routed", [False, True])
def test_outputs_past_two_billion(routed):
    """The last rows of a 4-bit product of 2^31 values and more are what they are by themselves."""
    import torch
    M, N, K, E = 2 ** 20 + 77, 2056, 64, 3
    x = torch.randn((M // (2 if routed else 1), K), generator=_generator(0), device="cuda").to(torch.bfloat16)
    q, s = gg.quantize_mx4(torch.randn((E, N, K), generator=_generator(1), device="cuda"))
    rows = torch.randint(0, x.shape[0], (M,), generator=_generator(2), device="cuda").to(torch.int32) if routed else None
    offsets = torch.tensor([0, 5, M - 400, M], dtype=torch.int32, device="cuda")
    y = gg.mx4_gemm(x, q, s, offsets=offsets, rows=rows)
    xs = x if rows is None else x[rows.long()]
    values = gg.mx4_values(*gg.quantize_mx4(xs[-1000:].contiguous())).double()
    for e, cut in ((1, slice(0, 600)), (2, slice(600, 1000))):
        w = gg.mx4_values(q[e], s[e]).double()
        want, size = values[cut] @ w.T, values[cut].abs() @ w.abs().T
        # (sums of 64 exact products in FP32, then one rounding)
        assert bool(((y[-1000:][cut].double() - want).abs() <= 2.0 ** -8 * want.abs() + 15 * 2.0 ** -23 * size).all())
