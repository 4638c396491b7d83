"""What the quantised expert layer takes, and how it says no."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


@pytest.fixture
def host_layer(monkeypatch):
    """A layer on the CPU, and nothing of it may reach the library's kernels."""
    import torch
    from moe_ragged_grouped_gb300 import experts
    gg_build.build()
    monkeypatch.setattr(experts.gg, "quantize_rows",
                        lambda w: (torch.zeros(w.shape, dtype=torch.int8), torch.zeros(w.shape[0])))

    def reached(*args, **more):
        raise AssertionError("a kernel's call was reached")
    for name in ("router_gemm", "int8_gemm"):
        monkeypatch.setattr(experts.gg, name, reached)
    z = torch.zeros
    return experts.Int8Experts(z(8, 64), z(8, 64, 64), z(8, 64, 32), 2)


@pytest.mark.parametrize("method", ["__call__", "route"])
def test_tokens_are_named_in_what_refuses_them(host_layer, method):
    import torch
    call = getattr(host_layer, method)
    for T in (0, 3):
        for dtype in (torch.float32, torch.float16, torch.int8):
            with pytest.raises(TypeError, match="x is"):
                call(torch.zeros((T, 64), dtype=dtype))
        for shape in ((T, 32), (T, 64, 1), (64,)):
            with pytest.raises(ValueError, match="x has shape"):
                call(torch.zeros(shape, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="contiguous"):
        call(torch.zeros((64, 3), dtype=torch.bfloat16).T)
    with pytest.raises(ValueError, match="x is on"):
        call(torch.zeros((3, 64), dtype=torch.bfloat16, device="meta"))


@pytest.mark.gpu
@pytest.mark.parametrize("E,top", [(4, 2), (13, 3), (1, 1)])
def test_expert_counts_that_are_no_multiple_of_eight(E, top):
    """The layer with E experts gives what one of 16 does whose other experts no token takes."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    from moe_ragged_grouped_gb300.experts import Int8Experts
    K, F = 256, 144
    g = torch.Generator(device="cuda").manual_seed(E)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    router, up, down = rand(E, K), rand(E, 2 * F, K), rand(E, K, F)
    more = lambda w, value: torch.cat([w, w.new_full((16 - E, *w.shape[1:]), value)])  # noqa: E731
    # (tokens whose first value is large, and a router that counts it against the others)
    x = rand(50, K)
    x[:, 0] = 100.0
    router[:, 0] = 0.0
    wide = more(router, 0.0)
    wide[E:, 0] = -1000.0
    x = x.to(torch.bfloat16)
    y = Int8Experts(router, up, down, top)(x, check=True)
    assert torch.equal(y, Int8Experts(wide, more(up, 1.0), more(down, 1.0), top)(x, check=True))
    expert, weight = Int8Experts(router, up, down, top).route(x)
    assert int(expert.max()) < E and expert.shape == weight.shape == (50, top)
