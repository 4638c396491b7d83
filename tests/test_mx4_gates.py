"""Gated values at the ends of FP32's range: the codes are the rounding of silu(g) u itself."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg
from test_mx4_gpu import gated, quantised, same, unpacked

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()


def check(gate, u):
    """Codes and scales, bit for bit."""
    import torch
    x = torch.cat([gate, u], dim=1).contiguous()
    code, byte = unpacked(*gg.quantize_mx4(x, act="silu_mul"))
    want = quantised(gated(x))
    assert same(byte, want[1]), (byte - want[1]).nonzero()[:4]
    assert same(code, want[0]), (code - want[0]).nonzero()[:4]


@pytest.mark.parametrize("up", [40, 50, 100, 127])
def test_subnormal_gates(up):
    """A gate below the normal range, halved by the sigmoid, does not fit FP32; with a large u the product does."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(up)
    whole = torch.randint(-64, 65, (512, 64), generator=g, device="cuda")
    whole[0, :4] = torch.tensor([12, 1, 3, 5], device="cuda")
    whole[0, 4:] = 0
    gate = (whole.double() * 2.0 ** -149).float()
    check(gate, torch.full_like(gate, 2.0 ** up))
    check(gate, -torch.full_like(gate, 2.0 ** up) * (1 + torch.rand(gate.shape, generator=g, device="cuda")).clamp(max=1.9))


@pytest.mark.parametrize("least", [-149, -130, -126, -120])
def test_tiny_gates_beside_ordinary_ones(least):
    """Rows in which some blocks have tiny gates and others lie on borders, so that all of a warp's are looked at again."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(-least)
    gate = torch.randn((256, 256), generator=g, device="cuda")
    tiny = torch.rand((256, 8), generator=g, device="cuda").repeat_interleave(32, dim=1) < 0.5
    u = torch.randn((256, 256), generator=g, device="cuda")
    power = torch.randint(least, least + 6, (256, 256), generator=g, device="cuda").double()
    gate = torch.where(tiny, (torch.sign(gate).double() * (1 + torch.rand((256, 256), generator=g, device="cuda").double()) * 2.0 ** power).float(), gate)
    u = torch.where(tiny, torch.sign(u) * 2.0 ** 126 * (1 + torch.rand((256, 256), generator=g, device="cuda")), u)
    # (the first block of every other row: values on a border)
    u[::2, :32] = (1.25 / (gate[::2, :32].double() / (1 + (-gate[::2, :32].double()).exp()))).clamp(-3e38, 3e38).float()
    u[::2, 0] = (4.5 / (gate[::2, 0].double() / (1 + (-gate[::2, 0].double()).exp()))).clamp(-3e38, 3e38).float()
    check(gate, u)


def test_at_the_largest_number():
    """Products that FP32 just holds, or just does not: a block is a NaN where the rounded product is infinite."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(1)
    gate = torch.zeros((4096, 32), device="cuda")
    u = torch.zeros((4096, 32), device="cuda")
    gate[:, 0] = 1.5 + 3 * torch.rand(4096, generator=g, device="cuda")
    largest = float(torch.finfo(torch.float32).max)
    s = gate[:, 0].double() / (1 + (-gate[:, 0].double()).exp())
    near = 1 + torch.randint(-8, 9, (4096,), generator=g, device="cuda").double() * 2.0 ** -25
    u[:, 0] = (largest * near / s).float()
    gate[:, 1:] = 1.0
    u[:, 1:] = torch.randn((4096, 31), generator=g, device="cuda") * 1e38
    check(gate, u)


@pytest.mark.parametrize("steps", [0, 8, 64])
def test_far_gates_on_borders(steps):
    """Gates from -50 to -20, whose exponentials carry the most error, a few of FP32's steps from a border between codes."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(steps)
    gate = -20 - 30 * torch.rand((8192, 32), generator=g, device="cuda")
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    want = mids[torch.randint(0, 7, (8192, 32), generator=g, device="cuda")].double()
    want[:, 0] = 4.0 + 3 * torch.rand(8192, generator=g, device="cuda").double()
    want[::7, 0] = 8.0
    want *= 1 + torch.randint(-steps, steps + 1, (8192, 32), generator=g, device="cuda").double() * 2.0 ** -23
    check(gate, (want / (gate.double() / (1 + (-gate.double()).exp()))).float())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_zeros_under_far_gates(dtype):
    """Zeros whatever their gate is: blocks of them, alone in a row and beside others; an infinite gate's are NaNs."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(7)
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    gate = torch.randn((60, 512), generator=g, device="cuda") * 10.0 ** torch.randint(0, 38, (60, 1), generator=g, device="cuda")
    gate[:20] = -90 * torch.rand((20, 512), generator=g, device="cuda")
    gate, u = gate.to(kind), torch.zeros((60, 512), dtype=kind, device="cuda")
    u[:, ::3] = -0.0
    u[1::4, :256] = torch.randn((15, 256), generator=g, device="cuda").to(kind)
    u[2::4, 500] = 1.0
    check(gate, u)
    gate[::5, 70], gate[1::5, 300], gate[2::5, 100] = float("-inf"), float("inf"), float("nan")
    check(gate, u)
    u[3::5, 33] = float("inf")
    gate[3::5, 33] = 0.0
    check(gate, u)
    x = torch.cat([torch.full((3, 64), -95.0, device="cuda"), torch.zeros((3, 64), device="cuda")], dim=1).to(kind)
    w = gg.quantize_mx4(torch.randn((16, 64), generator=g, device="cuda"))
    assert not gg.mx4_gemm(x, *w, act="silu_mul").any()
