"""The 4-bit products and their quantiser on the GPU, against 64-bit definitions.

The quantiser has to give the definition's codes and scales, bit for bit.  A
product of two 4-bit values with their powers of two is exact, so only the FP32
sums round: each of the ceil(K / 64) steps of the tensor cores may cut off at
the last place of a partial sum, which is at most A = sum |x w|, and so may the
additions within a step (64 products: six levels) and between the at most 8
parts of a divided reduction:

    |err| <= (ceil(K / 64) + 6 + 8) 2^-23 A,   for BF16 output 2^-8 |y| more.
"""
import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    return gg.load_library()


# ---------------------------------------------------------------- definitions

def power(e):
    """2^e in 64 bits by its bits (a power function may be off by a last place)."""
    import torch
    return ((e.long() + 1023) << 52).view(torch.float64)


def same(a, b):
    """Equal tensors (a value on its own, so that a failure does not print them)."""
    return a.shape == b.shape and bool((a == b).all())


GRID = [0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0]


def quantised(h):
    """Codes [R, K] (0 .. 15) and scale bytes [R, K / 32] of h [R, K] in 64 bits."""
    import torch
    b = h.view(h.shape[0], -1, 32)
    bad = ~torch.isfinite(b.float()).all(dim=2)
    m = torch.where(bad, torch.ones_like(b[:, :, 0]), b.abs().amax(dim=2))
    e = (torch.frexp(m).exponent - 3).clamp(min=-127)
    e = torch.where(m == 0, torch.full_like(e, -127), e)
    a = b.abs() * power(-e)[:, :, None]
    mid = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], dtype=torch.float64, device=h.device)
    odd_below = torch.tensor([False, True, False, True, False, True, False], device=h.device)   # ties go up from odd codes
    code = ((a[..., None] > mid) | ((a[..., None] == mid) & odd_below)).sum(dim=-1)
    code = code + 8 * (torch.signbit(b) & (code > 0)).long()
    code = torch.where(bad[:, :, None], torch.zeros_like(code), code)
    return code.view(h.shape), torch.where(bad, torch.full_like(e, 255), e + 127)


def unpacked(q, tiles):
    """Codes and scale bytes of packed rows and their tiles, element by element; a zero's sign does not count."""
    import torch
    R, K = q.shape[0], 2 * q.shape[1]
    code = torch.stack([q & 15, q >> 4], dim=-1).reshape(R, K).long()
    code = torch.where(code == 8, torch.zeros_like(code), code)
    r = torch.arange(R, device=q.device)[:, None]
    b = torch.arange(K // 32, device=q.device)[None, :]
    return code, tiles[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].long()


def gated(x):
    g, u = x.double().chunk(2, dim=1)
    return g / (1 + (-g).exp()) * u


def values(q, tiles):
    import torch
    code, byte = unpacked(q, tiles)
    grid = torch.tensor(GRID, dtype=torch.float64, device=q.device)
    v = torch.where(code < 8, grid[code & 7], -grid[code & 7])
    s = torch.where(byte == 255, torch.full(byte.shape, float("nan"), dtype=torch.float64, device=q.device),
                    power(byte - 127))
    return v * s.repeat_interleave(32, dim=1)


def check(got, x, w, sizes, rows=None, out_dtype="bf16"):
    """x [T, K] and w [E, N, K] in 64 bits."""
    import torch
    K = x.shape[1]
    if rows is not None:
        x = x[rows.long()]
    at = 0
    for e, n in enumerate(sizes):
        if n == 0:
            continue
        y, A = x[at:at + n] @ w[e].T, x[at:at + n].abs() @ w[e].abs().T
        tol = (-(-K // 64) + 14) * 2.0 ** -23 * A + (2.0 ** -8 * y.abs() if out_dtype == "bf16" else 0)
        err = (got[at:at + n].double() - y).abs()
        bad = ~(err <= tol)
        assert not bad.any(), (f"expert {e}: {int(bad.sum())} of {bad.numel()} outside, first at {bad.nonzero()[0].tolist()}, "
                               f"worst error {float((err / tol.clamp(min=1e-300)).max()):.3g} of the bound")
        at += n


def offsets_of(sizes):
    import torch
    return torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")


def randn(shape, seed, dtype="bf16"):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(shape, generator=g, device="cuda")
    x *= torch.exp2(torch.randint(-3, 4, shape[:-1] + (1,), generator=g, device="cuda").float())
    return x.to({"bf16": torch.bfloat16, "fp32": torch.float32}[dtype])


def weights(E, N, K, seed):
    q, s = gg.quantize_mx4(randn((E, N, K), seed))
    return q, s


def dense_values(q, s):
    import torch
    return torch.stack([values(a, b) for a, b in zip(q, s)])


# ---------------------------------------------------------------- quantiser


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K", [(1, 32), (2, 64), (7, 96), (8, 128), (9, 160), (33, 256), (127, 288), (128, 1024), (129, 1056),
                                 (300, 2080), (1, 8192), (5, 131040)])
def test_quantise(T, K, dtype):
    import torch
    x = randn((T, K), T + K, dtype)
    q, s = gg.quantize_mx4(x)
    code, byte = unpacked(q, s)
    want = quantised(x.double())
    assert same(byte, want[1]) and same(code, want[0])
    # the blocks past K are zeros, and so are the rows past T of tiles that the call made
    tail = s.transpose(-4, -2).reshape(s.shape[0] * 128, -1)
    assert not tail[:T, K // 32:].any() and not tail[T:].any()
    assert same(gg.mx4_values(q, s).double(), values(q, s))


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,K", [(1, 32), (3, 96), (64, 512), (129, 1056), (2048, 2048)])
def test_quantise_gated(T, K, dtype):
    import torch
    x = randn((T, 2 * K), T + K, dtype)
    q, s = gg.quantize_mx4(x, act="silu_mul")
    code, byte = unpacked(q, s)
    want = quantised(gated(x))
    assert same(byte, want[1]) and same(code, want[0])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantise_every_border(dtype):
    """Values on and beside every border between codes, in every binade of a scale, and exact powers of two as maxima."""
    import torch
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0, 6.0, 7.0, 7.9375], dtype=torch.float64)
    step = 2.0 ** -7 if dtype == "bf16" else 2.0 ** -23
    a = torch.cat([mids, mids * (1 + step), mids * (1 - step / 2), torch.tensor([0.0, -0.0], dtype=torch.float64)])
    row = torch.zeros(len(a), 32, dtype=torch.float64)
    row[:, 0], row[:, 1], row[:, 2] = 4.0, a, -a
    x = torch.cat([row * 2.0 ** p for p in (-126, -100, -3, 0, 1, 60, 120)]).cuda().to(
        torch.bfloat16 if dtype == "bf16" else torch.float32)
    q, s = gg.quantize_mx4(x)
    code, byte = unpacked(q, s)
    want = quantised(x.double())
    assert same(byte, want[1]) and same(code, want[0])


def test_quantise_gated_near_borders():
    """Gated values driven onto borders: u is chosen so that silu(g) u lies within FP32's error of a tie."""
    import torch
    g = torch.Generator(device="cuda").manual_seed(3)
    gate = torch.randn((4096, 32), generator=g, device="cuda") * 3
    mids = torch.tensor([0.25, 0.75, 1.25, 1.75, 2.5, 3.5, 5.0], device="cuda")
    want = mids[torch.randint(0, 7, (4096, 32), generator=g, device="cuda")].double()
    want[:, 0] = 4.0 + torch.rand(4096, generator=g, device="cuda").double()
    u = (want / (gate.double() / (1 + (-gate.double()).exp()))).float()
    x = torch.cat([gate, u], dim=1)
    q, s = gg.quantize_mx4(x, act="silu_mul")
    code, byte = unpacked(q, s)
    ref = quantised(gated(x))
    assert same(byte, ref[1]) and same(code, ref[0])


@pytest.mark.parametrize("value", [float("nan"), float("inf"), float("-inf")])
@pytest.mark.parametrize("act", [None, "silu_mul"])
def test_quantise_what_is_not_finite(value, act):
    """Its block is a NaN, the others are as they were; zeros and tiny values stay finite."""
    import torch
    K = 128
    x = randn((4, K * (2 if act else 1)), 5)
    x[1, 40] = value
    x[2] = 0
    x[3] = 1e-40
    q, s = gg.quantize_mx4(x, act=act)
    code, byte = unpacked(q, s)
    want = quantised(gated(x) if act else x.double())
    assert same(byte, want[1]) and same(code, want[0])
    assert byte[1].tolist().count(255) == 1 and byte[1, 1] == 255 and not byte[2].any()
    y = gg.mx4_gemm(x, *[t[0] for t in weights(1, 16, K, 1)], act=act, out_dtype="fp32")
    assert torch.isnan(y[1]).all() and torch.isfinite(y[[0, 2, 3]]).all()


# ---------------------------------------------------------------- products


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K", [
    (1, 8, 32), (1, 1000, 4096), (2, 24, 64), (3, 136, 2080), (5, 72, 96), (8, 4096, 640), (9, 40, 1024), (16, 128, 256),
    (17, 264, 160), (31, 128, 128), (33, 520, 1056), (64, 256, 512), (65, 1000, 384), (127, 640, 288), (129, 136, 544),
    (193, 264, 288), (225, 264, 800), (257, 520, 640), (1001, 392, 1024), (300, 256, 8192),
])
def test_dense(T, N, K, out_dtype):
    q, s = weights(1, N, K, T + N)
    x, xs = gg.quantize_mx4(randn((T, K), T * 7 + N + K))
    got = gg.mx4_gemm(x, q[0], s[0], xs=xs, out_dtype=out_dtype)
    check(got, values(x, xs), dense_values(q, s), [T], None, out_dtype)


@pytest.mark.parametrize("T", [1, 40, 200])
def test_exact_sums(T):
    """Products whose FP32 sums are exact in every order are those sums, bit for bit."""
    import torch
    K, N = 512, 264
    rng = np.random.default_rng(T)
    # whole numbers 0 .. 6 under scales of one: sums below 2^15
    grid = torch.tensor([0, 2, 4, 5, 6, 7], dtype=torch.uint8)
    def codes(r):
        c = grid[torch.from_numpy(rng.integers(0, 6, size=(r, K)))] + 8 * torch.from_numpy(rng.integers(0, 2, size=(r, K)).astype(np.uint8))
        return (c[:, ::2] | c[:, 1::2] << 4).cuda()
    ones = lambda r: torch.full(gg._mx4_tiles(r, K), 127, dtype=torch.uint8, device="cuda")  # noqa: E731
    x, w = codes(T), codes(N)
    got = gg.mx4_gemm(x, w, ones(N), xs=ones(T), out_dtype="fp32")
    assert same(got.double(), values(x, ones(T)) @ values(w, ones(N)).T)


SIZES = [
    [1], [0, 1, 0], [3, 0, 5, 1], [0, 0, 0, 7], [9, 8, 7, 16, 0, 1], [33, 1, 0, 64, 17],
    [130, 0, 2, 257, 31], [0, 500, 0, 100, 1, 1, 0],
]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("N,K", [(72, 96), (264, 544), (136, 1056)])
@pytest.mark.parametrize("routed", [False, True])
def test_grouped(sizes, N, K, routed, out_dtype):
    import torch
    E, M = len(sizes), sum(sizes)
    rng = np.random.default_rng(M + N + routed)
    T = max(1, M // 2) if routed else M
    q, s = weights(E, N, K, M + N)
    x, xs = gg.quantize_mx4(randn((T, K), M + K))
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda() if routed else None
    got = gg.mx4_gemm(x, q, s, xs=xs, offsets=offsets_of(sizes), rows=rows, out_dtype=out_dtype)
    check(got, values(x, xs), dense_values(q, s), sizes, rows, out_dtype)


@pytest.mark.parametrize("E,M", [(200, 40), (1024, 900), (1024, 8)])
def test_many_experts(E, M):
    rng = np.random.default_rng(E)
    sizes = [int(v) for v in rng.multinomial(M, [1 / E] * E)]
    N, K = 40, 96
    q, s = weights(E, N, K, E)
    x, xs = gg.quantize_mx4(randn((M, K), M))
    got = gg.mx4_gemm(x, q, s, xs=xs, offsets=offsets_of(sizes), out_dtype="fp32")
    check(got, values(x, xs), dense_values(q, s), sizes, None, "fp32")


@pytest.mark.parametrize("x_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("sizes", [[5], [40, 0, 3], [130, 300, 1]], ids=str)
def test_activations(sizes, act, x_dtype):
    """Quantised on the way as by themselves."""
    import torch
    E, M, N, K = len(sizes), sum(sizes), 136, 672
    q, s = weights(E, N, K, 9)
    x = randn((M, K * (2 if act else 1)), M, x_dtype)
    got = gg.mx4_gemm(x, q, s, offsets=offsets_of(sizes), act=act, out_dtype="fp32")
    xq, xs = gg.quantize_mx4(x, act=act)
    assert same(got, gg.mx4_gemm(xq, q, s, xs=xs, offsets=offsets_of(sizes), out_dtype="fp32"))
    check(got, values(xq, xs), dense_values(q, s), sizes, None, "fp32")


@pytest.mark.parametrize("M", [6, 300])
def test_rows_past_the_last_offset_and_bands(M):
    """Rows past offsets[E] and the memory around Y stay as they were."""
    import torch
    from gg_testutil import guarded_empty, guards_intact
    N, K = 136, 256
    sizes = [M // 2, 0, M // 3]
    q, s = weights(3, N, K, 2)
    x, xs = gg.quantize_mx4(randn((M, K), M))
    for out_dtype in ("bf16", "fp32"):
        buf, view, guard = guarded_empty((M, N), out_dtype)
        before = view[sum(sizes):].clone()
        gg.mx4_gemm(x, q, s, xs=xs, offsets=offsets_of(sizes), out_dtype=out_dtype, out=view)
        assert guards_intact(buf, guard, M * N, out_dtype)
        bits = torch.int16 if out_dtype == "bf16" else torch.int32
        assert same(view[sum(sizes):].view(bits), before.view(bits))
        check(view, values(x, xs), dense_values(q, s), sizes, None, out_dtype)


def test_device_errors():
    """Offsets and rows that do not hold are reported, and the next call works."""
    import torch
    N, K, M = 64, 128, 20
    q, s = weights(2, N, K, 1)
    x, xs = gg.quantize_mx4(randn((M, K), 1))
    good = offsets_of([12, 8])
    plan = gg.cake_gg_mx4_plan(2, M, M, N, K, "mx4", None, "fp32")
    work = gg.make_workspace(plan, "cuda")
    run = lambda offsets, rows=None: gg.mx4_gemm(x, q, s, xs=xs, offsets=offsets, rows=rows, out_dtype="fp32", plan=plan, workspace=work)  # noqa: E731
    for bad in ([1, 12, 20], [0, 12, 8], [0, 12, 21]):
        with pytest.raises(gg.CakeGGError) as err:
            run(torch.tensor(bad, dtype=torch.int32, device="cuda"))
        assert err.value.code == gg.CAKE_GG_ERR_BAD_OFFSETS
    rows = torch.arange(M, dtype=torch.int32, device="cuda")
    for at, value in ((0, -1), (19, M), (7, 2 ** 31 - 1), (7, -2 ** 31)):
        wrong = rows.clone()
        wrong[at] = value
        with pytest.raises(gg.CakeGGError) as err:
            run(good, wrong)
        assert err.value.code == gg.CAKE_GG_ERR_BAD_ROWS
    check(run(good, rows), values(x, xs), dense_values(q, s), [12, 8], rows, "fp32")


def test_no_rows():
    import torch
    q, s = weights(2, 64, 128, 1)
    x = torch.empty((0, 128), dtype=torch.bfloat16, device="cuda")
    assert gg.mx4_gemm(x, q, s, offsets=offsets_of([0, 0])).shape == (0, 64)
    assert [t.shape[0] for t in gg.quantize_mx4(x)] == [0, 0]


# ---------------------------------------------------------------- how a call behaves


def test_every_shape_of_the_kernel(monkeypatch):
    """Single CTAs, pairs, divided reductions, all tile sizes: ragged experts, routed and not, against 64 bits."""
    import torch
    sizes, N, K = [130, 0, 2, 257, 31], 392, 1056
    E, M = len(sizes), sum(sizes)
    q, s = weights(E, N, K, 4)
    w = dense_values(q, s)
    x, xs = gg.quantize_mx4(randn((M, K), 1))
    rows = torch.from_numpy(np.random.default_rng(0).permutation(M).astype(np.int32)).cuda()
    for pair, nt, splits in [(1, nt, 1) for nt in range(32, 193, 32)] + [(2, nt, 1) for nt in range(32, 193, 32)] + [(1, 32, 2), (1, 64, 3), (1, 32, 5)]:
        for name, value in (("PAIR", pair), ("ROWS_PER_TILE", nt), ("SPLITS", splits)):
            monkeypatch.setenv("CAKE_GG_MX4_" + name, str(value))
        for out_dtype in ("bf16", "fp32"):
            for r in (None, rows):
                got = gg.mx4_gemm(x, q, s, xs=xs, offsets=offsets_of(sizes), rows=r, out_dtype=out_dtype)
                check(got, values(x, xs), w, sizes, r, out_dtype)


@pytest.mark.parametrize("pair", [1, 2])
def test_same_bits_on_every_run_and_under_every_cap(pair, monkeypatch):
    import torch
    monkeypatch.setenv("CAKE_GG_MX4_PAIR", str(pair))
    sizes, N, K = [40, 300, 0, 77], 520, 800
    q, s = weights(4, N, K, 1)
    x = randn((sum(sizes), K), 2)
    first = gg.mx4_gemm(x, q, s, offsets=offsets_of(sizes), out_dtype="fp32")
    for cap in [0] * 5 + [1, 2, 7, 100]:
        assert torch.equal(first, gg.mx4_gemm(x, q, s, offsets=offsets_of(sizes), out_dtype="fp32", max_sms=cap))


@pytest.mark.parametrize("pair,splits", [(1, 1), (1, 2), (2, 1)])
def test_a_lost_copy_times_out(pair, splits, monkeypatch):
    """Every wait ends, the status says so, and the next call is right."""
    monkeypatch.setenv("CAKE_GG_MX4_PAIR", str(pair))
    monkeypatch.setenv("CAKE_GG_MX4_ROWS_PER_TILE", "64")
    monkeypatch.setenv("CAKE_GG_MX4_SPLITS", str(splits))
    T, N, K = 50, 264, 1056
    q, s = weights(1, N, K, 1)
    x, xs = gg.quantize_mx4(randn((T, K), 2))
    plan = gg.cake_gg_mx4_plan(1, T, T, N, K, "mx4", None, "fp32")
    assert (plan.pair, plan.splits) == (pair, splits)
    plan.timeout_ns = 100_000_000
    work = gg.make_workspace(plan, "cuda")
    plan.debug_flags = gg.CAKE_GG_DEBUG_DROP_FIRST_LOAD
    with pytest.raises(gg.CakeGGError) as err:
        gg.mx4_gemm(x, q[0], s[0], xs=xs, out_dtype="fp32", plan=plan, workspace=work)
    assert err.value.code == gg.CAKE_GG_ERR_TIMEOUT
    plan.debug_flags = 0
    got = gg.mx4_gemm(x, q[0], s[0], xs=xs, out_dtype="fp32", plan=plan, workspace=work)
    check(got, values(x, xs), dense_values(q, s), [T], None, "fp32")


@pytest.mark.parametrize("T", [3, 700])
def test_captured_on_another_stream(T):
    """A graph of quantising and product, replayed on new tokens and weights' rows."""
    import torch
    N, K = 264, 544
    sizes = [T // 3, T - T // 3]
    q, s = weights(2, N, K, 3)
    xs = [randn((T, K), 5 + i) for i in range(3)]
    want = [gg.mx4_gemm(x, q, s, offsets=offsets_of(sizes)) for x in xs]
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    with torch.cuda.stream(stream):
        x, off, out = xs[0].clone(), offsets_of(sizes), torch.empty((T, N), dtype=torch.bfloat16, device="cuda")
        plan = gg.cake_gg_mx4_plan(2, T, T, N, K)
        work = gg.make_workspace(plan, "cuda")
        run = lambda: gg.mx4_gemm(x, q, s, offsets=off, out=out, plan=plan, workspace=work, check=False)  # noqa: E731
        run()
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            run()
            run()
        for i in (1, 2, 0):
            x.copy_(xs[i])
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, want[i])


def test_weights_past_four_billion_values():
    """Codes past 2^31 bytes: the last expert's, whose rows are the last."""
    import torch
    E, N, K = 70, 8192, 8192
    q = torch.zeros((E, N, K // 2), dtype=torch.uint8, device="cuda")
    s = torch.zeros((E, *gg._mx4_tiles(N, K)), dtype=torch.uint8, device="cuda")
    q[-1], s[-1] = (t[0] for t in weights(1, N, K, 1))
    x, xs = gg.quantize_mx4(randn((20, K), 2))
    off = torch.zeros(E + 1, dtype=torch.int32)
    off[-1] = 20
    got = gg.mx4_gemm(x, q, s, xs=xs, offsets=off.cuda(), out_dtype="fp32")
    check(got, values(x, xs), dense_values(q[-1:], s[-1:]), [20], None, "fp32")


def test_on_a_stream_that_is_not_the_current_one():
    """Helpers given a stream: what they make belongs to it."""
    import torch
    N, K, T = 264, 544, 300
    q, s = weights(1, N, K, 3)
    x = randn((T, K), 1)
    want_q, want = gg.quantize_mx4(x), gg.mx4_gemm(x, q[0], s[0])
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for st in (stream, stream.cuda_stream):
        got_q, got = gg.quantize_mx4(x, stream=st), gg.mx4_gemm(x, q[0], s[0], stream=st)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got_q, want_q)) and torch.equal(got, want)


# ---------------------------------------------------------------- few rows


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("x_dtype", ["mx4", "bf16", "fp32"])
@pytest.mark.parametrize("T,E,K,N,routed", [
    (1, 1, 32, 8, False), (2, 1, 992, 136, False), (1, 1, 8192, 264, False), (3, 1, 1056, 1000, False), (15, 1, 1024, 1024, False),
    (1, 40, 288, 520, True), (2, 9, 2880, 256, True), (7, 3, 64, 120, True), (9, 300, 96, 40, False),
])
def test_few_rows(T, E, K, N, routed, x_dtype, out_dtype):
    """Dot products against 64 bits: one row and two a run, dense and by expert, codes and activations."""
    import torch
    rng = np.random.default_rng(T + K)
    M = 2 * T if routed else T
    sizes = [int(v) for v in rng.multinomial(M, [1 / E] * E)]
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda() if routed else None
    plan = gg.cake_gg_mx4_plan(E, M, T, N, K, x_dtype, None, out_dtype)
    assert plan.path == gg.CAKE_GG_MX4_ROWS
    q, s = weights(E, N, K, T + N)
    x = randn((T, K), T + K, "fp32" if x_dtype == "fp32" else "bf16")
    xq, xs = gg.quantize_mx4(x)
    scales = xs if x_dtype == "mx4" else None
    got = gg.mx4_gemm(xq if scales is not None else x, q, s, xs=scales, offsets=offsets_of(sizes) if E > 1 else None, rows=rows,
                      out_dtype=out_dtype)
    check(got, values(xq, xs), dense_values(q, s), sizes, rows, out_dtype)


@pytest.mark.parametrize("T", [1, 2])
def test_few_rows_of_every_scale(T):
    """One block: its sum is exact, so the output is that sum rounded, whatever the two scales are."""
    import torch
    N = 1024
    rng = np.random.default_rng(T)
    codes = lambda r: torch.from_numpy(rng.integers(0, 256, size=(r, 16)).astype(np.uint8)).cuda()  # noqa: E731
    tiles = lambda r: torch.from_numpy(rng.integers(0, 256, size=gg._mx4_tiles(r, 32)).astype(np.uint8)).cuda()  # noqa: E731
    w, ws = codes(N), tiles(N)
    ws[..., 1:] = 0                                              # (blocks that the rows do not have)
    for byte in (0, 1, 2, 3, 64, 127, 128, 200, 253, 254, 255):
        x, xs = codes(T), tiles(T)
        xs[...] = 0
        xs[..., 0] = byte
        got = gg.mx4_gemm(x, w, ws, xs=xs, out_dtype="fp32")
        want = (values(x, xs) @ values(w, ws).T).cpu().float()
        assert torch.allclose(got.cpu(), want, rtol=0, atol=0, equal_nan=True), byte


def test_few_rows_of_lost_tokens():
    """A row whose token does not exist is reported and is zeros; the others are right."""
    import torch
    N, K, M = 128, 256, 3
    q, s = weights(4, N, K, 1)
    x = randn((M, K), 1)
    rows = torch.tensor([0, 3, 2], dtype=torch.int32, device="cuda")
    for tokens in (gg.quantize_mx4(x), (x, None)):
        out = torch.empty((M, N), dtype=torch.float32, device="cuda")
        with pytest.raises(gg.CakeGGError) as err:
            gg.mx4_gemm(tokens[0], q, s, xs=tokens[1], offsets=offsets_of([1, 1, 0, 1]), rows=rows, out=out, out_dtype="fp32")
        assert err.value.code == gg.CAKE_GG_ERR_BAD_ROWS
        v, w = values(*gg.quantize_mx4(x)), dense_values(q, s)
        assert not out[1].any()
        check(out[0::2].contiguous(), v[0::2], w[0::3].contiguous(), [1, 1], None, "fp32")
