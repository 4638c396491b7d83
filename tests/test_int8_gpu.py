"""The 8-bit products and the row quantiser on the GPU, against 64-bit definitions.

Products of 8-bit integers are exact, so with S the exact integer sum the
kernels may differ from S * ws * xs in 64 bits only by the conversion of S to
FP32 (exact below 2^24, which the inputs here keep unless a test says
otherwise) and two FP32 multiplications: |err| <= 2^-22 |y|.  BF16 output has
to be the bits of (S * ws) * xs in FP32, rounded once.
"""
import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu

REL = 2.0 ** -22


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    return gg.load_library()


def _ints(shape, rng, lo=-128, hi=128):
    import torch
    return torch.from_numpy(rng.integers(lo, hi, size=shape, dtype=np.int8)).cuda()


def _scales(shape, rng):
    import torch
    return torch.from_numpy((rng.random(shape) + 0.5).astype(np.float32)).cuda()


def _want(q, xs, W, ws, sizes, rows=None):
    """S * ws * xs in 64 bits, and (S * ws) * xs in 32; S is exact (below 2^53)."""
    import torch
    q = q.double()
    if rows is not None:
        q, xs = q[rows.long()], xs[rows.long()]
    S, scale, at = [], [], 0
    for e, n in enumerate(sizes):
        S.append(q[at:at + n] @ W[e].double().T)
        scale.append(ws[e].expand(n, -1))
        at += n
    S, scale, xs = torch.cat(S), torch.cat(scale), xs[:at, None]
    return S * scale.double() * xs.double(), S.float() * scale * xs


def _close(got, want, out_dtype):
    import torch
    want64, want32 = want
    if out_dtype == "bf16":
        assert torch.equal(got, want32.to(torch.bfloat16))
        return
    err = (got.double() - want64).abs()
    bad = err > REL * want64.abs()
    assert not bad.any(), f"{int(bad.sum())} of {bad.numel()} outside, worst {float((err / want64.abs().clamp(min=1e-30)).max()):.3e}"


def _offsets(sizes):
    import torch
    return torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,N,K", [
    (1, 8, 16), (1, 1000, 4096), (2, 24, 48), (3, 136, 2064), (5, 72, 112), (8, 4096, 640), (9, 40, 1024),
    (17, 264, 176), (31, 128, 128), (33, 520, 1040), (64, 256, 256), (65, 1000, 384), (127, 640, 144),
    (129, 136, 528), (193, 264, 272), (257, 520, 640), (1001, 392, 1008),
])
def test_dense(T, N, K, out_dtype):
    rng = np.random.default_rng(T * 7 + N + K)
    q, W = _ints((T, K), rng), _ints((N, K), rng)
    xs, ws = _scales(T, rng), _scales(N, rng)
    got = gg.int8_gemm(q, W, ws, xs=xs, out_dtype=out_dtype)
    _close(got, _want(q, xs, W[None], ws[None], [T]), out_dtype)


SIZES = [
    [1], [0, 1, 0], [3, 0, 5, 1], [0, 0, 0, 7], [9, 8, 7, 16, 0, 1], [33, 1, 0, 64, 17],
    [130, 0, 2, 257, 31], [0, 500, 0, 100, 1, 1, 0],
]


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("sizes", SIZES, ids=str)
@pytest.mark.parametrize("N,K", [(72, 112), (264, 528)])
@pytest.mark.parametrize("routed", [False, True])
def test_grouped(sizes, N, K, routed, out_dtype):
    import torch
    E, M = len(sizes), sum(sizes)
    rng = np.random.default_rng(M + N + routed)
    T = max(1, M // 2) if routed else M
    q, W = _ints((T, K), rng), _ints((E, N, K), rng)
    xs, ws = _scales(T, rng), _scales((E, N), rng)
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda() if routed else None
    got = gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes), rows=rows, out_dtype=out_dtype)
    _close(got, _want(q, xs, W, ws, sizes, rows), out_dtype)


@pytest.mark.parametrize("E,M", [(200, 40), (1024, 900), (1024, 8)])
def test_many_experts(E, M):
    rng = np.random.default_rng(E)
    sizes = [int(v) for v in rng.multinomial(M, [1 / E] * E)]
    N, K = 40, 80
    q, W = _ints((M, K), rng), _ints((E, N, K), rng)
    xs, ws = _scales(M, rng), _scales((E, N), rng)
    got = gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes), out_dtype="fp32")
    _close(got, _want(q, xs, W, ws, sizes), "fp32")


@pytest.mark.parametrize("M", [6, 300])
def test_rows_past_the_last_offset_and_bands(M):
    """Rows past offsets[E] and the memory around Y stay as they were."""
    import torch
    rng = np.random.default_rng(5)
    sizes, N, K = [M // 2, 0, M - M // 2 - 2], 40, 64
    q, W, xs, ws = _ints((M, K), rng), _ints((3, N, K), rng), _scales(M, rng), _scales((3, N), rng)
    band = torch.full((M + 16, N), 7.0, dtype=torch.float32, device="cuda")
    out = band[8:8 + M]
    gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes), out_dtype="fp32", out=out)
    _close(out[:M - 2], _want(q, xs, W, ws, sizes), "fp32")
    assert (band[:8] == 7).all() and (band[8 + M - 2:] == 7).all()


@pytest.mark.parametrize("T,K", [(1, 4096), (40, 8192)])
def test_extreme_bytes_sum_exactly(T, K):
    """-128 everywhere: S = 2^14 K is a multiple of a large power of two, exact in FP32."""
    import torch
    q = torch.full((T, K), -128, dtype=torch.int8, device="cuda")
    W = torch.full((24, K), -128, dtype=torch.int8, device="cuda")
    one = torch.ones(T, device="cuda")
    got = gg.int8_gemm(q, W, torch.ones(24, device="cuda"), xs=one, out_dtype="fp32")
    assert (got == float(K * 128 * 128)).all()


def _rows_of(T, K, dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn((T, K), generator=g, device="cuda") * (0.1 + 10 * torch.rand((T, 1), generator=g, device="cuda"))
    return x.to(dtype)


def _gated(x):
    g, u = x.double().chunk(2, dim=1)
    return g / (1 + (-g).exp()) * u


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("T,K", [(1, 16), (1, 4096), (7, 48), (33, 1040), (3, 8192), (2, 40000), (5, 131056)])
def test_quantize_rows(T, K, act, dtype):
    """|q - h 127 / a| <= 1/2 plus FP32 error: h carries at most 6 roundings (2^-21 of it, the
    exponential's two ulp among them), a and 127 / a and the product 3 more: 127 * 2^-20 in all."""
    import torch
    x = _rows_of(T, K * (2 if act else 1), torch.bfloat16 if dtype == "bf16" else torch.float32, K + T)
    q, s = gg.quantize_rows(x, act=act)
    h = _gated(x) if act else x.double()
    a = h.abs().amax(dim=1)
    assert ((s.double() - a / 127).abs() <= 2.0 ** -20 * a / 127).all()
    assert ((q.double() - h * (127 / a)[:, None]).abs() <= 0.5 + 127 * 2.0 ** -20).all()
    assert int(q.abs().amax()) == 127


def test_quantize_rows_ties_go_to_even():
    import torch
    x = torch.tensor([[127.0, 0.5, 1.5, 2.5, -0.5, -1.5, -2.5, 126.5] + [0.0] * 8], device="cuda")
    q, s = gg.quantize_rows(x)
    assert float(s[0]) == 1.0
    assert q[0, :8].tolist() == [127, 0, 2, 2, 0, -2, -2, 126]


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_rows_that_hold_nothing_or_no_number(dtype):
    import torch
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    x = torch.ones((6, 32), dtype=dt, device="cuda")
    x[0] = 0.0
    x[1, 5] = float("nan")
    x[2, 31] = float("inf")
    x[3, 0] = float("-inf")
    x[4] = 2.0 ** -121
    q, s = gg.quantize_rows(x)
    assert torch.isnan(s[1:4]).all() and float(s[0]) == 0 and float(s[4]) == 0
    assert not q[:5].any() and (q[5] == 127).all()
    W, ws = torch.ones((8, 32), dtype=torch.int8, device="cuda"), torch.ones(8, device="cuda")
    y = gg.int8_gemm(x, W, ws, out_dtype="fp32")
    assert torch.isnan(y[1:4]).all() and not y[0].any() and not y[4].any()
    assert (y[5] == 127 * 32 * (s[5])).all()


@pytest.mark.parametrize("T", [3, 14, 90, 700])
def test_rows_without_numbers_stay_by_themselves(T):
    """A row that holds a NaN or an infinity gives NaN; its neighbours in the tile are as without it."""
    import torch
    rng = np.random.default_rng(T)
    N, K = 136, 400
    W, ws = _ints((N, K), rng), _scales(N, rng)
    x = _rows_of(T, K, torch.bfloat16, T)
    clean = gg.int8_gemm(x, W, ws)
    x[0, 7], x[T // 2, 0] = float("nan"), float("inf")
    got = gg.int8_gemm(x, W, ws)
    keep = torch.ones(T, dtype=torch.bool, device="cuda")
    keep[0] = keep[T // 2] = False
    assert torch.isnan(got[~keep]).all() and torch.equal(got[keep], clean[keep])


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("sizes,T,N,K", [([1], 1, 264, 1024), ([2, 0, 5], 7, 72, 112), ([40, 0, 90, 3], 50, 136, 528),
                                         ([300, 212], 512, 256, 256)])
def test_quantised_on_the_way(sizes, T, N, K, act, dtype):
    """Activations give the bits of quantising first and multiplying after."""
    import torch
    E, M = len(sizes), sum(sizes)
    rng = np.random.default_rng(M)
    x = _rows_of(T, K * (2 if act else 1), torch.bfloat16 if dtype == "bf16" else torch.float32, M)
    W, ws = _ints((E, N, K), rng), _scales((E, N), rng)
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda() if T != M else None
    q, s = gg.quantize_rows(x, act=act)
    for out_dtype in ("bf16", "fp32"):
        got = gg.int8_gemm(x, W, ws, offsets=_offsets(sizes), rows=rows, act=act, out_dtype=out_dtype)
        two = gg.int8_gemm(q, W, ws, xs=s, offsets=_offsets(sizes), rows=rows, out_dtype=out_dtype)
        assert torch.equal(got, two)
        _close(got, _want(q, s, W, ws, sizes, rows), out_dtype)


@pytest.mark.parametrize("M", [5, 150])
def test_same_bits_on_every_call_and_sm_cap(M):
    import torch
    rng = np.random.default_rng(M)
    sizes, N, K = [M // 3, 0, M - M // 3], 392, 1040
    x, W, ws = _rows_of(M, K, torch.bfloat16, M), _ints((3, N, K), rng), _scales((3, N), rng)
    offs = _offsets(sizes)
    first = gg.int8_gemm(x, W, ws, offsets=offs)
    for cap in (0, 0, 100, 7, 1):
        assert torch.equal(first, gg.int8_gemm(x, W, ws, offsets=offs, max_sms=cap))


@pytest.mark.parametrize("M", [4, 100])
def test_workspace_is_used_again_and_graphs_replay(M):
    import torch
    rng = np.random.default_rng(M)
    N, K = 264, 512
    W, ws = _ints((N, K), rng), _scales(N, rng)
    plan = gg.cake_gg_i8_plan(1, M, M, N, K)
    work = gg.make_workspace(plan, "cuda")
    x, y = torch.empty((M, K), dtype=torch.bfloat16, device="cuda"), torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    call = lambda: gg.int8_gemm(x, W, ws, out=y, plan=plan, workspace=work, check=False)
    x.copy_(_rows_of(M, K, torch.bfloat16, 1))
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in (2, 3, 4):
        x.copy_(_rows_of(M, K, torch.bfloat16, seed))
        call()
        one = y.clone()
        y.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, one)
        q, s = gg.quantize_rows(x)
        _close(y, _want(q, s, W[None], ws[None], [M]), "bf16")
    assert gg.cake_gg_check_status(work) == gg.CAKE_GG_OK


@pytest.mark.parametrize("M", [5, 90])
def test_side_stream(M):
    """Work queued on another stream sees that stream's earlier writes."""
    import torch
    rng = np.random.default_rng(9)
    N, K = 136, 2048
    W, ws = _ints((N, K), rng), _scales(N, rng)
    x = _rows_of(M, K, torch.bfloat16, 3)
    want = gg.int8_gemm(x, W, ws)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        late, w2 = torch.zeros_like(x), torch.zeros_like(W)
        torch.cuda._sleep(2_000_000)
        late.copy_(x)
        w2.copy_(W)
        got = gg.int8_gemm(late, w2, ws)
    side.synchronize()
    assert torch.equal(got, want)


@pytest.mark.parametrize("M", [6, 200])
@pytest.mark.parametrize("offsets", [[1, 3, 6], [0, 4, 3], [0, 2, 10 ** 6]])
def test_bad_offsets_are_reported(M, offsets):
    import torch
    rng = np.random.default_rng(1)
    q, W = _ints((M, 64), rng), _ints((2, 16, 64), rng)
    with pytest.raises(gg.CakeGGError) as err:
        gg.int8_gemm(q, W, _scales((2, 16), rng), xs=_scales(M, rng),
                     offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
    assert err.value.code == gg.CAKE_GG_ERR_BAD_OFFSETS


@pytest.mark.parametrize("M", [6, 200])
@pytest.mark.parametrize("bad", [-1, 11, 2 ** 31 - 1])
def test_bad_rows_are_reported(M, bad):
    import torch
    rng = np.random.default_rng(1)
    q, W = _ints((11, 64), rng), _ints((16, 64), rng)
    rows = torch.zeros(M, dtype=torch.int32, device="cuda")
    rows[M // 2] = bad
    with pytest.raises(gg.CakeGGError) as err:
        gg.int8_gemm(q, W, _scales(16, rng), xs=_scales(11, rng), rows=rows)
    assert err.value.code == gg.CAKE_GG_ERR_BAD_ROWS


def test_no_rows():
    import torch
    W, ws = torch.ones((16, 32), dtype=torch.int8, device="cuda"), torch.ones(16, device="cuda")
    x = torch.empty((0, 32), dtype=torch.bfloat16, device="cuda")
    assert gg.int8_gemm(x, W, ws).shape == (0, 16)
    q, s = gg.quantize_rows(x)
    assert q.shape == (0, 32) and s.shape == (0,)


def test_a_wait_that_runs_out_is_reported():
    """A dropped copy: the bounded waits end, the status says so, the next call is right again."""
    import torch
    rng = np.random.default_rng(2)
    M, N, K = 700, 264, 1040
    q, W, xs, ws = _ints((M, K), rng), _ints((N, K), rng), _scales(M, rng), _scales(N, rng)
    for rows in (64, M):
        plan = gg.cake_gg_i8_plan(1, rows, rows, N, K, "int8", None, "fp32")
        work = gg.make_workspace(plan, "cuda")
        out = torch.empty((rows, N), device="cuda")
        plan.debug_flags, plan.timeout_ns = gg.CAKE_GG_DEBUG_DROP_FIRST_LOAD, 50_000_000
        with pytest.raises(gg.CakeGGError) as err:
            gg.int8_gemm(q[:rows], W, ws, xs=xs[:rows], out_dtype="fp32", out=out, plan=plan, workspace=work)
        assert err.value.code == gg.CAKE_GG_ERR_TIMEOUT
        plan.debug_flags, plan.timeout_ns = 0, 2_000_000_000
        gg.int8_gemm(q[:rows], W, ws, xs=xs[:rows], out_dtype="fp32", out=out, plan=plan, workspace=work)
        _close(out, _want(q[:rows], xs[:rows], W[None], ws[None], [rows]), "fp32")


@pytest.mark.parametrize("env", [
    dict(PATH="0"), dict(PATH="2", ROWS_PER_TILE="16"), dict(PATH="2", ROWS_PER_TILE="32"),
    dict(PAIR="1", ROWS_PER_TILE="32", SPLITS="1"), dict(PAIR="1", ROWS_PER_TILE="32", SPLITS="3"),
    dict(PAIR="1", ROWS_PER_TILE="64", SPLITS="8"), dict(PAIR="1", ROWS_PER_TILE="128", SPLITS="1"),
    dict(PAIR="2", ROWS_PER_TILE="64", SPLITS="1"),
    dict(PAIR="2", ROWS_PER_TILE="128", SPLITS="1"), dict(PAIR="2", ROWS_PER_TILE="192", SPLITS="1"),
    dict(PAIR="1", ROWS_PER_TILE="96", SPLITS="2"), dict(PAIR="2", ROWS_PER_TILE="160", SPLITS="1"),
], ids=lambda e: "-".join(e.values()))
@pytest.mark.parametrize("routed", [False, True])
def test_every_tile_shape(env, routed, monkeypatch):
    """Each shape of tile on the same ragged rows, with one CTA or pair and with all."""
    import torch
    for k, v in dict(dict(PATH="1"), **env).items():
        monkeypatch.setenv("CAKE_GG_I8_" + k, v)
    rng = np.random.default_rng(4)
    sizes, N, K = [5, 0, 290, 1, 0, 33, 64, 17], 392, 1200
    E, M = len(sizes), sum(sizes)
    T = 77 if routed else M
    q, W, xs, ws = _ints((T, K), rng), _ints((E, N, K), rng), _scales(T, rng), _scales((E, N), rng)
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda() if routed else None
    want = _want(q, xs, W, ws, sizes, rows)
    for out_dtype in ("fp32", "bf16"):
        for cap in (0, 2):
            got = gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes), rows=rows, out_dtype=out_dtype, max_sms=cap)
            _close(got, want, out_dtype)


@pytest.mark.parametrize("T", [12, 100, 600])
@pytest.mark.parametrize("K", [4096, 32768, 131056])
def test_sums_past_24_bits(T, K):
    """One-signed bytes: sums past 2^24 are FP32 sums of K / 16 steps, each off by at most a unit in
    the last place of the running sum (2^-23 of it), and rounded three times more."""
    rng = np.random.default_rng(K)
    N = 64
    q, W = _ints((T, K), rng, 90, 128), _ints((N, K), rng, 90, 128)
    xs, ws = _scales(T, rng), _scales(N, rng)
    got = gg.int8_gemm(q, W, ws, xs=xs, out_dtype="fp32")
    want, _ = _want(q, xs, W[None], ws[None], [T])
    off = float(((got.double() - want).abs() / want.abs()).max())
    print(f"T {T} K {K}: {off:.3e}")
    assert off <= K / 16 * 2.0 ** -23 + 2.0 ** -21


@pytest.mark.parametrize("first", [1, 63, 160, 333, 409])
@pytest.mark.parametrize("x_dtype,act", [("int8", None), ("bf16", None), ("fp32", None), ("bf16", "silu_mul")])
@pytest.mark.parametrize("sizes", [[410], [5, 0, 290, 1, 0, 33, 64, 15]], ids=["dense", "grouped"])
def test_first_product(sizes, x_dtype, act, first, monkeypatch):
    """The rows divided between two products give the undivided call's bits, also where the second
    token pass of one call and the first of the next follow at once on the same workspace."""
    import torch
    E, N, K, M = len(sizes), 392, 1200, 410                     # (grouped: two rows past the last offset)
    rng = np.random.default_rng(first)
    W, ws = _ints((E, N, K), rng), _scales((E, N), rng)
    monkeypatch.setenv("CAKE_GG_I8_PATH", "1")
    plans = []
    for rows in (0, first):
        monkeypatch.setenv("CAKE_GG_I8_FIRST_ROWS", str(rows))
        plans.append(gg.cake_gg_i8_plan(E, M, M, N, K, x_dtype, act, "bf16"))
        assert plans[-1].first_rows == (rows if plans[-1].splits == 1 else 0)
    xs = _scales(M, rng) if x_dtype == "int8" else None
    inputs = []
    for seed in range(4):
        if x_dtype == "int8":
            inputs.append(_ints((M, K), rng))
        else:
            dtype = torch.bfloat16 if x_dtype == "bf16" else torch.float32
            inputs.append(_rows_of(M, 2 * K if act else K, dtype, seed))
    got = []
    for plan in plans:
        work = gg.make_workspace(plan, "cuda")
        outs = [torch.full((M, N), 7.0, dtype=torch.bfloat16, device="cuda") for _ in inputs]
        for x, out in zip(inputs * 3, outs * 3):
            gg.int8_gemm(x, W, ws, xs=xs, offsets=_offsets(sizes), act=act, out=out, plan=plan, workspace=work, check=False)
        assert gg.cake_gg_check_status(work) == gg.CAKE_GG_OK
        got.append(outs)
    for x, one, two in zip(inputs, *got):
        assert torch.equal(one, two)
        q, s = (x, xs) if xs is not None else gg.quantize_rows(x, act=act)
        used = sum(sizes)
        _close(two[:used], _want(q, s, W, ws, sizes), "bf16")
        assert (two[used:] == 7).all()


@pytest.mark.parametrize("E", [1, 6])
def test_first_product_by_its_own_rule(E):
    """A call long enough to be divided, as planned, against the same call undivided; routed rows
    leave it undivided, and a graph replays it."""
    import torch
    M, N, K = 12000, 2048, 8192
    rng = np.random.default_rng(E)
    W, ws = _ints((E, N, K), rng), _scales((E, N), rng)
    x = _rows_of(M, 2 * K, torch.bfloat16, 2)
    sizes = [M] if E == 1 else [0, 5000, 1, 1999, 0, 5000]
    plan, whole = (gg.cake_gg_i8_plan(E, M, M, N, K, "bf16", "silu_mul", "bf16") for _ in range(2))
    assert plan.first_rows > 0
    whole.first_rows = 0
    work = gg.make_workspace(plan, "cuda")
    out = torch.empty((M, N), dtype=torch.bfloat16, device="cuda")
    more = dict(offsets=_offsets(sizes), act="silu_mul", out=out, workspace=work)
    call = lambda p: gg.int8_gemm(x, W, ws, plan=p, **more)
    want = call(whole).clone()
    for _ in range(5):
        out.zero_()
        assert torch.equal(call(plan), want)
    rows = torch.arange(M, dtype=torch.int32, device="cuda")
    out.zero_()
    gg.int8_gemm(x, W, ws, rows=rows, plan=plan, **more)
    assert torch.equal(out, want)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        gg.int8_gemm(x, W, ws, plan=plan, check=False, **more)
    out.zero_()
    graph.replay()
    graph.replay()
    assert torch.equal(out, want)


@pytest.mark.parametrize("T,K", [(305, 16), (700, 272), (401, 512), (333, 528), (306, 1040), (310, 11008)])
@pytest.mark.parametrize("act", [None, "silu_mul"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_quantize_many_rows(T, K, act, dtype):
    """More rows than blocks of a row each start at once: several short rows in a block, the last block
    with fewer, and long rows by fewer threads.  Each row is what the same row alone gives (bit for bit:
    its values do not depend on the threads that share it)."""
    import torch
    x = _rows_of(T, 2 * K if act else K, torch.bfloat16 if dtype == "bf16" else torch.float32, T)
    q, s = gg.quantize_rows(x, act=act)
    for rows in (slice(0, 5), slice(T // 2, T // 2 + 3), slice(T - 3, T)):
        one_q, one_s = gg.quantize_rows(x[rows].contiguous(), act=act)
        assert torch.equal(q[rows], one_q) and torch.equal(s[rows], one_s)
    wide = q.int().abs().max(dim=1).values
    assert (wide == 127).all()                                   # the largest value of a row is 127


@pytest.mark.parametrize("sizes", [[5, 0, 3, 0, 0, 4, 0, 0, 0, 0, 0, 0], [12] + [0] * 11, [0] * 15 + [16], [1, 2] * 8 + [0] * 8])
@pytest.mark.parametrize("x_dtype", ["int8", "bf16"])
def test_few_rows_of_many_experts_that_meet(sizes, x_dtype):
    """Plans for rows that meet experts of their own, with rows that do not: longer runs than planned for."""
    import torch
    E, M, N, K = len(sizes), sum(sizes), 136, 2064
    rng = np.random.default_rng(M)
    W, ws = _ints((E, N, K), rng), _scales((E, N), rng)
    assert gg.cake_gg_i8_plan(E, M, M, N, K, x_dtype, None, "bf16").path == 0
    if x_dtype == "int8":
        q, xs = _ints((M, K), rng), _scales(M, rng)
        got = gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes))
    else:
        x = _rows_of(M, K, torch.bfloat16, 3)
        q, xs = gg.quantize_rows(x)
        got = gg.int8_gemm(x, W, ws, offsets=_offsets(sizes))
    _close(got, _want(q, xs, W, ws, sizes), "bf16")


@pytest.mark.parametrize("K", [16, 144, 400])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
def test_short_reductions(K, out_dtype):
    """One to four stages a tile and many tiles a CTA: a tile's scales are loaded during the one before."""
    import torch
    sizes = [700, 0, 1, 3000, 64, 33, 2000, 202]
    E, M, N, T = len(sizes), sum(sizes), 904, 1500
    rng = np.random.default_rng(K)
    q, W, xs, ws = _ints((T, K), rng), _ints((E, N, K), rng), _scales(T, rng), _scales((E, N), rng)
    rows = torch.from_numpy(rng.integers(0, T, size=M).astype(np.int32)).cuda()
    want = _want(q, xs, W, ws, sizes, rows)
    for cap in (0, 3):
        got = gg.int8_gemm(q, W, ws, xs=xs, offsets=_offsets(sizes), rows=rows, out_dtype=out_dtype, max_sms=cap)
        _close(got, want, out_dtype)
