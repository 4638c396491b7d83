"""Every kernel of the 8-bit products by name: errors, streams, graphs, rows without numbers, long sums.

The rules that choose a path move with the measurements; what has to hold on each of them is tested
here with the path, and the tensor-core path's shapes, set and asserted.
"""
import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu

# (overrides, rows that the form's own rule keeps it for); "rows" by the rows of a run: one and two are
# quantised by the blocks themselves, four after a token pass
FORMS = {
    "rows1": (dict(PATH=0), 1), "rows2": (dict(PATH=0), 2), "rows4": (dict(PATH=0), 7),
    "warps16": (dict(PATH=2, ROWS_PER_TILE=16), 13), "warps32": (dict(PATH=2, ROWS_PER_TILE=32), 31),
    "single32": (dict(PATH=1, PAIR=1, ROWS_PER_TILE=32, SPLITS=1), 40),
    "single96": (dict(PATH=1, PAIR=1, ROWS_PER_TILE=96, SPLITS=1), 200),
    "split3": (dict(PATH=1, PAIR=1, ROWS_PER_TILE=32, SPLITS=3), 40),
    "split8": (dict(PATH=1, PAIR=1, ROWS_PER_TILE=64, SPLITS=8), 100),
    "pair64": (dict(PATH=1, PAIR=2, ROWS_PER_TILE=64, SPLITS=1), 150),
    "pair192": (dict(PATH=1, PAIR=2, ROWS_PER_TILE=192, SPLITS=1), 500),
}


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    return gg.load_library()


@pytest.fixture(params=list(FORMS))
def form(request, monkeypatch):
    """Rows that the form takes; plans made from here on are its."""
    overrides, rows = FORMS[request.param]
    for k, v in overrides.items():
        monkeypatch.setenv("CAKE_GG_I8_" + k, str(v))
    plan = gg.cake_gg_i8_plan(1, rows, rows, 264, 2064)
    assert plan.path == overrides["PATH"]
    if plan.path == 1:
        assert (plan.pair, plan.tile_rows, plan.splits) == (overrides["PAIR"], overrides["ROWS_PER_TILE"], overrides["SPLITS"])
    return rows


def _ints(shape, rng, lo=-128, hi=128):
    import torch
    return torch.from_numpy(rng.integers(lo, hi, size=shape, dtype=np.int8)).cuda()


def _scales(shape, rng):
    import torch
    return torch.from_numpy((rng.random(shape) + 0.5).astype(np.float32)).cuda()


def _acts(T, K, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    return (torch.randn((T, K), generator=g, device="cuda") * (0.1 + torch.rand((T, 1), generator=g, device="cuda"))).to(torch.bfloat16)


def _want(x, W, ws):
    """(S * ws) * xs in FP32, rounded once, of one expert's rows; S is exact."""
    import torch
    q, xs = gg.quantize_rows(x)
    return ((q.double() @ W.double().T).float() * ws * xs[:, None]).to(torch.bfloat16)


@pytest.mark.parametrize("x_dtype", ["bf16", "int8"])
@pytest.mark.parametrize("offsets", [[1, 2, 3], [0, 4, 1], [0, 1, 10 ** 6], [0, -1, 1]])
def test_bad_offsets_are_reported(form, offsets, x_dtype):
    import torch
    rng = np.random.default_rng(1)
    off = torch.tensor(offsets, dtype=torch.int32, device="cuda")
    x = _acts(form, 2064, 0) if x_dtype == "bf16" else _ints((form, 2064), rng)
    xs = None if x_dtype == "bf16" else _scales(form, rng)
    with pytest.raises(gg.CakeGGError) as err:
        gg.int8_gemm(x, _ints((2, 16, 2064), rng), _scales((2, 16), rng), xs=xs, offsets=off)
    assert err.value.code == gg.CAKE_GG_ERR_BAD_OFFSETS


@pytest.mark.parametrize("x_dtype", ["bf16", "int8"])
@pytest.mark.parametrize("bad", [-1, 11, 2 ** 31 - 1, -2 ** 31])
def test_bad_rows_are_reported_and_the_others_right(form, bad, x_dtype):
    import torch
    rng = np.random.default_rng(1)
    T, N, K = 11, 136, 2064
    x, W, ws = _acts(T, K, 1), _ints((N, K), rng), _scales(N, rng)
    rows = torch.from_numpy(rng.integers(0, T, size=form).astype(np.int32)).cuda()
    want = _want(x, W, ws)[rows.long()]
    rows[form // 2] = bad
    plan = gg.cake_gg_i8_plan(1, form, T, N, K, x_dtype)
    work, out = gg.make_workspace(plan, "cuda"), torch.zeros((form, N), dtype=torch.bfloat16, device="cuda")
    q, s = gg.quantize_rows(x)
    more = dict(rows=rows, plan=plan, workspace=work, out=out, check=False)
    gg.int8_gemm(x, W, ws, **more) if x_dtype == "bf16" else gg.int8_gemm(q, W, ws, xs=s, **more)
    assert gg.cake_gg_check_status(work) == gg.CAKE_GG_ERR_BAD_ROWS
    keep = torch.arange(form, device="cuda") != form // 2
    assert torch.equal(out[keep], want[keep])
    rows[form // 2] = 0                                          # and the next call is right again
    gg.int8_gemm(x, W, ws, **more) if x_dtype == "bf16" else gg.int8_gemm(q, W, ws, xs=s, **more)
    assert gg.cake_gg_check_status(work) == gg.CAKE_GG_OK
    assert torch.equal(out, _want(x, W, ws)[rows.long()])


def test_rows_without_numbers_stay_by_themselves(form):
    import torch
    rng = np.random.default_rng(2)
    N, K = 136, 2064
    x, W, ws = _acts(form, K, 2), _ints((N, K), rng), _scales(N, rng)
    want = _want(x, W, ws)
    x[0, 7], x[form // 2, K - 1] = float("nan"), float("-inf")
    got = gg.int8_gemm(x, W, ws)
    keep = torch.ones(form, dtype=torch.bool, device="cuda")
    keep[0] = keep[form // 2] = False
    assert torch.isnan(got[~keep]).all() and torch.equal(got[keep], want[keep])


@pytest.mark.parametrize("routed", [False, True])
def test_graphs_replay(form, routed):
    """A captured call follows its inputs, weights, offsets and row numbers on every replay."""
    import torch
    rng = np.random.default_rng(3)
    N, K = 136, 2064
    x, W, ws = _acts(form, K, 0), _ints((2, N, K), rng), _scales((2, N), rng)
    off = torch.tensor([0, form, form], dtype=torch.int32, device="cuda")
    rows = torch.arange(form, dtype=torch.int32, device="cuda") if routed else None
    plan = gg.cake_gg_i8_plan(2, form, form, N, K)
    work, y = gg.make_workspace(plan, "cuda"), torch.empty((form, N), dtype=torch.bfloat16, device="cuda")
    call = lambda: gg.int8_gemm(x, W, ws, offsets=off, rows=rows, out=y, plan=plan, workspace=work, check=False)  # noqa: E731
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for seed in range(1, 5):
        cut = seed * form // 5
        x.copy_(_acts(form, K, seed))
        W.copy_(_ints((2, N, K), np.random.default_rng(seed)))
        off.copy_(torch.tensor([0, cut, form], dtype=torch.int32))
        if routed:
            rows.copy_(torch.randperm(form, generator=torch.Generator().manual_seed(seed)).to(torch.int32))
        y.zero_()
        graph.replay()
        src = x[rows.long()] if routed else x
        want = torch.cat([_want(src[a:b], W[e], ws[e]) for e, (a, b) in enumerate([(0, cut), (cut, form)]) if b > a])
        assert torch.equal(y, want)
    assert gg.cake_gg_check_status(work) == gg.CAKE_GG_OK


@pytest.mark.parametrize("x_dtype", ["bf16", "int8"])
def test_a_side_streams_late_writes_are_seen(form, x_dtype):
    """Weights, scales, offsets and rows written just before the call, on a stream that was kept busy:
    what a kernel reads before the one in front of it has ended must not be of these."""
    import torch
    rng = np.random.default_rng(4)
    N, K = 136, 2064
    x, W, ws = _acts(form, K, 5), _ints((2, N, K), rng), _scales((2, N), rng)
    off = torch.tensor([0, form // 3, form], dtype=torch.int32, device="cuda")
    rows = torch.randperm(form, generator=torch.Generator().manual_seed(1)).to(torch.int32).cuda()
    src = x[rows.long()]
    want = torch.cat([_want(src[a:b], W[e], ws[e]) for e, (a, b) in enumerate([(0, form // 3), (form // 3, form)]) if b > a])
    q, s = gg.quantize_rows(x)
    given = [q, s, W, ws, off, rows] if x_dtype == "int8" else [x, W, ws, off, rows]
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        with torch.cuda.stream(side):
            late = [torch.zeros_like(t) for t in given]
            late[-2][1:] = form
            torch.cuda._sleep(2_000_000)
            for to, t in zip(late, given):
                to.copy_(t)
            xs = late.pop(1) if x_dtype == "int8" else None
            got = gg.int8_gemm(late[0], late[1], late[2], xs=xs, offsets=late[3], rows=late[4])
        side.synchronize()
        assert torch.equal(got, want)


@pytest.mark.parametrize("cap", [0, 100, 7, 1])
def test_same_bits_under_every_sm_cap(form, cap):
    import torch
    rng = np.random.default_rng(6)
    x, W, ws = _acts(form, 2064, 6), _ints((392, 2064), rng), _scales(392, rng)
    want = _want(x, W, ws)
    for _ in range(3):
        assert torch.equal(gg.int8_gemm(x, W, ws, max_sms=cap), want)


@pytest.mark.parametrize("K", [4096, 32768, 131056])
def test_sums_past_24_bits(form, K, request):
    """One-signed bytes.  The few-row kernels add integers: exact, and three roundings (2^-22).  The others add
    FP32 in K / 16 steps, each off by at most a unit in the last place of the running sum (2^-23 of it)."""
    import torch
    rng = np.random.default_rng(K)
    N = 64
    if gg.cake_gg_i8_plan(1, form, form, N, K, "int8", None, "fp32").path == 0:
        bound = 2.0 ** -22
    else:
        bound = K / 16 * 2.0 ** -23 + 2.0 ** -21
    q, W = _ints((form, K), rng, 90, 128), _ints((N, K), rng, 90, 128)
    xs, ws = _scales(form, rng), _scales(N, rng)
    got = gg.int8_gemm(q, W, ws, xs=xs, out_dtype="fp32")
    want = (q.double() @ W.double().T) * ws.double() * xs.double()[:, None]
    off = float(((got.double() - want).abs() / want.abs()).max())
    print(f"{request.node.name}: {off:.3e}")
    assert off <= bound


@pytest.mark.parametrize("routed", [False, True])
def test_a_wait_that_runs_out_is_reported(form, routed):
    """A dropped copy: every role's waits end, the status says so, and the next call is right."""
    import torch
    rng = np.random.default_rng(8)
    N, K, T = 264, 2064, form
    plan = gg.cake_gg_i8_plan(1, form, T, N, K, "int8", None, "fp32")
    if plan.path != 1:
        return                                                   # (nothing in the other kernels waits with a limit)
    q, W, xs, ws = _ints((T, K), rng), _ints((N, K), rng), _scales(T, rng), _scales(N, rng)
    rows = torch.from_numpy(rng.integers(0, T, size=form).astype(np.int32)).cuda() if routed else None
    work, out = gg.make_workspace(plan, "cuda"), torch.empty((form, N), device="cuda")
    more = dict(xs=xs, rows=rows, out_dtype="fp32", out=out, plan=plan, workspace=work)
    plan.debug_flags, plan.timeout_ns = gg.CAKE_GG_DEBUG_DROP_FIRST_LOAD, 50_000_000
    with pytest.raises(gg.CakeGGError) as err:
        gg.int8_gemm(q, W, ws, **more)
    assert err.value.code == gg.CAKE_GG_ERR_TIMEOUT
    plan.debug_flags, plan.timeout_ns = 0, 2_000_000_000
    gg.int8_gemm(q, W, ws, **more)
    src, scale = (q, xs) if rows is None else (q[rows.long()], xs[rows.long()])
    want = (src.double() @ W.double().T) * ws.double() * scale.double()[:, None]
    assert ((out.double() - want).abs() <= 2.0 ** -22 * want.abs()).all()
