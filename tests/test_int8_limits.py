"""Sizes at the ends of what the 8-bit products take: plans, refusals, and index ranges."""
import ctypes

import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

ROWS, MMA, WARPS = 0, 1, 2


@pytest.fixture(scope="module", autouse=True)
def lib():
    gg_build.build()
    return gg.load_library()


def _gpu():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    return torch


@pytest.mark.parametrize("E,T,M,N,K", [(4, 2, 10000, 512, 1024), (8, 2, 1 << 24, 4096, 256), (4, 1, 64, 2048, 8192),
                                       (64, 2, 129, 2048, 4096), (2, 1, 3000, 1000, 512)])
def test_a_few_tokens_that_many_rows_name_are_many_rows(E, T, M, N, K):
    """More rows than experts times tokens: a token meets an expert more than once, and the few-row
    path would read an expert's weights again for every two rows."""
    assert gg.cake_gg_i8_plan(E, M, T, N, K).path == MMA


def test_a_token_through_experts_of_its_own_keeps_the_few_row_path():
    for E, T, M in ((32, 1, 4), (8, 1, 8), (32, 2, 8), (64, 2, 16), (32, 16, 16)):
        assert gg.cake_gg_i8_plan(E, M, T, 4096, 2048).path == ROWS


@pytest.mark.gpu
@pytest.mark.parametrize("x_dtype", ["int8", "bf16"])
def test_few_tokens_named_by_many_rows(x_dtype):
    torch = _gpu()
    E, T, M, N, K = 4, 2, 10000, 136, 272
    g = torch.Generator(device="cuda").manual_seed(0)
    W = torch.randint(-128, 128, (E, N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand((E, N), generator=g, device="cuda") + 0.5
    sizes = [5000, 0, 4999, 1]
    off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    rows = torch.randint(0, T, (M,), generator=g, device="cuda", dtype=torch.int32)
    x = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16)
    q, xs = gg.quantize_rows(x)
    got = gg.int8_gemm(q, W, ws, xs=xs, offsets=off, rows=rows) if x_dtype == "int8" else gg.int8_gemm(x, W, ws, offsets=off, rows=rows)
    e_of = torch.repeat_interleave(torch.arange(E, device="cuda"), torch.tensor(sizes, device="cuda"))
    sums = torch.einsum("tk,enk->ten", q.double(), W.double())          # every token through every expert
    t = rows.long()
    want = sums[t, e_of].float() * ws[e_of] * xs[t, None]
    assert torch.equal(got, want.to(torch.bfloat16))


@pytest.mark.parametrize("value", ["-1", "3", "7", "1000000"])
def test_a_path_that_is_none_is_no_override(value, monkeypatch):
    want = gg.cake_gg_i8_plan(1, 12, 12, 256, 1024).as_dict()
    monkeypatch.setenv("CAKE_GG_I8_PATH", value)
    assert gg.cake_gg_i8_plan(1, 12, 12, 256, 1024).as_dict() == want


@pytest.mark.parametrize("rows", ["0", "8", "48", "64", "192"])
@pytest.mark.parametrize("M", [12, 30])
def test_rows_that_a_path_cannot_take_are_no_override(M, rows, monkeypatch):
    """A documented value of another path's range: the call would refuse the plan it was written into."""
    want = gg.cake_gg_i8_plan(1, M, M, 256, 1024)
    assert want.path == WARPS and want.tile_rows in (16, 32)
    monkeypatch.setenv("CAKE_GG_I8_ROWS_PER_TILE", rows)
    assert gg.cake_gg_i8_plan(1, M, M, 256, 1024).as_dict() == want.as_dict()


def _raw_plan(E, M, T, N, K, x_dtype, path, monkeypatch):
    monkeypatch.setenv("CAKE_GG_I8_PATH", str(path))
    plan = gg.cake_gg_i8_plan(E, M, T, N, K, x_dtype)
    assert plan.path == path
    return plan


@pytest.mark.gpu
@pytest.mark.parametrize("path,M,N,K", [(ROWS, 1 << 24, 4096, 256), (WARPS, 1 << 24, 4096, 256), (MMA, 64, 1 << 24, 131056)],
                         ids=["rows", "warps", "mma"])
def test_a_refused_call_enqueues_nothing(path, M, N, K, monkeypatch):
    """Grids and strides past the hardware's limits, with activations: no token pass before the refusal.
    (Y, W and the row numbers are made up: no kernel that reads them can be launched.)"""
    torch = _gpu()
    T = 64
    plan = _raw_plan(1, M, T, N, K, "bf16", path, monkeypatch)
    x = torch.ones((T, K), dtype=torch.bfloat16, device="cuda")
    work = torch.full((int(plan.workspace_bytes),), 0x5A, dtype=torch.uint8, device="cuda")
    address = 1 << 20
    rc = gg.cake_gg_i8_gemm(plan, x, None, address if M != T else None, address, address, address, None, work,
                            stream=torch.cuda.current_stream().cuda_stream)
    torch.cuda.synchronize()
    assert rc != gg.CAKE_GG_OK
    assert bool((work == 0x5A).all())


@pytest.mark.parametrize("N", [2 ** 31 - 8, 2 ** 31 - 504])
@pytest.mark.parametrize("M", [1, 40, 4096])
def test_channels_whose_tiles_pass_32_bits_are_refused(N, M):
    """N rounded up to whole tiles has to fit the kernels' 32-bit channel numbers."""
    with pytest.raises(gg.CakeGGError) as err:
        gg.cake_gg_i8_plan(1, M, M, N, 16)
    assert err.value.code == gg.CAKE_GG_ERR_OVERFLOW
    plan = gg.cake_gg_i8_plan(1, M, M, 2 ** 31 - 512, 16)
    plan.N = N
    address = 1 << 20
    assert gg.cake_gg_i8_gemm(plan, address, None, None, address, address, address, None, address,
                              workspace_bytes=plan.workspace_bytes, stream=0) == gg.CAKE_GG_ERR_OVERFLOW


@pytest.mark.gpu
def test_routed_rows_up_to_2_31():
    """The last expert's one row is the last row there can be: its tile ends past 2^31, and what it
    reads of the row numbers must not.  (M * N passes 2^31 sixteen times.)"""
    torch = _gpu()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    M, T, N, K = 2 ** 31 - 1, 1000, 8, 16
    g = torch.Generator(device="cuda").manual_seed(0)
    q = torch.randint(-128, 128, (T, K), generator=g, device="cuda", dtype=torch.int8)
    W = torch.randint(-128, 128, (2, N, K), generator=g, device="cuda", dtype=torch.int8)
    xs, ws = torch.rand(T, generator=g, device="cuda") + 0.5, torch.rand((2, N), generator=g, device="cuda") + 0.5
    rows = torch.arange(M, dtype=torch.int32, device="cuda").remainder_(T)
    off = torch.tensor([0, M - 1, M], dtype=torch.int32, device="cuda")
    assert gg.cake_gg_i8_plan(2, M, T, N, K, "int8").path == MMA
    y = gg.int8_gemm(q, W, ws, xs=xs, offsets=off, rows=rows)
    each = ((q.double() @ W.double().transpose(1, 2)).float() * ws[:, None] * xs[:, None]).to(torch.bfloat16)
    for at in range(0, M, 1 << 27):
        end = min(at + (1 << 27), M - 1)
        assert torch.equal(y[at:end], each[0][rows[at:end].long()])
    assert torch.equal(y[M - 1], each[1][int(rows[M - 1])])


@pytest.mark.gpu
@pytest.mark.parametrize("path", [ROWS, MMA, WARPS])
def test_weights_past_2_31(path, monkeypatch):
    """More than 2^31 weights: the last expert's, and its last channels, are read where they lie."""
    torch = _gpu()
    E, N, K, M = 33, 8200, 8192, 9
    assert E * N * K > 2 ** 31
    monkeypatch.setenv("CAKE_GG_I8_PATH", str(path))
    W = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    for e in range(E):
        W[e] = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8)
    ws = torch.rand((E, N), device="cuda") + 0.5
    q, xs = torch.randint(-128, 128, (M, K), device="cuda", dtype=torch.int8), torch.rand(M, device="cuda") + 0.5
    sizes = [2] + [0] * (E - 3) + [3, 4]
    off = torch.tensor([0] + list(np.cumsum(sizes)), dtype=torch.int32, device="cuda")
    assert gg.cake_gg_i8_plan(E, M, M, N, K, "int8").path == path
    got = gg.int8_gemm(q, W, ws, xs=xs, offsets=off)
    want = torch.cat([(q[a:b].double() @ W[e].double().T).float() * ws[e] for a, b, e in ((0, 2, 0), (2, 5, E - 2), (5, 9, E - 1))])
    assert torch.equal(got, (want * xs[:, None]).to(torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("x_dtype", ["int8", "bf16"])
def test_outputs_past_2_31(x_dtype):
    """More than 2^31 outputs and tokens' values, not routed; activations are divided between two products."""
    torch = _gpu()
    if torch.cuda.mem_get_info()[0] < 64 << 30:
        pytest.skip("needs 64 GB")
    M, N, K = 525000, 4096, 4112
    assert M * N > 2 ** 31 and M * K > 2 ** 31
    W, ws = torch.randint(-128, 128, (N, K), device="cuda", dtype=torch.int8), torch.rand(N, device="cuda") + 0.5
    if x_dtype == "int8":
        q = torch.empty((M, K), dtype=torch.int8, device="cuda").random_(-128, 128)
        xs = torch.rand(M, device="cuda") + 0.5
        y = gg.int8_gemm(q, W, ws, xs=xs)
    else:
        x = torch.empty((M, K), dtype=torch.bfloat16, device="cuda").normal_()
        y = gg.int8_gemm(x, W, ws)
        q, xs = gg.quantize_rows(x)
    for at in (0, 130000, 262143, 400001, M - 500):
        rows = slice(at, at + 500)
        want = (q[rows].double() @ W.double().T).float() * ws * xs[rows, None]
        assert torch.equal(y[rows], want.to(torch.bfloat16))


@pytest.mark.gpu
@pytest.mark.parametrize("path", [ROWS, MMA, WARPS])
@pytest.mark.parametrize("K", [16, 32, 48, 64, 80, 112])
@pytest.mark.parametrize("x_dtype", ["int8", "bf16"])
def test_rows_shorter_than_a_step(path, K, x_dtype, monkeypatch):
    torch = _gpu()
    monkeypatch.setenv("CAKE_GG_I8_PATH", str(path))
    g = torch.Generator(device="cuda").manual_seed(K)
    for M, N in ((1, 8), (5, 40), (16, 72), (31, 264)):
        W = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
        ws = torch.rand(N, generator=g, device="cuda") + 0.5
        x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
        q, xs = gg.quantize_rows(x)
        got = gg.int8_gemm(q, W, ws, xs=xs) if x_dtype == "int8" else gg.int8_gemm(x, W, ws)
        want = (q.double() @ W.double().T).float() * ws * xs[:, None]
        assert torch.equal(got, want.to(torch.bfloat16))
