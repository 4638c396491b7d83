"""Helpers that are given a stream: what they allocate belongs to that stream.

Output and workspace that a helper allocates are written by kernels on the stream it was given.
A workspace's zero fill on another stream could run while the product does, and memory that goes
back to another stream's pool could be handed out while the product still uses it.
"""
import contextlib

import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

CURRENT, SIDE = 0x1000, 0x2000


class FakeStream:
    def __init__(self, handle):
        self.cuda_stream = handle


class FakeTensor:
    def __init__(self, shape, dtype, index=0):
        import torch
        self.shape, self.dtype = torch.Size(shape), dtype
        self.device, self.is_cuda, self.nbytes = torch.device("cuda", index), True, 1 << 30
        self.recorded = []

    def get_device(self):
        return self.device.index

    def is_contiguous(self):
        return True

    def dim(self):
        return len(self.shape)

    def numel(self):
        return self.shape.numel()

    def element_size(self):
        return 1 << 20

    def data_ptr(self):
        return 1 << 20

    def record_stream(self, stream):
        self.recorded.append(stream.cuda_stream)


class Calls:
    """The library's plans, with its compute calls recorded instead of made."""

    def __init__(self, lib):
        self._lib, self.streams = lib, []

    def __getattr__(self, name):
        if name in ("cake_gg_i8_gemm", "cake_gg_i8_quant", "cake_gg_fwd", "cake_gg_router_fp32"):
            return lambda *args: self.streams.append(args[-1]) or gg.CAKE_GG_OK
        return getattr(self._lib, name)


@pytest.fixture
def host(monkeypatch):
    """A torch whose streams and allocations are recorded: [(what, stream it belongs to)]."""
    import torch
    gg_build.build()
    calls = Calls(gg.load_library())
    at, made = [CURRENT], []
    monkeypatch.setattr(gg, "_lib", calls)
    monkeypatch.setattr(gg, "_current_device", lambda: 0)
    monkeypatch.setattr(gg, "_current_stream", lambda index: at[-1])

    @contextlib.contextmanager
    def within(stream):
        at.append(stream.cuda_stream)
        yield
        at.pop()

    def allocate(name):
        def make(shape, *more, dtype=None, device=None):
            shape = (shape,) if isinstance(shape, int) else shape
            t = FakeTensor(shape, dtype)
            made.append((name, at[-1], t))
            return t
        return make
    monkeypatch.setattr(torch.cuda, "stream", within)
    monkeypatch.setattr(torch.cuda, "ExternalStream", lambda handle, device=None: FakeStream(handle))
    monkeypatch.setattr(torch.cuda, "default_stream", lambda device=None: FakeStream(0))
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream(at[-1]))
    monkeypatch.setattr(torch, "empty", allocate("empty"))
    monkeypatch.setattr(torch, "zeros", allocate("zeros"))
    return calls, made


def _calls():
    import torch
    bf16, f32, i32 = torch.bfloat16, torch.float32, torch.int32
    x, W, off = FakeTensor((64, 256), bf16), FakeTensor((2, 128, 256), torch.int8), FakeTensor((3,), i32)
    return {
        "int8_gemm": lambda **m: gg.int8_gemm(x, W, FakeTensor((2, 128), f32), offsets=off, check=False, **m),
        "quantize_rows": lambda **m: gg.quantize_rows(x, **m),
        "grouped_gemm": lambda **m: gg.grouped_gemm("fwd", x, FakeTensor((2, 128, 256), bf16), off, check=False, **m),
        "router_gemm": lambda **m: gg.router_gemm(FakeTensor((64, 256), f32), FakeTensor((16, 256), f32), check=False, **m),
    }


@pytest.mark.parametrize("name", ["int8_gemm", "quantize_rows", "grouped_gemm", "router_gemm"])
@pytest.mark.parametrize("given", [None, CURRENT, SIDE, 0, "object"])
def test_allocations_belong_to_the_stream_of_the_call(name, given, host):
    calls, made = host
    stream = FakeStream(SIDE) if given == "object" else given
    handle = CURRENT if given is None else SIDE if given == "object" else given
    out = _calls()[name](stream=stream)
    assert [s or 0 for s in calls.streams] == [handle]
    assert made and all(at == handle for _, at, _ in made), [(what, hex(at)) for what, at, _ in made]
    # a result is read on the caller's stream: its memory waits for that one too
    for t in out if isinstance(out, tuple) else (out,):
        assert t.recorded == ([] if handle == CURRENT else [CURRENT])


@pytest.mark.gpu
@pytest.mark.parametrize("as_int", [False, True])
@pytest.mark.parametrize("M", [5, 33, 300])
def test_stream_argument_beside_a_busy_current_stream(M, as_int):
    """The memory the workspace will take is left dirty, and the current stream busy: nothing of it
    may show on the given stream.  Then memory of the workspace's size is written on the current stream
    while the product is still queued on the other."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    N, K = 264, 2048
    g = torch.Generator(device="cuda").manual_seed(M)
    x = torch.randn((M, K), generator=g, device="cuda").to(torch.bfloat16)
    W = torch.randint(-128, 128, (N, K), generator=g, device="cuda", dtype=torch.int8)
    ws = torch.rand(N, generator=g, device="cuda")
    want, (want_q, want_s) = gg.int8_gemm(x, W, ws), gg.quantize_rows(x)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if as_int else side
    size = int(gg.cake_gg_i8_plan(1, M, M, N, K).workspace_bytes)
    torch.cuda.synchronize()
    for check in (True, False, False):
        dirty = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        with torch.cuda.stream(side):
            other = torch.full((size,), 255, dtype=torch.uint8, device="cuda")
        torch.cuda.synchronize()
        del dirty, other
        torch.cuda._sleep(20_000_000)                    # the current stream: some 10 ms
        if not check:
            with torch.cuda.stream(side):
                torch.cuda._sleep(40_000_000)
        got = gg.int8_gemm(x, W, ws, stream=stream, check=check)
        q, s = gg.quantize_rows(x, stream=stream)
        over = [torch.full((size,), 255, dtype=torch.uint8, device="cuda") for _ in range(4)]
        side.synchronize()
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(q, want_q) and torch.equal(s, want_s)
        del over


@pytest.mark.gpu
def test_stream_argument_of_the_other_helpers():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    X, W = rand(300, 256).to(torch.bfloat16), rand(2, 128, 256).to(torch.bfloat16)
    off = torch.from_numpy(np.array([0, 100, 300], dtype=np.int32)).cuda()
    Xr, Wr = rand(256, 256), rand(16, 256)
    want, logits = gg.grouped_gemm("fwd", X, W, off), gg.router_gemm(Xr, Wr)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        torch.cuda._sleep(20_000_000)
        got, other = gg.grouped_gemm("fwd", X, W, off, stream=stream), gg.router_gemm(Xr, Wr, stream=stream)
        torch.cuda.current_stream().wait_stream(side)
        assert torch.equal(got, want) and torch.equal(other, logits)
