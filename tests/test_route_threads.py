"""Routing called by several threads at once: what a launch needs is a call's own or set once and for all."""
import threading

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


@pytest.mark.gpu
@pytest.mark.parametrize("E,sizes", [(1024, (40000, 65536)), (512, (100000, 150000))])
def test_two_threads_route_other_sizes(E, sizes):
    """Sizes whose blocks take more than 48 KB of shared memory, of one kernel, on a stream of each thread's own."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    g = torch.Generator(device="cuda").manual_seed(E)
    cases = [torch.randn((T, E), generator=g, device="cuda") for T in sizes]
    want = [gg.route(logits, 8) for logits in cases]
    torch.cuda.synchronize()
    start, failed = threading.Barrier(len(cases)), []

    def work(logits, want):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                plan = gg.cake_gg_route_plan(logits.shape[0], E, 8)
                space, out = gg.make_workspace(plan, "cuda"), gg.empty_routing(logits.shape[0], E, 8, "cuda")
                stream.synchronize()
                start.wait(60)
                for _ in range(1500):
                    gg.route(logits, 8, plan=plan, workspace=space, out=out)
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(out, want))
        except Exception as e:                                   # (a thread's own would be lost)
            failed.append(e)

    threads = [threading.Thread(target=work, args=a) for a in zip(cases, want)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed


@pytest.mark.gpu
@pytest.mark.parametrize("kind", ["mx4", "i8"])
def test_threads_multiply_at_once(kind):
    """Products of sizes that take every kernel, each thread's on a stream of its own: as by one thread."""
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    g = torch.Generator(device="cuda").manual_seed(3)
    N, K = 520, 1024
    w = torch.randn((N, K), generator=g, device="cuda")
    q, s = gg.quantize_mx4(w) if kind == "mx4" else gg.quantize_rows(w)
    multiply = gg.mx4_gemm if kind == "mx4" else gg.int8_gemm
    xs = [torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16) for T in (1, 2, 40, 700, 3000)]
    torch.cuda.synchronize()
    got, failed = [None] * len(xs), []
    start = threading.Barrier(len(xs))

    def work(i):
        try:
            stream = torch.cuda.Stream()
            with torch.cuda.stream(stream):
                start.wait(60)
                got[i] = [multiply(xs[i], q, s, out_dtype=kind, check=False) for kind in ("bf16", "fp32") * 20][-2:]
                stream.synchronize()
        except Exception as e:
            failed.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(xs))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert not failed, failed
    for x, (a, b) in zip(xs, got):
        assert torch.equal(a, multiply(x, q, s)) and torch.equal(b, multiply(x, q, s, out_dtype="fp32"))
