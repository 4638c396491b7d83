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
