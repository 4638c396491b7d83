"""What the quantised expert layer keeps between calls, and who may use it."""
import threading

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


class FakeStream:
    cuda_stream = 0x1000


@pytest.fixture
def host_layer(monkeypatch):
    """A layer on the CPU: its calls' buffers can be made there, its kernels cannot run."""
    import torch
    from moe_ragged_grouped_gb300 import experts
    gg_build.build()
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(experts.gg, "quantize_rows",
                        lambda w: (torch.zeros(w.shape, dtype=torch.int8), torch.zeros(w.shape[0])))
    z = torch.zeros
    return experts.Int8Experts(z(8, 64), z(8, 64, 64), z(8, 64, 32), 2)


def _tensors(kept):
    import torch
    if isinstance(kept, torch.Tensor):
        return [kept]
    return [t for part in kept for t in _tensors(part)] if isinstance(kept, tuple) else []


def test_threads_do_not_share_what_a_call_writes(host_layer):
    """Two threads' calls interleave on one stream: the first product of one may come between
    the two products of the other, and each call's token pass before the other's product."""
    import torch
    device, got = torch.device("cpu"), []
    got.append(_tensors(host_layer._for(40, device)))
    thread = threading.Thread(target=lambda: got.append(_tensors(host_layer._for(40, device))))
    thread.start()
    thread.join(60)
    mine, other = ({t.untyped_storage().data_ptr() for t in got[i]} for i in range(2))
    assert len(got[0]) == len(got[1]) >= 4 and not mine & other


def test_what_is_kept_does_not_grow_with_the_token_counts_seen(host_layer):
    """A server sees thousands of token counts: what the layer holds on to is bounded by the largest."""
    import torch
    from torch.multiprocessing.reductions import StorageWeakRef
    device, seen = torch.device("cpu"), {}
    for T in list(range(1, 60)) + [700] + list(range(60, 120)):
        for t in _tensors(host_layer._for(T, device)):
            storage = t.untyped_storage()
            seen[storage.data_ptr(), storage.nbytes()] = StorageWeakRef(storage)
            most = max(size for _, size in seen)
    kept = sum(size for (_, size), ref in seen.items() if not ref.expired())
    assert kept <= 4 * most, (kept, most)


def test_a_layer_is_freed_with_its_last_name(host_layer):
    """No cycle keeps its weights until a collection."""
    import gc
    import weakref

    import torch
    gc.disable()
    try:
        from moe_ragged_grouped_gb300.experts import Int8Experts
        z = torch.zeros
        layer = Int8Experts(z(8, 64), z(8, 64, 64), z(8, 64, 32), 2)
        layer._for(5, torch.device("cpu"))
        weights = weakref.ref(layer.up_q)
        del layer
        assert weights() is None
    finally:
        gc.enable()


def test_a_layer_can_be_copied_and_pickled(host_layer):
    """Its weights go along, what it keeps between calls does not."""
    import copy
    import pickle

    import torch
    device = torch.device("cpu")
    mine = {t.untyped_storage().data_ptr() for t in _tensors(host_layer._for(5, device))}
    for other in (copy.deepcopy(host_layer), pickle.loads(pickle.dumps(host_layer))):
        assert torch.equal(other.up_q, host_layer.up_q) and other.top_k == host_layer.top_k
        assert other.up_q.data_ptr() != host_layer.up_q.data_ptr()
        theirs = {t.untyped_storage().data_ptr() for t in _tensors(other._for(5, device))}
        assert theirs and not theirs & mine


def _gpu_layer(E=8, K=256, F=144, top=3):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    from moe_ragged_grouped_gb300.experts import Int8Experts
    g = torch.Generator(device="cuda").manual_seed(0)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    return Int8Experts(rand(E, K) / K ** 0.5, rand(E, 2 * F, K) / K ** 0.5, rand(E, K, F) / F ** 0.5, top), rand


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 40, 333])
def test_two_threads_on_one_stream(T, monkeypatch):
    """Calls of two threads, made to alternate after every product, give what each gives alone."""
    import torch
    layer, rand = _gpu_layer()
    xs = [rand(T, 256).to(torch.bfloat16) for _ in range(2)]
    want = [layer(x).clone() for x in xs]
    torch.cuda.synchronize()
    product, turn, got, failed = gg.int8_gemm, threading.Barrier(2), [None, None], []

    def after_both(*args, **more):
        out = product(*args, **more)
        turn.wait(60)
        return out

    monkeypatch.setattr(gg, "int8_gemm", after_both)

    def call(i):
        try:
            got[i] = [layer(xs[i]).clone() for _ in range(3)]
        except Exception as e:   # noqa: BLE001 (shown by the assertion)
            failed.append(e)
            turn.abort()

    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    assert not failed
    torch.cuda.synchronize()
    for outs, w in zip(got, want):
        assert all(torch.equal(o, w) for o in outs)


@pytest.mark.gpu
def test_memory_over_many_token_counts():
    """Device memory after calls of many token counts is what the largest of them needed, or less."""
    import torch
    layer, rand = _gpu_layer()
    x = rand(900, 256).to(torch.bfloat16)
    layer(x)
    torch.cuda.synchronize()
    base = torch.cuda.memory_allocated()
    for T in list(range(1, 200)) + list(range(850, 900, 3)):
        layer(x[:T])
    torch.cuda.synchronize()
    assert torch.cuda.memory_allocated() <= base + (1 << 16)


@pytest.mark.gpu
def test_a_status_is_not_lost_with_a_larger_workspace():
    """An error that an unchecked call recorded is reported by the next checked one on the stream,
    also when that one needs a larger workspace."""
    import torch
    layer, rand = _gpu_layer()
    x = rand(400, 256).to(torch.bfloat16)
    layer(x[:3])
    _, (_, work, _), _ = layer._for(3, x.device)
    work[:4].view(torch.int32).fill_(gg.CAKE_GG_ERR_TIMEOUT)
    with pytest.raises(gg.CakeGGError) as err:
        layer(x, check=True)
    assert err.value.code == gg.CAKE_GG_ERR_TIMEOUT
    layer(x, check=True)


@pytest.mark.gpu
def test_a_captured_call_keeps_its_buffers():
    """A graph's buffers stay its own when the layer's grow, or serve other calls, between replays."""
    import torch
    layer, rand = _gpu_layer()
    xs = [rand(T, 256).to(torch.bfloat16) for T in (20, 900)]
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        want = [layer(x).clone() for x in xs[::-1]][::-1]
    stream.synchronize()
    with torch.cuda.stream(stream):
        layer(xs[0])                                     # (warm, as a program does before it captures)
        graph = torch.cuda.CUDAGraph()
        stream.synchronize()
        with torch.cuda.graph(graph, stream=stream):
            out = layer(xs[0])
        for _ in range(3):
            assert torch.equal(layer(xs[1]), want[1])
            stream.synchronize()
            over = [torch.full((1 << 22,), 255, dtype=torch.uint8, device="cuda") for _ in range(8)]
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, want[0])
            del over
