"""The 4-bit expert layer: router, routing, routed product, gated product, rows' way back."""
import threading

import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


def test_layer_refuses():
    import torch
    from moe_ragged_grouped_gb300.experts import Mx4Experts
    z = torch.zeros
    good = z(4, 64), z(4, 64, 64), z(4, 64, 32)
    for router, up, down, top, more in [
        (*good, 5, {}), (*good, 0, {}), (z(3, 64), *good[1:], 2, {}), (z(4, 48), z(4, 64, 48), z(4, 48, 32), 2, {}),
        (z(4, 64), z(4, 32, 64), z(4, 64, 16), 2, {}), (*good, 2, dict(bias=z(3))), (*good, 2, dict(bias=z(4).double())),
    ]:
        with pytest.raises(ValueError):
            Mx4Experts(router, up, down, top, **more)


@pytest.fixture
def host_layer(monkeypatch):
    """A layer on the CPU: its calls' buffers can be made there, its kernels cannot run."""
    import torch
    from moe_ragged_grouped_gb300 import experts
    gg_build.build()

    class FakeStream:
        cuda_stream = 0x1000
    monkeypatch.setattr(torch.cuda, "current_stream", lambda device=None: FakeStream)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    u8 = torch.uint8
    monkeypatch.setattr(experts.gg, "quantize_mx4", lambda w: (torch.zeros((*w.shape[:2], w.shape[2] // 2), dtype=u8),
                                                               torch.zeros((w.shape[0], 1, 1, 32, 4, 4), dtype=u8)))
    z = torch.zeros
    return experts.Mx4Experts(z(8, 64), z(8, 64, 64), z(8, 64, 32), 2, bias=z(8))


def _tensors(kept):
    import torch
    if isinstance(kept, torch.Tensor):
        return [kept]
    return [t for part in kept for t in _tensors(part)] if isinstance(kept, (tuple, list)) else []


def test_buffers_are_a_threads_own_and_do_not_grow(host_layer):
    import torch
    device, got = torch.device("cpu"), []
    got.append(_tensors(host_layer._for(40, device)))
    thread = threading.Thread(target=lambda: got.append(_tensors(host_layer._for(40, device))))
    thread.start()
    thread.join(60)
    mine, other = ({t.untyped_storage().data_ptr() for t in got[i]} for i in range(2))
    assert len(got[0]) == len(got[1]) >= 8 and not mine & other
    from torch.multiprocessing.reductions import StorageWeakRef
    seen, most = {}, 0
    for T in list(range(1, 60)) + [700] + list(range(60, 120)):
        tensors = _tensors(host_layer._for(T, device))
        most = max(most, sum({t.untyped_storage().data_ptr(): t.untyped_storage().nbytes() for t in tensors}.values()))
        for t in tensors:
            seen[t.untyped_storage().data_ptr(), t.untyped_storage().nbytes()] = StorageWeakRef(t.untyped_storage())
    del tensors, t
    assert sum(size for (_, size), ref in seen.items() if not ref.expired()) <= 2 * most


def test_a_layer_can_be_copied_pickled_and_freed(host_layer):
    import copy
    import gc
    import pickle
    import weakref

    import torch
    host_layer._for(5, torch.device("cpu"))
    for other in (copy.deepcopy(host_layer), pickle.loads(pickle.dumps(host_layer))):
        assert torch.equal(other.up_q, host_layer.up_q) and other.options == host_layer.options and other.bias is not None
        other._for(5, torch.device("cpu"))
    gc.disable()
    try:
        weights = weakref.ref(other.up_q)
        del other
        assert weights() is None
    finally:
        gc.enable()


def _gpu_layer(E=8, K=256, F=160, top=3, seed=0, **options):
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    from moe_ragged_grouped_gb300.experts import Mx4Experts
    g = torch.Generator(device="cuda").manual_seed(seed)
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    if options.pop("biased", False):
        options["bias"] = rand(E) * 0.1
    return Mx4Experts(rand(E, K) / K ** 0.5, rand(E, 2 * F, K) / K ** 0.5, rand(E, K, F) / F ** 0.5, top, **options), rand


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 3, 40, 333])
@pytest.mark.parametrize("E,options", [
    (8, {}), (13, dict(score="sigmoid", biased=True, scale=2.5)),
    (16, dict(score="sigmoid", biased=True, groups=4, top_groups=2, group_score="top2")),
])
def test_layer_against_64_bits(T, E, options):
    """The layer's own quantised tensors multiplied in 64 bits.

    Each stage is bounded by itself: the choice and the weights by the routing's
    own test, h within 2^-8 (its rounding to BF16) and 2^-18 of the sum of its
    terms' magnitudes (the tensor cores' FP32 sums of at most 8 steps), y within
    2^-18 of the terms' magnitudes after it, and one BF16 rounding.
    """
    import torch
    K, F, top = 256, 160, 3
    layer, rand = _gpu_layer(E, K, F, top, seed=T, **options)
    x = rand(T, K).to(torch.bfloat16)
    y = layer(x, check=True)
    assert torch.equal(y, layer(x))                       # kept plans and workspaces
    expert, weight = layer.route(x)
    logits = gg.router_gemm(x.float(), layer.router)[:, :E]
    again = gg.route(logits, top, bias=layer.bias, **layer.options)
    assert torch.equal(expert, again.expert) and torch.equal(weight, again.weight)
    _, (_, _, h), _, _ = layer._for(T, x.device)
    order = torch.argsort(expert.reshape(-1).long(), stable=True)
    e_of, t_of = expert.reshape(-1)[order].long(), order // top
    tokens, up, down = (gg.mx4_values(q, s).double() for q, s in (gg.quantize_mx4(x), (layer.up_q, layer.up_s), (layer.down_q, layer.down_s)))
    product = lambda a, w: torch.einsum("mk,mnk->mn", a, w[e_of])  # noqa: E731
    want_h, size_h = product(tokens[t_of], up), product(tokens[t_of].abs(), up.abs())
    assert ((h.double() - want_h).abs() <= 2.0 ** -8 * want_h.abs() + 2.0 ** -18 * size_h).all()
    gated = gg.mx4_values(*gg.quantize_mx4(h, act="silu_mul")).double()
    w_of = weight.reshape(-1)[order, None].double()
    rows, sizes = product(gated, down) * w_of, product(gated.abs(), down.abs()) * w_of
    want, size = (torch.zeros(T, K, dtype=torch.float64, device="cuda").index_add_(0, t_of, v) for v in (rows, sizes))
    assert ((y.double() - want).abs() <= 2.0 ** -8 * want.abs() + 2.0 ** -18 * size).all()


@pytest.mark.gpu
def test_layer_without_tokens_and_on_other_streams():
    import torch
    layer, rand = _gpu_layer()
    none = torch.empty((0, 256), dtype=torch.bfloat16, device="cuda")
    assert layer(none).shape == (0, 256) and layer.route(none)[0].shape == (0, 3)
    x = rand(50, 256).to(torch.bfloat16)
    want = layer(x).clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        got = [layer(x) for _ in range(3)]
    stream.synchronize()
    assert all(torch.equal(g, want) for g in got)


@pytest.mark.gpu
def test_a_captured_call_replays_with_new_tokens():
    """Also when the layer's buffers serve other calls between replays."""
    import torch
    layer, rand = _gpu_layer()
    xs = [rand(20, 256).to(torch.bfloat16) for _ in range(3)]
    want = [layer(x).clone() for x in xs]
    other = rand(900, 256).to(torch.bfloat16)
    want_other = layer(other).clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        x = xs[0].clone()
        layer(x)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = layer(x)
        for i in (1, 2, 0):
            assert torch.equal(layer(other), want_other)
            x.copy_(xs[i])
            graph.replay()
            stream.synchronize()
            assert torch.equal(out, want[i])


@pytest.mark.gpu
def test_two_threads():
    import torch
    layer, rand = _gpu_layer()
    xs = [rand(T, 256).to(torch.bfloat16) for T in (40, 333)]
    want = [layer(x).clone() for x in xs]
    torch.cuda.synchronize()
    got, failed = [None, None], []

    def call(i):
        try:
            got[i] = [layer(xs[i]).clone() for _ in range(20)]
        except Exception as e:   # noqa: BLE001 (shown by the assertion)
            failed.append(e)
    threads = [threading.Thread(target=call, args=(i,)) for i in range(2)]
    for t in threads:
        t.start()
    for t in threads:
        t.join(120)
    torch.cuda.synchronize()
    assert not failed and all(torch.equal(o, w) for outs, w in zip(got, want) for o in outs)
