"""Routing, gathering and combining rows in training: their gradients, alone and around the grouped products."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg


def test_refusals_on_the_host():
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    gg_build.build()
    e, w = torch.zeros((4, 2), dtype=torch.int32), torch.zeros(4, 2)
    with pytest.raises(ValueError):
        ag.combine_rows(torch.zeros(7, 16), w, e)
    for call in (lambda: ag.combine_rows(torch.zeros(8, 16), w, e), lambda: ag.gather_rows(torch.zeros(4, 16), e),
                 lambda: ag.route(torch.zeros(4, 8), 2)):
        with pytest.raises(ValueError, match="CUDA"):
            call()


@pytest.fixture(scope="module")
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    return torch.device("cuda")


def _rand(*shape, seed=0):
    import torch
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


def layer_step(x, router, up, down, top, R, options):
    """One expert layer's forward and backward by the framework; gradients of x, router, up, down."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    leaves = [t.detach().clone().requires_grad_() for t in (x, router, up, down)]
    x, router, up, down = leaves
    r = ag.route(x.float() @ router.T, top, **options)
    X = ag.gather_rows(x, r.position)
    h = ag.grouped_linear(X, up, r.offsets)
    gate, lin = h.chunk(2, dim=1)
    Y = ag.grouped_linear((torch.nn.functional.silu(gate) * lin).contiguous(), down, r.offsets)
    y = ag.combine_rows(Y, r.weight, r.position, out_dtype="fp32")
    (y * R).sum().backward()
    return y.detach(), [t.grad for t in leaves], r


def layer_reference(x, router, up, down, top, R, options, expert):
    """The same in 64 bits by torch, with the experts as chosen."""
    import torch
    leaves = [t.detach().double().requires_grad_() for t in (x, router, up, down)]
    x, router, up, down = leaves
    logits = x @ router.T
    s = torch.sigmoid(logits) if options["score"] == "sigmoid" else torch.softmax(logits, dim=1)
    w = s.gather(1, expert.long())
    if options["renormalize"]:
        w = w / w.sum(dim=1, keepdim=True)
    y = torch.zeros_like(x)
    for e in range(up.shape[0]):
        t, j = (expert == e).nonzero(as_tuple=True)
        gate, lin = (x[t] @ up[e].T).chunk(2, dim=1)
        y = y.index_add(0, t, w[t, j, None] * ((torch.nn.functional.silu(gate) * lin) @ down[e].T))
    (y * R.double()).sum().backward()
    return y.detach(), [t.grad for t in leaves]


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 33, 400])
@pytest.mark.parametrize("options", [dict(score="softmax", renormalize=True), dict(score="softmax", renormalize=False),
                                     dict(score="sigmoid", renormalize=True)])
def test_a_run_of_them(cuda, T, options):
    """A whole expert layer in training.

    Between the stages values are rounded to BF16 five times on the way forward (x's
    products, the gate, the second product) and six back, each by 2^-8 at most of
    itself; relative to the gradients' norms, where roundings do not all point one
    way, that is within 12 * 2^-8.
    """
    import torch
    E, K, F, top = 6, 128, 64, 2
    x, router = _rand(T, K, seed=1).to(torch.bfloat16), _rand(E, K, seed=2) / K ** 0.5
    up, down = (_rand(E, 2 * F, K, seed=3) / K ** 0.5).to(torch.bfloat16), (_rand(E, K, F, seed=4) / F ** 0.5).to(torch.bfloat16)
    R = _rand(T, K, seed=5)
    y, grads, r = layer_step(x, router, up, down, top, R, options)
    want, want_grads = layer_reference(x, router, up, down, top, R, options, r.expert)
    for a, b in zip([y] + grads, [want] + want_grads):
        assert float((a.double() - b).norm()) <= 12 * 2.0 ** -8 * float(b.norm())
    again = layer_step(x, router, up, down, top, R, options)
    assert torch.equal(again[0], y) and all(torch.equal(a, b) for a, b in zip(again[1], grads))


@pytest.mark.gpu
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_each_against_autograd_in_64_bits(cuda, dtype):
    """Tolerances as in the kernels' own tests: d_rows one product, rounded; d_weight K 2^-24; sums of rows top_k 2^-24."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    T, top, K, E = 37, 3, 264, 9
    kind = torch.bfloat16 if dtype == "bf16" else torch.float32
    step = 2.0 ** -8 if dtype == "bf16" else 2.0 ** -23
    position = gg.route(_rand(T, E), top).position
    rows, w = _rand(T * top, K, seed=1).to(kind).requires_grad_(), _rand(T, top, seed=2).requires_grad_()
    y = ag.combine_rows(rows, w, position, out_dtype=dtype)
    G = _rand(T, K, seed=3).to(kind)
    y.backward(G)
    r64, w64 = rows.detach().double().requires_grad_(), w.detach().double().requires_grad_()
    ((r64[position.long()] * w64[:, :, None]).sum(dim=1)).backward(G.double())
    assert bool(((rows.grad.double() - r64.grad).abs() <= step * r64.grad.abs()).all())
    size = (G.double()[:, None, :] * r64.detach()[position.long()]).abs().sum(dim=2)
    assert bool(((w.grad.double() - w64.grad).abs() <= K * 2.0 ** -24 * size).all())
    x = _rand(T, K, seed=4).to(kind).requires_grad_()
    H = _rand(T * top, K, seed=5).to(kind)
    X = ag.gather_rows(x, position)
    assert bool((X[position.long()] == x.detach()[:, None, :]).all())
    X.backward(H)
    v = H.double()[position.long()]
    assert bool(((x.grad.double() - v.sum(dim=1)).abs() <= step * v.sum(dim=1).abs() + top * 2.0 ** -24 * v.abs().sum(dim=1)).all())


@pytest.mark.gpu
def test_gradients_that_are_not_dense_or_not_wanted(cuda):
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    r = ag.route(_rand(20, 8).requires_grad_(), 2)
    assert r.weight.requires_grad and not any(t.requires_grad for t in (r.expert, r.offsets, r.rows, r.position))
    rows = _rand(40, 64, seed=1).requires_grad_()
    y = ag.combine_rows(rows, r.weight.detach(), r.position, out_dtype="fp32")
    y.sum().backward()                                           # (a gradient expanded from one number)
    want = torch.zeros(40, device="cuda")
    want[r.position.long().flatten()] = r.weight.detach().flatten()
    assert bool((rows.grad == want[:, None]).all())
    logits = _rand(20, 8, seed=2).requires_grad_()
    r = ag.route(logits, 2, score="sigmoid", renormalize=False)
    r.weight[:, 0].sum().backward()                              # (zeros for the others, strided)
    s = torch.sigmoid(logits.detach().double())
    first = torch.zeros_like(s).scatter_(1, r.expert[:, :1].long(), 1.0)
    assert bool(((logits.grad.double() - first * s * (1 - s)).abs() <= 2.0 ** -16).all())
    with pytest.raises(RuntimeError):                            # there is no second derivative
        x = _rand(20, 8, seed=3).requires_grad_()
        (g,) = torch.autograd.grad(ag.route(x, 2).weight.square().sum(), x, create_graph=True)
        g.sum().backward()


@pytest.mark.gpu
def test_a_captured_step(cuda):
    """Forward and backward in a CUDA graph, replayed on new tokens."""
    import torch
    T, E, K, F, top = 48, 6, 128, 64, 2
    options = dict(score="softmax", renormalize=True)
    router = _rand(E, K, seed=2) / K ** 0.5
    up, down = (_rand(E, 2 * F, K, seed=3) / K ** 0.5).to(torch.bfloat16), (_rand(E, K, F, seed=4) / F ** 0.5).to(torch.bfloat16)
    R = _rand(T, K, seed=5)
    xs = [_rand(T, K, seed=10 + i).to(torch.bfloat16) for i in range(3)]
    want = [layer_step(x, router, up, down, top, R, options)[:2] for x in xs]
    x = xs[0].clone()
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        for _ in range(2):
            layer_step(x, router, up, down, top, R, options)
        stream.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            y, grads, _ = layer_step(x, router, up, down, top, R, options)
        for i in (1, 2, 0):
            x.copy_(xs[i])
            graph.replay()
            stream.synchronize()
            assert torch.equal(y, want[i][0]) and all(torch.equal(a, b) for a, b in zip(grads, want[i][1]))
