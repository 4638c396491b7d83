"""Gradients of routing and rows where a program asks for less than all of them, or hands over tensors that are not its own."""
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def cuda():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()


def _rand(*shape, seed=0):
    import torch
    return torch.randn(shape, generator=torch.Generator(device="cuda").manual_seed(seed), device="cuda")


@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_sums_without_weights(dtype, out_dtype):
    """Each row's gradient is its token's, in the rows' type: one rounding."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    T, top, K = 21, 3, 72
    kind = {"bf16": torch.bfloat16, "fp32": torch.float32}
    position = gg.route(_rand(T, 9), top).position
    rows = _rand(T * top, K, seed=1).to(kind[dtype]).requires_grad_()
    y = ag.combine_rows(rows, None, position, out_dtype=out_dtype)
    v = rows.detach().double()[position.long()]
    step = 2.0 ** -8 if out_dtype == "bf16" else 0.0
    assert bool(((y.double() - v.sum(dim=1)).abs() <= step * v.sum(dim=1).abs() + top * 2.0 ** -24 * v.abs().sum(dim=1)).all())
    G = _rand(T, K, seed=2).to(kind[out_dtype])
    y.backward(G)
    assert rows.grad.dtype == kind[dtype]
    assert torch.equal(rows.grad[position.long()], G.to(kind[dtype])[:, None, :].expand(-1, top, -1))


class _Watched:
    """The library, with the arguments of its gradient calls kept."""

    def __init__(self, lib, calls):
        self._lib, self._calls = lib, calls

    def __getattr__(self, name):
        f = getattr(self._lib, name)
        if name != "cake_gg_combine_grad":
            return f

        def call(*args):
            self._calls.append(args)
            return f(*args)
        return call


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_weights_that_are_frozen(dtype, monkeypatch):
    """Without a gradient of the weights no row is read, and none is kept for the backward pass."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    T, top, K = 21, 3, 72
    kind = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    r = gg.route(_rand(T, 9), top)
    rows = _rand(T * top, K, seed=1).to(kind).requires_grad_()
    G = _rand(T, K, seed=2)
    calls = []
    monkeypatch.setattr(gg, "_lib", _Watched(gg.load_library(), calls))
    ag.combine_rows(rows, r.weight, r.position, out_dtype="fp32").backward(G)
    (args,) = calls
    assert args[6] is None and args[11] is None                  # (rows, d_weight)
    want = (r.weight[:, :, None] * G[:, None, :]).to(kind)
    assert torch.equal(rows.grad[r.position.long()], want)
    # and with one as before
    rows.grad, weight = None, r.weight.clone().requires_grad_()
    ag.combine_rows(rows, weight, r.position, out_dtype="fp32").backward(G)
    assert torch.equal(rows.grad[r.position.long()], want)
    dots = G.double()[:, None, :] * rows.detach().double()[r.position.long()]
    assert bool(((weight.grad.double() - dots.sum(dim=2)).abs() <= K * 2.0 ** -24 * dots.abs().sum(dim=2)).all())


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
def test_gradients_at_odd_places(dtype):
    """A dense gradient that begins anywhere, as part of a flat buffer does."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    T, top, K, E = 8, 2, 64, 4
    kind = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    r = gg.route(_rand(T, E), top)

    def odd(f, *leaves):
        """Gradients through y = f(leaves), whose own begins at the second value of a buffer, and those of an aligned one."""
        both = []
        for front in (1, 16):
            xs = [t.detach().clone().requires_grad_() for t in leaves]
            y = f(*xs)
            buffer = _rand(front + y.numel(), seed=5)
            buffer[front:] = _rand(y.numel(), seed=6)
            flat = torch.cat([torch.zeros(front, dtype=y.dtype, device="cuda"), y.flatten()])
            flat.backward(buffer.to(y.dtype))
            both.append([t.grad for t in xs])
        return both

    rows, x = _rand(T * top, K, seed=1).to(kind), _rand(T, K, seed=2).to(kind)
    cases = [(lambda a: ag.gather_rows(a, r.position), x), (lambda a, w: ag.combine_rows(a, w, r.position, out_dtype=dtype), rows, r.weight),
             (lambda a: ag.combine_rows(a, r.weight, r.position, out_dtype=dtype), rows), (lambda a: ag.combine_rows(a, None, r.position, out_dtype=dtype), rows)]
    if dtype == "bf16":
        cases.append((lambda a, w: ag.grouped_linear(a, w, r.offsets), rows, _rand(E, 128, K, seed=3).to(kind)))
    for case in cases:
        a, b = odd(*case)
        assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_options_are_the_forward_calls():
    """An option given as a tensor that changes afterwards: the gradient is that of the forward call."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    G = _rand(20, 3, seed=4)

    def grad(change):
        logits = _rand(20, 8, seed=1).requires_grad_()
        scale, renormalize = torch.tensor(2.0), torch.tensor(True)
        w = ag.route(logits, 3, scale=scale, renormalize=renormalize).weight
        if change:
            scale.fill_(5.0)
            renormalize.fill_(False)
        w.backward(G)
        return logits.grad

    assert torch.equal(grad(True), grad(False))


@pytest.mark.parametrize("weights", ["trained", "frozen", "none"])
@pytest.mark.parametrize("T,top,K,dtype", [(5, 3, 8, "fp32"), (300, 2, 264, "bf16"), (40, 8, 4096, "fp32"), (70001, 2, 8, "bf16")])
def test_rows_that_no_token_takes(T, top, K, dtype, weights):
    """Positions outside the rows take none: the rows that are left have no part in the sums, so their gradient is zero."""
    import torch
    from moe_ragged_grouped_gb300 import autograd as ag
    kind = {"bf16": torch.bfloat16, "fp32": torch.float32}[dtype]
    M = T * top
    g = torch.Generator(device="cuda").manual_seed(M)
    position = torch.randperm(M, generator=g, device="cuda").view(T, top).to(torch.int32)
    out = torch.rand((T, top), generator=g, device="cuda") < 0.3
    out[0] = True
    position[out] = torch.where(torch.rand((T, top), generator=g, device="cuda") < 0.5, -1, M).to(torch.int32)[out]
    rows = _rand(M, K, seed=1).to(kind).requires_grad_()
    w = _rand(T, top, seed=2).requires_grad_(weights == "trained")
    G = _rand(T, K, seed=3)
    # (what the allocator gives again is not zeros)
    for _ in range(3):
        torch.full((M, K), float("nan"), dtype=kind, device="cuda")
    ag.combine_rows(rows, None if weights == "none" else w, position, out_dtype="fp32").backward(G)
    want = torch.zeros_like(rows)
    share = G[:, None, :] * (1.0 if weights == "none" else w.detach()[:, :, None])
    want[position[~out].long()] = share.expand(-1, top, -1)[~out].to(kind)
    assert torch.equal(rows.grad, want)
    if weights == "trained":
        assert not w.grad[out].any()


def test_zeros_in_the_rows_left_alone():
    """The named rows and the memory around stay as they were."""
    import torch
    from gg_testutil import guarded_empty, guards_intact
    for M, K, kind in ((1, 8, "bf16"), (33, 24, "fp32"), (1000, 520, "bf16")):
        position = torch.full((M, 1), -1, dtype=torch.int32, device="cuda")
        position[::3, 0] = torch.arange(M - 1, -1, -1, dtype=torch.int32, device="cuda")[::3]
        position[1::3, 0] = 2 ** 31 - 1
        buf, view, guard = guarded_empty((M, K), kind)
        bits = torch.int16 if kind == "bf16" else torch.int32
        before = view.clone().view(bits)
        work = torch.full((M,), 7, dtype=torch.uint8, device="cuda")
        assert gg.cake_gg_zero_unnamed_rows(M, M, 1, K, position, view, kind, work) == gg.CAKE_GG_OK
        named = torch.zeros(M, dtype=torch.bool, device="cuda")
        named[position[::3, 0].long()] = True
        assert guards_intact(buf, guard, M * K, kind) and not view[~named].any()
        assert torch.equal(view.view(bits)[named], before[named])


def test_zeros_on_another_stream():
    """The marks and the zeros go where the gradient goes."""
    import torch
    T, top, K = 3000, 2, 1024
    position = torch.randperm(T * top, generator=torch.Generator(device="cuda").manual_seed(1), device="cuda").view(T, top).to(torch.int32)
    position[::5] = -1
    G, rows, w = _rand(T, K, seed=1), _rand(T * top, K, seed=2), _rand(T, top, seed=3)
    want = gg.combine_grad(G, rows, position, w, zero_rest=True)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for st in (stream, stream.cuda_stream):
        got = gg.combine_grad(G, rows, position, w, stream=st, zero_rest=True)
        alone = gg.gather_rows(G, position, weight=w, stream=st, zero_rest=True)
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got, want)) and torch.equal(alone, want[0])
