"""Routing and the rows' way back on the GPU, against 64-bit definitions.

What is chosen, and how rows are numbered, has to be equal.  A weight is a few
FP32 operations on FP32 exponentials: the exponential is off by 2 units in the
last place and its argument by 2^-24 |l - max| of itself, a sum of up to 1024
terms by ten roundings more than its terms, a quotient and a product by 2^-24
each: with |l - max| <= 40 below 2^-17 of the value.  Gradients take differences
of such numbers: 2^-16 of the largest |g| w (of a sum of up to 32 terms of either
sign, 2^-16 of the sum of their magnitudes), and a rounding to BF16 adds 2^-8.
"""
import numpy as np
import pytest

from moe_ragged_grouped_gb300 import build as gg_build
from moe_ragged_grouped_gb300 import cake_gg as gg

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def lib():
    import torch
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    gg_build.build()
    return gg.load_library()


def same(a, b):
    return a.shape == b.shape and bool((a == b).all())


def probabilities(l, score):
    import torch
    l = l.double()
    return torch.sigmoid(l) if score == "sigmoid" else torch.softmax(l, dim=1)


def reference(logits, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max", renormalize=True, scale=1.0):
    """Experts, weights, offsets, rows, positions by numpy's stable sorts, in 64 bits."""
    T, E = logits.shape
    p = probabilities(logits, score).cpu().numpy()
    key = logits.double().cpu().numpy() if bias is None else p + bias.double().cpu().numpy()
    if groups > 1:
        by = key if bias is not None or group_score == "max" else p
        part = -np.sort(-by.reshape(T, groups, -1), axis=2)
        gs = part[:, :, 0] + part[:, :, 1] if group_score == "top2" else part[:, :, 0]
        best = np.argsort(-gs, axis=1, kind="stable")[:, :top_groups or groups]
        out = np.ones((T, groups), bool)
        np.put_along_axis(out, best, False, axis=1)
        key = np.where(np.repeat(out, E // groups, axis=1), -np.inf, key)
    expert = np.argsort(-key, axis=1, kind="stable")[:, :top_k]
    w = np.take_along_axis(p, expert, axis=1)
    if renormalize:
        w = w / w.sum(axis=1, keepdims=True)
    flat = expert.reshape(-1)
    order = np.argsort(flat, kind="stable")
    offsets = np.concatenate([[0], np.cumsum(np.bincount(flat, minlength=E))])
    position = np.empty_like(order)
    position[order] = np.arange(order.size)
    return expert, w * scale, offsets, order // top_k, position.reshape(T, top_k)


def check(got, want):
    expert, weight, offsets, rows, position = (t.cpu().numpy() for t in got)
    assert np.array_equal(expert, want[0])
    assert np.array_equal(offsets, want[2]) and np.array_equal(rows, want[3]) and np.array_equal(position, want[4])
    assert (np.abs(weight - want[1]) <= 2.0 ** -17 * np.abs(want[1])).all()


def make(T, E, seed, dtype="fp32", spread=2.0):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    l = torch.randn((T, E), generator=g, device="cuda") * spread
    bias = torch.randn(E, generator=g, device="cuda") * 0.1
    return l.to(torch.bfloat16 if dtype == "bf16" else torch.float32), bias


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,top_k", [
    (1, 1, 1), (1, 8, 2), (1, 32, 4), (2, 5, 5), (3, 33, 8), (31, 64, 6), (32, 32, 32), (33, 100, 3), (64, 256, 8), (65, 200, 31),
    (257, 12, 1), (300, 1024, 32), (1023, 40, 4), (1024, 512, 8), (1025, 256, 8), (1500, 7, 3), (2049, 1000, 9), (5000, 64, 6), (400001, 6, 2),
])
def test_route(T, E, top_k, score, dtype):
    logits, bias = make(T, E, T + E, dtype)
    for b, renormalize, scale in ((None, True, 1.0), (bias, False, 2.5)):
        o = dict(score=score, bias=b, renormalize=renormalize, scale=scale)
        check(gg.route(logits, top_k, **o), reference(logits, top_k, **o))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
@pytest.mark.parametrize("group_score", ["max", "top2"])
@pytest.mark.parametrize("T,E,top_k,groups,top_groups", [
    (1, 8, 2, 4, 1), (40, 256, 8, 8, 4), (33, 60, 5, 4, 3), (70, 64, 4, 32, 2), (50, 96, 6, 3, 3), (1100, 160, 6, 8, 3), (20, 1024, 8, 16, 2),
    (9, 14, 7, 2, 1),
])
def test_groups(T, E, top_k, groups, top_groups, group_score, with_bias, score):
    logits, bias = make(T, E, T * 3 + E)
    o = dict(score=score, bias=bias if with_bias else None, groups=groups, top_groups=top_groups, group_score=group_score)
    check(gg.route(logits, top_k, **o), reference(logits, top_k, **o))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_many_tokens(score):
    """Enough choices that some of them hang on the last places of FP32."""
    logits, bias = make(20000, 256, 1, spread=1.0)
    o = dict(score=score, bias=bias)
    check(gg.route(logits, 8, **o), reference(logits, 8, **o))
    o = dict(score=score, bias=bias, groups=8, top_groups=4, group_score="top2")
    check(gg.route(logits, 8, **o), reference(logits, 8, **o))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_ties(with_bias, score):
    """Equal keys go to the lowest index: all equal, equal in runs, and values one step apart."""
    import torch
    T, E = 70, 64
    logits = torch.zeros((T, E), device="cuda")
    logits[1] = torch.arange(E, device="cuda").div(7, rounding_mode="floor").float()
    logits[2] = -0.0
    logits[3, ::2] = -0.0
    near = torch.full((E,), 0.75, device="cuda")
    for i in range(4, 40):
        row = near.clone()
        row[i] = torch.nextafter(row[i], torch.tensor(2.0, device="cuda"))
        row[E - i] = torch.nextafter(row[E - i], torch.tensor(-2.0, device="cuda"))
        logits[i] = row
    bias = torch.full((E,), 0.25, device="cuda") if with_bias else None
    for top_k in (1, 8, 32):
        o = dict(score=score, bias=bias)
        check(gg.route(logits, top_k, **o), reference(logits, top_k, **o))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
def test_near_ties_with_bias(score):
    """score + bias within FP32's error of one another: biases make up for the scores' differences."""
    import torch
    E = 64
    g = torch.Generator(device="cuda").manual_seed(5)
    logits = torch.randn((1, E), generator=g, device="cuda").repeat(200, 1)
    p = probabilities(logits[:1], score)[0]
    bias = (0.9 - p).float()                                     # every key within a rounding of 0.9
    logits[1:] += torch.randn((199, E), generator=g, device="cuda") * 1e-6
    o = dict(score=score, bias=bias)
    check(gg.route(logits, 8, **o), reference(logits, 8, **o))
    o = dict(o, groups=8, top_groups=3, group_score="top2")
    check(gg.route(logits, 8, **o), reference(logits, 8, **o))
    o = dict(o, group_score="max")
    check(gg.route(logits, 8, **o), reference(logits, 8, **o))


def test_masked_experts():
    """Minus infinity and the type's lowest value as masks; rows with nothing left; NaNs last."""
    import torch
    ninf, low = float("-inf"), torch.finfo(torch.float32).min
    logits, _ = make(6, 16, 3)
    logits[0, 4:] = ninf
    logits[1, :] = ninf
    logits[2, 2:] = low
    logits[3, :] = low
    logits[4, 5] = float("nan")
    logits[5, :] = float("nan")
    got = gg.route(logits, 4)
    e, w = got.expert.cpu(), got.weight.cpu()
    assert sorted(e[0].tolist()) == [0, 1, 2, 3] and e[1].tolist() == [0, 1, 2, 3] and e[5].tolist() == [0, 1, 2, 3]
    assert sorted(e[2].tolist()) == [0, 1, 2, 3] and set(e[2, :2].tolist()) == {0, 1} and 5 not in e[4].tolist()
    assert bool((w[1] == 0).all()) and bool((w[3] == 0.25).all()) and bool((w[2, 2:] == 0).all())
    assert abs(float(w[0].sum()) - 1) < 1e-6 and bool(torch.isfinite(w[:5]).all()) and bool(torch.isnan(w[5]).all())
    for options in (dict(score="sigmoid"), dict(score="sigmoid", renormalize=False), dict(renormalize=False, score="softmax")):
        got = gg.route(logits, 4, **options)
        assert same(got.expert.cpu(), e)
        assert int(got.offsets[-1]) == 24 and same(got.position.flatten().sort().values.cpu(), torch.arange(24, dtype=torch.int32))
    w = gg.route(logits, 4, score="sigmoid").weight.cpu()
    assert bool((w[1] == 0).all()) and bool(torch.isfinite(w[:5]).all())
    # sigmoids that vanish in FP32 keep their ratios
    far = torch.full((1, 8), -200.0, device="cuda")
    far[0, 3] = -199.0
    w = gg.route(far, 2, score="sigmoid").weight.cpu()[0].double()
    assert abs(float(w[0] / w[1]) - np.e) < 1e-5
    # a bias that takes an expert out
    bias = torch.zeros(16, device="cuda")
    bias[7] = ninf
    plain, _ = make(50, 16, 8)
    o = dict(score="sigmoid", bias=bias)
    check(gg.route(plain, 5, **o), reference(plain, 5, **o))


def test_rows_apart_and_reuse():
    """Logits in a slice of columns; outputs and workspace used again; no tokens."""
    import torch
    for T in (5, 3000):
        wide, bias = make(T, 48, T)
        logits = wide[:, :40]
        plan = gg.cake_gg_route_plan(T, 40, 6)
        work, out = gg.make_workspace(plan, "cuda"), gg.empty_routing(T, 40, 6, "cuda")
        for _ in range(3):
            got = gg.route(logits, 6, plan=plan, workspace=work, out=out)
            assert all(a is b for a, b in zip(got, out))
            check(got, reference(logits.contiguous(), 6))
    got = gg.route(torch.empty((0, 16), device="cuda"), 4)
    assert got.expert.shape == (0, 4) and not got.offsets.any() and got.offsets.shape == (17,)


# ---------------------------------------------------------------- backward


def autograd_reference(logits, expert, d_weight, score, renormalize, scale):
    import torch
    l = logits.double().requires_grad_()
    w = probabilities(l, score).gather(1, expert.long())
    if renormalize:
        w = w / w.sum(dim=1, keepdim=True)
    (w * scale * d_weight.double()).sum().backward()
    return l.grad, (w * scale * d_weight.double()).abs().sum(dim=1, keepdim=True).detach()


@pytest.mark.parametrize("dtype", ["fp32", "bf16"])
@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
@pytest.mark.parametrize("T,E,top_k", [(1, 1, 1), (1, 32, 4), (3, 33, 8), (50, 100, 7), (65, 200, 31), (300, 1024, 32), (2049, 256, 8), (9, 500, 2)])
def test_route_grad(T, E, top_k, renormalize, score, dtype):
    import torch
    logits, _ = make(T, E, T + E + 1, dtype)
    expert = gg.route(logits, top_k, score=score).expert
    g = torch.randn((T, top_k), generator=torch.Generator(device="cuda").manual_seed(T), device="cuda")
    got = gg.route_grad(logits, expert, g, score=score, renormalize=renormalize, scale=1.5)
    want, size = autograd_reference(logits, expert, g, score, renormalize, 1.5)
    assert got.dtype == logits.dtype
    tol = 2.0 ** -16 * size + (2.0 ** -8 * want.abs() if dtype == "bf16" else 0)
    assert bool(((got.double() - want).abs() <= tol).all())
    if renormalize and top_k == 1:
        assert not got.any()                                     # a constant


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("renormalize", [False, True])
def test_route_grad_against_differences(renormalize, score):
    """The gradient as the slope of route()'s own weights."""
    import torch
    logits, _ = make(4, 16, 7)
    o = dict(score=score, renormalize=renormalize)
    first = gg.route(logits, 3, **o)
    g = torch.randn((4, 3), generator=torch.Generator(device="cuda").manual_seed(1), device="cuda")
    got = gg.route_grad(logits, first.expert, g, **o).double()
    h = 2.0 ** -7
    for e in range(16):
        total = []
        for sign in (1, -1):
            moved = logits.clone()
            moved[:, e] += sign * h
            r = gg.route(moved, 16, **dict(o, renormalize=False))
            at = torch.argsort(r.expert, dim=1)
            w = r.weight.double().gather(1, at).gather(1, first.expert.long())
            total.append(((w / w.sum(dim=1, keepdim=True) if renormalize else w) * g.double()).sum(dim=1))
        slope = (total[0] - total[1]) / (2 * h)
        # differences: h^2 / 6 of a third derivative (at most one here, times |g|), and
        # FP32's error of a weight over 2 h
        tol = (h * h / 6 + 2.0 ** -17 / h) * g.double().abs().sum(dim=1)
        assert bool(((slope - got[:, e]).abs() <= tol).all())


def test_route_grad_nobody():
    """Experts outside [0, E) take no part."""
    import torch
    logits, _ = make(2, 8, 1)
    expert = torch.tensor([[1, -1], [2 ** 31 - 1, 8]], dtype=torch.int32, device="cuda")
    got = gg.route_grad(logits, expert, torch.ones((2, 2), device="cuda"), score="sigmoid", renormalize=False)
    s = torch.sigmoid(logits[0, 1].double())
    assert abs(float(got[0, 1]) - float(s * (1 - s))) < 1e-6 and int((got != 0).sum()) == 1


# ---------------------------------------------------------------- rows


def rows_case(T, top_k, K, rows_dtype, seed):
    import torch
    g = torch.Generator(device="cuda").manual_seed(seed)
    position = torch.randperm(T * top_k, generator=g, device="cuda").view(T, top_k).to(torch.int32)
    r = torch.randn((T * top_k, K), generator=g, device="cuda").to(torch.bfloat16 if rows_dtype == "bf16" else torch.float32)
    return position, r, torch.rand((T, top_k), generator=g, device="cuda"), g


SHAPES = [(1, 1, 8), (1, 4, 6144), (3, 2, 24), (33, 8, 1000), (64, 32, 264), (129, 3, 2056), (300, 2, 8192), (5, 4, 16384)]


@pytest.mark.parametrize("rows_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("weighted", [False, True])
@pytest.mark.parametrize("T,top_k,K", SHAPES)
def test_combine(T, top_k, K, weighted, out_dtype, rows_dtype):
    """FP32 sums of top_k products in order: |err| <= top_k 2^-24 sum |w r|, and 2^-8 |y| for BF16."""
    position, r, w, _ = rows_case(T, top_k, K, rows_dtype, T + K)
    w = w if weighted else None
    got = gg.combine_rows(r, position, w, out_dtype=out_dtype)
    v = r.double()[position.long()] * (w.double()[:, :, None] if weighted else 1.0)
    tol = top_k * 2.0 ** -24 * v.abs().sum(dim=1) + (2.0 ** -8 * v.sum(dim=1).abs() if out_dtype == "bf16" else 0)
    assert bool(((got.double() - v.sum(dim=1)).abs() <= tol).all())


@pytest.mark.parametrize("rows_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,top_k,K", SHAPES)
def test_combine_grad(T, top_k, K, out_dtype, rows_dtype):
    """d_rows is one product, rounded; a dot product of K terms is off by K 2^-24 of the sum of their magnitudes."""
    import torch
    position, r, w, g = rows_case(T, top_k, K, rows_dtype, T + K)
    dy = torch.randn((T, K), generator=g, device="cuda").to(torch.bfloat16 if out_dtype == "bf16" else torch.float32)
    d_rows, d_weight = gg.combine_grad(dy, r, position, w)
    want = (w[:, :, None] * dy.float()[:, None, :]).to(r.dtype)
    assert same(d_rows[position.long()], want)
    dots = dy.double()[:, None, :] * r.double()[position.long()]
    assert bool(((d_weight.double() - dots.sum(dim=2)).abs() <= K * 2.0 ** -24 * dots.abs().sum(dim=2)).all())
    assert same(gg.gather_rows(dy, position)[position.long()], dy[:, None, :].expand(-1, top_k, -1))


def test_positions_that_are_no_rows():
    """They add nothing, get nothing, and nothing is read or written for them."""
    import torch
    from gg_testutil import guarded_empty, guards_intact
    T, top_k, K = 5, 3, 264
    position, r, w, _ = rows_case(T, top_k, K, "fp32", 1)
    position[0, 1], position[2] = -1, torch.tensor([T * top_k, 2 ** 31 - 1, -2 ** 31], dtype=torch.int32)
    ok = (position >= 0) & (position < T * top_k)
    want = (r.double()[position.clamp(0, T * top_k - 1).long()] * (w * ok)[:, :, None].double()).sum(dim=1)
    got = gg.combine_rows(r, position, w, out_dtype="fp32")
    assert bool(((got.double() - want).abs() <= 1e-5).all()) and not got[2].any()
    buf, view, guard = guarded_empty((T * top_k, K), "fp32")
    _, d_weight = gg.combine_grad(torch.ones((T, K), device="cuda"), r, position, w, out=view)
    assert guards_intact(buf, guard, T * top_k * K, "fp32") and not d_weight[~ok].any()
    named = torch.zeros(T * top_k, dtype=torch.bool, device="cuda")
    named[position[ok].long()] = True
    assert bool(torch.isnan(view[~named]).all()) and bool(torch.isfinite(view[named]).all())


def test_no_tokens():
    import torch
    none = torch.empty((0, 4), dtype=torch.int32, device="cuda")
    r = torch.empty((0, 64), device="cuda")
    assert gg.combine_rows(r, none, torch.empty((0, 4), device="cuda")).shape == (0, 64)
    d_rows, d_weight = gg.combine_grad(r, r, none, torch.empty((0, 4), device="cuda"))
    assert d_rows.shape == (0, 64) and d_weight.shape == (0, 4) and gg.gather_rows(r, none).shape == (0, 64)


# ---------------------------------------------------------------- how a call behaves


def test_chunks_of_many_experts():
    """Blocks that go through several chunks of their tokens, with the most shared memory that takes."""
    import torch
    for T, E, top_k in ((120000, 520, 2), (160000, 24, 3)):
        logits, _ = make(T, E, 1)
        got = gg.route(logits, top_k)
        expert = torch.sort(logits, dim=1, descending=True, stable=True).indices[:, :top_k]
        by, order = torch.sort(expert.reshape(-1), stable=True)
        position = torch.empty_like(order)
        position[order] = torch.arange(order.numel(), device="cuda")
        assert same(got.expert, expert) and same(got.position, position.view(T, top_k)) and same(got.rows, order // top_k)
        assert same(got.offsets, torch.searchsorted(by, torch.arange(E + 1, device="cuda")))


def test_same_bits_on_every_run():
    import torch
    logits, bias = make(3000, 200, 5)
    o = dict(score="sigmoid", bias=bias, groups=8, top_groups=3, group_score="top2")
    first = gg.route(logits, 6, **o)
    for _ in range(5):
        assert all(torch.equal(a, b) for a, b in zip(first, gg.route(logits, 6, **o)))


@pytest.mark.parametrize("T", [40, 3000])
def test_on_a_stream_that_is_not_the_current_one(T):
    """Helpers given a stream: what they make belongs to it, and they wait for nothing else."""
    import torch
    logits, bias = make(T, 64, T)
    position, r, w, _ = rows_case(T, 4, 264, "bf16", 1)
    want = gg.route(logits, 4, bias=bias), gg.combine_rows(r, position, w)
    grads = gg.route_grad(logits, want[0].expert, w), *gg.combine_grad(want[1], r, position, w), gg.gather_rows(want[1], position)
    torch.cuda.synchronize()
    stream = torch.cuda.Stream()
    for s in (stream, stream.cuda_stream):
        got = gg.route(logits, 4, bias=bias, stream=s), gg.combine_rows(r, position, w, stream=s)
        back = (gg.route_grad(logits, got[0].expert, w, stream=s), *gg.combine_grad(got[1], r, position, w, stream=s),
                gg.gather_rows(got[1], position, stream=s))
        stream.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(got[0], want[0])) and torch.equal(got[1], want[1])
        assert all(torch.equal(a, b) for a, b in zip(back, grads))


def test_captured():
    """One graph of routing, its gradient and the rows' way, replayed on new logits."""
    import torch
    for T in (30, 2000):
        ls = [make(T, 96, i)[0] for i in range(3)]
        rows = torch.randn((T * 5, 64), generator=torch.Generator(device="cuda").manual_seed(0), device="cuda")
        def step(l, **kept):
            r = gg.route(l, 5, score="sigmoid", **kept)
            y = gg.combine_rows(rows, r.position, r.weight, out_dtype="fp32")
            d_rows, d_weight = gg.combine_grad(y, rows, r.position, r.weight)
            return (*r, y, d_rows, gg.route_grad(l, r.expert, d_weight, score="sigmoid"))
        want = [step(l) for l in ls]
        torch.cuda.synchronize()
        stream = torch.cuda.Stream()
        with torch.cuda.stream(stream):
            l = ls[0].clone()
            plan = gg.cake_gg_route_plan(T, 96, 5)
            kept = dict(plan=plan, workspace=gg.make_workspace(plan, "cuda"))
            step(l, **kept)
            stream.synchronize()
            graph = torch.cuda.CUDAGraph()
            with torch.cuda.graph(graph, stream=stream):
                got = step(l, **kept)
            for i in (1, 2, 0):
                l.copy_(ls[i])
                graph.replay()
                stream.synchronize()
                assert all(torch.equal(a, b) for a, b in zip(got, want[i]))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("T,E,top_k", [(97, 1024, 9), (128, 700, 5), (129, 700, 5), (128, 512, 8), (129, 512, 8), (200, 384, 8), (256, 256, 8),
                                       (256, 130, 17), (257, 256, 8)])
def test_around_one_cluster(T, E, top_k, score):
    """As many tokens as one cluster of blocks takes, and one more; more experts than a block has threads."""
    logits, bias = make(T, E, T + E)
    for b in (None, bias):
        check(gg.route(logits, top_k, score=score, bias=b), reference(logits, top_k, score=score, bias=b))


def test_options_by_value():
    """An option given as a tensor counts with the value that it has at the call."""
    import torch
    logits, _ = make(40, 16, 3)
    scale, renormalize, groups = torch.tensor(1.0), torch.tensor(True), torch.tensor(1)
    call = lambda: gg.route(logits, 2, scale=scale, renormalize=renormalize, groups=groups, top_groups=1)  # noqa: E731
    first = call()
    scale.fill_(2.0)
    assert torch.equal(call().weight, 2.0 * first.weight)
    renormalize.fill_(False)
    groups.fill_(4)
    check(call(), reference(logits, 2, scale=2.0, renormalize=False, groups=4, top_groups=1))


@pytest.mark.parametrize("score", ["softmax", "sigmoid"])
@pytest.mark.parametrize("with_bias", [False, True])
def test_groups_that_are_close(with_bias, score):
    """Groups whose scores differ in the last places of FP32, not at all, or by which of two near experts counts."""
    import torch
    T, E, groups = 600, 128, 8
    logits, bias = make(T, E, 11)
    l = logits.view(T, groups, E // groups)
    g = torch.Generator(device="cuda").manual_seed(2)
    base = torch.rand((T, 1, 2), generator=g, device="cuda") + 2.0
    steps = torch.randint(-2, 3, (T, groups, 2), generator=g, device="cuda")
    l[:, :, 3:5] = base * (1 + steps * 2.0 ** -23)               # the two largest, some steps apart
    l[:200, :, 7] = l[:200, :, 4] * (1 - 2.0 ** -20)             # a third beside the second
    l[200:300, 1::2] = l[200:300, ::2]                           # groups that are the same
    if with_bias:
        bias = (torch.randint(0, 3, (E // groups,), generator=g, device="cuda").float() * 0.125).repeat(groups)
    for group_score in ("max", "top2"):
        o = dict(score=score, bias=bias if with_bias else None, groups=groups, top_groups=3, group_score=group_score)
        check(gg.route(logits, 6, **o), reference(logits, 6, **o))


SHORT = [(1000, 1, 8), (13, 2, 256), (1001, 4, 256), (9, 3, 264), (50, 5, 128), (77, 1, 520), (2, 1, 1024), (31, 2, 1032), (700, 6, 1000), (160, 3, 4104)]


@pytest.mark.parametrize("rows_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("out_dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("T,top_k,K", SHORT)
def test_short_rows(T, top_k, K, out_dtype, rows_dtype):
    """Several tokens a block, the last of them not there; and more blocks than multiprocessors."""
    test_combine(T, top_k, K, True, out_dtype, rows_dtype)
    test_combine_grad(T, top_k, K, out_dtype, rows_dtype)


@pytest.mark.parametrize("T,top_k,K", [(7, 2, 128), (301, 4, 256), (11, 3, 2056)])
def test_short_rows_and_what_is_beside_them(T, top_k, K):
    """Positions that are no rows, and the memory around what is written, by every kernel."""
    import torch
    from gg_testutil import guarded_empty, guards_intact
    position, r, w, _ = rows_case(T, top_k, K, "fp32", 1)
    position[::2, -1], position[T - 1, 0] = -1, T * top_k
    ok = (position >= 0) & (position < T * top_k)
    at = position.clamp(0, T * top_k - 1).long()
    buf, view, guard = guarded_empty((T, K), "fp32")
    gg.combine_rows(r, position, w, out=view, out_dtype="fp32")
    terms = r.double()[at] * (w * ok)[:, :, None].double()
    assert guards_intact(buf, guard, T * K, "fp32")
    assert bool(((view.double() - terms.sum(dim=1)).abs() <= top_k * 2.0 ** -24 * terms.abs().sum(dim=1)).all())
    for give in (lambda out: gg.combine_grad(r[:T], r, position, w, out=out)[1], lambda out: gg.gather_rows(r[:T], position, out=out)):
        buf, view, guard = guarded_empty((T * top_k, K), "fp32")
        got = give(view)
        assert guards_intact(buf, guard, T * top_k * K, "fp32")
        named = torch.zeros(T * top_k, dtype=torch.bool, device="cuda")
        named[position[ok].long()] = True
        assert bool(torch.isnan(view[~named]).all()) and bool(torch.isfinite(view[named]).all())
        if got.shape == (T, top_k):
            assert not got[~ok].any()
