"""Measured cases of the 8-bit integer products: dense, and grouped by expert with ragged sizes.

Each case is one pass of a quantised linear layer in serving.  Tokens come as
activations (BF16 or FP32) that the layer quantises row by row on the way, as
the output [gate | up] of a gated projection that it first turns into
silu(gate) * up, or as 8-bit rows with scales that an earlier step left:

    s[t] = max_k |x[t, k]| / 127        q[t, k] = round(x[t, k] * (127 / max_k |x[t, k]|))
    y[m, n] = s[r(m)] * ws[e(m), n] * sum_k q[r(m), k] * wq[e(m), n, k]

with 8-bit weights wq and a scale ws for each output channel; e(m) is the
expert that owns row m (one expert: the dense product) and r(m) the token that
row m was routed from (the row itself where nothing is routed).

Widths are those of the grouped GEMM's own workloads (dense 4096 / 5120 wide
projections; gate_up 6144 -> 4096 and down 2048 -> 6144 of the MoE layer,
4096-wide experts), token counts go from one to a long prefill.
"""
import math

import torch

own = False

OUT_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
IN_DTYPES = {"bf16": torch.bfloat16, "fp32": torch.float32, "int8": torch.int8}

# The most work a drawn case may have: that of the largest listed one.
MAX_FLOPS = 2.0 * 65536 * 4096 * 4096
MAX_WEIGHTS = 32 * 6144 * 4096


def _dense(name, T, K, N, x, out, act=False):
    return {"name": name, "op": "dense", "T": T, "E": 1, "top": 1, "K": K, "N": N, "x": x, "out": out, "act": act,
            "routed": False, "skew": 0.0, "empty": False}


def _grouped(name, T, E, top, K, N, x, out, act=False, routed=True, skew=0.0, empty=False):
    return {"name": name, "op": "grouped", "T": T, "E": E, "top": top, "K": K, "N": N, "x": x, "out": out, "act": act,
            "routed": routed, "skew": skew, "empty": empty}


def listed():
    return [
        # one sequence being decoded: a single token through a square projection
        _dense("dense one token", 1, 4096, 4096, "bf16", "bf16"),
        # a batch of sequences being decoded: a few dozen tokens, odd count
        _dense("dense 33 tokens", 33, 4096, 5120, "bf16", "bf16"),
        # a short odd prompt into a narrow head kept in FP32
        _dense("dense 3001 to 1000 fp32", 3001, 5120, 1000, "fp32", "fp32"),
        # a long prefill whose tokens an earlier step already quantised
        _dense("dense prefill 16384", 16384, 4096, 4096, "int8", "bf16"),
        # one token through its 4 of 32 experts: weights are all the traffic
        _grouped("up one token", 1, 32, 4, 6144, 4096, "bf16", "bf16"),
        # the same token's down products, gated on the way
        _grouped("down one token", 1, 32, 4, 2048, 6144, "bf16", "bf16", act=True, routed=False),
        # a decoding batch: every expert is read for a handful of rows each
        _grouped("up 64 tokens", 64, 32, 4, 6144, 4096, "bf16", "bf16", skew=0.5),
        _grouped("down 64 tokens", 64, 32, 4, 2048, 6144, "bf16", "bf16", act=True, routed=False, skew=0.5),
        # a short odd prompt over few wide experts, quantised tokens, FP32 sums kept
        _grouped("up 701 tokens fp32", 701, 8, 2, 4096, 2048, "int8", "fp32", skew=1.0),
        # prefill with skewed experts, one of them without a row
        _grouped("up prefill 8192", 8192, 32, 4, 6144, 4096, "bf16", "bf16", skew=0.8, empty=True),
        _grouped("down prefill 8192", 8192, 32, 4, 2048, 6144, "bf16", "bf16", act=True, routed=False, skew=0.8, empty=True),
        # the largest: many quantised tokens over few experts
        _grouped("up 32768 tokens", 32768, 8, 2, 4096, 4096, "int8", "bf16", skew=0.3),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def draw(rng):
    while True:
        K = _log_int(rng, 256, 8192, 16)
        N = _log_int(rng, 256, 8192, 8)
        out = rng.choice(["bf16", "bf16", "fp32"])
        x = rng.choice(["bf16", "bf16", "fp32", "int8"])
        act = x != "int8" and rng.random() < 0.3
        if rng.random() < 0.4:
            T = _log_int(rng, 1, 16384)
            case = _dense("", T, K, N, x, out, act)
        else:
            E = _log_int(rng, 2, 64)
            top = min(E - 1, rng.randint(1, 8))
            T = _log_int(rng, 1, 32768)
            case = _grouped("", T, E, max(1, top), K, N, x, out, act, routed=not act and rng.random() < 0.6,
                            skew=rng.choice([0.0, 0.3, 0.8, 1.2]), empty=rng.random() < 0.3)
        del case["name"]
        w = work(case)
        if w["flops"] <= MAX_FLOPS and case["E"] * K * N <= MAX_WEIGHTS and case["T"] * case["top"] * max(K, N) <= 1 << 29:
            return case


def _shares(case):
    """Each expert's share of the routing."""
    E = case["E"]
    p = [(e + 1.0) ** -case["skew"] for e in range(E)]
    if case["empty"]:
        p[E // 2] = 0.0
    total = sum(p)
    return [v / total for v in p]


def work(case):
    T, K, N, M = case["T"], case["K"], case["N"], case["T"] * case["top"]
    # experts that have a row (their weights are read), on average over the routing
    busy = 1.0
    if case["op"] == "grouped":
        busy = sum(1.0 - (1.0 - min(1.0, case["top"] * p)) ** T for p in _shares(case))
        busy = max(min(busy, case["E"], M), case["top"])
    x_rows = T if case["routed"] or case["op"] == "dense" else M
    x_size = {"int8": 1, "bf16": 2, "fp32": 4}[case["x"]]
    nbytes = x_rows * K * x_size * (2 if case["act"] else 1) + (4 * x_rows if case["x"] == "int8" else 0)
    nbytes += busy * (N * K + 4 * N) + M * N * {"bf16": 2, "fp32": 4}[case["out"]]
    nbytes += (4 * M if case["routed"] else 0) + (4 * (case["E"] + 1) if case["op"] == "grouped" else 0)
    return {"bytes": nbytes, "flops": 2.0 * M * N * K}


def _inputs(case, seed):
    """Tokens, weights, scales and the routing's offsets and rows, from the seed alone."""
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    T, E, top, K, N = (case[k] for k in ("T", "E", "top", "K", "N"))
    M = T * top
    rows, offsets, sizes = None, None, [M]
    if case["op"] == "grouped":
        # distinct experts of each token, drawn by their shares, rows sorted by expert
        share = torch.tensor(_shares(case), device="cuda")
        noise = -torch.log(-torch.log(torch.rand((T, E), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
        expert = torch.topk(torch.log(share) + noise, top, dim=1).indices.reshape(-1)
        order = torch.sort(expert, stable=True).indices
        counts = torch.bincount(expert, minlength=E)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        sizes = counts.tolist()
        if case["routed"]:
            rows = torch.div(order, top, rounding_mode="floor").to(torch.int32)
    x_rows = T if case["routed"] or case["op"] == "dense" else M
    width = 2 * K if case["act"] else K
    xs = None
    if case["x"] == "int8":
        x = (torch.randn((x_rows, K), generator=g, device="cuda") * 32.0).round_().clamp_(-127, 127).to(torch.int8)
        xs = (torch.rand(x_rows, generator=g, device="cuda") + 0.5) * 0.03
    else:
        # activations: some channels are louder than others, rows differ in size
        loud = 0.5 + torch.rand(width, generator=g, device="cuda") ** 4 * 4.0
        x = torch.randn((x_rows, width), generator=g, device="cuda") * loud
        x *= 0.5 + torch.rand((x_rows, 1), generator=g, device="cuda")
        x = x.to(IN_DTYPES[case["x"]])
    wq = torch.empty((E, N, K), dtype=torch.int8, device="cuda")
    for e in range(E):
        # normal weights whose largest of a channel lies near four deviations
        wq[e] = (torch.randn((N, K), generator=g, device="cuda") * 32.0).round_().clamp_(-127, 127)
    ws = (torch.rand((E, N), generator=g, device="cuda") + 0.5) / (32.0 * math.sqrt(K))
    if case["op"] == "dense":
        wq, ws = wq[0], ws[0]
    return {"x": x, "xs": xs, "wq": wq, "ws": ws, "offsets": offsets, "rows": rows, "sizes": sizes}


def prepare(case, seed):
    state = dict(_inputs(case, seed), act="silu_mul" if case["act"] else None, out=case["out"])
    if own:
        from moe_ragged_grouped_gb300 import cake_gg as gg
        M = sum(state["sizes"])
        state["plan"] = gg.cake_gg_i8_plan(case["E"], M, state["x"].shape[0], case["N"], case["K"], case["x"],
                                           state["act"], case["out"])
        state["workspace"] = gg.make_workspace(state["plan"], state["x"].device)
        state["y"] = torch.empty((M, case["N"]), dtype=OUT_DTYPES[case["out"]], device=state["x"].device)
    return state


def _quantised(x):
    """Integer rows (as FP32 values) and their scales."""
    amax = x.abs().amax(dim=1)
    inv = torch.where(amax > 0, torch.div(torch.full_like(amax, 127.0), amax), torch.zeros_like(amax))
    return torch.round(x * inv[:, None]), torch.div(amax, torch.full_like(amax, 127.0))


def run(state):
    if own:
        from moe_ragged_grouped_gb300 import cake_gg as gg
        return gg.int8_gemm(state["x"], state["wq"], state["ws"], xs=state["xs"], offsets=state["offsets"],
                            rows=state["rows"], act=state["act"], out_dtype=state["out"], out=state["y"],
                            plan=state["plan"], workspace=state["workspace"], check=False)
    x, xs = state["x"].float(), state["xs"]
    if state["act"]:
        gate, up = x.chunk(2, dim=1)
        x = gate / (1.0 + torch.exp(-gate)) * up
    if xs is None:
        x, xs = _quantised(x)
    if state["rows"] is not None:
        x, xs = x[state["rows"].long()], xs[state["rows"].long()]
    if state["offsets"] is None:
        y = (x @ state["wq"].float().T) * state["ws"]
    else:
        # the experts that have rows, one product each
        y = torch.cat([(rows @ w.float().T) * s
                       for rows, w, s in zip(x.split(state["sizes"]), state["wq"], state["ws"]) if rows.shape[0]])
    return (y * xs[:, None]).to(OUT_DTYPES[state["out"]])


def exact(case, seed):
    """The definition in 64 bits, an expert at a time."""
    s = _inputs(case, seed)
    x = s["x"].to(torch.float64)
    if case["act"]:
        K = case["K"]
        x = x[:, :K] * torch.sigmoid(x[:, :K]) * x[:, K:]
    if s["xs"] is None:
        scale = x.abs().max(dim=1, keepdim=True).values / 127.0
        q = torch.round(x / scale.clamp(min=1e-300))
    else:
        scale, q = s["xs"].to(torch.float64)[:, None], x
    if s["rows"] is not None:
        at = s["rows"].to(torch.int64)
        scale, q = scale[at], q[at]
    wq, ws = s["wq"].reshape(case["E"], case["N"], case["K"]), s["ws"].reshape(case["E"], case["N"])
    y = torch.zeros((q.shape[0], case["N"]), dtype=torch.float64, device=q.device)
    begin = 0
    for e, n in enumerate(s["sizes"]):
        end = begin + n
        if n:
            y[begin:end] = torch.matmul(q[begin:end], wq[e].to(torch.float64).t()).mul_(ws[e].to(torch.float64))
        begin = end
    return y * scale
