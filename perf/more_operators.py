"""Measured cases of an expert layer's routing, of its rows' way out and back, and of its 4-bit products.

route       Router logits l [T, E] to each token's experts and weights, and to the
            rows in expert order that the grouped products take.  Scores s are
            the softmax of a token's logits or their sigmoid; experts are chosen
            by s + bias (by the logits, which have the order of s, where no bias
            is given), the largest first, ties to the lowest index, and where
            experts come in groups only from the groups of the largest group
            scores (a group's largest, or the sum of its two largest).  Weights
            are the chosen experts' s, divided by their sum if asked, times a
            scale.  Rows are numbered by expert, then by token: offsets [E + 1],
            the token of each row, the row of each token's j-th expert.
            Backwards: the gradient of the logits from that of the weights.

combine     y[t] = sum_j w[t, j] r[position[t, j]] (or without weights), the rows'
            way back to their tokens.  Backwards: dr[position[t, j]] = w[t, j] dy[t] and
            dw[t, j] = <dy[t], r[position[t, j]]>; without weights dr is what takes tokens
            to their rows.

mx4         Products of 4-bit floating point (E2M1: 0, 0.5, 1, 1.5, 2, 3, 4, 6 and their
            negatives, two to a byte, the even one low) whose blocks of 32 along the
            reduction share a power of two (E8M0: 2^(byte - 127)), dense or grouped by
            expert, y[m, n] = sum_k x[r(m), k] w[e(m), n, k].  Activations are quantised
            on the way, after silu(g) * u of [g | u] if asked: a block's exponent
            is floor(log2(its largest magnitude)) - 2, values are rounded to nearest,
            ties to the even code, and held at 6.  Scales lie in tiles of 128 rows x
            4 blocks: [rows / 128, blocks / 4, row % 32, row % 128 / 32, block % 4].

Widths are those of the grouped GEMM's own workloads (dense 4096 / 5120 wide
projections; gate_up 6144 -> 4096 and down 2048 -> 6144 of 32 experts, 4096-wide ones
of 8; a router over 256), token counts go from one to a long prefill.
"""
import math

import torch

own = False

TYPES = {"bf16": torch.bfloat16, "fp32": torch.float32}
BYTES = {"bf16": 2, "fp32": 4, "mx4": 0.53125}

# The most work a drawn case of an operator may have: that of its largest listed one.
MOST_LOGITS = 16384 * 256
MOST_COMBINED = 8192 * 5 * 6144
MOST_FLOPS = 2.0 * 65536 * 4096 * 4096
MOST_WEIGHTS = 32 * 6144 * 4096


def _route(name, T, E, top, score, logits="fp32", bias=False, groups=1, top_groups=1, pair=False, norm=True, scale=1.0,
           back=False):
    return {"name": name, "op": "route", "T": T, "E": E, "top": top, "score": score, "logits": logits, "bias": bias,
            "groups": groups, "top_groups": top_groups, "pair": pair, "norm": norm, "scale": scale, "back": back}


def _combine(name, T, top, K, rows, out, weights=True, back=False):
    return {"name": name, "op": "combine", "T": T, "top": top, "K": K, "rows": rows, "out": out, "weights": weights,
            "back": back}


def _mx4(name, T, E, top, K, N, x, out, act=False, routed=False, skew=0.0, empty=False):
    return {"name": name, "op": "mx4", "T": T, "E": E, "top": top, "K": K, "N": N, "x": x, "out": out, "act": act,
            "routed": routed, "skew": skew, "empty": empty}


def listed():
    return [
        # one sequence being decoded: its token to 4 of 32 experts
        _route("route one token", 1, 32, 4, "softmax"),
        # a short odd prompt over many experts in groups, a bias keeping them balanced
        _route("route 301 tokens in groups", 301, 256, 8, "sigmoid", bias=True, groups=8, top_groups=4, pair=True, scale=2.5),
        # a training step's or a long prefill's tokens over as many
        _route("route 16384 tokens", 16384, 256, 8, "sigmoid", bias=True),
        # the training step's way back, through scores that were not renormalised
        _route("route 16384 tokens, back", 16384, 256, 8, "softmax", norm=False, back=True),
        # a decoding batch's rows, kept in FP32 between the second product and the sum
        _combine("combine 33 tokens", 33, 4, 6144, "fp32", "bf16"),
        # a prefill's rows
        _combine("combine 8192 tokens", 8192, 4, 6144, "bf16", "bf16"),
        # a training step's gradients, of the rows and of the routing weights
        _combine("combine 8191 tokens, back", 8191, 2, 4096, "bf16", "bf16", back=True),
        # one token through its 4 of 32 experts: weights are all the traffic
        _mx4("4-bit up one token", 1, 32, 4, 6144, 4096, "bf16", "bf16", routed=True),
        # a decoding batch: every expert is read for a handful of rows each
        _mx4("4-bit up 64 tokens", 64, 32, 4, 6144, 4096, "bf16", "bf16", routed=True, skew=0.5),
        # a short odd prompt into a narrow head, all in FP32
        _mx4("4-bit dense 3001 to 1000 fp32", 3001, 1, 1, 5120, 1000, "fp32", "fp32"),
        # the gated second product of a prefill with skewed experts, one of them without a row
        _mx4("4-bit down prefill 8192", 8192, 32, 4, 2048, 6144, "bf16", "bf16", act=True, skew=0.8, empty=True),
        # the largest: many tokens, quantised by an earlier step, over few experts
        _mx4("4-bit up 32768 tokens", 32768, 8, 2, 4096, 4096, "mx4", "bf16", routed=True, skew=0.3),
    ]


def _log_int(rng, lo, hi, step=1):
    return max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi))) / step)) * step)


def _draw_route(rng):
    T = _log_int(rng, 1, 65536)
    groups = rng.choice([1, 1, 2, 4, 8])
    E = _log_int(rng, 8, 512) // groups * groups
    score, bias = rng.choice(["softmax", "sigmoid"]), rng.random() < 0.5
    top_groups = rng.randint(1, groups)
    top = rng.randint(1, min(16, E // groups * top_groups))
    pair = groups > 1 and E // groups >= 2 and rng.random() < 0.5
    # (a single weight that is renormalised is a constant: training takes it as it is)
    return _route("", T, E, top, score, rng.choice(["fp32", "fp32", "bf16"]), bias, groups, top_groups, pair,
                  top > 1 and rng.random() < 0.6, rng.choice([1.0, 1.0, 2.5]), rng.random() < 0.4)


def _draw_combine(rng):
    back, weights = rng.random() < 0.5, rng.random() < 0.6
    rows, out = rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["bf16", "bf16", "fp32"])
    return _combine("", _log_int(rng, 1, 32768), rng.randint(1, 8), _log_int(rng, 256, 8192, 8), out if back else rows, out,
                    weights, back)


def _draw_mx4(rng):
    K, N = _log_int(rng, 256, 8192, 32), _log_int(rng, 256, 8192, 8)
    out, x = rng.choice(["bf16", "bf16", "fp32"]), rng.choice(["bf16", "bf16", "fp32", "mx4"])
    act = x != "mx4" and rng.random() < 0.3
    if rng.random() < 0.4:
        return _mx4("", _log_int(rng, 1, 32768), 1, 1, K, N, x, out, act)
    E = _log_int(rng, 2, 64)
    return _mx4("", _log_int(rng, 1, 32768), E, min(E - 1, rng.randint(1, 8)), K, N, x, out, act, not act and rng.random() < 0.6,
                rng.choice([0.0, 0.3, 0.8, 1.2]), rng.random() < 0.3)


def _drawable(case):
    if case["op"] == "route":
        return case["T"] * case["E"] <= MOST_LOGITS
    if case["op"] == "combine":
        return case["T"] * (case["top"] + 1) * case["K"] <= MOST_COMBINED
    rows = case["T"] * case["top"]
    return (2.0 * rows * case["N"] * case["K"] <= MOST_FLOPS and case["E"] * case["N"] * case["K"] <= MOST_WEIGHTS
            and rows * max(case["K"], case["N"]) <= 1 << 29)


def draw(rng):
    while True:
        case = rng.choice([_draw_route, _draw_combine, _draw_mx4, _draw_mx4])(rng)
        if _drawable(case):
            del case["name"]
            return case


def _shares(case):
    """Each expert's share of the routing."""
    E = case["E"]
    p = [(e + 1.0) ** -case["skew"] for e in range(E)]
    if case["empty"] and E > 1:
        p[E // 2] = 0.0
    total = sum(p)
    return [v / total for v in p]


def work(case):
    T, top = case["T"], case["top"]
    M = T * top
    if case["op"] == "route":
        E, size = case["E"], BYTES[case["logits"]]
        if case["back"]:
            # the logits that count: all of them where the scores of all are normalised
            read = T * E * size if case["score"] == "softmax" and not case["norm"] else M * size
            return {"bytes": read + 8 * M + T * E * size, "flops": 6.0 * T * E}
        return {"bytes": T * E * size + (4 * E if case["bias"] else 0) + 16 * M + 4 * (E + 1), "flops": 4.0 * T * E}
    if case["op"] == "combine":
        K, rows, out = case["K"], M * case["K"] * BYTES[case["rows"]], T * case["K"] * BYTES[case["out"]]
        weights = 4 * M if case["weights"] else 0
        if case["back"]:
            return {"bytes": out + rows + 4 * M + (rows + 2 * weights if case["weights"] else 0), "flops": 3.0 * M * K}
        return {"bytes": rows + out + 4 * M + weights, "flops": 2.0 * M * K}
    K, N = case["K"], case["N"]
    # experts that have a row (their weights are read), on average over the routing
    busy = 1.0
    if case["E"] > 1:
        busy = sum(1.0 - (1.0 - min(1.0, top * p)) ** T for p in _shares(case))
        busy = max(min(busy, case["E"], M), top)
    x_rows = T if case["routed"] else M
    nbytes = x_rows * K * BYTES[case["x"]] * (2 if case["act"] else 1) + busy * N * K * BYTES["mx4"] + M * N * BYTES[case["out"]]
    nbytes += (4 * M if case["routed"] else 0) + (4 * (case["E"] + 1) if case["E"] > 1 else 0)
    return {"bytes": nbytes, "flops": 2.0 * M * N * K}


# ---------------------------------------------------------------- inputs


def _generator(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def _to_rows(expert, E):
    """Rows in expert order of experts [T, top]: offsets, the token of each row, the row of each token's j-th expert."""
    flat = expert.reshape(-1).long()
    by_expert, order = torch.sort(flat, stable=True)
    offsets = torch.searchsorted(by_expert, torch.arange(E + 1, device=flat.device)).to(torch.int32)
    position = torch.empty_like(order)
    position[order] = torch.arange(order.numel(), device=flat.device)
    rows = torch.div(order, expert.shape[1], rounding_mode="floor").to(torch.int32)
    return offsets, rows, position.view(expert.shape).to(torch.int32)


def _routed_experts(g, T, top, shares):
    """Distinct experts of each token, drawn by their shares."""
    share = torch.tensor(shares, device="cuda")
    noise = -torch.log(-torch.log(torch.rand((T, len(shares)), generator=g, device="cuda").clamp_(1e-9, 1 - 1e-7)))
    return torch.topk(torch.log(share) + noise, top, dim=1).indices


def _route_inputs(case, seed):
    g = _generator(seed)
    T, E, top = case["T"], case["E"], case["top"]
    # some experts are liked by all tokens, some tokens are surer than others
    logits = torch.randn((T, E), generator=g, device="cuda") * (0.7 + torch.rand((T, 1), generator=g, device="cuda"))
    logits = (logits + 0.5 * torch.randn(E, generator=g, device="cuda")).to(TYPES[case["logits"]])
    # what balancing has added up: steps of one size up and down
    bias = 0.001 * torch.randint(-100, 101, (E,), generator=g, device="cuda") if case["bias"] else None
    state = {"logits": logits, "bias": bias}
    if case["back"]:
        state["expert"] = _choose(dict(case, **state))[0].to(torch.int32)
        state["d_weight"] = torch.randn((T, top), generator=g, device="cuda")
    return state


def _combine_inputs(case, seed):
    g = _generator(seed)
    T, top, K = case["T"], case["top"], case["K"]
    expert = _routed_experts(g, T, top, [1.0 / (e + 4) for e in range(max(8, top))])
    state = {"position": _to_rows(expert, max(8, top))[2], "weight": None}
    if case["weights"]:
        weight = torch.rand((T, top), generator=g, device="cuda") + 0.1
        state["weight"] = weight / weight.sum(dim=1, keepdim=True)
    if case["back"]:
        state["d_out"] = torch.randn((T, K), generator=g, device="cuda").to(TYPES[case["out"]])
    if case["weights"] or not case["back"]:
        state["r"] = torch.randn((T * top, K), generator=g, device="cuda").to(TYPES[case["rows"]])
    return state


def _mx4_inputs(case, seed):
    """Tokens, weights, scales and the routing's offsets and rows, from the seed alone."""
    g = _generator(seed)
    T, E, top, K, N = (case[k] for k in ("T", "E", "top", "K", "N"))
    M = T * top
    offsets, rows, sizes = None, None, [M]
    if E > 1:
        offsets, rows, _ = _to_rows(_routed_experts(g, T, top, _shares(case)), E)
        sizes = (offsets[1:] - offsets[:-1]).tolist()
    rows = rows if case["routed"] else None
    x_rows = T if case["routed"] else M
    # activations: some channels are louder than others, rows differ in size
    width = 2 * K if case["act"] else K
    loud = 0.5 + torch.rand(width, generator=g, device="cuda") ** 4 * 4.0
    x = torch.randn((x_rows, width), generator=g, device="cuda") * loud
    x *= 0.5 + torch.rand((x_rows, 1), generator=g, device="cuda")
    xs = None
    if case["x"] == "mx4":
        x, xs = _packed(x)
    else:
        x = x.to(TYPES[case["x"]])
    w = torch.empty((E, N, K // 2), dtype=torch.uint8, device="cuda")
    ws = torch.empty((E, -(-N // 128), -(-K // 128), 32, 4, 4), dtype=torch.uint8, device="cuda")
    for e in range(E):
        w[e], ws[e] = _packed(torch.randn((N, K), generator=g, device="cuda") / math.sqrt(K))
    if E == 1:
        w, ws = w[0], ws[0]
    return {"x": x, "xs": xs, "w": w, "ws": ws, "offsets": offsets, "rows": rows, "sizes": sizes}


_INPUTS = {"route": _route_inputs, "combine": _combine_inputs, "mx4": _mx4_inputs}


def _options(case):
    """The arguments of the framework's routing calls."""
    return {"score": case["score"], "groups": case["groups"], "top_groups": case["top_groups"],
            "group_score": "top2" if case["pair"] else "max", "renormalize": case["norm"], "scale": case["scale"]}


def prepare(case, seed):
    state = dict(case, **_INPUTS[case["op"]](case, seed))
    if own:
        # what a program keeps: plans, workspaces and the buffers that outputs go to
        from moe_ragged_grouped_gb300 import cake_gg as gg
        T, top = case["T"], case["top"]
        device = torch.device("cuda", torch.cuda.current_device())
        if case["op"] == "route" and not case["back"]:
            state["plan"] = gg.cake_gg_route_plan(T, case["E"], top)
            state["workspace"] = gg.make_workspace(state["plan"], device)
            state["routing"] = gg.empty_routing(T, case["E"], top, device)
        elif case["op"] == "route":
            state["d_logits"] = torch.empty_like(state["logits"])
        elif case["op"] == "combine" and not case["back"]:
            state["y"] = torch.empty((T, case["K"]), dtype=TYPES[case["out"]], device=device)
        elif case["op"] == "combine":
            state["d_rows"] = torch.empty((T * top, case["K"]), dtype=TYPES[case["rows"]], device=device)
        else:
            M = sum(state["sizes"])
            state["plan"] = gg.cake_gg_mx4_plan(case["E"], M, state["x"].shape[0], case["N"], case["K"], case["x"],
                                                "silu_mul" if case["act"] else None, case["out"])
            state["workspace"] = gg.make_workspace(state["plan"], device)
            state["y"] = torch.empty((M, case["N"]), dtype=TYPES[case["out"]], device=device)
    return state


# ---------------------------------------------------------------- plain forms


def _scores(s):
    """Scores of all experts, in 64 bits: the choice between two of them hangs on their last places."""
    l = s["logits"].double()
    if s["score"] == "sigmoid":
        return 1.0 / (1.0 + torch.exp(-l))
    e = torch.exp(l - l.amax(dim=1, keepdim=True))
    return e / e.sum(dim=1, keepdim=True)


def _choose(s):
    """Experts [T, top] of each token, and all experts' scores where they were needed."""
    T, E, top = s["T"], s["E"], s["top"]
    scores = _scores(s) if s["bias"] is not None or s["pair"] else None
    by = s["logits"].float()
    if s["bias"] is not None:
        by = scores + s["bias"].double()
    if s["groups"] > 1:
        within = (by if s["bias"] is not None or not s["pair"] else scores).view(T, s["groups"], -1)
        most = torch.sort(within, dim=2, descending=True).values
        score = most[:, :, 0] + most[:, :, 1] if s["pair"] else most[:, :, 0]
        first = torch.sort(score, dim=1, descending=True, stable=True).indices[:, :s["top_groups"]]
        kept = (first[:, :, None] == torch.arange(s["groups"], device=by.device)).any(dim=1)
        by = by.masked_fill(~kept.repeat_interleave(E // s["groups"], dim=1), -math.inf)
    return torch.sort(by, dim=1, descending=True, stable=True).indices[:, :top], scores


def _run_route(s):
    expert = _choose(s)[0]
    l = s["logits"].float()
    if s["score"] == "sigmoid":
        weight = 1.0 / (1.0 + torch.exp(-l.gather(1, expert)))
    else:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        weight = e.gather(1, expert) / e.sum(dim=1, keepdim=True)
    if s["norm"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    offsets, rows, position = _to_rows(expert, s["E"])
    return {"expert": expert.to(torch.int32), "weight": weight * s["scale"], "offsets": offsets, "rows": rows,
            "position": position}


def _run_route_back(s):
    l, at, g = s["logits"].float(), s["expert"].long(), s["d_weight"] * s["scale"]
    if s["score"] == "softmax" and not s["norm"]:
        e = torch.exp(l - l.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        inner = (g * p.gather(1, at)).sum(dim=1, keepdim=True)
        d = -p * inner
        return d.scatter_add(1, at, p.gather(1, at) * g).to(s["logits"].dtype)
    chosen = l.gather(1, at)
    if s["score"] == "softmax":
        e = torch.exp(chosen - chosen.amax(dim=1, keepdim=True))
        p = e / e.sum(dim=1, keepdim=True)
        d = p * (g - (g * p).sum(dim=1, keepdim=True))
    else:
        p = 1.0 / (1.0 + torch.exp(-chosen))
        if s["norm"]:
            total = p.sum(dim=1, keepdim=True)
            g = (g - (g * p).sum(dim=1, keepdim=True) / total) / total
        d = g * p / (1.0 + torch.exp(chosen))
    return torch.zeros_like(l).scatter_(1, at, d).to(s["logits"].dtype)


def _run_combine(s):
    r = s["r"].float()[s["position"].long()]
    if s["weight"] is not None:
        r = r * s["weight"][:, :, None]
    return r.sum(dim=1).to(TYPES[s["out"]])


def _run_combine_back(s):
    at, dy = s["position"].reshape(-1).long(), s["d_out"].float()
    d = dy[:, None, :].expand(-1, s["top"], -1)
    if s["weight"] is not None:
        d = d * s["weight"][:, :, None]
    d_rows = torch.empty((at.numel(), s["K"]), dtype=TYPES[s["rows"]], device=dy.device)
    d_rows[at] = d.reshape(-1, s["K"]).to(TYPES[s["rows"]])
    if s["weight"] is None:
        return {"d_rows": d_rows}
    return {"d_rows": d_rows, "d_weight": (s["r"].float()[s["position"].long()] * dy[:, None, :]).sum(dim=2)}


def _quantised(x):
    """Values of the 4-bit format in 32 bits, and the exponents of their blocks of 32: x [R, K] -> [R, K / 32, 32], [R, K / 32]."""
    x = x.view(x.shape[0], -1, 32)
    exponent = (torch.frexp(x.abs().amax(dim=2)).exponent - 3).clamp(min=-127)
    a = torch.ldexp(x.abs(), -exponent[:, :, None])
    a = torch.where(a < 2.0, torch.round(a * 2.0) * 0.5, torch.where(a < 4.0, torch.round(a), torch.round(a * 0.5) * 2.0))
    return torch.copysign(a.clamp(max=6.0), x).float(), exponent


def _packed(x):
    """The same as bytes: two codes each, and the exponents in tiles of 128 rows x 4 blocks."""
    values, exponent = _quantised(x)
    a = values.abs()
    code = torch.where(a < 2.0, a * 2.0, torch.where(a < 4.0, a + 2.0, a * 0.5 + 4.0)).to(torch.uint8)
    code = (code + 8 * torch.signbit(values).to(torch.uint8)).view(x.shape[0], -1, 2)
    R, B = exponent.shape
    tiles = torch.zeros((-(-R // 128) * 128, -(-B // 4) * 4), dtype=torch.uint8, device=x.device)
    tiles[:R, :B] = (exponent + 127).to(torch.uint8)
    tiles = tiles.view(-1, 4, 32, tiles.shape[1] // 4, 4).permute(0, 3, 2, 1, 4).contiguous()
    return code[:, :, 0] | code[:, :, 1] << 4, tiles


def _values(q, tiles):
    """The numbers that packed rows [R, K / 2] and their tiles of scales stand for, in 32 bits."""
    R, K = q.shape[0], q.shape[1] * 2
    table = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0, -0.0, -0.5, -1.0, -1.5, -2.0, -3.0, -4.0, -6.0], device=q.device)
    v = table[torch.stack([q & 15, q >> 4], dim=2).long()].view(R, K // 32, 32)
    exponent = tiles.permute(0, 3, 2, 1, 4).reshape(tiles.shape[0] * 128, -1)[:R, :K // 32]
    return torch.ldexp(v, exponent.to(torch.int32)[:, :, None] - 127).view(R, K)


def _run_mx4(s):
    if s["xs"] is not None:
        x = _values(s["x"], s["xs"])
    else:
        x = s["x"].float()
        if s["act"]:
            # in 64 bits: the value next to a border between two codes goes to the right one
            gate, up = s["x"].double().chunk(2, dim=1)
            x = gate / (1.0 + torch.exp(-gate)) * up
        values, exponent = _quantised(x)
        x = torch.ldexp(values, exponent[:, :, None]).view(values.shape[0], -1)
    if s["rows"] is not None:
        x = x[s["rows"].long()]
    if s["offsets"] is None:
        return (x @ _values(s["w"], s["ws"]).T).to(TYPES[s["out"]])
    # the experts that have rows, one product each
    return torch.cat([rows @ _values(w, ws).T
                      for rows, w, ws in zip(x.split(s["sizes"]), s["w"], s["ws"]) if rows.shape[0]]).to(TYPES[s["out"]])


def run(state):
    s = state
    if own:
        from moe_ragged_grouped_gb300 import cake_gg as gg
        if s["op"] == "route" and not s["back"]:
            return gg.route(s["logits"], s["top"], bias=s["bias"], plan=s["plan"], workspace=s["workspace"], out=s["routing"],
                            **_options(s))._asdict()
        if s["op"] == "route":
            return gg.route_grad(s["logits"], s["expert"], s["d_weight"], score=s["score"], renormalize=s["norm"],
                                 scale=s["scale"], out=s["d_logits"])
        if s["op"] == "combine" and not s["back"]:
            return gg.combine_rows(s["r"], s["position"], s["weight"], out_dtype=s["out"], out=s["y"])
        if s["op"] == "combine" and s["weight"] is None:
            return {"d_rows": gg.gather_rows(s["d_out"], s["position"], out=s["d_rows"])}
        if s["op"] == "combine":
            d_rows, d_weight = gg.combine_grad(s["d_out"], s["r"], s["position"], s["weight"], out=s["d_rows"])
            return {"d_rows": d_rows, "d_weight": d_weight}
        return gg.mx4_gemm(s["x"], s["w"], s["ws"], xs=s["xs"], offsets=s["offsets"], rows=s["rows"],
                           act="silu_mul" if s["act"] else None, out_dtype=s["out"], out=s["y"], plan=s["plan"],
                           workspace=s["workspace"], check=False)
    if s["op"] == "route":
        return _run_route_back(s) if s["back"] else _run_route(s)
    if s["op"] == "combine":
        return _run_combine_back(s) if s["back"] else _run_combine(s)
    return _run_mx4(s)


# ---------------------------------------------------------------- the definitions in 64 bits


def _exact_probabilities(case, logits):
    l = logits.to(torch.float64)
    return torch.sigmoid(l) if case["score"] == "sigmoid" else torch.softmax(l, dim=1)


def _exact_route(case, s):
    T, E, top = case["T"], case["E"], case["top"]
    p = _exact_probabilities(case, s["logits"])
    key = s["logits"].to(torch.float64) if s["bias"] is None else p + s["bias"].to(torch.float64)
    if case["groups"] > 1:
        group_key = key if s["bias"] is not None or not case["pair"] else p
        group = torch.topk(group_key.reshape(T, case["groups"], -1), 2 if case["pair"] else 1, dim=2).values.sum(dim=2)
        place = group.argsort(dim=1, descending=True, stable=True).argsort(dim=1)
        key = torch.where((place < case["top_groups"]).repeat_interleave(E // case["groups"], dim=1), key,
                          torch.full_like(key, -math.inf))
    expert = key.argsort(dim=1, descending=True, stable=True)[:, :top]
    weight = torch.take_along_dim(p, expert, 1)
    if case["norm"]:
        weight = weight / weight.sum(dim=1, keepdim=True)
    # a row's number: the rows of experts before its own, and of its own the tokens before it
    chosen = torch.zeros((T, E), dtype=torch.int64, device=p.device).scatter_(1, expert, 1)
    before = torch.cumsum(chosen, dim=0) - chosen
    offsets = torch.zeros(E + 1, dtype=torch.int64, device=p.device)
    offsets[1:] = torch.cumsum(chosen.sum(dim=0), dim=0)
    position = offsets[expert] + torch.take_along_dim(before, expert, 1)
    rows = torch.empty(T * top, dtype=torch.int64, device=p.device)
    rows[position.flatten()] = torch.arange(T, device=p.device).repeat_interleave(top)
    return {"expert": expert, "weight": weight * case["scale"], "offsets": offsets, "rows": rows, "position": position}


def _exact_route_back(case, s):
    # the chosen weights as a product with the scores' Jacobian, a token at a time in one batch
    at, g = s["expert"].to(torch.int64), s["d_weight"].to(torch.float64) * case["scale"]
    p = _exact_probabilities(case, s["logits"])
    d_p = torch.zeros_like(p)
    if case["norm"]:
        chosen = torch.take_along_dim(p, at, 1)
        total = chosen.sum(dim=1, keepdim=True)
        g = g / total - (g * chosen).sum(dim=1, keepdim=True) / total ** 2
    d_p.scatter_(1, at, g)
    if case["score"] == "sigmoid":
        return d_p * p * (1.0 - p)
    return p * (d_p - torch.einsum("te,te->t", p, d_p)[:, None])


def _exact_combine(case, s):
    y = torch.zeros((case["T"], case["K"]), dtype=torch.float64, device=s["r"].device)
    for j in range(case["top"]):
        part = s["r"].index_select(0, s["position"][:, j]).to(torch.float64)
        y += part if s["weight"] is None else part * s["weight"][:, j:j + 1].to(torch.float64)
    return y


def _exact_combine_back(case, s):
    dy = s["d_out"].to(torch.float64)
    out = {"d_rows": torch.empty((case["T"] * case["top"], case["K"]), dtype=torch.float64, device=dy.device)}
    if s["weight"] is not None:
        out["d_weight"] = torch.empty((case["T"], case["top"]), dtype=torch.float64, device=dy.device)
    for j in range(case["top"]):
        at = s["position"][:, j].to(torch.int64)
        out["d_rows"][at] = dy if s["weight"] is None else dy * s["weight"][:, j:j + 1].to(torch.float64)
        if s["weight"] is not None:
            out["d_weight"][:, j] = torch.einsum("tk,tk->t", dy, s["r"].index_select(0, at).to(torch.float64))
    return out


def _exact_rounded(h):
    """h [R, K] as the 4-bit format holds it: a code counts the borders below a value, those of odd codes themselves included."""
    blocks = h.reshape(h.shape[0], -1, 32)
    largest = blocks.abs().max(dim=2, keepdim=True).values
    power = torch.floor(torch.log2(largest))
    power += (torch.exp2(power + 1.0) <= largest).to(power.dtype)     # (a logarithm may fall short of a whole number)
    scale = torch.exp2((power - 2.0).clamp_(min=-127.0))
    a = blocks.abs() / scale
    code = sum([(a > b).to(torch.int8) for b in (0.25, 1.25, 2.5, 5.0)] + [(a >= b).to(torch.int8) for b in (0.75, 1.75, 3.5)])
    grid = torch.tensor([0.0, 0.5, 1.0, 1.5, 2.0, 3.0, 4.0, 6.0], dtype=torch.float64, device=h.device)
    return (grid[code.to(torch.int64)] * scale * torch.sign(blocks)).reshape(h.shape)


def _exact_values(q, tiles):
    """Packed rows in 64 bits, a column of 32 blocks' scales at a time."""
    R, half = q.shape
    out = torch.empty((R, 2 * half), dtype=torch.float64, device=q.device)
    for odd in (0, 1):
        code = (q >> (4 * odd)) & 15
        low = (code & 7).to(torch.float64)
        size = torch.where(low < 4, low / 2, torch.where(low < 6, low - 2, 2 * low - 8))
        out[:, odd::2] = torch.where(code > 7, -size, size)
    r = torch.arange(R, device=q.device)
    for b in range(2 * half // 32):
        byte = tiles[r // 128, b // 4, r % 32, r % 128 // 32, b % 4].to(torch.float64)
        out[:, 32 * b:32 * b + 32] *= torch.exp2(byte - 127.0)[:, None]
    return out


def _exact_mx4(case, s):
    if s["xs"] is not None:
        x = _exact_values(s["x"], s["xs"])
    else:
        h = s["x"].to(torch.float64)
        if case["act"]:
            h = torch.sigmoid(h[:, :case["K"]]) * h[:, :case["K"]] * h[:, case["K"]:]
        x = _exact_rounded(h)
    w, ws = (s["w"], s["ws"]) if case["E"] > 1 else (s["w"][None], s["ws"][None])
    M = sum(s["sizes"])
    y = torch.zeros((M, case["N"]), dtype=torch.float64, device=x.device)
    begin = 0
    for e, n in enumerate(s["sizes"]):
        if n:
            mine = x[begin:begin + n] if s["rows"] is None else x.index_select(0, s["rows"][begin:begin + n])
            torch.matmul(mine, _exact_values(w[e], ws[e]).t(), out=y[begin:begin + n])
        begin += n
    return y


def exact(case, seed):
    s = _INPUTS[case["op"]](case, seed)
    if case["op"] == "route":
        return _exact_route_back(case, s) if case["back"] else _exact_route(case, s)
    if case["op"] == "combine":
        return _exact_combine_back(case, s) if case["back"] else _exact_combine(case, s)
    return _exact_mx4(case, s)
