"""Mixture-of-experts layers in serving, with 8-bit or 4-bit weights and tokens.

    layer = Int8Experts(router, gate_up, down, top_k)
    y = layer(x)                               # x [T, K] bf16 -> y [T, K] bf16

Each token goes through the top_k experts of its router logits and their
outputs are added with softmax weights over those:

    p = softmax of the top_k of  x router^T
    y[t] = sum_j p[t, j] * down[e_j] (silu(g) * u),   [g | u] = gate_up[e_j] x[t]

The layer chains the library's calls as a server does: the FP32 router GEMM,
the grouped 8-bit product over rows routed by index (tokens quantised once,
gathered by expert), and the second grouped product, whose rows are gated and
quantised on the way.  Weights are quantised per output channel when the layer
is made.  Each thread keeps, for each device and stream, a workspace of the
largest size that it needed there and the two products' outputs of its last
call, which the next call of as many tokens writes again; y is a new tensor each
call.  Threads may call one layer at the same time, on one stream or several.
A call that is being captured in a CUDA graph has buffers of the graph's own.

    layer = Mx4Experts(router, gate_up, down, top_k, score="sigmoid", bias=bias, groups=8, top_groups=4)

is the same layer in 4-bit floating point with a power of two for each block of
32 values, in four calls of the library: the router's logits, the routing (with
all of cake_gg.route's choices), the two products, the rows' way back.
"""
from __future__ import annotations

import functools
import threading

import torch

from . import cake_gg as gg


def _plans(E, K, F, top_k, T):
    """Plans of a layer's call of T tokens: the router's, and the two products'."""
    M = T * top_k
    return (gg.cake_gg_router_plan(T, (E + 7) // 8 * 8, K), gg.cake_gg_i8_plan(E, M, T, 2 * F, K, "bf16", None, "bf16"),
            gg.cake_gg_i8_plan(E, M, M, K, F, "bf16", "silu_mul", "fp32"))


class Int8Experts:
    """Quantised experts: router [E, K] fp32, gate_up [E, 2 F, K] and down [E, K, F] bf16 or fp32 (CUDA)."""

    def __init__(self, router, gate_up, down, top_k):
        E, F2, K = gate_up.shape
        F = F2 // 2
        if tuple(router.shape) != (E, K) or tuple(down.shape) != (E, K, F) or F2 % 2:
            raise ValueError("shapes: router [E, K], gate_up [E, 2 F, K], down [E, K, F]")
        if not 1 <= top_k <= E:
            raise ValueError("top_k is 1 .. E")
        self.E, self.K, self.F, self.top_k = E, K, F, top_k
        # (the router product takes rows in eights: the rows added are cut off its logits)
        self.router = torch.nn.functional.pad(router.float(), (0, 0, 0, -E % 8)).contiguous()
        self.up_q, self.up_s = self._quantise(gate_up)
        self.down_q, self.down_s = self._quantise(down)
        self._keep_nothing()

    _plans = staticmethod(_plans)

    def _keep_nothing(self):
        self._planned = functools.lru_cache(maxsize=256)(functools.partial(self._plans, self.E, self.K, self.F, self.top_k))
        self._mine = threading.local()   # a thread's calls may interleave with another's on one stream

    def __getstate__(self):
        return {k: v for k, v in self.__dict__.items() if k not in ("_planned", "_mine")}

    def __setstate__(self, state):
        self.__dict__.update(state)
        self._keep_nothing()

    @staticmethod
    def _quantise(w):
        E, N, K = w.shape
        q, s = gg.quantize_rows(w.reshape(E * N, K).contiguous())
        return q.view(E, N, K), s.view(E, N)

    def _kept(self, device):
        """What the calling thread keeps for its current stream."""
        if torch.cuda.is_current_stream_capturing():
            return {}                      # (what is kept may be replaced while the graph still replays)
        return self._mine.__dict__.setdefault((str(device), torch.cuda.current_stream(device).cuda_stream), {})

    def _for(self, T, device):
        """A call's plans, each with its workspace, and the two products' outputs."""
        return self._buffers(T, device, self._kept(device))

    def _buffers(self, T, device, mine):
        route, up, down = self._planned(T)[:3]
        if "route" not in mine:
            mine["route"] = gg.make_workspace(route, device)         # (the same size for every T)
        # the products share a workspace: each call's kernels wait for those of the one before
        larger = up if up.workspace_bytes > down.workspace_bytes else down
        work = mine.get("products")
        if work is None or work.numel() < larger.workspace_bytes:
            grown = gg.make_workspace(larger, device)
            if work is not None:
                grown[:256] = work[:256]   # the header: a status that no check has reported yet
            mine["products"] = work = grown
        if mine.get("T") != T:
            mine.pop("out", None)
            M = T * self.top_k
            mine["out"] = (torch.empty((M, 2 * self.F), dtype=torch.bfloat16, device=device),
                           torch.empty((M, self.K), dtype=torch.float32, device=device))
            mine["T"] = T
        h, out = mine["out"]
        return (route, mine["route"]), (up, work, h), (down, work, out)

    def _check(self, x):
        """The layer's tokens, or a refusal that names what is wrong."""
        if x.dtype != torch.bfloat16:
            raise TypeError(f"x is {x.dtype}: torch.bfloat16 is needed")
        if x.dim() != 2 or x.shape[1] != self.K:
            raise ValueError(f"x has shape {tuple(x.shape)}: [T, {self.K}] is needed")
        if x.device != self.router.device:
            raise ValueError(f"x is on {x.device}, the layer on {self.router.device}")
        if not x.is_contiguous():
            raise ValueError("x is not contiguous")

    def route(self, x):
        """Experts [T, top_k] and weights [T, top_k] of each token."""
        self._check(x)
        return self._route(x, *self._for(x.shape[0], x.device)[0])

    def _route(self, x, plan, work):
        logits = gg.router_gemm(x.float(), self.router, plan=plan, workspace=work, check=False)
        top, expert = torch.topk(logits[:, :self.E], self.top_k, dim=1)
        return expert, torch.softmax(top, dim=1)

    def __call__(self, x, check=False):
        self._check(x)
        T = x.shape[0]
        if T == 0:
            return torch.empty_like(x)
        route, (up, work, h), (down, _, out) = self._for(T, x.device)
        expert, weight = self._route(x, *route)
        # rows in expert order, the token of each, and where each token's rows went
        flat = expert.reshape(-1)
        order = torch.argsort(flat, stable=True)
        rows = torch.div(order, self.top_k, rounding_mode="floor").to(torch.int32)
        counts = (flat[:, None] == torch.arange(self.E, device=x.device)).sum(dim=0)
        offsets = torch.cat([counts.new_zeros(1), counts.cumsum(0)]).to(torch.int32)
        gg.int8_gemm(x, self.up_q, self.up_s, offsets=offsets, rows=rows, out=h, plan=up, workspace=work, check=check)
        gg.int8_gemm(h, self.down_q, self.down_s, offsets=offsets, act="silu_mul", out_dtype="fp32", out=out, plan=down,
                     workspace=work, check=check)
        at = torch.empty_like(order)
        at[order] = torch.arange(order.numel(), device=x.device)
        return (out[at].view(T, self.top_k, self.K) * weight[:, :, None]).sum(dim=1).to(x.dtype)


def _mx4_plans(E, K, F, top_k, T):
    """Plans of a 4-bit layer's call of T tokens: the router's, the two products' and the routing's."""
    M = T * top_k
    return (gg.cake_gg_router_plan(T, (E + 7) // 8 * 8, K), gg.cake_gg_mx4_plan(E, M, T, 2 * F, K, "bf16", None, "bf16"),
            gg.cake_gg_mx4_plan(E, M, M, K, F, "bf16", "silu_mul", "fp32"), gg.cake_gg_route_plan(T, E, top_k))


class Mx4Experts(Int8Experts):
    """Experts in 4-bit floating point: router [E, K] fp32, gate_up [E, 2 F, K] and down [E, K, F] bf16 or fp32 (CUDA).

    K and F are multiples of 32.  score, bias, groups, top_groups, group_score,
    renormalize and scale are cake_gg.route's.
    """

    def __init__(self, router, gate_up, down, top_k, score="softmax", bias=None, groups=1, top_groups=None, group_score="max",
                 renormalize=True, scale=1.0):
        E, F2, K = gate_up.shape
        if K % 32 or F2 % 64:
            raise ValueError("K and F are multiples of 32")
        if bias is not None and (bias.dtype != torch.float32 or tuple(bias.shape) != (E,)):
            raise ValueError(f"bias is {bias.dtype} {tuple(bias.shape)}: float32 [{E}] is needed")
        self.bias = bias
        self.options = dict(score=score, groups=groups, top_groups=top_groups, group_score=group_score,
                            renormalize=renormalize, scale=scale)
        super().__init__(router, gate_up, down, top_k)

    _plans = staticmethod(_mx4_plans)

    @staticmethod
    def _quantise(w):
        return gg.quantize_mx4(w.contiguous())

    def _for(self, T, device):
        """A call's plans, each with its workspace, the two products' outputs, and the routing's."""
        mine = self._kept(device)
        products = self._buffers(T, device, mine)
        plan = self._planned(T)[3]
        if "choose" not in mine or mine["choose"].numel() < plan.workspace_bytes:
            mine["choose"] = gg.make_workspace(plan, device)
        if mine.get("routed") != T:
            mine["routing"] = gg.empty_routing(T, self.E, self.top_k, device)
            mine["routed"] = T
        return (*products, (plan, mine["choose"], mine["routing"]))

    def route(self, x):
        """Experts [T, top_k] and weights [T, top_k] of each token."""
        self._check(x)
        if x.shape[0] == 0:
            return gg.empty_routing(0, self.E, self.top_k, x.device)[:2]
        route, _, _, choose = self._for(x.shape[0], x.device)
        return tuple(t.clone() for t in self._routing(x, route, choose)[:2])

    def _routing(self, x, route, choose):
        logits = gg.router_gemm(x.float(), self.router, plan=route[0], workspace=route[1], check=False)
        plan, work, out = choose
        return gg.route(logits[:, :self.E], self.top_k, bias=self.bias, plan=plan, workspace=work, out=out, **self.options)

    def __call__(self, x, check=False):
        self._check(x)
        if x.shape[0] == 0:
            return torch.empty_like(x)
        route, (up, work, h), (down, _, out), choose = self._for(x.shape[0], x.device)
        r = self._routing(x, route, choose)
        gg.mx4_gemm(x, self.up_q, self.up_s, offsets=r.offsets, rows=r.rows, out=h, plan=up, workspace=work, check=check)
        gg.mx4_gemm(h, self.down_q, self.down_s, offsets=r.offsets, act="silu_mul", out_dtype="fp32", out=out, plan=down,
                    workspace=work, check=check)
        return gg.combine_rows(out, r.position, r.weight)


def main():
    """Run small layers on the GPU and compare each with the same layer in FP32 on the quantised weights."""
    g = torch.Generator(device="cuda").manual_seed(0)
    E, K, F, top_k = 8, 1024, 512, 2
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    weights = rand(E, K) / K ** 0.5, rand(E, 2 * F, K) / K ** 0.5, rand(E, K, F) / F ** 0.5
    for kind, values in ((Int8Experts, lambda q, s: q.float() * s[..., None]), (Mx4Experts, gg.mx4_values)):
        layer = kind(*weights, top_k)
        up, down = values(layer.up_q, layer.up_s), values(layer.down_q, layer.down_s)
        for T in (1, 16, 700):
            x = rand(T, K).to(torch.bfloat16)
            y = layer(x, check=True)
            expert, weight = layer.route(x)
            want = torch.zeros(T, K, device="cuda")
            for e in range(E):
                t, j = (expert == e).nonzero(as_tuple=True)
                gate, lin = (x[t].float() @ up[e].T).chunk(2, dim=1)
                want[t] += weight[t, j, None] * ((torch.nn.functional.silu(gate) * lin) @ down[e].T)
            err = float((y.float() - want).norm() / want.norm())
            print(f"{kind.__name__}, {T} tokens: relative difference from the unquantised activations {err:.4f}")


if __name__ == "__main__":
    main()
