"""A mixture-of-experts layer in serving, with 8-bit weights and tokens.

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

    def _keep_nothing(self):
        self._planned = functools.lru_cache(maxsize=256)(functools.partial(_plans, self.E, self.K, self.F, self.top_k))
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

    def _for(self, T, device):
        """A call's plans, each with its workspace, and the two products' outputs."""
        route, up, down = self._planned(T)
        if torch.cuda.is_current_stream_capturing():
            mine = {}                      # (what is kept may be replaced while the graph still replays)
        else:
            mine = self._mine.__dict__.setdefault((str(device), torch.cuda.current_stream(device).cuda_stream), {})
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


def main():
    """Run a small layer on the GPU and compare it with the same layer in FP32 on the quantised weights."""
    g = torch.Generator(device="cuda").manual_seed(0)
    E, K, F, top_k = 8, 1024, 512, 2
    rand = lambda *s: torch.randn(s, generator=g, device="cuda")  # noqa: E731
    layer = Int8Experts(rand(E, K) / K ** 0.5, rand(E, 2 * F, K) / K ** 0.5, rand(E, K, F) / F ** 0.5, top_k)
    for T in (1, 16, 700):
        x = rand(T, K).to(torch.bfloat16)
        y = layer(x, check=True)
        expert, weight = layer.route(x)
        up, down = layer.up_q.float() * layer.up_s[..., None], layer.down_q.float() * layer.down_s[..., None]
        want = torch.zeros(T, K, device="cuda")
        for e in range(E):
            t, j = (expert == e).nonzero(as_tuple=True)
            gate, lin = (x[t].float() @ up[e].T).chunk(2, dim=1)
            want[t] += weight[t, j, None] * ((torch.nn.functional.silu(gate) * lin) @ down[e].T)
        err = float((y.float() - want).norm() / want.norm())
        print(f"{T} tokens: relative difference from the unquantised activations {err:.4f}")


if __name__ == "__main__":
    main()
