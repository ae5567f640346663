"""One feed-forward block of a decoding step on FP8 block weights: norm, router, shared expert, routed
experts, residual stream.

    python examples/feed_forward.py [--tokens 16] [--hidden 2048] [--inter 1408] [--experts 16] [--top-k 4]

The block adds to the residual stream h [T, H] (bf16):

    x = rms_norm(h)
    ids, weights = route(x . Wr^T)                                     moe_route
    h = h + Wd . (silu(Wg . x) * (Wu . x))      shared expert          gemm_epilogue (activation; residual)
    h = h + sum_j weights[j] expert[ids[j]](x)  routed experts         moe_ffn (residual in place)

Weights are random; the program prints the block's time, eager and replayed from a HIP graph.
"""
import argparse
import os
import sys

import torch

sys.path.insert(0, os.path.dirname(os.path.dirname(os.path.abspath(__file__))))
import fine_grained_block_amd as fgb  # noqa: E402


def make_params(hidden: int, inter: int, experts: int, seed: int = 0, device="cuda", scale_fmt: str = "ue8m0") -> dict:
    """Random weights, quantized once: the shared expert's gate, up and down projections, the routed
    experts' stacked [gate; up] and down projections, the router and its selection bias."""
    gen = torch.Generator(device=device)
    gen.manual_seed(seed)

    def weight(n, k):
        return fgb.quantize_weight((0.02 * torch.randn((n, k), generator=gen, device=device)).to(torch.bfloat16), scale_fmt)

    stack = lambda ws: tuple(torch.stack(t) for t in zip(*ws))
    return {
        "norm": torch.ones(hidden, device=device),
        "router": torch.randn((experts, hidden), generator=gen, device=device) / hidden ** 0.5,
        "select_bias": 0.01 * torch.randn(experts, generator=gen, device=device),
        "gate": weight(inter, hidden), "up": weight(inter, hidden), "down": weight(hidden, inter),
        "w13": stack([weight(2 * inter, hidden) for _ in range(experts)]),
        "w2": stack([weight(hidden, inter) for _ in range(experts)]),
    }


def rms_norm(h: torch.Tensor, gain: torch.Tensor) -> torch.Tensor:
    f = h.float()
    return (f * torch.rsqrt(f.square().mean(-1, keepdim=True) + 1e-6) * gain).to(torch.bfloat16)


def feed_forward(h: torch.Tensor, p: dict, top_k: int, workspace: torch.Tensor | None = None) -> torch.Tensor:
    """The block on h bf16 [T, H] (T <= 64); returns the new residual stream."""
    x = rms_norm(h, p["norm"])
    ids, weights = fgb.moe_route(x.float() @ p["router"].t(), top_k, scoring="sigmoid", select_bias=p["select_bias"],
                                 scale=1.5)
    q, s = fgb.quantize(x)
    gated = fgb.gemm_epilogue(q, s, *p["gate"], activation="silu") * fgb.gemm(q, s, *p["up"])
    h = fgb.gemm_epilogue(*fgb.quantize(gated), *p["down"], residual=h)
    return fgb.moe_ffn(x, ids, weights, *p["w13"], *p["w2"], residual=h, out=h, workspace=workspace)


def main() -> None:
    ap = argparse.ArgumentParser(description=__doc__, formatter_class=argparse.RawDescriptionHelpFormatter)
    ap.add_argument("--tokens", type=int, default=16)
    ap.add_argument("--hidden", type=int, default=2048)
    ap.add_argument("--inter", type=int, default=1408)
    ap.add_argument("--experts", type=int, default=16)
    ap.add_argument("--top-k", type=int, default=4)
    a = ap.parse_args()
    p = make_params(a.hidden, a.inter, a.experts)
    h = torch.randn((a.tokens, a.hidden), device="cuda").to(torch.bfloat16)
    ws = torch.empty(fgb.moe_ffn_workspace_bytes(a.tokens, a.top_k, a.experts, a.hidden, a.inter), dtype=torch.uint8,
                     device="cuda")

    def timed(f, n=50):
        for _ in range(5):
            f()
        start, end = torch.cuda.Event(enable_timing=True), torch.cuda.Event(enable_timing=True)
        start.record()
        for _ in range(n):
            f()
        end.record()
        torch.cuda.synchronize()
        return start.elapsed_time(end) / n * 1e3

    step = lambda: feed_forward(h, p, a.top_k, ws)
    print(f"eager: {timed(step):.1f} us per block")
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step()
    print(f"graph: {timed(graph.replay):.1f} us per block; |h| {out.float().norm().item():.3f}")


if __name__ == "__main__":
    main()
