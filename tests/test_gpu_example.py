"""GPU: the example's feed-forward block (router, epilogue GEMMs, mixture-of-experts layer on one residual
stream) against a float32 composition of dequantized weights, and replayed from a graph.

Tolerance: the composition skips the activation quantization (E4M3 steps of at most 1/16 of a value,
uniform: 1.8% rms per operand, so below 4% of each projection's rms after two of them) and the block
adds to a residual stream of comparable size: 6% of the stream's change in the 2-norm."""
import importlib.util
import os

import pytest
import torch

import fine_grained_block_amd as fgb

pytestmark = pytest.mark.gpu

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def _example():
    spec = importlib.util.spec_from_file_location("feed_forward_example", os.path.join(ROOT, "examples", "feed_forward.py"))
    m = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(m)
    return m


def _dense(w_q, s_w):
    s = fgb.fp8_decode(s_w.contiguous(), fgb.UE8M0)
    w = fgb.fp8_decode(w_q.contiguous())
    return w * s.repeat_interleave(128, -2).repeat_interleave(128, -1)


@pytest.mark.parametrize("tokens", [1, 5, 33])
def test_feed_forward_block(dev, tokens):
    ex = _example()
    H, I, E, k = 512, 384, 6, 2
    p = ex.make_params(H, I, E, seed=tokens)
    h = torch.randn((tokens, H), generator=torch.Generator().manual_seed(tokens)).to(torch.bfloat16).to(dev)
    y = ex.feed_forward(h, p, k)
    x = ex.rms_norm(h, p["norm"])
    ids, w = fgb.moe_route(x.float() @ p["router"].t(), k, scoring="sigmoid", select_bias=p["select_bias"], scale=1.5)
    xf = x.float()
    ffn = lambda t, g, u, d: (torch.nn.functional.silu(t @ g.t()) * (t @ u.t())) @ d.t()
    change = ffn(xf, _dense(*p["gate"]), _dense(*p["up"]), _dense(*p["down"]))
    w13, w2 = _dense(*p["w13"]), _dense(*p["w2"])
    for t in range(tokens):
        for j in range(k):
            e = int(ids[t, j])
            change[t] += w[t, j] * ffn(xf[t:t + 1], w13[e, :I], w13[e, I:], w2[e])[0]
    err = (y.float() - h.float() - change).norm()
    assert err <= 0.06 * change.norm() + 2.0 ** -8 * y.float().norm()
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        out = ex.feed_forward(h, p, k)
    for _ in range(3):
        out.fill_(float("nan"))
        ex.feed_forward(h + 1, p, k)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, y)
