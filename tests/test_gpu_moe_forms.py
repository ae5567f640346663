"""GPU: the launch forms of the mixture-of-experts layer (fgb_moe_ffn) that need many experts or wide layers:
against the float64 oracle, and equal bit for bit with pitched rows, out = residual and a workspace full of
NaN patterns.

Tolerance: that of tests/test_gpu_moe_ffn.py, derived there (5e-3 of the experts' part in the 2-norm, single
elements sixteen times that).  The rules choose by min(T top_k, E), so the tokens here share a few of many
experts, one of them all of the tokens: the weights are drawn on the GPU and the oracle gets the experts that are read."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
import workloads
from tests.gemm_helpers import to_dev_bf16
from tests.test_gpu_moe_ffn import _check

pytestmark = pytest.mark.gpu

# T, E, top_k, H, I: quantization late (wide down, K-blocks of a segment odd), in gate+up or by the prep launch,
# K whole or sliced, one, two and four row tiles, wide and narrow down, experts whole or sliced
SHAPES = [(2, 6, 3, 5120, 1024), (1, 8, 8, 5248, 1408), (3, 6, 3, 2048, 2048), (7, 256, 37, 5248, 128),
          (20, 8, 3, 512, 1536), (9, 4, 2, 5376, 256), (16, 128, 8, 2560, 128), (9, 256, 29, 5248, 128),
          (20, 4, 2, 5248, 256), (18, 256, 15, 3712, 128), (20, 256, 13, 5248, 128), (40, 12, 2, 2048, 1024),
          (40, 4, 2, 5376, 256), (48, 256, 6, 5248, 128)]


def _draw(dev, T, E, k, H, I, fmt):
    gen = torch.Generator(device=dev)
    gen.manual_seed(T + E + H + I)

    def codes(n, m):  # finite codes, small magnitudes the most frequent
        c = torch.randn((E, n, m), generator=gen, device=dev, dtype=torch.float16).mul_(40).clamp_(-127, 127)
        c = c.to(torch.int16)
        return torch.where(c < 0, 0x80 - c - 1, c).clamp_(max=0xFE).to(torch.uint8).masked_fill_(c == 127, 0x7E)

    def scales(n, m):
        if fmt == "ue8m0":
            return torch.randint(112, 118, (E, n // 128, m // 128), generator=gen, device=dev).to(torch.uint8)
        return (0.5 + 1.5 * torch.rand((E, n // 128, m // 128), generator=gen, device=dev)) * 2.0 ** -13

    ops = [codes(2 * I, H), scales(2 * I, H), codes(H, I), scales(H, I)]
    g = np.random.default_rng([T, E, k, H, I])
    pool = np.sort(g.choice(E, size=min(E, k + 3), replace=False))
    ids = np.stack([np.r_[pool[1], g.choice(np.delete(pool, 1), size=k - 1, replace=False)] for _ in range(T)])
    return ops, pool, ids.astype(np.int32), (g.random((T, k)) + 0.1).astype(np.float32)


@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("fmt,act", [("f32", "silu"), ("ue8m0", "gelu")])
def test_form(dev, T, E, k, H, I, fmt, act):
    ops, pool, ids, w = _draw(dev, T, E, k, H, I, fmt)
    assert not any(bool(((o & 0x7F) == 0x7F).any()) for o in (ops[0], ops[2]))
    x = workloads.activations(T, H, key=(41, 70, T, H))
    res = torch.from_numpy(np.random.default_rng(6).standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(dev)
    args = (torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), *ops)
    y = fgb.moe_ffn(to_dev_bf16(x, dev), *args, activation=act, residual=res)
    used = torch.from_numpy(pool).to(dev)
    sub = [o[used].cpu().numpy() for o in ops]
    _check(y, x, np.searchsorted(pool, ids), w, sub, fmt, act, res.float().cpu().numpy().astype(np.float64))
    # the same with pitches, in place, on a workspace that holds NaN patterns, every row written and no other
    xb = torch.full((T, H + 64), 3.0, dtype=torch.bfloat16, device=dev)
    xb[:, :H] = to_dev_bf16(x, dev)
    buf = torch.full((T + 2, H + 32), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.full((fgb.moe_ffn_workspace_bytes(T, k, E, H, I),), 0xFF, dtype=torch.uint8, device=dev)
    out = buf[1:T + 1, 8:H + 8]
    out.copy_(res)
    fgb.moe_ffn(xb[:, :H], *args, activation=act, residual=out, out=out, workspace=ws)
    assert torch.equal(out.view(torch.int16), y.view(torch.int16))
    out.fill_(7.0)
    assert bool((buf == 7.0).all())
