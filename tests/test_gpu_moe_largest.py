"""GPU: the mixture-of-experts layer at its largest validated sizes (H = I = 32768, 2 GiB of gate and up codes
per expert: offsets past 31 bits within an expert and past 32 between experts).

The reference is the definition in torch operations on the GPU, weights widened 1024 rows at a time, products in
float64.  Tolerance: that of tests/test_gpu_moe_ffn.py, derived there (5e-3 of the 2-norm, and the rounding to
bf16, 2^-9)."""
import pytest
import torch

import fine_grained_block_amd as fgb

pytestmark = pytest.mark.gpu

N = 32768


def _quantized(v):
    """The values that the layer's 1x128-group codes of v stand for (scales amax * fl32(1 / 448))."""
    g = v.float().unflatten(-1, (-1, 128))
    s = g.abs().amax(-1, keepdim=True) * torch.tensor(1 / 448, dtype=torch.float32, device=v.device)
    q = (g / torch.where(s == 0, torch.ones_like(s), s)).clamp(-448, 448).to(torch.float8_e4m3fn)
    return (q.double() * s.double()).flatten(-2)


def _product(a, q, s):
    """a [T, K] float64 times the transpose of codes q [R, K] with block scales s [R / 128, K / 128]."""
    out = []
    for r in range(0, q.shape[0], 1024):
        w = q[r:r + 1024].view(torch.float8_e4m3fn).double()
        w = w * s[r // 128:r // 128 + 8].double().repeat_interleave(128, 0).repeat_interleave(128, 1)
        out.append(torch.mm(w, a.t().contiguous()).t())
    return torch.cat(out, 1)


@pytest.mark.parametrize("T", [1, 20, 64])
def test_largest_layer(dev, T):
    E, k = 2, 2
    gen = torch.Generator(device=dev)
    gen.manual_seed(T)

    def codes(*shape):  # finite: no 0x7F, no 0xFF
        q = torch.randint(0, 256, shape, generator=gen, device=dev, dtype=torch.uint8)
        return q.clamp_(max=0xFE).masked_fill_(q == 0x7F, 0x7E)

    scale = lambda *shape: (0.5 + torch.rand(shape, generator=gen, device=dev)) * 2.0 ** -16
    w13, s13 = codes(E, 2 * N, N), scale(E, 2 * N // 128, N // 128)
    w2, s2 = codes(E, N, N), scale(E, N // 128, N // 128)
    x = torch.randn((T, N), generator=gen, device=dev).to(torch.bfloat16)
    ids = torch.tensor([[1, -1], [0, 1], [1, 0], [0, -1]], dtype=torch.int32, device=dev).repeat(T // 4 + 1, 1)[:T].contiguous()
    w = torch.rand((T, k), generator=gen, device=dev) + 0.1
    y = fgb.moe_ffn(x, ids, w, w13, s13, w2, s2)
    xq, want = _quantized(x), torch.zeros((T, N), dtype=torch.float64, device=dev)
    for e in range(E):
        t, j = torch.nonzero(ids == e, as_tuple=True)
        if t.numel():
            gate, up = _product(xq[t], w13[e], s13[e]).split(N, 1)
            h = _quantized((gate * torch.sigmoid(gate) * up).float())
            want.index_add_(0, t, _product(h, w2[e], s2[e]) * w[t, j].double()[:, None])
    assert torch.isfinite(y).all() and want.norm() > 0
    err = (y.double() - want).norm(dim=1) / want.norm(dim=1)
    assert bool((err <= 5e-3 + 2.0 ** -9).all()), err.max()
    # every block of columns is in place
    part = (y.double() - want).unflatten(1, (-1, 128)).norm(dim=2) / want.unflatten(1, (-1, 128)).norm(dim=2)
    assert bool((part <= 4 * (5e-3 + 2.0 ** -9)).all()), part.max()
