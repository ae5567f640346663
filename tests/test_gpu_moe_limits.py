"""GPU: NaN and infinities in the mixture-of-experts layer (fgb_moe_ffn), through every launch form: a token
with a NaN comes out as NaN and one with an infinity not finite, an expert with a NaN weight or scale reaches
the tokens that are routed to it, and every other value is, bit for bit, that of a call without them."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
import workloads
from tests.gemm_helpers import to_dev_bf16
from tests.test_gpu_moe_ffn import _routing, _weights

pytestmark = pytest.mark.gpu

# late quantization; no prep launch, whole and sliced K; the prep launch, whole and sliced K, one to four row
# tiles; sliced experts in down
FORMS = [(1, 8, 2, 512, 512), (2, 8, 4, 1024, 384), (9, 12, 3, 512, 1024), (9, 6, 3, 4096, 256), (21, 40, 6, 640, 1024),
         (7, 32, 8, 7168, 256), (40, 6, 2, 1024, 256), (40, 6, 2, 2048, 256), (24, 6, 2, 2688, 256), (64, 12, 3, 128, 2048)]
BAD = 0x7FC1  # a bf16 NaN


def _call(dev, x, ids, w, ops, res):
    y = fgb.moe_ffn(to_dev_bf16(x, dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev),
                    *[torch.from_numpy(o).to(dev) for o in ops], residual=res, out_dtype=torch.float32)
    return y.cpu()


def _inputs(dev, T, E, k, H, I, fmt):
    x = workloads.activations(T, H, key=(31, 70, T, H))
    ops = list(_weights(E, H, I, 31, fmt))
    ids, w = _routing(T, E, k, 31)
    res = torch.randn((T, H), generator=torch.Generator().manual_seed(3)).to(dev)
    return x, ids, w + np.float32(0.1), ops, res


@pytest.mark.parametrize("T,E,k,H,I", FORMS)
@pytest.mark.parametrize("bits,kind", [(BAD, "nan"), (BAD | 0x8000, "nan"), (0x7F80, "inf"), (0xFF80, "inf")])
def test_token_with_a_nan_or_infinity(dev, T, E, k, H, I, bits, kind):
    x, ids, w, ops, res = _inputs(dev, T, E, k, H, I, "f32")
    if T > 2:
        ids[2] = -1  # a token with no expert here keeps its residual, whatever its row holds
    clean = _call(dev, x, ids, w, ops, res)
    assert torch.isfinite(clean).all()
    rows = sorted({0, T // 2, T - 1} | ({2} if T > 2 else set()))
    for i, t in enumerate(rows):
        x[t, (5 + 77 * i) % H] = bits
    y = _call(dev, x, ids, w, ops, res)
    for t in range(T):
        if t not in rows or (T > 2 and t == 2):
            assert torch.equal(y[t], clean[t]), t
        elif kind == "nan":
            assert torch.isnan(y[t]).all(), t
        else:
            assert not torch.isfinite(y[t]).any(), t


@pytest.mark.parametrize("T,E,k,H,I", FORMS)
@pytest.mark.parametrize("where", ["w13 scale", "w13 code", "w2 scale", "w2 code"])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_expert_with_a_nan(dev, T, E, k, H, I, where, fmt):
    x, ids, w, ops, res = _inputs(dev, T, E, k, H, I, fmt)
    clean = _call(dev, x, ids, w, ops, res)
    e = int(ids[T // 2, 0])
    nan_scale = np.nan if fmt == "f32" else 0xFF
    cols = slice(None)
    if where == "w13 scale":
        ops[1][e, I // 128 - 1, H // 128 - 1] = nan_scale     # the last gate block
    elif where == "w13 code":
        ops[0][e, I + 3, H - 1] = 0xFF                        # an up row
    elif where == "w2 scale":
        ops[3][e, 0, I // 128 - 1] = nan_scale
        cols = slice(0, 128)
    else:
        ops[2][e, H - 2, 0] = 0x7F
        cols = slice(H - 2, H - 1)
    y = _call(dev, x, ids, w, ops, res)
    hit = torch.from_numpy((ids == e).any(axis=1))
    assert hit.any() and torch.isnan(y[hit][:, cols]).all()
    want = clean.clone()
    want[hit.nonzero(as_tuple=True)[0][:, None], torch.arange(H)[cols]] = float("nan")
    assert torch.equal(torch.isnan(y), torch.isnan(want))
    assert torch.equal(torch.nan_to_num(y), torch.nan_to_num(want))
