"""GPU: NaN, infinities and huge finite values through the epilogue of every GEMM kernel
(fgb_w8a8_block_gemm_epilogue): a NaN or an infinity of the sum or of the bias comes out as the float64
formulas give it (NaN stays NaN, +inf stays +inf, relu(-inf) = 0), and finite sums beside it are untouched.

Sums are exact here (codes +-1, scales powers of two), so finite outputs are off only by the float32
activation, 1e-5 of the value (a few 2^-24 and the gelu fit's 1e-6), and one rounding to the output type;
an absolute 1e-30 covers tails that float32 exponentials flush to 0."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
from oracle import feedforward
from tests.gemm_helpers import ulp_bf16

pytestmark = pytest.mark.gpu

INF, NAN = float("inf"), float("nan")
ROWS = [0.0, 1.0, 2.0 ** -3, NAN, INF]                                # s_a * K of row m: ROWS[m % 5]
BIAS = [0.0, NAN, INF, -INF, 3.0, -3.0, 1e30, -1e30, 17.0, -17.0, 0.5]


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
# register kernel, per-wave ring (16 and 32 rows), shared ring whole and K-sliced, prefill K-sliced, 128 x 128,
# 256 x 128 and 256 x 256 tiles
@pytest.mark.parametrize("M,N,K", [(5, 256, 256), (5, 7168, 8192), (20, 10240, 4096), (40, 1024, 1024),
                                   (24, 6144, 4096), (200, 512, 8192), (129, 128, 256), (257, 4096, 1024),
                                   (1000, 8192, 1024)])
def test_nan_and_infinities(dev, M, N, K, act):
    sums = np.array([ROWS[m % 5] for m in range(M)])
    sign = np.where(np.arange(N) % 3 == 1, -1.0, 1.0)
    aq = torch.full((M, K), 0x38, dtype=torch.uint8, device=dev)      # 1.0
    wq = torch.from_numpy(np.where(sign < 0, 0xB8, 0x38).astype(np.uint8)).to(dev)[:, None].expand(N, K).contiguous()
    sa = torch.zeros((K // 128, (M + 3) // 4 * 4), device=dev)
    sa[:, :M] = torch.from_numpy((sums / K).astype(np.float32)).to(dev)
    sw = torch.ones((N // 128, K // 128), device=dev)
    b = np.array([BIAS[n % len(BIAS)] for n in range(N)])
    bias = torch.from_numpy(b.astype(np.float32)).to(dev)
    res = torch.full((M, N), 0.25, dtype=torch.bfloat16, device=dev)
    with np.errstate(all="ignore"):
        s = sums[:, None] * sign[None, :]
        want = feedforward.epilogue_ref(s, b.astype(np.float32).astype(np.float64), act)
        assert np.isnan(want).any() and np.isinf(want).any() and np.isfinite(want).any()
        for residual, odt in ((None, torch.float32), (None, torch.bfloat16), (res, torch.bfloat16), (res, torch.float32)):
            y = fgb.gemm_epilogue(aq, sa, wq, sw, bias=bias, activation=act, residual=residual, out_dtype=odt)
            got = y.float().cpu().numpy().astype(np.float64)
            w = want if residual is None else want + 0.25
            fine = np.isfinite(w)
            assert np.array_equal(np.isnan(got), np.isnan(w)), (residual is None, odt)
            assert np.array_equal(got[np.isinf(w)], w[np.isinf(w)])
            step = ulp_bf16(w[fine]) if odt == torch.bfloat16 else np.abs(w[fine]) * 2.0 ** -23
            assert np.all(np.abs(got[fine] - w[fine]) <= 1e-5 * np.abs(want[fine]) + step + 1e-30)
