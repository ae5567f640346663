"""GPU: the epilogue GEMM with more than 2^31 outputs: element offsets of output and residual past 31 bits, on
the 256 x 256 and 256 x 128 tiles and the 128 x 128 ones, against the plain GEMM, bit for bit (the float32 sum,
relu and the residual's addition are exact up to their own roundings)."""
import pytest
import torch

import fine_grained_block_amd as fgb

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(66001, 33024, 1024), (66001, 33024, 256), (66001, 32896, 128)])
def test_more_than_31_bits_of_outputs(dev, M, N, K):
    assert M * N > 1 << 31
    gen = torch.Generator(device=dev)
    gen.manual_seed(K)
    q, s = fgb.quantize(torch.randn((M, K), generator=gen, device=dev).to(torch.bfloat16))
    w, sw = fgb.quantize_weight(torch.randn((N, K), generator=gen, device=dev).to(torch.bfloat16))
    plain = fgb.gemm(q, s, w, sw, out_dtype=torch.float32)
    wide = torch.randn((M, N + 64), generator=gen, device=dev, dtype=torch.bfloat16)
    res = wide[:, 32:N + 32]
    y = fgb.gemm_epilogue(q, s, w, sw, activation="relu", residual=res)
    z = fgb.gemm_epilogue(q, s, w, sw, activation="relu")
    fgb.gemm_epilogue(q, s, w, sw, activation="relu", residual=res, out=res)
    for a in range(0, M, 8192):
        part = torch.relu(plain[a:a + 8192])
        assert torch.equal(z[a:a + 8192], part.to(torch.bfloat16)), a
        assert torch.equal(y[a:a + 8192], res[a:a + 8192]), a
    del z, plain
    wide = torch.randn((M, N + 64), generator=gen.manual_seed(K + 1), device=dev, dtype=torch.bfloat16)
    y2 = fgb.gemm_epilogue(q, s, w, sw, residual=wide[:, 32:N + 32], out_dtype=torch.float32)
    plain = fgb.gemm(q, s, w, sw, out_dtype=torch.float32)
    for a in range(0, M, 8192):
        assert torch.equal(y2[a:a + 8192], plain[a:a + 8192] + wide[a:a + 8192, 32:N + 32].float()), a
