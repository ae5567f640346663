"""GPU: the epilogue GEMM at the sizes where the plain GEMM walks several tiles per workgroup (more 256 x 256
tiles than CUs, K of 8 to 16 blocks): with nothing to apply the result is the plain GEMM's bit for bit, and
with an epilogue it is the epilogue, in float32, of the plain GEMM's float32 result, bit for bit where that
is exact (bias, relu, residual), ragged last rows and columns of narrower tiles included."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
from tests.gemm_helpers import oracle_operands, upload

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("M,N,K", [(4500, 8192, 1280), (8000, 4352, 2048), (8192, 8448, 1536), (1700, 24576, 1536), (2200, 16384, 1024)])
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_equal_to_the_plain_gemm(dev, M, N, K, fmt):
    aq, sa, wq, sw = oracle_operands(512, 512, K, key=N % 89, fmt=fmt)
    rm, rn = -(-M // 512), -(-N // 512)
    g = np.random.default_rng([M, N])
    # rows and columns repeat in an order of their own, so that no two tiles are alike
    pm, pn = np.tile(np.arange(512), rm)[g.permutation(512 * rm)][:M], np.tile(np.arange(4), rn)[g.permutation(4 * rn)][:N // 128]
    wq = wq.reshape(4, 128, K)[pn].reshape(N, K)
    dops = upload(aq[pm], sa[pm], wq, sw[pn], dev)
    plain, plain32 = fgb.gemm(*dops), fgb.gemm(*dops, out_dtype=torch.float32)
    assert torch.equal(plain.view(torch.int16), plain32.to(torch.bfloat16).view(torch.int16))
    assert torch.equal(fgb.gemm_epilogue(*dops).view(torch.int16), plain.view(torch.int16))
    bias = torch.from_numpy(g.standard_normal(N).astype(np.float32)).to(dev)
    res = torch.from_numpy(g.standard_normal((M, N)).astype(np.float32)).to(torch.bfloat16).to(dev)
    want = plain32 + bias
    assert torch.equal(fgb.gemm_epilogue(*dops, bias=bias), want.to(torch.bfloat16))
    want = torch.relu(want) + res.float()
    assert torch.equal(fgb.gemm_epilogue(*dops, bias=bias, activation="relu", residual=res), want.to(torch.bfloat16))
    assert torch.equal(fgb.gemm_epilogue(*dops, bias=bias, activation="relu", residual=res, out_dtype=torch.float32), want)
    out = res.clone()
    fgb.gemm_epilogue(*dops, bias=bias, activation="relu", residual=out, out=out)
    assert torch.equal(out, want.to(torch.bfloat16))
