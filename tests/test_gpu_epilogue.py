"""GPU: the block GEMM with bias, activation and residual in its epilogue
(fgb_w8a8_block_gemm_epilogue) against the float64 oracle, through the C-ABI.

Tolerance, derived: the GEMM's sum s carries the error that its own parity tests allow,
e = 2e-3 max|s|; every activation here has a slope of at most 1.13 in magnitude (gelu's maximum), so
the value before the residual is off by at most 1.13 e plus float32 roundings of the activation (a
few 2^-24 relative, covered by a further 1e-5 max|act|); the residual adds exactly; the result is
rounded once: half a bf16 ulp, taken as one ulp.  Without bias, activation and residual the result
is the plain GEMM's, bit for bit."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
import workloads
from oracle import feedforward, gemm
from tests.gemm_helpers import bf16_tensor_to_f64, oracle_operands, ulp_bf16, upload

pytestmark = pytest.mark.gpu


def _check(y, s, want):
    """y (device) against want, the epilogue of the oracle's sum s."""
    tol = 1.13 * 2e-3 * np.max(np.abs(s)) + 1e-5 * np.max(np.abs(want))
    got = y.float().cpu().numpy().astype(np.float64)
    bound = tol + (ulp_bf16(want) if y.dtype == torch.bfloat16 else np.abs(want) * 2.0 ** -23)
    bad = np.argwhere(np.abs(got - want) > bound)
    assert bad.size == 0, (bad[:5], got[tuple(bad[0])], want[tuple(bad[0])])


def _side(M, N, dtype, seed, dev):
    g = np.random.default_rng([seed, M, N])
    bits = lambda shape: torch.from_numpy(g.standard_normal(shape).astype(np.float32)).to(dtype).to(dev)
    return bits((N,)), bits((M, N))


# every kernel of the plan: register and per-wave ring kernels (M <= 16; the ring from 48 MiB), per-wave
# ring with 32 and 64 rows, shared ring with 2, 4 and 8 waves, one slice and several, 128 rows;
# prefill K-sliced, 128 x 128, 256 x 128 and 256 x 256 tiles, ragged last rows, column splits
SHAPES = [(1, 512, 1024), (16, 1024, 2048), (5, 7168, 8192), (11, 6272, 8192), (17, 256, 512), (40, 1024, 1024),
          (20, 6144, 4096), (24, 10240, 4096), (50, 6144, 4096), (100, 2048, 1024), (128, 20480, 512),
          (65, 1152, 8320), (200, 512, 8192), (129, 128, 256), (300, 1152, 512), (257, 4096, 1024),
          (1000, 8192, 1024), (1031, 4864, 1152)]


@pytest.mark.parametrize("M,N,K", SHAPES)
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_epilogue_every_path(dev, M, N, K, fmt):
    rows = min(M, 24)  # the oracle computes a sample of rows, the last one included
    ops = oracle_operands(M, min(N, 1280), K, key=N % 97, fmt=fmt)
    aq, sa, wq, sw = ops
    if N > wq.shape[0]:  # wide layers repeat the weight's rows (whole blocks)
        reps = -(-N // wq.shape[0])
        wq, sw = np.tile(wq, (reps, 1))[:N], np.tile(sw, (reps, 1))[:N // 128]
    dops = upload(aq, sa, wq, sw, dev)
    pick = np.unique(np.concatenate([np.linspace(0, M - 1, rows).astype(int), [M - 1]]))
    s = gemm.gemm_ref_fast(aq[pick], sa[pick], wq[:1280], sw[:10], fmt)
    s = np.tile(s, (1, -(-N // s.shape[1])))[:, :N]
    bias, res = _side(M, N, torch.bfloat16, 1, dev)
    plain = fgb.gemm(*dops)
    assert torch.equal(fgb.gemm_epilogue(*dops).view(torch.int16), plain.view(torch.int16))
    y = fgb.gemm_epilogue(*dops, bias=bias, activation="silu", residual=res)
    torch.cuda.synchronize()
    want = feedforward.epilogue_ref(s, bf16_tensor_to_f64(bias), "silu", bf16_tensor_to_f64(res)[pick])
    _check(y[torch.from_numpy(pick).to(dev)], s, want)


@pytest.mark.parametrize("act", ["none", "relu", "gelu", "gelu_tanh", "silu"])
@pytest.mark.parametrize("M,N,K", [(3, 256, 256), (33, 384, 1024), (300, 1024, 1024), (260, 4096, 1024)])
def test_activations_and_types(dev, M, N, K, act):
    aq, sa, wq, sw = oracle_operands(M, N, K, key=5)
    sa = sa * np.float32(0.2)  # sums of a few units: both tails of every activation
    s = gemm.gemm_ref_fast(aq, sa, wq, sw)
    dops = upload(aq, sa, wq, sw, dev)
    for bdt, rdt, odt in [(torch.float32, torch.bfloat16, torch.bfloat16), (torch.bfloat16, torch.float32, torch.float32),
                          (None, torch.float32, torch.bfloat16), (torch.float32, None, torch.float32),
                          (torch.bfloat16, torch.bfloat16, torch.float32)]:
        bias = None if bdt is None else _side(M, N, bdt, 2, dev)[0]
        res = None if rdt is None else _side(M, N, rdt, 3, dev)[1]
        y = fgb.gemm_epilogue(*dops, bias=bias, activation=act, residual=res, out_dtype=odt)
        f64 = lambda t: None if t is None else t.float().cpu().numpy().astype(np.float64)
        assert y.dtype == odt
        _check(y, s, feedforward.epilogue_ref(s, f64(bias), act, f64(res)))


@pytest.mark.parametrize("M,N,K", [(7, 512, 512), (48, 6144, 4096), (300, 1024, 1024), (1031, 4864, 1152)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_in_place_residual_and_pitches(dev, M, N, K, dtype):
    """out = residual (y += ...), with row pitches above the row lengths: equal to the separate call,
    and nothing outside the rows is touched."""
    aq, sa, wq, sw = oracle_operands(M, min(N, 1024), K, key=9)
    if N > 1024:
        wq, sw = np.tile(wq, (-(-N // 1024), 1))[:N], np.tile(sw, (-(-N // 1024), 1))[:N // 128]
    dops = upload(aq, sa, wq, sw, dev)
    bias, res = _side(M, N, dtype, 4, dev)
    want = fgb.gemm_epilogue(*dops, bias=bias, activation="gelu_tanh", residual=res, out_dtype=dtype)
    buf = torch.full((M + 2, N + 64), 7.5, dtype=dtype, device=dev)
    view = buf[1:M + 1, 32:N + 32]
    view.copy_(res)
    got = fgb.gemm_epilogue(*dops, bias=bias, activation="gelu_tanh", residual=view, out=view)
    assert got.data_ptr() == view.data_ptr()
    assert torch.equal(view, want)
    edge = buf.clone()
    edge[1:M + 1, 32:N + 32] = 7.5
    assert bool((edge == 7.5).all())


def test_saturated_activations(dev):
    """Sums far in both tails: no NaN from the exponential, and the limits are exact."""
    M, N, K = 4, 128, 128
    aq = torch.full((M, K), 0x38, dtype=torch.uint8, device=dev)  # 1.0
    sa = torch.ones((1, 4), device=dev)
    wq = torch.full((N, K), 0x38, dtype=torch.uint8, device=dev)
    sw = torch.ones((1, 1), device=dev)
    bias = torch.full((N,), -1128.0, device=dev)  # sum + bias = -1000
    bias[::2] = 872.0                             # +1000
    for act in ("relu", "gelu", "gelu_tanh", "silu"):
        y = fgb.gemm_epilogue(aq, sa, wq, sw, bias=bias, activation=act, out_dtype=torch.float32)
        assert bool((y[:, ::2] == 1000.0).all()) and bool((y[:, 1::2] == 0.0).all()), act


def test_epilogue_on_a_side_stream_and_graph(dev):
    """On another stream than the tensors' own, and replayed from a graph with eager work between."""
    M, N, K = 40, 6144, 4096  # K-sliced: two launches through the workspace
    aq, sa, wq, sw = oracle_operands(M, 512, K, key=13)
    dops = upload(aq, sa, np.tile(wq, (12, 1)), np.tile(sw, (12, 1)), dev)
    bias, res = _side(M, N, torch.bfloat16, 6, dev)
    ws = torch.empty(fgb.gemm_workspace_bytes(M, N, K), dtype=torch.uint8, device=dev)
    out = torch.empty((M, N), dtype=torch.bfloat16, device=dev)
    run = lambda: fgb.gemm_epilogue(*dops, bias=bias, activation="silu", residual=res, out=out, workspace=ws)
    run()
    torch.cuda.synchronize()
    want = out.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out.zero_()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(out, want)
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run()
    for _ in range(3):
        out.fill_(float("nan"))
        ws.fill_(255)
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
