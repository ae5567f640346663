"""GPU: the whole mixture-of-experts layer (fgb_moe_ffn) against the float64 oracle, through the C-ABI.

Tolerance, derived.  Gate and up sums are float32 sums of at most 256 scaled block sums, off by
eta <= 3e-6 of their 2-norm, so the gated product h is off by delta <= 2 eta |h|max.  Its E4M3 code then
flips to a neighbour, a step of at most |h|/8 away, with probability delta / step: the expected squared
change of the quantized row is sum(step * delta) <= |h|max eta |h|_1 / 4.  With |h|max <= 8 rms and
|h|_1 <= n rms over a group that is at most 2 eta n rms^2: 2.5e-3 of the 2-norm.  The same factor holds
for the layer's output (a linear map of h); the down products' 128-product sums add up to 1e-4 and the
bf16 rounding 2^-9.  The output's error is held to 5e-3 of the 2-norm of the experts' part, and single
elements to sixteen times its rms (few flips, one token) plus a bf16 step.  A wrong row, scale, block
or weight is an error of the order of 1, a scale an ulp off at ties of x of 1e-2."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
import workloads
from oracle import blockquant, feedforward as ff
from tests.gemm_helpers import bf16_tensor_to_f64, to_dev_bf16, ulp_bf16

pytestmark = pytest.mark.gpu


def _weights(E, H, I, seed, fmt):
    """Codes and scales of E experts (distinct blocks and scales: cheap random codes)."""
    g = np.random.default_rng([seed, E, H, I])
    codes = np.arange(256, dtype=np.uint8)
    codes = codes[(codes & 0x7F) != 0x7F]
    draw = lambda shape: codes[(g.standard_normal(shape) * 40 + 127).clip(0, codes.size - 1).astype(np.int64)]
    def scales(shape):
        if fmt == "ue8m0":
            return g.integers(112, 118, size=shape).astype(np.uint8)
        return (g.uniform(0.5, 2.0, size=shape) * 2.0 ** -13).astype(np.float32)
    return (draw((E, 2 * I, H)), scales((E, 2 * I // 128, H // 128)), draw((E, H, I)), scales((E, H // 128, I // 128)))


def _routing(T, E, k, seed, kind="random"):
    g = np.random.default_rng([seed, T, E, k])
    ids = np.stack([g.choice(E, size=k, replace=False) for _ in range(T)]).astype(np.int32)
    if kind == "one":        # every token's first choice is one expert: up to 64 rows in it
        ids[:, 0] = E - 1
        for t in range(T):   # keep the others distinct
            ids[t, 1:] = g.choice(E - 1, size=k - 1, replace=False)
    elif kind == "absent":
        ids[g.random(ids.shape) < 0.6] = -1
    return ids, g.random((T, k)).astype(np.float32)


def _check(y, x, ids, w, ops, fmt, act, residual=None):
    part = ff.moe_ffn_ref(x, ids, w, *ops, fmt=fmt, act=act)
    want = part if residual is None else part + residual
    got = y.float().cpu().numpy().astype(np.float64)
    assert np.isfinite(got).all()
    err = np.abs(got - want)
    ulp = ulp_bf16(want) if y.dtype == torch.bfloat16 else np.abs(want) * 2.0 ** -23
    rms = np.sqrt(np.mean(part ** 2))
    assert np.linalg.norm(got - want) <= 5e-3 * np.linalg.norm(part) + np.linalg.norm(ulp), \
        np.linalg.norm(got - want) / np.linalg.norm(part)
    assert np.all(err <= 16 * 5e-3 * np.maximum(np.abs(part), rms) + ulp)


def _run(dev, T, E, k, H, I, fmt="f32", act="silu", kind="random", seed=0, **kw):
    x = workloads.activations(T, H, key=(seed, 70, T, H))
    ops = _weights(E, H, I, seed, fmt)
    ids, w = _routing(T, E, k, seed, kind)
    dops = [torch.from_numpy(o).to(dev) for o in ops]
    y = fgb.moe_ffn(to_dev_bf16(x, dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), *dops,
                    activation=act, **kw)
    return y, x, ids, w, ops, dops


SHAPES = [(1, 1, 1, 128, 128), (1, 8, 2, 256, 384), (1, 32, 8, 1024, 512), (2, 4, 2, 128, 1152), (3, 16, 16, 384, 256),
          (7, 32, 8, 1024, 256), (16, 8, 2, 512, 512), (17, 3, 1, 256, 256), (33, 5, 2, 640, 384), (64, 32, 8, 512, 256),
          (64, 64, 16, 256, 128), (49, 1, 1, 256, 512), (64, 300, 4, 128, 128), (5, 1024, 3, 128, 128),
          (9, 6, 3, 4096, 256), (20, 6, 3, 2048, 256), (4, 8, 8, 1024, 1152), (16, 8, 1, 128, 256), (3, 70, 24, 256, 128),
          (40, 2, 1, 2048, 256), (16, 3, 2, 2048, 256), (24, 2, 2, 2432, 128), (1, 4, 1, 2048, 384),
          (8, 16, 4, 256, 1024), (50, 12, 3, 128, 2048), (1, 16, 16, 256, 2048), (3, 40, 8, 2304, 1152),
          (2, 2, 1, 8320, 128), (2, 2, 2, 128, 9600), (1, 1, 1, 32768, 128), (1, 1, 1, 128, 32768),
          (16, 6, 3, 2560, 384), (15, 32, 2, 2688, 512), (17, 32, 4, 2048, 512), (30, 3, 2, 2176, 256), (31, 3, 2, 2176, 256),
          (12, 8, 3, 4096, 2048)]


@pytest.mark.parametrize("T,E,k,H,I", SHAPES)
@pytest.mark.parametrize("fmt", ["f32", "ue8m0"])
def test_moe_matches_oracle(dev, T, E, k, H, I, fmt):
    y, x, ids, w, ops, _ = _run(dev, T, E, k, H, I, fmt, seed=1)
    assert y.dtype == torch.bfloat16 and y.shape == (T, H)
    _check(y, x, ids, w, ops, fmt, "silu")


@pytest.mark.parametrize("T", [15, 16, 17, 31, 32, 33, 48, 49, 63, 64])
@pytest.mark.parametrize("H", [384, 2304])
def test_one_popular_expert(dev, T, H):
    """All tokens in one expert: one to four activation tiles, the last one full or ragged; short rows
    (quantized where they are used) and longer ones (by the launch before)."""
    y, x, ids, w, ops, _ = _run(dev, T, 5, 2, H, 256, kind="one", seed=2)
    _check(y, x, ids, w, ops, "f32", "silu")


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh"])
@pytest.mark.parametrize("rdt,odt", [(torch.bfloat16, torch.bfloat16), (torch.float32, torch.float32),
                                     (torch.float32, torch.bfloat16), (None, torch.float32)])
def test_activations_and_residual_types(dev, act, rdt, odt):
    T, E, k, H, I = 9, 6, 2, 512, 256
    res = None
    if rdt is not None:
        res = torch.from_numpy(np.random.default_rng(4).standard_normal((T, H)).astype(np.float32)).to(rdt).to(dev)
    y, x, ids, w, ops, _ = _run(dev, T, E, k, H, I, act=act, seed=3, residual=res, out_dtype=odt)
    assert y.dtype == odt
    _check(y, x, ids, w, ops, "f32", act, None if res is None else res.float().cpu().numpy().astype(np.float64))


def test_absent_experts_repeats_and_empty_tokens(dev):
    """Ids outside 0 .. E-1 are skipped, a repeated id counts with the sum of its weights, a token with
    no expert here gets its residual (or zero)."""
    T, E, k, H, I = 40, 6, 4, 256, 256
    x = workloads.activations(T, H, key=(4, 70, T, H))
    ops = _weights(E, H, I, 4, "f32")
    g = np.random.default_rng(4)
    ids = g.integers(-2, E + 2, size=(T, k)).astype(np.int32)   # repeats within rows, -2, -1, E, E + 1
    ids[3] = -1
    ids[4] = [2 ** 31 - 1, -2 ** 31, E, -1]
    ids[5] = 2                                                  # one expert four times
    ids[6] = [1, 5, 1, 5]
    w = g.random((T, k)).astype(np.float32)
    res = g.standard_normal((T, H)).astype(np.float32)
    dops = [torch.from_numpy(o).to(dev) for o in ops]
    args = (to_dev_bf16(x, dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), *dops)
    rd = torch.from_numpy(res).to(dev)
    y = fgb.moe_ffn(*args, residual=rd, out_dtype=torch.float32)
    _check(y, x, ids, w, ops, "f32", "silu", res.astype(np.float64))
    assert torch.equal(y[3:5], rd[3:5])
    z = fgb.moe_ffn(*args)
    assert not z[3:5].any()
    none = fgb.moe_ffn(args[0], torch.full((T, k), -1, dtype=torch.int32, device=dev), *args[2:], residual=rd,
                       out_dtype=torch.float32)
    assert torch.equal(none, rd)


def test_zero_rows_and_zero_weights(dev):
    T, E, k, H, I = 4, 3, 2, 256, 256
    x = workloads.activations(T, H, key=(5, 70, T, H))
    x[1] = 0                       # a zero row: zero scales, zero codes
    x[2, :128] = 0x8000            # a group of -0
    ops = list(_weights(E, H, I, 5, "f32"))
    ops[0][1, :I] = 0              # an expert whose gate is zero: h = 0, zero scale
    ids = np.array([[0, 1], [1, 2], [0, 2], [1, 0]], dtype=np.int32)
    w = np.array([[1, 2], [3, 4], [0, 0], [0.5, -1]], dtype=np.float32)
    y = fgb.moe_ffn(to_dev_bf16(x, dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev),
                    *[torch.from_numpy(o).to(dev) for o in ops], out_dtype=torch.float32)
    _check(y, x, ids, w, ops, "f32", "silu")
    assert not y[1].any() and not y[2].any()


@pytest.mark.parametrize("T,E,k,H,I", [(21, 7, 3, 384, 256), (21, 12, 4, 256, 1280), (37, 3, 2, 2176, 256),
                                       (1, 8, 8, 1024, 1024), (5, 8, 2, 4096, 256)])
def test_pitches_in_place_and_workspace_contents(dev, T, E, k, H, I):
    """x, residual and out with row pitches above the row length, out = residual, a workspace that holds
    NaN patterns: equal, bit for bit, to the plain call, twice, and nothing outside out's rows is written."""
    g = np.random.default_rng(6)
    res = torch.from_numpy(g.standard_normal((T, H)).astype(np.float32)).to(torch.bfloat16).to(dev)
    y, x, ids, w, ops, dops = _run(dev, T, E, k, H, I, seed=6, residual=res)
    xb = torch.full((T, H + 64), 3.0, dtype=torch.bfloat16, device=dev)
    xb[:, :H] = to_dev_bf16(x, dev)
    buf = torch.full((T + 2, H + 32), 7.0, dtype=torch.bfloat16, device=dev)
    ws = torch.full((fgb.moe_ffn_workspace_bytes(T, k, E, H, I),), 0xFF, dtype=torch.uint8, device=dev)
    for _ in range(2):
        out = buf[1:T + 1, 8:H + 8]
        out.copy_(res)
        fgb.moe_ffn(xb[:, :H], torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev), *dops, residual=out, out=out,
                    workspace=ws)
        assert torch.equal(out.view(torch.int16), y.view(torch.int16))
        ws.fill_(0x7F)
    out.fill_(7.0)
    assert bool((buf == 7.0).all())


def test_no_tokens(dev):
    dops = [torch.from_numpy(o).to(dev) for o in _weights(2, 128, 128, 7, "f32")]
    y = fgb.moe_ffn(torch.empty((0, 128), dtype=torch.bfloat16, device=dev),
                    torch.empty((0, 2), dtype=torch.int32, device=dev), torch.empty((0, 2), device=dev), *dops)
    assert y.shape == (0, 128)


def test_router_into_layer_on_a_side_stream_and_in_a_graph(dev):
    """moe_route's result goes straight into moe_ffn; on another stream, and replayed from a graph with
    changed inputs and eager work between the replays."""
    T, E, k, H, I = 12, 16, 4, 512, 256
    x = to_dev_bf16(workloads.activations(T, H, key=(8, 70, T, H)), dev)
    dops = [torch.from_numpy(o).to(dev) for o in _weights(E, H, I, 8, "ue8m0")]
    logits = torch.randn((T, E), generator=torch.Generator().manual_seed(3)).to(dev)
    ws = torch.empty(fgb.moe_ffn_workspace_bytes(T, k, E, H, I), dtype=torch.uint8, device=dev)
    ids = torch.empty((T, k), dtype=torch.int32, device=dev)
    w = torch.empty((T, k), device=dev)
    y = torch.empty((T, H), dtype=torch.bfloat16, device=dev)

    def run(out):
        fgb.moe_route(logits, k, out=(ids, w))
        return fgb.moe_ffn(x, ids, w, *dops, residual=x, out=out, workspace=ws)

    want = [run(torch.empty_like(y)).clone()]
    first = logits.clone()
    logits.neg_()
    want.append(run(torch.empty_like(y)).clone())
    torch.cuda.synchronize()
    assert not torch.equal(want[0], want[1])
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        run(y)
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    assert torch.equal(y, want[1])
    g = torch.cuda.CUDAGraph()
    with torch.cuda.graph(g):
        run(y)
    for i in range(4):
        logits.copy_(first if i % 2 == 0 else -first)
        y.fill_(float("nan"))
        run(torch.empty_like(y))  # eager work between, on the same workspace
        torch.cuda.synchronize()
        g.replay()
        torch.cuda.synchronize()
        assert torch.equal(y, want[i % 2]), i


def test_large_layer_sampled(dev):
    """A layer of the MoE workload's size, 64 tokens: every token's row against the oracle on a sample of
    output columns (full intermediate)."""
    T, E, k, H, I = 64, 4, 2, 7168, 2048
    x = workloads.activations(T, H, key=(9, 70, T, H))
    ops = _weights(E, H, I, 9, "f32")
    ids, w = _routing(T, E, k, 9)
    y = fgb.moe_ffn(to_dev_bf16(x, dev), torch.from_numpy(ids).to(dev), torch.from_numpy(w).to(dev),
                    *[torch.from_numpy(o).to(dev) for o in ops])
    cols = np.r_[0:128, 3584:3712, 7040:7168]
    rows = np.unique(np.r_[0:8, 30:34, 60:64])
    sub = (ops[0], ops[1], ops[2][:, cols], ops[3][:, np.unique(cols // 128)])
    _check(y[torch.from_numpy(rows).to(dev)][:, torch.from_numpy(cols).to(dev)], x[rows], ids[rows], w[rows], sub, "f32", "silu")
