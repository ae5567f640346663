"""GPU: the router (fgb_moe_route) against the float64 oracle, through the C-ABI.

Without a selection bias the choice is a comparison of the logits as they are, so ids are equal.
Weights are float32 results of a few operations on exponentials of differences d of logits: relative
error at most (4 + |d|) 2^-23 per exponential (|d| <= 30 in these inputs), a sum of up to 1024 of
them and one division: 1e-5 relative is above every case.  With a selection bias, ids may differ
only between keys closer than their float32 rounding: 1e-5 * (1 + max |key|)."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
from oracle import feedforward as ff

pytestmark = pytest.mark.gpu


def _logits(T, E, seed, dtype, masked=0.0):
    g = np.random.default_rng([seed, T, E])
    l = torch.from_numpy((2.0 * g.standard_normal((T, E))).astype(np.float32))
    if masked:
        l[torch.from_numpy(g.random((T, E)) < masked)] = -float("inf")
    return l.to(dtype)


def _check(ids, w, l, k, **kw):
    eids, ew, _ = ff.route_ref(l.float().numpy(), k, **kw)
    assert np.array_equal(ids.cpu().numpy(), eids)
    assert np.allclose(w.cpu().numpy(), ew, rtol=1e-5, atol=0.0)


@pytest.mark.parametrize("T,E,k", [(1, 1, 1), (1, 8, 2), (3, 32, 8), (5, 63, 8), (4, 64, 32), (7, 65, 6), (64, 128, 8),
                                   (9, 129, 1), (6, 256, 8), (1025, 256, 8), (10, 257, 12), (3, 512, 32), (2, 513, 4),
                                   (5, 1024, 32), (33, 6, 6)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_route_matches_oracle(dev, T, E, k, dtype, scoring):
    for masked in (0.0, 0.4):
        l = _logits(T, E, 1, dtype, masked)
        d = l.to(dev)
        for renorm, scale in ((True, 1.0), (False, 2.5)):
            ids, w = fgb.moe_route(d, k, scoring=scoring, renormalize=renorm, scale=scale)
            assert ids.dtype == torch.int32 and w.dtype == torch.float32 and ids.shape == w.shape == (T, k)
            _check(ids, w, l, k, scoring=scoring, renormalize=renorm, scale=scale)


def test_ties_and_signed_zeros(dev):
    l = torch.zeros((4, 200))
    l[0, ::2] = -0.0             # one value: the lowest indices, in order
    l[1] = 3.0
    l[1, 64:128] = 5.0           # a tie within one register
    l[2, [199, 3, 67, 131]] = 7.0  # a tie across registers and lanes
    l[3] = torch.arange(200) // 50
    ids, w = fgb.moe_route(l.to(dev), 6)
    _check(ids, w, l, 6)
    assert ids[0].tolist() == [0, 1, 2, 3, 4, 5]


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_rows_with_few_or_no_open_experts_and_extreme_logits(dev, scoring):
    inf, low, big = float("inf"), torch.finfo(torch.float32).min, torch.finfo(torch.float32).max
    l = torch.full((9, 70), -inf)
    l[1, 69] = 4.0                        # fewer open experts than top_k
    l[2, :] = float("nan")
    l[3, [5, 66]] = torch.tensor([float("nan"), -2.0])
    l[4] = low                            # masked with the lowest value: ordinary, equal logits
    l[5] = -500.0 - torch.arange(70)      # scores below float32
    l[6] = 500.0 + torch.arange(70)
    l[7, [0, 30]] = torch.tensor([inf, 1.0])
    l[8] = torch.where(torch.arange(70) % 2 == 0, low, 0.0)
    for renorm in (True, False):
        ids, w = fgb.moe_route(l.to(dev), 5, scoring=scoring, renormalize=renorm)
        eids, ew, _ = ff.route_ref(l.numpy(), 5, scoring=scoring, renormalize=renorm)
        assert np.array_equal(ids.cpu().numpy(), eids)
        w = w.cpu().numpy()
        assert np.isfinite(w).all()
        # (scores below the smallest normal float32 may come out as 0)
        assert np.allclose(w, ew, rtol=1e-5, atol=2.0 ** -126)
        assert ids[0].tolist() == [-1] * 5 and not w[0].any() and ids[2].tolist() == [-1] * 5 and not w[2].any()


@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_selection_bias(dev, scoring):
    T, E, k = 200, 96, 6
    l = _logits(T, E, 3, torch.float32, 0.2)
    bias = torch.from_numpy(np.random.default_rng(8).standard_normal(E).astype(np.float32)) * 0.3
    bias[7] = -5.0                        # never chosen while others are open
    ids, w = fgb.moe_route(l.to(dev), k, scoring=scoring, select_bias=bias.to(dev), scale=1.5)
    eids, ew, keys = ff.route_ref(l.numpy(), k, scoring=scoring, select_bias=bias.numpy(), scale=1.5)
    ids, w = ids.cpu().numpy(), w.cpu().numpy()
    rows = np.arange(T)[:, None]
    near = 1e-5 * (1 + np.abs(keys[np.isfinite(keys)]).max())
    assert np.all(np.abs(keys[rows, ids] - keys[rows, eids]) <= near)
    same = (ids == eids).all(axis=1)
    assert same.mean() > 0.95 and np.allclose(w[same], ew[same], rtol=1e-5)
    # a bias does not enter the weights: they are those of the chosen experts' scores
    assert np.allclose(w.sum(1), 1.5, rtol=1e-5)


def test_pitch_out_buffers_and_offsets(dev):
    """Rows at an odd pitch and an odd element offset; given outputs; nothing outside them is written."""
    T, E, k = 37, 50, 4
    for dtype in (torch.bfloat16, torch.float32):
        l = _logits(T, E, 5, dtype)
        buf = torch.full((T, 2 * E + 3), 99.0, dtype=dtype, device=dev)
        view = buf[:, 1:E + 1]
        view.copy_(l)
        ids = torch.full((T + 2, k), 77, dtype=torch.int32, device=dev)
        w = torch.full((T + 2, k), 77.0, device=dev)
        got = fgb.moe_route(view, k, out=(ids[1:T + 1], w[1:T + 1]))
        assert got[0].data_ptr() == ids[1].data_ptr()
        _check(ids[1:T + 1], w[1:T + 1], l, k)
        assert (ids[[0, T + 1]] == 77).all() and (w[[0, T + 1]] == 77).all()


def test_empty_and_many_rows(dev):
    ids, w = fgb.moe_route(torch.zeros((0, 16), device=dev), 4)
    assert ids.shape == (0, 4) and w.shape == (0, 4)
    l = _logits(70001, 16, 6, torch.bfloat16)
    ids, w = fgb.moe_route(l.to(dev), 2, scoring="sigmoid")
    pick = np.r_[0:300, 69000:70001]
    _check(ids[torch.from_numpy(pick).to(dev)], w[torch.from_numpy(pick).to(dev)], l[pick], 2, scoring="sigmoid")


@pytest.mark.parametrize("E,k", [(1, 1), (7, 7), (16, 16), (17, 4), (64, 6), (65, 16), (128, 8), (130, 1), (255, 11),
                                 (256, 8), (256, 16), (256, 17)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_many_tokens_equal_few(dev, E, k, dtype):
    """Thousands of tokens in one call: rows equal, bit for bit, to those of calls of fewer tokens (the sums'
    order is the same), and to the oracle; odd counts, masked and empty rows, ties, a row pitch, garbage in the
    outputs."""
    T = 6157
    l = _logits(T, E, 7, dtype, 0.3)
    l[5::97] = -float("inf")
    l[11::89] = 0.5
    l[13::83] = float("nan")
    buf = torch.full((T, E + 3), 9.0, dtype=dtype, device=dev)
    buf[:, :E] = l.to(dev)
    d = buf[:, :E]
    bias = torch.from_numpy(np.random.default_rng(8).standard_normal(E).astype(np.float32)).to(dev)
    pick = np.r_[0:40, 3000:3040, T - 40:T]
    for scoring in ("softmax", "sigmoid"):
        for renorm, b in ((True, None), (False, None), (True, bias), (False, bias)):
            out = (torch.full((T, k), 77, dtype=torch.int32, device=dev), torch.full((T, k), float("nan"), device=dev))
            fgb.moe_route(d, k, scoring=scoring, select_bias=b, renormalize=renorm, out=out)
            for a in range(0, T, 2053):
                ids, w = fgb.moe_route(d[a:a + 2053], k, scoring=scoring, select_bias=b, renormalize=renorm)
                assert torch.equal(out[0][a:a + 2053], ids) and torch.equal(out[1][a:a + 2053], w)
            if b is None:
                at = torch.from_numpy(pick).to(dev)
                _check(out[0][at], out[1][at], l[pick], k, scoring=scoring, renormalize=renorm)
