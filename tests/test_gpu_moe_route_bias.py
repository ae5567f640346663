"""GPU: NaN and infinities in the router's selection bias, few tokens and thousands, and its CPU oracle."""
import numpy as np
import pytest
import torch

import fine_grained_block_amd as fgb
from oracle import feedforward as ff

NAN, INF = float("nan"), float("inf")


def test_oracle_nan_bias():
    l = np.array([[0.0, 1.0, 2.0, 3.0], [-np.inf, -np.inf, 5.0, -np.inf]])
    ids, w, _ = ff.route_ref(l, 2, "sigmoid", select_bias=[NAN, 0.0, NAN, -INF], renormalize=False)
    assert ids.tolist() == [[1, 3], [-1, -1]] and np.allclose(w[0], 1 / (1 + np.exp([-1.0, -3.0]))) and not w[1].any()


@pytest.mark.gpu
@pytest.mark.parametrize("T", [1, 5, 6200])
@pytest.mark.parametrize("E,k", [(8, 3), (70, 6), (256, 8), (300, 4)])
@pytest.mark.parametrize("scoring", ["softmax", "sigmoid"])
def test_bias_nan_and_infinities(dev, T, E, k, scoring):
    """An expert with a NaN bias (either sign) is never selected, +inf comes first (the lowest index of two),
    -inf last; the weights are the scores, which no bias enters (the softmax keeps those experts' shares)."""
    g = np.random.default_rng([T, E])
    # selection keys a whole step apart, so that the float32 rounding of score + bias decides nothing
    l = torch.from_numpy(g.standard_normal((T, E)).astype(np.float32))
    bias = torch.from_numpy(2.0 * g.permutation(E).astype(np.float32))
    bias[1], bias[E - 1], bias[3], bias[6], bias[5] = NAN, -NAN, INF, INF, -INF
    ids, w = fgb.moe_route(l.to(dev), k, scoring=scoring, select_bias=bias.to(dev), renormalize=False)
    eids, ew, _ = ff.route_ref(l.numpy(), k, scoring=scoring, select_bias=bias.numpy(), renormalize=False)
    assert np.array_equal(ids.cpu().numpy(), eids)
    assert (eids[:, :2] == [3, 6]).all() and not np.isin(eids, [1, E - 1]).any()
    assert np.allclose(w.cpu().numpy(), ew, rtol=1e-5, atol=2.0 ** -126)
    none = torch.full((E,), NAN, device=dev)
    ids, w = fgb.moe_route(l.to(dev), k, scoring=scoring, select_bias=none)
    assert (ids == -1).all() and not w.any()
