"""Closed forms that pin the float64 oracle of the feed-forward operators (CPU)."""
import math

import numpy as np
import pytest

from oracle import feedforward as ff


def test_activations_closed_forms():
    v = np.array([-40.0, -3.0, -1.0, 0.0, 0.5, 2.0, 40.0])
    assert np.array_equal(ff.activate(v, "none"), v)
    assert np.array_equal(ff.activate(v, "relu"), [0, 0, 0, 0, 0.5, 2, 40])
    # v Phi(v) + (-v) Phi(-v) ... gelu(v) - gelu(-v) = v; the same for silu and the tanh form
    for act in ("gelu", "silu", "gelu_tanh"):
        assert np.allclose(ff.activate(v, act) - ff.activate(-v, act), v, rtol=1e-14, atol=1e-14)
    assert ff.activate(np.array([1.0]), "gelu")[0] == pytest.approx(0.8413447460685429, rel=1e-14)  # Phi(1)
    assert ff.activate(np.array([math.log(3.0)]), "silu")[0] == pytest.approx(0.75 * math.log(3.0), rel=1e-14)
    # the tanh form is an approximation of gelu: within 5e-4 everywhere
    w = np.linspace(-6, 6, 2001)
    d = np.abs(ff.activate(w, "gelu_tanh") - ff.activate(w, "gelu"))
    assert 1e-5 < d.max() < 5e-4
    with pytest.raises(ValueError):
        ff.activate(v, "tanh")


def test_activation_slopes():
    """The slope bound that the GPU tolerance uses, by differences: at most 1.13."""
    w = np.linspace(-12, 12, 240001)
    for act in ("none", "relu", "gelu", "gelu_tanh", "silu"):
        slope = np.abs(np.diff(ff.activate(w, act)) / np.diff(w)).max()
        assert slope < 1.13, (act, slope)


def test_epilogue_order():
    s = np.array([[1.0, -2.0]])
    y = ff.epilogue_ref(s, bias=[1.0, 1.0], act="relu", residual=[[10.0, 20.0]])
    assert np.array_equal(y, [[12.0, 20.0]])  # bias inside the activation, the residual outside
    assert np.array_equal(ff.epilogue_ref(s), s)
