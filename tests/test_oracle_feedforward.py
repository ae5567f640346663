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


def test_route_closed_forms():
    l = np.array([[0.0, math.log(2.0), math.log(5.0), -np.inf], [1.0, 1.0, 1.0, 1.0], [-np.inf] * 4,
                  [np.nan, -np.inf, 3.0, -np.inf]])
    ids, w, _ = ff.route_ref(l, 2, "softmax", renormalize=False)
    assert ids.tolist() == [[2, 1], [0, 1], [-1, -1], [2, -1]]  # ties: the lowest index; masked rows end in -1
    assert np.allclose(w, [[5 / 8, 2 / 8], [0.25, 0.25], [0, 0], [1, 0]])
    _, w, _ = ff.route_ref(l, 2, "softmax", renormalize=True, scale=2.5)
    assert np.allclose(w[0], [2.5 * 5 / 7, 2.5 * 2 / 7])
    # a selection bias moves the choice and not the weights
    ids, w, _ = ff.route_ref(l, 2, "sigmoid", select_bias=[10.0, 0, 0, 0], renormalize=False)
    assert ids[0].tolist() == [0, 2] and np.allclose(w[0], [0.5, 5 / 6])
    # scores far below the smallest double keep their ratios: e^-800 / (e^-800 + e^-801)
    _, w, _ = ff.route_ref(np.array([[-800.0, -801.0]]), 2, "sigmoid")
    assert np.allclose(w, [[1 / (1 + math.exp(-1)), 1 / (1 + math.exp(1))]])


def test_group_quant_f64_matches_the_quantizer_on_its_inputs():
    """On bf16 rows whose scale is exact (group maximum 448 * 2^k) both quantizers agree exactly."""
    from oracle import blockquant, fp8
    import workloads
    x = np.random.default_rng(5).integers(-448, 449, size=(6, 256)).astype(np.float32)
    x[:, ::128] = 448.0
    x[1] *= np.float32(2.0 ** -5)
    x[2, :128] = 0.0
    bits = workloads.f32_to_bf16_bits(x)
    q, s = blockquant.act_quant(bits)
    want = fp8.dec_e4m3(q) * np.repeat(s.astype(np.float64), 128, axis=1)
    assert np.array_equal(ff.group_quant_f64(workloads.bf16_bits_to_f32(bits).astype(np.float64)), want)


def test_layer_quant_scale():
    """The layer's scale: a float32 product with fl32(1/448); codes equal to the activation quantizer's
    except where the scales differ."""
    from oracle import blockquant
    import workloads
    bits = workloads.activations(64, 1024, key=(5, 1, 2, 3))
    q, s = ff.layer_quant(bits)
    q2, s2 = blockquant.act_quant(bits)
    ulp = np.spacing(s2)
    assert np.all(np.abs(s - s2) <= ulp) and 0.1 < np.mean(s != s2) < 0.9
    same = np.repeat(s == s2, 128, axis=1)
    assert np.array_equal(q[same], q2[same])
    zero = np.zeros((1, 128), dtype=np.uint16)
    zero[0, 3] = 0x8000
    q, s = ff.layer_quant(zero)
    assert s[0, 0] == 0 and q[0, 3] == 0x80 and not q[0, [0, 1, 2, 4]].any()


def test_moe_closed_form():
    """One-hot weights and values the codes hold exactly: gate = x0, up = x1, h = relu-like branch of gelu."""
    from oracle import fp8
    import workloads
    H = I = 128
    x = np.zeros((2, H), dtype=np.float32)
    x[0, :2] = [448.0, 7.0]
    x[1, :2] = [448.0, 14.0]
    one = int(fp8.enc_e4m3_sat(np.array([1.0]))[0])
    w13 = np.zeros((3, 2 * I, H), dtype=np.uint8)
    w13[:, 0, 0] = one       # gate[0] = x[0]
    w13[:, I, 1] = one       # up[0] = x[1]
    w2 = np.zeros((3, H, I), dtype=np.uint8)
    w2[:, 5, 0] = one        # y[5] = h[0]
    s13, s2 = np.ones((3, 2, 1), np.float32), np.ones((3, 1, 1), np.float32)
    s2[1] = 2.0
    ids = np.array([[0, 1], [1, -1]])
    w = np.array([[0.5, 0.25], [1.0, 9.0]])
    y = ff.moe_ffn_ref(workloads.f32_to_bf16_bits(x), ids, w, w13, s13, w2, s2, act="gelu", residual=np.ones((2, H)))
    want = np.ones((2, H))
    want[0, 5] += 448 * 7 * (0.5 + 0.25 * 2)
    want[1, 5] += 448 * 14 * 2
    assert np.allclose(y, want, rtol=1e-14)
    # an expert named twice counts with the sum of its weights
    y2 = ff.moe_ffn_ref(workloads.f32_to_bf16_bits(x), np.array([[0, 0], [7, -1]]), w, w13, s13, w2, s2, act="gelu")
    assert np.allclose(y2[0, 5], 448 * 7 * 0.75) and not y2[1].any()
