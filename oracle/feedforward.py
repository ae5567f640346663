"""Reference of the operators around the block GEMM (test infrastructure, CPU, float64): the GEMM's
epilogue (bias, activation, residual), the router of a mixture of experts, and the whole
mixture-of-experts layer on FP8 block weights (the expert matmuls of Transformers "Fine-grained
FP8", "DeepGEMM fast path").

Parity unpinned: the pages print no values for these; the definitions below are pinned by closed
forms in tests/test_oracle_feedforward.py.
"""
from __future__ import annotations

import math

import numpy as np

from . import blockquant, fp8, gemm

_erfc = np.vectorize(math.erfc, otypes=[np.float64])


def activate(v, act: str) -> np.ndarray:
    """act(v) in float64: none, relu, gelu (v Phi(v)), gelu_tanh (its tanh form), silu (v sigmoid(v))."""
    v = np.asarray(v, dtype=np.float64)
    if act == "none":
        return v
    if act == "relu":
        return np.maximum(v, 0.0)
    if act == "gelu":
        return 0.5 * v * _erfc(-v / math.sqrt(2.0)) if v.size else v
    if act == "gelu_tanh":
        return 0.5 * v * (1.0 + np.tanh(math.sqrt(2.0 / math.pi) * (v + 0.044715 * v ** 3)))
    if act == "silu":
        with np.errstate(over="ignore"):
            return v / (1.0 + np.exp(-v))
    raise ValueError("unknown activation")


def epilogue_ref(s, bias=None, act: str = "none", residual=None) -> np.ndarray:
    """act(s + bias) + residual in float64, s the GEMM's float64 result."""
    y = np.asarray(s, dtype=np.float64)
    if bias is not None:
        y = y + np.asarray(bias, dtype=np.float64)[None, :]
    y = activate(y, act)
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)


def route_ref(logits, top_k: int, scoring: str = "softmax", select_bias=None, renormalize: bool = True,
              scale: float = 1.0):
    """Top-k experts of every row and their weights in float64.

    Keys are the logits, or score + select_bias; ties go to the lowest index; experts at -inf (or NaN)
    are never selected and have no share, experts with a NaN bias are never selected.  Returns (ids int32 [T, k], weights float64 [T, k], keys
    float64 [T, E] with -inf for masked experts)."""
    l = np.asarray(logits, dtype=np.float64)
    l = np.where(np.isnan(l), -np.inf, np.minimum(l, np.finfo(np.float32).max))
    T, E = l.shape
    ids = np.full((T, top_k), -1, dtype=np.int32)
    weights = np.zeros((T, top_k), dtype=np.float64)
    keys = np.full((T, E), -np.inf)
    for t in range(T):
        open_ = np.nonzero(l[t] > -np.inf)[0]
        if open_.size == 0:
            continue
        v = l[t, open_]
        if scoring == "softmax":
            logp = v - v.max()
            logp = logp - math.log(np.exp(logp).sum())
        else:  # log sigmoid(v)
            logp = np.minimum(v, 0.0) - np.log1p(np.exp(-np.abs(v)))
        key = v if select_bias is None else np.exp(logp) + np.asarray(select_bias, dtype=np.float64)[open_]
        there = ~np.isnan(key)
        if not there.any():
            continue
        open_, logp, key = open_[there], logp[there], key[there]
        keys[t, open_] = key
        order = np.lexsort((open_, -key))[:top_k]
        lp = logp[order]
        w = np.exp(lp - lp.max()) / np.exp(lp - lp.max()).sum() if renormalize else np.exp(lp)
        ids[t, :order.size] = open_[order]
        weights[t, :order.size] = w * scale
    return ids, weights, keys


def layer_quant(x):
    """The layer's quantization of bf16 rows: s = fl32(amax * fl32(1 / 448)), codes E4M3(fl32(x / s))
    (the activation quantizer divides amax by 448: scales an ulp apart, hence other codes at ties)."""
    xf = blockquant._as_f32(x)
    g = xf.reshape(xf.shape[0], -1, blockquant.GROUP)
    s = (np.abs(g).max(axis=2) * (np.float32(1.0) / np.float32(448.0))).astype(np.float32)
    return blockquant._quantize_groups(g, s).reshape(xf.shape), s


def group_quant_f64(v):
    """The values that the 1x128-group E4M3 quantization of float64 rows stands for (scales and
    quotients in float64)."""
    v = np.asarray(v, dtype=np.float64)
    g = v.reshape(v.shape[0], -1, blockquant.GROUP)
    s = np.abs(g).max(axis=2, keepdims=True) / 448.0
    q = fp8.dec_e4m3(fp8.enc_e4m3_sat(np.where(s > 0, g / np.where(s > 0, s, 1.0), 0.0)))
    return (q * s).reshape(v.shape)


def moe_ffn_ref(x, ids, weights, w13_q, s_w13, w2_q, s_w2, fmt: str = "f32", act: str = "silu", residual=None):
    """The whole mixture-of-experts layer in float64: x bf16 bits [T, H]; ids int [T, k] (outside
    0 .. E-1: skipped); weights [T, k]; w13_q [E, 2I, H] (gate rows, then up rows); w2_q [E, H, I]."""
    T, E, I = x.shape[0], w2_q.shape[0], w2_q.shape[2]
    xq, xs = layer_quant(x)
    y = np.zeros((T, w2_q.shape[1]), dtype=np.float64)
    ids, weights = np.asarray(ids), np.asarray(weights, dtype=np.float64)
    for e in range(E):
        rows = np.nonzero((ids == e).any(axis=1))[0]
        if rows.size == 0:
            continue
        gu = gemm.gemm_ref_fast(xq[rows], xs[rows], w13_q[e], s_w13[e], fmt)
        h = group_quant_f64(activate(gu[:, :I], act) * gu[:, I:])
        sw = np.repeat(np.repeat(gemm._w_scales(s_w2[e], fmt), 128, axis=0), 128, axis=1)
        o = h @ (fp8.dec_e4m3(w2_q[e]) * sw).T
        y[rows] += o * np.where(ids[rows] == e, weights[rows], 0.0).sum(axis=1)[:, None]
    return y if residual is None else y + np.asarray(residual, dtype=np.float64)
