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
