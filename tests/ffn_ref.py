"""Plain 64-bit definitions of the gated projection, its gradients, the 8-bit
quantisation and the 8-bit product, for the tests."""

import math

import numpy as np

_erf = np.vectorize(math.erf, otypes=[np.float64])
erfc = np.vectorize(math.erfc, otypes=[np.float64])
C = math.sqrt(2 / math.pi)
ACTS = ("silu", "gelu", "gelu_tanh", "relu")


def _sigmoid(v):
    e = np.exp(-np.abs(v))
    return np.where(v >= 0, 1, e) / (1 + e)


def act(name, v):
    if name == "silu":
        return v * _sigmoid(v)
    if name == "gelu":
        return 0.5 * v * (1 + _erf(v / math.sqrt(2)))
    if name == "gelu_tanh":
        return 0.5 * v * (1 + np.tanh(C * (v + 0.044715 * v ** 3)))
    return np.maximum(v, 0)


def slope(name, v):
    if name == "silu":
        s = _sigmoid(v)
        return s * (1 + v * (1 - s))
    if name == "gelu":
        return 0.5 * (1 + _erf(v / math.sqrt(2))) + v * np.exp(-0.5 * v * v) / math.sqrt(2 * math.pi)
    if name == "gelu_tanh":
        t = np.tanh(C * (v + 0.044715 * v ** 3))
        return 0.5 * (1 + t) + 0.5 * v * (1 - t * t) * C * (1 + 3 * 0.044715 * v * v)
    return (v > 0).astype(np.float64)


def forward(name, x, wg, wu):
    """h, gate, up."""
    g, u = x @ wg.T, x @ wu.T
    return act(name, g) * u, g, u


def backward(name, x, wg, wu, g, u, d_h):
    """d_x, d_w_gate, d_w_up, d_gate, d_up."""
    dg, du = d_h * u * slope(name, g), d_h * act(name, g)
    return dg @ wg + du @ wu, dg.T @ x, du.T @ x, dg, du


def quantize(x):
    """codes and f32 scales of rows whose values are exact in f32."""
    most = np.abs(x).max(axis=1) if x.shape[1] else np.zeros(x.shape[0])
    fine = np.isfinite(most)
    scale = np.where(fine, (np.where(fine, most, 0).astype(np.float32) * (np.float32(1) / np.float32(127))), np.float32(np.nan))
    s = scale.astype(np.float64)
    live = fine & (s > 0)
    # two f32 numbers' quotient lies at least 2^-26 of itself away from any middle that it is not: 64 bits decide
    q = np.rint(np.where(live[:, None], x, 0) / np.where(live, s, 1)[:, None])
    return np.clip(q, -127, 127).astype(np.int8), scale.astype(np.float32)
