"""fp64 CPU oracle of a block's projections: the matrix product with bias, activation and residual,
the gated feed-forward block, and the head norms with rotary positions.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Every function follows the operator's
definition in numpy fp64 and shares no code with the GPU library.
"""
from __future__ import annotations

import numpy as np
from scipy.special import erfc, expit

from .block_oracle import _f64, rotary

__all__ = ["activation", "linear", "linear_bwd", "gated_ffn", "gated_ffn_bwd", "head_norm_rotary", "head_norm_rotary_bwd"]

ACTIVATIONS = ("none", "relu", "gelu", "gelu_tanh", "silu")


def activation(z, name):
    """(value, derivative) of an activation: z P(z) with a distribution function P, or a threshold."""
    z = _f64(z)
    if name == "none":
        return z, np.ones_like(z)
    if name == "relu":
        return np.where(z > 0, z, 0.0), np.where(z > 0, 1.0, 0.0)
    if name == "gelu":
        p = 0.5 * erfc(-z / np.sqrt(2.0))
        return z * p, p + z * np.exp(-0.5 * z * z) / np.sqrt(2.0 * np.pi)
    if name == "gelu_tanh":
        c = np.sqrt(2.0 / np.pi)
        p = expit(2 * c * (z + 0.044715 * z ** 3))
        return z * p, p + z * p * (1 - p) * 2 * c * (1 + 3 * 0.044715 * z * z)
    if name == "silu":
        p = expit(z)
        return z * p, p + z * p * (1 - p)
    raise ValueError(name)


def linear(x, weight, bias=None, residual=None, act="none"):
    """(act(z) + residual, z) with z = x weight^T + bias."""
    z = _f64(x) @ _f64(weight).T
    if bias is not None:
        z = z + _f64(bias)
    y = activation(z, act)[0]
    return (y if residual is None else y + _f64(residual)), z


def linear_bwd(x, weight, grad_y, pre=None, act="none"):
    """(grad_x, grad_weight, grad_bias) for rows x [R, K] and the forward's pre-activations."""
    gz = _f64(grad_y)
    if act != "none":
        gz = gz * activation(pre, act)[1]
    return gz @ _f64(weight), gz.T @ _f64(x), gz.sum(0)


def gated_ffn(x, w_gate, w_up, w_down, residual=None, act="silu"):
    """(y, gate, up): y = (act(x w_gate^T) * (x w_up^T)) w_down^T + residual."""
    g, u = _f64(x) @ _f64(w_gate).T, _f64(x) @ _f64(w_up).T
    y = (activation(g, act)[0] * u) @ _f64(w_down).T
    return (y if residual is None else y + _f64(residual)), g, u


def gated_ffn_bwd(x, w_gate, w_up, w_down, gate, up, grad_y, act="silu"):
    """(grad_x, grad_w_gate, grad_w_up, grad_w_down) for rows x [R, D]."""
    x, gy, u = _f64(x), _f64(grad_y), _f64(up)
    a, slope = activation(gate, act)
    gh = gy @ _f64(w_down)
    gg, gu = gh * u * slope, gh * a
    return gg @ _f64(w_gate) + gu @ _f64(w_up), gg.T @ x, gu.T @ x, gy.T @ (a * u)


def head_norm_rotary(x, positions, freq, weight=None, eps=1e-6, interleaved=True, scale=1.0):
    """scale * turn(x / sqrt(mean(x^2) + eps) * weight) of x [B, H, N, d] (turn: `rotary`)."""
    x = _f64(x)
    y = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    return rotary(y if weight is None else y * _f64(weight), positions, freq, interleaved, scale)


def head_norm_rotary_bwd(x, positions, freq, grad, weight=None, eps=1e-6, interleaved=True, scale=1.0):
    """(gradient of x, gradient of weight)."""
    x = _f64(x)
    r = 1.0 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    g = rotary(_f64(grad), positions, freq, interleaved, scale, backward=True)
    v = g if weight is None else g * _f64(weight)
    gx = r * (v - x * r * np.mean(v * x * r, -1, keepdims=True))
    return gx, (g * x * r).sum((0, 1, 2))
