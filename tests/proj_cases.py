"""Error bounds of the projections, shared by their GPU tests.

In units of U = 2^-24 (half a step of fp32).  A sum of n products in the matrix cores is off by
at most 2 n + 16 of the sum of the products' absolute values: n additions of half a step each,
twice that for cores that cut instead of rounding, a few for joining split sums.  An activation
is off by 16 |z| (its distribution function by 6: the polynomial 1.3, exponential, reciprocal
and products the rest) and moves by at most 1.2 of what z is off by; its slope is off by 24 of
one.  What is kept in the type t between two products is off by half(t) / U of its value more.
"""
import numpy as np

import oracle as O
from block_cases import TYPES, U, half

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def total(n):
    return 2 * n + 16


def step(dtype):
    return half(TYPES[dtype]) / U


def linear_bounds(x, w, b, r, act):
    """Bounds of (y, pre) before their own rounding."""
    x, w = np.abs(x), np.abs(w)
    z = O.linear(x, w, None if b is None else np.abs(b))[1]
    bz = total(x.shape[1]) * z
    return 1.2 * bz + 20 * z + (0 if r is None else 4 * np.abs(r)), bz


def linear_bwd_bounds(x, w, gy, pre, act, dtype):
    x, w, gy = np.abs(x), np.abs(w), np.abs(gy)
    if act == "none":
        gz, bz = gy, 0 * gy
    else:
        gz = gy * np.abs(O.activation(pre, act)[1])
        bz = step(dtype) * gz + 24 * gy
    n = len(x)
    return (bz @ w + total(w.shape[0]) * (gz @ w), bz.T @ x + total(n) * (gz.T @ x),
            (24 * gy + 0 * gz).sum(0) + total(n) * gz.sum(0))


def ffn_bounds(x, wg, wu, wd, r, act, dtype):
    """Bounds of (y, gate, up)."""
    x = np.abs(x)
    g, u = x @ np.abs(wg).T, x @ np.abs(wu).T                     # the sums of absolute values
    bg, bu = total(x.shape[1]) * g, total(x.shape[1]) * u
    return bg, bu


def ffn_y_bound(g, u, bg, bu, wd, r, act, dtype):
    a = O.activation(g, act)[0]
    h = np.abs(a * u)
    bh = (1.2 * bg + 16 * np.abs(g)) * np.abs(u) + np.abs(a) * bu + 4 * h + step(dtype) * h
    wd = np.abs(wd)
    return 1.01 * (bh @ wd.T + total(wd.shape[1]) * (h @ wd.T) + (0 if r is None else 4 * np.abs(r)))


def ffn_bwd_bounds(x, wg, wu, wd, gate, up, gy, act, dtype):
    x, wg, wu, ad, ay, u = (np.abs(v) for v in (x, wg, wu, wd, gy, up))
    a, s = O.activation(gate, act)
    a, s, g = np.abs(a), np.abs(s), np.abs(gate)
    gh, mh = np.abs(gy @ wd), ay @ ad
    bh = total(gy.shape[1]) * mh
    st = step(dtype)
    gu, gg, h = gh * a, gh * u * s, a * u
    bu = bh * a + 16 * g * gh + (4 + st) * gu
    bg = bh * u * s + 24 * gh * u + (4 + st) * gg
    bp = 16 * g * u + (4 + st) * h
    n = total(len(x))
    bx = bg @ wg + bu @ wu + total(2 * len(wg)) * (gg @ wg + gu @ wu)
    return tuple(1.01 * v for v in (bx, bg.T @ x + n * (gg.T @ x), bu.T @ x + n * (gu.T @ x), ay.T @ bp + n * (ay.T @ h)))


def pair_sizes(x, rot, interleaved):
    """|a| + |b| of each element's pair."""
    m = np.abs(x).copy()
    if interleaved:
        s = m[..., 0:rot:2] + m[..., 1:rot:2]
        m[..., 0:rot:2] = m[..., 1:rot:2] = s
    else:
        s = m[..., :rot // 2] + m[..., rot // 2:rot]
        m[..., :rot // 2] = m[..., rot // 2:rot] = s
    return m
