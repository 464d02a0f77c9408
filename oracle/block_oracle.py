"""fp64 CPU oracle of the operators around the retention in a block: layer normalisation,
rotary positions, the short causal convolution and the selective state-space scan.

TEST INFRASTRUCTURE ONLY, like the rest of this package.  Every function follows the
operator's definition token by token in numpy fp64 and shares no code with the GPU library.

The backward functions take ``magnitude=True`` for error bounds: every product then enters
the sums with its absolute value, so the result bounds what the rounding errors of the
sums' terms are relative to.  (For the scan the decays stay what they are.)
"""
from __future__ import annotations

import numpy as np

__all__ = ["layer_norm", "layer_norm_bwd", "rotary", "causal_conv", "causal_conv_bwd", "selective_scan",
           "selective_scan_bwd", "softplus"]


def _f64(x):
    return None if x is None else np.asarray(x, dtype=np.float64)


def _sigmoid(x):
    return 0.5 * (1.0 + np.tanh(0.5 * x))


def softplus(x):
    """log(1 + e^x)."""
    return np.logaddexp(0.0, _f64(x))


def layer_norm(x, weight=None, bias=None, eps=1e-5):
    """(y, mean, rstd) over the last axis."""
    x = _f64(x)
    mean = np.mean(x, axis=-1)
    rstd = 1.0 / np.sqrt(np.mean((x - mean[..., None]) ** 2, axis=-1) + eps)
    y = (x - mean[..., None]) * rstd[..., None]
    if weight is not None:
        y = y * _f64(weight)
    if bias is not None:
        y = y + _f64(bias)
    return y, mean, rstd


def layer_norm_bwd(x, weight, mean, rstd, grad_y, magnitude=False):
    """(grad_x, grad_weight, grad_bias) for rows x [R, D] with their statistics."""
    a = np.abs if magnitude else (lambda v: v)
    x, g, mean, rstd = _f64(x), _f64(grad_y), _f64(mean)[:, None], _f64(rstd)[:, None]
    xh = (x - mean) * rstd
    v = g if weight is None else g * _f64(weight)
    m1, m2 = np.mean(a(v), -1, keepdims=True), np.mean(a(v * xh), -1, keepdims=True)
    if magnitude:
        # x - mean is rounded relative to its operands
        xh = (np.abs(x) + np.abs(mean)) * rstd
        return rstd * (np.abs(v) + m1 + xh * m2), np.sum(np.abs(g) * xh, 0), np.sum(np.abs(g), 0)
    return rstd * (v - m1 - xh * m2), np.sum(g * xh, 0), np.sum(g, 0)


def rotary(x, positions, freq, interleaved=True, scale=1.0, magnitude=1.0, backward=False):
    """x [B, H, N, d]; positions [N] or [B, N]; the first 2 len(freq) elements of a head turn as
    complex numbers by e^(i p f) (backward: e^(-i p f))."""
    x, freq = _f64(x), _f64(freq)
    p = np.asarray(positions, dtype=np.float64)
    p = np.broadcast_to(p, (x.shape[0], x.shape[2]))
    w = magnitude * np.exp((-1j if backward else 1j) * p[:, None, :, None] * freq)
    r = 2 * len(freq)
    out = x.copy()
    if interleaved:
        c = (x[..., 0:r:2] + 1j * x[..., 1:r:2]) * w
        out[..., 0:r:2], out[..., 1:r:2] = c.real, c.imag
    else:
        c = (x[..., :r // 2] + 1j * x[..., r // 2:r]) * w
        out[..., :r // 2], out[..., r // 2:r] = c.real, c.imag
    return out * scale


def _conv_parts(x, weight, bias, state_in, n):
    """xs, pre and the windows of one sequence of n tokens."""
    K = weight.shape[1]
    xs = np.concatenate([state_in, x[:n]])
    pre = np.zeros((n, x.shape[1]))
    for t in range(n):
        pre[t] = bias + sum(weight[:, j] * xs[t + j] for j in range(K))
    return xs, pre


def causal_conv(x, weight, bias=None, silu=False, state_in=None, lengths=None):
    """(y, state_out) for x [B, N, D], weight [D, K]; rows behind a length are zero."""
    x, weight = _f64(x), _f64(weight)
    B, N, D = x.shape
    K = weight.shape[1]
    bias = np.zeros(D) if bias is None else _f64(bias)
    s0 = np.zeros((B, K - 1, D)) if state_in is None else _f64(state_in)
    y, s1 = np.zeros((B, N, D)), np.zeros((B, K - 1, D))
    for b in range(B):
        n = N if lengths is None else int(lengths[b])
        xs, pre = _conv_parts(x[b], weight, bias, s0[b], n)
        y[b, :n] = pre * _sigmoid(pre) if silu else pre
        s1[b] = xs[n:n + K - 1]
    return y, s1


def causal_conv_bwd(x, weight, grad_y, bias=None, silu=False, state_in=None, grad_state_out=None, lengths=None,
                    magnitude=False):
    """(grad_x, grad_weight, grad_bias, grad_state_in)."""
    a = np.abs if magnitude else (lambda v: v)
    x, weight, g = _f64(x), _f64(weight), _f64(grad_y)
    B, N, D = x.shape
    K = weight.shape[1]
    bias = np.zeros(D) if bias is None else _f64(bias)
    s0 = np.zeros((B, K - 1, D)) if state_in is None else _f64(state_in)
    gs1 = np.zeros((B, K - 1, D)) if grad_state_out is None else _f64(grad_state_out)
    gx, gw, gb, gs0 = np.zeros((B, N, D)), np.zeros((D, K)), np.zeros(D), np.zeros((B, K - 1, D))
    for b in range(B):
        n = N if lengths is None else int(lengths[b])
        xs, pre = _conv_parts(x[b], weight, bias, s0[b], n)
        gp = g[b, :n].copy()
        if silu:
            s = _sigmoid(pre)
            gp = gp * (s + pre * s * (1 - s))
        gxs = np.zeros((n + K - 1, D))
        for t in range(n):
            for j in range(K):
                gxs[t + j] += a(gp[t] * weight[:, j])
                gw[:, j] += a(gp[t] * xs[t + j])
            gb += a(gp[t])
        gxs[n:] += a(gs1[b])
        gx[b, :n], gs0[b] = gxs[K - 1:], gxs[:K - 1]
    return gx, gw, gb, gs0


def selective_scan(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, use_softplus=False, state_in=None, lengths=None):
    """(y, state_out): the recurrence token by token.  x, dt, z [B, N, D]; Bm, Cm [B, N, G, S];
    A [D, S]; state [B, D, S]; rows behind a length are zero."""
    x, raw, A, Bm, Cm = _f64(x), _f64(dt), _f64(A), _f64(Bm), _f64(Cm)
    B, N, ch = x.shape
    group = np.arange(ch) // (ch // Bm.shape[2])
    raw = raw if dt_bias is None else raw + _f64(dt_bias)
    dt = softplus(raw) if use_softplus else raw
    skip = np.zeros(ch) if D is None else _f64(D)
    h = np.zeros((B, ch, A.shape[1])) if state_in is None else _f64(state_in).copy()
    y = np.zeros((B, N, ch))
    for b in range(B):
        for t in range(N if lengths is None else int(lengths[b])):
            h[b] = np.exp(dt[b, t][:, None] * A) * h[b] + (dt[b, t] * x[b, t])[:, None] * Bm[b, t][group]
            y[b, t] = np.sum(Cm[b, t][group] * h[b], -1) + skip * x[b, t]
    if z is not None:
        y = y * (_f64(z) * _sigmoid(_f64(z)))
    return y, h


def selective_scan_bwd(x, dt, A, Bm, Cm, grad_y, D=None, z=None, dt_bias=None, use_softplus=False, state_in=None,
                       grad_state_out=None, lengths=None, magnitude=False):
    """(grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_z, grad_dt_bias, grad_state_in)."""
    a = np.abs if magnitude else (lambda v: v)
    x, raw, A, Bm, Cm, g = a(_f64(x)), _f64(dt), _f64(A), a(_f64(Bm)), a(_f64(Cm)), a(_f64(grad_y))
    B, N, ch = x.shape
    G, S = Bm.shape[2:]
    group = np.arange(ch) // (ch // G)
    raw = raw if dt_bias is None else raw + _f64(dt_bias)
    dt = softplus(raw) if use_softplus else raw
    dtm = a(dt)
    skip = np.zeros(ch) if D is None else a(_f64(D))
    h0 = np.zeros((B, ch, S)) if state_in is None else a(_f64(state_in))
    w = np.zeros((B, ch, S)) if grad_state_out is None else a(_f64(grad_state_out)).copy()
    gx, gdt, gz = np.zeros((B, N, ch)), np.zeros((B, N, ch)), np.zeros((B, N, ch))
    gA, gB, gC, gD = np.zeros((ch, S)), np.zeros((B, N, G, S)), np.zeros((B, N, G, S)), np.zeros(ch)
    for b in range(B):
        n = N if lengths is None else int(lengths[b])
        hs = [h0[b]]
        for t in range(n):
            hs.append(np.exp(dt[b, t][:, None] * A) * hs[-1] + (dtm[b, t] * x[b, t])[:, None] * Bm[b, t][group])
        for t in reversed(range(n)):
            gt = g[b, t]
            if z is not None:
                zt = _f64(z)[b, t]
                s = _sigmoid(zt)
                ys = np.sum(Cm[b, t][group] * hs[t + 1], -1) + skip * x[b, t]
                gz[b, t] = gt * ys * (a(s) + a(zt * s * (1 - s)))
                gt = gt * a(zt * s)
            adj = Cm[b, t][group] * gt[:, None] + w[b]
            dec = np.exp(dt[b, t][:, None] * A)
            du = np.sum(adj * Bm[b, t][group], -1)
            q = adj * hs[t] * dec
            gx[b, t] = du * dtm[b, t] + skip * gt
            d = du * x[b, t] + np.sum(q * a(A), -1)
            gdt[b, t] = d * _sigmoid(raw[b, t]) if use_softplus else d
            gA += q * dtm[b, t][:, None]
            gD += gt * x[b, t]
            np.add.at(gB[b, t], group, adj * (dtm[b, t] * x[b, t])[:, None])
            np.add.at(gC[b, t], group, hs[t + 1] * gt[:, None])
            w[b] = adj * dec
    return gx, gdt, gA, gB, gC, gD, gz, gdt.sum((0, 1)), w
