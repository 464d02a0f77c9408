"""Pins of the fp64 oracle of the operators around the retention (oracle/block_oracle.py):
hand-worked values, closed forms, the retention oracle as a special case of the scan,
central differences for every backward, and planted mistakes that a pin rejects."""
import inspect

import numpy as np
import pytest

import oracle as O
from oracle import block_oracle as BO


def rng(seed):
    return np.random.default_rng(seed)


def differences(f, args, names, step=1e-5):
    """Central differences of the scalar f(**args) by every element of the named arguments."""
    out = []
    for nm in names:
        base = args[nm]
        g = np.zeros_like(base)
        for i in np.ndindex(*base.shape):
            hi, lo = base.copy(), base.copy()
            hi[i] += step
            lo[i] -= step
            g[i] = (f(**{**args, nm: hi}) - f(**{**args, nm: lo})) / (2 * step)
        out.append(g)
    return out


def close(a, b, tol=2e-8):
    """Central differences with a step of 1e-5 in fp64: truncation ~1e-10, rounding ~1e-11 of the value."""
    assert np.max(np.abs(a - b)) <= tol * max(1.0, np.max(np.abs(b))), np.max(np.abs(a - b))


# -------------------------------------------------------------------------------------- layer norm
def test_layer_norm_by_hand():
    # (1, 3, 5, 7): mean 4, deviations -3 -1 1 3, variance 5; eps 4 makes the root 3
    y, mean, rstd = O.layer_norm(np.array([[1.0, 3, 5, 7]]), np.array([1.0, 2, 3, 4]), np.array([0.0, 0, 1, 1]), eps=4.0)
    assert np.allclose(mean, 4) and np.allclose(rstd, 1 / 3)
    assert np.allclose(y, [[-1, -2 / 3, 2, 5]])


def test_layer_norm_is_shift_and_scale_free():
    x = rng(1).standard_normal((3, 17))
    assert np.allclose(O.layer_norm(x, eps=0.0)[0], O.layer_norm(5 * x - 2, eps=0.0)[0])


def test_layer_norm_backward_differences():
    r = rng(2)
    a = dict(x=r.standard_normal((3, 5)), weight=r.standard_normal(5), bias=r.standard_normal(5))
    g = r.standard_normal((3, 5))
    f = lambda **k: float(np.sum(g * O.layer_norm(k["x"], k["weight"], k["bias"], 1e-2)[0]))   # noqa: E731
    _, mean, rstd = O.layer_norm(a["x"], eps=1e-2)
    for got, ref in zip(O.layer_norm_bwd(a["x"], a["weight"], mean, rstd, g), differences(f, a, a)):
        close(got, ref)


# ------------------------------------------------------------------------------------------ rotary
def test_rotary_by_hand_and_layouts():
    f = np.array([np.pi / 2, np.pi])
    x = np.arange(1.0, 6.0).reshape(1, 1, 1, 5)
    # position 1: the first pair turns by a quarter, the second by a half; the fifth element passes
    assert np.allclose(O.rotary(x, [1], f)[0, 0, 0], [-2, 1, -3, -4, 5])
    assert np.allclose(O.rotary(x, [1], f, interleaved=False)[0, 0, 0], [-3, -2, 1, -4, 5])
    assert np.allclose(O.rotary(x, [0], f, scale=2.0)[0, 0, 0], 2 * x[0, 0, 0])


def test_rotary_agrees_with_the_layer_oracle():
    x = rng(3).standard_normal((2, 3, 7, 8))
    f = 10000.0 ** (-np.arange(0, 8, 2) / 8)
    assert np.allclose(O.rotary(x, np.arange(7), f), O.rope_interleaved(x), atol=1e-13)


def test_rotary_backward_is_the_transpose():
    r = rng(4)
    x, g, f = r.standard_normal((2, 3, 5, 6)), r.standard_normal((2, 3, 5, 6)), r.random(2)
    pos = r.integers(0, 1000, (2, 5))
    for inter in (True, False):
        lhs = np.sum(g * O.rotary(x, pos, f, inter, 0.7, 1.3))
        assert np.isclose(lhs, np.sum(x * O.rotary(g, pos, f, inter, 0.7, 1.3, backward=True)))


# -------------------------------------------------------------------------------- causal convolution
def test_causal_conv_by_hand_and_split():
    x = np.array([1.0, 2, 3, 4]).reshape(1, 4, 1)
    w = np.array([[10.0, 1.0]])
    y, s = O.causal_conv(x, w, np.array([0.5]))
    assert np.allclose(y[0, :, 0], [1.5, 12.5, 23.5, 34.5]) and np.allclose(s, 4)
    r = rng(5)
    x, w = r.standard_normal((2, 9, 3)), r.standard_normal((3, 4))
    y, s = O.causal_conv(x, w, silu=True)
    y1, s1 = O.causal_conv(x[:, :2], w, silu=True)
    y2, s2 = O.causal_conv(x[:, 2:], w, silu=True, state_in=s1)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(s, s2)
    yl, sl = O.causal_conv(x, w, silu=True, lengths=[9, 2])
    assert np.allclose(yl[1, :2], y[1, :2]) and not yl[1, 2:].any() and np.allclose(sl[1], s1[1])


@pytest.mark.parametrize("silu", [False, True])
def test_causal_conv_backward_differences(silu):
    r = rng(6)
    a = dict(x=r.standard_normal((2, 4, 2)), weight=r.standard_normal((2, 3)), bias=r.standard_normal(2),
             state_in=r.standard_normal((2, 2, 2)))
    g, gs, n = r.standard_normal((2, 4, 2)), r.standard_normal((2, 2, 2)), [4, 1]

    def f(**k):
        y, s = O.causal_conv(k["x"], k["weight"], k["bias"], silu, k["state_in"], n)
        return float(np.sum(g * y) + np.sum(gs * s))

    got = O.causal_conv_bwd(a["x"], a["weight"], g, a["bias"], silu, a["state_in"], gs, n)
    for u, v in zip(got, differences(f, a, ("x", "weight", "bias", "state_in"))):
        close(u, v)


# ------------------------------------------------------------------------------------ selective scan
def scan_case(seed, B=2, N=5, D=4, G=2, S=3):
    r = rng(seed)
    return dict(x=r.standard_normal((B, N, D)), dt=r.standard_normal((B, N, D)), A=-r.random((D, S)) - 0.1,
                Bm=r.standard_normal((B, N, G, S)), Cm=r.standard_normal((B, N, G, S)), D=r.standard_normal(D),
                z=r.standard_normal((B, N, D)), dt_bias=r.standard_normal(D), state_in=r.standard_normal((B, D, S)))


def test_selective_scan_by_hand():
    ln2 = np.log(2.0)
    one = np.ones((1, 2, 1))
    y, h = O.selective_scan(one * [[[3.0], [1.0]]], one, np.array([[-ln2]]), np.ones((1, 2, 1, 1)),
                            2 * np.ones((1, 2, 1, 1)), D=np.array([10.0]), state_in=np.full((1, 1, 1), 4.0))
    # h: 4 -> 4/2 + 3 = 5 -> 5/2 + 1 = 3.5; y = 2 h + 10 x
    assert np.allclose(y[0, :, 0], [40, 17]) and np.allclose(h, 3.5)


def test_selective_scan_contains_the_gated_retention():
    """One decay for all channels and states, A = -1 and dt_t: the gated retention with
    q = C, k = B, v = dt x and log-decay -dt."""
    r = rng(7)
    B, N, D, S = 2, 11, 5, 4
    x, Bm, Cm = r.standard_normal((B, N, D)), r.standard_normal((B, N, 1, S)), r.standard_normal((B, N, 1, S))
    dt = np.repeat(r.random((B, N, 1)), D, 2)
    s0 = r.standard_normal((B, D, S))
    y, h = O.selective_scan(x, dt, -np.ones((D, S)), Bm, Cm, state_in=s0)
    o, s = O.gated_retention_recurrent(Cm.transpose(0, 2, 1, 3), Bm.transpose(0, 2, 1, 3), (dt * x)[:, None], -dt[:, None, :, 0],
                                       s0.transpose(0, 2, 1)[:, None])
    assert np.allclose(o[:, 0], y, atol=1e-12) and np.allclose(s[:, 0].transpose(0, 2, 1), h, atol=1e-12)


def test_selective_scan_split_and_lengths():
    a = scan_case(8, N=7)
    y, h = O.selective_scan(**a, use_softplus=True)
    cut = {k: (v[:, :3] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in a.items()}
    rest = {k: (v[:, 3:] if k in ("x", "dt", "Bm", "Cm", "z") else v) for k, v in a.items()}
    y1, h1 = O.selective_scan(**cut, use_softplus=True)
    y2, h2 = O.selective_scan(**{**rest, "state_in": h1}, use_softplus=True)
    assert np.allclose(np.concatenate([y1, y2], 1), y) and np.allclose(h, h2)
    yl, hl = O.selective_scan(**a, use_softplus=True, lengths=[0, 3])
    assert not yl[0].any() and np.allclose(hl[0], a["state_in"][0]) and np.allclose(hl[1], h1[1])


@pytest.mark.parametrize("gate,sp", [(True, True), (False, False)])
def test_selective_scan_backward_differences(gate, sp):
    a = scan_case(9, N=4)
    if not gate:
        a.pop("z")
    r = rng(10)
    g, gs, n = r.standard_normal(a["x"].shape), r.standard_normal(a["state_in"].shape), [4, 2]

    def f(**k):
        y, h = O.selective_scan(**k, use_softplus=sp, lengths=n)
        return float(np.sum(g * y) + np.sum(gs * h))

    got = dict(zip(("x", "dt", "A", "Bm", "Cm", "D", "z", "dt_bias", "state_in"),
                   O.selective_scan_bwd(a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], g, a["D"], a.get("z"), a["dt_bias"], sp,
                                        a["state_in"], gs, n)))
    for nm, ref in zip(a, differences(f, a, a)):
        close(got[nm], ref, 1e-7)


def test_magnitudes_bound_the_gradients():
    a = scan_case(11)
    g = rng(12).standard_normal(a["x"].shape)
    args = (a["x"], a["dt"], a["A"], a["Bm"], a["Cm"], g, a["D"], a["z"], a["dt_bias"], True, a["state_in"])
    for v, m in zip(O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True)):
        assert np.all(np.abs(v) <= m + 1e-12)


MISTAKES = {   # function, text, planted text, test that rejects it
    "norm: variance about zero": ("layer_norm", "(x - mean[..., None]) ** 2", "x ** 2", test_layer_norm_by_hand),
    "norm: mean of the gradient kept": ("layer_norm_bwd", "rstd * (v - m1 - xh * m2)", "rstd * (v - xh * m2)",
                                        test_layer_norm_backward_differences),
    "rotary: halves as adjacent pairs": ("rotary", "if interleaved:", "if True:", test_rotary_by_hand_and_layouts),
    "rotary: backward turns on": ("rotary", "-1j if backward else 1j", "1j", test_rotary_backward_is_the_transpose),
    "conv: weights reversed": ("_conv_parts", "weight[:, j]", "weight[:, K - 1 - j]", test_causal_conv_by_hand_and_split),
    "conv: state one row late": ("causal_conv", "xs[n:n + K - 1]", "np.concatenate([xs, xs])[n + 1:n + K]",
                                 test_causal_conv_by_hand_and_split),
    "scan: input undiscretised": ("selective_scan", "(dt[b, t] * x[b, t])", "x[b, t]",
                                  test_selective_scan_contains_the_gated_retention),
    "scan: read before the update": ("selective_scan", "np.sum(Cm[b, t][group] * h[b], -1)",
                                     "np.sum(Cm[b, t][group] * (h[b] - (dt[b, t] * x[b, t])[:, None] * Bm[b, t][group]), -1)",
                                     test_selective_scan_by_hand),
    "scan: adjoint undecayed": ("selective_scan_bwd", "w[b] = adj * dec", "w[b] = adj",
                                lambda: test_selective_scan_backward_differences(True, True)),
    "scan: dA from the new state": ("selective_scan_bwd", "q = adj * hs[t] * dec", "q = adj * hs[t + 1]",
                                    lambda: test_selective_scan_backward_differences(True, True)),
}


@pytest.mark.parametrize("name", MISTAKES)
def test_planted_mistakes_are_rejected(name, monkeypatch):
    fn, text, planted, pin = MISTAKES[name]
    source = inspect.getsource(getattr(BO, fn))
    assert source.count(text) >= 1
    scope = dict(vars(BO))
    exec(source.replace(text, planted), scope)
    if fn.startswith("_"):      # a part: the functions that call it have to find the planted one
        for whole in ("causal_conv", "causal_conv_bwd"):
            exec(inspect.getsource(getattr(BO, whole)), scope)
            monkeypatch.setattr(O, whole, scope[whole])
    else:
        monkeypatch.setattr(O, fn, scope[fn])
    with pytest.raises(AssertionError):
        pin()
