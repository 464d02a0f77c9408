"""Pins of the fp64 oracle of the projections (oracle/proj_oracle.py): hand-worked values, closed
forms, central differences for every backward, and planted mistakes that a pin rejects."""
import inspect
import math

import numpy as np
import pytest

import oracle as O
from oracle import proj_oracle as PO
from test_oracle_block import close, differences, rng

ACTS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


def by_hand():
    """Values of the activations at 1 and -2: the normal distribution's 0.841344746 and 0.022750132,
    the logistic function's 0.731058579 and 0.119202922, tanh by its exponentials."""
    th = lambda z: math.tanh(math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3))   # noqa: E731
    return {"none": (1.0, -2.0), "relu": (1.0, 0.0), "gelu": (0.841344746068543, -2 * 0.022750131948179),
            "gelu_tanh": (0.5 * (1 + th(1.0)), -(1 + th(-2.0))), "silu": (0.731058578630005, -2 * 0.119202922022118)}


def pins(act):
    one, two = by_hand()[act]
    v, _ = O.activation(np.array([1.0, -2.0, 0.0]), act)
    assert np.allclose(v, [one, two, 0.0], rtol=1e-12, atol=1e-14)
    z = np.array([-3.1, -1.0, -0.2, 0.3, 0.9, 2.7])
    close(O.activation(z, act)[1], (O.activation(z + 1e-5, act)[0] - O.activation(z - 1e-5, act)[0]) / 2e-5)


@pytest.mark.parametrize("act", ACTS)
def test_activations(act):
    pins(act)
    v, s = O.activation(np.array([-1e4, 1e4]), act)
    assert np.allclose(v, [-1e4 if act == "none" else 0, 1e4]) and np.allclose(s, [float(act == "none"), 1])


def test_linear_by_hand():
    # [1 2] [[3 4], [5 6]]^T + [1 -20] = [12 -3]; relu, residual
    y, z = O.linear([[1.0, 2]], [[3.0, 4], [5, 6]], [1.0, -20], [[0.5, 0.25]], "relu")
    assert np.array_equal(z, [[12, -3]]) and np.array_equal(y, [[12.5, 0.25]])
    gx, gw, gb = O.linear_bwd([[1.0, 2]], [[3.0, 4], [5, 6]], [[2.0, 7]], [[12.0, -3]], "relu")
    assert np.array_equal(gx, [[6, 8]]) and np.array_equal(gw, [[2, 4], [0, 0]]) and np.array_equal(gb, [2, 0])


@pytest.mark.parametrize("act", ACTS)
def test_linear_backward_differences(act):
    r = rng(3)
    a = dict(x=r.standard_normal((4, 3)), w=r.standard_normal((5, 3)), b=r.standard_normal(5))
    g = r.standard_normal((4, 5))
    f = lambda **k: float(np.sum(g * O.linear(k["x"], k["w"], k["b"], None, act)[0]))   # noqa: E731
    z = O.linear(a["x"], a["w"], a["b"])[1]
    for got, ref in zip(O.linear_bwd(a["x"], a["w"], g, z, act), differences(f, a, a)):
        close(got, ref)


def test_gated_ffn_by_hand():
    # g = 2, u = -3 for one hidden element, relu: h = -6; y = -6 [1 -1] + residual
    y, g, u = O.gated_ffn([[1.0, 1]], [[1.0, 1]], [[-1.0, -2]], [[1.0], [-1]], [[0.5, 0.5]], "relu")
    assert g == 2 and u == -3 and np.array_equal(y, [[-5.5, 6.5]])


def ffn_pin(mod):
    r = rng(4)
    a = dict(x=r.standard_normal((3, 4)), wg=r.standard_normal((5, 4)), wu=r.standard_normal((5, 4)),
             wd=r.standard_normal((4, 5)))
    gy = r.standard_normal((3, 4))
    f = lambda **k: float(np.sum(gy * O.gated_ffn(k["x"], k["wg"], k["wu"], k["wd"], act="gelu")[0]))   # noqa: E731
    _, g, u = O.gated_ffn(**{k: v for k, v in zip(("x", "w_gate", "w_up", "w_down"), a.values())}, act="gelu")
    for got, ref in zip(mod["gated_ffn_bwd"](*a.values(), g, u, gy, "gelu"), differences(f, a, a)):
        close(got, ref)


def test_gated_ffn_backward_differences():
    ffn_pin(vars(PO))


def test_gated_ffn_is_linear_in_up_and_down():
    r = rng(5)
    x, wg, wu, wd = (r.standard_normal(s) for s in ((3, 4), (6, 4), (6, 4), (4, 6)))
    y = O.gated_ffn(x, wg, wu, wd)[0]
    assert np.allclose(O.gated_ffn(x, wg, 3 * wu, wd)[0], 3 * y) and np.allclose(O.gated_ffn(x, wg, wu, -2 * wd)[0], -2 * y)


def test_head_norm_by_hand():
    # (3, 4): mean square 12.5, eps 12.5 makes the root 5; position 0 does not turn
    y = O.head_norm_rotary(np.array([[[[3.0, 4]]]]), [0], [1.0], [1.0, 2.0], 12.5, scale=10.0)
    assert np.allclose(y, [[[[6, 16]]]])
    # a quarter turn of (a, b) is (-b, a)
    y = O.head_norm_rotary(np.array([[[[3.0, 4]]]]), [1], [np.pi / 2], None, 12.5)
    assert np.allclose(y, [[[[-0.8, 0.6]]]])


def heads_pin(mod, interleaved):
    r = rng(6)
    a = dict(x=r.standard_normal((2, 2, 3, 6)), w=r.standard_normal(6))
    g, freq, pos = r.standard_normal((2, 2, 3, 6)), [0.7, 0.1], [[3, 4, 5], [0, 9, 2]]
    f = lambda **k: float(np.sum(g * O.head_norm_rotary(k["x"], pos, freq, k["w"], 1e-2, interleaved, 0.5)))   # noqa: E731
    for got, ref in zip(mod["head_norm_rotary_bwd"](a["x"], pos, freq, g, a["w"], 1e-2, interleaved, 0.5),
                        differences(f, a, a)):
        close(got, ref)


@pytest.mark.parametrize("interleaved", [True, False])
def test_head_norm_backward_differences(interleaved):
    heads_pin(vars(PO), interleaved)


def test_head_norm_rotary_is_the_norm_then_the_rotation():
    x = rng(7).standard_normal((2, 3, 5, 8))
    freq = [0.9, 0.3]
    y = x / np.sqrt((x ** 2).mean(-1, keepdims=True) + 1e-6)
    assert np.allclose(O.head_norm_rotary(x, range(5), freq), O.rotary(y, range(5), freq))


MISTAKES = [
    ("z * p * (1 - p)\n    raise", "z * p\n    raise", lambda m: pins_of(m, "silu")),
    ("0.5 * erfc(-z", "0.5 * erfc(z", lambda m: pins_of(m, "gelu")),
    ("(1 + 3 * 0.044715 * z * z)", "(1 + 0.044715 * z * z)", lambda m: pins_of(m, "gelu_tanh")),
    ("gg, gu = gh * u * slope, gh * a", "gg, gu = gh * u * a, gh * slope", ffn_pin),
    ("gy.T @ (a * u)", "gy.T @ a", ffn_pin),
    ("gg @ _f64(w_gate) + gu @ _f64(w_up)", "gu @ _f64(w_gate) + gg @ _f64(w_up)", ffn_pin),
    ("np.mean(v * x * r, -1", "np.mean(g * x * r, -1", lambda m: heads_pin(m, True)),
    ("interleaved, scale, backward=True", "interleaved, scale, backward=False", lambda m: heads_pin(m, False)),
    ("return gx, (g * x * r)", "return gx, (v * x * r)", lambda m: heads_pin(m, True)),
]


def pins_of(mod, act):
    real = PO.activation
    try:
        O.activation = mod["activation"]
        pins(act)
    finally:
        O.activation = real


@pytest.mark.parametrize("i", range(len(MISTAKES)))
def test_planted_mistakes_are_rejected(i):
    good, bad, pin = MISTAKES[i]
    src = inspect.getsource(PO).replace("from .block_oracle", "from oracle.block_oracle")
    assert src.count(good) == 1
    mod = {"__name__": "planted"}
    exec(compile(src.replace(good, bad), "planted", "exec"), mod)
    with pytest.raises(AssertionError):
        pin(mod)
