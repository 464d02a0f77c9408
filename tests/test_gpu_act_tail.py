"""The activations where they are small, and their slopes at ordinary values, relative to what they are.

Counting roundings, in units of U = 2^-24 (half a step of fp32), for z < 0, where an activation is z P(z)
with a small P:
  gelu       the tail of the normal distribution is a polynomial times e^(-z^2/2): the fit 2, its terms,
             their argument and a reciprocal 12, exponential and products 8; the exponent is rounded three
             times (square, constant, product), each 1 of z^2/2.  In all 1.5 z^2 + 24.
  silu       1 / (1 + e^-z): the exponent's constant and product 1 each of |z|, the rest 16.  2 |z| + 16.
  gelu_tanh  the same of q = 2 sqrt(2/pi) (z + 0.044715 z^3), whose own products are 6 more of |q|.  8 |q| + 16.
A slope is P + z P' with the same errors of both terms, and 8 for what P' takes besides.  For z >= 0 nothing
is small, and the errors are 16 of |z| (24 of one for a slope).  bf16 results are rounded once more.
P is held in fp32, whose smallest whole-precision value is T = 2^-126; below it P may be zero, which moves
z P by |z| T and the slope P + z P (1 - P) q' by (1 + |z| q') T, q' being 1 (silu) or the derivative of q.  The tail of
gelu is that small only below -13.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, U, half  # noqa: E402

T = 2.0 ** -126
SMOOTH = ["gelu", "gelu_tanh", "silu"]


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def grid(dtype):
    """(CUDA column, fp64 row) of pre-activations from -12 to 12."""
    z = torch.linspace(-12, 12, 6007).to(TYPES[dtype])
    return z.cuda()[:, None], z.double().numpy()


def steps(z, act):
    a = np.abs(z)
    if act == "gelu":
        return 1.5 * a * a + 24
    if act == "silu":
        return 2 * a + 16
    return 8 * 2 * np.sqrt(2 / np.pi) * (a + 0.044715 * a ** 3) + 16


def growth(z, act):
    """q' of an activation z / (1 + e^-q)."""
    return 2 * np.sqrt(2 / np.pi) * (1 + 3 * 0.044715 * z * z) if act == "gelu_tanh" else np.ones_like(z)


def inside(got, ref, room):
    got = got.double().cpu().numpy().reshape(-1)
    over = np.abs(got - ref) / room
    i = int(np.argmax(over))
    assert over[i] <= 1, f"{i}: {got[i]} for {ref[i]}, {over[i]:.2f} of the bound"


def value_room(z, ref, act, dtype):
    return np.where(z < 0, steps(z, act) * np.abs(ref), 16 * np.abs(z)) * U + half(TYPES[dtype]) * np.abs(ref) + np.abs(z) * T + T


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_small_values_keep_their_bits(act, dtype):
    print(f"\n[case] small values {act} {dtype}", flush=True)
    z, zr = grid(dtype)
    one = torch.ones(1, 1, device="cuda", dtype=TYPES[dtype])
    ref = O.activation(zr, act)[0]
    inside(R().linear_fwd(z, one, activation=act), ref, value_room(zr, ref, act, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_values_of_the_gradient(act, dtype):
    """The gated product, which the gradient of w_down forms again from gate and up."""
    print(f"\n[case] small values of the gradient {act} {dtype}", flush=True)
    z, zr = grid(dtype)
    F, t = len(zr), TYPES[dtype]
    x, one, row = (torch.ones(s, device="cuda", dtype=t) for s in ((1, 1), (F, 1), (1, F)))
    got = R().gated_ffn_bwd(x, one, one, row, z.view(1, F), row, x, activation=act)[3]
    ref = O.activation(zr, act)[0]
    inside(got, ref, value_room(zr, ref, act, dtype))


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", SMOOTH)
def test_slopes(act, dtype):
    print(f"\n[case] slopes {act} {dtype}", flush=True)
    z, zr = grid(dtype)
    one = torch.ones(1, 1, device="cuda", dtype=TYPES[dtype])
    got = R().linear_bwd(z, one, torch.ones_like(z), pre=z, activation=act)[0]
    value, ref = O.activation(zr, act)
    p = np.abs(value) / np.maximum(np.abs(zr), 1e-30)
    terms = np.abs(p) + np.abs(ref - p)
    inside(got, ref, np.where(zr < 0, (steps(zr, act) + 8) * terms, 24) * U + half(TYPES[dtype]) * np.abs(ref)
           + (1 + np.abs(zr) * growth(zr, act)) * T)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("act", ["none", "relu"] + SMOOTH)
def test_both_directions_agree_at_the_ends_of_the_type(act, dtype):
    """Where P is 0, 1/2 or 1, the gated product that the gradient of w_down forms again is the forward's, NaN where
    that is NaN: a gate of minus infinity, whose gelu is 0, leaves the gradients finite."""
    print(f"\n[case] ends {act} {dtype}", flush=True)
    t = TYPES[dtype]
    gate = torch.tensor([float("-inf"), -3e38, -1e4, -0.0, 0.0, 1e4, 3e38, float("inf"), float("nan")], device="cuda").to(t)
    F = len(gate)
    x, one, row = (torch.ones(s, device="cuda", dtype=t) for s in ((1, 1), (F, 1), (1, F)))
    forward = R().linear_fwd(gate[:, None], x, activation=act)[:, 0]
    gx, _, _, gwd = R().gated_ffn_bwd(x, one, one, row, gate[None], row, x, activation=act)
    both = torch.isnan(forward) & torch.isnan(gwd[0])
    assert (both | (forward == gwd[0])).all(), (forward, gwd)
    if act in ("relu", "gelu"):
        gx = R().gated_ffn_bwd(x, one[:1], one[:1], row[:, :1], gate[None, :1], row[:, :1], x, activation=act)[0]
        assert gx.item() == 0.0
