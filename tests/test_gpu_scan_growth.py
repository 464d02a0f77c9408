"""The selective scan where decays are above one (A dt > 0), so that the factor of a whole segment
of tokens is beyond fp32 (e^8 a token and more, e^128 over 16 of them) though each token's is not:
a state of zero stays zero whatever multiplies it, and a tiny one grows to what it is.

Bounds as in test_gpu_scan.py where the tokens that grow carry nothing and the others decay.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import check, draw  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def case(B, N, D, S, dtype, lo, hi):
    """No state before token hi; tokens lo .. hi - 1 grow."""
    t, v = {}, {}
    for i, (name, shape) in enumerate((("x", (B, N, D)), ("Bm", (B, N, 1, S)), ("Cm", (B, N, 1, S)))):
        t[name], v[name] = draw(30 + i, shape, dtype)
    t["x"][:, :hi] = 0
    r = np.random.default_rng(40)
    t["A"] = torch.tensor(r.uniform(0.9, 1.5, (D, S))).float().cuda()
    dt = -r.uniform(0.05, 0.5, (B, N, D))
    dt[:, lo:hi] = 8.0
    t["dt"] = torch.tensor(dt).to(t["x"].dtype).cuda()
    return t, {n: a.double().cpu().numpy() for n, a in t.items()}


NAMES = ("x", "dt", "A", "Bm", "Cm")
SIZES = [(1, 700, 20, 16), (2, 1600, 20, 16), (1, 1700, 37, 5), (1, 900, 70, 40)]   # composed by one wave and by 16


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,S", SIZES)
def test_forward(B, N, D, S, dtype):
    print(f"\n[case] scan growth fwd {B} {N} {D} {S} {dtype}", flush=True)
    t, v = case(B, N, D, S, dtype, 50, 350)
    y, h = R().selective_scan_fwd(*(t[n] for n in NAMES), return_state=True)
    ry, rh = O.selective_scan(*(v[n] for n in NAMES))
    m = {n: np.abs(a) for n, a in v.items()}
    # |dt x| enters through x; dt is negative wherever x is not zero
    my, mh = O.selective_scan(-m["x"], v["dt"], v["A"], m["Bm"], m["Cm"])
    k = 8 * N + 4 * S + 64
    check(h, rh, np.abs(mh), k, "state")
    check(y, ry, np.abs(my), k, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,S", SIZES)
def test_backward(B, N, D, S, dtype):
    """No state enters the tokens that grow, and no adjoint: gradients in front of them only."""
    print(f"\n[case] scan growth bwd {B} {N} {D} {S} {dtype}", flush=True)
    lo, hi = 250, 450
    t, v = case(B, N, D, S, dtype, lo, hi)
    g, gr = draw(50, (B, N, D), dtype)
    g[:, lo:], gr[:, lo:] = 0, 0
    got = R().selective_scan_bwd(*(t[n] for n in NAMES), g, return_grad_state_in=True)
    args = (*(v[n] for n in NAMES), gr)
    assert np.abs(O.selective_scan_bwd(*args)[0][:, :lo]).min() > 0
    for i, (a, r, m) in enumerate(zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True))):
        if a is not None:
            check(a, r, m, 20 * N + 8 * S + 256, i)


@pytest.mark.parametrize("N", [700, 1600])
def test_a_tiny_state_grows(N):
    """A state of 2^-120 that grows by 2^5 a token over 40 tokens, 2^200 in all, and stays.  Of an
    exponent, log2(e), its product with A and that with dt are rounded, 3 u of it, so 3 u of 200
    in all (the sums of dt are whole numbers); each token's power and product add 3 u, 40 times:
    720 u, and the read-out's or the channels' sum of a few terms."""
    print(f"\n[case] scan growth tiny {N}", flush=True)
    D, S = 8, 4
    z = torch.zeros(1, N, D, device="cuda")
    dt = z.clone()
    dt[:, 60:100] = 5.0
    A = torch.full((D, S), float(np.log(2.0)), device="cuda")
    one = torch.ones(1, N, 1, S, device="cuda")
    s0 = torch.full((1, D, S), 2.0 ** -120, device="cuda")
    y, h = R().selective_scan_fwd(z, dt, A, one, one, state_in=s0, return_state=True)
    ref, rh = O.selective_scan(*(a.double().cpu().numpy() for a in (z, dt, A, one, one)), state_in=s0.double().cpu().numpy())
    assert np.isfinite(rh).all() and rh.min() > 2.0 ** 79
    check(h, rh, rh, 740, "state")
    check(y, ref, ref, 740, "y")
    g = torch.zeros(1, N, D, device="cuda")
    g[:, -1] = 2.0 ** -80
    got = R().selective_scan_bwd(z, dt, A, one, one, g, state_in=s0, return_grad_state_in=True)
    args = (*(a.double().cpu().numpy() for a in (z, dt, A, one, one, g)),)
    refs = O.selective_scan_bwd(*args, state_in=s0.double().cpu().numpy())
    check(got[8], refs[8], refs[8], 740, "grad_state_in")
    check(got[4], refs[4], refs[4], 740, "grad_C")
