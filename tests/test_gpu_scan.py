"""The selective scan, forward, backward and one token, against the fp64 oracle.

Counting roundings: a step multiplies the state by a decay that is off by (3 + 2 |dt A|) u and
adds one term of 12 roundings (softplus, two products); what is left of a state after the sum
of |dt A| reached L is e^-L of it, and L e^-L <= 0.4, so N steps are off by at most 8 N u
relative to the recurrence over absolute values, plus the read-out's sum over S states and the
gate: k = 8 N + 4 S + 64.  Backward: the same once more for the adjoint, and sums over 64
channels and their blocks, or over tokens: k = 20 N + 8 S + 256.  The gate's derivative
s + z s (1 - s) crosses zero at z = -1.2785, where its two terms are 0.218 each and the
roundings of both stay: its magnitude is the sum of theirs, not |their sum| (at z = -1.278493
that sum is 6e-6, and half a step of 0.218 already 2e-3 of it).
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


def case(B, N, D, G, S, dtype, wide=False, seed=0):
    """Inputs as (tensors, fp64 values): dt around softplus(-3), decays that last from a token
    to the whole sequence."""
    t, v = {}, {}

    def put(name, shape, dt_=dtype, scale=1.0, cut=None):
        t[name], v[name] = draw(seed + len(t), shape, dt_, scale)
        if cut is not None:
            t[name], v[name] = t[name][..., cut:cut + D], v[name][..., cut:cut + D]

    put("x", (B, N, 2 * D) if wide else (B, N, D), cut=D if wide else None)
    put("z", (B, N, 2 * D) if wide else (B, N, D), cut=0 if wide else None)
    put("dt", (B, N, D))
    bc, bcv = draw(seed + 50, (B, N, 3 + 2 * G * S) if wide else (B, N, 2 * G * S), dtype)
    o = 3 if wide else 0
    for i, nm in enumerate(("Bm", "Cm")):
        lo = o + i * G * S
        t[nm], v[nm] = bc[..., lo:lo + G * S].unflatten(-1, (G, S)), bcv[..., lo:lo + G * S].reshape(B, N, G, S)
    if not wide:
        t["Bm"], t["Cm"] = t["Bm"].contiguous(), t["Cm"].contiguous()
    a = -np.exp(np.random.default_rng(seed + 60).uniform(-3, 3, (D, S)))
    t["A"] = torch.tensor(a).float().cuda()
    v["A"] = t["A"].double().cpu().numpy()
    put("D", (D,), "f32")
    put("dt_bias", (D,), "f32")
    t["dt_bias"] -= 3
    v["dt_bias"] = t["dt_bias"].double().cpu().numpy()
    put("state_in", (B, D, S), "f32")
    return t, v


def fwd_args(t, names=("x", "dt", "A", "Bm", "Cm")):
    return tuple(t[n] for n in names)


def mags(v, sp, lengths=None, gate=True):
    """The recurrence over absolute values: (y, state)."""
    m = {n: np.abs(v[n]) for n in ("x", "Bm", "Cm", "D", "state_in")}
    raw = v["dt"] + v["dt_bias"]
    dt = O.softplus(raw) if sp else raw
    N = v["x"].shape[1]
    # absolute inputs with the decays as they are: |dt x| enters through x
    x = m["x"] * np.abs(dt) / np.where(dt == 0, 1, dt)
    y, h = O.selective_scan(x, dt, v["A"], m["Bm"], m["Cm"], None, None, None, False, m["state_in"], lengths)
    y = np.abs(y) + m["D"] * m["x"]
    if gate:
        z = v["z"]
        y = y * np.abs(z) * (0.5 + 0.5 * np.tanh(z / 2))
    return y, np.abs(h)


CASES = [
    # B, N, D, G, S, wide: one token, odd channels and states, groups smaller than a
    # workgroup's channels, tiles that end inside, enough tokens for several segments
    (1, 1, 1, 1, 1, False), (2, 3, 5, 1, 16, False), (1, 33, 64, 1, 16, True), (2, 70, 100, 2, 16, False),
    (1, 64, 96, 3, 8, True), (2, 40, 48, 1, 32, False), (1, 50, 40, 2, 20, True), (1, 45, 24, 1, 64, False),
    (1, 37, 17, 1, 47, True), (1, 600, 66, 1, 16, False), (1, 300, 20, 1, 33, False), (1, 520, 12, 4, 4, True),
    (3, 129, 130, 1, 13, False), (2, 40, 128, 1, 8, False), (1, 90, 36, 1, 8, True), (40, 33, 260, 2, 16, False),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,G,S,wide", CASES)
def test_forward(B, N, D, G, S, wide, dtype):
    print(f"\n[case] scan fwd {B} {N} {D} {G} {S} {wide} {dtype}", flush=True)
    t, v = case(B, N, D, G, S, dtype, wide)
    y, h = R().selective_scan_fwd(*fwd_args(t), D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True,
                                  state_in=t["state_in"], return_state=True)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"])
    my, mh = mags(v, True)
    k = 8 * N + 4 * S + 64
    check(h, rh, mh, k, "state")
    check(y, ry, my, k, "y")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,G,S", [(2, 50, 70, 1, 16), (1, 300, 8, 2, 5)])
def test_forward_with_nothing_optional(B, N, D, G, S, dtype):
    print(f"\n[case] scan fwd plain {B} {N} {D} {G} {S} {dtype}", flush=True)
    t, v = case(B, N, D, G, S, dtype, False, 5)
    t["dt"], v["dt"] = t["dt"].abs() * 0.25, np.abs(v["dt"]) * 0.25      # a quarter is exact in either type
    y = R().selective_scan_fwd(*fwd_args(t))
    ry, _ = O.selective_scan(*fwd_args(v))
    v["D"], v["dt_bias"], v["state_in"] = np.zeros(D), np.zeros(D), np.zeros((B, D, S))
    check(y, ry, mags(v, False, gate=False)[0], 8 * N + 4 * S + 64)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,G,S,wide", CASES)
def test_backward(B, N, D, G, S, wide, dtype):
    print(f"\n[case] scan bwd {B} {N} {D} {G} {S} {wide} {dtype}", flush=True)
    t, v = case(B, N, D, G, S, dtype, wide, 100)
    g, gr = draw(200, (B, N, D), dtype)
    gs, gsr = draw(201, (B, D, S), "f32")
    got = R().selective_scan_bwd(*fwd_args(t), g, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True,
                                 state_in=t["state_in"], grad_state_out=gs, return_grad_state_in=True)
    args = (*fwd_args(v), gr, v["D"], v["z"], v["dt_bias"], True, v["state_in"], gsr)
    names = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_state_in")
    for a, r, m, nm in zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True), names):
        check(a, r, m, 20 * N + 8 * S + 256, nm)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_backward_with_nothing_optional(dtype):
    print(f"\n[case] scan bwd plain {dtype}", flush=True)
    B, N, D, G, S = 2, 50, 70, 1, 16
    t, v = case(B, N, D, G, S, dtype, False, 5)
    t["dt"], v["dt"] = t["dt"].abs() * 0.25, np.abs(v["dt"]) * 0.25
    g, gr = draw(210, (B, N, D), dtype)
    got = R().selective_scan_bwd(*fwd_args(t), g)
    assert [x is None for x in got] == [False] * 5 + [True] * 3
    ref, mag = (O.selective_scan_bwd(*fwd_args(v), gr, magnitude=m) for m in (False, True))
    for a, r, m in zip(got[:5], ref, mag):
        check(a, r, m, 20 * N + 8 * S + 256)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [70, 530])
def test_lengths(N, dtype):
    """Padded sequences, of no token and of all of them among them, ending in the first, a
    middle and the last segment; NaN behind the ends."""
    print(f"\n[case] scan lengths {N} {dtype}", flush=True)
    n = [N, 0, 1, 33, N - 1]
    B, D, G, S = 5, 20, 1, 16
    t, v = case(B, N, D, G, S, dtype, False, 300)
    g, gr = draw(310, (B, N, D), dtype)
    gs, gsr = draw(311, (B, D, S), "f32")
    for i, m in enumerate(n):
        for x in (t["x"], t["dt"], t["z"], t["Bm"], t["Cm"], g):
            x[i, m:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True, state_in=t["state_in"], lengths=lengths)
    out = torch.full((B, N, D), 7.0, dtype=t["x"].dtype, device="cuda")
    y, h = R().selective_scan_fwd(*fwd_args(t), **kw, return_state=True, out=out)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"], n)
    my, mh = mags(v, True, n)
    k = 8 * N + 4 * S + 64
    check(h, rh, mh, k, "state")
    for i, m in enumerate(n):
        check(y[i, :m], ry[i, :m], my[i, :m], k, "y")
        assert bool((y[i, m:] == 7).all())
    got = R().selective_scan_bwd(*fwd_args(t), g, **kw, grad_state_out=gs, return_grad_state_in=True)
    args = (*fwd_args(v), gr, v["D"], v["z"], v["dt_bias"], True, v["state_in"], gsr, n)
    for a, r, m in zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True)):
        check(a, r, m, 20 * N + 8 * S + 256)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,D,G,S", [(1, 1, 1, 1), (3, 70, 2, 16), (2, 33, 1, 5), (4, 64, 1, 32), (2, 20, 1, 61),
                                     (128, 256, 1, 16)])
def test_step_continues_a_prompt(B, D, G, S, dtype):
    """Tokens one at a time from a prompt's state: the recurrence of the whole sequence."""
    print(f"\n[case] scan step {B} {D} {G} {S} {dtype}", flush=True)
    N, cut = 9, 4
    t, v = case(B, N, D, G, S, dtype, True, 400)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"])
    my, mh = mags(v, True)
    seq = ("x", "dt", "z", "Bm", "Cm")
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], softplus=True)
    a = {m: t[m][:, :cut].contiguous() for m in seq}
    _, state = R().selective_scan_fwd(a["x"], a["dt"], t["A"], a["Bm"], a["Cm"], z=a["z"], state_in=t["state_in"],
                                      return_state=True, **kw)
    k = 8 * N + 4 * S + 64
    for i in range(cut, N):
        s = {m: t[m][:, i] for m in seq}
        y = R().selective_scan_step(s["x"], s["dt"], t["A"], s["Bm"], s["Cm"], state, z=s["z"], **kw)
        check(y, ry[:, i], my[:, i], k, f"y {i}")
    check(state, rh, mh, k, "state")


def test_state_in_place_and_split():
    """A prompt in two parts, the state updated in place, against the whole sequence's recurrence.
    (Not bit for bit against one call: a sequence may be cut into segments that the parts are
    not, and a segment's entry state is composed, which rounds in another order.)"""
    print("\n[case] scan in place", flush=True)
    t, v = case(2, 128, 70, 1, 16, "bf16", False, 500)
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], softplus=True)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"])
    my, mh = mags(v, True)
    state, ys = t["state_in"].clone(), []
    for lo in (0, 64):
        p = {m: t[m][:, lo:lo + 64].contiguous() for m in ("x", "dt", "z", "Bm", "Cm")}
        got = R().selective_scan_fwd(p["x"], p["dt"], t["A"], p["Bm"], p["Cm"], z=p["z"], state_in=state, state_out=state,
                                     **kw)
        ys.append(got[0])
        assert got[1] is state
    k = 8 * 128 + 4 * 16 + 64
    check(torch.cat(ys, 1), ry, my, k, "y")
    check(state, rh, mh, k, "state")
    # segmented, in place: the entry states are composed before any state is written
    t, v = case(1, 700, 12, 1, 16, "f32", False, 510)
    kw = dict(D=t["D"], dt_bias=t["dt_bias"], softplus=True)
    y, h = R().selective_scan_fwd(*fwd_args(t), state_in=t["state_in"], return_state=True, **kw)
    assert R().scan_workspace_bytes(1, 700, 12, 1, 16) > 0
    state = t["state_in"].clone()
    y2, _ = R().selective_scan_fwd(*fwd_args(t), state_in=state, state_out=state, **kw)
    assert torch.equal(y2, y) and torch.equal(state, h)


def test_extreme_step_sizes():
    """Steps that forget everything or keep everything, raw values far out on both sides."""
    print("\n[case] scan extreme steps", flush=True)
    B, N, D, S = 1, 40, 8, 16
    t, v = case(B, N, D, 1, S, "f32", False, 520)
    raw = np.array([-200.0, -100, -30, 0, 15, 25, 90, 200])
    t["dt"] = torch.tensor(np.broadcast_to(raw, (B, N, D)).copy()).float().cuda()
    v["dt"] = t["dt"].double().cpu().numpy()
    v["dt_bias"] = np.zeros(D)
    y, h = R().selective_scan_fwd(*fwd_args(t), softplus=True, state_in=t["state_in"], return_state=True)
    ry, rh = O.selective_scan(*fwd_args(v), None, None, None, True, v["state_in"])
    v["D"] = np.zeros(D)
    my, mh = mags(v, True, gate=False)
    k = 8 * N + 4 * S + 64
    check(h, rh, mh, k, "state")
    check(y, ry, my, k, "y")


def test_no_tokens():
    print("\n[case] scan without tokens", flush=True)
    t, _ = case(2, 3, 16, 1, 16, "bf16", False, 530)
    cut = {m: t[m][:, :0].contiguous() for m in ("x", "dt", "z", "Bm", "Cm")}
    a = (cut["x"], cut["dt"], t["A"], cut["Bm"], cut["Cm"])
    y, h = R().selective_scan_fwd(*a, state_in=t["state_in"], return_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(h, t["state_in"])
    gs = torch.randn(2, 16, 16, device="cuda")
    got = R().selective_scan_bwd(*a, cut["x"], D=t["D"], dt_bias=t["dt_bias"], state_in=t["state_in"], grad_state_out=gs,
                                 return_grad_state_in=True)
    assert not got[2].any() and not got[5].any() and not got[7].any() and torch.equal(got[8], gs)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,S", [(40, 16), (300, 16), (90, 13), (50, 64)])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_channels_do_not_meet(N, S, dtype, bad):
    """A channel whose inputs are NaN or infinite leaves every other channel's results as they
    are, bit for bit (the gradients of B, C and the sums over channels are the exception)."""
    print(f"\n[case] scan channels {N} {S} {dtype} {bad}", flush=True)
    B, D, G, c = 2, 70, 1, 5
    t, _ = case(B, N, D, G, S, dtype, False, 700)
    g, _ = draw(720, (B, N, D), dtype)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True, state_in=t["state_in"])

    def run():
        y, h = R().selective_scan_fwd(*fwd_args(t), **kw, return_state=True)
        b = R().selective_scan_bwd(*fwd_args(t), g, **kw, return_grad_state_in=True)
        return {"y": y, "state": h.transpose(1, 2), "gx": b[0], "gdt": b[1], "gA": b[2].t(), "gD": b[5], "gz": b[6],
                "gbias": b[7], "gstate": b[8].transpose(1, 2)}

    want = {n: v.clone() for n, v in run().items()}
    t["x"][:, N // 3, c] = bad
    got = run()
    assert not bool(torch.isfinite(got["y"][..., c]).all())
    for n, v in got.items():
        w = want[n].clone()
        w[..., c] = v[..., c] = 0
        assert torch.equal(v, w), n
