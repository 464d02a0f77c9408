"""The selective scan cut into more than 48 segments, whose entry states sixteen waves compose: counts
just above that, not a multiple of 16 (waves with fewer segments than others, and with none), and
in the hundreds; (channel, state) pairs that leave lanes of the last workgroup idle; lengths that
end in any segment.  Bounds as in test_gpu_scan.py."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import check, draw  # noqa: E402
from test_gpu_scan import case, fwd_args, mags  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def segments(B, N, D, G, S):
    """Segments of a sequence, forward, by the workspace that they need."""
    floats = R().scan_workspace_bytes(B, N, D, G, S) // 4
    assert floats % (B * D * (S + 1)) == 0
    return floats // (B * D * (S + 1))


def segments_back(B, N, D, G, S):
    """The same of the backward (D / G up to the channels of a workgroup, one block a group)."""
    tiles = -(-N // 16)
    up = lambda n: -(-n // 4) * 4                                                # noqa: E731
    block = 64 if S <= 16 else 32 if S <= 32 else 16
    nblk = G * -(-(D // G) // block)
    have = R().scan_bwd_workspace_bytes(B, N, D, G, S) // 4
    fits = [n for n in range(2, tiles + 1) if
            2 * up(B * n * D * S) + up(B * n * D) + up(B * tiles * D * S) + up(B * tiles * D) + up(2 * nblk * B * N * S) +
            up(B * n * (S + 2) * D) == have]
    assert len(fits) == 1
    return fits[0]


CASES = [
    # B, N, D, G, S, segments forward and backward
    (1, 800, 37, 1, 5, 50, 50), (2, 816, 130, 2, 13, 51, 51), (1, 1040, 20, 1, 16, 65, 65), (1, 4100, 8, 2, 3, 171, 129),
    (2, 1600, 33, 1, 40, 100, 100), (1, 3300, 64, 1, 16, 138, 104),
]


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,G,S,fwd,bwd", CASES)
def test_forward(B, N, D, G, S, fwd, bwd, dtype):
    print(f"\n[case] scan segments fwd {B} {N} {D} {G} {S} {dtype}", flush=True)
    assert segments(B, N, D, G, S) == fwd > 48 and B * D * S <= 32768
    t, v = case(B, N, D, G, S, dtype, True, 900)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True)
    y, h = R().selective_scan_fwd(*fwd_args(t), state_in=t["state_in"], return_state=True, **kw)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"])
    my, mh = mags(v, True)
    k = 8 * N + 4 * S + 64
    check(h, rh, mh, k, "state")
    check(y, ry, my, k, "y")
    for _ in range(3):                       # the state in place, and the same bits from call to call
        state = t["state_in"].clone()
        y2, _ = R().selective_scan_fwd(*fwd_args(t), state_in=state, state_out=state, **kw)
        assert torch.equal(y2, y) and torch.equal(state, h)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,N,D,G,S,fwd,bwd", CASES)
def test_backward(B, N, D, G, S, fwd, bwd, dtype):
    print(f"\n[case] scan segments bwd {B} {N} {D} {G} {S} {dtype}", flush=True)
    assert segments_back(B, N, D, G, S) == bwd > 48
    t, v = case(B, N, D, G, S, dtype, True, 1000)
    g, gr = draw(1020, (B, N, D), dtype)
    gs, gsr = draw(1021, (B, D, S), "f32")
    run = lambda: R().selective_scan_bwd(*fwd_args(t), g, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True,  # noqa: E731
                                         state_in=t["state_in"], grad_state_out=gs, return_grad_state_in=True)
    got = run()
    args = (*fwd_args(v), gr, v["D"], v["z"], v["dt_bias"], True, v["state_in"], gsr)
    names = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_state_in")
    for a, r, m, nm in zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True), names):
        check(a, r, m, 20 * N + 8 * S + 256, nm)
    for a, b in zip(run(), got):
        assert torch.equal(a, b)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N", [800, 1611])
def test_lengths(N, dtype):
    """Sequences of no token, one, to the middle of a segment and of all, NaN behind their ends."""
    print(f"\n[case] scan segments lengths {N} {dtype}", flush=True)
    B, D, G, S = 5, 19, 1, 16
    assert segments(B, N, D, G, S) > 48 and segments_back(B, N, D, G, S) > 48
    n = [N, 0, 1, N // 2 + 5, N - 1]
    t, v = case(B, N, D, G, S, dtype, False, 1100)
    g, gr = draw(1120, (B, N, D), dtype)
    gs, gsr = draw(1121, (B, D, S), "f32")
    for i, m in enumerate(n):
        for x in (t["x"], t["dt"], t["z"], t["Bm"], t["Cm"], g):
            x[i, m:] = float("nan")
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True, state_in=t["state_in"], lengths=lengths)
    y, h = R().selective_scan_fwd(*fwd_args(t), **kw, return_state=True)
    ry, rh = O.selective_scan(*fwd_args(v), v["D"], v["z"], v["dt_bias"], True, v["state_in"], n)
    my, mh = mags(v, True, n)
    k = 8 * N + 4 * S + 64
    check(h, rh, mh, k, "state")
    check(y, ry, my, k, "y")                 # rows behind the ends are zero in both
    got = R().selective_scan_bwd(*fwd_args(t), g, **kw, grad_state_out=gs, return_grad_state_in=True)
    args = (*fwd_args(v), gr, v["D"], v["z"], v["dt_bias"], True, v["state_in"], gsr, n)
    for a, r, m in zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True)):
        check(a, r, m, 20 * N + 8 * S + 256)
