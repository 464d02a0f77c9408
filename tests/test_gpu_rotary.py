"""Rotary positions against complex multiplication in fp64.

Counting roundings: cosine and sine (u each), two products, a sum, the scale: k = 8 relative to
(|a| + |b|) times the scales covers either element of a pair.
"""
import math

import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import check, draw  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def sizes(x, rot, interleaved):
    """|a| + |b| of each element's pair."""
    m = np.abs(x).copy()
    if interleaved:
        s = m[..., 0:rot:2] + m[..., 1:rot:2]
        m[..., 0:rot:2] = m[..., 1:rot:2] = s
    else:
        s = m[..., :rot // 2] + m[..., rot // 2:rot]
        m[..., :rot // 2] = m[..., rot // 2:rot] = s
    return m


CASES = [
    # B, Hq, Hk, N, d, rot: whole heads and parts, packs and odd sizes, one token, keys with
    # fewer heads, more heads than a thread takes
    (2, 3, 3, 37, 64, 64), (1, 4, 1, 100, 128, 64), (2, 2, 0, 9, 80, 80), (3, 1, 2, 5, 10, 6), (1, 1, 1, 1, 256, 256),
    (5, 32, 32, 1, 128, 128), (1, 20, 7, 300, 96, 48), (2, 2, 2, 33, 36, 34), (1, 2, 2, 7, 2, 2), (1, 1, 1, 4, 255, 2),
    (300, 17, 5, 4, 32, 32),
]


@pytest.mark.parametrize("back", [False, True])
@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", CASES)
def test_parity(B, Hq, Hk, N, d, rot, dtype, interleaved, back):
    print(f"\n[case] rotary {B} {Hq} {Hk} {N} {d} {rot} {dtype} {interleaved} {back}", flush=True)
    q, qr = draw(1, (B, Hq, N, d), dtype)
    k, kr = draw(2, (B, Hk, N, d), dtype) if Hk else (None, None)
    freq = R().rotary_frequencies(rot)
    table = R().rotary_table(freq, N + 50)
    f = R().rotary_bwd if back else R().rotary_fwd
    got = f(q, k, table, offset=50, interleaved=interleaved, q_scale=0.75, k_scale=0.1)
    got = got if Hk else (got, None)
    for g, x, scale in ((got[0], qr, 0.75), (got[1], kr, 0.1)):
        if g is not None:
            ref = O.rotary(x, np.arange(N) + 50, freq.numpy(), interleaved, scale, backward=back)
            check(g, ref, sizes(x, rot, interleaved) * scale, 8)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_strides_and_in_place(dtype):
    print(f"\n[case] rotary strides {dtype}", flush=True)
    B, H, N, d, rot = 3, 5, 11, 64, 32
    joint, _ = draw(3, (B, N, 3, H, d), dtype)          # q, k, v of one projection
    q, k = (joint[:, :, i].transpose(1, 2) for i in (0, 1))
    freq = R().rotary_frequencies(rot, base=500.0)
    table = R().rotary_table(freq, 70)
    pos = torch.randint(0, 70, (B, N), device="cuda")
    for p in (pos, pos[0].contiguous()):
        got = R().rotary_fwd(q, k, table, positions=p)
        for g, x in zip(got, (q, k)):
            assert g.is_contiguous()
            xr = x.double().cpu().numpy()
            check(g, O.rotary(xr, p.cpu().numpy(), freq.numpy()), sizes(xr, rot, True), 8)
    v_before, want = joint[:, :, 2].clone(), R().rotary_fwd(q, k, table, positions=pos)
    out = R().rotary_fwd(q, k, table, positions=pos, out_q=q, out_k=k)     # both inside the joint rows
    assert out[0] is q and torch.equal(q, want[0]) and torch.equal(k, want[1])
    assert torch.equal(joint[:, :, 2], v_before)


def test_backward_undoes_the_rotation():
    print("\n[case] rotary there and back", flush=True)
    q, qr = draw(4, (2, 3, 50, 64), "f32")
    freq = R().rotary_frequencies(64)
    table = R().rotary_table(freq, 50)
    back = R().rotary_bwd(R().rotary_fwd(q, None, table), None, table)
    check(back, qr, sizes(sizes(qr, 64, True), 64, True), 20)


def test_far_positions_and_scalings():
    """The table is what fp64 gives at positions of millions, for every scaling."""
    print("\n[case] rotary table", flush=True)
    first, n = 3_000_000, 100
    for scaling in ("none", "linear", "base", "ramp"):
        freq = R().rotary_frequencies(64, scaling=scaling, factor=8.0, original_length=4096)
        t = R().rotary_table(freq, n, first=first, magnitude=1.25).double().cpu().numpy()
        ang = (first + np.arange(n))[:, None] * freq.numpy()
        ref = 1.25 * np.stack((np.cos(ang), np.sin(ang)), -1)
        # one rounding to fp32, and an angle of 3e6 that two fp64 products may round apart by 2^-31
        assert np.max(np.abs(t - ref)) <= 1.25 * (2.0 ** -24 + 2.0 ** -30)


def test_frequencies():
    f = R().rotary_frequencies(8).numpy()
    assert np.allclose(f, 10000.0 ** (-np.arange(4) / 4))
    assert np.allclose(R().rotary_frequencies(8, scaling="linear", factor=4).numpy(), f / 4)
    b = R().rotary_frequencies(8, scaling="base", factor=4).numpy()
    assert np.isclose(b[0], f[0]) and np.isclose(b[-1], f[-1] / 4)
    r = R().rotary_frequencies(8, scaling="ramp", factor=4, original_length=int(2 * math.pi * 16), fast=8, slow=1).numpy()
    # 16, 1.6, 0.16, 0.016 turns: left alone, blended, divided, divided
    assert np.isclose(r[0], f[0]) and f[1] / 4 < r[1] < f[1] and np.allclose(r[2:], f[2:] / 4)


def test_unknown_positions_give_nan_rows_only():
    print("\n[case] rotary unknown positions", flush=True)
    q, _ = draw(5, (1, 2, 6, 16), "bf16")
    table = R().rotary_table(R().rotary_frequencies(8), 10)
    pos = torch.tensor([0, -1, 9, 10, 3, 1 << 40], device="cuda")
    got = R().rotary_fwd(q, None, table, positions=pos)
    bad = torch.tensor([False, True, False, True, False, True], device="cuda")
    assert torch.isnan(got[:, :, bad, :8]).all() and not torch.isnan(got[:, :, ~bad]).any()
    assert torch.equal(got[..., 8:], q[..., 8:])


def test_empty():
    q = torch.empty(0, 3, 5, 16, device="cuda")
    table = R().rotary_table(R().rotary_frequencies(16), 5)
    assert R().rotary_fwd(q, None, table).shape == q.shape
    assert R().rotary_table(R().rotary_frequencies(16), 0).shape == (0, 8, 2)
