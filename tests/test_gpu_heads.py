"""Head norms with rotary positions and their gradients, against the fp64 oracle.

Counting roundings, in units of 2^-24: a row's sum of d squares d, the root and its reciprocal 4,
of which the root takes half; two products, the turn (8, of both of a pair's elements): d + 32
covers every element of the forward; the gradient's second sum d more.  A weight's gradient sums
over all rows, one term after another at most.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402
from proj_cases import pair_sizes  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


CASES = [
    # B, Hq, Hk, N, d, rot: whole heads and parts, packs and odd sizes, one token, no keys, keys with fewer heads,
    # more heads than a thread takes, more rows than workgroups
    (2, 3, 3, 37, 64, 64), (1, 4, 1, 100, 128, 64), (2, 2, 0, 9, 80, 80), (3, 1, 2, 5, 10, 6), (1, 1, 1, 1, 256, 256),
    (5, 32, 32, 1, 128, 128), (1, 20, 7, 300, 96, 48), (2, 2, 2, 33, 36, 34), (1, 2, 2, 7, 2, 2), (1, 1, 1, 4, 255, 2),
    (300, 17, 5, 4, 32, 32), (1, 1, 1, 5, 256, 128), (2, 1, 1, 3000, 16, 16),
]


def ref_sizes(x, weight, eps, rot, interleaved, scale):
    """(normalised rows, the sizes that the forward's errors are relative to)."""
    xh = x / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    w = 1.0 if weight is None else weight
    return xh, pair_sizes(xh * w, rot, interleaved) * scale


def bwd_sizes(x, g, weight, eps, rot, interleaved, scale):
    r = 1 / np.sqrt(np.mean(x * x, -1, keepdims=True) + eps)
    xh, v = np.abs(x) * r, pair_sizes(g, rot, interleaved) * scale
    vw = v * (1.0 if weight is None else np.abs(weight))
    return r * (vw + xh * np.mean(vw * xh, -1, keepdims=True)), (v * xh).sum((0, 1, 2))


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("B,Hq,Hk,N,d,rot", CASES)
def test_parity(B, Hq, Hk, N, d, rot, dtype, wtype, interleaved):
    print(f"\n[case] heads {B} {Hq} {Hk} {N} {d} {rot} {dtype}/{wtype} {interleaved}", flush=True)
    q, qr = draw(1, (B, Hq, N, d), dtype, 2.0)
    k, kr = draw(2, (B, Hk, N, d), dtype, 0.5) if Hk else (None, None)
    gq, gqr = draw(3, (B, Hq, N, d), dtype)
    gk, gkr = draw(4, (B, Hk, N, d), dtype) if Hk else (None, None)
    (qw, qwr), (kw, kwr) = draw(5, (d,), wtype), draw(6, (d,), wtype)
    freq = R().rotary_frequencies(rot)
    table = R().rotary_table(freq, N + 50)
    kw_ = dict(q_weight=qw, k_weight=kw if Hk else None, eps=1e-5, offset=50, interleaved=interleaved, q_scale=0.75, k_scale=0.1)
    got = R().head_norm_rotary_fwd(q, k, table, **kw_)
    got = got if Hk else (got, None)
    pos, f = np.arange(N) + 50, freq.numpy()
    for g, x, w, scale in ((got[0], qr, qwr, 0.75), (got[1], kr, kwr, 0.1)):
        if g is not None:
            check(g, O.head_norm_rotary(x, pos, f, w, 1e-5, interleaved, scale), ref_sizes(x, w, 1e-5, rot, interleaved, scale)[1],
                  d + 32)
    got = R().head_norm_rotary_bwd(q, k, table, gq, gk, **kw_)
    rows = B * N
    for g, gw, x, gr, w, scale, H in ((got[0], got[2], qr, gqr, qwr, 0.75, Hq), (got[1], got[3], kr, gkr, kwr, 0.1, Hk)):
        if g is None:
            assert gw is None
            continue
        assert gw.dtype == TYPES[wtype]
        rx, rw = O.head_norm_rotary_bwd(x, pos, f, gr, w, 1e-5, interleaved, scale)
        mx, mw = bwd_sizes(x, gr, w, 1e-5, rot, interleaved, scale)
        check(g, rx, mx, 2 * d + 64, "x")
        check(gw, rw, mw, rows * H + d + 64, "weight")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_positions_strides_and_in_place(dtype):
    print(f"\n[case] heads strides {dtype}", flush=True)
    B, H, N, d, rot = 3, 5, 11, 64, 32
    joint, _ = draw(7, (B, N, 3, H, d), dtype)           # q, k, v of one projection
    q, k = (joint[:, :, i].transpose(1, 2) for i in (0, 1))
    freq = R().rotary_frequencies(rot, base=500.0)
    table = R().rotary_table(freq, 40)
    pos = torch.randint(0, 40, (B, N), device="cuda")
    w = draw(8, (d,), "f32")[0]
    ref = R().head_norm_rotary_fwd(q.contiguous(), k.contiguous(), table, w, None, positions=pos)
    o = O.head_norm_rotary(q.double().cpu().numpy(), pos.cpu().numpy(), freq.numpy(), w.double().cpu().numpy(), 1e-6)
    check(ref[0], o, ref_sizes(q.double().cpu().numpy(), w.double().cpu().numpy(), 1e-6, rot, True, 1.0)[1], d + 32)
    out = R().head_norm_rotary_fwd(q, k, table, w, None, positions=pos)
    assert all(torch.equal(a, b) for a, b in zip(out, ref))
    for i in range(B):                                   # one row of positions for all sequences
        one = R().head_norm_rotary_fwd(q[i:i + 1], k[i:i + 1], table, w, None, positions=pos[i])
        assert torch.equal(one[0], ref[0][i:i + 1]) and torch.equal(one[1], ref[1][i:i + 1])
    gq, gk = (draw(9 + i, (B, N, H, d), dtype)[0].transpose(1, 2) for i in (0, 1))
    a = R().head_norm_rotary_bwd(q, k, table, gq, gk, w, None, positions=pos)
    b = R().head_norm_rotary_bwd(q.contiguous(), k.contiguous(), table, gq.contiguous(), gk.contiguous(), w, None, positions=pos)
    assert all(torch.equal(u, v) for u, v in zip(a[:3], b[:3])) and a[3] is None
    c = R().head_norm_rotary_bwd(q, k, table, gq, gk, w, None, positions=pos, out_q=gq, out_k=gk)
    assert c[0] is gq and torch.equal(gq, a[0]) and torch.equal(gk, a[1]) and torch.equal(c[2], a[2])
    v = joint[:, :, 2].clone()
    R().head_norm_rotary_fwd(q, k, table, w, None, positions=pos, out_q=q, out_k=k)       # in the joint rows
    assert torch.equal(q, ref[0]) and torch.equal(k, ref[1]) and torch.equal(joint[:, :, 2], v)


def test_unknown_positions_and_rows_of_zeros():
    print("\n[case] heads unknown positions", flush=True)
    table = R().rotary_table(R().rotary_frequencies(16), 8)
    q = draw(20, (1, 2, 4, 24), "f32")[0]
    q[0, 0, 1] = 0
    pos = torch.tensor([0, 1, 8, -1], device="cuda")
    y = R().head_norm_rotary_fwd(q, None, table, positions=pos)
    assert torch.isnan(y[:, :, 2:, :16]).all() and torch.isfinite(y[:, :, 2:, 16:]).all() and torch.isfinite(y[:, :, :2]).all()
    assert not y[0, 0, 1].any()
    z = R().head_norm_rotary_fwd(torch.zeros_like(q), None, table, eps=0.0)     # 0 / 0
    assert torch.isnan(z).all()


def test_nothing_to_do():
    print("\n[case] heads empty", flush=True)
    table = R().rotary_table(R().rotary_frequencies(16), 8)
    w = torch.ones(24, device="cuda")
    for shape in ((0, 2, 4, 24), (2, 2, 0, 24), (2, 0, 4, 24)):
        q = torch.empty(shape, device="cuda")
        assert R().head_norm_rotary_fwd(q, None, table, w).shape == shape
        g = R().head_norm_rotary_bwd(q, None, table, q, None, w)
        assert g[0].shape == shape and not g[2].any()


def test_repeats_bit_for_bit():
    print("\n[case] heads repeat", flush=True)
    table = R().rotary_table(R().rotary_frequencies(64), 500)
    q, g = draw(30, (2, 9, 500, 128), "bf16")[0], draw(31, (2, 9, 500, 128), "bf16")[0]
    w = draw(32, (128,), "bf16")[0]
    a, b = (R().head_norm_rotary_bwd(q, q, table, g, g, w, w) for _ in range(2))
    assert all(torch.equal(u, v) for u, v in zip(a, b))
