"""The gated feed-forward block and its gradients, against the fp64 oracle (bounds: proj_cases)."""
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402
from proj_cases import ffn_bounds, ffn_bwd_bounds, ffn_y_bound  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


# one token; widths that are whole and cut units; tiles cut in each direction; few tokens; many
SIZES = [(1, 1, 1), (1, 64, 128), (2, 30, 50), (7, 256, 512), (16, 128, 200), (50, 77, 129), (128, 128, 256), (129, 96, 136),
         (300, 264, 392), (260, 65, 1111), (1000, 40, 24)]


def make(M, D, F, dtype, seed=0):
    shapes = [((M, D), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((D, F), F ** -0.5), ((M, D), 1.0)]
    both = [draw(seed + i, s, dtype, c) for i, (s, c) in enumerate(shapes)]
    return [b[0] for b in both], [b[1] for b in both]


@pytest.mark.parametrize("act", ["silu", "gelu", "gelu_tanh", "relu", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", SIZES)
def test_forward(M, D, F, dtype, act):
    print(f"\n[case] ffn {M} {D} {F} {dtype} {act}", flush=True)
    (x, wg, wu, wd, r), (xr, gr, ur, dr, rr) = make(M, D, F, dtype)
    y, g, u = R().gated_ffn_fwd(x, wg, wu, wd, residual=r, activation=act, return_pre=True)
    ry, rg, ru = O.gated_ffn(xr, gr, ur, dr, rr, act)
    bg, bu = ffn_bounds(xr, gr, ur, dr, rr, act, dtype)
    check(g, rg, bg, 1, "gate")
    check(u, ru, bu, 1, "up")
    check(y, ry, ffn_y_bound(rg, ru, bg, bu, dr, rr, act, dtype), 1, "y")
    bare = R().gated_ffn_fwd(x, wg, wu, wd, activation=act)
    check(bare, O.gated_ffn(xr, gr, ur, dr, None, act)[0], ffn_y_bound(rg, ru, bg, bu, dr, None, act, dtype), 1, "bare")


@pytest.mark.parametrize("act", ["silu", "gelu", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", SIZES + [(3000, 64, 64), (2500, 33, 70)])
def test_backward(M, D, F, dtype, act):
    print(f"\n[case] ffn bwd {M} {D} {F} {dtype} {act}", flush=True)
    (x, wg, wu, wd, gy), (xr, gr, ur, dr, yr) = make(M, D, F, dtype, 10)
    g, gtr = draw(16, (M, F), dtype, 1.5)
    u, upr = draw(17, (M, F), dtype)
    got = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy, activation=act)
    ref = O.gated_ffn_bwd(xr, gr, ur, dr, gtr, upr, yr, act)
    for a, b, m, what in zip(got, ref, ffn_bwd_bounds(xr, gr, ur, dr, gtr, upr, yr, act, dtype),
                             ("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")):
        check(a, b, m, 1, what)
    gx = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy, activation=act, weight_grad=False)
    assert torch.equal(gx[0], got[0]) and gx[1:] == (None, None, None)
    gw = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy, activation=act, x_grad=False)
    assert gw[0] is None and all(torch.equal(a, b) for a, b in zip(gw[1:], got[1:]))


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_slices_and_odd_addresses(dtype):
    print(f"\n[case] ffn slices {dtype}", flush=True)
    D, F = 64, 96
    for off in (0, 1):
        buf, br = draw(20, (2, 45, 150), dtype)
        x, xr = buf[..., off:off + D], br[..., off:off + D].reshape(90, D)
        flat, fr = draw(21, (off + 3 * D * F,), dtype, 0.1)
        # one weight at an odd address, the others not
        wg, gr = flat[off:off + D * F].view(F, D), fr[off:off + D * F].reshape(F, D)
        wu, ur = draw(22, (F, D), dtype, 0.1)
        wd, dr = draw(23, (D, F), dtype, 0.1)
        y, g, u = R().gated_ffn_fwd(x, wg, wu, wd, return_pre=True)
        ry, rg, ru = O.gated_ffn(xr, gr, ur, dr)
        bg, bu = ffn_bounds(xr, gr, ur, dr, None, "silu", dtype)
        check(y.view(90, D), ry, ffn_y_bound(rg, ru, bg, bu, dr, None, "silu", dtype), 1, "y")
        gy, yr = draw(24, (2, 45, D), dtype)
        yr = yr.reshape(90, D)
        got = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy)
        gk, uk = (v.double().cpu().numpy().reshape(90, F) for v in (g, u))
        ref = O.gated_ffn_bwd(xr, gr, ur, dr, gk, uk, yr)
        for a, b, m in zip((got[0].view(90, D),) + got[1:], ref, ffn_bwd_bounds(xr, gr, ur, dr, gk, uk, yr, "silu", dtype)):
            check(a, b, m, 1)


def test_residual_in_place():
    print("\n[case] ffn in place", flush=True)
    (x, wg, wu, wd, r), _ = make(70, 136, 200, "bf16", 30)
    y = R().gated_ffn_fwd(x, wg, wu, wd, residual=r)
    r2 = r.clone()
    assert R().gated_ffn_fwd(x, wg, wu, wd, residual=r2, out=r2) is r2 and torch.equal(r2, y)


def test_no_rows():
    print("\n[case] ffn without rows", flush=True)
    for t in TYPES.values():
        x = torch.empty(0, 24, device="cuda", dtype=t)
        wg, wd = torch.ones(40, 24, device="cuda", dtype=t), torch.ones(24, 40, device="cuda", dtype=t)
        y, g, u = R().gated_ffn_fwd(x, wg, wg, wd, return_pre=True)
        assert y.shape == (0, 24) and g.shape == u.shape == (0, 40)
        got = R().gated_ffn_bwd(x, wg, wg, wd, g, u, y)
        assert got[0].shape == (0, 24) and not any(v.any() for v in got[1:])


def test_nan_stays_in_its_row():
    print("\n[case] ffn NaN", flush=True)
    (x, wg, wu, wd, r), _ = make(140, 72, 100, "bf16", 40)
    clean = R().gated_ffn_fwd(x, wg, wu, wd, residual=r)
    x[139, 71] = float("nan")
    y = R().gated_ffn_fwd(x, wg, wu, wd, residual=r)
    assert torch.isnan(y[139]).all() and torch.equal(y[:139], clean[:139])


@pytest.mark.parametrize("M,D,F", [(4096, 512, 2048), (3000, 520, 1368)])
def test_many_tiles(M, D, F):
    """Enough tiles for every size of them, against products in fp64 on the GPU."""
    print(f"\n[case] ffn many {M} {D} {F}", flush=True)
    (x, wg, wu, wd, r), _ = make(M, D, F, "bf16", 50)
    y, g, u = R().gated_ffn_fwd(x, wg, wu, wd, residual=r, return_pre=True)
    xd, gd, ud, dd = (v.double() for v in (x, wg, wu, wd))
    # products in fp64, the operator's roundings (gate, up: bf16 as they are returned; product: bf16)
    rg, ru = xd @ gd.T, xd @ ud.T
    for got, ref, w in ((g, rg, gd), (u, ru, ud)):
        assert ((got.double() - ref).abs() <= 2.0 ** -8 * ref.abs() + 2.0 ** -24 * (2 * D + 16) * (xd.abs() @ w.abs().T)).all()
    h = rg * torch.sigmoid(rg) * ru
    ry = h @ dd.T + r.double()
    room = 2.0 ** -8 * (ry.abs() + 1.05 * h.abs() @ dd.abs().T) + 2.0 ** -24 * (2 * F + 16) * (h.abs() @ dd.abs().T)
    room = room + 2.0 ** -24 * 2 * (2 * D + 40) * ((xd.abs() @ gd.abs().T) * ru.abs() + (xd.abs() @ ud.abs().T) * rg.abs()) @ dd.abs().T
    assert ((y.double() - ry).abs() <= room).all()
    gy = torch.randn(M, D, device="cuda").bfloat16()
    got = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy)
    yd, gk, uk = gy.double(), g.double(), u.double()
    s = torch.sigmoid(gk)
    gh = yd @ dd
    gg, gu, h = gh * uk * (s + gk * s * (1 - s)), gh * gk * s, gk * s * uk
    refs = (gg @ gd + gu @ ud, gg.T @ xd, gu.T @ xd, yd.T @ h)
    eh = 2.0 ** -24 * (2 * D + 64) * (yd.abs() @ dd.abs())
    eg = eh * uk.abs() * 1.2 + 2.0 ** -8 * 1.01 * gg.abs()
    eu = eh * gk.abs() + 2.0 ** -8 * 1.01 * gu.abs()
    n = 2.0 ** -24 * (2 * M + 4 * F + 16)
    rooms = (eg @ gd.abs() + eu @ ud.abs() + n * (gg.abs() @ gd.abs() + gu.abs() @ ud.abs()),
             eg.T @ xd.abs() + n * gg.abs().T @ xd.abs(), eu.T @ xd.abs() + n * gu.abs().T @ xd.abs(),
             yd.abs().T @ (2.0 ** -8 * 1.01 * h.abs() + 2.0 ** -24 * 24 * gk.abs() * uk.abs()) + n * yd.abs().T @ h.abs())
    for a, b, m in zip(got, refs, rooms):
        assert ((a.double() - b).abs() <= 2.0 ** -8 * b.abs() + 1.05 * m).all()


@pytest.mark.parametrize("F", [100, 101, 104])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_infinities_do_not_meet_padding(dtype, F):
    """Everything positive: an infinity in a row makes that row infinite, not NaN, whether or not
    the hidden width is a multiple of 16 bytes."""
    M, D = 40, 72
    gen = torch.Generator().manual_seed(5)
    t = lambda *s: (torch.rand(s, generator=gen) * 0.1 + 0.01).to("cuda", TYPES[dtype])
    x, gy, wg, wu, wd = t(M, D), t(M, D), t(F, D), t(F, D), t(D, F)
    clean, gate, up = R().gated_ffn_fwd(x, wg, wu, wd, return_pre=True)
    grad = R().gated_ffn_bwd(x, wg, wu, wd, gate, up, gy)[0]
    x2, gy2 = x.clone(), gy.clone()
    x2[39, 3] = gy2[39, 3] = float("inf")
    y = R().gated_ffn_fwd(x2, wg, wu, wd)
    assert torch.isposinf(y[39]).all() and torch.equal(y[:39], clean[:39])
    g = R().gated_ffn_bwd(x, wg, wu, wd, gate, up, gy2)[0]
    assert torch.isposinf(g[39]).all() and torch.equal(g[:39], grad[:39])
