"""Layer normalisation, forward and backward, against the fp64 oracle.

Counting roundings: a sum over D columns is at most D / 256 terms in a lane's order (wide
rows) or 64 and then a tree of 10 levels; with the elementwise steps, k = 128 covers every
width here.  The deviation x - mean is rounded relative to its operands.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def case(rows, D, dtype, wtype, seed=0):
    x, xr = draw(seed, (rows, D), dtype, 2.0)
    w, wr = draw(seed + 1, (D,), wtype)
    b, br = draw(seed + 2, (D,), wtype)
    g, gr = draw(seed + 3, (rows, D), dtype)
    return (x, w, b, g), (xr, wr, br, gr)


def fwd_mag(xr, wr, br, mean, rstd, y):
    size = (np.abs(xr) + np.abs(mean)[:, None] + np.mean(np.abs(xr), 1, keepdims=True)) * rstd[:, None]
    # the root's error moves the normalised value with it
    wide = 1 + 2 * np.mean(np.abs(xr), 1, keepdims=True) * rstd[:, None]
    w = np.abs(wr) if wr is not None else 1.0
    return size * wide * w + (np.abs(br) if br is not None else 0.0)


TYPE_PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]
# one row and many; below, at and across the widths of each kernel: a wave's packs, a
# workgroup's, wider than its registers; odd widths (rows that start at odd addresses)
SIZES = [(1, 1), (3, 7), (5, 64), (130, 511), (33, 513), (9, 1024), (700, 1111), (17, 2048), (6, 2049), (10, 4100),
         (3, 8192), (5, 8193), (3, 16384), (3, 16385), (2, 20001)]


@pytest.mark.parametrize("dtype,wtype", TYPE_PAIRS)
@pytest.mark.parametrize("rows,D", SIZES)
def test_forward(rows, D, dtype, wtype):
    print(f"\n[case] norm fwd {rows}x{D} {dtype}/{wtype}", flush=True)
    (x, w, b, _), (xr, wr, br, _) = case(rows, D, dtype, wtype)
    y, mean, rstd = R().layer_norm_fwd(x, w, b, eps=1e-5, return_stats=True)
    ry, rm, rr = O.layer_norm(xr, wr, br, 1e-5)
    size = np.mean(np.abs(xr), 1)
    check(mean, rm, size, 128, "mean")
    check(rstd, rr, rr * (1 + 2 * size * rr), 128, "rstd")
    check(y, ry, fwd_mag(xr, wr, br, rm, rr, ry), 128, "y")


@pytest.mark.parametrize("dtype,wtype", TYPE_PAIRS)
@pytest.mark.parametrize("rows,D", SIZES + [(5000, 96), (2500, 300)])
def test_backward(rows, D, dtype, wtype):
    print(f"\n[case] norm bwd {rows}x{D} {dtype}/{wtype}", flush=True)
    (x, w, b, g), (xr, wr, br, gr) = case(rows, D, dtype, wtype, 10)
    _, rm, rr = O.layer_norm(xr, eps=1e-5)
    mean, rstd = (torch.tensor(v).float().cuda() for v in (rm, rr))
    stats = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    got = R().layer_norm_bwd(x, w, mean, rstd, g)
    assert got[1].dtype == got[2].dtype == TYPES[wtype]
    ref = O.layer_norm_bwd(xr, wr, *stats, gr)
    mag = O.layer_norm_bwd(xr, wr, *stats, gr, magnitude=True)
    # sums over rows: at most rows / 64 in a lane's order (wide rows), 48 partial sums, a tree
    for v, r, m, what in zip(got, ref, mag, ("grad_x", "grad_weight", "grad_bias")):
        check(v, r, m, 128 + rows / 64, what)


def test_without_weights_and_with_parts():
    print("\n[case] norm without weights", flush=True)
    (x, w, b, g), (xr, wr, br, gr) = case(20, 200, "bf16", "f32", 20)
    ry, rm, rr = O.layer_norm(xr)
    check(R().layer_norm_fwd(x), ry, fwd_mag(xr, None, None, rm, rr, ry), 128)
    assert torch.equal(R().layer_norm_fwd(x.view(4, 5, 200)).view(20, 200), R().layer_norm_fwd(x))
    ry = O.layer_norm(xr, None, br)[0]
    check(R().layer_norm_fwd(x, None, b), ry, fwd_mag(xr, None, br, rm, rr, ry), 128)
    _, mean, rstd = R().layer_norm_fwd(x, return_stats=True)
    full = R().layer_norm_bwd(x, w, mean, rstd, g)
    assert R().layer_norm_bwd(x, None, mean, rstd, g)[1] is None
    parts = R().layer_norm_bwd(x, w, mean, rstd, g, bias_grad=False, weight_grad=False)
    assert parts[1] is None and parts[2] is None and torch.equal(parts[0], full[0])
    assert torch.equal(R().layer_norm_bwd(x, w, mean, rstd, g, weight_grad=False)[2], full[2])


def test_no_rows():
    print("\n[case] norm without rows", flush=True)
    x, w = torch.empty(0, 30, device="cuda"), torch.ones(30, device="cuda")
    y, mean, rstd = R().layer_norm_fwd(x, w, w, return_stats=True)
    assert y.shape == (0, 30) and mean.shape == (0,)
    gx, gw, gb = R().layer_norm_bwd(x, w, mean, rstd, x)
    assert gx.shape == (0, 30) and not gw.any() and not gb.any()


def test_a_row_of_nan_stays_one_row():
    print("\n[case] norm NaN row", flush=True)
    (x, w, b, g), _ = case(9, 600, "bf16", "bf16", 30)
    clean = R().layer_norm_fwd(x, w, b)
    x[4, 17] = float("nan")
    y = R().layer_norm_fwd(x, w, b)
    assert torch.isnan(y[4]).all() and torch.equal(y[:4], clean[:4]) and torch.equal(y[5:], clean[5:])


def test_large_offset_keeps_the_variance():
    """Columns far from zero: the squared deviations are summed about the mean."""
    print("\n[case] norm offset", flush=True)
    x, xr = draw(40, (4, 1500), "f32")
    x, xr = x + 1000.0, (x + 1000.0).double().cpu().numpy()
    _, mean, rstd = R().layer_norm_fwd(x, return_stats=True)
    _, rm, rr = O.layer_norm(xr)
    # the mean is off by k u 1000 at most, which moves the variance by its square only, and
    # each deviation by half a step of 1000: 2 u 1000 relative to the root
    check(mean, rm, np.full(4, 1000.0), 128, "mean")
    check(rstd, rr, rr * 1001, 4, "rstd")
