"""The projection with its epilogue and its gradients, against the fp64 oracle (bounds: proj_cases)."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402
from proj_cases import ACTS, linear_bounds, linear_bwd_bounds  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


# one row and one column; steps of the reduction that are whole, cut inside a 16-byte unit and at
# one; tiles that are whole and cut; few rows; a long reduction with few tiles (split)
SIZES = [(1, 1, 1), (1, 64, 64), (3, 8, 24), (5, 130, 7), (16, 128, 256), (33, 100, 72), (128, 128, 128), (130, 129, 65),
         (300, 257, 200), (129, 40, 1111), (1000, 96, 33), (64, 64, 4096), (700, 384, 512)]


def make(M, N, K, dtype, bdtype, seed=0):
    x, xr = draw(seed, (M, K), dtype)
    w, wr = draw(seed + 1, (N, K), dtype, K ** -0.5)
    b, br = draw(seed + 2, (N,), bdtype)
    r, rr = draw(seed + 3, (M, N), dtype)
    return (x, w, b, r), (xr, wr, br, rr)


@pytest.mark.parametrize("act", ACTS)
@pytest.mark.parametrize("dtype,bdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_forward(M, N, K, dtype, bdtype, act):
    print(f"\n[case] linear {M} {N} {K} {dtype}/{bdtype} {act}", flush=True)
    (x, w, b, r), (xr, wr, br, rr) = make(M, N, K, dtype, bdtype)
    y, pre = R().linear_fwd(x, w, b, residual=r, activation=act, return_pre=True)
    ry, rz = O.linear(xr, wr, br, rr, act)
    by, bz = linear_bounds(xr, wr, br, rr, act)
    check(pre, rz, bz, 1, "pre")
    check(y, ry, by, 1, "y")
    plain = R().linear_fwd(x, w, activation=act)
    by, _ = linear_bounds(xr, wr, None, None, act)
    check(plain, O.linear(xr, wr, None, None, act)[0], by, 1, "without bias and residual")


@pytest.mark.parametrize("act", ["none", "gelu", "silu"])
@pytest.mark.parametrize("dtype,bdtype", [("bf16", "bf16"), ("bf16", "f32"), ("f32", "f32")])
@pytest.mark.parametrize("M,N,K", SIZES + [(5000, 24, 40), (4096, 64, 64), (2500, 65, 30)])
def test_backward(M, N, K, dtype, bdtype, act):
    print(f"\n[case] linear bwd {M} {N} {K} {dtype}/{bdtype} {act}", flush=True)
    (x, w, _, _), (xr, wr, _, _) = make(M, N, K, dtype, bdtype, 10)
    gy, gr = draw(14, (M, N), dtype)
    z, zr = draw(15, (M, N), dtype, 1.5)
    got = R().linear_bwd(x, w, gy, pre=None if act == "none" else z, activation=act, bias_dtype=TYPES[bdtype])
    assert got[2].dtype == TYPES[bdtype]
    ref = O.linear_bwd(xr, wr, gr, zr, act)
    for g, v, m, what in zip(got, ref, linear_bwd_bounds(xr, wr, gr, zr, act, dtype), ("grad_x", "grad_weight", "grad_bias")):
        check(g, v, m, 1, what)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("off", [0, 1, 8])
def test_slices_of_wider_rows(dtype, off):
    """A column slice that starts at any element, of rows of any width, and weights at odd addresses."""
    print(f"\n[case] linear slices {dtype} {off}", flush=True)
    for wide in (200, 201):
        buf, br = draw(20, (3, 70, wide), dtype)
        x, xr = buf[..., off:off + 72], br[..., off:off + 72].reshape(210, 72)
        wb, wbr = draw(21, (off + 48 * 72,), dtype, 0.1)
        w, wr = wb[off:].view(48, 72), wbr[off:].reshape(48, 72)
        y = R().linear_fwd(x, w, activation="silu")
        assert y.shape == (3, 70, 48)
        check(y.view(210, 48), O.linear(xr, wr, act="silu")[0], linear_bounds(xr, wr, None, None, "silu")[0], 1, "y")
        gy, gr = draw(22, (3, 70, 48), dtype)
        gx, gw, gb = R().linear_bwd(x, w, gy)
        gr = gr.reshape(210, 48)
        for g, v, m in zip((gx.view(210, 72), gw, gb), O.linear_bwd(xr, wr, gr), linear_bwd_bounds(xr, wr, gr, None, "none", dtype)):
            check(g, v, m, 1)


def test_residual_in_place_and_parts():
    print("\n[case] linear in place", flush=True)
    (x, w, b, r), _ = make(150, 130, 96, "bf16", "bf16", 30)
    y = R().linear_fwd(x, w, b, residual=r, activation="gelu")
    r2 = r.clone()
    assert R().linear_fwd(x, w, b, residual=r2, activation="gelu", out=r2) is r2 and torch.equal(r2, y)
    gy = torch.randn(150, 130, device="cuda").bfloat16()
    full = R().linear_bwd(x, w, gy)
    for i, kw in enumerate((dict(weight_grad=False, bias_grad=False), dict(x_grad=False, bias_grad=False),
                            dict(x_grad=False, weight_grad=False))):
        part = R().linear_bwd(x, w, gy, **kw)
        for j in range(3):
            assert torch.equal(part[j], full[j]) if i == j else part[j] is None


def test_no_rows():
    print("\n[case] linear without rows", flush=True)
    for dtype in TYPES.values():
        x, w = torch.empty(0, 30, device="cuda", dtype=dtype), torch.ones(20, 30, device="cuda", dtype=dtype)
        y, pre = R().linear_fwd(x, w, activation="relu", return_pre=True)
        assert y.shape == pre.shape == (0, 20)
        gx, gw, gb = R().linear_bwd(x, w, y)
        assert gx.shape == (0, 30) and not gw.any() and not gb.any()
        gx, gw, gb = R().linear_bwd(x, w, y, pre=pre, activation="relu")
        assert not gw.any() and not gb.any()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_nan_and_infinity_stay_in_their_rows(dtype):
    """Rows and columns that pad tiles, and what lies beside a slice, are never part of a sum."""
    print(f"\n[case] linear NaN {dtype}", flush=True)
    (x, w, b, r), _ = make(200, 150, 100, dtype, "f32", 40)
    clean = R().linear_fwd(x, w, b, residual=r, activation="silu")
    x2 = x.clone()
    x2[77, 3] = float("nan")
    y = R().linear_fwd(x2, w, b, residual=r, activation="silu")
    assert torch.isnan(y[77]).all()
    keep = torch.arange(200, device="cuda") != 77
    assert torch.equal(y[keep], clean[keep])
    w2 = w.clone()
    w2[149, 99] = float("inf")
    y = R().linear_fwd(x, w2, b, residual=r)
    assert torch.equal(y[:, :149], R().linear_fwd(x, w, b, residual=r)[:, :149]) and not torch.isfinite(y[:, 149]).any()
    # a slice between columns of NaN
    wide = torch.full((200, 300), float("nan"), device="cuda", dtype=TYPES[dtype])
    wide[:, 104:204] = x
    assert torch.equal(R().linear_fwd(wide[:, 104:204], w, b, residual=r, activation="silu"), clean)
    gy = torch.randn(200, 150, device="cuda").to(TYPES[dtype])
    a, c = R().linear_bwd(wide[:, 104:204], w, gy), R().linear_bwd(x, w, gy)
    assert all(torch.equal(u, v) for u, v in zip(a, c))


@pytest.mark.parametrize("act", ACTS)
def test_far_values_of_the_activations(act):
    """Pre-activations to the ends of the type, and infinities of the sign that a limit exists for."""
    print(f"\n[case] linear far {act}", flush=True)
    z = torch.tensor([0.0, -0.0, 1e-30, -1e-30, 20.0, -20.0, 1e4, -1e4, 3e38, -3e38, float("inf")], device="cuda")[:, None]
    one = torch.ones(1, 1, device="cuda")
    y = R().linear_fwd(z, one, activation=act).double().cpu().numpy()
    with np.errstate(all="ignore"):
        ref, slope = O.activation(z.double().cpu().numpy(), act)
        slope = np.where(np.abs(z.cpu().numpy()) > 1e3, O.activation(np.clip(z.double().cpu().numpy(), -1e3, 1e3), act)[1], slope)
    fin = np.isfinite(ref)
    assert np.all(np.abs(y - ref)[fin] <= 16 * 2.0 ** -24 * np.abs(z.cpu().numpy())[fin] + 1e-37)
    assert np.isposinf(y[-1, 0])
    g = R().linear_bwd(z, one, torch.ones_like(z), pre=z, activation=act)[0].double().cpu().numpy()
    assert np.all(np.abs(g - slope) <= 24 * 2.0 ** -24)
    nan = torch.full((1, 1), float("nan"), device="cuda")
    assert torch.isnan(R().linear_fwd(nan, one, activation=act)).all()


@pytest.mark.parametrize("M,N,K", [(4096, 2048, 768), (2000, 4096, 520), (8192, 1032, 1024)])
def test_many_tiles(M, N, K):
    """Enough tiles for every size of them, against products in fp64 on the GPU."""
    print(f"\n[case] linear many {M} {N} {K}", flush=True)
    (x, w, b, r), _ = make(M, N, K, "bf16", "f32", 50)
    gy = torch.randn(M, N, device="cuda").bfloat16()
    xd, wd, gd = x.double(), w.double(), gy.double()
    z = xd @ wd.T + b.double()
    mag = xd.abs() @ wd.abs().T + b.double().abs()
    for got, ref, bound in (
            (R().linear_fwd(x, w, b), z, (2 * K + 16) * mag),
            (R().linear_bwd(x, w, gy)[0], gd @ wd, (2 * N + 16) * (gd.abs() @ wd.abs())),
            (R().linear_bwd(x, w, gy)[1], gd.T @ xd, (2 * M + 16) * (gd.abs().T @ xd.abs()))):
        room = 2.0 ** -8 * ref.abs() + 1.01 * 2.0 ** -24 * bound
        assert ((got.double() - ref).abs() <= room).all()
