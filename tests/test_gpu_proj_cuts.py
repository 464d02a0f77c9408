"""Products whose tiles are cut along the reduction in each way (all of them, the last round's, none; few
parts and many; both phases of a gradient), and tensors of more than 2^31 elements, against products in
fp64 on the GPU (bounds: proj_cases' counting)."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TYPES = {"bf16": (torch.bfloat16, 2.0 ** -8), "f32": (torch.float32, 2.0 ** -24)}


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def draw(seed, *shape, dtype, scale=1.0):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def inside(got, ref, bound, half):
    over = (got.double() - ref).abs() - (half * ref.abs() + 1.01 * U * bound)
    assert (over <= 0).all(), over.max().item()


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(12000, 777, 64), (8192, 5000, 1024), (12000, 1500, 4096), (12000, 200, 4096), (300, 4096, 4096),
                                   (12000, 1500, 2048), (300, 4096, 2048), (1000, 777, 2048), (300, 200, 1000), (5000, 777, 64),
                                   (40, 136, 9000), (2200, 1048, 4104)])
def test_linear(M, N, K, dtype):
    print(f"\n[case] cuts {M} {N} {K} {dtype}", flush=True)
    t, half = TYPES[dtype]
    if dtype == "f32":
        M = M // 2 + 1
    x, w = draw(1, M, K, dtype=t), draw(2, N, K, dtype=t, scale=K ** -0.5)
    b, r, gy = draw(3, N, dtype=torch.float32), draw(4, M, N, dtype=t), draw(5, M, N, dtype=t)
    xd, wd, gd = x.double(), w.double(), gy.double()
    z, mag = xd @ wd.T + b.double(), xd.abs() @ wd.abs().T + b.double().abs()
    y, pre = R().linear_fwd(x, w, b, residual=r, activation="silu", return_pre=True)
    inside(pre, z, (2 * K + 16) * mag, half)
    inside(y, z * torch.sigmoid(z) + r.double(), 1.2 * (2 * K + 16) * mag + 20 * z.abs() + 4 * r.double().abs(), half)
    gx, gw, gb = R().linear_bwd(x, w, gy)
    inside(gx, gd @ wd, (2 * N + 16) * (gd.abs() @ wd.abs()), half)
    inside(gw, gd.T @ xd, (2 * M + 16) * (gd.abs().T @ xd.abs()), half)
    inside(gb, gd.sum(0), (2 * M + 16) * gd.abs().sum(0), half)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", [(200, 1032, 520), (128, 2048, 1024), (5000, 200, 136), (2500, 520, 1400)])
def test_gated_ffn(M, D, F, dtype):
    print(f"\n[case] cuts ffn {M} {D} {F} {dtype}", flush=True)
    t, half = TYPES[dtype]
    x, gy = draw(1, M, D, dtype=t), draw(2, M, D, dtype=t)
    wg, wu = (draw(3 + i, F, D, dtype=t, scale=D ** -0.5) for i in range(2))
    wd = draw(5, D, F, dtype=t, scale=F ** -0.5)
    xd, gd, ud, dd, yd = (v.double() for v in (x, wg, wu, wd, gy))
    y, g, u = R().gated_ffn_fwd(x, wg, wu, wd, activation="relu", return_pre=True)
    rg, ru = xd @ gd.T, xd @ ud.T
    bg, bu = ((2 * D + 16) * (xd.abs() @ w.abs().T) for w in (gd, ud))
    inside(g, rg, bg, half)
    inside(u, ru, bu, half)
    h = rg.clamp(min=0) * ru
    bh = bg * ru.abs() + rg.abs() * bu + (half / U + 4) * h.abs()
    inside(y, h @ dd.T, 1.01 * (bh @ dd.abs().T) + (2 * F + 16) * (h.abs() @ dd.abs().T), half)
    got = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy, activation="relu")
    gk, uk = g.double(), u.double()
    gh, mh = yd @ dd, (2 * D + 16) * (yd.abs() @ dd.abs())
    a, s = gk.clamp(min=0), (gk > 0).double()
    gg, gu, h = gh * uk * s, gh * a, a * uk
    eg, eu, eh = mh * uk.abs() * s + (half / U + 4) * gg.abs(), mh * a + (half / U + 4) * gu.abs(), (half / U + 4) * h.abs()
    n = 2 * M + 16
    inside(got[0], gg @ gd + gu @ ud, 1.01 * (eg @ gd.abs() + eu @ ud.abs()) + (4 * F + 16) * (gg.abs() @ gd.abs() + gu.abs() @ ud.abs()), half)
    inside(got[1], gg.T @ xd, 1.01 * eg.T @ xd.abs() + n * gg.abs().T @ xd.abs(), half)
    inside(got[2], gu.T @ xd, 1.01 * eu.T @ xd.abs() + n * gu.abs().T @ xd.abs(), half)
    inside(got[3], yd.T @ h, 1.01 * yd.abs().T @ eh + n * yd.abs().T @ h.abs(), half)


def test_more_than_2_31_elements():
    """Outputs, gradients and pre-activations of 2.2e9 elements: the last rows and columns."""
    print("\n[case] cuts large", flush=True)
    M, N, K = 66001, 33000, 24
    t, half = TYPES["bf16"]
    x, w = draw(1, M, K, dtype=t), draw(2, N, K, dtype=t)
    y, pre = R().linear_fwd(x, w, activation="relu", return_pre=True)
    rows = torch.tensor([0, 1, 40000, 65279, 65280, 66000], device="cuda")
    z = x[rows].double() @ w.double().T
    bound = (2 * K + 16) * (x[rows].double().abs() @ w.double().abs().T)
    inside(pre[rows], z, bound, half)
    inside(y[rows], z.clamp(min=0), 1.2 * bound, half)
    gx, gw, gb = R().linear_bwd(x, w, y, pre=pre, activation="relu")
    gd = y[rows].double() * (pre[rows] > 0)
    inside(gx[rows], gd @ w.double(), (2 * N + 16) * (gd.abs() @ w.double().abs()), half)
    cols = torch.tensor([0, 17, 32999], device="cuda")
    gd = y[:, cols].double() * (pre[:, cols] > 0)
    inside(gw[cols], gd.T @ x.double(), (2 * M + 16) * (gd.abs().T @ x.double().abs()), half)
    inside(gb[cols], gd.sum(0), (2 * M + 16) * gd.abs().sum(0), half)
