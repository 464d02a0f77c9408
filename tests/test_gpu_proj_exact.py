"""Products of whole numbers, whose sums are exact in fp32 in any order: every result is known to the last bit.

|sum| < 2^24 of all partial sums, so a product that keeps its operands and its (partial, cut, joined) sums in
fp32 gives the exact sum, and one that rounds any of them to fewer bits does not: one fp32 operand has 11 or
12 bits, more than bf16's 8, and the sums have more.  bf16 results are the exact sums rounded once, and
what a product hands to the next in bf16 is the exact value rounded once: the references round there too.
"""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"bf16": torch.bfloat16, "f32": torch.float32}
TOP = 1 << 24


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def whole(seed, shape, most, dtype):
    """Whole numbers from -most to most (fp32 beyond what bf16 holds)."""
    g = torch.Generator().manual_seed(seed)
    v = torch.randint(-most, most + 1, shape, generator=g)
    t = v.to(TYPES[dtype])
    assert torch.equal(t.long(), v)
    return t.cuda(), v.double().cuda()


def most_of(n, dtype):
    """The largest operand against -1, 0 and 1 in sums of n."""
    return 200 if dtype == "bf16" else min(4095, (TOP - 1) // n)


def exactly(got, ref, what):
    assert ref.abs().max() < TOP
    want = ref.to(got.dtype)          # exact in fp32; to bf16 one rounding from the exact value
    bad = (got != want).sum().item()
    assert bad == 0, f"{what}: {bad} of {got.numel()} differ, {got[got != want][:3]} for {want[got != want][:3]}"


# few rows (one and two blocks), one cut tile, all tiles cut, the last round's, none; long reductions, odd widths
SIZES = [(1, 4096, 1024), (16, 777, 4096), (17, 200, 4001), (32, 2048, 4096), (33, 200, 4096), (128, 1024, 4096), (300, 4096, 2048),
         (6001, 1500, 4096), (12000, 200, 4096), (8192, 2560, 512), (2200, 1048, 4104), (40, 136, 9000)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear(M, N, K, dtype):
    print(f"\n[case] exact linear {M} {N} {K} {dtype}", flush=True)
    for swap in (False, True):        # which operand has the bits
        x, xr = whole(1, (M, K), 1 if swap else most_of(K + 3, dtype), dtype)
        w, wr = whole(2, (N, K), most_of(K + 3, dtype) if swap else 1, dtype)
        b, br = whole(3, (N,), 90, "f32")
        y, pre = R().linear_fwd(x, w, b, activation="relu", return_pre=True)
        ref = xr @ wr.T + br
        exactly(pre, ref, "pre")
        exactly(y, ref.clamp(min=0), "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", SIZES)
def test_linear_gradients(M, N, K, dtype):
    print(f"\n[case] exact linear bwd {M} {N} {K} {dtype}", flush=True)
    gy, gr = whole(4, (M, N), most_of(max(M, N), dtype), dtype)
    x, xr = whole(5, (M, K), 1, dtype)
    w, wr = whole(6, (N, K), 1, dtype)
    z, zr = whole(7, (M, N), 9, dtype)
    for act, g in (("none", gr), ("relu", gr * (zr > 0))):
        gx, gw, gb = R().linear_bwd(x, w, gy, pre=z, activation=act, bias_dtype=torch.float32)
        exactly(gx, g @ wr, "grad_x")
        exactly(gw, g.T @ xr, "grad_weight")
        exactly(gb, g.sum(0), "grad_bias")


FFN = [(1, 64, 200), (16, 128, 1032), (30, 77, 333), (64, 256, 1024), (200, 1032, 520), (1100, 200, 136), (4000, 264, 1400)]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", FFN)
def test_gated_ffn(M, D, F, dtype):
    """Gate and up are exact, the gated product is rounded to the type once, and so is the result."""
    print(f"\n[case] exact ffn {M} {D} {F} {dtype}", flush=True)
    t = TYPES[dtype]
    x, xr = whole(1, (M, D), 2, dtype)
    (wg, gr), (wu, ur), (wd, dr), (r, rr) = (whole(2 + i, s, 1, dtype) for i, s in enumerate(((F, D), (F, D), (D, F), (M, D))))
    y, g, u = R().gated_ffn_fwd(x, wg, wu, wd, residual=r, activation="relu", return_pre=True)
    rg, ru = xr @ gr.T, xr @ ur.T
    exactly(g, rg, "gate")
    exactly(u, ru, "up")
    h = (rg.clamp(min=0) * ru).to(t).double()
    assert (h.abs() @ dr.abs().T).max() < TOP
    exactly(y, h @ dr.T + rr, "y")


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", FFN)
def test_gated_ffn_gradients(M, D, F, dtype):
    """The gradients of gate and up and the gated product are rounded to the type once, and so are the results."""
    print(f"\n[case] exact ffn bwd {M} {D} {F} {dtype}", flush=True)
    t = TYPES[dtype]
    (x, xr), (wg, gr), (wu, ur), (wd, dr), (gy, yr) = (whole(10 + i, s, 1, dtype)
                                                       for i, s in enumerate(((M, D), (F, D), (F, D), (D, F), (M, D))))
    g, gk = whole(16, (M, F), 5, dtype)
    u, uk = whole(17, (M, F), 5, dtype)
    got = R().gated_ffn_bwd(x, wg, wu, wd, g, u, gy, activation="relu")
    gh, on, a = yr @ dr, (gk > 0).double(), gk.clamp(min=0)
    gg, gu, h = ((gh * uk * on).to(t).double(), (gh * a).to(t).double(), (a * uk).to(t).double())
    assert (gg.abs() @ gr.abs() + gu.abs() @ ur.abs()).max() < TOP and (gg.abs().T @ xr.abs()).max() < TOP
    for o, ref, what in zip(got, (gg @ gr + gu @ ur, gg.T @ xr, gu.T @ xr, yr.T @ h),
                            ("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")):
        exactly(o, ref, what)
