"""The short causal convolution, forward, backward and one token, against the fp64 oracle.

Counting roundings: K + 1 steps and the activation's 8, k = 16, relative to |bias| + sum |w x|
(silu's slope is at most 1.1).  Backward: an error of pre moves silu' by half of it at most, so
the terms' relative error is (16 + 8 mag_pre) u; sums over tokens add 32 steps in a walk, 32
walks in LDS at most, 48 partial sums: k = 160 + 8 max mag_pre.
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


def case(B, N, D, K, dtype, wtype, wide=False, seed=0):
    x, xr = draw(seed, (B, N, 2 * D if wide else D), dtype)
    if wide:
        x, xr = x[..., D:], xr[..., D:]
    w, wr = draw(seed + 1, (D, K), wtype, 0.6)
    b, br = draw(seed + 2, (D,), wtype)
    s, sr = draw(seed + 3, (B, K - 1, D), dtype)
    return (x, w, b, s), (xr, wr, br, sr)


def pre_mag(xr, wr, br, sr):
    return O.causal_conv(np.abs(xr), np.abs(wr), None if br is None else np.abs(br), False,
                         None if sr is None else np.abs(sr))[0]


CASES = [
    # B, N, D, K, wide: one token, fewer tokens than taps, odd widths, tiles that end inside
    (1, 1, 8, 4, False), (2, 2, 5, 4, False), (3, 3, 64, 3, True), (2, 70, 33, 2, False), (1, 257, 96, 4, True),
    (2, 40, 2048, 4, False), (4, 129, 72, 3, False), (1, 1000, 7, 4, True), (3, 600, 640, 4, False),
]
TYPE_PAIRS = [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")]


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype,wtype", TYPE_PAIRS)
@pytest.mark.parametrize("B,N,D,K,wide", CASES)
def test_forward(B, N, D, K, wide, dtype, wtype, silu):
    print(f"\n[case] conv fwd {B} {N} {D} {K} {wide} {dtype}/{wtype} {silu}", flush=True)
    (x, w, b, s), (xr, wr, br, sr) = case(B, N, D, K, dtype, wtype, wide)
    y, s1 = R().causal_conv_fwd(x, w, b, silu=silu, state_in=s, return_state=True)
    ry, rs = O.causal_conv(xr, wr, br, silu, sr)
    check(y, ry, pre_mag(xr, wr, br, sr), 16, "y")
    assert np.array_equal(s1.double().cpu().numpy(), rs)
    # without a bias and a state
    y = R().causal_conv_fwd(x, w, silu=silu)
    check(y, O.causal_conv(xr, wr, None, silu)[0], pre_mag(xr, wr, None, None), 16, "plain y")


@pytest.mark.parametrize("big", [False, True])
def test_large_forward_uses_the_long_walk(big):
    """Sizes on both sides of the rule that picks the tokens of a thread; equal results."""
    B, N, D = (8, 2049, 2048) if big else (1, 333, 2048)
    print(f"\n[case] conv long walk {big}", flush=True)
    g = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(B, N, D, generator=g, device="cuda").bfloat16()
    w, b = torch.randn(D, 4, generator=g, device="cuda").bfloat16(), torch.randn(D, generator=g, device="cuda").bfloat16()
    y, s = R().causal_conv_fwd(x, w, b, return_state=True)
    xs = torch.cat((torch.zeros(B, 3, D, device="cuda"), x.float()), 1)
    ref = b.float() + sum(w.float()[:, j] * xs[:, j:j + N] for j in range(4))
    size = b.float().abs() + sum(w.float()[:, j].abs() * xs[:, j:j + N].abs() for j in range(4))
    # both sums are off by 5 roundings at most, the output by half a step
    assert bool(((y.float() - ref).abs() <= 2.0 ** -8 * ref.abs() + 10 * 2.0 ** -24 * size).all())
    assert torch.equal(s, x[:, -3:])


@pytest.mark.parametrize("silu", [False, True])
@pytest.mark.parametrize("dtype,wtype", TYPE_PAIRS)
@pytest.mark.parametrize("B,N,D,K,wide", CASES)
def test_backward(B, N, D, K, wide, dtype, wtype, silu):
    print(f"\n[case] conv bwd {B} {N} {D} {K} {wide} {dtype}/{wtype} {silu}", flush=True)
    (x, w, b, s), (xr, wr, br, sr) = case(B, N, D, K, dtype, wtype, wide, 10)
    g, gr = draw(20, (B, N, D), dtype)
    gs, gsr = draw(21, (B, K - 1, D), dtype)
    got = R().causal_conv_bwd(x, w, g, b, silu=silu, state_in=s, grad_state_out=gs, return_grad_state_in=True)
    args = (xr, wr, gr, br, silu, sr, gsr)
    k = 160 + 8 * pre_mag(xr, wr, br, sr).max()
    names = ("grad_x", "grad_weight", "grad_bias", "grad_state_in")
    mags = O.causal_conv_bwd(*args, magnitude=True)
    # where silu' is near zero the error is relative to |g|, not to |g silu'|
    flat = O.causal_conv_bwd(xr, wr, gr, br, False, sr, gsr, magnitude=True)
    for v, r, m, f, nm in zip(got, O.causal_conv_bwd(*args), mags, flat, names):
        check(v, r, np.maximum(m, f), k, nm)
    plain = R().causal_conv_bwd(x, w, g, silu=silu)
    assert plain[2] is None
    check(plain[0], O.causal_conv_bwd(xr, wr, gr, None, silu)[0], O.causal_conv_bwd(xr, wr, gr, None, False, magnitude=True)[0],
          k, "plain grad_x")


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_lengths(dtype):
    """Padded sequences, of no token and of all of them among them; NaN behind the ends."""
    print(f"\n[case] conv lengths {dtype}", flush=True)
    B, N, D, K = 6, 75, 40, 4
    (x, w, b, s), (xr, wr, br, sr) = case(B, N, D, K, dtype, dtype, False, 30)
    n = [75, 0, 1, 2, 64, 33]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    g, gr = draw(40, (B, N, D), dtype)
    gs, gsr = draw(41, (B, K - 1, D), dtype)
    for i, m in enumerate(n):
        x[i, m:], g[i, m:] = float("nan"), float("nan")
    out = torch.full((B, N, D), 7.0, dtype=x.dtype, device="cuda")
    y, s1 = R().causal_conv_fwd(x, w, b, silu=True, state_in=s, return_state=True, lengths=lengths, out=out)
    ry, rs = O.causal_conv(xr, wr, br, True, sr, n)
    mag = pre_mag(xr, wr, br, sr)
    for i, m in enumerate(n):
        check(y[i, :m], ry[i, :m], mag[i, :m], 16)
        assert bool((y[i, m:] == 7).all())
    assert np.array_equal(s1.double().cpu().numpy(), rs)
    got = R().causal_conv_bwd(x, w, g, b, silu=True, state_in=s, grad_state_out=gs, lengths=lengths,
                              return_grad_state_in=True)
    ref = O.causal_conv_bwd(xr, wr, gr, br, True, sr, gsr, n)
    flat = O.causal_conv_bwd(xr, wr, gr, br, False, sr, gsr, n, magnitude=True)
    for v, r, f in zip(got, ref, flat):
        check(v, r, 1.1 * f, 160 + 8 * mag.max())
    # lengths outside 0 .. N count as 0 and N
    wild = torch.tensor([99, -5, 1, 2, 64, 33], dtype=torch.int32, device="cuda")
    again = R().causal_conv_fwd(x, w, b, silu=True, state_in=s, lengths=wild, out=torch.full_like(out, 7.0))
    assert torch.equal(again, y)


@pytest.mark.parametrize("dtype,wtype", TYPE_PAIRS)
@pytest.mark.parametrize("B,D,K", [(1, 1, 2), (3, 33, 3), (128, 256, 4), (7, 2048, 4)])
def test_step_continues_a_prompt(B, D, K, dtype, wtype):
    print(f"\n[case] conv step {B} {D} {K} {dtype}/{wtype}", flush=True)
    N = 6
    (x, w, b, s), _ = case(B, N, D, K, dtype, wtype, True, 50)
    y, s1 = R().causal_conv_fwd(x, w, b, silu=True, state_in=s, return_state=True)
    state = s.clone()
    for t in range(N):
        assert torch.equal(R().causal_conv_step(x[:, t], w, state, b, silu=True), y[:, t]), t
    assert torch.equal(state, s1)


def test_no_tokens():
    print("\n[case] conv without tokens", flush=True)
    (x, w, b, s), _ = case(2, 3, 16, 4, "bf16", "bf16", False, 60)
    y, s1 = R().causal_conv_fwd(x[:, :0].contiguous(), w, b, state_in=s, return_state=True)
    assert y.shape == (2, 0, 16) and torch.equal(s1, s)
    gs = torch.randn(2, 3, 16, device="cuda").bfloat16()
    gx, gw, gb, gs0 = R().causal_conv_bwd(x[:, :0].contiguous(), w, x[:, :0].contiguous(), b, state_in=s, grad_state_out=gs,
                                          return_grad_state_in=True)
    assert gx.numel() == 0 and not gw.any() and not gb.any() and torch.equal(gs0, gs)
