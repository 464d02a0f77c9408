"""Rows behind the sequences of a padded batch, in outputs that the binding allocates: zeros,
whatever the memory held.  (A gradient sums y^T g over all rows of a padded batch; g is zero
behind the ends, and zero times a NaN that an earlier tensor left there would be NaN.)"""
import numpy as np
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TYPES = {"f32": torch.float32, "bf16": torch.bfloat16}


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def draw(seed, shape, dtype, scale=1.0):
    v = np.random.default_rng(seed).standard_normal(shape) * scale
    return torch.tensor(v).to(TYPES[dtype]).cuda()


def poison(shape, dtype):
    """Leaves NaN in the memory that the next tensors of this size get."""
    junk = [torch.full(shape, float("nan"), dtype=TYPES[dtype], device="cuda") for _ in range(4)]
    torch.cuda.synchronize()
    del junk


def ends(B, N):
    n = [N, 0, 1, N // 2 + 1, max(N - 1, 0)][:B]
    return n, torch.tensor(n, dtype=torch.int32, device="cuda")


def compare(y, want, n):
    for i, m in enumerate(n):
        assert torch.equal(y[i, :m], want[i, :m]), (i, m)
        assert not bool(y[i, m:].ne(0).any()), (i, m)        # NaN differs from zero too


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,K", [(75, 40, 4), (1, 8, 2), (130, 33, 3), (3, 64, 4), (700, 256, 4)])
def test_convolution(N, D, K, dtype):
    print(f"\n[case] conv padding {N} {D} {K} {dtype}", flush=True)
    B = 5
    x, w, b = draw(1, (B, N, D), dtype), draw(2, (D, K), dtype, 0.6), draw(3, (D,), dtype)
    s = draw(4, (B, K - 1, D), dtype)
    n, lengths = ends(B, N)
    out = torch.full((B, N, D), 7.0, dtype=TYPES[dtype], device="cuda")
    kw = dict(silu=True, state_in=s, lengths=lengths)
    want, state = R().causal_conv_fwd(x, w, b, return_state=True, out=out, **kw)
    for i, m in enumerate(n):
        assert bool((want[i, m:] == 7).all())                # a given output's rows stay
    poison((B, N, D), dtype)
    y, st = R().causal_conv_fwd(x, w, b, return_state=True, **kw)
    compare(y, want, n)
    assert torch.equal(st, state)


@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("N,D,G,S", [(40, 70, 1, 16), (1, 5, 1, 3), (530, 20, 2, 16), (300, 66, 1, 13), (90, 64, 1, 64)])
def test_scan(N, D, G, S, dtype):
    print(f"\n[case] scan padding {N} {D} {G} {S} {dtype}", flush=True)
    B = 5
    x, dt, z = (draw(i, (B, N, D), dtype) for i in (1, 2, 3))
    Bm, Cm = (draw(i, (B, N, G, S), dtype) for i in (4, 5))
    A = -torch.exp(draw(6, (D, S), "f32"))
    n, lengths = ends(B, N)
    out = torch.full((B, N, D), 7.0, dtype=TYPES[dtype], device="cuda")
    kw = dict(D=draw(7, (D,), "f32"), z=z, dt_bias=draw(8, (D,), "f32"), softplus=True, state_in=draw(9, (B, D, S), "f32"),
              lengths=lengths)
    want, state = R().selective_scan_fwd(x, dt, A, Bm, Cm, return_state=True, out=out, **kw)
    for i, m in enumerate(n):
        assert bool((want[i, m:] == 7).all())
    poison((B, N, D), dtype)
    y, st = R().selective_scan_fwd(x, dt, A, Bm, Cm, return_state=True, **kw)
    compare(y, want, n)
    assert torch.equal(st, state)
