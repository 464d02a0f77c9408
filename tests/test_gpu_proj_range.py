"""The projections and head norms at the ends of what they take: widths of 2^20, more than 2^27 rows, views whose
offsets pass 32 bits, heads that are shared or stored in another order, more tokens than one launch holds,
threads that call at the same time.  (Bounds: proj_cases' and the head norms' counting, on the GPU in fp64.)"""
import threading

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
@pytest.mark.parametrize("M,N,K", [(1, 40, 1 << 20), (20, 33, (1 << 20) - 1), (100, 24, 1 << 20), (3, 1 << 20, 8), (70, (1 << 20) - 3, 9)])
def test_the_widest(M, N, K, dtype):
    print(f"\n[case] widest {M} {N} {K} {dtype}", flush=True)
    t, half = TYPES[dtype]
    x, w, gy = draw(1, M, K, dtype=t), draw(2, N, K, dtype=t, scale=K ** -0.5), draw(3, M, N, dtype=t)
    xd, wd, gd = x.double(), w.double(), gy.double()
    inside(R().linear_fwd(x, w), xd @ wd.T, (2 * K + 16) * (xd.abs() @ wd.abs().T), half)
    gx, gw, gb = R().linear_bwd(x, w, gy)
    inside(gx, gd @ wd, (2 * N + 16) * (gd.abs() @ wd.abs()), half)
    inside(gw, gd.T @ xd, (2 * M + 16) * (gd.abs().T @ xd.abs()), half)
    inside(gb, gd.sum(0), (2 * M + 16) * gd.abs().sum(0), half)


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_most_rows(dtype):
    """Whole numbers, whose sums are exact, in 2^27 + 77 rows."""
    print(f"\n[case] most rows {dtype}", flush=True)
    t, _ = TYPES[dtype]
    M = (1 << 27) + 77
    g = torch.Generator(device="cuda")
    g.manual_seed(4)
    x, gy = (torch.randint(-1, 2, (M, 1), generator=g, device="cuda", dtype=torch.int8) for _ in range(2))
    want = (x * gy).sum(dtype=torch.int64).item(), gy.sum(dtype=torch.int64).item()
    assert max(map(abs, want)) < 1 << 24
    x, gy, w = x.to(t), gy.to(t), torch.full((1, 1), 3.0, dtype=t, device="cuda")
    assert torch.equal(R().linear_fwd(x, w, activation="relu"), (3 * x).clamp(min=0))
    gx, gw, gb = R().linear_bwd(x, w, gy, bias_dtype=torch.float32)
    assert torch.equal(gx, 3 * gy)
    assert gb.item() == want[1] and gw.item() == torch.tensor(float(want[0])).to(t).item()


def norms(q, w, table, pos, eps=1e-6):
    """Head norms with interleaved rotary positions in fp64."""
    x = q.double()
    x = x / (x.square().mean(-1, keepdim=True) + eps).sqrt() * w.double()
    rot = 2 * table.shape[1]
    c, s = (table.double()[pos][..., i] for i in (0, 1))
    a, b = x[..., 0:rot:2], x[..., 1:rot:2]
    y = x.clone()
    y[..., 0:rot:2], y[..., 1:rot:2] = a * c - b * s, a * s + b * c
    return y


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
def test_heads_with_far_strides_and_shared_heads(dtype):
    print(f"\n[case] heads far {dtype}", flush=True)
    t, half = TYPES[dtype]
    B, H, N, d = 2, 3, 5, 64
    far = (1 << 31) + 64
    buf = torch.zeros(far + H * N * d, dtype=t, device="cuda")
    q = buf.as_strided((B, H, N, d), (far, d, H * d, 1))                # token-major, a batch beyond 2^31 elements
    q.copy_(draw(5, B, H, N, d, dtype=t))
    k = draw(6, B, 1, N, d, dtype=t).expand(B, H, N, d)                 # one head for all
    w, table = draw(7, d, dtype=t), R().rotary_table(R().rotary_frequencies(d), N)
    out = torch.zeros(far + H * N * d, dtype=t, device="cuda").as_strided(q.shape, q.stride())
    oq, ok = R().head_norm_rotary_fwd(q, k, table, w, w, out_q=out)
    assert oq is out
    pos = torch.arange(N, device="cuda")
    size = d + 32
    for got, x in ((oq, q), (ok, k)):
        ref = norms(x, w, table, pos)
        pairs = norms(x, w, table[:1], 0 * pos).abs()                   # (turned by nothing)
        pairs = (pairs[..., 0::2] + pairs[..., 1::2]).repeat_interleave(2, -1)
        inside(got, ref, size * pairs, half)
    g = draw(8, B, H, N, d, dtype=t)
    a = R().head_norm_rotary_bwd(q, k, table, g, g, w, w, out_q=out)
    b = R().head_norm_rotary_bwd(q.contiguous(), k.contiguous(), table, g, g, w, w)
    assert all(torch.equal(u, v) for u, v in zip(a, b))


@pytest.mark.parametrize("interleaved", [True, False])
def test_heads_of_more_tokens_than_a_launch(interleaved):
    """Single pairs, four tokens a workgroup: more than 2^22 workgroups."""
    print(f"\n[case] heads many tokens {interleaved}", flush=True)
    N = (1 << 24) + 5
    q = draw(9, 1, 1, N, 2, dtype=torch.float32)
    table = R().rotary_table(R().rotary_frequencies(2), 64)
    pos = (torch.arange(N, device="cuda") * 7) % 64
    y = R().head_norm_rotary_fwd(q, None, table, positions=pos, interleaved=interleaved)
    ref = norms(q, torch.ones(2, device="cuda"), table, pos)
    pairs = norms(q, torch.ones(2, device="cuda"), table[:1], 0 * pos).abs().sum(-1, keepdim=True)
    inside(y, ref, 34 * pairs, U)
    w = torch.ones(2, device="cuda")
    gx, _, gw, _ = R().head_norm_rotary_bwd(q, None, table, y, None, w, positions=pos, interleaved=interleaved)
    # the gradient of |y|^2 / 2, which is 1 - eps r^2 of a row: along x it vanishes but for eps
    x = q.double()
    ms = x.square().mean(-1, keepdim=True) + 1e-6
    xh = x / ms.sqrt()
    ref = (xh - xh * xh.square().mean(-1, keepdim=True)) / ms.sqrt()
    size = (xh.abs() + pairs.double() + xh.abs() * (pairs * xh.abs()).mean(-1, keepdim=True)) / ms.sqrt()
    inside(gx, ref, 2 * (34 + 68) * size, U)
    inside(gw, xh.square().sum((0, 1, 2)), (N + 68) * (pairs * xh.abs()).sum((0, 1, 2)), U)


def test_threads_call_at_the_same_time():
    """Each thread has a stream of its own and sizes of its own; every result is the lone call's."""
    print("\n[case] threads", flush=True)
    t = torch.bfloat16
    sizes = [(3, 136, 200), (40, 264, 65), (300, 1000, 520), (128, 4096, 1024)]
    data = [(draw(20 + i, M, K, dtype=t), draw(30 + i, N, K, dtype=t, scale=K ** -0.5), draw(40 + i, M, N, dtype=t))
            for i, (M, N, K) in enumerate(sizes)]
    call = lambda x, w, g, **k: (R().linear_fwd(x, w, activation="gelu", **k), *R().linear_bwd(x, w, g, **k))
    want = [call(*v) for v in data]
    torch.cuda.synchronize()
    got, errors = [None] * len(data), []

    def work(i):
        try:
            s = torch.cuda.Stream()
            got[i] = [call(*data[(i + j) % len(data)], stream=s) for j in range(40)]
            s.synchronize()
        except Exception as e:      # noqa: BLE001 (raised below)
            errors.append(e)

    threads = [threading.Thread(target=work, args=(i,)) for i in range(len(data))]
    for th in threads:
        th.start()
    for th in threads:
        th.join()
    assert not errors, errors
    for i, calls in enumerate(got):
        for j, out in enumerate(calls):
            assert all(torch.equal(a, b) for a, b in zip(out, want[(i + j) % len(data)])), (i, j)
