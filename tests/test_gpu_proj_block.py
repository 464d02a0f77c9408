"""The projections as a block uses them: between norms, rotary positions and the retention, in
training against differences of the whole, on streams, in captured graphs over one workspace."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import draw  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def rel(a, b):
    a = a.detach().double().cpu().numpy()
    return float(np.max(np.abs(a - b)) / np.max(np.abs(b)))


B, N, D, H, d, F = 2, 70, 96, 3, 32, 200
T = B * N


def weights(dtype):
    """(tensors, fp64 values) of a block: norms, q, k, v and output projections, head norms, feed-forward."""
    shapes = dict(n1=(D,), wq=(H * d, D), wk=(H * d, D), wv=(H * d, D), qn=(d,), kn=(d,), wo=(D, H * d), n2=(D,), wg=(F, D),
                  wu=(F, D), wd=(D, F))
    t, r = {}, {}
    for i, (n, s) in enumerate(shapes.items()):
        t[n], r[n] = draw(100 + i, s, dtype, 1.0 if len(s) == 1 else s[1] ** -0.5)
    return t, r


def heads(y):
    return y.view(B, N, H, d).transpose(1, 2)


def oracle_block(x, w, gamma, freq):
    h = O.layer_norm(x, w["n1"])[0]
    q, k, v = (np.transpose((h @ w[n].T).reshape(B, N, H, d), (0, 2, 1, 3)) for n in ("wq", "wk", "wv"))
    pos = np.arange(N)
    q = O.head_norm_rotary(q, pos, freq, w["qn"], 1e-6)
    k = O.head_norm_rotary(k, pos, freq, w["kn"], 1e-6, scale=d ** -0.5)
    o = np.transpose(O.retention_recurrent(q, k, v, gamma)[0], (0, 2, 1, 3)).reshape(B, N, H * d)
    x = x + o @ w["wo"].T
    return O.gated_ffn(O.layer_norm(x, w["n2"])[0].reshape(T, D), w["wg"], w["wu"], w["wd"], x.reshape(T, D))[0].reshape(B, N, D)


def block(x, w, gamma, table):
    h = R().layer_norm_fwd(x, w["n1"])
    # q, k and v in one product, read as column slices
    joint = R().linear_fwd(h, torch.cat((w["wq"], w["wk"], w["wv"])))
    q, k, v = (joint[..., i * H * d:(i + 1) * H * d].unflatten(-1, (H, d)).transpose(1, 2) for i in range(3))
    q, k = R().head_norm_rotary_fwd(q, k, table, w["qn"], w["kn"], k_scale=d ** -0.5)
    o = R().retention_chunkwise_fwd(q, k, v.contiguous(), gamma, 64)
    x = R().linear_fwd(o.transpose(1, 2).reshape(B, N, H * d), w["wo"], residual=x)
    return R().gated_ffn_fwd(R().layer_norm_fwd(x, w["n2"]), w["wg"], w["wu"], w["wd"], residual=x)


@pytest.mark.parametrize("dtype,tol", [("f32", 1e-4), ("bf16", 3e-2)])
def test_a_block(dtype, tol):
    """The whole block against the oracles', relative to the largest output: eight operators, whose
    roundings of at most 2^-8 (bf16) add up to 3e-2; in fp32 their sums of up to 200 terms stay below 1e-4."""
    print(f"\n[case] block {dtype}", flush=True)
    x, xr = draw(99, (B, N, D), dtype)
    w, wr = weights(dtype)
    gamma = torch.tensor([0.9, 0.97, 1.0])
    freq = R().rotary_frequencies(d)
    y = block(x, w, gamma.cuda(), R().rotary_table(freq, N))
    assert rel(y, oracle_block(xr, wr, gamma.double().numpy(), freq.numpy())) <= tol


def test_a_training_step_against_differences():
    """<g, y> of the feed-forward half and a projection behind a head norm, fp32: the chained
    gradients against central differences of the fp64 oracles along random directions."""
    print("\n[case] chained gradients", flush=True)
    x, xr = draw(98, (T, D), "f32")
    w, wr = weights("f32")
    g, gr = draw(97, (T, D), "f32")
    gq, gqr = draw(96, (B, H, N, d), "f32")
    freq = R().rotary_frequencies(d)
    table = R().rotary_table(freq, N)

    def whole(x, w):
        y, pre = O.linear(x, w["wo"][:, :D], None, x, "gelu")
        y = O.gated_ffn(y, w["wg"], w["wu"], w["wd"], y)[0]
        q = np.transpose((x @ w["wq"].T).reshape(B, N, H, d), (0, 2, 1, 3))
        return np.sum(gr * y) + np.sum(gqr * O.head_norm_rotary(q, np.arange(N), freq.numpy(), w["qn"], 1e-6))

    wo = w["wo"][:, :D].contiguous()
    y1, pre = R().linear_fwd(x, wo, residual=x, activation="gelu", return_pre=True)
    _, gate, up = R().gated_ffn_fwd(y1, w["wg"], w["wu"], w["wd"], residual=y1, return_pre=True)
    gy, gwg, gwu, gwd = R().gated_ffn_bwd(y1, w["wg"], w["wu"], w["wd"], gate, up, g)
    gy = gy + g                                             # the residual's
    gx, gwo, _ = R().linear_bwd(x, wo, gy, pre=pre, activation="gelu", bias_grad=False)
    q = heads(R().linear_fwd(x, w["wq"]).view(B, N, H * d))
    gqq, _, gqn, _ = R().head_norm_rotary_bwd(q, None, table, gq, None, w["qn"])
    gx2, gwq, _ = R().linear_bwd(x, w["wq"], gqq.transpose(1, 2).reshape(T, H * d), bias_grad=False)
    gwo_full = torch.zeros_like(w["wo"])
    gwo_full[:, :D] = gwo
    got = dict(x=gx + gy + gx2, wo=gwo_full, wg=gwg, wu=gwu, wd=gwd, wq=gwq, qn=gqn)
    rng, step = np.random.default_rng(7), 1e-5
    for n, v in got.items():
        base = xr if n == "x" else wr[n]
        for _ in range(3):
            e = rng.standard_normal(base.shape)
            hi, lo = base + step * e, base - step * e
            ref = ((whole(hi, wr) - whole(lo, wr)) if n == "x" else (whole(xr, {**wr, n: hi}) - whole(xr, {**wr, n: lo}))) / (2 * step)
            have = float(np.sum(v.double().cpu().numpy() * e))
            size = float(np.sqrt(np.sum(v.double().cpu().numpy() ** 2)))       # of a random direction's value
            assert abs(have - ref) <= 1e-4 * size, (n, have, ref)


def calls(M, dtype):
    """Each operator with rows M as (name, call with a workspace or none)."""
    x, w = draw(60, (M, 136), dtype)[0], draw(61, (264, 136), dtype, 0.1)[0]
    wd, gy = draw(62, (136, 264), dtype, 0.1)[0], draw(63, (M, 264), dtype)[0]
    odd, wodd = draw(64, (M, 65), dtype)[0], draw(65, (70, 65), dtype, 0.1)[0]
    gyo = draw(66, (M, 70), dtype)[0]
    z, g2 = draw(67, (M, 264), dtype)[0], draw(68, (M, 136), dtype)[0]
    q, hw = draw(69, (2, 3, M, 32), dtype)[0], draw(70, (32,), dtype)[0]
    table = R().rotary_table(R().rotary_frequencies(32), M)
    torch.cuda.synchronize()
    f = R()
    return [
        ("linear", lambda **k: (f.linear_fwd(x, w, activation="gelu", **k),)),
        ("linear odd", lambda **k: (f.linear_fwd(odd, wodd, **k),)),
        ("linear bwd", lambda **k: f.linear_bwd(x, w, gy, pre=z, activation="silu", **k)),
        ("linear bwd odd", lambda **k: f.linear_bwd(odd, wodd, gyo, **k)),
        ("ffn", lambda **k: f.gated_ffn_fwd(x, w, w, wd, return_pre=True, **k)),
        ("ffn bwd", lambda **k: f.gated_ffn_bwd(x, w, w, wd, z, gy, g2, **k)),
        ("heads bwd", lambda **k: f.head_norm_rotary_bwd(q, q, table, q, q, hw, hw, **k)),
    ]


@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M", [3, 300])
def test_graphs_over_one_workspace(M, dtype):
    """Two captured graphs of all operators whose calls share one workspace, replayed in turn with
    eager work between, give what eager calls give, bit for bit."""
    print(f"\n[case] graphs {M} {dtype}", flush=True)
    ops = calls(M, dtype)
    want = [op() for _, op in ops]
    ws = torch.empty(32 << 20, dtype=torch.uint8, device="cuda")
    for _, op in ops:                                       # (with the workspace, before the capture)
        op(workspace=ws)
    torch.cuda.synchronize()
    graphs = []
    for _ in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            out = [op(workspace=ws) for _, op in ops]
        graphs.append((g, out))
    for turn in range(3):
        for g, out in graphs:
            for o in out:
                for t in o:
                    if t is not None:
                        t.fill_(7.0)
            ws.fill_(0xFF)                                  # (NaN in both types)
            g.replay()
            torch.cuda.synchronize()
            for (name, op), o, ref in zip(ops, out, want):
                for a, b in zip(o, ref):
                    assert (a is None and b is None) or torch.equal(a, b), (turn, name)
            again = ops[turn][1]()
            assert all(b is None or torch.equal(a, b) for a, b in zip(again, want[turn]))


def test_streams_and_repeats():
    """Calls on streams of their own, at the same time, with workspaces of their own, repeat the
    results of one after the other; so do calls again."""
    print("\n[case] streams", flush=True)
    ops = calls(500, "bf16")
    want = [op() for _, op in ops]
    torch.cuda.synchronize()
    streams = [torch.cuda.Stream() for _ in range(3)]
    outs = []
    for i in range(9):
        for j, (_, op) in enumerate(ops):
            s = streams[(i + j) % 3]
            outs.append((j, op(stream=s)))
    torch.cuda.synchronize()
    for j, o in outs:
        assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(o, want[j])), ops[j][0]


def test_poisoned_memory_is_not_read():
    """Workspaces of NaN, and outputs over memory that held NaN, change nothing."""
    print("\n[case] poisoned", flush=True)
    for dtype in ("bf16", "f32"):
        for M in (5, 130, 1100):
            for name, op in calls(M, dtype):
                want = op()
                ws = torch.full((64 << 20,), 0xFF, dtype=torch.uint8, device="cuda")
                got = op(workspace=ws)
                assert all((a is None and b is None) or torch.equal(a, b) for a, b in zip(got, want)), (name, M, dtype)


def test_what_lies_around_is_left_alone():
    """Outputs inside larger buffers, at odd addresses: nothing before or behind them is written."""
    print("\n[case] guards", flush=True)
    for dtype in ("bf16", "f32"):
        for M, Nn, K in ((1, 5, 40), (20, 33, 65), (130, 70, 64), (300, 129, 130)):
            x, w = draw(80, (M, K), dtype)[0], draw(81, (Nn, K), dtype)[0]
            want = R().linear_fwd(x, w)
            buf = torch.full((M * Nn + 2002,), 3.0, dtype=x.dtype, device="cuda")
            out = buf[1001:1001 + M * Nn].view(M, Nn)
            R().linear_fwd(x, w, out=out)
            assert torch.equal(out, want) and (buf[:1001] == 3).all() and (buf[1001 + M * Nn:] == 3).all()


def test_profile_kinds():
    print("\n[case] profile", flush=True)
    ops = calls(300, "bf16")
    R().profile_enable(True)
    for _, op in ops:
        op()
    kinds = R().profile_read()
    R().profile_enable(False)
    for n in ("projection", "projection_pass", "head_norm_rotary", "gradient_sums"):
        assert kinds[n]["launches"] > 0, kinds
