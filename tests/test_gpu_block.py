"""The block operators together, as a stack runs them: a retention block (norm, rotary, gated
retention) and a scan block (norm, convolution, scan), as prompts, token by token and backward;
in captured graphs, on other streams and with shared workspaces.

Whole chains run in fp32 and are held to the fp32 tolerance of the retention's tests, 1e-4 of the
largest reference value: each operator's own bound is a few hundred u = 2^-24 of its magnitudes
(their own tests), a chain of four with gains of order one stays below 2000 u = 1.2e-4 in the
worst case and the tolerance's norm is taken over the largest value.
"""
import numpy as np
import pytest

import oracle as O
from retnet_retention_fwd_amd import inputs as I

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

TOL = 1e-4


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def rel(got, ref):
    g = got.detach().double().cpu().numpy()
    assert np.all(np.isfinite(g))
    return float(np.max(np.abs(g - ref)) / np.max(np.abs(ref)))


def draw(rng, *shape, scale=1.0, dtype=torch.float32):
    t = torch.tensor(rng.standard_normal(shape) * scale).to(dtype)
    return t.cuda(), t.double().numpy()


def retention_case(seed, B=2, N=37, H=3, d=32):
    """Rows of width H*d that are q's, k's and v's source at once (no projections)."""
    r = np.random.default_rng(seed)
    c = {"x": draw(r, B, N, H * d), "w": draw(r, H * d), "b": draw(r, H * d),
         "g": I.to_dtype(I.logsigmoid(r.standard_normal((B, H, N))) / 16.0, "f32")}
    c["g"] = (c["g"][0].cuda(), c["g"][1])
    return c, R().rotary_frequencies(d, base=500.0)


def test_retention_block_prompt_and_tokens():
    print("\n[case] retention block", flush=True)
    B, N, H, d, cut = 2, 37, 3, 32, 20
    c, freq = retention_case(1)
    x, w, b, g = (c[n][0] for n in ("x", "w", "b", "g"))
    table = R().rotary_table(freq, 64)
    n_ref = O.layer_norm(c["x"][1], c["w"][1], c["b"][1])[0].reshape(B, N, H, d).transpose(0, 2, 1, 3)
    q_ref = O.rotary(n_ref, np.arange(N), freq.numpy())
    k_ref = q_ref * d ** -0.5
    o_ref, s_ref = O.gated_retention_recurrent(q_ref, k_ref, n_ref, c["g"][1])

    def mixer(rows, first):
        """Norm and rotation of rows [B, n, H*d] at positions first ..: q, k, v of [B,H,n,d]."""
        y = R().layer_norm_fwd(rows, w, b)
        heads = y.view(B, -1, H, d).transpose(1, 2)          # token-major, as a projection leaves it
        q, k = R().rotary_fwd(heads, heads, table, offset=first, k_scale=d ** -0.5)
        return q, k, heads.contiguous()

    q, k, v = mixer(x, 0)
    o, S = R().gated_retention_chunkwise_fwd(q, k, v, g, 16, return_state=True)
    assert rel(o, o_ref) <= TOL and rel(S, s_ref) <= TOL
    # a prompt and then tokens, each at its own position
    q, k, v = mixer(x[:, :cut].contiguous(), 0)
    _, S = R().gated_retention_chunkwise_fwd(q, k, v, g[:, :, :cut].contiguous(), 16, return_state=True)
    for t in range(cut, N):
        q, k, v = mixer(x[:, t:t + 1].contiguous(), t)
        o = R().gated_retention_decode_step(q[:, :, 0].contiguous(), k[:, :, 0].contiguous(), v[:, :, 0].contiguous(),
                                            g[:, :, t].contiguous(), S)
        assert rel(o, o_ref[:, :, t]) <= TOL, t
    assert rel(S, s_ref) <= TOL


def scan_block_case(seed, B=2, N=70, D=40, S=16, K=4, dtype=torch.float32):
    r = np.random.default_rng(seed)
    c = {"x": draw(r, B, N, D, dtype=dtype), "w": draw(r, D, dtype=dtype), "b": draw(r, D, dtype=dtype),
         "cw": draw(r, D, K, scale=0.6, dtype=dtype), "cb": draw(r, D, scale=0.2, dtype=dtype),
         "dt": draw(r, B, N, D, dtype=dtype), "Bm": draw(r, B, N, 1, S, dtype=dtype), "Cm": draw(r, B, N, 1, S, dtype=dtype),
         "z": draw(r, B, N, D, dtype=dtype), "D": draw(r, D), "bias": draw(r, D)}
    a = -np.exp(r.uniform(-2, 2, (D, S)))
    A = torch.tensor(a).float()
    c["A"] = (A.cuda(), A.double().numpy())
    return c


def scan_block_ref(v):
    y, mean, rstd = O.layer_norm(v["x"], v["w"], v["b"])
    u, cs = O.causal_conv(y, v["cw"], v["cb"], True)
    o, hs = O.selective_scan(u, v["dt"], v["A"], v["Bm"], v["Cm"], v["D"], v["z"], v["bias"], True)
    return y, mean, rstd, u, cs, o, hs


def test_scan_block_prompt_and_tokens():
    print("\n[case] scan block", flush=True)
    c = scan_block_case(2)
    t, v = ({n: p[i] for n, p in c.items()} for i in (0, 1))
    *_, cs_ref, o_ref, hs_ref = scan_block_ref(v)
    N, cut = 70, 45
    kw = dict(D=t["D"], dt_bias=t["bias"], softplus=True)
    y = R().layer_norm_fwd(t["x"], t["w"], t["b"])
    u, cs = R().causal_conv_fwd(y, t["cw"], t["cb"], silu=True, return_state=True)
    o, hs = R().selective_scan_fwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], return_state=True, **kw)
    assert rel(o, o_ref) <= TOL and rel(hs, hs_ref) <= TOL and rel(cs, cs_ref) <= TOL
    # a padded prompt of `cut` tokens, then one token at a time
    n = torch.full((2,), cut, dtype=torch.int32, device="cuda")
    u, cs = R().causal_conv_fwd(y, t["cw"], t["cb"], silu=True, return_state=True, lengths=n)
    _, hs = R().selective_scan_fwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], z=t["z"], return_state=True, lengths=n, **kw)
    for i in range(cut, N):
        y1 = R().layer_norm_fwd(t["x"][:, i].contiguous(), t["w"], t["b"])
        u1 = R().causal_conv_step(y1, t["cw"], cs, t["cb"], silu=True)
        o1 = R().selective_scan_step(u1, t["dt"][:, i], t["A"], t["Bm"][:, i], t["Cm"][:, i], hs, z=t["z"][:, i], **kw)
        assert rel(o1, o_ref[:, i]) <= TOL, i
    assert rel(hs, hs_ref) <= TOL and rel(cs, cs_ref) <= TOL


def scan_block_grads(t, go, workspaces=None):
    """Forward and backward of norm -> convolution -> scan for the gradient `go` of its output."""
    ws = workspaces or {}
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], softplus=True)
    y, mean, rstd = R().layer_norm_fwd(t["x"], t["w"], t["b"], return_stats=True)
    u = R().causal_conv_fwd(y, t["cw"], t["cb"], silu=True)
    o = R().selective_scan_fwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], workspace=ws.get("scan"), **kw)
    gu, *rest = R().selective_scan_bwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], go, workspace=ws.get("scan_bwd"), **kw)
    gy, gcw, gcb = R().causal_conv_bwd(y, t["cw"], gu, t["cb"], silu=True, workspace=ws.get("conv"))
    gx, gw, gb = R().layer_norm_bwd(t["x"], t["w"], mean, rstd, gy, workspace=ws.get("norm"))
    return (o, gx, gw, gb, gcw, gcb, *rest)


def test_scan_block_backward():
    print("\n[case] scan block backward", flush=True)
    c = scan_block_case(3)
    t, v = ({n: p[i] for n, p in c.items()} for i in (0, 1))
    go, gor = draw(np.random.default_rng(4), 2, 70, 40)
    got = scan_block_grads(t, go)
    y, mean, rstd, u, _, o, _ = scan_block_ref(v)
    gu, *rest, _ = O.selective_scan_bwd(u, v["dt"], v["A"], v["Bm"], v["Cm"], gor, v["D"], v["z"], v["bias"], True)
    gy, gcw, gcb, _ = O.causal_conv_bwd(y, v["cw"], gu, v["cb"], True)
    gx, gw, gb = O.layer_norm_bwd(v["x"].reshape(140, 40), v["w"], mean.ravel(), rstd.ravel(), gy.reshape(140, 40))
    gx = gx.reshape(2, 70, 40)
    for a, r in zip(got, (o, gx, gw, gb, gcw, gcb, *rest)):
        assert rel(a, r) <= TOL, (rel(a, r), tuple(a.shape))


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_results_repeat(dtype):
    """No order of execution shows in the results: ten runs, the same bits."""
    print("\n[case] repeats", flush=True)
    c = scan_block_case(5, B=3, N=300, D=200, dtype=dtype)
    t = {n: p[0] for n, p in c.items()}
    go, _ = draw(np.random.default_rng(6), 3, 300, 200, dtype=dtype)
    first = scan_block_grads(t, go)
    for _ in range(9):
        for a, b in zip(scan_block_grads(t, go), first):
            assert torch.equal(a, b)


def workspaces(B, N, D, S, K, code):
    from retnet_retention_fwd_amd import _block
    need = {"scan": R().scan_workspace_bytes(B, N, D, 1, S), "scan_bwd": R().scan_bwd_workspace_bytes(B, N, D, 1, S),
            "conv": _block._fn("causal_conv_bwd_workspace_bytes")(B, N, D, K, code),
            "norm": _block._fn("layer_norm_bwd_workspace_bytes")(B * N, D, code)}
    return {n: torch.empty(max(b, 1), dtype=torch.uint8, device="cuda") for n, b in need.items()}


def test_graphs_with_shared_workspaces():
    """Two captured training steps over one set of workspaces, replayed in turn with eager work
    between and new inputs in place: every replay's results are the eager ones'."""
    print("\n[case] graphs", flush=True)
    B, N, D = 2, 600, 72
    ws = workspaces(B, N, D, 16, 4, 1)
    sets = []
    for seed in (7, 8):
        c = scan_block_case(seed, B=B, N=N, D=D, dtype=torch.bfloat16)
        sets.append(({n: p[0] for n, p in c.items()}, draw(np.random.default_rng(seed + 10), B, N, D, dtype=torch.bfloat16)[0]))
    eager = [[a.clone() for a in scan_block_grads(t, go, ws)] for t, go in sets]
    torch.cuda.synchronize()
    graphs = []
    for t, go in sets:
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.stream(side):
            with torch.cuda.graph(graph, stream=side):
                out = scan_block_grads(t, go, ws)
        torch.cuda.current_stream().wait_stream(side)
        graphs.append((graph, out))
    for rep in range(4):
        for (graph, out), want in zip(graphs, eager):
            for a in out:
                a.zero_()
            graph.replay()
            torch.cuda.synchronize()
            for a, b in zip(out, want):
                assert torch.equal(a, b), rep
        scan_block_grads(*sets[rep % 2], ws)
        torch.cuda.synchronize()
    # other values in the captured inputs
    (t, go), (graph, out) = sets[0], graphs[0]
    t["x"].mul_(0.5)
    go.neg_()
    graph.replay()
    torch.cuda.synchronize()
    for a, b in zip(out, scan_block_grads(t, go, ws)):
        assert torch.equal(a, b)


def test_graph_of_decode_tokens():
    """A captured token of both mixers: its states move on with every replay."""
    print("\n[case] decode graph", flush=True)
    B, D, S, K, H, d = 3, 40, 16, 4, 2, 32
    c = scan_block_case(9, B=B, N=1, D=D)
    t = {n: p[0][:, 0].contiguous() if n in ("x", "dt", "Bm", "Cm", "z") else p[0] for n, p in c.items()}
    table = R().rotary_table(R().rotary_frequencies(d), 16)
    pos = torch.zeros(B, 1, dtype=torch.int64, device="cuda")
    q = torch.randn(B, H, 1, d, device="cuda", generator=torch.Generator("cuda").manual_seed(1))
    cs0 = torch.randn(B, K - 1, D, device="cuda", generator=torch.Generator("cuda").manual_seed(2))
    hs0 = torch.randn(B, D, S, device="cuda", generator=torch.Generator("cuda").manual_seed(3))

    def token(cs, hs):
        y = R().layer_norm_fwd(t["x"], t["w"], t["b"])
        u = R().causal_conv_step(y, t["cw"], cs, t["cb"], silu=True)
        o = R().selective_scan_step(u, t["dt"], t["A"], t["Bm"], t["Cm"], hs, D=t["D"], z=t["z"], dt_bias=t["bias"], softplus=True)
        rq, rk = R().rotary_fwd(q, q, table, positions=pos, interleaved=False)
        pos.add_(1)
        return o, rq, rk

    cs, hs = cs0.clone(), hs0.clone()
    want = []
    for _ in range(5):
        want.append([a.clone() for a in (*token(cs, hs), cs, hs)])
    pos.zero_()
    cs, hs = cs0.clone(), hs0.clone()
    torch.cuda.synchronize()
    graph, side = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        with torch.cuda.graph(graph, stream=side):
            out = token(cs, hs)
    torch.cuda.current_stream().wait_stream(side)
    for rep in range(5):
        graph.replay()
        torch.cuda.synchronize()
        for a, b in zip((*out, cs, hs), want[rep]):
            assert torch.equal(a, b), rep
        R().layer_norm_fwd(t["x"], t["w"], t["b"])


def test_explicit_stream():
    """stream= names a side stream: outputs and workspaces that the wrappers allocate belong to it,
    so memory that the current stream frees and reuses meanwhile is not theirs."""
    print("\n[case] explicit stream", flush=True)
    B, N, D = 2, 600, 72
    c = scan_block_case(11, B=B, N=N, D=D, dtype=torch.bfloat16)
    t = {n: p[0] for n, p in c.items()}
    go, _ = draw(np.random.default_rng(12), B, N, D, dtype=torch.bfloat16)
    kw = dict(D=t["D"], z=t["z"], dt_bias=t["bias"], softplus=True)
    table = R().rotary_table(R().rotary_frequencies(24), N)
    heads = t["x"].view(B, N, 3, 24).transpose(1, 2)

    def work(s):
        y, mean, rstd = R().layer_norm_fwd(t["x"], t["w"], t["b"], return_stats=True, stream=s)
        u = R().causal_conv_fwd(y, t["cw"], t["cb"], silu=True, stream=s)
        o, h = R().selective_scan_fwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], return_state=True, stream=s, **kw)
        g = R().selective_scan_bwd(u, t["dt"], t["A"], t["Bm"], t["Cm"], go, stream=s, **kw)
        gy, gcw, gcb = R().causal_conv_bwd(y, t["cw"], g[0], t["cb"], silu=True, stream=s)
        gn = R().layer_norm_bwd(t["x"], t["w"], mean, rstd, gy, stream=s)
        return (y, u, o, h, *g, gcw, gcb, *gn, *R().rotary_fwd(heads, heads, table, stream=s),
                R().rotary_table(R().rotary_frequencies(24), N, stream=s))

    ref = work(None)
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    outs = []
    for _ in range(3):
        side.wait_stream(torch.cuda.current_stream())
        outs.append(work(side))
        junk = [torch.full((n,), 255, dtype=torch.uint8, device="cuda") for n in (B * N * D * 2, B * N * D * 4, 1 << 20)]
        del junk
    side.synchronize()
    torch.cuda.synchronize()
    for out in outs:
        for a, b in zip(out, ref):
            assert torch.equal(a, b)
