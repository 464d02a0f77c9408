"""The operators that stand in front of, beside and in place of the retention in a block: what is measured.

Four operators, in each direction that a user runs them:

  norm    layer normalisation in front of a mixer: forward, and backward with the weight's and bias's gradients
  rotary  rotation of queries and keys by their positions, the step before the retention: forward and backward
  conv    the short causal convolution in front of the selective scan: prompt, backward, one token
  scan    the selective state-space scan (per-channel, per-token decays): prompt, backward, one token

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once), or, with
`own` set, through retnet_retention_fwd_amd.  Sizes: model width 1024, inner width 2048 (twice the model
width), heads of 128, 2048 to 16384 tokens and a decode batch of 128 are this repository's layer, train,
long and decode workloads.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EB = {"bf16": 2, "f32": 4}


# ------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the pre-normalisation of a training step: 8 sequences of 2048 tokens, inner width, bf16 weights
        dict(name="norm fwd train", op="norm", way="fwd", rows=16384, D=2048, dtype="bf16", wtype="bf16", bias=True),
        # its gradient in a float32 model of an odd width, with float32 weights
        dict(name="norm bwd odd f32", op="norm", way="bwd", rows=8200, D=1111, dtype="f32", wtype="f32", bias=True),
        # a long prompt's queries and keys, rotated whole, as the projections leave them (token-major rows)
        dict(name="rotary prompt", op="rotary", way="fwd", B=1, H=16, Hk=16, N=16384, d=128, rot=128, dtype="bf16",
             interleaved=True, major="token", scaling=1.0, ragged=False),
        # the rotation's gradient in a training step, halves of a part of the head, scaled for a longer context
        dict(name="rotary bwd half", op="rotary", way="bwd", B=4, H=8, Hk=8, N=2048, d=128, rot=64, dtype="bf16",
             interleaved=False, major="head", scaling=4.0, ragged=False),
        # one token of 128 sequences, each at a position of its own
        dict(name="rotary token", op="rotary", way="fwd", B=128, H=32, Hk=32, N=1, d=128, rot=128, dtype="bf16",
             interleaved=True, major="head", scaling=1.0, ragged=True),
        # prompts of different lengths, padded, read from one half of a wider projection, with a state to keep
        dict(name="conv prompt", op="conv", way="fwd", B=2, N=8191, D=2048, K=4, dtype="bf16", silu=True, wide=True,
             ragged=True),
        # the convolution's gradient in a training step
        dict(name="conv bwd train", op="conv", way="bwd", B=4, N=2048, D=2048, K=4, dtype="bf16", silu=True,
             wide=False, ragged=False),
        # one token of 128 sequences
        dict(name="conv token", op="conv", way="step", B=128, N=1, D=2048, K=4, dtype="bf16", silu=True, wide=False,
             ragged=False),
        # a training step's forward scan, gated
        dict(name="scan train", op="scan", way="fwd", B=4, N=2048, D=2048, G=1, S=16, dtype="bf16", gate=True,
             wide=False, ragged=False),
        # one long prompt continued from a state: few channels, many tokens
        dict(name="scan long", op="scan", way="fwd", B=1, N=16384, D=2048, G=1, S=16, dtype="bf16", gate=True,
             wide=True, ragged=False),
        # a training step's gradients of everything the scan takes
        dict(name="scan bwd train", op="scan", way="bwd", B=4, N=2048, D=2048, G=1, S=16, dtype="bf16", gate=True,
             wide=False, ragged=False),
        # one token of 128 sequences
        dict(name="scan token", op="scan", way="step", B=128, N=1, D=2048, G=1, S=16, dtype="bf16", gate=True,
             wide=False, ragged=False),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op, way = rng.choice([("norm", "fwd"), ("norm", "bwd"), ("rotary", "fwd"), ("rotary", "bwd"), ("conv", "fwd"),
                          ("conv", "bwd"), ("conv", "step"), ("scan", "fwd"), ("scan", "bwd"), ("scan", "step")])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "norm":
        D = _spread(rng, 64, 8192)
        rows = _spread(rng, 1, max(1, min(32768, (1 << 25) // D)))
        wtype = rng.choice([dtype, "f32"])
        return dict(op=op, way=way, rows=rows, D=D, dtype=dtype, wtype=wtype, bias=rng.random() < 0.7)
    if op == "rotary":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        rot = rng.choice([d, d, d // 2])
        H = _spread(rng, 1, 32)
        Hk = rng.choice([H, H, max(1, H // 4)])
        B = _spread(rng, 1, 64)
        N = _spread(rng, 1, max(1, min(32768, (1 << 25) // (B * H * d))))
        return dict(op=op, way=way, B=B, H=H, Hk=Hk, N=N, d=d, rot=rot, dtype=dtype, interleaved=rng.random() < 0.5,
                    major=rng.choice(["head", "token"]), scaling=rng.choice([1.0, 4.0]), ragged=rng.random() < 0.4)
    wide, ragged = rng.random() < 0.5, way != "step" and rng.random() < 0.4
    if op == "conv":
        D = _spread(rng, 64, 8192)
        B = _spread(rng, 1, 256) if way == "step" else _spread(rng, 1, 16)
        N = 1 if way == "step" else _spread(rng, 1, max(1, min(16384, (1 << 24) // (B * D))))
        return dict(op=op, way=way, B=B, N=N, D=D, K=rng.choice([2, 3, 4, 4]), dtype=dtype, silu=rng.random() < 0.7,
                    wide=wide, ragged=ragged)
    G = rng.choice([1, 1, 2, 4])
    D = G * _spread(rng, 32, 4096 // G)
    S = rng.choice([8, 16, 16, 16, 32, rng.randint(1, 24)])
    most = (1 << 24) // D * 16 // max(16, S)
    B = _spread(rng, 1, min(256, max(1, most))) if way == "step" else _spread(rng, 1, 8)
    N = 1 if way == "step" else _spread(rng, 1, max(1, min(16384, most // B)))
    return dict(op=op, way=way, B=B, N=N, D=D, G=G, S=S, dtype=dtype, gate=rng.random() < 0.7, wide=wide,
                ragged=ragged)


# ------------------------------------------------------------------------------------------------------ inputs
def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def _rows(g, case, *lead, width):
    """[*lead, width] rows; with `wide`, one half of rows twice as wide, as a joint projection leaves them."""
    t = DT[case["dtype"]]
    if case["wide"]:
        return _normal(g, *lead, 2 * width, dtype=t)[..., :width]
    return _normal(g, *lead, width, dtype=t)


def _lengths(g, case):
    """Tokens of each padded sequence (None: all of them): the longest one fills the batch."""
    if not case["ragged"]:
        return None
    n = torch.randint(1, case["N"] + 1, (case["B"],), generator=g, device="cuda", dtype=torch.int32)
    n[0] = case["N"]
    return n


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    t = DT[case["dtype"]]
    if case["op"] == "norm":
        rows, D, wt = case["rows"], case["D"], DT[case["wtype"]]
        s["x"] = (_normal(g, rows, D, scale=2.0) + _normal(g, rows, 1)).to(t)   # a residual stream's rows
        s["w"] = (1.0 + _normal(g, D, scale=0.2)).to(wt)
        s["b"] = _normal(g, D, scale=0.2, dtype=wt) if case["bias"] else None
        s["eps"] = 1e-5
        if case["way"] == "bwd":
            x = s["x"].double()
            mean = x.mean(1)
            s["mean"] = mean.float()
            s["rstd"] = ((x - mean[:, None]).square().mean(1) + s["eps"]).rsqrt().float()
            s["gy"] = _normal(g, rows, D, dtype=t)
    elif case["op"] == "rotary":
        B, H, Hk, N, d, rot = (case[k] for k in ("B", "H", "Hk", "N", "d", "rot"))
        far = N + (4096 if case["ragged"] else 0)          # positions that the kept table covers
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot) / case["scaling"]
        ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * freq
        s["freq"], s["table"] = freq, torch.stack((ang.cos(), ang.sin()), dim=-1).float()

        def heads(h):
            if case["major"] == "token":
                return _normal(g, B, N, h, d, dtype=t).transpose(1, 2)
            return _normal(g, B, h, N, d, dtype=t)

        s["q"], s["k"] = heads(H), heads(Hk)
        s["pos"] = None
        if case["ragged"]:                                 # each sequence continues at a position of its own
            s["pos"] = torch.randint(0, 4096, (B, 1), generator=g, device="cuda") + torch.arange(N, device="cuda")
        s["k_scale"] = d ** -0.5
    elif case["op"] == "conv":
        B, N, D, K = (case[k] for k in ("B", "N", "D", "K"))
        s["x"] = _rows(g, case, *([B, N] if case["way"] != "step" else [B]), width=D)
        s["w"], s["b"] = _normal(g, D, K, scale=K ** -0.5, dtype=t), _normal(g, D, scale=0.2, dtype=t)
        s["state"] = _normal(g, B, K - 1, D, dtype=t)
        s["lengths"] = _lengths(g, case)
        if case["way"] == "fwd":
            s["y"] = torch.zeros(B, N, D, dtype=t, device="cuda")
        if case["way"] == "bwd":
            s["gy"], s["gstate"] = _normal(g, B, N, D, dtype=t), _normal(g, B, K - 1, D, dtype=t)
    else:
        B, N, D, G, S = (case[k] for k in ("B", "N", "D", "G", "S"))
        lead = [B, N] if case["way"] != "step" else [B]
        s["x"] = _rows(g, case, *lead, width=D)
        s["z"] = _rows(g, case, *lead, width=D) if case["gate"] else None
        s["dt"] = _normal(g, *lead, D, scale=0.5, dtype=t)
        rank = 32 if case["wide"] else 0                   # B and C as column slices behind a low-rank part
        bc = _normal(g, *lead, rank + 2 * G * S, dtype=t)
        s["Bm"] = bc[..., rank:rank + G * S].unflatten(-1, (G, S))
        s["Cm"] = bc[..., rank + G * S:].unflatten(-1, (G, S))
        s["A"] = -torch.arange(1, S + 1, dtype=torch.float32, device="cuda") * torch.exp(_normal(g, D, S, scale=0.2))
        s["Dskip"] = _normal(g, D)
        step = torch.exp(torch.rand(D, generator=g, device="cuda") * math.log(100.0) + math.log(1e-3))
        s["bias"] = step + torch.log(-torch.expm1(-step))  # softplus(bias) spreads over 1e-3 .. 1e-1
        s["state"] = _normal(g, B, D, S, scale=0.5)
        s["lengths"] = _lengths(g, case)
        if case["way"] == "fwd":
            s["y"] = torch.zeros(B, N, D, dtype=t, device="cuda")
        if case["way"] == "bwd":
            s["gy"], s["gstate"] = _normal(g, B, N, D, dtype=t), _normal(g, B, D, S, scale=0.1)
    return s


# ------------------------------------------------------------------------------------------------- plain forms
def _sigmoid(x):
    return 1.0 / (1.0 + torch.exp(-x))


def _softplus(x):
    return torch.where(x > 20.0, x, torch.log1p(torch.exp(torch.clamp(x, max=20.0))))


def _plain_norm(s):
    x = s["x"].float()
    w = s["w"].float()
    if s["way"] == "fwd":
        mean = x.mean(1, keepdim=True)
        xc = x - mean
        rstd = (xc.square().mean(1, keepdim=True) + s["eps"]).rsqrt()
        y = xc * rstd * w
        y = y if s["b"] is None else y + s["b"].float()
        return y.to(s["x"].dtype), mean[:, 0], rstd[:, 0]
    gy = s["gy"].float()
    xh = (x - s["mean"][:, None]) * s["rstd"][:, None]
    gw = gy * w
    gx = (gw - gw.mean(1, keepdim=True) - xh * (gw * xh).mean(1, keepdim=True)) * s["rstd"][:, None]
    gb = None if s["b"] is None else gy.sum(0).to(s["w"].dtype)
    return gx.to(s["x"].dtype), (gy * xh).sum(0).to(s["w"].dtype), gb


def _plain_rotary(s):
    N, rot = s["N"], s["rot"]
    cs = s["table"][:N][None] if s["pos"] is None else s["table"][s["pos"]]      # [1 or B, N, rot/2, 2]
    c, sn = cs[..., 0][:, None], cs[..., 1][:, None]
    sn = -sn if s["way"] == "bwd" else sn

    def turn(x, scale):
        f = x.float()
        part, rest = f[..., :rot], f[..., rot:]
        a, b = (part[..., 0::2], part[..., 1::2]) if s["interleaved"] else (part[..., :rot // 2], part[..., rot // 2:])
        a, b = a * c - b * sn, a * sn + b * c
        part = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
        return (torch.cat((part, rest), -1) * scale).to(x.dtype)

    return turn(s["q"], 1.0), turn(s["k"], s["k_scale"])


def _in_length(s):
    """[B, N, 1]: whether a token is one of its sequence's, or None where all are."""
    if s["lengths"] is None:
        return None
    return (torch.arange(s["N"], device="cuda")[None, :] < s["lengths"][:, None])[..., None]


def _windows(xs, w, N):
    """sum_j w[:, j] xs[:, j : j + N] for xs [B, N + K - 1, D]."""
    return sum(w[:, j] * xs[:, j:j + N] for j in range(w.shape[1]))


def _plain_conv(s):
    K, N = s["K"], s["N"]
    t = s["x"].dtype
    w, b = s["w"].float(), s["b"].float()
    x = s["x"].float() if s["way"] != "step" else s["x"].float()[:, None]
    xs = torch.cat((s["state"].float(), x), 1)                                   # [B, K-1+N, D]
    pre = _windows(xs, w, N) + b
    keep = _in_length(s)
    tail = torch.arange(K - 1, device="cuda")[None] + (N if keep is None else s["lengths"][:, None])
    tail = tail.expand(s["B"], K - 1)[..., None].expand(-1, -1, s["D"])
    if s["way"] != "bwd":
        y = pre * _sigmoid(pre) if s["silu"] else pre
        last = xs.gather(1, tail).to(t)
        if s["way"] == "step":
            s["state"].copy_(last)
            return y[:, 0].to(t), s["state"]
        return (y if keep is None else torch.where(keep, y, 0.0)).to(t), last
    gp = s["gy"].float()
    if s["silu"]:
        sg = _sigmoid(pre)
        gp = gp * (sg + pre * sg * (1.0 - sg))
    gp = gp if keep is None else torch.where(keep, gp, 0.0)
    pad = torch.zeros(s["B"], K - 1, s["D"], device="cuda")
    gxs = _windows(torch.cat((pad, gp, pad), 1), w.flip(1), N + K - 1)
    gxs = gxs.scatter_add(1, tail, s["gstate"].float())
    gw = torch.stack([(gp * xs[:, j:j + N]).sum((0, 1)) for j in range(K)], 1)
    return gxs[:, K - 1:].to(t), gw.to(t), gp.sum((0, 1)).to(t), gxs[:, :K - 1].to(t)


def _doubling(a, u):
    """h_t = a_t h_(t-1) + u_t along axis 1 for all t, by doubling the span that each step covers."""
    a, h, k = a.clone(), u.clone(), 1
    while k < h.shape[1]:
        h[:, k:] += a[:, k:] * h[:, :-k]
        a[:, k:] = a[:, k:] * a[:, :-k]
        k *= 2
    return h


def _plain_scan(s):
    t, B, N, D, G, S = s["x"].dtype, s["B"], s["N"], s["D"], s["G"], s["S"]
    lift = (lambda v: v.float()[:, None]) if s["way"] == "step" else (lambda v: v.float())
    x, raw = lift(s["x"]), lift(s["dt"]) + s["bias"]
    dt = _softplus(raw)
    keep = _in_length(s)
    if keep is not None:                   # a token behind its sequence's last leaves the state as it is
        dt = torch.where(keep, dt, 0.0)
    spread = lambda v: lift(v).repeat_interleave(D // G, 2)                      # noqa: E731  [B, N, D, S]
    Bd, Cd = spread(s["Bm"]), spread(s["Cm"])
    a = torch.exp(dt[..., None] * s["A"])
    u = (dt * x)[..., None] * Bd
    u[:, 0] += a[:, 0] * s["state"]
    h = _doubling(a, u)
    ys = (h * Cd).sum(-1) + x * s["Dskip"]
    z = None if s["z"] is None else lift(s["z"])
    if s["way"] != "bwd":
        y = ys if z is None else ys * (z * _sigmoid(z))
        if s["way"] == "step":
            s["state"].copy_(h[:, 0])
            return y[:, 0].to(t), s["state"]
        return (y if keep is None else torch.where(keep, y, 0.0)).to(t), h[:, -1].contiguous()
    gy = s["gy"].float()
    gy = gy if keep is None else torch.where(keep, gy, 0.0)
    gz = None
    if z is not None:
        sg = _sigmoid(z)
        gz, gy = (gy * ys * (sg + z * sg * (1.0 - sg))).to(t), gy * (z * sg)
    # adjoint: g_t = C_t gy_t + a_(t+1) g_(t+1), with the final state's gradient behind the last token
    c = gy[..., None] * Cd
    c[:, -1] += s["gstate"]
    later = torch.cat((torch.ones_like(a[:, :1]), a[:, 1:].flip(1)), 1)
    gh = _doubling(later, c.flip(1)).flip(1)
    before = torch.cat((s["state"][:, None], h[:, :-1]), 1)
    ga = gh * before * a                                                         # d / d (dt A)
    gu = (gh * Bd).sum(-1)
    gdt = (ga * s["A"]).sum(-1) + gu * x
    graw = gdt * _sigmoid(raw)
    graw = graw if keep is None else torch.where(keep, graw, 0.0)
    groups = lambda v: v.unflatten(2, (G, D // G)).sum(3)                        # noqa: E731  [B, N, G, S]
    return ((gu * dt + gy * s["Dskip"]).to(t), graw.to(t), (ga * dt[..., None]).sum((0, 1)),
            groups(gh * (dt * x)[..., None]).to(t), groups(h * gy[..., None]).to(t), (gy * x).sum((0, 1)), gz,
            graw.sum((0, 1)), gh[:, 0] * a[:, 0])


PLAIN = {"norm": _plain_norm, "rotary": _plain_rotary, "conv": _plain_conv, "scan": _plain_scan}


# --------------------------------------------------------------------------------------------------- own calls
def _own(s):
    import retnet_retention_fwd_amd as R
    op, way = s["op"], s["way"]
    if op == "norm":
        if way == "fwd":
            return R.layer_norm_fwd(s["x"], s["w"], s["b"], eps=s["eps"], return_stats=True)
        return R.layer_norm_bwd(s["x"], s["w"], s["mean"], s["rstd"], s["gy"], bias_grad=s["b"] is not None)
    if op == "rotary":
        f = R.rotary_fwd if way == "fwd" else R.rotary_bwd
        return f(s["q"], s["k"], s["table"], positions=s["pos"], interleaved=s["interleaved"], k_scale=s["k_scale"])
    if op == "conv":
        if way == "fwd":
            return R.causal_conv_fwd(s["x"], s["w"], s["b"], silu=s["silu"], state_in=s["state"], return_state=True,
                                     lengths=s["lengths"])      # which writes the rows behind the ends as zeros
        if way == "step":
            return R.causal_conv_step(s["x"], s["w"], s["state"], s["b"], silu=s["silu"]), s["state"]
        return R.causal_conv_bwd(s["x"], s["w"], s["gy"], s["b"], silu=s["silu"], state_in=s["state"],
                                 grad_state_out=s["gstate"], lengths=s["lengths"], return_grad_state_in=True)
    if way == "fwd":
        return R.selective_scan_fwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], D=s["Dskip"], z=s["z"],
                                    dt_bias=s["bias"], softplus=True, state_in=s["state"], return_state=True,
                                    lengths=s["lengths"])
    if way == "step":
        return R.selective_scan_step(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["state"], D=s["Dskip"], z=s["z"],
                                     dt_bias=s["bias"], softplus=True), s["state"]
    return R.selective_scan_bwd(s["x"], s["dt"], s["A"], s["Bm"], s["Cm"], s["gy"], D=s["Dskip"], z=s["z"],
                                dt_bias=s["bias"], softplus=True, state_in=s["state"], grad_state_out=s["gstate"],
                                lengths=s["lengths"], return_grad_state_in=True)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; operations of the formulas, an exponential as one."""
    e = EB[case["dtype"]]
    if case["op"] == "norm":
        n, D, we = case["rows"] * case["D"], case["D"], EB[case["wtype"]]
        nb = 1 + int(case["bias"])
        if case["way"] == "fwd":
            return {"bytes": 2 * n * e + nb * D * we + 8 * case["rows"], "flops": 8 * n}
        return {"bytes": 3 * n * e + (1 + nb) * D * we + 8 * case["rows"], "flops": 13 * n}
    if case["op"] == "rotary":
        n = case["B"] * (case["H"] + case["Hk"]) * case["N"]
        table = case["N"] * case["rot"] * 4 * (case["B"] if case["ragged"] else 1)
        return {"bytes": 2 * n * case["d"] * e + table, "flops": 3 * n * case["rot"]}
    B, N, D = case["B"], case["N"], case["D"]
    n = B * N * D
    if case["op"] == "conv":
        K = case["K"]
        st = 2 * B * (K - 1) * D * e
        if case["way"] == "bwd":
            return {"bytes": 3 * n * e + 2 * D * (K + 1) * e + 1.5 * st, "flops": n * (6 * K + 10)}
        return {"bytes": 2 * n * e + D * (K + 1) * e + st, "flops": n * (2 * K + 4)}
    G, S = case["G"], case["S"]
    st, par, gate = 4 * B * D * S, 4 * D * (S + 2), int(case["gate"])
    bc = 2 * B * N * G * S * e
    if case["way"] == "bwd":        # reads x, dt, gy, B, C (z), writes the gradients of x, dt, B, C (z)
        return {"bytes": (5 + 2 * gate) * n * e + 2 * bc + 3 * st + 2 * par, "flops": n * (22 * S + 20)}
    return {"bytes": (3 + gate) * n * e + bc + 2 * st + par, "flops": n * (7 * S + 12)}


# ------------------------------------------------------------------------------------------------------- exact
def _exact_norm(s):
    x, w = s["x"].double(), s["w"].double()
    D = x.shape[1]
    if s["way"] == "fwd":
        mean = x.sum(1) / D
        var = (x * x).sum(1) / D - mean * mean
        rstd = 1.0 / torch.sqrt(var + s["eps"])
        y = (x - mean[:, None]) * (rstd[:, None] * w[None])
        return (y if s["b"] is None else y + s["b"].double()), mean, rstd
    xh = (x - s["mean"].double()[:, None]) * s["rstd"].double()[:, None]
    gy = s["gy"].double()
    v = gy * w
    dots = torch.stack((v.sum(1), (v * xh).sum(1))) / D
    gx = s["rstd"].double()[:, None] * (v - dots[0][:, None] - xh * dots[1][:, None])
    return gx, (gy * xh).sum(0), None if s["b"] is None else gy.sum(0)


def _exact_rotary(s):
    pos = torch.arange(s["N"], device="cuda")[None] if s["pos"] is None else s["pos"]
    turn = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), pos[..., None].double() * s["freq"])
    turn = (turn if s["way"] == "fwd" else turn.conj())[:, None]
    rot = s["rot"]

    def one(x, scale):
        x = x.double()
        if s["interleaved"]:
            c = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * turn
            part = torch.view_as_real(c).flatten(-2)
        else:
            c = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * turn
            part = torch.cat((c.real, c.imag), -1)
        return torch.cat((part, x[..., rot:]), -1) * scale

    return one(s["q"], 1.0), one(s["k"], s["k_scale"])


def _exact_conv(s):
    B, N, D, K = s["B"], s["N"], s["D"], s["K"]
    x = s["x"].double() if s["way"] != "step" else s["x"].double()[:, None]
    w, b, state = s["w"].double(), s["b"].double(), s["state"].double()
    n = [N] * B if s["lengths"] is None else s["lengths"].tolist()
    y, last = torch.zeros(B, N, D, dtype=torch.float64, device="cuda"), []
    gx, gs = torch.zeros_like(y), []
    gw, gb = torch.zeros(D, K, dtype=torch.float64, device="cuda"), torch.zeros(D, dtype=torch.float64, device="cuda")
    for i in range(B):
        xs = torch.cat((state[i], x[i, :n[i]]))
        win = xs.unfold(0, K, 1)                                   # [n, D, K]
        pre = (win * w).sum(-1) + b
        sg = torch.sigmoid(pre)
        if s["way"] != "bwd":
            y[i, :n[i]] = pre * sg if s["silu"] else pre
            last.append(xs[n[i]:])
            continue
        gp = s["gy"][i, :n[i]].double() * (sg * (1 + pre * (1 - sg)) if s["silu"] else 1.0)
        gw += (win * gp[..., None]).sum(0)
        gb += gp.sum(0)
        gxs = torch.zeros_like(xs)
        gxs[n[i]:] += s["gstate"][i].double()
        for j in range(K):
            gxs[j:j + n[i]] += gp * w[:, j]
        gx[i, :n[i]] = gxs[K - 1:]
        gs.append(gxs[:K - 1])
    if s["way"] == "bwd":
        return gx, gw, gb, torch.stack(gs)
    return (y[:, 0] if s["way"] == "step" else y), torch.stack(last)


def _exact_scan(s):
    B, N, D, G, S = s["B"], s["N"], s["D"], s["G"], s["S"]
    lift = (lambda v: v[:, None]) if s["way"] == "step" else (lambda v: v)
    x, Bm, Cm = (lift(s[k]) for k in ("x", "Bm", "Cm"))
    raw = lift(s["dt"]).double() + s["bias"].double()
    dt = torch.logaddexp(raw, torch.zeros_like(raw))
    n = torch.full((B,), N, device="cuda") if s["lengths"] is None else s["lengths"]
    A, skip = s["A"].double(), s["Dskip"].double()
    of = lambda v, i: v[:, i].double().repeat_interleave(D // G, 1)              # noqa: E731  [B, D, S]
    h = s["state"].double()
    ys = torch.zeros(B, N, D, dtype=torch.float64, device="cuda")
    seen = []
    for i in range(N):
        if s["way"] == "bwd":
            seen.append(h)
        on = (i < n)[:, None, None]
        xi = x[:, i].double()
        new = torch.exp(dt[:, i, :, None] * A) * h + (dt[:, i] * xi)[..., None] * of(Bm, i)
        h = torch.where(on, new, h)
        ys[:, i] = torch.where(on[..., 0], (h * of(Cm, i)).sum(-1) + skip * xi, 0.0)
    if s["way"] != "bwd":
        if s["z"] is not None:
            z = lift(s["z"]).double()
            ys = ys * z * torch.sigmoid(z)
        return (ys[:, 0] if s["way"] == "step" else ys), h
    gy = s["gy"].double() * (torch.arange(N, device="cuda")[None, :] < n[:, None])[..., None]
    gz = None
    if s["z"] is not None:
        z = s["z"].double()
        sg = torch.sigmoid(z)
        gz, gy = gy * ys * sg * (1 + z * (1 - sg)), gy * z * sg
    gx, gdt = torch.zeros_like(ys), torch.zeros_like(ys)
    gB = torch.zeros(B, N, G, S, dtype=torch.float64, device="cuda")
    gC, gA = torch.zeros_like(gB), torch.zeros_like(A)
    later = s["gstate"].double()                                                 # gradient of the state behind token i
    for i in reversed(range(N)):
        on = (i < n)[:, None, None]
        xi, di, gi = x[:, i].double(), dt[:, i], gy[:, i]
        a = torch.exp(di[..., None] * A)
        b = of(Bm, i)
        now = a * seen[i] + (di * xi)[..., None] * b
        gh = torch.where(on, later + gi[..., None] * of(Cm, i), 0.0)
        gu = (gh * b).sum(-1)
        ga = gh * seen[i] * a
        gx[:, i] = gu * di + gi * skip
        gdt[:, i] = (gu * xi + (ga * A).sum(-1)) * torch.sigmoid(raw[:, i])
        gB[:, i] = (gh * (di * xi)[..., None]).unflatten(1, (G, D // G)).sum(2)
        gC[:, i] = (now * gi[..., None]).unflatten(1, (G, D // G)).sum(2)
        gA += (ga * di[..., None]).sum(0)
        later = torch.where(on, gh * a, later)
    return gx, gdt, gA, gB, gC, (gy * x.double()).sum((0, 1)), gz, gdt.sum((0, 1)), later


def exact(case, seed):
    s = prepare(case, seed)
    return {"norm": _exact_norm, "rotary": _exact_rotary, "conv": _exact_conv, "scan": _exact_scan}[case["op"]](s)
