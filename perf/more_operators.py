"""The projections, the feed-forward half and the head norms of a block around the retention: what is measured.

Three operators, in each direction that a user runs them:

  linear  a projection: matrix product with bias, activation and residual in its epilogue; its gradients
  ffn     the gated feed-forward block: gate and up projections, activation, product, down projection, residual;
          its gradients
  heads   root-mean-square norms of queries and keys for each head with the rotation by their positions in the
          same pass, the step between the projections and the retention; its gradients

`run` computes them in their plain form (elementary torch operations in 32 bits, rounded once), or, with
`own` set, through retnet_retention_fwd_amd.  Sizes: model widths 1024 and 2048, heads of 128, 2048 tokens of 4
sequences, prompts of 16384 tokens, a decode batch of 128 sequences with 32 heads (width 4096) are this
repository's layer, train, long and decode workloads; feed-forward widths are two to four times the model's.
"""
import math

import torch

own = False

DT = {"bf16": torch.bfloat16, "f32": torch.float32}
EB = {"bf16": 2, "f32": 4}
ACTIVATIONS = ["none", "relu", "gelu", "gelu_tanh", "silu"]


# ------------------------------------------------------------------------------------------------------- cases
def listed():
    return [
        # the output projection of one token of 128 sequences, added to the residual stream
        dict(name="linear token", op="linear", way="fwd", M=128, K=4096, N=4096, dtype="bf16", act="none", bias=False,
             residual=True, pre=False, wide=False),
        # the first projection of a training step's feed-forward, pre-activations kept for the gradient
        dict(name="linear train", op="linear", way="fwd", M=8192, K=1024, N=4096, dtype="bf16", act="gelu", bias=True,
             residual=False, pre=True, wide=False),
        # a float32 model of odd widths, reading a column slice of a wider projection
        dict(name="linear odd f32", op="linear", way="fwd", M=2047, K=1111, N=777, dtype="f32", act="silu", bias=True,
             residual=True, pre=False, wide=True),
        # the gradients of that first projection in a training step
        dict(name="linear bwd train", op="linear", way="bwd", M=8192, K=1024, N=4096, dtype="bf16", act="gelu",
             bias=True, residual=False, pre=True, wide=False),
        # gradients of a ragged batch's rows in odd widths
        dict(name="linear bwd odd", op="linear", way="bwd", M=3001, K=1111, N=777, dtype="bf16", act="none", bias=True,
             residual=False, pre=False, wide=False),
        # a single token of a single sequence, where the weights' bytes and the launches count
        dict(name="ffn one token", op="ffn", way="fwd", M=1, K=1024, N=4096, dtype="bf16", act="silu", residual=True,
             pre=False),
        # one token of 128 sequences
        dict(name="ffn token", op="ffn", way="fwd", M=128, K=2048, N=8192, dtype="bf16", act="silu", residual=True,
             pre=False),
        # a long prompt
        dict(name="ffn prompt", op="ffn", way="fwd", M=16384, K=2048, N=5632, dtype="bf16", act="silu", residual=True,
             pre=False),
        # the gradients of a training step
        dict(name="ffn bwd train", op="ffn", way="bwd", M=8192, K=1024, N=2816, dtype="bf16", act="silu",
             residual=False, pre=True),
        # a long prompt's queries and keys as the projections leave them (token-major rows)
        dict(name="heads prompt", op="heads", way="fwd", B=1, H=16, Hk=16, N=16384, d=128, rot=128, dtype="bf16",
             wtype="bf16", interleaved=True, major="token", ragged=False),
        # the gradients in a training step, halves of a part of the head
        dict(name="heads bwd train", op="heads", way="bwd", B=4, H=8, Hk=8, N=2048, d=128, rot=64, dtype="bf16",
             wtype="f32", interleaved=False, major="token", ragged=False),
        # one token of 128 sequences, each at a position of its own
        dict(name="heads token", op="heads", way="fwd", B=128, H=32, Hk=32, N=1, d=128, rot=128, dtype="bf16",
             wtype="bf16", interleaved=True, major="head", ragged=True),
    ]


def _spread(rng, lo, hi):
    """A whole number between lo and hi, even over its logarithm."""
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def _width(rng, lo, hi):
    """A width: most models' are multiples of 64, some are odd."""
    n = _spread(rng, lo, hi)
    return n if n < 64 or rng.random() < 0.4 else n // 64 * 64


def draw(rng):
    op = rng.choice(["linear", "ffn", "heads"])
    way = rng.choice(["fwd", "fwd", "bwd"])
    dtype = rng.choice(["bf16", "bf16", "f32"])
    if op == "heads":
        d = rng.choice([32, 64, 80, 96, 128, 256])
        H = _spread(rng, 1, 32)
        B = _spread(rng, 1, 64)
        return dict(op=op, way=way, B=B, H=H, Hk=rng.choice([H, H, max(1, H // 4)]),
                    N=_spread(rng, 1, max(1, min(32768, (1 << 25) // (B * H * d)))), d=d, rot=rng.choice([d, d, d // 2]),
                    dtype=dtype, wtype=rng.choice([dtype, "f32"]), interleaved=rng.random() < 0.5,
                    major=rng.choice(["head", "token"]), ragged=rng.random() < 0.4)
    K, N = _width(rng, 32, 8192), _width(rng, 32, 8192)
    most = 1 << (34 if op == "ffn" else 35)                # of M K N; float32's matrix rate is a fraction of bfloat16's
    most //= 8 if dtype == "f32" else 1
    M = _spread(rng, 1, max(1, min(16384, most // (K * N))))
    act = rng.choice(ACTIVATIONS) if op == "linear" else rng.choice(["silu", "silu", "gelu", "gelu_tanh", "relu"])
    case = dict(op=op, way=way, M=M, K=K, N=N, dtype=dtype, act=act, residual=way == "fwd" and rng.random() < 0.5,
                pre=act != "none" or op == "ffn" if way == "bwd" else rng.random() < 0.3)
    if op == "linear":
        case.update(bias=rng.random() < 0.6, wide=rng.random() < 0.3)
    return case


# ------------------------------------------------------------------------------------------------------ inputs
def _normal(g, *shape, scale=1.0, dtype=torch.float32):
    return (torch.randn(*shape, generator=g, device="cuda") * scale).to(dtype)


def prepare(case, seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    s = dict(case)
    t = DT[case["dtype"]]
    if case["op"] == "heads":
        B, H, Hk, N, d, rot = (case[k] for k in ("B", "H", "Hk", "N", "d", "rot"))
        far = N + (4096 if case["ragged"] else 0)          # positions that the kept table covers
        freq = 10000.0 ** (-torch.arange(0, rot, 2, dtype=torch.float64, device="cuda") / rot)
        ang = torch.arange(far, dtype=torch.float64, device="cuda")[:, None] * freq
        s["freq"], s["table"] = freq, torch.stack((ang.cos(), ang.sin()), dim=-1).float()

        def heads(h, scale):
            if case["major"] == "token":
                return _normal(g, B, N, h, d, scale=scale, dtype=t).transpose(1, 2)
            return _normal(g, B, h, N, d, scale=scale, dtype=t)

        s["q"], s["k"] = heads(H, 2.0), heads(Hk, 0.5)
        wt = DT[case["wtype"]]
        s["qw"], s["kw"] = ((1.0 + _normal(g, d, scale=0.2)).to(wt) for _ in range(2))
        s["eps"], s["k_scale"] = 1e-6, d ** -0.5
        s["pos"] = None
        if case["ragged"]:                                 # each sequence continues at a position of its own
            s["pos"] = torch.randint(0, 4096, (B, 1), generator=g, device="cuda") + torch.arange(N, device="cuda")
        if case["way"] == "bwd":
            s["gq"], s["gk"] = heads(H, 1.0), heads(Hk, 1.0)
        return s
    M, K, N = case["M"], case["K"], case["N"]
    if case["op"] == "linear":
        s["x"] = _normal(g, M, 2 * K if case["wide"] else K, dtype=t)[:, :K]
        s["w"] = _normal(g, N, K, scale=K ** -0.5, dtype=t)
        s["b"] = _normal(g, N, scale=0.2, dtype=t) if case["bias"] else None
        s["r"] = _normal(g, M, N, dtype=t) if case["residual"] else None
        if case["way"] == "bwd":
            s["gy"] = _normal(g, M, N, dtype=t)
            s["z"] = None
            if case["pre"]:                                # kept by the forward
                z = s["x"].float() @ s["w"].float().T
                s["z"] = (z if s["b"] is None else z + s["b"].float()).to(t)
        return s
    s["x"] = _normal(g, M, K, dtype=t)
    s["wg"], s["wu"] = (_normal(g, N, K, scale=K ** -0.5, dtype=t) for _ in range(2))
    s["wd"] = _normal(g, K, N, scale=N ** -0.5, dtype=t)
    s["r"] = _normal(g, M, K, dtype=t) if case["residual"] else None
    if case["way"] == "bwd":
        s["gy"] = _normal(g, M, K, dtype=t)
        s["g"], s["u"] = ((s["x"].float() @ s[w].float().T).to(t) for w in ("wg", "wu"))
    return s


# ------------------------------------------------------------------------------------------------- plain forms
_C, _C3 = math.sqrt(2.0 / math.pi), 0.044715


def _act(z, act):
    if act == "relu":
        return torch.clamp(z, min=0.0)
    if act == "gelu":
        return 0.5 * z * (1.0 + torch.erf(z * math.sqrt(0.5)))
    if act == "gelu_tanh":
        return 0.5 * z * (1.0 + torch.tanh(_C * (z + _C3 * z * z * z)))
    if act == "silu":
        return z / (1.0 + torch.exp(-z))
    return z


def _slope(z, act):
    if act == "relu":
        return (z > 0.0).to(z.dtype)
    if act == "gelu":
        return 0.5 * (1.0 + torch.erf(z * math.sqrt(0.5))) + z * torch.exp(-0.5 * z * z) / math.sqrt(2.0 * math.pi)
    if act == "gelu_tanh":
        th = torch.tanh(_C * (z + _C3 * z * z * z))
        return 0.5 * (1.0 + th) + 0.5 * z * (1.0 - th * th) * _C * (1.0 + 3.0 * _C3 * z * z)
    if act == "silu":
        sg = 1.0 / (1.0 + torch.exp(-z))
        return sg * (1.0 + z * (1.0 - sg))
    return torch.ones_like(z)


def _plain_linear(s):
    t, x, w = s["x"].dtype, s["x"].float(), s["w"].float()
    if s["way"] == "fwd":
        z = x @ w.T
        z = z if s["b"] is None else z + s["b"].float()
        y = _act(z, s["act"])
        y = (y if s["r"] is None else y + s["r"].float()).to(t)
        return (y, z.to(t)) if s["pre"] else y
    gz = s["gy"].float()
    if s["z"] is not None:
        gz = gz * _slope(s["z"].float(), s["act"])
    return (gz @ w).to(t), (gz.T @ x).to(t), gz.sum(0).to(t) if s["bias"] else None


def _plain_ffn(s):
    t = s["x"].dtype
    x, wg, wu, wd = (s[k].float() for k in ("x", "wg", "wu", "wd"))
    if s["way"] == "fwd":
        g, u = x @ wg.T, x @ wu.T
        y = (_act(g, s["act"]) * u) @ wd.T
        y = (y if s["r"] is None else y + s["r"].float()).to(t)
        return (y, g.to(t), u.to(t)) if s["pre"] else y
    g, u, gy = s["g"].float(), s["u"].float(), s["gy"].float()
    a, gh = _act(g, s["act"]), gy @ wd
    gg, gu = gh * u * _slope(g, s["act"]), gh * a
    return ((gg @ wg + gu @ wu).to(t), (gg.T @ x).to(t), (gu.T @ x).to(t), (gy.T @ (a * u)).to(t))


def _plain_heads(s):
    N, rot = s["N"], s["rot"]
    cs = s["table"][:N][None] if s["pos"] is None else s["table"][s["pos"]]      # [1 or B, N, rot/2, 2]
    c, sn = cs[..., 0][:, None], cs[..., 1][:, None]

    def turn(f, sn):
        part, rest = f[..., :rot], f[..., rot:]
        a, b = (part[..., 0::2], part[..., 1::2]) if s["interleaved"] else (part[..., :rot // 2], part[..., rot // 2:])
        a, b = a * c - b * sn, a * sn + b * c
        part = torch.stack((a, b), -1).flatten(-2) if s["interleaved"] else torch.cat((a, b), -1)
        return torch.cat((part, rest), -1)

    def fwd(x, w, scale):
        f = x.float()
        r = (f.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
        return (turn(f * r * w.float(), sn) * scale).to(x.dtype)

    def bwd(x, w, gy, scale):
        f = x.float()
        r = (f.square().mean(-1, keepdim=True) + s["eps"]).rsqrt()
        xh, g = f * r, turn(gy.float(), -sn) * scale
        v = g * w.float()
        gx = r * (v - xh * (v * xh).mean(-1, keepdim=True))
        return gx.to(x.dtype), (g * xh).sum((0, 1, 2)).to(w.dtype)

    if s["way"] == "fwd":
        return fwd(s["q"], s["qw"], 1.0), fwd(s["k"], s["kw"], s["k_scale"])
    (gq, gqw), (gk, gkw) = bwd(s["q"], s["qw"], s["gq"], 1.0), bwd(s["k"], s["kw"], s["gk"], s["k_scale"])
    return gq, gk, gqw, gkw


PLAIN = {"linear": _plain_linear, "ffn": _plain_ffn, "heads": _plain_heads}


# --------------------------------------------------------------------------------------------------- own calls
def _own(s):
    import retnet_retention_fwd_amd as R
    op, fwd = s["op"], s["way"] == "fwd"
    if op == "linear":
        if fwd:
            return R.linear_fwd(s["x"], s["w"], s["b"], residual=s["r"], activation=s["act"], return_pre=s["pre"])
        return R.linear_bwd(s["x"], s["w"], s["gy"], pre=s["z"], activation=s["act"], bias_grad=s["bias"])
    if op == "ffn":
        if fwd:
            return R.gated_ffn_fwd(s["x"], s["wg"], s["wu"], s["wd"], residual=s["r"], activation=s["act"],
                                   return_pre=s["pre"])
        return R.gated_ffn_bwd(s["x"], s["wg"], s["wu"], s["wd"], s["g"], s["u"], s["gy"], activation=s["act"])
    kw = dict(q_weight=s["qw"], k_weight=s["kw"], eps=s["eps"], positions=s["pos"], interleaved=s["interleaved"],
              k_scale=s["k_scale"])
    if fwd:
        return R.head_norm_rotary_fwd(s["q"], s["k"], s["table"], **kw)
    return R.head_norm_rotary_bwd(s["q"], s["k"], s["table"], s["gq"], s["gk"], **kw)


def run(state):
    return _own(state) if own else PLAIN[state["op"]](state)


# -------------------------------------------------------------------------------------------------------- work
def work(case):
    """Each input read once, each output written once; operations of the formulas, a function as one."""
    e, fwd = EB[case["dtype"]], case["way"] == "fwd"
    if case["op"] == "heads":
        n = case["B"] * (case["H"] + case["Hk"]) * case["N"]
        table = case["N"] * case["rot"] * 4 * (case["B"] if case["ragged"] else 1)
        w = 2 * case["d"] * EB[case["wtype"]]
        if fwd:
            return {"bytes": 2 * n * case["d"] * e + table + w, "flops": n * (5 * case["d"] + 3 * case["rot"])}
        return {"bytes": 3 * n * case["d"] * e + table + 2 * w, "flops": n * (12 * case["d"] + 3 * case["rot"])}
    M, K, N, pre = case["M"], case["K"], case["N"], int(case["pre"])
    if case["op"] == "linear":
        b = int(case["bias"]) * N
        if fwd:
            el = M * K + N * K + b + M * N * (1 + int(case["residual"]) + pre)
            return {"bytes": el * e, "flops": 2 * M * N * K + 4 * M * N}
        return {"bytes": (2 * (M * K + N * K) + b + M * N * (1 + pre)) * e, "flops": 4 * M * N * K + 6 * M * N}
    if fwd:
        el = M * K * (2 + int(case["residual"])) + 3 * N * K + 2 * M * N * pre
        return {"bytes": el * e, "flops": 6 * M * N * K + 6 * M * N}
    return {"bytes": (3 * M * K + 6 * N * K + 2 * M * N) * e, "flops": 12 * M * N * K + 12 * M * N}


# ------------------------------------------------------------------------------------------------------- exact
def _exact_act(z, act):
    """(value, slope) from the definitions: x P(x) with a distribution P, or a threshold."""
    if act == "none":
        return z, torch.ones_like(z)
    if act == "relu":
        on = z > 0
        return torch.where(on, z, 0.0), on.double()
    if act == "silu":
        p = torch.sigmoid(z)
        return z * p, p + z * p * torch.sigmoid(-z)
    if act == "gelu":
        p = 0.5 * torch.erfc(-z / math.sqrt(2.0))
        return z * p, p + z * torch.exp(-z * z / 2) * (0.5 / math.pi) ** 0.5
    q = 2 * math.sqrt(2 / math.pi) * (z + 0.044715 * z ** 3)                     # (1 + tanh(q/2)) / 2 = sigmoid(q)
    p = torch.sigmoid(q)
    return z * p, p + z * p * torch.sigmoid(-q) * 2 * math.sqrt(2 / math.pi) * (1 + 3 * 0.044715 * z ** 2)


def _exact_linear(s):
    x, w = s["x"].double(), s["w"].double()
    if s["way"] == "fwd":
        z = torch.matmul(x, w.t())
        if s["b"] is not None:
            z += s["b"].double()
        y = _exact_act(z, s["act"])[0]
        if s["r"] is not None:
            y = y + s["r"].double()
        return (y, z) if s["pre"] else y
    gz = s["gy"].double()
    if s["act"] != "none":
        gz = gz * _exact_act(s["z"].double(), s["act"])[1]
    return torch.matmul(gz, w), torch.matmul(gz.t(), x), gz.sum(0) if s["bias"] else None


def _exact_ffn(s):
    x, wg, wu, wd = (s[k].double() for k in ("x", "wg", "wu", "wd"))
    if s["way"] == "fwd":
        g, u = torch.matmul(x, wg.t()), torch.matmul(x, wu.t())
        y = torch.matmul(_exact_act(g, s["act"])[0] * u, wd.t())
        if s["r"] is not None:
            y = y + s["r"].double()
        return (y, g, u) if s["pre"] else y
    u, gy = s["u"].double(), s["gy"].double()
    a, da = _exact_act(s["g"].double(), s["act"])
    gwd = torch.matmul(gy.t(), a * u)
    gh = torch.matmul(gy, wd)
    both = torch.cat((gh * da * u, gh * a), 1)                                   # beside each other: [M, 2 N]
    gx = torch.matmul(both, torch.cat((wg, wu), 0))
    gw = torch.matmul(both.t(), x)
    return gx, gw[:s["N"]], gw[s["N"]:], gwd


def _exact_heads(s):
    pos = torch.arange(s["N"], device="cuda")[None] if s["pos"] is None else s["pos"]
    unit = torch.polar(torch.ones(1, dtype=torch.float64, device="cuda"), pos[..., None].double() * s["freq"])[:, None]
    rot, inter = s["rot"], s["interleaved"]

    def turn(x, by):
        if inter:
            z = torch.complex(x[..., 0:rot:2], x[..., 1:rot:2]) * by
            part = torch.view_as_real(z).flatten(-2)
        else:
            z = torch.complex(x[..., :rot // 2], x[..., rot // 2:rot]) * by
            part = torch.cat((z.real, z.imag), -1)
        return torch.cat((part, x[..., rot:]), -1)

    def one(x, w, scale, gy):
        x, w = x.double(), w.double()
        d = x.shape[-1]
        size = torch.sqrt((x * x).sum(-1, keepdim=True) / d + s["eps"])
        if gy is None:
            return turn(w * (x / size), unit) * scale
        back = turn(gy.double(), unit.conj()) * scale
        gw = (back * (x / size)).flatten(0, 2).sum(0)
        back = back * w
        return back / size - x * ((back * x).sum(-1, keepdim=True) / (d * size ** 3)), gw

    if s["way"] == "fwd":
        return one(s["q"], s["qw"], 1.0, None), one(s["k"], s["kw"], s["k_scale"], None)
    (gq, gqw), (gk, gkw) = one(s["q"], s["qw"], 1.0, s["gq"]), one(s["k"], s["kw"], s["k_scale"], s["gk"])
    return gq, gk, gqw, gkw


def exact(case, seed):
    s = prepare(case, seed)
    return {"linear": _exact_linear, "ffn": _exact_ffn, "heads": _exact_heads}[case["op"]](s)
