"""Refusals of the operators around the retention (no GPU: every call here fails validation
and returns before anything is enqueued)."""
import ctypes

import pytest

from retnet_retention_fwd_amd import _block, _lib

torch = pytest.importorskip("torch")

OK, ERR_NULL, ERR_SHAPE, ERR_DTYPE, ERR_UNSUPPORTED, ERR_WORKSPACE, ERR_ALIAS, ERR_HIP = range(8)
FAKE, MB = 1 << 40, 1 << 20
F32, BF16 = 0, 1


def at(i):
    return FAKE + i * 64 * MB


def call(name, defaults, **kw):
    assert not set(kw) - set(defaults), set(kw) - set(defaults)
    return _block._fn(name)(*{**defaults, **kw}.values())


def test_signatures_cover_the_header():
    for n in _block.SIGNATURES:
        assert n in _lib.EXPORTED


def norm_fwd(**kw):
    return call("layer_norm_fwd", dict(x=at(0), w=at(1), b=at(2), y=at(3), mean=at(4), rstd=at(5), rows=8, D=64, eps=1e-5,
                                       dt=BF16, wt=BF16, stream=None), **kw)


def norm_bwd(**kw):
    return call("layer_norm_bwd", dict(x=at(0), w=at(1), mean=at(2), rstd=at(3), gy=at(4), gx=at(5), gw=at(6), gb=at(7),
                                       rows=8, D=64, dt=BF16, wt=BF16, ws=at(8), wsb=64 * MB, stream=None), **kw)


def test_layer_norm():
    assert norm_fwd(dt=5) == ERR_DTYPE and norm_fwd(wt=7) == ERR_DTYPE
    assert norm_fwd(dt=F32, wt=BF16) == ERR_DTYPE
    assert norm_fwd(rows=-1) == ERR_SHAPE and norm_fwd(D=0) == ERR_SHAPE and norm_fwd(eps=-1.0) == ERR_SHAPE
    assert norm_fwd(eps=float("nan")) == ERR_SHAPE
    assert norm_fwd(D=(1 << 20) + 1) == ERR_UNSUPPORTED and norm_fwd(rows=1 << 40) == ERR_UNSUPPORTED
    assert norm_fwd(rows=(1 << 63) - 1, D=1 << 20) == ERR_UNSUPPORTED
    assert norm_fwd(x=None) == ERR_NULL and norm_fwd(y=None) == ERR_NULL
    assert norm_fwd(y=at(0)) == ERR_ALIAS and norm_fwd(mean=at(5) + 4) == ERR_ALIAS and norm_fwd(y=at(1) + 2) == ERR_ALIAS
    assert norm_fwd(rows=0) == OK
    assert norm_bwd(dt=F32, wt=BF16) == ERR_DTYPE and norm_bwd(D=-2) == ERR_SHAPE
    assert norm_bwd(mean=None) == ERR_NULL and norm_bwd(gx=None) == ERR_NULL
    assert norm_bwd(gx=at(4)) == ERR_ALIAS and norm_bwd(gw=at(7)) == ERR_ALIAS and norm_bwd(ws=at(0)) == ERR_ALIAS
    need = _block._fn("layer_norm_bwd_workspace_bytes")(8, 64, BF16)
    assert need > 0
    assert norm_bwd(ws=None) == ERR_WORKSPACE and norm_bwd(wsb=need - 1) == ERR_WORKSPACE
    assert norm_bwd(ws=at(8) + 4) == ERR_WORKSPACE
    assert norm_bwd(rows=0, gw=None, gb=None, ws=None, wsb=0) == OK
    assert _block._fn("layer_norm_bwd_workspace_bytes")(-1, 64, BF16) == 0


def strides(q=None, oq=None, k=None, ok=None, H=4, N=8, d=64):
    dense = (H * N * d, N * d, d)
    return (ctypes.c_longlong * 12)(*(q or dense), *(oq or dense), *(k or dense), *(ok or dense))


def rotary(name="rotary_fwd", **kw):
    return call(name, dict(q=at(0), k=at(1), oq=at(2), ok=at(3), st=strides(), table=at(4), length=100, pos=None, batched=0,
                           first=0, B=2, Hq=4, Hk=4, N=8, d=64, rot=64, inter=1, qs=1.0, ks=1.0, dt=BF16, stream=None), **kw)


@pytest.mark.parametrize("name", ["rotary_fwd", "rotary_bwd"])
def test_rotary(name):
    c = lambda **kw: rotary(name, **kw)  # noqa: E731
    assert c(dt=3) == ERR_DTYPE
    assert c(B=-1) == ERR_SHAPE and c(rot=0) == ERR_SHAPE and c(rot=3) == ERR_SHAPE and c(rot=66) == ERR_SHAPE
    assert c(first=-1) == ERR_SHAPE and c(first=93) == ERR_SHAPE and c(length=7) == ERR_SHAPE and c(length=-1) == ERR_SHAPE
    assert c(d=258, rot=64) == ERR_UNSUPPORTED and c(B=1 << 20, N=1 << 10) == ERR_UNSUPPORTED
    assert c(B=1 << 16, N=1 << 20) == ERR_UNSUPPORTED
    assert c(Hq=40000, Hk=40000) == ERR_UNSUPPORTED and c(length=1 << 62) == ERR_UNSUPPORTED
    assert c(st=strides(q=(1 << 62, 512, 64))) == ERR_SHAPE and c(st=strides(oq=(2048, 1 << 62, 64))) == ERR_SHAPE
    assert c(q=None) == ERR_NULL and c(ok=None) == ERR_NULL and c(table=None) == ERR_NULL and c(st=None) == ERR_NULL
    assert c(st=strides(q=(-1, 512, 64))) == ERR_SHAPE
    assert c(oq=at(0) + 128) == ERR_ALIAS                       # partly over its input
    assert c(oq=at(1)) == ERR_ALIAS and c(oq=at(3)) == ERR_ALIAS and c(ok=at(4)) == ERR_ALIAS
    assert c(oq=at(0), st=strides(oq=(2048, 64, 256))) == ERR_ALIAS   # in place in another order
    assert c(st=strides(oq=(0, 512, 64))) == ERR_ALIAS          # batches of the output over each other
    assert c(st=strides(oq=(2048, 512, 32))) == ERR_ALIAS
    assert c(B=0) == OK and c(N=0) == OK and c(Hq=0, Hk=0) == OK


def test_rotary_table():
    f = lambda **kw: call("rotary_table", dict(t=at(0), f=at(1), pairs=32, first=0, n=10, m=1.0, s=None), **kw)  # noqa: E731
    assert f(pairs=0) == ERR_SHAPE and f(n=-1) == ERR_SHAPE and f(first=-1) == ERR_SHAPE
    assert f(pairs=129) == ERR_UNSUPPORTED and f(n=1 << 32) == ERR_UNSUPPORTED and f(first=1 << 41) == ERR_UNSUPPORTED
    assert f(t=None) == ERR_NULL and f(f=None) == ERR_NULL and f(f=at(0) + 8) == ERR_ALIAS and f(n=0) == OK


def conv_fwd(**kw):
    return call("causal_conv_fwd", dict(x=at(0), ldx=64, w=at(1), b=at(2), y=at(3), si=at(4), so=at(5), n=at(6), B=2, N=8,
                                        D=64, K=4, silu=1, dt=BF16, wt=BF16, stream=None), **kw)


def conv_bwd(**kw):
    return call("causal_conv_bwd", dict(x=at(0), ldx=64, w=at(1), b=at(2), si=at(3), gy=at(4), gso=at(5), n=at(6), gx=at(7),
                                        gw=at(8), gb=at(9), gsi=at(10), B=2, N=8, D=64, K=4, silu=1, dt=BF16, wt=BF16,
                                        ws=at(11), wsb=64 * MB, stream=None), **kw)


def conv_step(**kw):
    return call("causal_conv_step", dict(x=at(0), ldx=64, w=at(1), b=at(2), s=at(3), y=at(4), B=2, D=64, K=4, silu=1,
                                         dt=BF16, wt=BF16, stream=None), **kw)


@pytest.mark.parametrize("f", [conv_fwd, conv_bwd, conv_step])
def test_causal_conv(f):
    assert f(dt=9) == ERR_DTYPE and f(dt=F32, wt=BF16) == ERR_DTYPE
    assert f(B=-1) == ERR_SHAPE and f(D=0) == ERR_SHAPE and f(K=0) == ERR_SHAPE and f(ldx=63) == ERR_SHAPE
    assert f(K=1) == ERR_UNSUPPORTED and f(K=5) == ERR_UNSUPPORTED
    assert f(B=1 << 20, D=1 << 14, ldx=1 << 14) == ERR_UNSUPPORTED
    assert f(ldx=1 << 26) == ERR_UNSUPPORTED and f(ldx=1 << 62) == ERR_UNSUPPORTED
    assert f(x=None) == ERR_NULL and f(w=None) == ERR_NULL


def test_causal_conv_buffers():
    assert conv_fwd(y=at(0)) == ERR_ALIAS and conv_fwd(so=at(4)) == ERR_ALIAS and conv_fwd(so=at(3) + 2) == ERR_ALIAS
    assert conv_fwd(y=None) == ERR_NULL and conv_fwd(B=0) == OK and conv_fwd(N=0, so=None) == OK
    assert conv_fwd(y=at(0) + 128, ldx=128) == ERR_ALIAS        # between the rows that are read
    assert conv_step(s=at(0)) == ERR_ALIAS and conv_step(y=at(3)) == ERR_ALIAS and conv_step(s=None) == ERR_NULL
    assert conv_step(B=0) == OK
    assert conv_bwd(gx=at(4)) == ERR_ALIAS and conv_bwd(gsi=at(5)) == ERR_ALIAS and conv_bwd(gw=at(9)) == ERR_ALIAS
    assert conv_bwd(gy=None) == ERR_NULL and conv_bwd(gx=None) == ERR_NULL
    need = _block._fn("causal_conv_bwd_workspace_bytes")(2, 8, 64, 4, BF16)
    assert need > 0 and conv_bwd(ws=None) == ERR_WORKSPACE and conv_bwd(wsb=need - 1) == ERR_WORKSPACE
    assert conv_bwd(ws=at(11) + 8) == ERR_WORKSPACE
    assert conv_bwd(B=1 << 26, N=1, D=1, ldx=1) == ERR_UNSUPPORTED       # more workgroups than a launch takes
    assert conv_bwd(B=1, N=(1 << 31) - 1, D=1, ldx=1) == ERR_UNSUPPORTED   # steps ahead of a token would wrap
    assert conv_bwd(N=0, gw=None, gb=None, gsi=None, ws=None) == OK


SCAN_IN = dict(x=at(0), dt=at(1), A=at(2), Bm=at(3), Cm=at(4), D=at(5), z=at(6), bias=at(7))
SCAN_LD = dict(ldx=64, lddt=64, ldz=64, ldb=16, ldc=16)


def scan_fwd(**kw):
    return call("selective_scan_fwd", dict(**SCAN_IN, y=at(8), si=at(9), so=at(10), n=at(11), **SCAN_LD, B=2, N=8, ch=64, G=1,
                                           S=16, sp=1, dtype=BF16, ws=at(12), wsb=64 * MB, stream=None), **kw)


def scan_bwd(**kw):
    return call("selective_scan_bwd", dict(**SCAN_IN, si=at(8), gy=at(9), gso=at(10), n=at(11), gx=at(12), gdt=at(13), gA=at(14),
                                           gB=at(15), gC=at(16), gD=at(17), gz=at(18), gbias=at(19), gsi=at(20), **SCAN_LD, B=2,
                                           N=8, ch=64, G=1, S=16, sp=1, dtype=BF16, ws=at(21), wsb=64 * MB, stream=None), **kw)


def scan_step(**kw):
    return call("selective_scan_step", dict(**SCAN_IN, s=at(8), y=at(9), **SCAN_LD, B=2, ch=64, G=1, S=16, sp=1, dtype=BF16,
                                            stream=None), **kw)


@pytest.mark.parametrize("f", [scan_fwd, scan_bwd, scan_step])
def test_selective_scan(f):
    assert f(dtype=9) == ERR_DTYPE
    assert f(B=-1) == ERR_SHAPE and f(S=0) == ERR_SHAPE and f(G=0) == ERR_SHAPE and f(ch=0) == ERR_SHAPE
    assert f(G=3, ldb=48, ldc=48) == ERR_SHAPE                  # groups that do not divide the channels
    for ld in ("ldx", "lddt", "ldz"):
        assert f(**{ld: 63}) == ERR_SHAPE
        assert f(**{ld: 1 << 26}) == ERR_UNSUPPORTED
    assert f(ldb=15) == ERR_SHAPE and f(ldc=15) == ERR_SHAPE and f(ldb=1 << 62) == ERR_UNSUPPORTED
    assert f(S=65, ldb=65, ldc=65) == ERR_UNSUPPORTED
    assert f(B=1 << 20, ch=1 << 12, ldx=1 << 12, lddt=1 << 12, ldz=1 << 12) == ERR_UNSUPPORTED
    for p in ("x", "dt", "A", "Bm", "Cm"):
        assert f(**{p: None}) == ERR_NULL, p


def test_selective_scan_buffers():
    assert scan_fwd(y=at(6)) == ERR_ALIAS and scan_fwd(so=at(9) + 4) == ERR_ALIAS and scan_fwd(so=at(8)) == ERR_ALIAS
    assert scan_fwd(y=None) == ERR_NULL and scan_fwd(B=0) == OK and scan_fwd(N=0, so=None) == OK
    assert scan_step(s=at(2)) == ERR_ALIAS and scan_step(y=at(0)) == ERR_ALIAS and scan_step(y=None) == ERR_NULL
    assert scan_step(B=0) == OK
    for a, b in (("gx", 9), ("gdt", 12), ("gA", 2), ("gB", 16), ("gD", 19), ("gz", 6), ("gsi", 10), ("ws", 0)):
        assert scan_bwd(**{a: at(b)}) == ERR_ALIAS, a
    for p in ("gy", "gx", "gdt", "gA", "gB", "gC", "gz"):
        assert scan_bwd(**{p: None}) == ERR_NULL, p
    need = _block.scan_bwd_workspace_bytes(2, 8, 64, 1, 16)
    assert need > 0 and scan_bwd(ws=None) == ERR_WORKSPACE and scan_bwd(wsb=need - 1) == ERR_WORKSPACE
    assert scan_bwd(ws=at(21) + 4) == ERR_WORKSPACE
    need = _block.scan_workspace_bytes(1, 4096, 64, 1, 16)       # few channels, many tokens: segments
    assert need > 0 and _block.scan_workspace_bytes(2, 8, 64, 1, 16) == 0
    long = dict(B=1, N=4096)
    assert scan_fwd(**long, ws=None) == ERR_WORKSPACE and scan_fwd(**long, wsb=need - 1) == ERR_WORKSPACE
    assert scan_fwd(**long, ws=at(12) + 4) == ERR_WORKSPACE
    assert _block.scan_workspace_bytes(-1, 8, 64, 1, 16) == 0 and _block.scan_bwd_workspace_bytes(2, 8, 64, 3, 16) == 0


def test_binding_refuses_host_tensors():
    import retnet_retention_fwd_amd as R
    x = torch.zeros(2, 3, 8)
    for f in (lambda: R.layer_norm_fwd(x), lambda: R.causal_conv_fwd(x, torch.zeros(8, 4)),
              lambda: R.selective_scan_fwd(x, x, torch.zeros(8, 4), x, x), lambda: R.rotary_fwd(x[None], None, x)):
        with pytest.raises(ValueError, match="GPU tensor"):
            f()


def test_row_strides():
    """What _rows takes and gives, on tensors that only claim to be on the GPU."""
    class Seen(torch.Tensor):
        is_cuda = True

    def seen(t):
        return t.as_subclass(Seen)

    wide = torch.zeros(3, 5, 24)
    assert _block._rows(seen(wide), "x", None, None, None) == 24
    assert _block._rows(seen(wide[..., 8:16]), "x", None, None, None) == 24
    assert _block._rows(seen(wide[:, :1, :8]), "x", None, None, None) == 120   # one token: batches are its rows
    assert _block._rows(seen(wide[0, :, :8]), "x", None, None, None) == 24
    bc = wide[..., 4:20].unflatten(-1, (2, 8))
    assert _block._rows(seen(bc), "B", None, None, (3, 5, 2, 8), inner=2) == 24
    for bad in (wide[..., ::2], wide.transpose(1, 2), wide[:, ::2].transpose(0, 1), wide[:, :3],
                torch.zeros(1, 5, 8).expand(3, 5, 8), torch.zeros(3, 1, 8).expand(3, 5, 8)):
        with pytest.raises(ValueError):
            _block._rows(seen(bad), "x", None, None, None)


def test_weight_types():
    class Seen(torch.Tensor):
        is_cuda = True

    x = torch.zeros(2, 8, dtype=torch.bfloat16).as_subclass(Seen)
    w = torch.zeros(8).as_subclass(Seen)
    assert _block._weights(w, w, x, (8,), 8) == F32 and _block._weights(None, None, x, (8,), 8) == F32
    assert _block._weights(w.bfloat16(), None, x, (8,), 8) == BF16
    with pytest.raises(TypeError):
        _block._weights(w.half(), None, x, (8,), 8)
    with pytest.raises(TypeError):
        _block._weights(w, w.bfloat16(), x, (8,), 8)
    with pytest.raises(ValueError):
        _block._weights(w[:4], None, x, (8,), 8)


def test_frequency_arguments():
    f = _block.rotary_frequencies
    for bad in (dict(rot=7), dict(rot=0), dict(rot=8, base=1.0), dict(rot=8, factor=0.5), dict(rot=2, scaling="base"),
                dict(rot=8, scaling="ramp"), dict(rot=8, scaling="ramp", original_length=10, fast=1, slow=2),
                dict(rot=8, scaling="other")):
        with pytest.raises(ValueError):
            f(**bad)
