"""More refusals of the operators around the retention (no GPU: every call here fails validation
and returns before anything is enqueued)."""
import pytest

torch = pytest.importorskip("torch")

from retnet_retention_fwd_amd import _block  # noqa: E402
from test_block_abi import (BF16, ERR_ALIAS, ERR_DTYPE, ERR_NULL, ERR_SHAPE, ERR_UNSUPPORTED, ERR_WORKSPACE, F32, MB,  # noqa: E402
                            OK, SCAN_IN, SCAN_LD, at, call, rotary, scan_bwd)


def conv_padded(**kw):
    return call("causal_conv_fwd_padded", dict(x=at(0), ldx=64, w=at(1), b=at(2), y=at(3), si=at(4), so=at(5), n=at(6), B=2,
                                               N=8, D=64, K=4, silu=1, dt=BF16, wt=BF16, stream=None), **kw)


def scan_padded(**kw):
    return call("selective_scan_fwd_padded", dict(**SCAN_IN, y=at(8), si=at(9), so=at(10), n=at(11), **SCAN_LD, B=2, N=8,
                                                  ch=64, G=1, S=16, sp=1, dtype=BF16, ws=at(12), wsb=64 * MB, stream=None),
                **kw)


def test_padded_forms():
    """They check what the forms beside them check."""
    c, s = conv_padded, scan_padded
    assert c(dt=9) == ERR_DTYPE and c(dt=F32, wt=BF16) == ERR_DTYPE and s(dtype=9) == ERR_DTYPE
    assert c(B=-1) == ERR_SHAPE and c(ldx=63) == ERR_SHAPE and s(S=0) == ERR_SHAPE and s(ldb=15) == ERR_SHAPE
    assert c(K=5) == ERR_UNSUPPORTED and s(S=65, ldb=65, ldc=65) == ERR_UNSUPPORTED
    assert c(x=None) == ERR_NULL and c(y=None) == ERR_NULL and s(A=None) == ERR_NULL and s(y=None) == ERR_NULL
    assert c(y=at(0)) == ERR_ALIAS and c(y=at(6)) == ERR_ALIAS and s(y=at(6)) == ERR_ALIAS and s(so=at(11)) == ERR_ALIAS
    assert s(B=1, N=4096, ws=None) == ERR_WORKSPACE and s(B=1, N=4096, ws=at(12) + 4) == ERR_WORKSPACE
    assert c(B=0) == OK and c(N=0, so=None) == OK and s(B=0) == OK and s(N=0, so=None) == OK


def test_padded_forms_take_the_same_arguments():
    for n in ("causal_conv_fwd", "selective_scan_fwd"):
        assert _block.SIGNATURES[n] == _block.SIGNATURES[n + "_padded"]


@pytest.mark.parametrize("name", ["rotary_fwd", "rotary_bwd"])
def test_positions_need_a_table(name):
    """An unknown position turns its row into NaN, but a table without rows has no row to read."""
    assert rotary(name, length=0, pos=at(5)) == ERR_SHAPE
    assert rotary(name, length=0, pos=at(5), batched=1) == ERR_SHAPE
    assert rotary(name, length=0) == ERR_SHAPE
    assert rotary(name, length=0, pos=at(5), N=0) == OK


def test_launches_of_whole_workgroups():
    """Element counts whose last, partly idle workgroup would bring a launch to 2^32 threads."""
    table = lambda **kw: call("rotary_table", dict(t=at(0), f=1 << 39, pairs=2, first=0, n=10, m=1.0, s=None), **kw)  # noqa: E731
    assert table(n=(1 << 31) - 1) == ERR_UNSUPPORTED
    # 2 B N G S elements of the gradients of B and C, one a thread
    for f in (scan_padded, scan_bwd):
        assert f(B=1, N=(1 << 30) - 1, ch=2, G=1, S=2, ldx=2, lddt=2, ldz=2, ldb=2, ldc=2) == ERR_UNSUPPORTED
    assert _block.scan_bwd_workspace_bytes(1, (1 << 30) - 1, 2, 1, 2) == 0
    assert _block.scan_bwd_workspace_bytes(1, (1 << 30) - 64, 2, 1, 2) > 0


class Seen(torch.Tensor):
    """A tensor that only claims to be on the GPU."""
    is_cuda = True


def seen(*shape, dtype=None):
    return torch.zeros(*shape, dtype=dtype).as_subclass(Seen)


def test_arguments_of_the_wrong_kind_are_named():
    R = _block
    x, w = seen(2, 3, 8), seen(8, 4)
    for f in (lambda: R.causal_conv_fwd(seen(8), w), lambda: R.causal_conv_step(seen(8), w, seen(2, 3, 8)),
              lambda: R.selective_scan_fwd(seen(8), x, seen(8, 4), x, x),
              lambda: R.selective_scan_step(seen(8), x, seen(8, 4), x, seen(2, 8, 4), x)):
        with pytest.raises(ValueError, match="x must be"):
            f()
    for f in (lambda: R.layer_norm_fwd(seen(2, 8), [1.0] * 8), lambda: R.causal_conv_fwd(x, [[1.0] * 4] * 8)):
        with pytest.raises(TypeError, match="weight must be a torch.Tensor"):
            f()
    with pytest.raises(TypeError, match="bias must be a torch.Tensor"):
        R.layer_norm_fwd(seen(2, 8), None, 1.0)
    with pytest.raises(TypeError, match="positions must be a torch.Tensor"):
        R._positions([0, 1, 2], None, 1, 3)


def test_table_is_built_where_it_is_asked_for():
    freq = _block.rotary_frequencies(8)
    with pytest.raises(ValueError, match="device"):
        _block.rotary_table(freq, 4, device="cpu")
    with pytest.raises(ValueError, match="device"):
        _block._table_device(torch.device("cuda", 0), "cuda:1")
    assert _block._table_device(torch.device("cuda", 1), None) == torch.device("cuda", 1)
    assert _block._table_device(torch.device("cuda", 1), "cuda") == torch.device("cuda", 1)
    assert _block._table_device(torch.device("cpu"), "cuda:1") == torch.device("cuda", 1)
