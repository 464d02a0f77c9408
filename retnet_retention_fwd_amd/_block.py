"""ctypes binding of the operators that stand around the retention in a block: layer
normalisation, rotary positions, the short causal convolution and the selective scan (the
second half of include/retention.h).

Argument marshalling only, as in _lib.py: torch provides device memory and the stream.
Activations are [B, N, D] with adjacent channels; a column slice of a wider projection is
taken in place (its rows are one stride apart over the whole batch).  Work runs on the
tensors' device, on its current stream or on `stream`.
"""
from __future__ import annotations

import contextlib
import ctypes
import math

from ._lib import RETN_BF16, RETN_F32, _check, _dtype_code, _require, lib

_vp, _i, _ll, _f, _sz = ctypes.c_void_p, ctypes.c_int, ctypes.c_longlong, ctypes.c_float, ctypes.c_size_t

#: Argument types of the entry points, by name; the result is a status unless named below.
SIGNATURES = {
    "layer_norm_fwd": [_vp] * 6 + [_ll, _i, _f, _i, _i, _vp],
    "layer_norm_bwd": [_vp] * 8 + [_ll, _i, _i, _i, _vp, _sz, _vp],
    "layer_norm_bwd_workspace_bytes": [_ll, _i, _i],
    "rotary_table": [_vp, _vp, _i, _ll, _ll, _f, _vp],
    "rotary_fwd": [_vp] * 6 + [_ll, _vp, _i, _ll] + [_i] * 7 + [_f, _f, _i, _vp],
    "rotary_bwd": [_vp] * 6 + [_ll, _vp, _i, _ll] + [_i] * 7 + [_f, _f, _i, _vp],
    "causal_conv_fwd": [_vp, _ll] + [_vp] * 6 + [_i] * 7 + [_vp],
    "causal_conv_fwd_padded": [_vp, _ll] + [_vp] * 6 + [_i] * 7 + [_vp],
    "causal_conv_bwd": [_vp, _ll] + [_vp] * 10 + [_i] * 7 + [_vp, _sz, _vp],
    "causal_conv_bwd_workspace_bytes": [_i] * 5,
    "causal_conv_step": [_vp, _ll] + [_vp] * 4 + [_i] * 6 + [_vp],
    "selective_scan_fwd": [_vp] * 12 + [_ll] * 5 + [_i] * 7 + [_vp, _sz, _vp],
    "selective_scan_fwd_padded": [_vp] * 12 + [_ll] * 5 + [_i] * 7 + [_vp, _sz, _vp],
    "selective_scan_workspace_bytes": [_i] * 5,
    "selective_scan_bwd": [_vp] * 21 + [_ll] * 5 + [_i] * 7 + [_vp, _sz, _vp],
    "selective_scan_bwd_workspace_bytes": [_i] * 5,
    "selective_scan_step": [_vp] * 10 + [_ll] * 5 + [_i] * 6 + [_vp],
}

_Strides = _ll * 12
_HERE = contextlib.nullcontext()
_T = None


def _torch():
    """torch, imported by the first call (importing the package does not)."""
    global _T
    if _T is None:
        import torch
        _T = torch
    return _T


def _binder(signatures):
    """The library's functions with these argument types, each looked up once."""
    bound = {}

    def fn(name):
        f = bound.get(name)
        if f is None:
            f = getattr(lib(), name)
            f.argtypes = signatures[name]
            f.restype = _sz if name.endswith("_bytes") else _i
            bound[name] = f
        return f
    return fn


_fn = _binder(SIGNATURES)


def _ptr(t):
    return None if t is None else t.data_ptr()


def _on(dev, stream):
    """A context in which the tensors' device is current and allocations belong to the stream
    that the kernels run on, and that stream's handle.  The current stream of the current
    device needs no context."""
    torch = _torch()
    if stream is None and torch.cuda.current_device() == dev.index:
        return _HERE, torch._C._cuda_getCurrentRawStream(dev.index)
    stack = contextlib.ExitStack()
    if torch.cuda.current_device() != dev.index:
        stack.enter_context(torch.cuda.device(dev))
    if stream is None:
        return stack, torch._C._cuda_getCurrentRawStream(dev.index)
    if stream.device != dev:
        stack.close()
        raise ValueError(f"stream is on {stream.device}, the tensors on {dev}")
    stack.enter_context(torch.cuda.stream(stream))
    return stack, stream.cuda_stream


def _code(t):
    """Type code of the activations."""
    torch = _torch()
    return RETN_BF16 if t.dtype is torch.bfloat16 else RETN_F32 if t.dtype is torch.float32 else _dtype_code(t)


def _shape(t, name, shape):
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must be {list(shape)}, got {list(t.shape)}")


def _dense(t, name, dtype, dev, shape):
    """A contiguous tensor of this type, device and shape."""
    try:       # what holds as a rule, at the price of four attributes
        if t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous():
            return
    except AttributeError:
        pass
    _require(t, name, dtype, dev)
    _shape(t, name, shape)


def _given(t, name, dtype, dev, shape):
    """An optional contiguous tensor of this type and shape."""
    if t is not None:
        _dense(t, name, dtype, dev, shape)


def _rows(t, name, dtype, dev, shape, inner=1):
    """A [B, N, ...] (or [B, ...]) tensor whose tokens lie one stride apart; its `inner` last
    axes are contiguous.  Returns that stride."""
    try:       # contiguous, as a rule
        if dev is None:
            if inner == 1 and dtype is None and shape is None and t.is_contiguous() and t.get_device() >= 0 and t.dim() > 1:
                return t.shape[-1]
        elif t.dtype is dtype and t.shape == shape and t.get_device() == dev.index and t.is_contiguous():
            return shape[-1] if inner == 1 else shape[-1] * shape[-2]
    except AttributeError:
        pass
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be a GPU tensor")
    if dev is not None and t.device != dev:
        raise ValueError(f"{name} is on {t.device}, expected {dev}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    size, step = t.shape, t.stride()
    if shape is not None and size != shape:
        _shape(t, name, shape)
    if len(size) <= inner:
        raise ValueError(f"{name} must be [B,N,...] or [B,...], got {list(size)}")
    width = 1
    for i in range(1, inner + 1):
        if step[-i] != width and size[-i] != 1:
            raise ValueError(f"{name}: the elements of a token must be contiguous")
        width *= size[-i]
    if len(size) - inner == 1:
        ld = step[0] if size[0] > 1 else width
    else:
        B, N = size[0], size[1]
        ld = step[1] if N > 1 else step[0] if B > 1 else width
        if B > 1 and N > 1 and step[0] != N * ld:
            raise ValueError(f"{name}: tokens must lie one stride apart over the whole batch")
    if ld < width:
        if t.numel() > 0:
            raise ValueError(f"{name}: tokens overlap")
        return width
    return ld


def _weights(w, b, x, w_shape, D):
    """Type code of weight and bias: fp32 or x's type, one for both."""
    torch = _torch()
    first = w if w is not None else b
    if first is None:
        return RETN_F32
    if not isinstance(first, torch.Tensor):
        raise TypeError(f"{'bias' if w is None else 'weight'} must be a torch.Tensor")
    if first.dtype not in (torch.float32, x.dtype):
        raise TypeError(f"weight and bias must be float32 or {x.dtype}, got {first.dtype}")
    _given(w, "weight", first.dtype, x.device, w_shape)
    _given(b, "bias", first.dtype, x.device, (D,))
    return _code(first)


def _space(need, workspace, dev):
    """The caller's workspace or a new one; its size."""
    torch = _torch()
    if workspace is None:
        if need == 0:
            return None, 0
        workspace = torch.empty(need, dtype=torch.uint8, device=dev)
    else:
        _require(workspace, "workspace", None, dev)
    return workspace, workspace.numel() * workspace.element_size()


def _lengths(lengths, dev, B):
    _given(lengths, "lengths", _torch().int32, dev, (B,))


# ------------------------------------------------------------------------------------ layer norm
def layer_norm_fwd(x, weight=None, bias=None, eps=1e-5, return_stats=False, out=None, stream=None):
    """Layer normalisation over the last axis of x [..., D] (bf16 or fp32): (x - mean) * rstd *
    weight + bias.  weight, bias [D]: fp32 or x's type.  Returns y, or (y, mean, rstd) with the
    fp32 statistics [...] that layer_norm_bwd takes."""
    torch = _torch()
    _require(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D] with D >= 1")
    D, dev = x.shape[-1], x.device
    rows = x.numel() // D
    wcode = _weights(weight, bias, x, (D,), D)
    code = _code(x)
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, x.shape)
        y = torch.empty_like(x) if out is None else out
        mean = rstd = None
        if return_stats:
            mean, rstd = torch.empty((2,) + x.shape[:-1], dtype=torch.float32, device=dev)
        _check(_fn("layer_norm_fwd")(_ptr(x), _ptr(weight), _ptr(bias), _ptr(y), _ptr(mean), _ptr(rstd), rows, D,
                                     float(eps), code, wcode, s), "layer_norm_fwd")
    return (y, mean, rstd) if return_stats else y


def layer_norm_bwd(x, weight, mean, rstd, grad_y, bias_grad=True, weight_grad=True, workspace=None, stream=None):
    """Backward of layer_norm_fwd: (grad_x, grad_weight, grad_bias); grad_weight is None without
    a weight or with weight_grad=False, grad_bias (of weight's type, or fp32) with bias_grad=False."""
    torch = _torch()
    _require(x, "x")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., D] with D >= 1")
    D, dev = x.shape[-1], x.device
    rows = x.numel() // D
    _dense(grad_y, "grad_y", x.dtype, dev, x.shape)
    _dense(mean, "mean", torch.float32, dev, x.shape[:-1])
    _dense(rstd, "rstd", torch.float32, dev, x.shape[:-1])
    wcode = _weights(weight, None, x, (D,), D)
    wt = torch.float32 if weight is None else weight.dtype
    code = _code(x)
    on, s = _on(dev, stream)
    with on:
        gx = torch.empty_like(x)
        gw = torch.empty(D, dtype=wt, device=dev) if weight is not None and weight_grad else None
        gb = torch.empty(D, dtype=wt, device=dev) if bias_grad else None
        need = 0 if gw is None and gb is None else _fn("layer_norm_bwd_workspace_bytes")(rows, D, code)
        ws, nbytes = _space(need, workspace, dev)
        _check(_fn("layer_norm_bwd")(_ptr(x), _ptr(weight), _ptr(mean), _ptr(rstd), _ptr(grad_y), _ptr(gx), _ptr(gw),
                                     _ptr(gb), rows, D, code, wcode, _ptr(ws), nbytes, s), "layer_norm_bwd")
    return gx, gw, gb


# ---------------------------------------------------------------------------------------- rotary
def rotary_frequencies(rot, base=10000.0, scaling="none", factor=1.0, original_length=None, fast=32.0, slow=1.0):
    """Angular frequencies [rot/2] (fp64, host) of the rotary schedule base^(-2i/rot), scaled for
    contexts `factor` times the length that a model was trained on:

    "none"    the plain schedule
    "linear"  every frequency divided by factor (positions interpolated)
    "base"    the base multiplied by factor^(rot/(rot-2)): the slowest pair is interpolated by
              factor, the fastest is left alone
    "ramp"    pairs that turn more than `fast` times over original_length are left alone, those
              that turn less than `slow` times are divided by factor, the others blended
              linearly in their number of turns
    """
    torch = _torch()
    if rot < 2 or rot % 2:
        raise ValueError("rot must be even and at least 2")
    if not base > 1 or not factor >= 1:
        raise ValueError("base must be above 1 and factor at least 1")
    if scaling == "base":
        if rot < 4:
            raise ValueError('"base" scaling needs rot >= 4')
        base = base * factor ** (rot / (rot - 2))
    i = torch.arange(0, rot, 2, dtype=torch.float64)
    freq = torch.exp(-math.log(base) * i / rot)
    if scaling == "linear":
        freq = freq / factor
    elif scaling == "ramp":
        if original_length is None or not fast > slow:
            raise ValueError('"ramp" scaling needs original_length, and fast above slow')
        turns = original_length * freq / (2 * math.pi)
        keep = ((turns - slow) / (fast - slow)).clamp(0, 1)
        freq = freq * (keep + (1 - keep) / factor)
    elif scaling not in ("none", "base"):
        raise ValueError(f"unknown scaling {scaling!r}")
    return freq


def _table_device(at, device):
    """The GPU of a table of frequencies at `at`: the one asked for, theirs, or the current one."""
    torch = _torch()
    dev = torch.device("cuda" if device is None else device)
    if dev.type != "cuda":
        raise ValueError(f"device must be a GPU, got {dev}")
    if at.type == "cuda":
        if dev.index not in (None, at.index):
            raise ValueError(f"device is {dev}, freq is on {at}")
        return at
    return dev if dev.index is not None else torch.device("cuda", torch.cuda.current_device())


def rotary_table(freq, count, first=0, magnitude=1.0, device=None, stream=None):
    """Table [count, rot/2, 2] fp32 of magnitude * (cos, sin) for positions first ..
    first + count - 1 and the angular frequencies freq [rot/2] (rotary_frequencies)."""
    torch = _torch()
    if not isinstance(freq, torch.Tensor) or freq.dim() != 1 or freq.dtype != torch.float64:
        raise TypeError("freq must be a float64 tensor [rot/2]")
    dev = _table_device(freq.device, device)
    on, s = _on(dev, stream)
    with on:
        f = freq.to(dev).contiguous()
        table = torch.empty((count, f.numel(), 2), dtype=torch.float32, device=dev)
        _check(_fn("rotary_table")(_ptr(table), _ptr(f), f.numel(), int(first), int(count), float(magnitude), s),
               "rotary_table")
    return table


def _heads(t, name, dtype, dev, shape):
    """Strides of a [B,H,N,d] tensor with adjacent head elements."""
    torch = _torch()
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch.Tensor")
    if t.get_device() < 0:
        raise ValueError(f"{name} must be a GPU tensor")
    if t.dim() != 4:
        raise ValueError(f"{name} must be [B,H,N,d]")
    if dtype is not None and (t.dtype is not dtype or t.get_device() != dev.index):
        raise TypeError(f"{name} must be {dtype} on {dev}, got {t.dtype} on {t.device}")
    if shape is not None and t.shape != shape:
        _shape(t, name, shape)
    step = t.stride()
    if step[3] != 1 and t.shape[3] != 1:
        raise ValueError(f"{name}: the elements of a head must be contiguous")
    return step[:3]


def _positions(positions, dev, B, N):
    """Whether they are one row a sequence, and their address."""
    torch = _torch()
    if not isinstance(positions, torch.Tensor):
        raise TypeError("positions must be a torch.Tensor")
    batched = int(positions.dim() == 2)
    _dense(positions, "positions", torch.int64, dev, (B, N) if batched else (N,))
    return batched, positions.data_ptr()


def _rotary(fn, q, k, table, positions, offset, interleaved, q_scale, k_scale, out_q, out_k, stream):
    torch = _torch()
    sq = _heads(q, "q", None, None, None)
    B, Hq, N, d = q.shape
    dev, t, code = q.device, q.dtype, _code(q)
    if not isinstance(table, torch.Tensor) or table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be [positions, rot/2, 2]")
    far, half, _ = table.shape
    _dense(table, "table", torch.float32, dev, (far, half, 2))
    sk = sok = (0, 0, 0)
    Hk = pk = pok = 0
    if k is not None:
        sk = _heads(k, "k", t, dev, None)
        Hk, pk = k.shape[1], k.data_ptr()
        if k.shape != (B, Hk, N, d):
            raise ValueError(f"k must be [{B}, Hk, {N}, {d}], got {list(k.shape)}")
    batched, pp = (0, None) if positions is None else _positions(positions, dev, B, N)
    on, s = _on(dev, stream)
    with on:
        if out_q is None:
            out_q = q.new_empty((B, Hq, N, d))
            soq = (Hq * N * d, N * d, d)
        else:
            soq = _heads(out_q, "out_q", t, dev, q.shape)
        if k is not None:
            if out_k is None:
                out_k = k.new_empty((B, Hk, N, d))
                sok = (Hk * N * d, N * d, d)
            else:
                sok = _heads(out_k, "out_k", t, dev, k.shape)
            pok = out_k.data_ptr()
        _check(_fn(fn)(q.data_ptr(), pk, out_q.data_ptr(), pok, _Strides(*sq, *soq, *sk, *sok), table.data_ptr(), far, pp,
                       batched, offset, B, Hq, Hk, N, d, 2 * half, 1 if interleaved else 0, q_scale, k_scale, code, s), fn)
    return out_q if k is None else (out_q, out_k)


def rotary_fwd(q, k, table, positions=None, offset=0, interleaved=True, q_scale=1.0, k_scale=1.0, out_q=None,
               out_k=None, stream=None):
    """Rotary positions of q [B,Hq,N,d] and k [B,Hk,N,d] (or None): the first rot = 2 *
    table.shape[1] elements of each head turn by the table's row of their token's position, the
    rest pass, all are scaled.  Any strides with adjacent head elements; outputs are [B,H,N,d]
    contiguous unless given (out_q=q, out_k=k: in place).  positions: int64 [N] or [B,N], or
    None for offset + n.  Returns (q', k'), or q' alone without k."""
    return _rotary("rotary_fwd", q, k, table, positions, offset, interleaved, q_scale, k_scale, out_q, out_k, stream)


def rotary_bwd(grad_q, grad_k, table, positions=None, offset=0, interleaved=True, q_scale=1.0, k_scale=1.0,
               out_q=None, out_k=None, stream=None):
    """Backward of rotary_fwd (the transposed rotation, the same scales): gradients of q and k."""
    return _rotary("rotary_bwd", grad_q, grad_k, table, positions, offset, interleaved, q_scale, k_scale, out_q,
                   out_k, stream)


# ------------------------------------------------------------------------------- causal convolution
def _conv_shapes(x, weight, bias, dims):
    ldx = _rows(x, "x", None, None, None)
    if x.dim() != dims:
        raise ValueError("x must be " + ("[B,N,D]" if dims == 3 else "[B,D]"))
    D = x.shape[-1]
    if weight is not None and not isinstance(weight, _torch().Tensor):
        raise TypeError("weight must be a torch.Tensor")
    if weight is None or weight.dim() != 2 or weight.shape[0] != D:
        raise ValueError(f"weight must be [{D}, K]")
    return ldx, D, weight.shape[1], _weights(weight, bias, x, weight.shape, D)


def causal_conv_fwd(x, weight, bias=None, silu=False, state_in=None, return_state=False, lengths=None, out=None,
                    state_out=None, stream=None):
    """Causal convolution of each channel of x [B,N,D] over its last K tokens with weight [D,K]
    (K 2, 3 or 4), plus bias [D], with an optional silu.  state_in / state_out [B,K-1,D]: the
    tokens in front of the first and the last K-1 tokens.  lengths [B] int32: tokens of each
    sequence of a padded batch; the rows of y behind them are zero, or, in a given `out`, left as
    they were.  Returns y, or (y, state_out)."""
    torch = _torch()
    ldx, D, K, wcode = _conv_shapes(x, weight, bias, 3)
    B, N, dev, code = x.shape[0], x.shape[1], x.device, _code(x)
    _given(state_in, "state_in", x.dtype, dev, (B, K - 1, D))
    _lengths(lengths, dev, B)
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, (B, N, D))
        _given(state_out, "state_out", x.dtype, dev, (B, K - 1, D))
        y = torch.empty((B, N, D), dtype=x.dtype, device=dev) if out is None else out
        if state_out is None and return_state:
            state_out = torch.empty((B, max(K - 1, 0), D), dtype=x.dtype, device=dev)
        fn = "causal_conv_fwd" if out is not None else "causal_conv_fwd_padded"     # fresh memory is written whole
        _check(_fn(fn)(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(y), _ptr(state_in), _ptr(state_out), _ptr(lengths),
                       B, N, D, K, int(bool(silu)), code, wcode, s), fn)
    return (y, state_out) if state_out is not None else y


def causal_conv_bwd(x, weight, grad_y, bias=None, silu=False, state_in=None, grad_state_out=None, lengths=None,
                    return_grad_state_in=False, workspace=None, stream=None):
    """Backward of causal_conv_fwd: (grad_x, grad_weight, grad_bias), plus grad_state_in when
    return_grad_state_in is set; grad_bias is None without a bias."""
    torch = _torch()
    ldx, D, K, wcode = _conv_shapes(x, weight, bias, 3)
    B, N, dev, code = x.shape[0], x.shape[1], x.device, _code(x)
    _dense(grad_y, "grad_y", x.dtype, dev, x.shape)
    _given(state_in, "state_in", x.dtype, dev, (B, K - 1, D))
    _given(grad_state_out, "grad_state_out", x.dtype, dev, (B, K - 1, D))
    _lengths(lengths, dev, B)
    on, s = _on(dev, stream)
    with on:
        gx = torch.empty((B, N, D), dtype=x.dtype, device=dev)
        gw = torch.empty((D, K), dtype=weight.dtype, device=dev)
        gb = torch.empty(D, dtype=weight.dtype, device=dev) if bias is not None else None
        gs = torch.empty((B, max(K - 1, 0), D), dtype=x.dtype, device=dev) if return_grad_state_in else None
        ws, nbytes = _space(_fn("causal_conv_bwd_workspace_bytes")(B, N, D, K, code), workspace, dev)
        _check(_fn("causal_conv_bwd")(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(state_in), _ptr(grad_y),
                                      _ptr(grad_state_out), _ptr(lengths), _ptr(gx), _ptr(gw), _ptr(gb), _ptr(gs), B, N,
                                      D, K, int(bool(silu)), code, wcode, _ptr(ws), nbytes, s), "causal_conv_bwd")
    return (gx, gw, gb, gs) if return_grad_state_in else (gx, gw, gb)


def causal_conv_step(x, weight, state, bias=None, silu=False, out=None, stream=None):
    """One token of causal_conv_fwd: y [B,D] from x [B,D] and the state [B,K-1,D], which moves
    up by one row in place."""
    torch = _torch()
    ldx, D, K, wcode = _conv_shapes(x, weight, bias, 2)
    B, dev, code = x.shape[0], x.device, _code(x)
    _dense(state, "state", x.dtype, dev, (B, K - 1, D))
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, (B, D))
        y = x.new_empty((B, D)) if out is None else out
        _check(_fn("causal_conv_step")(_ptr(x), ldx, _ptr(weight), _ptr(bias), _ptr(state), _ptr(y), B, D, K,
                                       int(bool(silu)), code, wcode, s), "causal_conv_step")
    return y


# --------------------------------------------------------------------------------- selective scan
def _scan_shapes(x, dt, A, Bm, Cm, D, z, dt_bias, step):
    """Checks the inputs that every form takes; (token strides, sizes, type code)."""
    torch = _torch()
    ldx = _rows(x, "x", None, None, None)
    if x.dim() != (2 if step else 3):
        raise ValueError("x must be " + ("[B,D]" if step else "[B,N,D]"))
    dev, t, shape = x.device, x.dtype, tuple(x.shape)
    lead, ch, code = shape[:-1], shape[-1], _code(x)
    lddt = _rows(dt, "dt", t, dev, shape)
    ldz = _rows(z, "z", t, dev, shape) if z is not None else 0
    if not isinstance(A, torch.Tensor) or A.dim() != 2 or A.shape[0] != ch:
        _require(A, "A", torch.float32, dev)
        raise ValueError(f"A must be [{ch}, S]")
    S = A.shape[1]
    _dense(A, "A", torch.float32, dev, (ch, S))
    if not isinstance(Bm, torch.Tensor) or Bm.dim() != len(lead) + 2:
        raise ValueError("Bm must be " + ("[B,G,S]" if step else "[B,N,G,S]"))
    G = Bm.shape[-2]
    ldb = _rows(Bm, "Bm", t, dev, lead + (G, S), inner=2)
    ldc = _rows(Cm, "Cm", t, dev, lead + (G, S), inner=2)
    _given(D, "D", torch.float32, dev, (ch,))
    _given(dt_bias, "dt_bias", torch.float32, dev, (ch,))
    return (ldx, lddt, ldz, ldb, ldc), G, S, code


def scan_workspace_bytes(B, N, D, G, S) -> int:
    """Bytes of workspace selective_scan_fwd needs for these sizes."""
    return int(_fn("selective_scan_workspace_bytes")(B, N, D, G, S))


def scan_bwd_workspace_bytes(B, N, D, G, S) -> int:
    """Bytes of workspace selective_scan_bwd needs for these sizes."""
    return int(_fn("selective_scan_bwd_workspace_bytes")(B, N, D, G, S))


def selective_scan_fwd(x, dt, A, Bm, Cm, D=None, z=None, dt_bias=None, softplus=False, state_in=None,
                       return_state=False, lengths=None, out=None, state_out=None, workspace=None, stream=None):
    """Selective state-space scan: h_t = exp(dt_t A) h_(t-1) + dt_t x_t B_t, y_t = (C_t . h_t + D x_t)
    silu(z_t), with dt_t = dt + dt_bias or its softplus.

    x, dt, z [B,N,D] and Bm, Cm [B,N,G,S] (bf16 or fp32, token strides allowed); A [D,S], D and
    dt_bias [D], state_in and state_out [B,D,S] fp32 (state_out may be state_in); lengths [B] int32:
    tokens of each sequence of a padded batch; the rows of y behind them are zero, or, in a given
    `out`, left as they were.  Returns y [B,N,D], or (y, state_out)."""
    torch = _torch()
    ld, G, S, code = _scan_shapes(x, dt, A, Bm, Cm, D, z, dt_bias, False)
    (B, N, ch), dev = x.shape, x.device
    _given(state_in, "state_in", torch.float32, dev, (B, ch, S))
    _lengths(lengths, dev, B)
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, (B, N, ch))
        _given(state_out, "state_out", torch.float32, dev, (B, ch, S))
        y = torch.empty((B, N, ch), dtype=x.dtype, device=dev) if out is None else out
        if state_out is None and return_state:
            state_out = torch.empty((B, ch, S), dtype=torch.float32, device=dev)
        ws, nbytes = _space(scan_workspace_bytes(B, N, ch, G, S), workspace, dev)
        fn = "selective_scan_fwd" if out is not None else "selective_scan_fwd_padded"     # fresh memory is written whole
        _check(_fn(fn)(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z), _ptr(dt_bias), _ptr(y),
                       _ptr(state_in), _ptr(state_out), _ptr(lengths), *ld, B, N, ch, G, S, int(bool(softplus)), code,
                       _ptr(ws), nbytes, s), fn)
    return (y, state_out) if state_out is not None else y


def selective_scan_bwd(x, dt, A, Bm, Cm, grad_y, D=None, z=None, dt_bias=None, softplus=False, state_in=None,
                       grad_state_out=None, lengths=None, return_grad_state_in=False, workspace=None, stream=None):
    """Backward of selective_scan_fwd: (grad_x, grad_dt, grad_A, grad_B, grad_C, grad_D, grad_z,
    grad_dt_bias), plus grad_state_in when return_grad_state_in is set.  Gradients of absent
    inputs are None; grad_dt is that of dt as it was passed."""
    torch = _torch()
    ld, G, S, code = _scan_shapes(x, dt, A, Bm, Cm, D, z, dt_bias, False)
    (B, N, ch), dev, t = x.shape, x.device, x.dtype
    _dense(grad_y, "grad_y", t, dev, x.shape)
    _given(state_in, "state_in", torch.float32, dev, (B, ch, S))
    _given(grad_state_out, "grad_state_out", torch.float32, dev, (B, ch, S))
    _lengths(lengths, dev, B)
    on, s = _on(dev, stream)
    with on:
        full = lambda: torch.empty((B, N, ch), dtype=t, device=dev)                         # noqa: E731
        f32 = lambda *shape: torch.empty(shape, dtype=torch.float32, device=dev)           # noqa: E731
        gx, gdt, gz = full(), full(), full() if z is not None else None
        gA, gB, gC = f32(ch, S), torch.empty((B, N, G, S), dtype=t, device=dev), torch.empty((B, N, G, S), dtype=t,
                                                                                             device=dev)
        gD, gbias = f32(ch) if D is not None else None, f32(ch) if dt_bias is not None else None
        gs = f32(B, ch, S) if return_grad_state_in else None
        ws, nbytes = _space(scan_bwd_workspace_bytes(B, N, ch, G, S), workspace, dev)
        _check(_fn("selective_scan_bwd")(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                         _ptr(dt_bias), _ptr(state_in), _ptr(grad_y), _ptr(grad_state_out),
                                         _ptr(lengths), _ptr(gx), _ptr(gdt), _ptr(gA), _ptr(gB), _ptr(gC), _ptr(gD),
                                         _ptr(gz), _ptr(gbias), _ptr(gs), *ld, B, N, ch, G, S, int(bool(softplus)), code,
                                         _ptr(ws), nbytes, s), "selective_scan_bwd")
    grads = (gx, gdt, gA, gB, gC, gD, gz, gbias)
    return grads + (gs,) if return_grad_state_in else grads


def selective_scan_step(x, dt, A, Bm, Cm, state, D=None, z=None, dt_bias=None, softplus=False, out=None, stream=None):
    """One token of selective_scan_fwd: y [B,D] from x, dt, z [B,D] and Bm, Cm [B,G,S]; the state
    [B,D,S] fp32 is updated in place."""
    torch = _torch()
    ld, G, S, code = _scan_shapes(x, dt, A, Bm, Cm, D, z, dt_bias, True)
    (B, ch), dev = x.shape, x.device
    _dense(state, "state", torch.float32, dev, (B, ch, S))
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, (B, ch))
        y = x.new_empty((B, ch)) if out is None else out
        _check(_fn("selective_scan_step")(_ptr(x), _ptr(dt), _ptr(A), _ptr(Bm), _ptr(Cm), _ptr(D), _ptr(z),
                                          _ptr(dt_bias), _ptr(state), _ptr(y), *ld, B, ch, G, S, int(bool(softplus)),
                                          code, s), "selective_scan_step")
    return y
