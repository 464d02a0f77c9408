"""ctypes binding of a block's projections: the matrix product with bias, activation and residual
in its epilogue, the gated feed-forward block, and the norms of queries and keys for each head
with rotary positions in the same pass (the last part of include/retention.h).

Argument marshalling only, as in _block.py.  x is [..., K] with adjacent elements; a column slice
of a wider projection is taken in place.  Weights are [out, in], of x's type.  Work runs on the
tensors' device, on its current stream or on `stream`.
"""
from __future__ import annotations

import functools

from ._block import _binder, _code, _dense, _f, _given, _heads, _i, _ll, _on, _positions, _ptr, _space, _sz, _torch, _vp, _weights
from ._lib import RETN_BF16, RETN_F32, _check, _require

#: Argument types of the entry points, by name; the result is a status unless named below.
SIGNATURES = {
    "linear_fwd": [_vp, _ll] + [_vp] * 5 + [_ll] + [_i] * 5 + [_vp, _sz, _vp],
    "linear_workspace_bytes": [_ll] + [_i] * 4,
    "linear_bwd": [_vp, _ll] + [_vp] * 6 + [_ll] + [_i] * 5 + [_vp, _sz, _vp],
    "linear_bwd_workspace_bytes": [_ll] + [_i] * 5,
    "gated_ffn_fwd": [_vp, _ll] + [_vp] * 7 + [_ll] + [_i] * 4 + [_vp, _sz, _vp],
    "gated_ffn_workspace_bytes": [_ll] + [_i] * 4,
    "gated_ffn_bwd": [_vp, _ll] + [_vp] * 10 + [_ll] + [_i] * 4 + [_vp, _sz, _vp],
    "gated_ffn_bwd_workspace_bytes": [_ll] + [_i] * 4,
    "head_norm_rotary_fwd": [_vp] * 8 + [_ll, _vp, _i, _ll] + [_i] * 7 + [_f] * 3 + [_i, _i, _vp],
    "head_norm_rotary_bwd": [_vp] * 12 + [_ll, _vp, _i, _ll] + [_i] * 7 + [_f] * 3 + [_i, _i, _vp, _sz, _vp],
    "head_norm_rotary_bwd_workspace_bytes": [_i],
}

#: Activations by name: z, max(z, 0), z times the normal distribution function, its tanh form,
#: z sigmoid(z).
ACTIVATIONS = {"none": 0, "relu": 1, "gelu": 2, "gelu_tanh": 3, "silu": 4}

_Strides12, _Strides18 = _ll * 12, _ll * 18
_fn = _binder(SIGNATURES)


def _activation(name):
    try:
        return ACTIVATIONS[name]
    except (KeyError, TypeError):
        raise ValueError(f"activation must be one of {sorted(ACTIVATIONS)}, got {name!r}") from None


def _x(x):
    """(rows, width, row stride, type code) of x [..., K]: rows lie one stride apart."""
    torch = _torch()
    if not isinstance(x, torch.Tensor):
        raise TypeError("x must be a torch.Tensor")
    if not x.is_cuda:
        raise ValueError("x must be a GPU tensor")
    if x.dim() < 1 or x.shape[-1] < 1:
        raise ValueError("x must be [..., K] with K >= 1")
    K = x.shape[-1]
    if x.is_contiguous():
        return x.numel() // K, K, K, _code(x)
    size, step = x.shape, x.stride()
    if step[-1] != 1 and K != 1:
        raise ValueError("x: the elements of a row must be contiguous")
    rows, ld = 1, None
    for n, s in zip(reversed(size[:-1]), reversed(step[:-1])):
        if n != 1:
            if ld is None:
                ld = s
            elif s != rows * ld:
                raise ValueError("x: rows must lie one stride apart")
        rows *= n
    if rows == 0 or ld is None:
        ld = K
    if ld < K:
        raise ValueError("x: rows overlap")
    return rows, K, ld, _code(x)


def _aligned(code, *widths_and_addresses):
    """Whether widths (in elements, the first three) and addresses are multiples of 16 bytes."""
    a, b, c, *addresses = widths_and_addresses
    if (a | b | c) & (7 if code == RETN_BF16 else 3):
        return 0
    bits = 0
    for p in addresses:
        bits |= p
    return 0 if bits & 15 else 1


@functools.lru_cache(maxsize=4096)
def _bytes(name, *sizes):
    """A workspace query, asked once for the same sizes."""
    return _fn(name)(*sizes)


def _matrix(w, name, x, shape=None):
    """A contiguous weight of x's type and device."""
    if shape is None:
        try:       # what holds as a rule
            if w.dtype is x.dtype and w.get_device() == x.get_device() and w.is_contiguous() and w.dim() == 2 and w.shape[0] > 0:
                return
        except AttributeError:
            pass
        _require(w, name, x.dtype, x.device)
        if w.dim() != 2 or w.shape[0] < 1:
            raise ValueError(f"{name} must be [out, in]")
        return
    _dense(w, name, x.dtype, x.device, shape)


def _dtype(dtype):
    torch = _torch()
    codes = {torch.float32: RETN_F32, torch.bfloat16: RETN_BF16}
    if dtype not in codes:
        raise TypeError(f"dtype must be float32 or bfloat16, got {dtype}")
    return codes[dtype]


# ------------------------------------------------------------------------------------ projection
def linear_workspace_bytes(rows, N, K, dtype, aligned=False) -> int:
    """Bytes of workspace linear_fwd needs for these sizes; `aligned`: pointers, row strides and
    widths are multiples of 16 bytes (False is always enough)."""
    return int(_fn("linear_workspace_bytes")(rows, N, K, _dtype(dtype), int(aligned)))


def linear_bwd_workspace_bytes(rows, N, K, dtype, activation="none", aligned=False) -> int:
    """Bytes of workspace linear_bwd needs for these sizes."""
    return int(_fn("linear_bwd_workspace_bytes")(rows, N, K, _activation(activation), _dtype(dtype), int(aligned)))


def linear_fwd(x, weight, bias=None, residual=None, activation="none", return_pre=False, out=None, workspace=None,
               stream=None):
    """act(x weight^T + bias) + residual for x [..., K] and weight [N, K]: one pass, the sums in
    fp32 and rounded once.  bias [N]: fp32 or x's type; residual [..., N].  Returns y [..., N], or
    (y, pre) with the sums before the activation, which linear_bwd takes.  `out` may be the
    residual itself."""
    torch = _torch()
    act = _activation(activation)
    rows, K, ld, code = _x(x)
    dev = x.device
    _matrix(weight, "weight", x)
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight must be [N, {K}], got {list(weight.shape)}")
    bcode = RETN_F32 if bias is None else _weights(None, bias, x, None, N)
    shape = x.shape[:-1] + (N,)
    _given(residual, "residual", x.dtype, dev, shape)
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, shape)
        y = x.new_empty(shape) if out is None else out
        pre = x.new_empty(shape) if return_pre else None
        px, pw = x.data_ptr(), weight.data_ptr()
        need = _bytes("linear_workspace_bytes", rows, N, K, code, _aligned(code, ld, K, N, px, pw))
        ws, nbytes = _space(need, workspace, dev)
        _check(_fn("linear_fwd")(px, ld, pw, _ptr(bias), _ptr(residual), y.data_ptr(), _ptr(pre), rows, N, K, act,
                                 code, bcode, _ptr(ws), nbytes, s), "linear_fwd")
    return (y, pre) if return_pre else y


def linear_bwd(x, weight, grad_y, pre=None, activation="none", bias_grad=True, x_grad=True, weight_grad=True,
               bias_dtype=None, workspace=None, stream=None):
    """Backward of linear_fwd: (grad_x, grad_weight, grad_bias), each None where it is not asked
    for.  `pre` is the forward's for an activation; grad_bias has bias_dtype (fp32 or x's type, by
    default x's).  The residual's gradient is grad_y."""
    torch = _torch()
    act = _activation(activation)
    rows, K, ld, code = _x(x)
    dev = x.device
    _matrix(weight, "weight", x)
    N = weight.shape[0]
    if weight.shape[1] != K:
        raise ValueError(f"weight must be [N, {K}], got {list(weight.shape)}")
    shape = x.shape[:-1] + (N,)
    _dense(grad_y, "grad_y", x.dtype, dev, shape)
    if act and pre is None:
        raise ValueError("an activation's backward needs pre, the forward's")
    if act:
        _dense(pre, "pre", x.dtype, dev, shape)
    bdtype = x.dtype if bias_dtype is None else bias_dtype
    if bdtype not in (torch.float32, x.dtype):
        raise TypeError(f"bias_dtype must be float32 or {x.dtype}, got {bdtype}")
    on, s = _on(dev, stream)
    with on:
        gx = x.new_empty(x.shape) if x_grad else None
        gw = torch.empty_like(weight) if weight_grad else None
        px, pw = x.data_ptr(), weight.data_ptr()
        gb = torch.empty(N, dtype=bdtype, device=dev) if bias_grad else None
        need = _bytes("linear_bwd_workspace_bytes", rows, N, K, act, code, _aligned(code, ld, K, N, px, pw, grad_y.data_ptr()))
        ws, nbytes = _space(need, workspace, dev)
        _check(_fn("linear_bwd")(px, ld, pw, _ptr(pre) if act else None, _ptr(grad_y), _ptr(gx), _ptr(gw),
                                 _ptr(gb), rows, N, K, act, code, RETN_F32 if bdtype is torch.float32 else RETN_BF16,
                                 _ptr(ws), nbytes, s), "linear_bwd")
    return gx, gw, gb


# ------------------------------------------------------------------------ gated feed-forward block
def gated_ffn_workspace_bytes(rows, D, F, dtype, aligned=False) -> int:
    """Bytes of workspace gated_ffn_fwd needs for these sizes (aligned: as linear_workspace_bytes)."""
    return int(_fn("gated_ffn_workspace_bytes")(rows, D, F, _dtype(dtype), int(aligned)))


def gated_ffn_bwd_workspace_bytes(rows, D, F, dtype, aligned=False) -> int:
    """Bytes of workspace gated_ffn_bwd needs for these sizes."""
    return int(_fn("gated_ffn_bwd_workspace_bytes")(rows, D, F, _dtype(dtype), int(aligned)))


def _ffn_weights(x, K, w_gate, w_up, w_down):
    _matrix(w_gate, "w_gate", x)
    F = w_gate.shape[0]
    _matrix(w_gate, "w_gate", x, (F, K))
    _matrix(w_up, "w_up", x, (F, K))
    _matrix(w_down, "w_down", x, (K, F))
    return F


def gated_ffn_fwd(x, w_gate, w_up, w_down, residual=None, activation="silu", return_pre=False, out=None, workspace=None,
                  stream=None):
    """Gated feed-forward block (act(x w_gate^T) * (x w_up^T)) w_down^T + residual for x [..., D],
    w_gate and w_up [F, D], w_down [D, F], residual [..., D].  Returns y [..., D], or (y, gate, up)
    with both projections [..., F], which gated_ffn_bwd takes.  `out` may be the residual itself."""
    torch = _torch()
    act = _activation(activation)
    rows, D, ld, code = _x(x)
    dev = x.device
    F = _ffn_weights(x, D, w_gate, w_up, w_down)
    _given(residual, "residual", x.dtype, dev, x.shape)
    on, s = _on(dev, stream)
    with on:
        _given(out, "out", x.dtype, dev, x.shape)
        y = x.new_empty(x.shape) if out is None else out
        gate = up = None
        if return_pre:
            gate, up = x.new_empty(x.shape[:-1] + (F,)), x.new_empty(x.shape[:-1] + (F,))
        px = x.data_ptr()
        addresses = px, w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr()
        need = _bytes("gated_ffn_workspace_bytes", rows, D, F, code, _aligned(code, ld, D, F, *addresses))
        ws, nbytes = _space(need, workspace, dev)
        _check(_fn("gated_ffn_fwd")(px, ld, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(residual), _ptr(y), _ptr(gate),
                                    _ptr(up), rows, D, F, act, code, _ptr(ws), nbytes, s), "gated_ffn_fwd")
    return (y, gate, up) if return_pre else y


def gated_ffn_bwd(x, w_gate, w_up, w_down, gate, up, grad_y, activation="silu", x_grad=True, weight_grad=True,
                  workspace=None, stream=None):
    """Backward of gated_ffn_fwd: (grad_x, grad_w_gate, grad_w_up, grad_w_down), None where not
    asked for.  gate and up are the forward's; the residual's gradient is grad_y."""
    torch = _torch()
    act = _activation(activation)
    rows, D, ld, code = _x(x)
    dev = x.device
    F = _ffn_weights(x, D, w_gate, w_up, w_down)
    _dense(gate, "gate", x.dtype, dev, x.shape[:-1] + (F,))
    _dense(up, "up", x.dtype, dev, x.shape[:-1] + (F,))
    _dense(grad_y, "grad_y", x.dtype, dev, x.shape)
    on, s = _on(dev, stream)
    with on:
        gx = x.new_empty(x.shape) if x_grad else None
        px = x.data_ptr()
        gw = [torch.empty_like(w) if weight_grad else None for w in (w_gate, w_up, w_down)]
        addresses = px, w_gate.data_ptr(), w_up.data_ptr(), w_down.data_ptr(), grad_y.data_ptr()
        need = _bytes("gated_ffn_bwd_workspace_bytes", rows, D, F, code, _aligned(code, ld, D, F, *addresses))
        ws, nbytes = _space(need, workspace, dev)
        _check(_fn("gated_ffn_bwd")(px, ld, _ptr(w_gate), _ptr(w_up), _ptr(w_down), _ptr(gate), _ptr(up), _ptr(grad_y),
                                    _ptr(gx), *map(_ptr, gw), rows, D, F, act, code, _ptr(ws), nbytes, s), "gated_ffn_bwd")
    return (gx, *gw)


# ---------------------------------------------------------------------- head norms and positions
def _norm_weights(q_weight, k_weight, x, d):
    """Type code and type of the head norms' weights: fp32 or x's type, one for both."""
    torch = _torch()
    first = q_weight if q_weight is not None else k_weight
    if first is None:
        return RETN_F32, torch.float32
    if not isinstance(first, torch.Tensor):
        raise TypeError(f"{'k_weight' if q_weight is None else 'q_weight'} must be a torch.Tensor")
    if first.dtype not in (torch.float32, x.dtype):
        raise TypeError(f"q_weight and k_weight must be float32 or {x.dtype}, got {first.dtype}")
    _given(q_weight, "q_weight", first.dtype, x.device, (d,))
    _given(k_weight, "k_weight", first.dtype, x.device, (d,))
    return _code(first), first.dtype


def _sides(q, k, table, q_weight, k_weight, positions):
    """What both directions take: (device, sizes, strides of q and k, pointers and codes)."""
    torch = _torch()
    sq = _heads(q, "q", None, None, None)
    B, Hq, N, d = q.shape
    dev = q.device
    if not isinstance(table, torch.Tensor) or table.dim() != 3 or table.shape[2] != 2:
        raise ValueError("table must be [positions, rot/2, 2]")
    _dense(table, "table", torch.float32, dev, table.shape)
    sk, Hk = (0, 0, 0), 0
    if k is not None:
        sk = _heads(k, "k", q.dtype, dev, None)
        Hk = k.shape[1]
        if k.shape != (B, Hk, N, d):
            raise ValueError(f"k must be [{B}, Hk, {N}, {d}], got {list(k.shape)}")
    wcode, wt = _norm_weights(q_weight, k_weight, q, d)
    batched, pos = (0, None) if positions is None else _positions(positions, dev, B, N)
    return dev, (B, Hq, Hk, N, d), sq, sk, batched, pos, _code(q), wcode, wt


def _heads_out(out, like, name):
    """A contiguous [B,H,N,d] output, or the given one, and its strides."""
    B, H, N, d = like.shape
    if out is None:
        return like.new_empty((B, H, N, d)), (H * N * d, N * d, d)
    return out, _heads(out, name, like.dtype, like.device, like.shape)


def head_norm_rotary_fwd(q, k, table, q_weight=None, k_weight=None, eps=1e-6, positions=None, offset=0, interleaved=True,
                         q_scale=1.0, k_scale=1.0, out_q=None, out_k=None, stream=None):
    """Root-mean-square norm of each head's row of q [B,Hq,N,d] and k [B,Hk,N,d] (or None) over
    its d elements, times q_weight (k_weight) [d] (fp32 or q's type, None: ones), then rotary
    positions as rotary_fwd's, in one pass.  Strides, outputs, table, positions and scales are
    rotary_fwd's; out_q=q, out_k=k: in place.  Returns (q', k'), or q' alone without k."""
    dev, (B, Hq, Hk, N, d), sq, sk, batched, pos, code, wcode, _ = _sides(q, k, table, q_weight, k_weight, positions)
    on, s = _on(dev, stream)
    with on:
        out_q, soq = _heads_out(out_q, q, "out_q")
        sok = (0, 0, 0)
        if k is not None:
            out_k, sok = _heads_out(out_k, k, "out_k")
        _check(_fn("head_norm_rotary_fwd")(_ptr(q), _ptr(k), _ptr(out_q), None if k is None else _ptr(out_k),
                                           _Strides12(*sq, *soq, *sk, *sok), _ptr(q_weight), _ptr(k_weight), _ptr(table),
                                           table.shape[0], pos, batched, offset, B, Hq, Hk, N, d, 2 * table.shape[1],
                                           1 if interleaved else 0, eps, q_scale, k_scale, code, wcode, s),
               "head_norm_rotary_fwd")
    return out_q if k is None else (out_q, out_k)


def head_norm_rotary_bwd(q, k, table, grad_q, grad_k, q_weight=None, k_weight=None, eps=1e-6, positions=None, offset=0,
                         interleaved=True, q_scale=1.0, k_scale=1.0, weight_grad=True, out_q=None, out_k=None,
                         workspace=None, stream=None):
    """Backward of head_norm_rotary_fwd for the gradients grad_q and grad_k of its outputs:
    (gradient of q, of k, of q_weight, of k_weight), None where there is no such input or, for the
    weights, with weight_grad=False.  The other arguments are the forward's; out_q=grad_q,
    out_k=grad_k: in place."""
    torch = _torch()
    dev, (B, Hq, Hk, N, d), sq, sk, batched, pos, code, wcode, wt = _sides(q, k, table, q_weight, k_weight, positions)
    sgq = _heads(grad_q, "grad_q", q.dtype, dev, q.shape)
    sgk = (0, 0, 0) if k is None else _heads(grad_k, "grad_k", q.dtype, dev, k.shape)
    on, s = _on(dev, stream)
    with on:
        out_q, soq = _heads_out(out_q, q, "out_q")
        sok = (0, 0, 0)
        if k is not None:
            out_k, sok = _heads_out(out_k, k, "out_k")
        gqw = torch.empty(d, dtype=wt, device=dev) if q_weight is not None and weight_grad else None
        gkw = torch.empty(d, dtype=wt, device=dev) if k is not None and k_weight is not None and weight_grad else None
        need = 0 if gqw is None and gkw is None else _bytes("head_norm_rotary_bwd_workspace_bytes", d)
        ws, nbytes = _space(need, workspace, dev)
        k_in = (None, None, None) if k is None else (_ptr(k), _ptr(grad_k), _ptr(out_k))
        _check(_fn("head_norm_rotary_bwd")(_ptr(q), k_in[0], _ptr(grad_q), k_in[1], _ptr(out_q), k_in[2],
                                           _Strides18(*sq, *sgq, *soq, *sk, *sgk, *sok), _ptr(q_weight), _ptr(k_weight),
                                           _ptr(gqw), _ptr(gkw), _ptr(table), table.shape[0], pos, batched, offset, B, Hq,
                                           Hk, N, d, 2 * table.shape[1], 1 if interleaved else 0, eps, q_scale, k_scale,
                                           code, wcode, _ptr(ws), nbytes, s), "head_norm_rotary_bwd")
    return out_q, out_k if k is not None else None, gqw, gkw
