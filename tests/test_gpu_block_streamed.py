"""Gradients of the convolution and the scan of 8 MiB and more, which are stored past the caches, with
ragged lengths, at whole and at cut channel widths.  Bounds as in test_gpu_conv.py and
test_gpu_scan.py."""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

import test_gpu_conv as C  # noqa: E402
import test_gpu_scan as S  # noqa: E402
from block_cases import TYPES, check, draw  # noqa: E402

MIB8 = 8 << 20


def R():
    import retnet_retention_fwd_amd as R_
    return R_


@pytest.mark.parametrize("dtype,N,D", [("bf16", 701, 2048), ("bf16", 703, 2051), ("f32", 345, 2052), ("f32", 351, 2049)])
def test_convolution(dtype, N, D):
    print(f"\n[case] conv streamed {N} {D} {dtype}", flush=True)
    B, K = 3, 4
    assert B * N * D * TYPES[dtype].itemsize >= MIB8
    (x, w, b, s), (xr, wr, br, sr) = C.case(B, N, D, K, dtype, dtype, False, 70)
    g, gr = draw(80, (B, N, D), dtype)
    gs, gsr = draw(81, (B, K - 1, D), dtype)
    n = [N, N // 2 + 1, 2]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    got = R().causal_conv_bwd(x, w, g, b, silu=True, state_in=s, grad_state_out=gs, lengths=lengths,
                              return_grad_state_in=True)
    args = (xr, wr, gr, br)
    ref = O.causal_conv_bwd(*args, True, sr, gsr, n)
    flat = O.causal_conv_bwd(*args, False, sr, gsr, n, magnitude=True)      # silu' is 1.1 at most
    k = 160 + 8 * C.pre_mag(xr, wr, br, sr).max()
    for v, r, m, nm in zip(got, ref, flat, ("grad_x", "grad_weight", "grad_bias", "grad_state_in")):
        check(v, r, 1.1 * m, k, nm)


@pytest.mark.parametrize("dtype,N,D", [("bf16", 172, 8192), ("bf16", 175, 8191), ("f32", 171, 4100), ("f32", 173, 4099)])
def test_scan(dtype, N, D):
    print(f"\n[case] scan streamed {N} {D} {dtype}", flush=True)
    B, G, St = 3, 1, 4
    assert B * N * D * TYPES[dtype].itemsize >= MIB8
    t, v = S.case(B, N, D, G, St, dtype, False, 800)
    g, gr = draw(820, (B, N, D), dtype)
    gs, gsr = draw(821, (B, D, St), "f32")
    n = [N, N // 2 + 1, 17]
    lengths = torch.tensor(n, dtype=torch.int32, device="cuda")
    got = R().selective_scan_bwd(*S.fwd_args(t), g, D=t["D"], z=t["z"], dt_bias=t["dt_bias"], softplus=True,
                                 state_in=t["state_in"], grad_state_out=gs, lengths=lengths, return_grad_state_in=True)
    args = (*S.fwd_args(v), gr, v["D"], v["z"], v["dt_bias"], True, v["state_in"], gsr, n)
    # sums over channels: of 8192 of them at most, 64 a workgroup as there and 128 workgroups in a row
    k = 20 * N + 8 * St + 256 + 128
    names = ("grad_x", "grad_dt", "grad_A", "grad_B", "grad_C", "grad_D", "grad_z", "grad_dt_bias", "grad_state_in")
    for a, r, m, nm in zip(got, O.selective_scan_bwd(*args), O.selective_scan_bwd(*args, magnitude=True), names):
        check(a, r, m, k, nm)
