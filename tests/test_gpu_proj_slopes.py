"""Gradients of the projection and the gated feed-forward block behind the activations that the parity
tests leave out, against the fp64 oracle (bounds: proj_cases)."""
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402
from proj_cases import ffn_bwd_bounds, linear_bwd_bounds  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


@pytest.mark.parametrize("act", ["gelu_tanh", "relu"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,N,K", [(1, 1, 1), (5, 130, 7), (33, 100, 72), (130, 129, 65), (300, 257, 200), (700, 384, 512), (2500, 65, 30)])
def test_linear(M, N, K, dtype, act):
    print(f"\n[case] slopes linear {M} {N} {K} {dtype} {act}", flush=True)
    (x, xr), (w, wr), (gy, gr) = draw(1, (M, K), dtype), draw(2, (N, K), dtype, K ** -0.5), draw(3, (M, N), dtype)
    z, zr = draw(4, (M, N), dtype, 1.5)
    got = R().linear_bwd(x, w, gy, pre=z, activation=act, bias_dtype=torch.float32)
    for g, v, m, what in zip(got, O.linear_bwd(xr, wr, gr, zr, act), linear_bwd_bounds(xr, wr, gr, zr, act, dtype),
                             ("grad_x", "grad_weight", "grad_bias")):
        check(g, v, m, 1, what)


@pytest.mark.parametrize("act", ["gelu_tanh", "none"])
@pytest.mark.parametrize("dtype", ["bf16", "f32"])
@pytest.mark.parametrize("M,D,F", [(1, 1, 1), (7, 256, 512), (50, 77, 129), (129, 96, 136), (300, 264, 392), (2500, 33, 70)])
def test_gated_ffn(M, D, F, dtype, act):
    print(f"\n[case] slopes ffn {M} {D} {F} {dtype} {act}", flush=True)
    shapes = [((M, D), 1.0), ((F, D), D ** -0.5), ((F, D), D ** -0.5), ((D, F), F ** -0.5), ((M, F), 1.5), ((M, F), 1.0), ((M, D), 1.0)]
    t, r = zip(*(draw(10 + i, s, dtype, c) for i, (s, c) in enumerate(shapes)))
    got = R().gated_ffn_bwd(*t, activation=act)
    for a, b, m, what in zip(got, O.gated_ffn_bwd(*r, act), ffn_bwd_bounds(*r, act, dtype),
                             ("grad_x", "grad_w_gate", "grad_w_up", "grad_w_down")):
        check(a, b, m, 1, what)
