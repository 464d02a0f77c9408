"""Layer normalisation of more rows than workgroups, so that each walks over several rows with the
next one in flight, and of tensors of 8 MiB and more, which are loaded and stored past the caches;
odd widths end in a cut pack.  Bounds as in test_gpu_norm.py."""
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check  # noqa: E402
from test_gpu_norm import case, fwd_mag  # noqa: E402

import numpy as np  # noqa: E402

MIB8 = 8 << 20


def R():
    import retnet_retention_fwd_amd as R_
    return R_


# forward: at most 2048 workgroups of four rows (up to 1024 columns) or of one
@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,D", [(2051, 2048), (4099, 1111), (8203, 515), (2053, 4099)])
def test_forward(rows, D, dtype, wtype):
    print(f"\n[case] norm large fwd {rows}x{D} {dtype}/{wtype}", flush=True)
    assert rows > 2048 * (4 if D <= 1024 else 1) and rows * D * TYPES[dtype].itemsize >= MIB8
    (x, w, b, _), (xr, wr, br, _) = case(rows, D, dtype, wtype)
    y, mean, rstd = R().layer_norm_fwd(x, w, b, eps=1e-5, return_stats=True)
    ry, rm, rr = O.layer_norm(xr, wr, br, 1e-5)
    size = np.mean(np.abs(xr), 1)
    check(mean, rm, size, 128, "mean")
    check(rstd, rr, rr * (1 + 2 * size * rr), 128, "rstd")
    check(y, ry, fwd_mag(xr, wr, br, rm, rr, ry), 128, "y")


# backward: at most 512 workgroups of four rows, then 768, 512 and 256 of one
@pytest.mark.parametrize("dtype,wtype", [("f32", "f32"), ("bf16", "bf16"), ("bf16", "f32")])
@pytest.mark.parametrize("rows,D,most", [(4411, 961, 2048), (2053, 2047, 768), (2049, 2048, 768), (1031, 4100, 256),
                                         (517, 8191, 256), (359, 12001, 256)])
def test_backward(rows, D, most, dtype, wtype):
    print(f"\n[case] norm large bwd {rows}x{D} {dtype}/{wtype}", flush=True)
    assert rows > most and rows * D * TYPES[dtype].itemsize >= MIB8
    (x, w, _, g), (xr, wr, _, gr) = case(rows, D, dtype, wtype, 10)
    _, rm, rr = O.layer_norm(xr, eps=1e-5)
    mean, rstd = (torch.tensor(v).float().cuda() for v in (rm, rr))
    stats = mean.double().cpu().numpy(), rstd.double().cpu().numpy()
    got = R().layer_norm_bwd(x, w, mean, rstd, g)
    ref = O.layer_norm_bwd(xr, wr, *stats, gr)
    mag = O.layer_norm_bwd(xr, wr, *stats, gr, magnitude=True)
    for v, r, m, what in zip(got, ref, mag, ("grad_x", "grad_weight", "grad_bias")):
        check(v, r, m, 128 + rows / 64, what)
