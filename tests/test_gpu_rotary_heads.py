"""Rotary positions with enough tokens that a thread walks over several heads: batches of four heads
in flight, a batch that the head count cuts, one that begins with queries and ends with keys (other
memory, strides and scale).  Bounds as in test_gpu_rotary.py.
"""
import numpy as np
import pytest

import oracle as O

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu

from block_cases import TYPES, check, draw  # noqa: E402
from test_gpu_rotary import sizes  # noqa: E402


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def heads_of_a_thread(tokens, heads, d, rot, dtype, interleaved):
    """The launcher's rule: the most heads up to 16 that leave 2^17 threads."""
    v, rest = 16 // TYPES[dtype].itemsize, d - rot
    part = rot if interleaved else rot // 2
    units = part // v + rest // v if part % v == 0 and rest % v == 0 else rot // 2 + rest
    per = 16
    while per > 1 and tokens * units * -(-heads // per) < 1 << 17:
        per //= 2
    return per


def one(q, k, qr, kr, freq, table, N, rot, interleaved, back, **out):
    f = R().rotary_bwd if back else R().rotary_fwd
    got = f(q, k, table, offset=3, interleaved=interleaved, q_scale=0.75, k_scale=0.1, **out)
    for g, x, scale in ((got[0], qr, 0.75), (got[1], kr, 0.1)):
        ref = O.rotary(x, np.arange(N) + 3, freq.numpy(), interleaved, scale, backward=back)
        check(g, ref, sizes(x, rot, interleaved) * scale, 8)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
@pytest.mark.parametrize("Hq,Hk,per,back", [(17, 5, 16, False), (16, 16, 16, True), (3, 6, 8, True), (3, 4, 4, False)])
def test_packs(Hq, Hk, per, back, dtype, interleaved):
    d = rot = 32
    # units of a token: 4 (bf16, pairs adjacent), 8 (fp32) or half of these
    N = 65536 // (d // (16 // TYPES[dtype].itemsize) // (1 if interleaved else 2))
    print(f"\n[case] rotary heads {Hq} {Hk} {N} {dtype} {interleaved} {back}", flush=True)
    assert heads_of_a_thread(N, Hq + Hk, d, rot, dtype, interleaved) == per
    freq = R().rotary_frequencies(rot)
    table = R().rotary_table(freq, N + 3)
    # queries head-major, keys token-major inside wider rows
    q, qr = draw(1, (1, Hq, N, d), dtype)
    wide, wr = draw(2, (1, N, Hk + 1, d), dtype)
    k, kr = wide[:, :, 1:].transpose(1, 2), wr[:, :, 1:].transpose(0, 2, 1, 3)
    one(q, k, qr, kr, freq, table, N, rot, interleaved, back)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_in_place_in_joint_rows(dtype, interleaved):
    B, N, Hq, Hk, d, rot = 2, 8192, 10, 5, 64, 32
    print(f"\n[case] rotary heads in place {dtype} {interleaved}", flush=True)
    assert heads_of_a_thread(B * N, Hq + Hk, d, rot, dtype, interleaved) >= 8      # the third batch of four crosses
    freq = R().rotary_frequencies(rot)
    table = R().rotary_table(freq, N + 3)
    joint, jr = draw(3, (B, N, Hq + 2 * Hk, d), dtype)
    q, k = joint[:, :, :Hq].transpose(1, 2), joint[:, :, Hq:Hq + Hk].transpose(1, 2)
    rest = joint[:, :, Hq + Hk:].clone()
    qr, kr = jr[:, :, :Hq].transpose(0, 2, 1, 3), jr[:, :, Hq:Hq + Hk].transpose(0, 2, 1, 3)
    one(q, k, qr, kr, freq, table, N, rot, interleaved, False, out_q=q, out_k=k)
    assert torch.equal(joint[:, :, Hq + Hk:], rest)


@pytest.mark.parametrize("interleaved", [True, False])
@pytest.mark.parametrize("dtype", ["f32", "bf16"])
def test_single_elements(dtype, interleaved):
    """An odd head: pairs and single elements instead of packs, 18 heads as 16 and 2."""
    N, Hq, Hk, d, rot = 4096, 13, 5, 33, 6
    print(f"\n[case] rotary heads odd {dtype} {interleaved}", flush=True)
    assert heads_of_a_thread(N, Hq + Hk, d, rot, dtype, interleaved) == 16
    freq = R().rotary_frequencies(rot)
    table = R().rotary_table(freq, N + 3)
    q, qr = draw(4, (1, Hq, N, d), dtype)
    k, kr = draw(5, (1, Hk, N, d), dtype)
    one(q, k, qr, kr, freq, table, N, rot, interleaved, False)
