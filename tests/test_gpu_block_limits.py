"""Calls near the documented limits of the operators around the retention."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def R():
    import retnet_retention_fwd_amd as R_
    return R_


@pytest.mark.parametrize("interleaved", [True, False])
def test_rotary_of_more_workgroups_than_a_launch_takes(interleaved):
    """17 million tokens of one head of 130 elements, two of them turned: 129 units leave a workgroup
    of 256 threads one token, 4.4e9 threads in all, where a launch takes 2^32.  The elements that
    are not turned pass unchanged.  The kernel's two turned ones and the comparison's are off by
    four roundings of fp32 each at most, and the kernel's by the rounding to bf16, half a step of
    a value that is itself off by those eight: 8 (1 + 2^-8) < 9."""
    N, d, far = 17_000_001, 130, 64
    print(f"\n[case] rotary limits {N} {d} {interleaved}", flush=True)
    q = torch.empty(1, 1, N, d, dtype=torch.bfloat16, device="cuda")
    q.uniform_(-1, 1, generator=torch.Generator("cuda").manual_seed(1))
    pos = torch.arange(N, device="cuda") % far
    table = R().rotary_table(R().rotary_frequencies(2), far)
    got = R().rotary_fwd(q, None, table, positions=pos, interleaved=interleaved)
    step = 1 << 22
    for lo in range(0, N, step):
        g, x = got[0, 0, lo:lo + step], q[0, 0, lo:lo + step]
        assert torch.equal(g[:, 2:], x[:, 2:])
        c, s = table[pos[lo:lo + step], 0].unbind(-1)
        a, b = x[:, 0].float(), x[:, 1].float()
        for have, want in ((g[:, 0].float(), a * c - b * s), (g[:, 1].float(), a * s + b * c)):
            room = 2.0 ** -8 * want.abs() + 9 * 2.0 ** -24 * (a.abs() + b.abs())
            assert bool(((have - want).abs() <= room).all())
