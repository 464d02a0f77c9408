"""Launches of the projections by kind: a forward sums no gradients, and a cut product's join is a kind of its own."""
import pytest

torch = pytest.importorskip("torch")
pytestmark = pytest.mark.gpu


def R():
    import retnet_retention_fwd_amd as R_
    return R_


def launches(op):
    """Launches of each kind that one call makes."""
    op()
    torch.cuda.synchronize()
    R().profile_enable(True)
    try:
        op()
        return {k: v["launches"] for k, v in R().profile_read().items() if isinstance(v, dict) and v["launches"]}
    finally:
        R().profile_enable(False)


def test_a_forward_sums_no_gradients():
    print("\n[case] profile of forwards", flush=True)
    draw = lambda *s: torch.randn(s, device="cuda").bfloat16()
    x, w, wd = draw(128, 2048), draw(4096, 2048), draw(2048, 4096)
    # 32 and 64 tiles with 32 steps and more each: their reduction is cut
    assert launches(lambda: R().linear_fwd(x, w)) == {"projection": 1, "projection_join": 1}
    assert launches(lambda: R().gated_ffn_fwd(x, w, w, wd)) == {"projection": 2, "projection_join": 2}
    # few rows are not
    assert launches(lambda: R().linear_fwd(x[:16], w)) == {"projection": 1}


def test_a_backward_names_its_sums():
    print("\n[case] profile of a backward", flush=True)
    draw = lambda *s: torch.randn(s, device="cuda").bfloat16()
    x, w, gy = draw(2048, 136), draw(264, 136), draw(2048, 264)
    got = launches(lambda: R().linear_bwd(x, w, gy))
    assert got["projection"] == 2 and got["gradient_sums"] == 1 and got["projection_join"] >= 1    # grad_bias; grad_weight
    assert "projection_join" not in launches(lambda: R().linear_bwd(x, w, gy, x_grad=False, weight_grad=False))
