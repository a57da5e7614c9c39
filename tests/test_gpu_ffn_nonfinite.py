"""A row of the gated feed-forward that is not finite: its output, and the gradients that it enters, say so."""
import pytest

from tests.test_gpu_ffn import _dev, _inputs, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("M,H,F", [(7, 64, 40), (300, 256, 264)])
def test_a_row_that_is_not_finite(torch, M, H, F, kind, bad):
    import dflash2_block_drafter_gb300 as d
    x, wg, wu, dh = (_dev(torch, t) for t in _inputs(M, M, H, F))
    at, rest = 5, [i for i in range(M) if i != 5]
    wg[:, 3] = wg[:, 3].abs() + 0.125  # (an infinite gate, never a product of zero and infinity)
    wu[:, 3] = wu[:, 3].abs() + 0.125
    h0, pre0 = d.dflash2_gated_ffn(x, wg, wu, act=kind, want_pre=True)
    dx0, _, _ = d.dflash2_gated_ffn_backward(dh, pre0, x, wg, wu, act=kind)
    x[at, 3] = bad
    h, pre = d.dflash2_gated_ffn(x, wg, wu, act=kind, want_pre=True)
    dx, dwg, dwu = d.dflash2_gated_ffn_backward(dh, pre, x, wg, wu, act=kind)
    assert d.dflash2_poll_error() == 0
    assert not h[at].isfinite().any() and torch.equal(h[rest], h0[rest]) and torch.equal(pre[rest], pre0[rest])
    words = pre[at] & 0xFFFF, (pre[at] >> 16) & 0xFFFF
    for w in words:  # exponent bits all set; mantissa 0 for an infinity
        assert bool(((w & 0x7E00) == 0x7E00).all()) and bool((((w & 0x1FF) != 0) == (bad != bad)).all())
    assert not dx[at].isfinite().any() and torch.equal(dx[rest], dx0[rest])
    assert not dwg.isfinite().any() and not dwu.isfinite().any()


def test_an_infinite_up_product_keeps_its_sign(torch):
    """g finite, u of either sign infinite: the kept words are infinities of that sign."""
    import dflash2_block_drafter_gb300 as d
    x = torch.zeros(3, 64, dtype=torch.bfloat16, device="cuda")
    x[:, 0] = 1.0
    wg = torch.full((8, 64), 0.5, dtype=torch.bfloat16, device="cuda")
    wu = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
    wu[:4, 0], wu[4:, 0] = float("inf"), -float("inf")
    h, pre = d.dflash2_gated_ffn(x, wg, wu, want_pre=True)
    words = (pre >> 16) & 0xFFFF
    assert bool((words[:, :4] == 0x7E00).all()) and bool((words[:, 4:] == 0xFE00).all())
    assert d.dflash2_poll_error() == 0
