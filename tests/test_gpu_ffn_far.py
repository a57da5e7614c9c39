"""The gated feed-forward where rows lie more than 2^32 elements apart, against float64 at some of them."""
import numpy as np
import pytest

from tests import test_gpu_ffn as T
from tests.test_gpu_ffn import S, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def test_offsets_past_32_bits(torch):
    import dflash2_block_drafter_gb300 as d
    M, H, F = 2 ** 22 + 5, 64, 1032
    g = torch.Generator(device="cuda").manual_seed(3)
    rnd = lambda *s, std=1.0: torch.empty(s, dtype=torch.bfloat16, device="cuda").normal_(0.0, std, generator=g)
    x, wg, wu, dh = rnd(M, H), rnd(F, H, std=H ** -0.5), rnd(F, H, std=H ** -0.5), rnd(M, F, std=0.01)
    h, pre = d.dflash2_gated_ffn(x, wg, wu, want_pre=True)
    dx, dwg, dwu = d.dflash2_gated_ffn_backward(dh, pre, x, wg, wu)
    assert d.dflash2_poll_error() == 0
    rows = torch.tensor([0, 1, 2 ** 31 // F, 2 ** 31 // F + 1, 2 ** 32 // F, 2 ** 32 // F + 1, M - 2, M - 1], device="cuda")
    sx, sdh, sg, su = (T._host(t[rows]) if t.numel() > F * H else T._host(t) for t in (x, dh, wg, wu))
    want, gg, uu = S.gated_ffn(sx, sg, su, "silu")
    assert np.all(np.abs(T._host(h[rows]) - want) <= T._forward_bound(sx, sg, su, gg, uu, "silu"))
    kg, ku = T._kept(pre[rows].cpu().numpy().view(np.uint32))
    for got, ref, w in ((kg, gg, sg), (ku, uu, su)):
        assert np.all(np.abs(got - ref) <= (1 + T.U) * H * T.E * T._abs_product(sx, w.T) + 2.0 ** -10 * np.abs(ref) + 2.0 ** -40)
    wdx, _, _, dg, du = S.gated_ffn_backward(sdh, kg, ku, sx, sg, su, "silu")
    # dg and du: one bf16 rounding each and a few fp32 steps of their terms; fp32 sums; one rounding of the result
    eg = T.U * np.abs(dg) + 64 * T.E * np.abs(sdh * ku) * (1 + np.abs(kg))
    eu = T.U * np.abs(du) + 64 * T.E * np.abs(sdh * kg)
    b = eg @ np.abs(sg) + eu @ np.abs(su) + 2 * F * T.E * ((np.abs(dg) + eg) @ np.abs(sg) + (np.abs(du) + eu) @ np.abs(su))
    assert np.all(np.abs(T._host(dx[rows]) - wdx) <= (1 + T.U) * b + T.U * np.abs(wdx) + 1e-30)
    # the weights' gradients run over every row: roundings are independent, far below the result
    fg, fu = torch.zeros(F, H, dtype=torch.float64, device="cuda"), torch.zeros(F, H, dtype=torch.float64, device="cuda")
    wg64, wu64 = wg.double(), wu.double()
    for at in range(0, M, 1 << 18):
        xs, ds = x[at:at + (1 << 18)].double(), dh[at:at + (1 << 18)].double()
        a, c = xs @ wg64.T, xs @ wu64.T
        s = torch.sigmoid(a)
        fg += (ds * c * s * (1 + a * (1 - s))).T @ xs
        fu += (ds * a * s).T @ xs
    for got, ref in ((dwg, fg), (dwu, fu)):
        assert float((got.double() - ref).square().mean().sqrt()) <= 0.02 * float(ref.square().mean().sqrt())
