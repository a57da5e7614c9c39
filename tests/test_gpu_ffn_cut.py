"""Products of the gated feed-forward whose tiles are cut into shares, one for each of the three: the same bits from
repeated calls, replayed graphs, and calls on two streams with workspaces of their own. That tiles are cut shows in
the workspace: the partial tiles at its start are written, and nothing else of it is up to its flags."""
import numpy as np
import pytest

from tests.test_gpu_ffn import _dev, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


# (far from the sizes where the rule changes: 36 tiles of 200 k-blocks, 4 of 200, 8 of 128, on 66 to 80 pairs)
@pytest.mark.parametrize("what,M,H,F", [("forward", 300, 12800, 2304), ("dx", 500, 512, 6400), ("dw", 8192, 512, 512)])
def test_cut_tiles_give_the_same_bits(torch, what, M, H, F):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(M)
    f = lambda *s, std=1.0: _dev(torch, (std * rng.standard_normal(s, dtype=np.float32)))
    x, wg, wu, dh = f(M, H), f(F, H, std=H ** -0.5), f(F, H, std=H ** -0.5), f(M, F, std=0.01)
    share = d.dflash2_gated_ffn_workspace_bytes(M, H, F, 0)  # (H a multiple of 64: partial tiles and flags only)
    new = lambda: torch.full((d.dflash2_gated_ffn_workspace_bytes(M, H, F, 1),), 255, dtype=torch.uint8, device="cuda")
    _, pre = d.dflash2_gated_ffn(x, wg, wu, want_pre=True)

    def step(ws):
        if what == "forward":
            return d.dflash2_gated_ffn(x, wg, wu, want_pre=True, workspace=ws)
        return [t for t in d.dflash2_gated_ffn_backward(dh, pre, x, wg, wu, want_dx=what == "dx", want_dw=what == "dw",
                                                        workspace=ws) if t is not None]

    same = lambda p, q: all(torch.equal(a, b) for a, b in zip(p, q))
    ws = new()
    want = step(ws)
    assert bool((ws[:share // 2] != 255).any()), "no tile was cut"
    assert same(want, step(new())) and all(same(want, step(ws)) for _ in range(3))
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = step(ws)
    for _ in range(3):
        for t in out:
            t.zero_()
        graph.replay()
        torch.cuda.synchronize()
        assert same(want, out)
    streams, spaces, results = [torch.cuda.Stream() for _ in range(2)], [new(), new()], []
    torch.cuda.synchronize()
    for s, w in zip(streams, spaces):
        with torch.cuda.stream(s):
            results.append([step(w) for _ in range(3)])
    torch.cuda.synchronize()
    assert d.dflash2_poll_error() == 0
    assert all(same(want, r) for per in results for r in per)


def test_cut_tiles_against_float64(torch):
    """A cut forward product: fp32 sums of 12800 products (each rounding at most 2^-24 of the sum of their sizes), |act'|
    at most 1.13, one bf16 rounding, 2^-8; roundings being independent, the mean square stays below that rounding's."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(1)
    M, H, F = 300, 12800, 2304
    f = lambda *s, std=1.0: _dev(torch, (std * rng.standard_normal(s, dtype=np.float32)))
    x, wg, wu = f(M, H), f(F, H, std=H ** -0.5), f(F, H, std=H ** -0.5)
    h = d.dflash2_gated_ffn(x, wg, wu)
    assert d.dflash2_poll_error() == 0
    g, u = x.double() @ wg.double().T, x.double() @ wu.double().T
    eg, eu = (H * 2.0 ** -24 * (x.double().abs() @ w.double().abs().T) for w in (wg, wu))
    a = g * torch.sigmoid(g)
    err = (h.double() - a * u).abs()
    assert bool((err <= 2.0 ** -8 * (a * u).abs() + 1.01 * (1.13 * eg * (u.abs() + eu) + a.abs() * eu) + 1e-6).all())
    assert float(err.square().mean()) <= 2.0 ** -16 * float((a * u).square().mean())
