"""GPU parity of the gated feed-forward sublayer and its gradients against float64."""
import numpy as np
import pytest

from oracle import sublayer_oracle as S

pytestmark = pytest.mark.gpu

U = 2.0 ** -8   # bf16: half a step, relative
E = 2.0 ** -24  # fp32


@pytest.fixture(scope="module")
def torch():
    from tests.gpu_util import require_gpu
    return require_gpu()


def _dev(torch, x):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(torch.bfloat16)


def _host(t):
    return t.double().cpu().numpy()


def _inputs(seed, M, H, F):
    rng = np.random.default_rng(seed)
    f = lambda *s, std=1.0: S.bf16(std * rng.normal(size=s))
    return f(M, H), f(F, H, std=H ** -0.5), f(F, H, std=H ** -0.5), f(M, F, std=0.01)


def _abs_product(a, b):
    return np.abs(a) @ np.abs(b)


def _forward_bound(x, wg, wu, g, u, kind):
    """|h - exact|: g and u carry fp32 accumulation of K products (K 2^-24 sum |.|); the gate's
    exponential and quotient a few fp32 steps (32 covers the argument's rounding at |g| < 16); one
    bf16 rounding of the result. |act'| <= 1.13."""
    K = x.shape[1]
    eg, eu = (K * E * _abs_product(x, w.T) for w in (wg, wu))
    a = np.abs(S.act(g, kind)[0])
    return (1.13 * eg * np.abs(u) + a * eu + 1.13 * eg * eu + 32 * E * (a + np.abs(g) * E) * np.abs(u)) * (1 + U) + \
        U * a * np.abs(u) + 1e-30


def _keep(g, u):
    """The kept words: sign, 6 exponent bits (bias 31), 9 mantissa bits each, ties to even."""
    def half(x):
        m, e = np.frexp(np.abs(x))
        e = np.where(x == 0, -30, np.maximum(e - 1, -30))                      # steps of 2^-39 below 2^-30
        units = np.rint(np.abs(x) / 2.0 ** (e - 9))     # 512 .. 1024, or less for the smallest
        code = ((e + 30) * 512 + units).astype(np.uint32)
        return (np.signbit(x).astype(np.uint32) << 15) | code
    return (half(g) | (half(u) << 16)).astype(np.uint32)


def _kept(words):
    def value(h):
        e, m = (h >> 9) & 63, h & 511
        v = np.where(e > 0, (512.0 + m) * 2.0 ** (e.astype(np.float64) - 31 - 9), m * 2.0 ** -39)
        return np.where(h & 0x8000, -v, v)
    return value(words & 0xFFFF), value(words >> 16)


SIZES = [(1, 8, 8), (1, 2560, 72), (48, 5128, 1096), (128, 640, 13824), (16, 64, 128), (3, 200, 136), (130, 72, 1000), (257, 512, 392), (64, 1352, 2600), (300, 2568, 264),
         (1000, 128, 512)]


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,F", SIZES)
def test_forward(torch, M, H, F, kind):
    import dflash2_block_drafter_gb300 as d
    x, wg, wu, _ = _inputs(M + F, M, H, F)
    want, g, u = S.gated_ffn(x, wg, wu, kind)
    h, pre = d.dflash2_gated_ffn(_dev(torch, x), _dev(torch, wg), _dev(torch, wu), act=kind, want_pre=True)
    assert d.dflash2_poll_error() == 0
    assert np.all(np.abs(_host(h) - want) <= _forward_bound(x, wg, wu, g, u, kind))
    for got, ref, w in zip(_kept(pre.cpu().numpy().view(np.uint32)), (g, u), (wg, wu)):
        # 10 significant bits: half a step is 2^-10, and 2^-40 below 2^-30
        assert np.all(np.abs(got - ref) <= (1 + U) * H * E * _abs_product(x, w.T) + 2.0 ** -10 * np.abs(ref) + 2.0 ** -40)
    h2 = d.dflash2_gated_ffn(_dev(torch, x), _dev(torch, wg), _dev(torch, wu), act=kind)
    assert torch.equal(h, h2)  # the same bits, with and without the kept products


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,F", SIZES)
def test_backward(torch, M, H, F, kind):
    """From given pre-activations (exact in the kept form), so that the bound is the backward pass's own: dg and
    du carry one bf16 rounding (and a few fp32 steps) each, the products fp32 accumulation, the
    results one bf16 rounding."""
    import dflash2_block_drafter_gb300 as d
    x, wg, wu, dh = _inputs(M + F, M, H, F)
    _, g, u = S.gated_ffn(x, wg, wu, kind)
    words = _keep(g, u)
    g, u = _kept(words)
    dx, dwg, dwu, dg, du = S.gated_ffn_backward(dh, g, u, x, wg, wu, kind)
    pre = torch.from_numpy(words.view(np.int32)).cuda()
    args = (_dev(torch, dh), pre, _dev(torch, x), _dev(torch, wg), _dev(torch, wu))
    got = d.dflash2_gated_ffn_backward(*args, act=kind)
    assert d.dflash2_poll_error() == 0
    # act' is a sum of terms up to 1 + |g|: its fp32 error is a few steps of those, not of the sum
    eg = U * np.abs(dg) + 64 * E * np.abs(dh * u) * (1 + np.abs(g))
    eu = U * np.abs(du) + 64 * E * np.abs(dh * g)
    ag, au = np.abs(dg) + eg, np.abs(du) + eu
    bounds = (eg @ np.abs(wg) + eu @ np.abs(wu) + 2 * F * E * (ag @ np.abs(wg) + au @ np.abs(wu)),
              eg.T @ np.abs(x) + M * E * ag.T @ np.abs(x), eu.T @ np.abs(x) + M * E * au.T @ np.abs(x))
    for t, ref, b, name in zip(got, (dx, dwg, dwu), bounds, ("dx", "dw_gate", "dw_up")):
        err = np.abs(_host(t) - ref)
        assert np.all(err <= (1 + U) * b + U * np.abs(ref) + 1e-30), f"{name}: {np.max(err / (b + U * np.abs(ref) + 1e-30))}"
        # roundings are independent: the mean square is far below the square of the worst case
        rms = np.sqrt(np.mean(err ** 2))
        assert rms <= 0.02 * np.sqrt(np.mean(ref ** 2)), f"{name}: relative rms {rms / np.sqrt(np.mean(ref**2))}"
    only_dx = d.dflash2_gated_ffn_backward(*args, act=kind, want_dw=False)
    only_dw = d.dflash2_gated_ffn_backward(*args, act=kind, want_dx=False)
    assert only_dx[1] is None and only_dw[0] is None
    assert torch.equal(only_dx[0], got[0]) and torch.equal(only_dw[1], got[1]) and torch.equal(only_dw[2], got[2])


def test_gradient_against_differences(torch):
    """The gradients through both calls against central differences of the float64 forward pass."""
    import dflash2_block_drafter_gb300 as d
    M, H, F = 33, 72, 40
    x, wg, wu, dh = _inputs(0, M, H, F)
    h, pre = d.dflash2_gated_ffn(*(_dev(torch, t) for t in (x, wg, wu)), want_pre=True)
    grads = d.dflash2_gated_ffn_backward(_dev(torch, dh), pre, *(_dev(torch, t) for t in (x, wg, wu)))
    rng = np.random.default_rng(1)
    f = lambda a, b, c: (S.gated_ffn(a, b, c, "silu")[0] * dh).sum()
    for i, grad in enumerate(grads):
        step = [rng.normal(size=t.shape) if j == i else 0.0 for j, t in enumerate((x, wg, wu))]
        e = 1e-5
        diff = (f(x + e * step[0], wg + e * step[1], wu + e * step[2]) -
                f(x - e * step[0], wg - e * step[1], wu - e * step[2])) / (2 * e)
        along = (_host(grad) * step[i]).sum()
        # rounding of g, u, dg or du, and of the gradient: independent, 2^-8 / sqrt 3 each
        size = np.sqrt((_host(grad) ** 2 * step[i] ** 2).sum())
        spread = np.sqrt(((np.abs(dh) @ np.ones((F, 1))) ** 2).sum())
        assert abs(diff - along) <= 8 * U * (size + spread)


@pytest.mark.parametrize("M,H,F", [(1001, 1544, 1736), (16, 5120, 1024), (2048, 1024, 2048)])
def test_shares_give_the_same_bits(torch, M, H, F):
    """Sizes whose tiles do not fill the SMs (k-blocks dealt out in shares): repeated calls, replayed
    graphs, and calls on two streams with their own workspaces agree bit for bit."""
    import dflash2_block_drafter_gb300 as d
    x, wg, wu, dh = (_dev(torch, t) for t in _inputs(5, M, H, F))
    n = d.dflash2_gated_ffn_workspace_bytes(M, H, F, 1)
    new = lambda: torch.full((n,), 255, dtype=torch.uint8, device="cuda")
    ws = new()

    def step(ws):
        h, pre = d.dflash2_gated_ffn(x, wg, wu, want_pre=True, workspace=ws)
        return (h, *d.dflash2_gated_ffn_backward(dh, pre, x, wg, wu, workspace=ws))

    want = step(ws)
    for _ in range(3):
        assert all(torch.equal(a, b) for a, b in zip(want, step(ws)))
    graph = torch.cuda.CUDAGraph()
    torch.cuda.synchronize()
    with torch.cuda.graph(graph):
        out = step(ws)
    for _ in range(3):
        for t in out:
            t.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(want, out))
    streams = [torch.cuda.Stream() for _ in range(2)]
    spaces = [new(), new()]
    torch.cuda.synchronize()
    results = []
    for s, w in zip(streams, spaces):
        with torch.cuda.stream(s):
            results.append([step(w) for _ in range(3)])
    torch.cuda.synchronize()
    assert d.dflash2_poll_error() == 0
    for per in results:
        for r in per:
            assert all(torch.equal(a, b) for a, b in zip(want, r))


def test_no_rows_and_large_values(torch):
    import dflash2_block_drafter_gb300 as d
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(16, 64, dtype=torch.bfloat16, device="cuda")
    h, pre = d.dflash2_gated_ffn(z, w, w, want_pre=True)
    assert h.shape == (0, 16)
    dx, dwg, dwu = d.dflash2_gated_ffn_backward(torch.empty(0, 16, dtype=torch.bfloat16, device="cuda"), pre, z, w, w)
    assert dx.shape == (0, 64) and not dwg.any() and not dwu.any()
    # gates far out: act saturates to g or 0 without an overflow on the way
    for kind in ("silu", "gelu_tanh"):
        x = torch.zeros(2, 64, dtype=torch.bfloat16, device="cuda")
        x[0, 0], x[1, 0] = 128.0, -128.0
        wg = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
        wg[:, 0] = 64.0
        wu = torch.zeros(8, 64, dtype=torch.bfloat16, device="cuda")
        wu[:, 0] = 1.0
        h = d.dflash2_gated_ffn(x, wg, wu, act=kind)
        assert bool((h[0] == 128.0 * 64.0 * 128.0).all()) and not h[1].any()
    assert d.dflash2_poll_error() == 0
