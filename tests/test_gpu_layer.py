"""A whole drafter layer (conv sites, projections, attention over the 4-bit cache, gated feed-forward)
against its float64 statement, eagerly and replayed from a CUDA graph."""
import numpy as np
import pytest

from oracle import dflash2_oracle as O
from oracle import sublayer_oracle as S
from synth import inputs as I
from tests.parity import assert_close_scaled

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    from tests.gpu_util import require_gpu
    return require_gpu()


@pytest.mark.parametrize("B,G,window", [(3, 16, 0), (1, 8, 40), (20, 16, 0)])
def test_layer_matches_float64(torch, B, G, window):
    from dflash2_block_drafter_gb300 import dflash2_poll_error
    from dflash2_block_drafter_gb300.layer import LayerRunner, LayerWeights
    from dflash2_block_drafter_gb300.tail import SiteWeights, to_device
    H, Hq, Hkv, D, F, gs, page = 256, 6, 2, 64, 640, 16, 32
    rng = np.random.default_rng(B)
    sites = [I.conv_site(B, f"site{i}", B, G, H, gs, "bf16") for i in range(2)]
    f = lambda *s, std=1.0: S.bf16(std * rng.normal(size=s))
    dev = lambda x: torch.from_numpy(np.ascontiguousarray(x)).cuda().to(torch.bfloat16)
    w_qkv, w_o = f((Hq + 2 * Hkv) * D, H, std=H ** -0.5), f(H, Hq * D, std=(Hq * D) ** -0.5)
    w_gate, w_up, w_down = f(F, H, std=H ** -0.5), f(F, H, std=H ** -0.5), f(H, F, std=F ** -0.5)
    site = lambda s: SiteWeights(to_device(s.w_kp), to_device(s.base), to_device(s.norm_w))
    lens = [int(n) for n in rng.integers(0, 300, B)]
    need = [-(-n // page) for n in lens]
    width = max(1, max(need))
    run = LayerRunner(LayerWeights(site(sites[0]), dev(w_qkv), dev(w_o), site(sites[1]), dev(w_gate), dev(w_up),
                                   dev(w_down)), B, G, Hq, Hkv, D, sum(need) + 1, width, page, gs, window=window)
    run.cache.fill_(255)
    table = np.zeros((B, width), np.int32)
    at, K, V = 1, [], []
    for b, n in enumerate(lens):
        table[b, :need[b]] = np.arange(at, at + need[b])
        at += need[b]
        k, v = f(n, Hkv, D), f(n, Hkv, D)
        i = np.arange(n)
        run.append_context(dev(k), dev(v), torch.from_numpy(table[b, i // page].astype(np.int64) * page + i % page).cuda())
        K.append(S.kv4_values(k))
        V.append(S.kv4_values(v))
    x = f(B, G, H)
    tab, ctx = torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda")
    dx = dev(x)
    got = run.forward(dx, tab, ctx).clone()
    assert dflash2_poll_error() == 0

    # the same in float64
    def conv(i, n, norm):
        s = sites[i]
        return O.conv_prepare(n, I.to_f64(s.norm_w) if norm else None, 1e-6, I.to_f64(s.w_kp), s.base.astype(np.float64), gs)[:2]
    a, d1 = conv(0, x, True)
    qkv = a @ w_qkv.T
    o = np.zeros((B, G, Hq, D))
    for b in range(B):
        q, k, v = np.split(qkv[b], [Hq * D, (Hq + Hkv) * D], axis=-1)
        o[b], _ = S.attention(q.reshape(G, Hq, D), np.concatenate([K[b], k.reshape(G, Hkv, D)]),
                              np.concatenate([V[b], v.reshape(G, Hkv, D)]), S.seen(G, lens[b], G, False, window), D ** -0.5)
    mid = O.conv_finish(o.reshape(B, G, -1) @ w_o.T, d1, sites[0].base.astype(np.float64), gs, x)
    n = O.rms_norm(mid, I.to_f64(sites[1].norm_w), 1e-6)
    a, d1 = conv(1, n, False)
    h, _, _ = S.gated_ffn(a.reshape(B * G, H), w_gate, w_up, "silu")
    want = O.conv_finish((h @ w_down.T).reshape(B, G, H), d1, sites[1].base.astype(np.float64), gs, mid)
    assert_close_scaled(got.double().cpu().numpy(), want, what="layer")

    graph = run.capture(dx, tab, ctx)
    run.x.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.equal(run.x, got)
    # lengths are read at replay: an empty context still gives the block's own rows
    ctx.zero_()
    graph.replay()
    torch.cuda.synchronize()
    assert torch.isfinite(run.x.float()).all() and not torch.equal(run.x, got)
    assert dflash2_poll_error() == 0
