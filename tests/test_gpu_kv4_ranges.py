"""Attention over the 4-bit cache where a CTA's range holds many tiles, many items, or a small part of one item;
extreme magnitudes and scales; replays of items that many ranges share."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import S, _cached, _check, _dev, _host, _rows, _run, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("G,Hq,Hkv,D", [(1, 8, 2, 128), (4, 16, 2, 64), (4, 16, 2, 128), (10, 16, 2, 128), (5, 24, 2, 64)])
def test_many_tiles_a_range_and_the_same_bits_every_time(torch, G, Hq, Hkv, D):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(G * D + Hq)
    lens = [int(n) for n in rng.integers(900, 3600, 48)]
    lens[5], lens[11] = 0, 4096
    cache, table, ctx, K, V = _cached(torch, d, rng, lens, Hkv, D, 128)
    q = _rows(rng, len(lens), G, Hq, D)
    kn, vn = _rows(rng, len(lens), G, Hkv, D), _rows(rng, len(lens), G, Hkv, D)
    args = (_dev(torch, q), cache, table, ctx, 128, D ** -0.5)
    kw = dict(k_new=_dev(torch, kn), v_new=_dev(torch, vn))
    out = d.dflash2_kv4_attention(*args, **kw)
    for _ in range(20):
        assert torch.equal(out, d.dflash2_kv4_attention(*args, **kw))
    assert d.dflash2_poll_error() == 0
    want, sd = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        want[b], sd[b] = S.attention(q[b], np.concatenate([K[b], kn[b]]), np.concatenate([V[b], vn[b]]),
                                     S.seen(G, n, G, False, 0), D ** -0.5)
    _check(_host(out), want, sd, f"G={G} {Hq}/{Hkv} D={D}")


@pytest.mark.parametrize("B,Hkv,D", [(300, 1, 64), (65, 3, 128), (33, 8, 64)])
@pytest.mark.parametrize("new", [False, True])
def test_many_short_sequences(torch, B, Hkv, D, new):
    lens = [int(n) for n in np.random.default_rng(B).integers(0, 40, B)]
    _run(torch, B, lens, 1, 2 * Hkv, Hkv, D, 16, new=new)


@pytest.mark.parametrize("scale", [0.0, -0.125, 4.0])
def test_scales_of_any_sign(torch, scale):
    _run(torch, 3, [200, 5], 3, 4, 2, 64, 32, scale=scale)


@pytest.mark.parametrize("qm,km,vm", [(0.0, 1.0, 1.0), (1e-30, 1e30, 1e-20), (1e18, 1e-18, 1e25), (1.0, 0.0, 0.0),
                                      (1e10, 1e-10, 1e-30)])
def test_magnitudes(torch, qm, km, vm):
    """The powers of two that operands are divided by hold from the smallest to the largest bf16 numbers."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(17)
    T, G, Hq, Hkv, D, page = 150, 2, 4, 2, 64, 32
    k, v = S.bf16(_rows(rng, T, Hkv, D) * km), S.bf16(_rows(rng, T, Hkv, D) * vm)
    q = S.bf16(_rows(rng, 1, G, Hq, D) * qm)
    cache = d.dflash2_kv4_cache(5, Hkv, D, page)
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), torch.arange(T, device="cuda"), cache, page)
    table = torch.arange(5, dtype=torch.int32, device="cuda")[None]
    ctx = torch.tensor([T], dtype=torch.int32, device="cuda")
    out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, 0.125)
    assert d.dflash2_poll_error() == 0
    want, sd = S.attention(q[0], S.kv4_values(k), S.kv4_values(v), S.seen(G, T, 0, False, 0), 0.125)
    unit = max(vm, 1e-38)
    _check(_host(out)[0] / unit, want / unit, sd / unit, f"q {qm} k {km} v {vm}")


@pytest.mark.parametrize("n,G,Hq,Hkv", [(20000, 1, 4, 1), (9000, 10, 8, 1), (3000, 2, 16, 2)])
def test_shared_items_in_a_graph(torch, n, G, Hq, Hkv):
    """An item cut into a hundred parts, a dozen, or a few: eager and replayed results have the same bits, also
    when another call's results lie in between."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(n)
    D, page = 128, 256
    cache, table, ctx, K, V = _cached(torch, d, rng, [n, 100], Hkv, D, page)
    q, q2 = _rows(rng, 2, G, Hq, D), _rows(rng, 2, G, Hq, D)
    x = _dev(torch, q)
    first = d.dflash2_kv4_attention(x, cache, table, ctx, page, 0.1)
    other = d.dflash2_kv4_attention(_dev(torch, q2), cache, table, ctx, page, 0.1)
    stream = torch.cuda.Stream()
    stream.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(stream):
        d.dflash2_kv4_attention(x, cache, table, ctx, page, 0.1)
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph, stream=stream):
            out = d.dflash2_kv4_attention(x, cache, table, ctx, page, 0.1)
    torch.cuda.current_stream().wait_stream(stream)
    for y, want in ((q, first), (q2, other), (q, first)):
        x.copy_(_dev(torch, y))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    assert d.dflash2_poll_error() == 0
    for b, m in enumerate((n, 100)):
        want, sd = S.attention(q[b], K[b], V[b], S.seen(G, m, 0, False, 0), 0.1)
        _check(_host(first)[b], want, sd, f"{m} keys")
