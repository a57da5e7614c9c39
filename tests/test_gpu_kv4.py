"""GPU parity of the 4-bit key/value cache: rows in and out bit for bit, attention against float64."""
import numpy as np
import pytest

from oracle import sublayer_oracle as S

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module")
def torch():
    from tests.gpu_util import require_gpu
    return require_gpu()


def _rows(rng, *shape):
    return S.bf16(rng.normal(size=shape))


def _dev(torch, x):
    return torch.from_numpy(np.ascontiguousarray(x)).to("cuda").to(torch.bfloat16)


def _host(t):
    return t.double().cpu().numpy()


def _cached(torch, d, rng, lens, heads, D, page, spare=2):
    """A cache holding sequences of the given lengths in shuffled pages: (cache, table, ctx, K, V lists
    of float64 values). Pages are filled by append in one shuffled call; the rest of the cache is 0xFF
    bytes (codes 15 with NaN scales), which no call may let through."""
    need = [-(-n // page) for n in lens]
    pages = sum(need) + spare
    cache = d.dflash2_kv4_cache(pages, heads, D, page)
    cache.fill_(255)
    order = rng.permutation(pages)
    table = np.full((len(lens), max(1, max(need))), 10 ** 6, np.int32)  # unused entries are not looked at
    slots, ks, vs, at = [], [], [], 0
    for b, n in enumerate(lens):
        table[b, :need[b]] = order[at:at + need[b]]
        at += need[b]
        i = np.arange(n)
        slots.append(table[b, i // page].astype(np.int64) * page + i % page)
        ks.append(_rows(rng, n, heads, D))
        vs.append(_rows(rng, n, heads, D))
    total = sum(lens)
    if total:
        mix = rng.permutation(total)
        d.dflash2_kv4_append(_dev(torch, np.concatenate(ks)[mix]), _dev(torch, np.concatenate(vs)[mix]),
                             torch.from_numpy(np.concatenate(slots)[mix]).cuda(), cache, page)
    return (cache, torch.from_numpy(table).cuda(), torch.tensor(lens, dtype=torch.int32, device="cuda"),
            [S.kv4_values(k) for k in ks], [S.kv4_values(v) for v in vs])


def _check(got, want, sd, what):
    """Rounding errors are independent and within half a step each: no element beyond 8 standard
    deviations (and fp32 noise), and the mean square within twice its expectation (+ 1e-12)."""
    err = np.abs(got - want)
    assert np.isfinite(got).all(), f"{what}: not finite"
    assert np.all(err <= 8 * sd + 1e-5), f"{what}: {np.max(err / (sd + 1e-9))} standard deviations"
    assert np.mean(err ** 2) <= 2 * np.mean(sd ** 2) + 1e-12, f"{what}: mean square {np.mean(err**2)} of {np.mean(sd**2)}"


def _run(torch, seed, lens, G, Hq, Hkv, D, page, causal=False, window=0, new=True, scale=None):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(seed)
    B = len(lens)
    cache, table, ctx, K, V = _cached(torch, d, rng, lens, Hkv, D, page)
    q = _rows(rng, B, G, Hq, D)
    kn, vn = _rows(rng, B, G, Hkv, D), _rows(rng, B, G, Hkv, D)
    scale = D ** -0.5 if scale is None else scale
    # q, k and v as slices of one fused projection's rows
    fused = _dev(torch, np.concatenate([q.reshape(B, G, -1), kn.reshape(B, G, -1), vn.reshape(B, G, -1)], -1))
    nq, nk = Hq * D, Hkv * D
    kw = dict(k_new=fused[..., nq:nq + nk].unflatten(-1, (Hkv, D)),
              v_new=fused[..., nq + nk:].unflatten(-1, (Hkv, D))) if new else {}
    out = d.dflash2_kv4_attention(fused[..., :nq].unflatten(-1, (Hq, D)), cache, table, ctx, page, scale,
                                  causal=causal, window=window, **kw)
    assert d.dflash2_poll_error() == 0
    want, sd = np.zeros((B, G, Hq, D)), np.zeros((B, G, Hq, D))
    for b, n in enumerate(lens):
        k, v = (np.concatenate([K[b], kn[b]]), np.concatenate([V[b], vn[b]])) if new else (K[b], V[b])
        want[b], sd[b] = S.attention(q[b], k, v, S.seen(G, n, G if new else 0, causal, window), scale)
    _check(_host(out), want, sd, f"attention {lens} G={G} {Hq}/{Hkv} D={D} page={page}")


@pytest.mark.parametrize("T,heads,D,page", [(1, 1, 64, 16), (33, 3, 128, 64), (1000, 2, 64, 32), (257, 8, 128, 256)])
def test_rows_round_trip_bit_for_bit(torch, T, heads, D, page):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(T)
    k, v = _rows(rng, T, heads, D), _rows(rng, T, heads, D)
    k[0, 0, :64] = 0.5                       # a constant group: scale 0
    k[-1, -1, :64] = np.linspace(-3e38, 3e38, 64)[0]
    v[0, 0, :64] = S.bf16(np.linspace(1e-30, 2e-30, 64))
    k = S.bf16(k)
    pages = -(-T // page) + 1
    cache = d.dflash2_kv4_cache(pages, heads, D, page)
    cache.zero_()
    slots = rng.permutation(pages * page)[:T].astype(np.int64)
    skip = rng.random(T) < 0.1
    slots_in = np.where(skip, -1, slots)
    s = torch.from_numpy(slots_in).cuda()
    wide = torch.zeros(T, 2 * heads * D + 8, dtype=torch.bfloat16, device="cuda")
    wide[:, :heads * D] = _dev(torch, k).flatten(1)
    wide[:, heads * D:2 * heads * D] = _dev(torch, v).flatten(1)
    d.dflash2_kv4_append(wide[:, :heads * D].unflatten(1, (heads, D)),
                         wide[:, heads * D:2 * heads * D].unflatten(1, (heads, D)), s, cache, page)
    kr, vr = d.dflash2_kv4_read(cache, s, D, page)
    assert d.dflash2_poll_error() == 0
    for got, x in ((kr, k), (vr, v)):
        want = np.where(skip[:, None, None], 0.0, S.bf16(S.kv4_values(x)))
        np.testing.assert_array_equal(_host(got), want)
    # the bytes themselves, of one row
    r = int(np.nonzero(~skip)[0][0])
    pg, at = divmod(int(slots[r]), page)
    gran = cache[pg, 0, 0, at // 16].cpu().numpy()
    code, scale, bias = S.kv4_quantise(k[r, 0])
    row = gran[at % 16 * (D // 2):(at % 16 + 1) * (D // 2)]
    np.testing.assert_array_equal(np.stack([row & 15, row >> 4], -1).ravel(), code.ravel())
    par = gran[16 * D // 2:].view(np.uint16).reshape(16, D // 64, 2)[at % 16].astype(np.uint32) << 16
    np.testing.assert_array_equal(par.view(np.float32), np.stack([scale, bias], -1).astype(np.float32))


def test_skipped_rows_leave_the_cache_alone_and_bad_slots_are_recorded(torch):
    import dflash2_block_drafter_gb300 as d
    cache = d.dflash2_kv4_cache(2, 2, 64, 16)
    cache.fill_(7)
    k = torch.ones(3, 2, 64, dtype=torch.bfloat16, device="cuda")
    d.dflash2_kv4_append(k, k, torch.tensor([-1, -5, -2 ** 40], device="cuda"), cache, 16)
    assert d.dflash2_poll_error() == 0 and bool((cache == 7).all())
    d.dflash2_kv4_append(k, k, torch.tensor([32, 2 ** 40, -1], device="cuda"), cache, 16)
    assert d.dflash2_poll_error() == -6 and bool((cache == 7).all())
    kr, vr = d.dflash2_kv4_read(cache, torch.tensor([32], device="cuda"), 64, 16)
    assert d.dflash2_poll_error() == -6 and not kr.any() and not vr.any()
    none = torch.empty(0, 2, 64, dtype=torch.bfloat16, device="cuda")
    d.dflash2_kv4_append(none, none, torch.empty(0, dtype=torch.int64, device="cuda"), cache, 16)
    assert d.dflash2_poll_error() == 0


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("lens,G,Hq,Hkv,page", [
    ([1], 1, 1, 1, 16), ([17], 1, 4, 1, 16), ([31, 32, 33], 1, 8, 2, 64), ([129, 0, 4000], 1, 10, 2, 256),
    ([100, 15], 3, 4, 4, 32), ([700, 64], 16, 10, 2, 64), ([300], 64, 3, 1, 128), ([65, 1], 7, 24, 2, 16),
    ([513], 1, 64, 1, 64)])
def test_attention_with_own_rows(torch, D, lens, G, Hq, Hkv, page):
    _run(torch, G + D, lens, G, Hq, Hkv, D, page)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("new", [False, True])
@pytest.mark.parametrize("causal,window", [(True, 0), (True, 1), (True, 40), (False, 25), (False, 2), (True, 333)])
def test_attention_masks(torch, D, new, causal, window):
    # contexts shorter than the rows leave causal rows without a key (no own rows): they give zeros
    _run(torch, window, [0, 3, 16, 50, 345, 1030], 9, 6, 2, D, 16, causal=causal, window=window, new=new)


@pytest.mark.parametrize("G,Hq,Hkv", [(1, 8, 1), (16, 5, 1)])
def test_attention_split_over_a_long_context(torch, G, Hq, Hkv):
    _run(torch, 5, [9001], G, Hq, Hkv, 128, 64)
    _run(torch, 6, [9001, 0, 2500], G, Hq, Hkv, 64, 16, causal=True, window=3000)


def test_attention_large_scores_and_equal_bits(torch):
    """Scores of hundreds (one key takes everything) stay finite; repeated calls give the same bits."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(3)
    cache, table, ctx, K, V = _cached(torch, d, rng, [5000, 4097], 2, 128, 64)
    q = _dev(torch, 30 * rng.normal(size=(2, 4, 4, 128)))
    a = d.dflash2_kv4_attention(q, cache, table, ctx, 64, 1.0)
    assert torch.isfinite(a.float()).all()
    for _ in range(3):
        assert torch.equal(a, d.dflash2_kv4_attention(q, cache, table, ctx, 64, 1.0))
    assert d.dflash2_poll_error() == 0


def test_attention_in_a_graph_and_on_another_stream(torch):
    """Lengths and pages are read when the call runs: a captured call follows them."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(4)
    cache, table, ctx, K, V = _cached(torch, d, rng, [3000, 100], 2, 64, 32)
    q = _dev(torch, rng.normal(size=(2, 1, 8, 64)))
    out = torch.empty_like(q)
    ws = torch.empty(max(256, d.dflash2_kv4_attention_workspace_bytes(2, 1, 8, 2, 64, 32, table.shape[1])),
                     dtype=torch.uint8, device="cuda")
    call = lambda: d.dflash2_kv4_attention(q, cache, table, ctx, 32, 0.125, out=out, workspace=ws)
    call()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for lens in ([3000, 100], [17, 0], [2048, 99]):
        ctx.copy_(torch.tensor(lens, dtype=torch.int32))
        want = d.dflash2_kv4_attention(q, cache, table, ctx, 32, 0.125)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, want)
    with torch.cuda.stream(side):
        other = d.dflash2_kv4_attention(q, cache, table, ctx, 32, 0.125)
    side.synchronize()
    assert torch.equal(other, want)
    assert d.dflash2_poll_error() == 0


def test_attention_bad_pages_and_lengths_are_recorded(torch):
    """A page outside the cache hides its tokens; a length outside the table's range is clamped."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(8)
    cache, table, ctx, K, V = _cached(torch, d, rng, [64], 1, 64, 16)
    q = _rows(rng, 1, 1, 2, 64)
    for bad in (-1, 10 ** 6):
        t = table.clone()
        t[0, 1] = bad
        got = _host(d.dflash2_kv4_attention(_dev(torch, q), cache, t, ctx, 16, 0.125))
        assert d.dflash2_poll_error() == -6
        see = np.ones((1, 64), bool)
        see[:, 16:32] = False
        _check(got[0], *S.attention(q[0], K[0], V[0], see, 0.125), "one page missing")
    full = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, 16, 0.125)
    over = d.dflash2_kv4_attention(_dev(torch, q), cache, table, torch.tensor([65], dtype=torch.int32, device="cuda"),
                                   16, 0.125)
    assert d.dflash2_poll_error() == -1 and torch.equal(full, over)
    under = d.dflash2_kv4_attention(_dev(torch, q), cache, table, torch.tensor([-3], dtype=torch.int32, device="cuda"),
                                    16, 0.125)
    assert d.dflash2_poll_error() == -1 and not under.any()
    # pages that a window has left behind may be gone
    t = table.clone()
    t[0, :2] = -1
    got = _host(d.dflash2_kv4_attention(_dev(torch, q), cache, t, ctx, 16, 0.125, window=30))
    assert d.dflash2_poll_error() == 0
    _check(got[0], *S.attention(q[0], K[0], V[0], S.seen(1, 64, 0, False, 30), 0.125), "window past freed pages")


def test_cache_offsets_past_32_bits(torch):
    """A cache of more than 4 GiB: its last pages are reached."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(9)
    page, heads, D = 4096, 8, 128
    pages = (5 << 30) // d.dflash2_kv4_page_bytes(heads, D, page)
    cache = d.dflash2_kv4_cache(pages, heads, D, page)
    n = 70
    k, v = _rows(rng, n, heads, D), _rows(rng, n, heads, D)
    slots = torch.arange(pages * page - page, pages * page - page + n, device="cuda")
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), slots, cache, page)
    kr, _ = d.dflash2_kv4_read(cache, slots, D, page)
    np.testing.assert_array_equal(_host(kr), S.bf16(S.kv4_values(k)))
    q = _rows(rng, 1, 1, heads, D)
    got = d.dflash2_kv4_attention(_dev(torch, q), cache, torch.tensor([[pages - 1]], dtype=torch.int32, device="cuda"),
                                  torch.tensor([n], dtype=torch.int32, device="cuda"), page, D ** -0.5)
    assert d.dflash2_poll_error() == 0
    _check(_host(got)[0], *S.attention(q[0], S.kv4_values(k), S.kv4_values(v), np.ones((1, n), bool), D ** -0.5), "far page")
