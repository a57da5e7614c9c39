"""Attention over the 4-bit cache with scores and values far from one another: one call, float64 statements."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import S, _cached, _check, _dev, _host, _rows, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _fill(torch, d, k, v, page):
    """A cache of one sequence's rows k, v [n, heads, D] in pages in order: (cache, table, ctx)."""
    n, heads, D = k.shape
    pages = max(1, -(-n // page))
    cache = d.dflash2_kv4_cache(pages, heads, D, page)
    cache.fill_(255)
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), torch.arange(n, device="cuda"), cache, page)
    return (cache, torch.arange(pages, dtype=torch.int32, device="cuda")[None],
            torch.tensor([n], dtype=torch.int32, device="cuda"))


@pytest.mark.parametrize("qm,km,scale", [(1e3, 1e3, 0.125), (1e4, 1e4, 0.125), (1e6, 1e2, 1.0), (1e8, 1e8, 0.125),
                                         (1e15, 1e15, 0.1), (1.0, 1.0, 3e7), (1e-3, 1.0, 1e12)])
@pytest.mark.parametrize("G,Hq,first", [(1, 2, 3), (2, 4, 600), (10, 8, 1299), (16, 5, 700)])
def test_large_finite_scores(torch, qm, km, scale, G, Hq, first):
    """Scores up to 2^110 (an fp32 product near 2^28 is rounded by more than the slack that scores have over their
    row's reference). One key stands out by a factor of two for rows of either sign, so that it takes everything."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(first + G)
    n, D, page = 1300, 64, 32
    u = rng.choice([-1.0, 1.0], D)
    size = rng.uniform(0.5, 0.9, (n, 1, 1))
    size[first], size[(first + n // 2) % n] = 2.0, -2.0
    k, v = S.bf16(km * size * u), _rows(rng, n, 1, D)
    q = S.bf16(qm * rng.choice([-1.0, 1.0], (1, G, Hq, 1)) * rng.uniform(1.0, 2.0, (1, G, Hq, 1)) * u)
    cache, table, ctx = _fill(torch, d, k, v, page)
    out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, scale)
    assert d.dflash2_poll_error() == 0
    want, sd = S.attention(q[0], S.kv4_values(k), S.kv4_values(v), np.ones((G, n), bool), scale)
    # everything is one key's value: only its operand's and the result's roundings count
    assert np.all(np.abs(_host(out)[0] - want) <= 2 ** -7 * np.abs(want) + 1e-5)


def test_large_random_scores(torch):
    """Scores of hundreds of millions with no key far ahead: finite, within the values' range, the same bits again."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(12)
    cache, table, ctx, K, V = _cached(torch, d, rng, [3000, 129, 1], 2, 128, 64)
    for size in (3e6, 1e9):
        q = _dev(torch, size * rng.normal(size=(3, 5, 8, 128)))
        a = d.dflash2_kv4_attention(q, cache, table, ctx, 64, 1.0)
        assert d.dflash2_poll_error() == 0
        top = max(np.abs(v).max() for v in V)
        assert torch.isfinite(a.float()).all() and float(a.abs().max()) <= top * (1 + 2 ** -6) and bool(a.any(-1).all())
        assert torch.equal(a, d.dflash2_kv4_attention(q, cache, table, ctx, 64, 1.0))


@pytest.mark.parametrize("new", [False, True])
@pytest.mark.parametrize("causal", [False, True])
@pytest.mark.parametrize("window", [2 ** 31 - 1, 2 ** 31 - 60, 2 ** 31, 2 ** 40])
def test_windows_that_leave_nothing_out(torch, new, causal, window):
    """Also where rows stand before the first key (contexts shorter than the rows, no own rows)."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(21)
    lens, G, Hq, Hkv, D, page = [0, 2, 3, 5, 150, 1], 9, 4, 2, 64, 16
    cache, table, ctx, K, V = _cached(torch, d, rng, lens, Hkv, D, page)
    q = _dev(torch, _rows(rng, len(lens), G, Hq, D))
    kw = dict(causal=causal)
    if new:
        kw.update(k_new=_dev(torch, _rows(rng, len(lens), G, Hkv, D)), v_new=_dev(torch, _rows(rng, len(lens), G, Hkv, D)))
    want = d.dflash2_kv4_attention(q, cache, table, ctx, page, 0.125, **kw)
    got = d.dflash2_kv4_attention(q, cache, table, ctx, page, 0.125, window=window, **kw)
    assert d.dflash2_poll_error() == 0 and torch.equal(got, want)
    assert bool(want[1].any()) and bool(want[2].any())


def _check_rows(got, want, sd, unit, what):
    """Row by row (rows differ in size): `unit` is what 1 stands for in the row's absolute allowance."""
    for t in np.ndindex(got.shape[:2]):
        _check(got[t] / unit[t], want[t] / unit[t], sd[t] / unit[t], f"{what} row {t}")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("e", [12, 16, 24, 60])
def test_one_value_row_far_larger(torch, D, e):
    """A value row 2^e above the rest is felt by the rows that give it weight, and by no other: rows to which causal
    order or the window hides it, and rows whose score for it is far below, give what the rest gives."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(e)
    n, G, R, page = 300, 4, 3, 16
    for place in ("own row", "window's edge", "low score"):
        k, v = _rows(rng, n, 1, D), _rows(rng, n, 1, D)
        kn, vn = _rows(rng, 1, G, 1, D), _rows(rng, 1, G, 1, D)
        q = _rows(rng, 1, G, R, D)
        causal, window = place == "own row", 50 if place == "window's edge" else 0
        if place == "own row":
            vn[0, 2] *= 2.0 ** e
        elif place == "window's edge":
            v[n - window + 1] *= 2.0 ** e  # (the last key of row 0 and of no other; own rows follow at n)
        else:
            q = np.abs(q)
            k[40], v[40] = -30.0, v[40] * 2.0 ** e
        cache, table, ctx = _fill(torch, d, k, v, page)
        out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, D ** -0.5, k_new=_dev(torch, kn),
                                      v_new=_dev(torch, vn), causal=causal, window=window)
        assert d.dflash2_poll_error() == 0
        K, V = np.concatenate([S.kv4_values(k), kn[0]]), np.concatenate([S.kv4_values(v), vn[0]])
        want, sd = S.attention(q[0], K, V, S.seen(G, n, G, causal, window), D ** -0.5)
        unit = np.maximum(1.0, np.abs(want).max(-1))
        _check_rows(_host(out)[0], want, sd, unit, f"{place} 2^{e}")


@pytest.mark.parametrize("D", [64, 128])
def test_value_rows_of_every_size(torch, D):
    """Value rows from 2^-60 to 2^60, in an order that meets the largest late, over many tiles and parts."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(D)
    n, G, R, page = 5000, 2, 2, 64
    k, v = _rows(rng, n, 1, D), _rows(rng, n, 1, D) * 2.0 ** np.round(np.linspace(-60, 60, n))[:, None, None]
    q = _rows(rng, 1, G, R, D)
    cache, table, ctx = _fill(torch, d, k, v, page)
    out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, D ** -0.5)
    assert d.dflash2_poll_error() == 0
    want, sd = S.attention(q[0], S.kv4_values(k), S.kv4_values(v), np.ones((G, n), bool), D ** -0.5)
    _check_rows(_host(out)[0], want, sd, np.abs(want).max(-1), "sizes")


@pytest.mark.parametrize("sink", [0.0, 2.0 ** -8, 1.0])
@pytest.mark.parametrize("gap", [8.0, 14.0])
def test_a_key_that_takes_nearly_everything(torch, gap, sink):
    """The first key's score stands `gap` above the rest; its value is small. What is left of the output is the
    rest's, each of them a small probability."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(int(gap))
    n, D, page, G, R = 6000, 64, 64, 1, 4
    k, v = 0.02 * _rows(rng, n, 1, D), _rows(rng, n, 1, D) + 1.0
    q = np.ones((1, G, R, D))
    k[0], v[0] = gap / 8.0, v[0] * sink
    k, v = S.bf16(k), S.bf16(v)
    cache, table, ctx = _fill(torch, d, k, v, page)
    out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, 0.125)
    assert d.dflash2_poll_error() == 0
    want, sd = S.attention(q[0], S.kv4_values(k), S.kv4_values(v), np.ones((G, n), bool), 0.125)
    _check_rows(_host(out)[0], want, sd, np.abs(want).max(-1), f"gap {gap}")


def _sizes_case(torch, d, rng, n, G, R, D, page, causal=False, window=0):
    k, v = _rows(rng, n, 1, D), _rows(rng, n, 1, D)
    kn, vn, q = _rows(rng, 1, G, 1, D), _rows(rng, 1, G, 1, D), _rows(rng, 1, G, R, D)
    return k, v, kn, vn, q, S.seen(G, n, G, causal, window)


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
@pytest.mark.parametrize("what", ["own key", "own value", "cached"])
@pytest.mark.parametrize("n,G,R", [(300, 4, 2), (5000, 16, 5), (40, 1, 1)])
def test_keys_and_values_that_are_not_finite(torch, D, bad, what, n, G, R):
    """They give NaN to the rows that see them, and nothing to the others (hidden by causal order, or by the window)."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(n + D)
    window = 30 if what == "cached" else 0
    causal = True
    k, v, kn, vn, q, see = _sizes_case(torch, d, rng, n, G, R, D, 16, causal, window)
    cache, table, ctx = _fill(torch, d, k, v, 16)
    if what == "cached":  # (its parameters, in one granule, of the first key that row 0's window holds)
        at = n - window + 1
        par = cache[at // 16, 0, :, at % 16 // 16, 16 * D // 2:].reshape(2, 16, -1)
        par[:, at % 16] = torch.tensor([0xC0, 0x7F] if np.isnan(bad) else [0x80, 0x7F], dtype=torch.uint8).repeat(
            D // 32).cuda()
        cache[at // 16, 0, :, 0, 16 * D // 2:] = par.reshape(2, -1)
        sees = see[:, at]
    else:
        (kn if what == "own key" else vn)[0, G // 2, 0, 7] = bad
        if what == "own key":
            q[..., 7] = np.abs(q[..., 7]) + 0.5  # (an infinite score above, not below)
        sees = see[:, n + G // 2]
    out = _host(d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, 16, D ** -0.5, k_new=_dev(torch, kn),
                                        v_new=_dev(torch, vn), causal=causal, window=window))[0]
    assert d.dflash2_poll_error() == 0
    assert sees.any() and np.isnan(out[sees]).all()
    see = see & ~sees[:, None]
    fine = lambda x: np.where(np.isfinite(x), x, 0.0)
    want, sd = S.attention(q[0], np.concatenate([S.kv4_values(k), fine(kn[0])]),
                           np.concatenate([S.kv4_values(v), fine(vn[0])]), see, D ** -0.5)
    if not sees.all():
        _check(out[~sees], want[~sees], sd[~sees], "rows that do not see it")


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf"), 1e30, 2.0 ** -100])
def test_one_query_row_unlike_the_others(torch, D, bad):
    """A query row that is not finite gives NaN, one of another size what it should, and neither touches the rest."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(5)
    for n, G, R in ((300, 3, 2), (4000, 16, 5), (0, 2, 1)):
        k, v, kn, vn, q, see = _sizes_case(torch, d, rng, n, G, R, D, 16)
        at = (0, G - 1, R - 1)
        q[at] = S.bf16(q[at] * bad) if np.isfinite(bad) else q[at]
        if not np.isfinite(bad):
            q[at][1] = bad
        cache, table, ctx = _fill(torch, d, k if n else _rows(rng, 1, 1, D), v if n else _rows(rng, 1, 1, D), 16)
        if n == 0:
            ctx.zero_()
        out = _host(d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, 16, D ** -0.5, k_new=_dev(torch, kn),
                                            v_new=_dev(torch, vn)))[0]
        assert d.dflash2_poll_error() == 0
        K, V = np.concatenate([S.kv4_values(k), kn[0]]), np.concatenate([S.kv4_values(v), vn[0]])
        mask = np.ones((G, R), bool)
        if abs(bad) != 2.0 ** -100:
            mask[at[1:]] = False
            got = out[at[1:]]
            assert np.isfinite(got).all() if np.isfinite(bad) else np.isnan(got).all()
        q[at] = q[at] if np.isfinite(bad) else 0.0
        want, sd = S.attention(q[0], K, V, see, D ** -0.5)
        _check(out[mask], want[mask], sd[mask], f"rows beside {bad}")


@pytest.mark.parametrize("n", [0, 100, 5000])
def test_query_rows_of_every_size(torch, n):
    """Rows from 2^-30 to 2^30 over keys of 2^28: the small rows' scores are moderate, the large rows take one key."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(n)
    G, R, D = 8, 2, 64
    k, v, kn, vn, q, see = _sizes_case(torch, d, rng, max(n, 1), G, R, D, 16)
    size = 2.0 ** np.array([-30, -28, -26, -40, 30, -27, -29, 10])
    q *= size[None, :, None, None]
    k, kn = k * 2.0 ** 28, kn * 2.0 ** 28
    cache, table, ctx = _fill(torch, d, k, v, 16)
    ctx.fill_(n)
    out = _host(d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, 16, D ** -0.5, k_new=_dev(torch, kn),
                                        v_new=_dev(torch, vn)))[0]
    assert d.dflash2_poll_error() == 0
    K, V = np.concatenate([S.kv4_values(k)[:n], kn[0]]), np.concatenate([S.kv4_values(v)[:n], vn[0]])
    want, sd = S.attention(q[0], K, V, np.ones((G, n + G), bool), D ** -0.5)
    small = size < 2.0 ** -20
    _check(out[small], want[small], sd[small], "small rows")
    assert np.isfinite(out).all()


@pytest.mark.parametrize("D", [64, 128])
def test_own_rows_with_strong_channels(torch, D):
    """Own rows whose channels differ by 2^8 to 2^12 keep the small ones to 11 significant bits, as the bound's."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(D + 1)
    G, R, page = 16, 2, 16
    for e in (8, 12):
        kn, vn, q = _rows(rng, 1, G, 1, D), _rows(rng, 1, G, 1, D), _rows(rng, 1, G, R, D)
        vn[..., 3] *= 2.0 ** e
        kn[..., 5] *= 2.0 ** e
        q[..., 5] = 0.0
        cache, table, _ = _fill(torch, d, _rows(rng, 1, 1, D), _rows(rng, 1, 1, D), page)
        ctx = torch.zeros(1, dtype=torch.int32, device="cuda")
        out = d.dflash2_kv4_attention(_dev(torch, q), cache, table, ctx, page, D ** -0.5, k_new=_dev(torch, kn),
                                      v_new=_dev(torch, vn))
        assert d.dflash2_poll_error() == 0
        want, _ = S.attention(q[0], kn[0], vn[0], np.ones((G, G), bool), D ** -0.5)
        # the channels apart from the strong one: bf16's half step of the result; 2^-11 of the weighted values for each
        # of the probability's, the value's and (through a score below 2 in size) the key's rounding
        big = np.abs(vn[0, :, 0]).copy()
        big[:, 3] = 0
        keep = np.arange(D) != 3
        err = np.abs(_host(out)[0] - want)[..., keep]
        assert np.all(err <= 2.0 ** -8 * np.abs(want[..., keep]) + 4 * 2.0 ** -11 * big.max()), e
