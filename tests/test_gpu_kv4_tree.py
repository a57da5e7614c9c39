"""GPU parity of attention for trees of drafted tokens over the 4-bit cache, against float64."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import S, _cached, _check, _dev, _host, _rows, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _tree(rng, G, kind):
    if kind == "chain":
        return np.arange(G) - 1
    if kind == "roots":
        return np.full(G, -1)
    if kind == "wide":                       # every row below the first
        return np.where(np.arange(G) > 0, 0, -1)
    if kind == "small":                      # the last half is not there
        return np.where(np.arange(G) < (G + 1) // 2, np.maximum(-1, np.arange(G) // 2 - 1), -2)
    if kind == "none":
        return np.full(G, -3)
    return np.array([int(rng.integers(-1, t)) if t else -1 for t in range(G)])


def _call(torch, d, rng, lens, G, Hq, Hkv, D, page, parents, window, scale=None, spoil=True):
    """(result, inputs): own rows that are not there hold NaN where `spoil`."""
    B = len(lens)
    cache, table, ctx, K, V = _cached(torch, d, rng, lens, Hkv, D, page)
    q, kn, vn = _rows(rng, B, G, Hq, D), _rows(rng, B, G, Hkv, D), _rows(rng, B, G, Hkv, D)
    scale = D ** -0.5 if scale is None else scale
    there = np.array([[bool(x) for x in T.lines(p)] for p in parents])
    held = [np.where(there[:, :, None, None], x, np.nan) if spoil else x for x in (q, kn, vn)]
    fused = _dev(torch, np.concatenate([x.reshape(B, G, -1) for x in held], -1))
    nq, nk = Hq * D, Hkv * D
    args = (fused[..., :nq].unflatten(-1, (Hq, D)), cache, table, ctx, page, scale,
            fused[..., nq:nq + nk].unflatten(-1, (Hkv, D)), fused[..., nq + nk:].unflatten(-1, (Hkv, D)),
            torch.tensor(parents, dtype=torch.int32, device="cuda"))
    out = d.dflash2_kv4_attention_tree(*args, window=window)
    want, sd = np.zeros(q.shape), np.zeros(q.shape)
    for b, n in enumerate(lens):
        want[b], sd[b] = S.attention(q[b], np.concatenate([K[b], kn[b]]), np.concatenate([V[b], vn[b]]),
                                     T.tree_seen(parents[b], n, window), scale)
    return out, want, sd, args


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("kind", ["chain", "roots", "wide", "small", "none", "any"])
@pytest.mark.parametrize("lens,G,Hq,Hkv,page", [([1], 1, 1, 1, 16), ([0], 2, 4, 2, 16), ([300, 0, 129], 13, 10, 2, 64),
                                                ([700, 64], 33, 3, 1, 32), ([513, 1], 64, 5, 1, 128), ([90], 64, 16, 2, 16)])
def test_trees(torch, D, kind, lens, G, Hq, Hkv, page):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(G + D)
    parents = np.stack([_tree(rng, G, kind) for _ in lens])
    out, want, sd, _ = _call(torch, d, rng, lens, G, Hq, Hkv, D, page, parents, 0)
    assert d.dflash2_poll_error() == 0
    _check(_host(out), want, sd, f"{kind} {lens} G={G}")
    assert not _host(out)[want == 0].any()


@pytest.mark.parametrize("window", [1, 2, 5, 40, 333])
def test_windows_follow_each_rows_position(torch, window):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(window)
    lens, G = [0, 3, 50, 345, 1030], 40
    parents = np.stack([_tree(rng, G, k) for k in ("chain", "any", "chain", "any", "small")])
    for D, Hq, Hkv in ((64, 6, 2), (128, 4, 4), (128, 5, 1)):
        out, want, sd, _ = _call(torch, d, rng, lens, G, Hq, Hkv, D, 16, parents, window)
        assert d.dflash2_poll_error() == 0
        _check(_host(out), want, sd, f"window {window} D={D}")


def test_a_chain_is_causal_attention(torch):
    """(Both within their roundings of the same numbers; how the work is cut, and so the order of sums, differs.)"""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(1)
    for lens, G, window in (([700, 20, 0], 16, 0), ([900, 5], 24, 100), ([3000], 64, 100)):
        parents = np.stack([_tree(rng, G, "chain") for _ in lens])
        out, want, sd, a = _call(torch, d, rng, lens, G, 8, 2, 128, 64, parents, window)
        same = d.dflash2_kv4_attention(*a[:6], k_new=a[6], v_new=a[7], causal=True, window=window)
        _check(_host(out), want, sd, "tree")
        _check(_host(same), want, sd, "causal")
    assert d.dflash2_poll_error() == 0


@pytest.mark.parametrize("D,G,Hq,Hkv", [(128, 20, 5, 1), (128, 64, 10, 2), (64, 64, 4, 1), (64, 33, 12, 1), (128, 64, 64, 1)])
def test_many_rows_a_key_head(torch, D, G, Hq, Hkv):
    """100 to 4096 rows a head: several tiles of rows; ragged contexts, absent rows, a window."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(Hq + D)
    lens = [0, 1, 127, 128, 129, 640, 2000]
    parents = np.stack([_tree(rng, G, "any" if b % 2 else "small") for b in range(len(lens))])
    for window in (0, 300):
        out, want, sd, a = _call(torch, d, rng, lens, G, Hq, Hkv, D, 32, parents, window)
        assert d.dflash2_poll_error() == 0
        _check(_host(out), want, sd, f"{G} x {Hq}/{Hkv} D={D} window {window}")
        assert not _host(out)[want == 0].any()
        for _ in range(3):
            assert torch.equal(out, d.dflash2_kv4_attention_tree(*a, window=window))


@pytest.mark.parametrize("G,scale", [(8, 0.1), (40, 0.1), (40, -0.2), (40, 0.0)])
def test_key_and_value_rows_of_very_different_sizes(torch, G, scale):
    """Cached rows that lie up to 2^40 apart inside a tile, zero rows, and scales of any sign: each value within its own
    rounding (the largest keys are made small enough not to decide everything)."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(7)
    n, Hq, Hkv, D, page = 700, 8, 2, 128, 64
    size = lambda lo, hi: np.exp2(rng.integers(lo, hi, (n, Hkv, 1)))
    k, v = S.bf16(_rows(rng, n, Hkv, D) * size(-20, 1)), S.bf16(_rows(rng, n, Hkv, D) * size(-20, 20))
    k[5], v[9], k[200:210] = 0, 0, 0
    cache = d.dflash2_kv4_cache(11, Hkv, D, page)
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), torch.arange(n, device="cuda"), cache, page)
    q, kn, vn = _rows(rng, 1, G, Hq, D), _rows(rng, 1, G, Hkv, D), _rows(rng, 1, G, Hkv, D)
    q = S.bf16(q * np.exp2(rng.integers(-3, 3, (1, G, Hq, 1))))
    parents = np.array([_tree(rng, G, "any")])
    out = d.dflash2_kv4_attention_tree(_dev(torch, q), cache, torch.arange(11, dtype=torch.int32, device="cuda")[None],
                                       torch.tensor([n], dtype=torch.int32, device="cuda"), page, scale, _dev(torch, kn),
                                       _dev(torch, vn), torch.tensor(parents, dtype=torch.int32, device="cuda"))
    assert d.dflash2_poll_error() == 0
    want, sd = S.attention(q[0], np.concatenate([S.kv4_values(k), kn[0]]), np.concatenate([S.kv4_values(v), vn[0]]),
                           T.tree_seen(parents[0], n), scale)
    unit = np.abs(want).max()
    _check(_host(out)[0] / unit, want / unit, sd / unit, f"G={G} scale {scale}")


def test_a_long_context_many_trees_and_large_scores(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(2)
    for lens, G, Hq, Hkv, scale in (([9001], 16, 10, 2, None), ([9001, 0, 2500], 48, 5, 1, None),
                                    ([int(n) for n in rng.integers(0, 400, 70)], 7, 4, 2, None), ([800, 33], 20, 4, 2, 3.0)):
        parents = np.stack([_tree(rng, G, "any" if b % 3 else "small") for b in range(len(lens))])
        out, want, sd, a = _call(torch, d, rng, lens, G, Hq, Hkv, 128, 64, parents, 0, scale)
        _check(_host(out), want, sd, f"{len(lens)} trees of {G}")
        for _ in range(3):
            assert torch.equal(out, d.dflash2_kv4_attention_tree(*a))
    assert d.dflash2_poll_error() == 0


def test_bad_parents_are_recorded_and_hide_what_is_below(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(3)
    for bad in ([0], [-1, 1], [-1, 0, 64, 2, 1], [-1, 2 ** 31 - 1, 1, 0], [5, 0, -1, 2]):
        out, want, sd, _ = _call(torch, d, rng, [40], len(bad), 2, 1, 64, 16, np.array([bad]), 0)
        assert d.dflash2_poll_error() == -6, bad
        _check(_host(out), want, sd, f"{bad}")
        assert not _host(out)[want == 0].any()


def test_what_is_not_finite_stays_with_the_rows_that_see_it(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(4)
    parents = np.array([[-1, 0, 0, 1, 2]])
    for i in (6, 7):  # a NaN in row 1's key, or value: rows 1 and 3 see it
        _, want, sd, a = _call(torch, d, rng, [50], 5, 4, 2, 64, 16, parents, 0)
        a = list(a)
        a[i] = a[i].clone()
        a[i][0, 1, :, 3] = float("nan")
        a[13 - i] = a[13 - i].clone()  # (the same strides)
        got = _host(d.dflash2_kv4_attention_tree(*a))[0]
        assert np.isnan(got[[1, 3]]).any(-1).all()
        _check(got[[0, 2, 4]], want[0, [0, 2, 4]], sd[0, [0, 2, 4]], "the others")
    assert d.dflash2_poll_error() == 0


def test_trees_in_a_graph_and_on_another_stream(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(5)
    lens, G = [900, 100], 24
    first, want, sd, a = _call(torch, d, rng, lens, G, 8, 2, 128, 32, np.stack([_tree(rng, G, "any")] * 2), 0, spoil=False)
    out = torch.empty_like(first)
    ws = torch.empty(d.dflash2_kv4_attention_workspace_bytes(2, G, 8, 2, 128, 32, a[2].shape[1]), dtype=torch.uint8,
                     device="cuda")
    call = lambda: d.dflash2_kv4_attention_tree(*a, out=out, workspace=ws)
    call()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        call()
    for kind in ("chain", "small", "any", "none"):
        a[8].copy_(torch.tensor(np.stack([_tree(rng, G, kind)] * 2), dtype=torch.int32))
        fresh = d.dflash2_kv4_attention_tree(*a)
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(out, fresh)
        side.wait_stream(torch.cuda.current_stream())
        other = d.dflash2_kv4_attention_tree(*a, stream=side)
        side.synchronize()
        assert torch.equal(other, fresh)
    assert d.dflash2_poll_error() == 0
