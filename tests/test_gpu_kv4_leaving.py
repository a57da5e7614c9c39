"""GPU: attention over the 4-bit cache launched back to back, so that a CTA's shared and tensor memory serve the next launch's
CTA as soon as it has left. Every launch gives the first one's bits."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import S, _cached, _check, _dev, _host, _rows, torch  # noqa: F401 (fixture)
from tests.test_gpu_kv4_tree import _tree

pytestmark = pytest.mark.gpu

LAUNCHES, REPLAYS = 40, 25


def _repeat(torch, call, out):
    """LAUNCHES a graph, REPLAYS of it: each launch against the first one's result."""
    import dflash2_block_drafter_gb300 as d
    call(out[0])
    first = out[0].clone()
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        for i in range(LAUNCHES):
            call(out[i % len(out)])
    for r in range(REPLAYS):
        out.fill_(float("nan"))
        graph.replay()
        torch.cuda.synchronize()
        for o in out:
            assert torch.equal(o, first), f"replay {r}"
    assert d.dflash2_poll_error() == 0


def _inputs(torch, rng, lens, G, Hq, Hkv, D, page):
    import dflash2_block_drafter_gb300 as d
    B = len(lens)
    cache, table, ctx, _, _ = _cached(torch, d, rng, lens, Hkv, D, page)
    q, k, v = (_dev(torch, _rows(rng, B, G, h, D)) for h in (Hq, Hkv, Hkv))
    out = torch.empty((8, B, G, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(max(1, d.dflash2_kv4_attention_workspace_bytes(B, G, Hq, Hkv, D, page, table.shape[1])),
                     dtype=torch.uint8, device="cuda")
    return cache, table, ctx, q, k, v, out, ws


# ranges of one, two, three and more tiles; 16, 32, 64 and 80 rows a CTA; several items a CTA, and items cut into parts
@pytest.mark.parametrize("lens,G,Hq,Hkv,D", [([0], 4, 2, 2, 64), ([100] * 3, 4, 8, 2, 128), ([200], 40, 1, 1, 64),
                                             ([129, 300, 0], 16, 10, 2, 128), ([4000], 1, 16, 2, 128),
                                             ([700] * 40, 16, 20, 4, 128), ([9000], 64, 5, 1, 64)])
def test_blocks_and_trees_behind_one_another(torch, lens, G, Hq, Hkv, D):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(len(lens) + G)
    cache, table, ctx, q, k, v, out, ws = _inputs(torch, rng, lens, G, Hq, Hkv, D, 32)
    _repeat(torch, lambda o: d.dflash2_kv4_attention(q, cache, table, ctx, 32, D ** -0.5, k_new=k, v_new=v, causal=True, out=o,
                                                     workspace=ws), out)
    parents = torch.tensor(np.stack([_tree(rng, G, "any") for _ in lens]), dtype=torch.int32, device="cuda")
    _repeat(torch, lambda o: d.dflash2_kv4_attention_tree(q, cache, table, ctx, 32, D ** -0.5, k, v, parents, out=o,
                                                          workspace=ws), out)


@pytest.mark.parametrize("G,Hq,D", [(4, 4, 64), (16, 10, 128), (64, 6, 128)])
def test_references_raised_in_every_tile(torch, G, Hq, D):
    """Scores that grow by 12 powers of two a tile: the warps leave their common path for the raise, and wait for the last
    product, in each of a range's several tiles. (40 sequences over the same pages.)"""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(G)
    B, Hkv, n, page = 40, 2, 1500, 64
    k, v, q = _rows(rng, n, Hkv, D), _rows(rng, n, Hkv, D), _rows(rng, B, G, Hq, D)
    k[:, :, 0] = S.bf16(np.arange(n) // 128 * 12.0 * np.log(2.0))[:, None]
    q[..., 0] = S.bf16(D ** 0.5)
    kn, vn = _rows(rng, B, G, Hkv, D), _rows(rng, B, G, Hkv, D)
    cache = d.dflash2_kv4_cache(-(-n // page), Hkv, D, page)
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), torch.arange(n, device="cuda"), cache, page)
    table = torch.arange(cache.shape[0], dtype=torch.int32, device="cuda").repeat(B, 1)
    ctx = torch.full((B,), n, dtype=torch.int32, device="cuda")
    parents = np.stack([_tree(rng, G, "any") for _ in range(B)])
    args = [_dev(torch, q), cache, table, ctx, page, D ** -0.5, _dev(torch, kn), _dev(torch, vn),
            torch.tensor(parents, dtype=torch.int32, device="cuda")]
    out = torch.empty((8, B, G, Hq, D), dtype=torch.bfloat16, device="cuda")
    ws = torch.empty(d.dflash2_kv4_attention_workspace_bytes(B, G, Hq, Hkv, D, page, table.shape[1]), dtype=torch.uint8,
                     device="cuda")
    _repeat(torch, lambda o: d.dflash2_kv4_attention_tree(*args, out=o, workspace=ws), out)
    K, V = S.kv4_values(k), S.kv4_values(v)
    for b in (0, 17, B - 1):
        want, sd = S.attention(q[b], np.concatenate([K, kn[b]]), np.concatenate([V, vn[b]]), T.tree_seen(parents[b], n), D ** -0.5)
        _check(_host(out[0])[b], want, sd, f"G={G}, sequence {b}")


def test_two_graphs_of_one_workspace_in_turn(torch):
    """A graph of blocks and one of trees, cut into other parts, replayed one after the other over the same workspace."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(1)
    made = []
    for lens, G, Hq, Hkv, D in (([5000, 40], 16, 10, 2, 128), ([3000] * 3, 40, 4, 1, 64)):
        cache, table, ctx, q, k, v, out, _ = _inputs(torch, rng, lens, G, Hq, Hkv, D, 32)
        parents = torch.tensor(np.stack([_tree(rng, G, "any") for _ in lens]), dtype=torch.int32, device="cuda")
        size = d.dflash2_kv4_attention_workspace_bytes(len(lens), G, Hq, Hkv, D, 32, table.shape[1])
        made.append((cache, table, ctx, q, k, v, out[0], parents, D, size))
    ws = torch.empty(max(m[-1] for m in made), dtype=torch.uint8, device="cuda")
    block, tree = made
    calls = [lambda: d.dflash2_kv4_attention(block[3], *block[:3], 32, block[8] ** -0.5, k_new=block[4], v_new=block[5],
                                             out=block[6], workspace=ws),
             lambda: d.dflash2_kv4_attention_tree(tree[3], *tree[:3], 32, tree[8] ** -0.5, tree[4], tree[5], tree[7], out=tree[6],
                                                  workspace=ws)]
    first, graphs = [], []
    for call, m in zip(calls, made):
        call()
        torch.cuda.synchronize()
        first.append(m[6].clone())
        graphs.append(torch.cuda.CUDAGraph())
        with torch.cuda.graph(graphs[-1]):
            call()
    for r in range(200):
        for m in made:
            m[6].fill_(float("nan"))
        for g in graphs:
            g.replay()
        if r % 3 == 0:
            calls[r % 2]()  # and an eager call between
        torch.cuda.synchronize()
        for m, want in zip(made, first):
            assert torch.equal(m[6], want), f"round {r}"
    assert d.dflash2_poll_error() == 0
