"""Rounds of tree decoding with the operators one after the other: pages for what was kept, its rows into the cache, attention
of the next trees, their candidates. Each step against its statement, over what the whole run so far has made."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import S, _check, _dev, _host, _rows, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

B, G, HQ, HKV, D, V, PAGE, PAGES, WIDTH, LONG = 4, 12, 8, 2, 64, 10, 16, 23, 9, 144


class _Run:
    """Static buffers, so that a round can be captured."""

    def __init__(self, torch, rng):
        from dflash2_block_drafter_gb300 import dflash2_kv4_attention_workspace_bytes, dflash2_kv4_cache
        from dflash2_block_drafter_gb300.layer import ContextPages
        i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")
        self.torch, self.pages, self.cache = torch, ContextPages(B, PAGES, WIDTH, PAGE), dflash2_kv4_cache(PAGES, HKV, D, PAGE)
        # of each sequence, position and token (all different, so that roundings are independent)
        self.rows = {n: _rows(rng, B, LONG, V, h, D).reshape(B, LONG, V, h, D) for n, h in (("q", HQ), ("k", HKV), ("v", HKV))}
        self.table = {n: _dev(torch, x) for n, x in self.rows.items()}
        self.w = _dev(torch, rng.standard_normal((HQ * D, V)))
        self.change, self.place = i32(B), i32(B, G)
        self.kept, self.tokens, self.parents, self.depth = (i32(B, G) for _ in range(4))
        self.sequence = torch.arange(B, device="cuda")[:, None]
        self.history, self.prompt, self.length = i32(B, LONG), i32(B), i32(B)
        self.penalty = torch.tensor([1.0, 1.3, 2.0, 0.9], device="cuda")
        self.presence = torch.tensor([0.0, 0.5, 0.0, 0.1], device="cuda")
        self.attn_ws = torch.empty(dflash2_kv4_attention_workspace_bytes(B, G, HQ, HKV, D, PAGE, WIDTH), dtype=torch.uint8,
                                   device="cuda")

    def rows_of(self, name, position, token):
        return self.table[name][self.sequence, position.long().clamp(0, LONG - 1), token.long()]

    def round(self):
        import dflash2_block_drafter_gb300 as d
        slots, self.positions = self.pages.gain(self.change, place=self.place)
        self.slots, at = slots, self.pages.lengths[:, None] + self.depth
        d.dflash2_kv4_append(*(self.rows_of(n, self.positions, self.kept).flatten(0, 1) for n in "kv"), slots.flatten(), self.cache,
                             PAGE)
        q, k, v = (self.rows_of(n, at, self.tokens) for n in "qkv")
        self.out = d.dflash2_kv4_attention_tree(q, self.cache, self.pages.table, self.pages.lengths, PAGE, D ** -0.5, k, v,
                                                self.parents, workspace=self.attn_ws)
        self.logits = (self.out.view(B * G, HQ * D).float() @ self.w.float()).to(self.torch.bfloat16)
        self.best, self.value, _ = d.dflash2_logits_topk(
            self.logits, 1, requests=B, history=self.history, prompt_len=self.prompt, history_len=self.length,
            repetition=self.penalty, presence=self.presence, tokens=self.tokens.view(-1), parents=self.parents.view(-1))


def _draft(rng, root):
    """A tree below a token: (tokens, parents), a row's children all different."""
    tokens, parents, used = [root], [-1], {}
    while len(tokens) < G:
        p = int(rng.integers(0, len(tokens)))
        free = [t for t in range(V) if t not in used.setdefault(p, set())]
        t = int(rng.choice(free))
        used[p].add(t)
        tokens.append(t)
        parents.append(p)
    return tokens, parents


def _rounds(torch, captured):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(11)
    run = _Run(torch, rng)
    # what the run has made, in plain form: each sequence's tokens, and those in the cache (all but its last, in the end)
    history = [list(rng.integers(0, V, n)) for n in (30, 1, 17, 5)]
    prompt, cached, path = [len(h) for h in history], [[] for _ in range(B)], [None] * B
    state = dict(ctx=np.zeros(B, int), table=np.full((B, WIDTH), -1), queue=np.arange(PAGES), state=(0, PAGES))
    outs, graph, accepted = [], None, 0
    for r in range(14):
        change, place, kept = np.zeros(B, int), np.full((B, G), -1), np.zeros((B, G), int)
        for b in range(B):
            if r == 9 and b == 2:  # done: its pages go back, and a new sequence takes its place
                change[b], cached[b], history[b], prompt[b], path[b] = -state["ctx"][b], [], [3, 1], 2, None
                continue
            if path[b] is None:    # the prompt, G tokens at a time
                new = history[b][len(cached[b]):-1][:G]
                rows = list(range(len(new)))
                kept[b, rows] = new
            else:                  # what was kept of the tree before
                rows, kept[b] = path[b], tokens[b]
            place[b, rows] = np.arange(len(rows))
            change[b] = len(rows)
            cached[b] = cached[b] + [int(t) for t in kept[b, rows]]
        want = T.plan(state["ctx"], change, state["table"], state["queue"], state["state"], PAGE, PAGES, place=place)
        assert not want["bad"] and [len(c) for c in cached] == list(want["ctx"])
        state = {k: want[k] for k in state}
        drafts = [_draft(rng, int(h[-1])) for h in history]
        tokens, parents = np.array([x[0] for x in drafts]), np.array([x[1] for x in drafts])
        hist = np.zeros((B, LONG), int)
        for b in range(B):
            hist[b, :len(history[b])] = history[b]
            if len(cached[b]) + 1 < len(history[b]):  # (a tree needs its sequence's whole context)
                parents[b] = -2
        depth = np.array([[max(0, len(x) - 1) for x in T.lines(p)] for p in parents])
        for t, x in ((run.depth, depth), (run.change, change), (run.place, place), (run.kept, kept), (run.tokens, tokens), (run.parents, parents),
                     (run.history, hist), (run.prompt, prompt), (run.length, [len(h) - 1 for h in history])):
            t.copy_(torch.from_numpy(np.asarray(x, np.int32)))
        if captured and r > 0:
            if graph is None:
                graph = torch.cuda.CUDAGraph()
                with torch.cuda.graph(graph):
                    run.round()
            graph.replay()
        else:
            run.round()
        assert d.dflash2_poll_error() == 0
        for name, x in (("ctx", run.pages.lengths), ("slots", run.slots), ("positions", run.positions), ("table", run.pages.table),
                        ("queue", run.pages.free), ("state", run.pages.state)):
            np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=f"{name}, round {r}")
        out, logits = _host(run.out), run.logits.float().cpu().numpy().reshape(B, G, V)
        best = run.best.cpu().numpy().reshape(B, G)
        for b in range(B):
            old, lines = np.array(cached[b], int), T.lines(parents[b])
            at = len(old) + depth[b]
            k, v = ([S.kv4_values(run.rows[n][b, np.arange(len(old)), old])] if len(old) else [] for n in "kv")
            q, kn, vn = (run.rows[n][b, at, tokens[b]] for n in "qkv")
            o, sd = S.attention(q, np.concatenate(k + [kn]), np.concatenate(v + [vn]), T.tree_seen(parents[b], len(old)),
                                D ** -0.5)
            _check(out[b], o, sd, f"round {r}, sequence {b}")
            before = history[b][:-1]
            for t in range(G):
                if not lines[t]:
                    assert best[b, t] == -1 and not out[b, t].any()
                    continue
                counts, in_prompt = np.zeros(V, int), np.zeros(V, bool)
                in_prompt[before[:prompt[b]]] = True
                np.add.at(counts, np.array(before[prompt[b]:], int), 1)
                np.add.at(counts, tokens[b][lines[t]], 1)
                y = T.adjust(logits[b, t], counts, in_prompt, float(run.penalty[b]), 0.0, float(run.presence[b]))
                assert best[b, t] == T.best(y, 1)[0]
            path[b] = None
            if lines[0]:  # from the root down, as long as a child is what its parent's row says
                path[b] = [0]
                while True:
                    below = [t for t in range(G) if parents[b, t] == path[b][-1] and tokens[b, t] == best[b, path[b][-1]]]
                    if not below:
                        break
                    path[b].append(below[0])
                history[b] = history[b] + [int(tokens[b][t]) for t in path[b][1:]] + [int(best[b, path[b][-1]])]
                accepted += len(path[b]) - 1
        outs.append((run.out.clone(), run.best.clone(), run.value.clone()))
    return outs, accepted


def test_rounds_of_tree_decoding(torch):
    eager, accepted = _rounds(torch, False)
    replayed, _ = _rounds(torch, True)
    assert accepted > 0
    for r, (a, b) in enumerate(zip(eager, replayed)):
        for x, y in zip(a, b):
            assert torch.equal(x, y), f"round {r}: a replayed round differs from an eager one"
