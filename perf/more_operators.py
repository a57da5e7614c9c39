"""The operators of a step that drafts and verifies trees of tokens, as cases in a plain form or by the library.

Three operators stand around the paged 4-bit key/value cache and the head's logits:

* the page plan: from each sequence's length and the tokens that it gains or drops, the cache slots of new rows, the
  page tables and the queue of free pages;
* attention of a tree of drafted tokens: a row sees the cached context, its ancestors' rows and its own;
* candidates from logits: penalties for repeated tokens (those of a drafted row's ancestors among them), token
  biases and a grammar mask, then the K best tokens of each row, and the adjusted logits where they are wanted.

``own`` selects the form: False computes with elementary torch operations (whole numbers in 64 bits, the rest in fp32),
True calls the library. Both start from what ``prepare`` returns. ``exact`` states the same results again in float64.
"""
import math

import numpy as np
import torch

own = False

GROUP = 64    # values per quantisation group of the cache
GRANULE = 16  # tokens whose codes and parameters lie together in the cache


# ---------------------------------------------------------------------------------------- cases
def listed():
    plan = dict(op="plan", page=64, ctx_min=0, ctx_max=4096, grow=16, finish=0.0, rows=0, place=0, short=False)
    tree = dict(op="tree", q_heads=40, heads=8, dim=128, page=64, window=0, absent=False)
    pick = dict(op="pick", vocab=248320, dtype="float32", history=1024, tokens=False, ragged=False, bias=0, mask=False,
                out=False, k=16)
    return [
        # after each verified block of a serving batch: the accepted rows of 64 blocks of 16 find their slots
        dict(plan, name="plan_accept", batch=64, place=16),
        # prompts enter the cache in small pages, packed one behind the other, into free pages that run short
        dict(plan, name="plan_prompts", batch=24, page=16, ctx_max=0, grow=8192, rows=98304, short=True),
        # a large batch of single tokens; some sequences are done and give their pages back
        dict(plan, name="plan_tokens", batch=4096, page=32, ctx_max=2048, grow=1, finish=0.05, rows=4096),
        # one small tree over a short context: latency
        dict(tree, name="tree_8", batch=1, rows=8, ctx_min=1024, ctx_max=1024),
        # one full tree over a long context
        dict(tree, name="tree_64_long", batch=1, rows=64, ctx_min=32768, ctx_max=32768),
        # a serving batch of trees with ragged contexts; some trees are smaller than the batch's rows
        dict(tree, name="tree_batch", batch=32, rows=32, ctx_min=256, ctx_max=4096, absent=True),
        # small pages, 64-wide heads, a window, odd counts, empty contexts
        dict(tree, name="tree_window", batch=23, rows=13, q_heads=12, heads=4, dim=64, page=16, ctx_min=0, ctx_max=3001,
             window=1000, absent=True),
        # the candidates of one draft block's 15 rows: latency
        dict(pick, name="pick_block", batch=1, rows=15),
        # of 64 draft blocks
        dict(pick, name="pick_64", batch=64, rows=15),
        # one sampled token for each of 64 requests under a grammar, with biases; the adjusted logits go to a sampler
        dict(pick, name="pick_grammar", batch=64, rows=1, dtype="bfloat16", bias=40, mask=True, out=True, history=4096),
        # verification of trees: ancestors count as repeated, each node has its grammar state, the best token is wanted
        dict(pick, name="pick_tree", batch=12, rows=48, dtype="bfloat16", tokens=True, ragged=True, mask=True, k=1),
        # a draft vocabulary of odd size, long histories
        dict(pick, name="pick_odd", batch=7, rows=9, vocab=32771, history=30000, tokens=True, bias=3, out=True, k=5),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["plan", "tree", "tree", "pick", "pick", "pick"])
    if op == "plan":
        batch = _log_int(rng, 1, 4096)
        place = rng.choice([0, 0, 1, 5, 16, 33, 64])
        grow = place if place else _log_int(rng, 1, max(1, min(16384, 196608 // batch)))
        ctx_max = rng.choice([0, _log_int(rng, 1, max(1, min(8192, 16777216 // batch)))])
        return dict(op="plan", batch=batch, page=rng.choice([16, 32, 64, 128, 256]), ctx_min=rng.choice([0, ctx_max // 2]),
                    ctx_max=ctx_max, grow=grow, finish=rng.choice([0.0, 0.1]), place=place,
                    rows=0 if place else batch * grow + rng.choice([0, 3]), short=rng.random() < 0.3)
    if op == "tree":
        heads = rng.choice([1, 2, 4, 8])
        ratio = rng.choice([1, 2, 3, 4, 5, 6, 8])
        rows = rng.choice([1, 2, 5, 8, 13, 16, 26, 32, 48, 63, 64])
        batch = _log_int(rng, 1, 64)
        # the whole batch's scores stay below those of 32 trees of 32 rows over 4096 tokens
        room = 32 * 32 * 40 * 4096 // (batch * rows * heads * ratio)
        ctx_max = _log_int(rng, 1, max(1, min(32768, room, 64 * 8192 // batch)))
        return dict(op="tree", batch=batch, rows=rows, q_heads=heads * ratio, heads=heads, dim=rng.choice([64, 128, 128]),
                    page=rng.choice([16, 32, 64, 64, 128, 256]), ctx_min=rng.choice([0, 1, ctx_max // 2, ctx_max]),
                    ctx_max=ctx_max, window=rng.choice([0, 0, _log_int(rng, 1, max(1, ctx_max))]),
                    absent=rng.random() < 0.5)
    vocab = _log_int(rng, 1000, 248320)
    tokens = rng.random() < 0.4
    rows = rng.choice([1, 1, 2, 7, 15, 15, 31, 64])
    out = rng.random() < 0.4
    room = 64 * 15 * 248320 // (vocab * rows * (2 if out else 1))
    return dict(op="pick", batch=_log_int(rng, 1, max(1, min(256, room))), rows=rows, vocab=vocab,
                dtype=rng.choice(["float32", "bfloat16"]), history=rng.choice([0, _log_int(rng, 1, 32768)]),
                tokens=tokens, ragged=rng.random() < 0.5, bias=rng.choice([0, 0, 1, _log_int(rng, 2, 300)]),
                mask=rng.random() < 0.5, out=out, k=rng.choice([1, 4, 16, 16]))


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _ints(values):
    return torch.tensor(values, dtype=torch.int32, device="cuda")


def _prepare_plan(case, seed, st):
    r = np.random.default_rng(seed)
    B, page, grow = case["batch"], case["page"], case["grow"]
    ctx = r.integers(case["ctx_min"], case["ctx_max"] + 1, B)
    change = r.integers(min(1, case["place"]), grow + 1, B) if grow > 1 else np.ones(B, np.int64)
    change = np.where(r.random(B) < case["finish"], -ctx, change)
    width = -(-(case["ctx_max"] + grow) // page) + 1
    used = -(-ctx // page)
    need = int(np.maximum(0, -(-(ctx + change) // page) - used).sum())
    pages = B * (-(-case["ctx_max"] // page) + -(-grow // page) + 1)  # (the cache's)
    order = r.permutation(pages)
    table = np.zeros((B, width), np.int64)
    at = np.cumsum(used) - used
    col = np.arange(width)[None, :]
    table = np.where(col < used[:, None], order[np.minimum(at[:, None] + col, pages - 1)], 0)
    waiting = order[int(used.sum()):]
    if case["short"]:  # others hold the rest
        waiting = waiting[:max(1, need * 3 // 4)]
    head = int(r.integers(0, pages))
    queue = np.full(pages, -1)
    queue[(head + np.arange(waiting.size)) % pages] = waiting
    st.update(ctx=_ints(ctx), change=_ints(change), table=_ints(table), queue=_ints(queue),
              state=_ints([head, waiting.size]), pages=pages, place_of=None)
    if case["place"]:
        # the rows that a verified block or tree keeps, in order; the others go nowhere
        G = case["place"]
        rank = np.argsort(r.random((B, G)), 1)
        keep = np.argsort(rank, 1) < np.clip(change, 0, G)[:, None]
        st["place_of"] = _ints(np.where(keep, np.cumsum(keep, 1) - 1, -1))
    if own:
        n = (B, case["place"]) if case["place"] else (case["rows"],)
        new = lambda *s, t=torch.int32: torch.empty(s, dtype=t, device="cuda")
        st["outs"] = dict(ctx_out=new(B), state_out=new(2), offsets=new(B + 1), slots=new(*n, t=torch.int64),
                          positions=new(*n))


def _keys_values(g, tokens, heads, dim):
    """Keys with a few strong channels (as rotary keys have) and plain values, [tokens, heads, dim]."""
    channel = torch.ones(heads, dim, device="cuda")
    strong = torch.randint(0, dim, (heads, 3), generator=g, device="cuda")
    channel.scatter_(1, strong, 4.0)
    k = (torch.randn(tokens, heads, dim, generator=g, device="cuda") * channel).to(torch.bfloat16)
    return k, _normal(g, tokens, heads, dim)


def _granule_bytes(dim):
    return GRANULE * (dim // 2 + dim // GROUP * 4)


def _pack(x, pages, page):
    """[pages * page, heads, dim] rows as one side of the cache: [pages, heads, page / 16, granule]."""
    heads, dim = x.shape[1], x.shape[2]
    f = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    scale, bias = ((hi - lo) / 15.0).to(torch.bfloat16), lo.to(torch.bfloat16)
    code = ((f - bias.float()) / scale.float()).round().clamp(0.0, 15.0).to(torch.uint8).flatten(-2)
    packed = code[..., 0::2] | (code[..., 1::2] << 4)
    par = torch.cat([scale, bias], -1).contiguous().view(torch.uint8).flatten(-2)

    def order(t):
        t = t.view(pages, page // GRANULE, GRANULE, heads, -1).permute(0, 3, 1, 2, 4)
        return t.reshape(pages, heads, page // GRANULE, -1)

    return torch.cat([order(packed), order(par)], -1)


def _make_cache(g, pages, page, heads, dim):
    out = torch.empty(pages, heads, 2, page // GRANULE, _granule_bytes(dim), dtype=torch.uint8, device="cuda")
    step = max(1, 65536 // page)
    for p0 in range(0, pages, step):
        n = min(step, pages - p0)
        k, v = _keys_values(g, n * page, heads, dim)
        out[p0:p0 + n, :, 0] = _pack(k, n, page)
        out[p0:p0 + n, :, 1] = _pack(v, n, page)
    return out


def _trees(r, batch, rows, absent):
    """Parents of each row: -1 for a root, an earlier row else; -2 for rows behind the end of a smaller tree. Rows
    lean towards recent parents, as the best candidates are followed deepest."""
    par = np.empty((batch, rows), np.int64)
    for b in range(batch):
        n = int(r.integers(0, rows + 1)) if absent and b % 2 else rows
        for t in range(rows):
            near = t - 1 - int(r.integers(0, t + 1) * r.random()) if t else -1
            par[b, t] = max(-1, near) if t < n else -2
    return par


def _prepare_tree(case, seed, st):
    g, r = _gen(seed), np.random.default_rng(seed)
    B, G, heads, dim, page = case["batch"], case["rows"], case["heads"], case["dim"], case["page"]
    lens = r.integers(case["ctx_min"], case["ctx_max"] + 1, B)
    lens[0], lens[-1] = case["ctx_min"], case["ctx_max"]
    need = -(-lens // page)
    pages, width = int(need.sum()) + 2, max(1, int(need.max()))
    order = r.permutation(pages)
    at = np.cumsum(need) - need
    col = np.arange(width)[None, :]
    st["table"] = _ints(np.where(col < need[:, None], order[np.minimum(at[:, None] + col, pages - 1)], 0))
    st["cache"] = _make_cache(g, pages, page, heads, dim)
    st["lens"] = _ints(lens)
    st["scale"] = dim ** -0.5
    st["parents"] = _ints(_trees(r, B, G, case["absent"]))
    nq, nk = case["q_heads"] * dim, heads * dim
    qkv = torch.empty(B, G, nq + 2 * nk, dtype=torch.bfloat16, device="cuda")
    qkv[..., :nq] = _normal(g, B, G, nq)
    k, v = _keys_values(g, B * G, heads, dim)
    qkv[..., nq:nq + nk] = k.view(B, G, -1)
    qkv[..., nq + nk:] = v.view(B, G, -1)
    st["q"] = qkv[..., :nq].unflatten(-1, (case["q_heads"], dim))
    st["k_new"] = qkv[..., nq:nq + nk].unflatten(-1, (heads, dim))
    st["v_new"] = qkv[..., nq + nk:].unflatten(-1, (heads, dim))
    if own:
        import dflash2_block_drafter_gb300 as d
        st["out"] = torch.empty(B, G, case["q_heads"], dim, dtype=torch.bfloat16, device="cuda")
        n = d.dflash2_kv4_attention_workspace_bytes(B, G, case["q_heads"], heads, dim, page, width)
        st["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")


def _row_counts(r, case):
    """Rows of each request: all `rows`, or between one and that, half of the batch's in all."""
    B, G = case["batch"], case["rows"]
    if not case["ragged"] or G == 1:
        return np.full(B, G)
    more = r.permutation(B * (G - 1))[:B * (G - 1) // 2] // (G - 1)
    return 1 + np.bincount(more, minlength=B)


def _zipf(g, vocab, *shape):
    """Token ids whose frequency falls with the id, as a vocabulary's do."""
    u = torch.rand(*shape, generator=g, device="cuda", dtype=torch.float64)
    return (torch.exp(u * math.log(vocab + 1)) - 1).long().clamp(0, vocab - 1).to(torch.int32)


def _prepare_pick(case, seed, st):
    g, r = _gen(seed), np.random.default_rng(seed)
    B, V, n = case["batch"], case["vocab"], case["history"]
    counts = _row_counts(r, case)
    offsets = np.concatenate([[0], np.cumsum(counts)])
    M = int(offsets[-1])
    st["request"] = torch.from_numpy(np.repeat(np.arange(B), counts)).cuda()
    st["offsets"] = _ints(offsets) if case["ragged"] else None
    x = torch.randn(M, V, generator=g, device="cuda") * 2 - 0.4 * torch.log1p(torch.arange(V, device="cuda"))
    st["history"] = st["prompt"] = st["length"] = st["tokens"] = st["parents"] = None
    st["bias_ids"] = st["bias_values"] = st["mask"] = None
    if n:
        length = r.integers(0, n + 1, B)
        length[-1] = n
        st["history"] = _zipf(g, V, B, n)
        st["length"] = _ints(length)
        st["prompt"] = _ints((length * r.random(B)).astype(np.int64))
        # what was said is likely again
        recent = st["history"][:, -64:].long()[st["request"]]
        x.scatter_add_(1, recent, torch.full(recent.shape, 1.5, device="cuda"))
    if case["tokens"]:
        par = [_trees(r, 1, int(c), False)[0] for c in counts]
        st["parents"] = _ints(np.concatenate(par))
        st["tokens"] = _zipf(g, V, M)
    st["logits"] = x.to(getattr(torch, case["dtype"]))
    one = lambda lo, hi: torch.from_numpy(r.uniform(lo, hi, B).astype(np.float32)).cuda()
    st["repetition"], st["frequency"], st["presence"] = one(1.0, 1.5), one(-0.2, 1.0), one(-0.2, 1.0)
    if case["bias"]:
        ids = _zipf(g, V, B, case["bias"])
        spread = torch.rand(B, case["bias"], generator=g, device="cuda")
        st["bias_ids"] = torch.where(spread < 0.1, torch.full_like(ids, -1), ids)
        st["bias_values"] = torch.randn(B, case["bias"], generator=g, device="cuda") * 4
    if case["mask"]:
        # a grammar leaves a few tokens, about half of them, or all; now and then none
        words = -(-V // 32)
        some = np.array([1.0, 0.5, 20.0 / V, 2000.0 / V, 0.0])[r.choice(5, M, p=[0.3, 0.3, 0.2, 0.17, 0.03])]
        share = torch.from_numpy(some).cuda().float()
        st["mask"] = torch.empty(M, words, dtype=torch.int32, device="cuda")
        bit = 2 ** torch.arange(32, dtype=torch.int64, device="cuda")
        for m0 in range(0, M, 64):
            u = torch.rand(min(64, M - m0), words * 32, generator=g, device="cuda")
            w = ((u < share[m0:m0 + 64, None]).unflatten(1, (words, 32)) * bit).sum(-1)
            st["mask"][m0:m0 + 64] = torch.where(w >= 2 ** 31, w - 2 ** 32, w).to(torch.int32)
    if own:
        st["outs"] = dict(cand=torch.empty(M, case["k"], dtype=torch.int32, device="cuda"),
                          unary=torch.empty(M, case["k"], dtype=torch.float32, device="cuda"))
        if case["out"]:
            st["outs"]["out"] = torch.empty_like(st["logits"])


def prepare(case, seed):
    st = dict(case)
    {"plan": _prepare_plan, "tree": _prepare_tree, "pick": _prepare_pick}[case["op"]](case, seed, st)
    return st


# ------------------------------------------------------------------------------- the plain forms
def _plain_plan(st):
    page, T, Q = st["page"], st["rows"], st["pages"]
    ctx, ch, table, queue = (st[n].long() for n in ("ctx", "change", "table", "queue"))
    head, count = st["state"].long()
    B, width = table.shape
    zero = torch.zeros_like(ctx)
    fits = (ctx >= 0) & (ctx <= width * page) & (ctx + ch >= 0) & (ctx + ch <= width * page)
    p0, p1 = (ctx + page - 1) // page, (ctx + ch + page - 1) // page
    need = torch.where(fits, (p1 - p0).clamp(min=0), zero)
    granted = fits & ((need == 0) | (need.cumsum(0) <= count))
    rows = torch.where(granted, ch.clamp(min=0), zero)
    if st["place_of"] is None:
        granted = granted & ((rows == 0) | (rows.cumsum(0) <= T))
        rows = torch.where(granted, rows, zero)
    taken = torch.where(granted, need, zero)
    given = torch.where(granted, (p0 - p1).clamp(min=0), zero)
    ctx_out = torch.where(granted, ctx + ch, ctx)
    offsets = torch.cat([zero[:1], rows.cumsum(0)])

    def owner(n, size):
        """For items 0 .. size - 1 laid out sequence by sequence, n of each: (its sequence, its place there, is there)."""
        i = torch.arange(size, device="cuda")
        end = n.cumsum(0)
        b = torch.searchsorted(end, i, right=True).clamp(max=B - 1)
        return b, i - (end - n)[b], i < end[-1]

    at = torch.arange(Q, device="cuda")
    b, j, there = owner(taken, Q)                                    # pages taken
    flat = torch.cat([table.flatten(), zero[:1]])                    # (the last entry takes what goes nowhere)
    where = torch.where(there, b * width + p0[b] + j, torch.full_like(b, B * width))
    flat = flat.scatter(0, where, queue[(head + at) % Q])
    table2 = flat[:-1].view(B, width)
    b, j, there = owner(given, Q)                                    # pages given back
    old = table[b, (p1[b] + j).clamp(0, width - 1)]
    pad = torch.cat([queue, zero[:1]])
    queue2 = pad.scatter(0, torch.where(there, (head + count + at) % Q, torch.full_like(at, Q)), old)[:-1]
    state = torch.stack([(head + taken.sum()) % Q, count - taken.sum() + given.sum()])
    if st["place_of"] is None:
        b, j, there = owner(rows, T)
    else:
        j = st["place_of"].long()
        b = torch.arange(B, device="cuda").view(B, 1).expand_as(j)
        there = (j >= 0) & (j < rows[b])
    pos = ctx[b] + j
    entry = table2[b, (pos // page).clamp(0, width - 1)]
    slots = torch.where(there, entry * page + pos % page, torch.full_like(pos, -1))
    pos = torch.where(there, pos, torch.full_like(pos, -1))
    i32 = torch.int32
    return (ctx_out.to(i32), state.to(i32), offsets.to(i32), slots, pos.to(i32), table2.to(i32), queue2.to(i32))


def _plain_cached(cache, table, side, page, dim):
    """fp32 rows of one side of the cache in the order of `table`: [B, heads, width * page, dim]."""
    raw = cache[table.long(), :, side]                                   # [B, width, heads, granules, bytes]
    B, width, heads, gran, _ = raw.shape
    nb = GRANULE * dim // 2
    by = raw[..., :nb].view(B, width, heads, gran, GRANULE, dim // 2)
    code = torch.stack([by & 15, by >> 4], -1).flatten(-2).float()       # [..., dim]
    par = raw[..., nb:].contiguous().view(torch.bfloat16).float().view(B, width, heads, gran, GRANULE, dim // GROUP, 2)
    val = par[..., :1] * code.unflatten(-1, (-1, GROUP)) + par[..., 1:]
    return val.flatten(-2).permute(0, 2, 1, 3, 4, 5).reshape(B, heads, width * page, dim)


def _line(parents, deepest):
    """[..., G, G] whether row j is row t or one of its ancestors, and [..., G] how many ancestors t has (-1: t is not
    there). parents [..., G]: -1 a root, -2 not there."""
    G = parents.shape[-1]
    me = torch.arange(G, device=parents.device)
    at = torch.where(parents >= -1, me.expand_as(parents), torch.full_like(parents, -1))
    line = torch.zeros(*parents.shape, G, dtype=torch.bool, device=parents.device)
    for _ in range(deepest):
        line |= at.unsqueeze(-1) == me
        at = torch.where(at >= 0, parents.gather(-1, at.clamp(min=0)).clamp(min=-1), at)
    return line, line.sum(-1) - 1


def _plain_tree(st):
    B, G, R = st["batch"], st["rows"], st["q_heads"] // st["heads"]
    dim, page, heads = st["dim"], st["page"], st["heads"]
    K = _plain_cached(st["cache"], st["table"], 0, page, dim)
    V = _plain_cached(st["cache"], st["table"], 1, page, dim)
    L = K.shape[2]
    lens = st["lens"].long().view(B, 1)
    at = torch.arange(L, device="cuda").view(1, L)
    there = at < lens
    V = torch.where(there.view(B, 1, L, 1), V, torch.zeros_like(V))
    K = torch.cat([K, st["k_new"].float().transpose(1, 2)], 2)
    V = torch.cat([V, st["v_new"].float().transpose(1, 2)], 2)
    line, depth = _line(st["parents"].long(), G)
    see = there.view(B, 1, L) & (depth >= 0).view(B, G, 1)
    if st["window"] > 0:
        see = see & (at.view(1, 1, L) > (lens + depth).view(B, G, 1) - st["window"])
        line = line & (depth.view(B, 1, G) > depth.view(B, G, 1) - st["window"])
    see = torch.cat([see, line], 2)
    q = st["q"].float().view(B, G, heads, R, dim).permute(0, 2, 1, 3, 4).reshape(B, heads, G * R, dim)
    s = (q @ K.transpose(2, 3)).view(B, heads, G, R, -1) * st["scale"]
    s = s.masked_fill(~see.view(B, 1, G, 1, -1), float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    den = p.sum(-1, keepdim=True)
    p = p / torch.where(den > 0, den, torch.ones_like(den))
    o = (p.view(B, heads, G * R, -1) @ V).view(B, heads, G, R, dim)
    return o.permute(0, 2, 1, 3, 4).reshape(B, G, heads * R, dim).to(torch.bfloat16)


def _allowed(mask, V):
    """[M, V] truth values of a bit mask's rows."""
    bits = torch.arange(32, dtype=torch.int32, device="cuda")
    return ((mask.unsqueeze(-1) >> bits) & 1).flatten(1)[:, :V] != 0


def _plain_pick(st):
    x, req, V = st["logits"].float(), st["request"], st["vocab"]
    M, B = x.shape[0], st["batch"]
    said = torch.zeros(B, V, dtype=torch.int32, device="cuda")        # how often each token was generated
    prompt = torch.zeros(B, V, dtype=torch.int32, device="cuda")
    if st["history"] is not None:
        at = torch.arange(st["history"].shape[1], device="cuda").view(1, -1)
        h = st["history"].long()
        in_prompt = at < torch.minimum(st["prompt"], st["length"]).view(B, 1)
        prompt.scatter_add_(1, h, in_prompt.int())
        said.scatter_add_(1, h, ((at < st["length"].view(B, 1)) & ~in_prompt).int())
    count = said[req]
    seen = prompt[req] > 0
    if st["tokens"] is not None:
        off = torch.zeros(B + 1, dtype=torch.long, device="cuda")
        off[1:] = torch.bincount(req, minlength=B).cumsum(0)
        G = st["rows"]
        row = off[req]                                                # each row's request's first row
        grid = torch.full((B, G), -2, dtype=torch.long, device="cuda")
        mine = torch.arange(M, device="cuda") - row
        grid[req, mine] = st["parents"].long()
        line = _line(grid, G)[0][req, mine].int()                     # [M, G]
        tok = torch.zeros(B, G, dtype=torch.long, device="cuda")
        tok[req, mine] = st["tokens"].long()
        count.scatter_add_(1, tok[req], line)
    seen |= count > 0
    rep, freq, pres = (st[n][req].view(M, 1) for n in ("repetition", "frequency", "presence"))
    x = torch.where(seen, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (freq * count.float() + pres * (count > 0).float())
    if st["bias_ids"] is not None:
        ids = st["bias_ids"].long()
        earlier = torch.ones(ids.shape[1], ids.shape[1], dtype=torch.bool, device="cuda").tril(-1)
        first = (ids >= 0) & ~((ids.unsqueeze(2) == ids.unsqueeze(1)) & earlier).any(2)   # a token's first entry counts
        dense = torch.zeros(B, V, device="cuda")
        dense.scatter_add_(1, ids.clamp(min=0), torch.where(first, st["bias_values"], torch.zeros_like(st["bias_values"])))
        x = x + dense[req]
    if st["mask"] is not None:
        x = torch.where(_allowed(st["mask"], V), x, torch.full_like(x, float("-inf")))
    # the k best, the lowest token first among equals
    token = torch.arange(V, dtype=torch.int32, device="cuda").expand(M, V)
    left = torch.ones(M, V, dtype=torch.bool, device="cuda")
    low, cand, unary = torch.full_like(x, float("-inf")), [], []
    for _ in range(st["k"]):
        top = torch.where(left, x, low).amax(1, keepdim=True)
        pick = torch.where(left & (x == top), token, torch.full_like(token, V)).amin(1, keepdim=True)
        left.scatter_(1, pick.long(), False)
        cand.append(pick)
        unary.append(top)
    got = torch.cat(cand, 1), torch.cat(unary, 1)
    return got + (x.to(st["logits"].dtype),) if st["out"] else got


# ------------------------------------------------------------------------------------- the passes
def run(state):
    st = state
    if not own:
        return {"plan": _plain_plan, "tree": _plain_tree, "pick": _plain_pick}[st["op"]](st)
    import dflash2_block_drafter_gb300 as d
    if st["op"] == "plan":
        got = d.dflash2_kv4_plan(st["ctx"], st["change"], st["table"], st["queue"], st["state"], st["page"], st["pages"],
                                 rows=st["rows"], place=st["place_of"], **st["outs"])
        return got + (st["table"], st["queue"])
    if st["op"] == "tree":
        return d.dflash2_kv4_attention_tree(st["q"], st["cache"], st["table"], st["lens"], st["page"], st["scale"],
                                            st["k_new"], st["v_new"], st["parents"], window=st["window"], out=st["out"],
                                            workspace=st["workspace"])
    got = d.dflash2_logits_topk(st["logits"], st["k"], requests=st["batch"], row_offsets=st["offsets"],
                                history=st["history"], prompt_len=st["prompt"], history_len=st["length"],
                                repetition=st["repetition"], frequency=st["frequency"], presence=st["presence"],
                                tokens=st["tokens"], parents=st["parents"], bias_ids=st["bias_ids"],
                                bias=st["bias_values"], mask=st["mask"], **st["outs"])
    return got if st["out"] else got[:2]


# ---------------------------------------------------------------------------------------- the work
def _mean(lo, hi):
    return (lo + hi) / 2


def work(case):
    B = case["batch"]
    if case["op"] == "plan":
        rows = B * case["place"] if case["place"] else case["rows"]
        moved = B * _mean(min(1, case["place"]), case["grow"]) * (1 - case["finish"])
        paged = (moved + case["finish"] * B * _mean(case["ctx_min"], case["ctx_max"])) / case["page"]
        # lengths in and out, offsets, each row's slot and position (and place), each page that changes hands
        by = 16 * B + rows * 12 + (4 * rows if case["place"] else 0) + 8 * paged
        return {"bytes": int(by), "flops": int(8 * (rows + B + paged))}
    if case["op"] == "tree":
        G, D = case["rows"], case["dim"]
        mid = _mean(case["ctx_min"], case["ctx_max"])
        keys = case["ctx_max"] if B == 1 else (case["ctx_min"] + case["ctx_max"] + (B - 2) * mid) / B
        if case["window"]:
            keys = min(keys, case["window"])
        rows = B * G * (0.75 if case["absent"] and B > 1 else 1.0)
        by = B * keys * case["heads"] * 2 * (D // 2 + D // GROUP * 4) + 2 * B * G * case["q_heads"] * D * 2
        by += 2 * B * G * case["heads"] * D * 2 + 4 * B * G
        return {"bytes": int(by), "flops": int(4 * D * case["q_heads"] * rows * (keys + math.sqrt(G)))}
    V, size = case["vocab"], 4 if case["dtype"] == "float32" else 2
    rows = B + B * (case["rows"] - 1) // 2 if case["ragged"] else B * case["rows"]
    by = rows * V * size * (2 if case["out"] else 1) + rows * 8 * case["k"] + B * _mean(0, case["history"]) * 4
    by += (rows * -(-V // 32) * 4 if case["mask"] else 0) + (8 * rows if case["tokens"] else 0) + 8 * B * case["bias"]
    return {"bytes": int(by), "flops": int(2 * rows * V)}


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_plan(st):
    """Sequence by sequence, with the queue as a list."""
    page, T, Q = st["page"], st["rows"], st["pages"]
    ctx, ch, table, queue = (st[n].cpu().numpy().astype(np.int64) for n in ("ctx", "change", "table", "queue"))
    head, count = st["state"].tolist()
    B, width = table.shape
    place = None if st["place_of"] is None else st["place_of"].cpu().numpy()
    shape = T if place is None else place.shape
    slots, pos = np.full(shape, -1, np.int64), np.full(shape, -1, np.int64)
    out, off = ctx.copy(), np.zeros(B + 1, np.int64)
    taken, back, asked, filled, full = 0, [], 0, 0, False
    new = table.copy()
    for b in range(B):
        off[b + 1] = off[b]
        end = ctx[b] + ch[b]
        if not (0 <= ctx[b] <= width * page and 0 <= end <= width * page):
            continue
        have, want = -(-ctx[b] // page), -(-end // page)
        if want > have:
            asked += want - have
            if asked > count:
                continue
        gain = max(0, ch[b])
        if place is None and gain:
            if full or filled + gain > T:
                full = True
                continue
            filled += gain
        for i in range(have, want):
            new[b, i] = queue[(head + taken) % Q]
            taken += 1
        back += table[b, want:have].tolist()
        out[b] = end
        off[b + 1] = off[b] + gain
        if gain:
            p = ctx[b] + np.arange(gain)
            s = new[b, p // page] * page + p % page
            if place is None:
                slots[off[b]:off[b + 1]], pos[off[b]:off[b + 1]] = s, p
            else:
                ok = (place[b] >= 0) & (place[b] < gain)
                slots[b, ok], pos[b, ok] = s[place[b, ok]], p[place[b, ok]]
    waiting = queue.copy()
    for i, p in enumerate(back):
        waiting[(head + count + i) % Q] = p
    state = np.array([(head + taken) % Q, count - taken + len(back)])
    return tuple(torch.from_numpy(np.ascontiguousarray(a)).cuda() for a in (out, state, off, slots, pos, new, waiting))


def _exact_read(cache, pages, n, head, side, dim):
    """Cached rows 0 .. n - 1 of one sequence and head, float64 [n, dim]."""
    blob = cache[pages.long(), head, side].reshape(-1, cache.shape[-1])  # granules in order
    codes = blob[:, :GRANULE * dim // 2].reshape(-1, dim // 2)
    par = blob[:, GRANULE * dim // 2:].contiguous().view(torch.bfloat16).double().reshape(-1, dim // GROUP, 2)
    val = torch.empty(codes.shape[0], dim, dtype=torch.float64, device=cache.device)
    val[:, 0::2] = (codes % 16).double()
    val[:, 1::2] = torch.div(codes, 16, rounding_mode="floor").double()
    for i in range(dim // GROUP):
        val[:, i * GROUP:(i + 1) * GROUP] *= par[:, i, 0:1]
        val[:, i * GROUP:(i + 1) * GROUP] += par[:, i, 1:2]
    return val[:n]


def _lines(parents):
    """Each row's list of rows from its root down to itself; empty for a row that is not there."""
    lines = []
    for t, p in enumerate(parents):
        lines.append([] if p < -1 else (lines[p] if p >= 0 else []) + [t])
    return lines


def _exact_tree(st):
    B, G, heads, dim = st["batch"], st["rows"], st["heads"], st["dim"]
    R, window = st["q_heads"] // heads, st["window"]
    out = torch.zeros(B, G, st["q_heads"], dim, dtype=torch.float64, device="cuda")
    parents = st["parents"].tolist()
    for b, n in enumerate(st["lens"].tolist()):
        see = torch.zeros(G, n + G, dtype=torch.bool)
        for t, line in enumerate(_lines(parents[b])):
            if line:
                at = n + len(line) - 1                               # the row's position
                see[t, max(0, at - window + 1) if window else 0:n] = True
                see[t, [n + j for j in (line[-window:] if window else line)]] = True
        see = see.cuda()
        some = see.any(1)
        for h in range(heads):
            K = torch.cat([_exact_read(st["cache"], st["table"][b], n, h, 0, dim), st["k_new"][b, :, h].double()])
            V = torch.cat([_exact_read(st["cache"], st["table"][b], n, h, 1, dim), st["v_new"][b, :, h].double()])
            for j in range(R):
                s = st["q"][b, :, h * R + j].double() @ K.T * st["scale"]
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                out[b, some, h * R + j] = torch.softmax(s[some], -1) @ V
    return out


def _step(x):
    """A step's result as fp32 holds it: the adjusted logits are defined with each step rounded to fp32, so that which
    of two nearly equal tokens comes first does not depend on who computes it."""
    return x.float().double()


def _exact_pick(st):
    """Row by row: the few tokens that something applies to, one vector of them at a time."""
    logits, V, B = st["logits"], st["vocab"], st["batch"]
    req = st["request"].tolist()
    first = [req.index(b) for b in range(B)] + [len(req)]
    parents = st["parents"].tolist() if st["parents"] is not None else None
    tokens = st["tokens"].tolist() if st["tokens"] is not None else None
    cand, unary, outs = [], [], []
    for b in range(B):
        said = torch.zeros(V, dtype=torch.float64, device="cuda")
        known = torch.zeros(V, dtype=torch.bool, device="cuda")
        if st["history"] is not None:
            n = int(st["length"][b])
            p = min(int(st["prompt"][b]), n)
            h = st["history"][b].long()
            known[h[:p]] = True
            said += torch.bincount(h[p:n], minlength=V).double()
        rep, freq, pres = (st[k][b].double() for k in ("repetition", "frequency", "presence"))
        bias = {}
        if st["bias_ids"] is not None:
            for i, v in zip(st["bias_ids"][b].tolist(), st["bias_values"][b].tolist()):
                if i >= 0:
                    bias.setdefault(i, v)
        lines = _lines(parents[first[b]:first[b + 1]]) if parents is not None else None
        for m in range(first[b], first[b + 1]):
            c = said
            if lines is not None:
                c = said.clone()
                for t in lines[m - first[b]]:
                    c[tokens[first[b] + t]] += 1
            x = logits[m].double()
            hit = ((c > 0) | known).nonzero().view(-1)
            v = x[hit]
            v = _step(torch.where(v > 0, v / rep, v * rep))
            x[hit] = _step(v - _step(_step(freq * c[hit]) + pres * (c[hit] > 0)))
            if bias:
                at = torch.tensor(list(bias), device="cuda")
                x[at] = _step(x[at] + torch.tensor(list(bias.values()), dtype=torch.float64, device="cuda"))
            if st["mask"] is not None:
                w = st["mask"][m].long() & 0xFFFFFFFF
                at = torch.arange(V, device="cuda")
                x[(w[at // 32] >> (at % 32)) % 2 == 0] = -math.inf
            top, at = torch.sort(x, descending=True, stable=True)
            cand.append(at[:st["k"]].clone())
            unary.append(top[:st["k"]].clone())
            if st["out"]:
                outs.append(x)
    got = torch.stack(cand), torch.stack(unary)
    return got + (torch.stack(outs),) if st["out"] else got


def exact(case, seed):
    st = prepare(case, seed)
    return {"plan": _exact_plan, "tree": _exact_tree, "pick": _exact_pick}[case["op"]](st)
