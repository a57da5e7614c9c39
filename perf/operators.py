"""The drafter's sublayer operators, as cases that can be run in a plain form or by the library.

Three operators stand around the block-local tail:

* rows of the 4-bit key/value cache: quantise rows of keys and values into cache slots and read
  slots back (affine codes 0..15 in groups of 64 along the head: value = scale * code + bias);
* attention of each sequence's G query rows (one token, or a draft block) over its cached context
  and, unquantised, the block's own rows;
* the gated feed-forward product act(x Wg^T) * (x Wu^T), and its gradients.

``own`` selects the form: False computes with elementary torch operations in fp32, True calls the
library. Both start from what ``prepare`` returns. ``exact`` states the same results in float64.
"""
import math

import torch

own = False

GROUP = 64    # values per quantisation group
GRANULE = 16  # tokens whose codes and parameters lie together in the cache


# ---------------------------------------------------------------------------------------- cases
def listed():
    rows = dict(op="rows", heads=8, dim=128, page=64, stride_extra=5120, skip=False)
    att = dict(op="attention", q_heads=40, heads=8, dim=128, page=64, causal=False, window=0, new=True)
    ffn = dict(op="ffn", hidden=5120, inter=13824, act="silu", train=False)
    return [
        # the accepted rows of one draft block enter the cache: pure latency
        dict(rows, name="rows_block", tokens=16),
        # a long prompt's keys and values, slices of a fused q/k/v product; some rows are padding
        dict(rows, name="rows_prompt", tokens=32768, skip=True),
        # one sequence, one token at a time
        dict(att, name="token_1", batch=1, rows=1, ctx_min=1024, ctx_max=1024, new=False),
        # a serving batch of single tokens with ragged contexts
        dict(att, name="token_64", batch=64, rows=1, ctx_min=1, ctx_max=8192, new=False),
        # one draft block (anchor + 15 masks, bidirectional inside the block) over a long context
        dict(att, name="block_long", batch=1, rows=16, ctx_min=32768, ctx_max=32768),
        # 64 draft blocks with ragged contexts
        dict(att, name="block_64", batch=64, rows=16, ctx_min=256, ctx_max=4096),
        # causal rows over a sliding window in small pages; 64-wide heads, odd counts, empty contexts
        dict(att, name="window_causal", batch=23, rows=7, q_heads=12, heads=4, dim=64, page=16, ctx_min=0,
             ctx_max=3001, causal=True, window=1000),
        # the gate/up sublayer of one draft block: a weight stream
        dict(ffn, name="ffn_block", rows=16),
        # of 64 draft blocks: tensor-core bound
        dict(ffn, name="ffn_64", rows=1024),
        # odd sizes and the other activation
        dict(ffn, name="ffn_odd", rows=333, hidden=1352, inter=3592, act="gelu_tanh"),
        # a training step of the drafter's sublayer: product and all gradients
        dict(ffn, name="train_4096", rows=4096, train=True),
        # a ragged training batch of a narrower drafter
        dict(ffn, name="train_odd", rows=1001, hidden=2568, inter=6920, act="gelu_tanh", train=True),
    ]


def _log_int(rng, lo, hi):
    return min(hi, max(lo, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))))


def draw(rng):
    op = rng.choice(["rows", "attention", "attention", "ffn", "ffn", "train"])
    if op == "rows":
        dim = rng.choice([64, 128])
        return dict(op="rows", heads=rng.choice([1, 2, 4, 5, 8]), dim=dim, page=rng.choice([16, 32, 64, 128, 256]),
                    tokens=_log_int(rng, 1, 32768), stride_extra=rng.choice([0, 8, 1024, 5120]),
                    skip=rng.random() < 0.5)
    if op == "attention":
        heads = rng.choice([1, 2, 4, 8])
        ratio = rng.choice([1, 2, 3, 4, 5, 6, 8])
        rows = rng.choice([1, 1, 2, 5, 8, 16, 16, 24, 32])
        batch = _log_int(rng, 1, 64)
        # the whole batch's scores stay below those of 64 blocks of 16 rows over 4096 tokens
        room = 64 * 16 * 40 * 4096 // (batch * rows * heads * ratio)
        ctx_max = _log_int(rng, 1, max(1, min(32768, room, 64 * 8192 // batch)))
        causal = rng.random() < 0.4
        return dict(op="attention", batch=batch, rows=rows, q_heads=heads * ratio, heads=heads,
                    dim=rng.choice([64, 128, 128]), page=rng.choice([16, 32, 64, 64, 128, 256]),
                    ctx_min=rng.choice([0, 1, ctx_max // 2, ctx_max]), ctx_max=ctx_max, causal=causal,
                    window=rng.choice([0, 0, _log_int(rng, 1, max(1, ctx_max))]), new=rng.random() < 0.7)
    train = op == "train"
    hidden = 8 * _log_int(rng, 8, 640)
    inter = 8 * _log_int(rng, 8, 1728)
    return dict(op="ffn", rows=_log_int(rng, 1, 4096), hidden=hidden, inter=inter,
                act=rng.choice(["silu", "gelu_tanh"]), train=train)


# ------------------------------------------------------------------------------------ the inputs
def _gen(seed):
    return torch.Generator(device="cuda").manual_seed(seed)


def _normal(g, *shape, std=1.0):
    return (torch.randn(*shape, generator=g, device="cuda", dtype=torch.float32) * std).to(torch.bfloat16)


def _keys_values(g, tokens, heads, dim):
    """Keys with a few strong channels (as rotary keys have) and plain values, [tokens, heads, dim]."""
    channel = torch.ones(heads, dim, device="cuda")
    strong = torch.randint(0, dim, (heads, 3), generator=g, device="cuda")
    channel.scatter_(1, strong, 4.0)
    k = (torch.randn(tokens, heads, dim, generator=g, device="cuda") * channel).to(torch.bfloat16)
    return k, _normal(g, tokens, heads, dim)


def _granule_bytes(dim):
    return GRANULE * (dim // 2 + dim // GROUP * 4)


def _quantise(x):
    """Codes, scales and biases of [..., dim] rows: one group per 64 values."""
    f = x.float().unflatten(-1, (-1, GROUP))
    lo, hi = f.amin(-1, keepdim=True), f.amax(-1, keepdim=True)
    scale = ((hi - lo) / 15.0).to(torch.bfloat16)
    bias = lo.to(torch.bfloat16)
    s, b = scale.float(), bias.float()
    code = torch.where(s > 0, ((f - b) / s).round().clamp(0.0, 15.0), torch.zeros_like(f))
    return code, scale, bias


def _pack(x, pages, page):
    """[pages * page, heads, dim] rows as one side of the cache: [pages, heads, page / 16, granule]."""
    heads, dim = x.shape[1], x.shape[2]
    code, scale, bias = _quantise(x)
    code = code.to(torch.uint8).flatten(-2)                              # [T, heads, dim]
    packed = code[..., 0::2] | (code[..., 1::2] << 4)                    # [T, heads, dim / 2]
    par = torch.cat([scale, bias], -1).contiguous().view(torch.uint8)    # [T, heads, groups, 4] bytes
    par = par.flatten(-2)

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


def _lengths(case, seed):
    r = torch.Generator().manual_seed(seed)
    lo, hi = case["ctx_min"], case["ctx_max"]
    n = torch.randint(lo, hi + 1, (case["batch"],), generator=r).tolist()
    n[-1] = hi
    if case["batch"] > 1:
        n[0] = lo
    return n


def prepare(case, seed):
    g = _gen(seed)
    st = dict(case)
    if case["op"] == "rows":
        T, heads, dim, page = case["tokens"], case["heads"], case["dim"], case["page"]
        k, v = _keys_values(g, T, heads, dim)
        fused = torch.zeros(T, 2 * heads * dim + case["stride_extra"], dtype=torch.bfloat16, device="cuda")
        fused[:, :heads * dim] = k.flatten(1)
        fused[:, heads * dim:2 * heads * dim] = v.flatten(1)
        st["k"] = fused[:, :heads * dim].unflatten(1, (heads, dim))
        st["v"] = fused[:, heads * dim:2 * heads * dim].unflatten(1, (heads, dim))
        pages = -(-T // page) + 3
        slots = torch.randperm(pages * page, generator=g, device="cuda")[:T]
        if case["skip"]:
            slots = torch.where(torch.rand(T, generator=g, device="cuda") < 0.05, torch.full_like(slots, -1), slots)
        st["slots"] = slots
        st["cache"] = torch.zeros(pages, heads, 2, page // GRANULE, _granule_bytes(dim), dtype=torch.uint8,
                                  device="cuda")
    elif case["op"] == "attention":
        B, G, heads, dim, page = case["batch"], case["rows"], case["heads"], case["dim"], case["page"]
        lens = _lengths(case, seed)
        need = [-(-n // page) for n in lens]
        pages = sum(need) + 2
        width = max(1, max(need))
        order = torch.randperm(pages, generator=g, device="cuda")
        table = torch.zeros(B, width, dtype=torch.int32, device="cuda")
        at = 0
        for b, n in enumerate(need):
            table[b, :n] = order[at:at + n]
            at += n
        st["cache"] = _make_cache(g, pages, page, heads, dim)
        st["table"] = table
        st["lens"] = torch.tensor(lens, dtype=torch.int32, device="cuda")
        st["scale"] = dim ** -0.5
        qkv = torch.empty(B, G, (case["q_heads"] + 2 * heads) * dim, dtype=torch.bfloat16, device="cuda")
        nq = case["q_heads"] * dim
        qkv[..., :nq] = _normal(g, B, G, nq)
        k, v = _keys_values(g, B * G, heads, dim)
        qkv[..., nq:nq + heads * dim] = k.view(B, G, -1)
        qkv[..., nq + heads * dim:] = v.view(B, G, -1)
        st["q"] = qkv[..., :nq].unflatten(-1, (case["q_heads"], dim))
        st["k_new"] = qkv[..., nq:nq + heads * dim].unflatten(-1, (heads, dim)) if case["new"] else None
        st["v_new"] = qkv[..., nq + heads * dim:].unflatten(-1, (heads, dim)) if case["new"] else None
        if own:
            import dflash2_block_drafter_gb300 as d
            st["out"] = torch.empty(B, G, case["q_heads"], dim, dtype=torch.bfloat16, device="cuda")
            n = d.dflash2_kv4_attention_workspace_bytes(B, G, case["q_heads"], heads, dim, page, width)
            st["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
    else:
        M, H, F = case["rows"], case["hidden"], case["inter"]
        st["x"] = _normal(g, M, H)
        st["wg"] = _normal(g, F, H, std=H ** -0.5)
        st["wu"] = _normal(g, F, H, std=H ** -0.5)
        if case["train"]:
            st["dh"] = _normal(g, M, F, std=1e-2)
        if own:
            import dflash2_block_drafter_gb300 as d
            new = lambda *s: torch.empty(*s, dtype=torch.bfloat16, device="cuda")
            st["h"] = new(M, F)
            n = d.dflash2_gated_ffn_workspace_bytes(M, H, F, int(case["train"]))
            st["workspace"] = torch.empty(max(n, 256), dtype=torch.uint8, device="cuda")
            if case["train"]:
                st["pre"] = new(2, M, F)
                st["dx"], st["dwg"], st["dwu"] = new(M, H), new(F, H), new(F, H)
    return st


# ------------------------------------------------------------------------------- the plain forms
def _plain_rows(st):
    out = []
    keep = (st["slots"] >= 0).view(-1, 1, 1)
    for x in (st["k"], st["v"]):
        code, scale, bias = _quantise(x)
        val = (scale.float() * code + bias.float()).flatten(-2)
        out.append(torch.where(keep, val, torch.zeros_like(val)).to(torch.bfloat16))
    return tuple(out)


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


def _plain_attention(st):
    B, G, R = st["batch"], st["rows"], st["q_heads"] // st["heads"]
    dim, page, heads = st["dim"], st["page"], st["heads"]
    K = _plain_cached(st["cache"], st["table"], 0, page, dim)
    V = _plain_cached(st["cache"], st["table"], 1, page, dim)
    L = K.shape[2]
    lens = st["lens"].long().view(B, 1)
    at = torch.arange(L, device="cuda").view(1, L)
    there = at < lens                                                    # [B, L]
    pos = at.expand(B, L)
    total = lens
    if st["k_new"] is not None:
        K = torch.cat([K, st["k_new"].float().transpose(1, 2)], 2)
        V = torch.cat([V, st["v_new"].float().transpose(1, 2)], 2)
        mine = torch.arange(G, device="cuda").view(1, G)
        pos = torch.cat([pos, lens + mine], 1)
        there = torch.cat([there, torch.ones(B, G, dtype=torch.bool, device="cuda")], 1)
        total = lens + G
    V = torch.where(there.view(B, 1, -1, 1), V, torch.zeros_like(V))
    row = total - G + torch.arange(G, device="cuda").view(1, G)          # [B, G] positions of the query rows
    see = there.view(B, 1, -1).expand(B, G, -1)
    if st["causal"]:
        see = see & (pos.view(B, 1, -1) <= row.view(B, G, 1))
    if st["window"] > 0:
        see = see & (pos.view(B, 1, -1) > row.view(B, G, 1) - st["window"])
    q = st["q"].float().view(B, G, heads, R, dim).permute(0, 2, 1, 3, 4).reshape(B, heads, G * R, dim)
    s = (q @ K.transpose(2, 3)).view(B, heads, G, R, -1) * st["scale"]
    s = s.masked_fill(~see.view(B, 1, G, 1, -1), float("-inf"))
    top = s.amax(-1, keepdim=True)
    p = torch.exp(s - torch.where(torch.isinf(top), torch.zeros_like(top), top))
    den = p.sum(-1, keepdim=True)
    p = p / torch.where(den > 0, den, torch.ones_like(den))
    o = (p.view(B, heads, G * R, -1) @ V).view(B, heads, G, R, dim)
    return o.permute(0, 2, 1, 3, 4).reshape(B, G, heads * R, dim).to(torch.bfloat16)


def _act(g, kind):
    """act(g) and act'(g)."""
    if kind == "silu":
        s = 1.0 / (1.0 + torch.exp(-g))
        return g * s, s * (1.0 + g * (1.0 - s))
    c = math.sqrt(2.0 / math.pi)
    t = torch.tanh(c * (g + 0.044715 * g * g * g))
    return 0.5 * g * (1.0 + t), 0.5 * (1.0 + t) + 0.5 * g * (1.0 - t * t) * c * (1.0 + 3.0 * 0.044715 * g * g)


def _plain_ffn(st):
    x, wg, wu = st["x"].float(), st["wg"].float(), st["wu"].float()
    g, u = x @ wg.t(), x @ wu.t()
    a, da = _act(g, st["act"])
    h = (a * u).to(torch.bfloat16)
    if not st["train"]:
        return h
    dh = st["dh"].float()
    dg, du = dh * u * da, dh * a
    dx = dg @ wg + du @ wu
    return tuple(t.to(torch.bfloat16) for t in (h, dx, dg.t() @ x, du.t() @ x))


# ------------------------------------------------------------------------------------- the passes
def run(state):
    st = state
    if not own:
        return {"rows": _plain_rows, "attention": _plain_attention, "ffn": _plain_ffn}[st["op"]](st)
    import dflash2_block_drafter_gb300 as d
    if st["op"] == "rows":
        d.dflash2_kv4_append(st["k"], st["v"], st["slots"], st["cache"], st["page"])
        return d.dflash2_kv4_read(st["cache"], st["slots"], st["dim"], st["page"])
    if st["op"] == "attention":
        return d.dflash2_kv4_attention(st["q"], st["cache"], st["table"], st["lens"], st["page"], st["scale"],
                                       k_new=st["k_new"], v_new=st["v_new"], causal=st["causal"],
                                       window=st["window"], out=st["out"], workspace=st["workspace"])
    if not st["train"]:
        return d.dflash2_gated_ffn(st["x"], st["wg"], st["wu"], act=st["act"], out=st["h"],
                                   workspace=st["workspace"])
    h = d.dflash2_gated_ffn(st["x"], st["wg"], st["wu"], act=st["act"], out=st["h"], pre=st["pre"],
                            workspace=st["workspace"])
    dx, dwg, dwu = d.dflash2_gated_ffn_backward(st["dh"], st["pre"], st["x"], st["wg"], st["wu"], act=st["act"],
                                                dx=st["dx"], dw_gate=st["dwg"], dw_up=st["dwu"],
                                                workspace=st["workspace"])
    return h, dx, dwg, dwu


# ---------------------------------------------------------------------------------------- the work
def _seen(case, n):
    """(cached keys that some row sees, visible (row, key) pairs) of one head and n cached tokens."""
    G, N = case["rows"], case["rows"] if case["new"] else 0
    total, pairs, first = n + N, 0, n
    for t in range(G):
        row = total - G + t
        hi = min(total, row + 1) if case["causal"] else total
        lo = max(0, row - case["window"] + 1) if case["window"] > 0 else 0
        pairs += max(0, hi - lo)
        if hi > lo:
            first = min(first, lo)
    return n - first, pairs


def work(case):
    if case["op"] == "rows":
        n = case["tokens"] * case["heads"] * case["dim"] * 2             # keys and values
        coded = case["tokens"] * case["heads"] * 2 * (case["dim"] // 2 + case["dim"] // GROUP * 4)
        return {"bytes": 2 * n * 2 + 2 * coded + 16 * case["tokens"], "flops": 8 * n}
    if case["op"] == "attention":
        B, G, D = case["batch"], case["rows"], case["dim"]
        if B == 1 or case["ctx_min"] == case["ctx_max"]:
            lens = [case["ctx_max"]] * B
        else:                                                            # the mean of the drawn lengths
            mid = (case["ctx_min"] + case["ctx_max"]) // 2
            lens = [case["ctx_min"]] + [mid] * (B - 2) + [case["ctx_max"]]
        keys = pairs = 0
        for n in lens:
            k, p = _seen(case, n)
            keys += k
            pairs += p
        row = D // 2 + D // GROUP * 4
        by = keys * case["heads"] * 2 * row + 2 * B * G * case["q_heads"] * D * 2
        if case["new"]:
            by += 2 * B * G * case["heads"] * D * 2
        return {"bytes": by, "flops": 4 * D * pairs * case["q_heads"]}
    M, H, F = case["rows"], case["hidden"], case["inter"]
    by, fl = 2 * (M * H + 2 * F * H + M * F), 4 * M * F * H
    if case["train"]:
        by += 2 * (M * F + M * H + 2 * F * H)
        fl += 8 * M * F * H
    return {"bytes": by, "flops": fl}


# ---------------------------------------------------------------------------------- in 64 bits
def _exact_side(rows):
    """The values the 4-bit codes of [..., dim] rows stand for, group by group."""
    x = rows.double()
    parts = []
    for g0 in range(0, x.shape[-1], GROUP):
        v = x[..., g0:g0 + GROUP]
        lo = v.min(-1, keepdim=True).values
        step = ((v.max(-1, keepdim=True).values - lo) / 15.0).to(torch.bfloat16).double()
        base = lo.to(torch.bfloat16).double()
        n = torch.where(step > 0, torch.round((v - base) / torch.where(step > 0, step, 1.0)), 0.0)
        parts.append(n.clamp(0, 15) * step + base)
    return torch.cat(parts, -1)


def _exact_read(cache, pages, n, head, side, page, dim):
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


def _exact_attention(st):
    B, G, heads, dim = st["batch"], st["rows"], st["heads"], st["dim"]
    R = st["q_heads"] // heads
    out = torch.zeros(B, G, st["q_heads"], dim, dtype=torch.float64, device="cuda")
    for b, n in enumerate(st["lens"].tolist()):
        total = n + (G if st["k_new"] is not None else 0)
        key = torch.arange(total, device="cuda")
        row = (total - G + torch.arange(G, device="cuda")).view(G, 1)
        see = torch.ones(G, total, dtype=torch.bool, device="cuda")
        if st["causal"]:
            see &= key <= row
        if st["window"] > 0:
            see &= row - key < st["window"]
        if total == 0:
            continue
        some = see.any(1)
        pages = st["table"][b]
        for h in range(heads):
            K = _exact_read(st["cache"], pages, n, h, 0, st["page"], dim)
            V = _exact_read(st["cache"], pages, n, h, 1, st["page"], dim)
            if total > n:
                K = torch.cat([K, st["k_new"][b, :, h].double()])
                V = torch.cat([V, st["v_new"][b, :, h].double()])
            for j in range(R):
                hq = h * R + j
                s = st["q"][b, :, hq].double() @ K.T * st["scale"]
                s = torch.where(see, s, torch.full_like(s, -math.inf))
                w = torch.softmax(s[some], -1)
                out[b, some, hq] = w @ V
    return out


def _exact_ffn(st):
    x, wg, wu = (st[n].double() for n in ("x", "wg", "wu"))
    g, u = x.mm(wg.T), x.mm(wu.T)
    if st["act"] == "silu":
        sig = torch.sigmoid(g)
        a, slope = g * sig, sig + g * sig * (1 - sig)
    else:
        k = (2 / math.pi) ** 0.5
        t = torch.tanh(k * (g + 0.044715 * g ** 3))
        a = g * (1 + t) / 2
        slope = (1 + t) / 2 + g / 2 * (1 - t ** 2) * k * (1 + 0.134145 * g ** 2)
    if not st["train"]:
        return a * u
    dh = st["dh"].double()
    dg, du = dh * u * slope, dh * a
    return a * u, dg.mm(wg) + du.mm(wu), dg.T.mm(x), du.T.mm(x)


def exact(case, seed):
    st = prepare(case, seed)
    if case["op"] == "rows":
        keep = (st["slots"] >= 0).view(-1, 1, 1)
        return tuple(torch.where(keep, _exact_side(st[n]), 0.0) for n in ("k", "v"))
    if case["op"] == "attention":
        return _exact_attention(st)
    return _exact_ffn(st)
