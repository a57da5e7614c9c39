"""GPU parity of candidates from logits: ids, values and adjusted logits bit for bit (every step is rounded to fp32 in the
definition; bf16 outputs are its values rounded once)."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import S, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _case(rng, B, rows, V, dtype="float32", history=0, tokens=None, ragged=False, bias=0, mask=None, penalties=True,
          behind=0):
    """Host arrays of a call; `behind` rows of no request follow the last one."""
    counts = np.full(B, rows) if not ragged else rng.integers(0, rows + 1, B)
    off = np.concatenate([[0], np.cumsum(counts)]).astype(np.int32)
    M = int(off[-1]) + behind
    x = (3 * rng.normal(size=(M, V))).astype(np.float32)
    c = dict(B=B, M=M, V=V, off=off, ragged=ragged or behind > 0, dtype=dtype,
             logits=S.bf16(x).astype(np.float32) if dtype == "bfloat16" else x)
    zipf = lambda *s: np.minimum(V - 1, np.exp(rng.random(s) * np.log(V + 1)) - 1).astype(np.int32)
    if history:
        c["history"], c["length"] = zipf(B, history), rng.integers(0, history + 1, B).astype(np.int32)
        c["length"][-1] = history
        c["prompt"] = (c["length"] * rng.random(B)).astype(np.int32)
    if tokens:
        c["tokens"] = zipf(M)
        if tokens != "chain":
            c["parents"] = np.concatenate([[int(rng.integers(-1, t)) if t and rng.random() > 0.1 else -1 for t in range(n)]
                                           for n in counts] + [np.zeros(behind, int)]).astype(np.int32)
    if penalties:
        c["rep"], c["freq"], c["pres"] = (rng.uniform(lo, hi, B).astype(np.float32) for lo, hi in
                                          ((0.8, 1.6), (-0.5, 1.0), (-0.5, 1.0)))
    if bias:
        c["ids"] = np.where(rng.random((B, bias)) < 0.2, -rng.integers(1, 5, (B, bias)), zipf(B, bias)).astype(np.int32)
        c["bias"] = (4 * rng.normal(size=(B, bias))).astype(np.float32)
    if mask is not None:
        c["mask"] = rng.random((M, V)) < mask
    return c


def _words(allowed):
    M, V = allowed.shape
    bits = np.zeros((M, -(-V // 32) * 32), np.uint8)
    bits[:, :V] = allowed
    return np.packbits(bits, axis=1, bitorder="little").view(np.int32)


def _want(c, K):
    """(cand, unary, out), rows of no request None."""
    M, V, B = c["M"], c["V"], c["B"]
    cand, unary, out = [None] * M, [None] * M, [None] * M
    for b in range(B):
        lo, hi = c["off"][b], c["off"][b + 1]
        base, prompt = np.zeros(V, int), np.zeros(V, bool)
        if "history" in c:
            h, p, n = c["history"][b], c["prompt"][b], c["length"][b]
            ok = lambda t: t[(t >= 0) & (t < V)]
            prompt[ok(h[:min(p, n)])] = True
            np.add.at(base, ok(h[min(p, n):n]), 1)
        bias = {}
        if "ids" in c:
            for i, v in zip(c["ids"][b], c["bias"][b]):
                if 0 <= i < V:
                    bias.setdefault(int(i), v)
        par = c["parents"][lo:hi] if "parents" in c else np.arange(hi - lo) - 1
        lines = T.lines(par) if "tokens" in c else None
        for m in range(lo, hi):
            n = base
            if lines is not None:
                line = lines[m - lo]
                if not line:
                    cand[m], unary[m] = np.full(K, -1), np.full(K, -np.inf, np.float32)
                    continue
                n = base.copy()
                for j in line:
                    t = c["tokens"][lo + j]
                    if 0 <= t < V:
                        n[t] += 1
            y = T.adjust(c["logits"][m], n, prompt, *(c[k][b] if k in c else z for k, z in (("rep", 1), ("freq", 0), ("pres", 0))),
                         bias, c["mask"][m] if "mask" in c else None)
            cand[m] = T.best(y, K)
            unary[m] = y[cand[m]]
            out[m] = y
    return cand, unary, out


def _args(torch, c, pad=0, shift=0):
    """Device arguments. Rows of logits lie V + pad apart, `shift` elements behind an aligned address."""
    dt = getattr(torch, c["dtype"])
    dev = lambda x: None if x is None else torch.from_numpy(np.ascontiguousarray(x)).cuda()
    flat = torch.full((shift + c["M"] * (c["V"] + pad),), float("nan"), dtype=dt, device="cuda")
    logits = flat[shift:].view(c["M"], c["V"] + pad)[:, :c["V"]]
    logits.copy_(dev(c["logits"]))
    kw = dict(requests=c["B"], row_offsets=dev(c["off"]) if c["ragged"] else None)
    for name, key in (("history", "history"), ("prompt_len", "prompt"), ("history_len", "length"), ("repetition", "rep"),
                      ("frequency", "freq"), ("presence", "pres"), ("tokens", "tokens"), ("parents", "parents"),
                      ("bias_ids", "ids"), ("bias", "bias")):
        kw[name] = dev(c.get(key))
    kw["mask"] = dev(_words(c["mask"])) if "mask" in c else None
    return logits, kw


def _check(torch, c, K, want_out=True, pad=0, shift=0, error=0, in_place=False):
    import dflash2_block_drafter_gb300 as d
    logits, kw = _args(torch, c, pad, shift)
    cand = torch.full((c["M"], K), -77, dtype=torch.int32, device="cuda") if K else None
    unary = torch.full((c["M"], K), 77.0, device="cuda") if K else None
    out = None
    if in_place:
        out = logits
    elif want_out:
        out = torch.full((c["M"], c["V"] + pad), 77.0, dtype=logits.dtype, device="cuda")[:, :c["V"]]
    before = None if out is None else out.float().cpu().numpy()
    got = d.dflash2_logits_topk(logits, K, cand=cand, unary=unary, out=out, **kw)
    assert d.dflash2_poll_error() == error
    wc, wu, wo = _want(c, K)
    for m in range(c["M"]):
        if K and wc[m] is None:
            assert (got[0][m] == -77).all() and (got[1][m] == 77).all(), f"row {m} of no request"
        elif K:
            np.testing.assert_array_equal(got[0][m].cpu().numpy(), wc[m], err_msg=f"ids of row {m}")
            np.testing.assert_array_equal(got[1][m].cpu().numpy(), wu[m], err_msg=f"values of row {m}")
        if out is not None:
            want = before[m] if wo[m] is None else wo[m]
            if c["dtype"] == "bfloat16" and wo[m] is not None:
                want = torch.from_numpy(want).to(torch.bfloat16).float().numpy()
            np.testing.assert_array_equal(out[m].float().cpu().numpy(), want, err_msg=f"logits of row {m}")
    return got


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,rows,V,K", [(1, 1, 1, 1), (1, 1, 16, 16), (2, 3, 100, 5), (3, 2, 1000, 16), (1, 5, 1024, 1),
                                        (1, 1, 16384, 16), (2, 2, 16385, 16), (1, 2, 50001, 3), (40, 1, 2500, 16)])
def test_raw_logits(torch, dtype, B, rows, V, K):
    _check(torch, _case(np.random.default_rng(V), B, rows, V, dtype), K)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("tokens,ragged", [(None, False), ("chain", False), ("tree", True), ("tree", False)])
def test_everything_at_once(torch, dtype, tokens, ragged):
    rng = np.random.default_rng(7)
    for B, rows, V, history, bias in ((3, 5, 1200, 400, 6), (9, 64, 700, 33, 1), (2, 33, 20011, 3000, 200)):
        c = _case(rng, B, rows, V, dtype, history, tokens, ragged, bias, 0.6, behind=3 if ragged else 0)
        _check(torch, c, 16)
        _check(torch, c, 1, want_out=False)
        _check(torch, c, 0, in_place=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("B,rows,V", [(20, 10, 3001), (50, 10, 17501), (50, 10, 2001), (500, 1, 37)])
def test_more_rows_than_three_a_multiprocessor(torch, dtype, B, rows, V):
    """Fewer threads a row from 153 and 457 rows on, by the rows' length; then rows of equal values, whose every token
    reaches the bound."""
    rng = np.random.default_rng(V)
    c = _case(rng, B, rows, V, dtype, 150, "tree", False, 3, 0.6)
    _check(torch, c, 16)
    _check(torch, c, 2, in_place=True)
    c = _case(rng, B, rows, V, dtype)
    c["logits"][::2] = 1.5
    _check(torch, c, 16, want_out=False)


@pytest.mark.parametrize("part", ["history", "tokens", "bias", "mask", "penalties"])
def test_each_part_alone(torch, part):
    rng = np.random.default_rng(8)
    kw = dict(history=dict(history=300), tokens=dict(tokens="tree"), bias=dict(bias=20), mask=dict(mask=0.5),
              penalties=dict(penalties=True))[part]
    _check(torch, _case(rng, 3, 4, 1500, **dict(dict(penalties=part in ("history", "tokens", "penalties")), **kw)), 16)


@pytest.mark.parametrize("V", [248320, 300001])
def test_a_whole_vocabulary(torch, V):
    rng = np.random.default_rng(9)
    for B, rows, dtype in ((1, 1, "float32"), (3, 5, "bfloat16"), (40, 2, "float32")):
        _check(torch, _case(rng, B, rows, V, dtype, history=2000, tokens="tree", bias=4, mask=0.9), 16)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("pad,shift", [(0, 0), (1, 0), (3, 1), (8, 2), (5, 7)])
def test_strides_and_alignments(torch, dtype, pad, shift):
    c = _case(np.random.default_rng(10), 3, 3, 2311, dtype, history=100, bias=3, mask=0.7)
    _check(torch, c, 16, pad=pad, shift=shift)
    _check(torch, c, 8, pad=pad, shift=shift, in_place=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_masks_that_leave_few_tokens_or_none(torch, dtype):
    rng = np.random.default_rng(12)
    c = _case(rng, 12, 1, 40000, dtype, history=50, bias=2, mask=0.0)
    for m in range(12):  # 0, 1, 2, 4, .. tokens, scattered or side by side
        n = 0 if m == 0 else 2 ** (m - 1)
        c["mask"][m, rng.permutation(40000)[:n] if m % 2 else np.arange(777, 777 + n)] = True
    _check(torch, c, 16)
    c["logits"][3, :] = -np.inf
    c["logits"][5, c["mask"][5]] = [np.inf] * 16
    _check(torch, c, 16)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_ties_orders_and_odd_values(torch, dtype):
    """Rows in ascending, descending and equal order, with zeros of both signs, infinities, NaN of both signs and the type's
    lowest value."""
    rng = np.random.default_rng(13)
    V = 40000
    c = _case(rng, 14, 1, V, dtype, history=20, mask=None)
    x = c["logits"]
    x[0] = 1.5
    x[1] = 0.0
    x[1, ::3] = -0.0
    x[2] = np.sort(x[2])
    x[3] = np.sort(x[3])[::-1]
    x[4] = rng.integers(0, 3, V)
    x[5, rng.permutation(V)[:40]] = np.nan
    x[6, rng.permutation(V)[:5]] = -np.float32(np.nan)
    x[7] = -np.inf
    x[7, [5, 39999]] = -3e38
    x[8] = np.inf
    x[9] = np.nan
    x[10] = -3.3895313892515355e38  # bf16's lowest value
    x[11, 1000:2000] = 50.0         # a thousand equal ones side by side
    x[12, 0:V:256] = np.linspace(50, 60, len(x[12, 0:V:256]))  # the best fall to few threads
    x[13, 8192:8260] = 1e38
    if dtype == "bfloat16":
        c["logits"] = torch.from_numpy(x).to(torch.bfloat16).float().numpy()
    _check(torch, c, 16)


def test_long_histories_and_repeated_indices(torch):
    rng = np.random.default_rng(14)
    c = _case(rng, 2, 3, 5000, history=70000, tokens="chain", bias=300)
    c["history"][0, :66000] = 4321                                    # a count past 16 bits
    c["prompt"][0], c["length"][0] = 0, 66000
    c["tokens"][:] = 4321                                             # and once more for each ancestor
    c["ids"][0, :] = 17                                               # the first entry of a token counts
    c["ids"][1, ::2] = 4999
    _check(torch, c, 16)


def test_empty_histories_and_prompt_bounds(torch):
    rng = np.random.default_rng(15)
    c = _case(rng, 6, 2, 900, history=40)
    c["length"][:] = [0, 1, 40, 40, 40, 7]
    c["prompt"][:] = [0, 1, 40, 0, 100, -5]  # a prompt longer than the history, or negative: all of it, none of it
    _check(torch, {**c, "prompt": np.maximum(c["prompt"], 0)}, 16)
    import dflash2_block_drafter_gb300 as d
    logits, kw = _args(torch, c)
    a = d.dflash2_logits_topk(logits, 16, **kw)
    logits, kw = _args(torch, {**c, "prompt": np.clip(c["prompt"], 0, c["length"])})
    b = d.dflash2_logits_topk(logits, 16, **kw)
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1]) and d.dflash2_poll_error() == 0


def test_bad_indices_lengths_and_spans_are_recorded(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(16)
    V = 3000
    for key, at, value in (("history", (0, 0), V), ("history", (1, 3), -1), ("tokens", 2, V + 5), ("tokens", 0, -1),
                           ("ids", (1, 1), 2 ** 31 - 1), ("parents", 2, 2), ("parents", 4, 99)):
        c = _case(rng, 2, 4, V, history=30, tokens="tree", bias=3)
        c["length"][:] = 30
        c["parents"][:] = [-1, 0, 1, 2] * 2
        c[key][at] = value
        _check(torch, c, 16, error=-6)
    c = _case(rng, 2, 2, V, history=30)
    for n, as_if in ((31, 30), (-1, 0), (2 ** 31 - 1, 30)):
        c["length"][0] = n
        logits, kw = _args(torch, c)
        got = d.dflash2_logits_topk(logits, 4, **kw)
        assert d.dflash2_poll_error() == -1
        c["length"][0] = as_if
        logits, kw = _args(torch, c)
        want = d.dflash2_logits_topk(logits, 4, **kw)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1]) and d.dflash2_poll_error() == 0
    # spans outside the rows
    c = _case(rng, 3, 4, V)
    logits, kw = _args(torch, c)
    for off in ([0, 4, 8, 13], [-1, 4, 8, 12], [0, 9, 8, 12]):
        kw["row_offsets"] = torch.tensor(off, dtype=torch.int32, device="cuda")
        d.dflash2_logits_topk(logits, 4, **kw)
        assert d.dflash2_poll_error() == -1, off
    # drafted rows past the 64th are left as they were
    c = _case(rng, 1, 70, 500, tokens="chain", behind=0)
    c["ragged"] = True
    logits, kw = _args(torch, c)
    cand = torch.full((70, 4), -77, dtype=torch.int32, device="cuda")
    d.dflash2_logits_topk(logits, 4, cand=cand, **kw)
    assert d.dflash2_poll_error() == -1
    assert (cand[64:] == -77).all() and (cand[:64] >= 0).all()
    np.testing.assert_array_equal(cand[:64].cpu().numpy(), np.stack(_want(c, 4)[0][:64]))


def test_trees_with_rows_that_are_not_there(torch):
    c = _case(np.random.default_rng(17), 3, 20, 800, history=50, tokens="tree")
    c["parents"].reshape(3, 20)[1, 12:] = -2
    c["parents"].reshape(3, 20)[2, :] = -5
    _check(torch, c, 16)


def test_in_a_graph_on_another_stream_and_two_at_once(torch):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(18)
    a, b = (_case(rng, 5, 3, 30000, "bfloat16", history=200, tokens="tree", bias=3, mask=0.5) for _ in range(2))
    (x, kx), (y, ky) = _args(torch, a), _args(torch, b)
    wx, wy = d.dflash2_logits_topk(x, 16, **kx), d.dflash2_logits_topk(y, 16, **ky)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for _ in range(5):
        gy = d.dflash2_logits_topk(y, 16, stream=side, **ky)
        gx = d.dflash2_logits_topk(x, 16, **kx)
        torch.cuda.synchronize()
        assert torch.equal(gx[0], wx[0]) and torch.equal(gx[1], wx[1])
        assert torch.equal(gy[0], wy[0]) and torch.equal(gy[1], wy[1])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph, stream=side):
        got = d.dflash2_logits_topk(x, 16, **kx)
    for src, want in ((y, d.dflash2_logits_topk(y, 16, **kx)), (x.clone(), wx)):
        x.copy_(src)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert d.dflash2_poll_error() == 0


def test_rows_past_32_bits(torch):
    """Logits of more than 2^32 elements: the last rows are reached."""
    import dflash2_block_drafter_gb300 as d
    V, M = 1 << 18, (1 << 14) + 5
    x = torch.zeros(M, V, dtype=torch.bfloat16, device="cuda")
    x[:, 3] = 1.0
    at = torch.arange(M, device="cuda") * 7 % V
    x[torch.arange(M, device="cuda"), at] = 2.0
    cand, unary, _ = d.dflash2_logits_topk(x, 2)
    assert d.dflash2_poll_error() == 0
    assert torch.equal(cand[:, 0].long(), at)
    assert torch.equal(cand[:, 1].long(), torch.where(at == 3, 0, 3)) and (unary[:, 0] == 2).all()
