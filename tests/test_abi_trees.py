"""Host-side refusals of the page plan, tree attention and candidate calls (no GPU): a status before anything is
launched, and the Python binding's checks of shapes, types and strides."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)      # aligned, never dereferenced: validation fails first
FAKE_MIS = ctypes.c_void_p(0x10002)  # misaligned for 16 bytes and for fp32


@pytest.fixture(scope="module")
def lib():
    from dflash2_block_drafter_gb300 import _build
    import dflash2_block_drafter_gb300 as pkg
    _build.build()
    return pkg.library()


def _plan(lib, **kw):
    a = dict(ctx=FAKE, change=FAKE, table=FAKE, queue=FAKE, state=FAKE, place=None, B=4, G=0, rows=16, width=8, page=64,
             pages=100, cap=100, ctx_out=FAKE, state_out=FAKE, off=FAKE, slots=FAKE, pos=FAKE)
    a.update(kw)
    return lib.dflash2_kv4_plan(a["ctx"], a["change"], a["table"], a["queue"], a["state"], a["place"], a["B"], a["G"],
                                a["rows"], a["width"], a["page"], a["pages"], a["cap"], a["ctx_out"], a["state_out"],
                                a["off"], a["slots"], a["pos"], None)


def test_plan_rejects_bad_arguments(lib):
    for bad in (dict(B=0), dict(B=8193), dict(page=48), dict(page=8), dict(page=8192), dict(pages=0), dict(cap=0),
                dict(width=0), dict(width=2 ** 26), dict(rows=-1), dict(rows=2 ** 31 - 1), dict(ctx=None), dict(change=None),
                dict(table=None), dict(queue=None), dict(state=None), dict(ctx_out=None), dict(state_out=None),
                dict(off=None), dict(slots=None), dict(pos=None), dict(place=FAKE, G=0), dict(place=FAKE, G=2 ** 30),
                dict(place=FAKE, G=4, slots=None)):
        assert _plan(lib, **bad) == -1, bad


def test_plan_refuses_counts_that_its_steps_would_pass(lib):
    for bad in (dict(rows=2 ** 31 - 1024), dict(cap=2 ** 31 - 1024), dict(B=8191, place=FAKE, G=262176)):
        assert _plan(lib, **bad) == -1, bad


def _tree(lib, **kw):
    a = dict(q=FAKE, qs=5120, cache=FAKE, table=FAKE, ctx=FAKE, kn=FAKE, vn=FAKE, ns=1024, par=FAKE, B=2, G=16, Hq=40, Hkv=8,
             D=128, page=64, pages=10, width=4, window=0, scale=0.1, dtype=0, out=FAKE, ws=None, wsb=0)
    a.update(kw)
    return lib.dflash2_kv4_attention_tree(a["q"], a["qs"], a["cache"], a["table"], a["ctx"], a["kn"], a["vn"], a["ns"],
                                          a["par"], a["B"], a["G"], a["Hq"], a["Hkv"], a["D"], a["page"], a["pages"],
                                          a["width"], a["window"], a["scale"], a["dtype"], a["out"], a["ws"], a["wsb"], None)


def test_tree_attention_rejects_bad_arguments(lib):
    assert _tree(lib, dtype=1) == -2
    for bad in (dict(par=None), dict(kn=None), dict(vn=None), dict(kn=None, vn=None), dict(G=65), dict(G=0), dict(B=0),
                dict(Hq=41), dict(D=96), dict(page=24), dict(q=None), dict(out=FAKE_MIS), dict(qs=5112), dict(ns=1000),
                dict(window=-1), dict(scale=float("nan"))):
        assert _tree(lib, **bad) == -1, bad
    need = lib.dflash2_kv4_attention_workspace_bytes(2, 16, 40, 8, 128, 64, 4)
    assert _tree(lib) == -4 and _tree(lib, ws=FAKE, wsb=need - 1) == -4


def _pick(lib, **kw):
    a = dict(logits=FAKE, stride=1000, M=8, V=1000, dtype=1, B=4, off=None, hist=FAKE, hs=50, prompt=FAKE, length=FAKE,
             max_len=50, rep=FAKE, freq=FAKE, pres=FAKE, tokens=FAKE, parents=FAKE, ids=FAKE, bias=FAKE, nb=3, mask=FAKE,
             ms=32, K=16, cand=FAKE, unary=FAKE, out=FAKE, os=1000, ws=None, wsb=0)
    a.update(kw)
    return lib.dflash2_logits_topk(a["logits"], a["stride"], a["M"], a["V"], a["dtype"], a["B"], a["off"], a["hist"], a["hs"],
                                   a["prompt"], a["length"], a["max_len"], a["rep"], a["freq"], a["pres"], a["tokens"],
                                   a["parents"], a["ids"], a["bias"], a["nb"], a["mask"], a["ms"], a["K"], a["cand"],
                                   a["unary"], a["out"], a["os"], a["ws"], a["wsb"], None)


def test_candidates_reject_bad_arguments(lib):
    for bad in (dict(dtype=2), dict(M=-1), dict(B=0), dict(V=0), dict(V=2 ** 22 + 1), dict(K=-1), dict(K=17), dict(V=15),
                dict(M=9), dict(logits=None), dict(cand=None), dict(unary=None), dict(K=0, out=None), dict(logits=FAKE_MIS),
                dict(out=FAKE_MIS), dict(stride=999), dict(os=999), dict(length=None), dict(max_len=-1),
                dict(max_len=2 ** 20), dict(hs=49), dict(tokens=None), dict(M=65 * 4), dict(nb=-1), dict(nb=2048),
                dict(ids=None), dict(bias=None), dict(ms=31)):
        assert _pick(lib, **bad) == -1, bad
    need = lib.dflash2_logits_topk_workspace_bytes(8, 1000, 4, 0, 50, 1, 3, 16)
    assert need > 0 and _pick(lib) == -4 and _pick(lib, ws=FAKE, wsb=need - 1) == -4
    assert _pick(lib, ws=ctypes.c_void_p(0x10010), wsb=need) == -1  # not 256-byte aligned
    assert lib.dflash2_logits_topk_workspace_bytes(8, 0, 4, 0, 50, 1, 3, 16) == 0
    assert _pick(lib, M=2 ** 25, B=2 ** 25, V=2 ** 20, stride=2 ** 20, os=2 ** 20, ms=2 ** 15) == -1
    assert _pick(lib, M=0, logits=None, cand=None, unary=None, out=None) == 0  # no rows: nothing to do


def test_python_checks():
    torch = pytest.importorskip("torch")
    import dflash2_block_drafter_gb300 as d
    i32 = torch.int32
    ints = lambda *s: torch.zeros(*s, dtype=i32)
    plan = lambda **kw: d.dflash2_kv4_plan(**dict(dict(
        ctx_len=ints(4), change=ints(4), page_table=ints(4, 2), free_pages=ints(9), free_state=ints(2), page_size=16,
        num_pages=9, rows=8), **kw))
    for match, bad in (("ctx_len and change", dict(change=ints(3))), ("page_table", dict(page_table=ints(3, 2))),
                       ("free_pages", dict(free_state=ints(3))), ("place", dict(place=ints(3, 2))),
                       ("slots holds", dict(slots=torch.zeros(7, dtype=torch.int64))),
                       ("offsets holds", dict(offsets=ints(4))), ("state_out holds", dict(state_out=ints(1))),
                       ("ctx_out holds", dict(ctx_out=ints(3))), ("positions holds", dict(positions=ints(7)))):
        with pytest.raises(ValueError, match=match):
            plan(**bad)
    with pytest.raises(ValueError, match="CUDA"):
        plan()
    pick = lambda **kw: d.dflash2_logits_topk(**dict(dict(logits=torch.zeros(4, 64), K=4), **kw))
    with pytest.raises(ValueError, match="CUDA"):
        pick()
    with pytest.raises(ValueError, match="logits must be"):
        pick(logits=torch.zeros(64))
    with pytest.raises(ValueError, match="dtype"):
        pick(logits=torch.zeros(4, 64, dtype=torch.float16))
    with pytest.raises(ValueError, match="row_offsets"):
        pick(requests=3, row_offsets=ints(3))
    with pytest.raises(ValueError, match="needs k_new"):
        d.dflash2_kv4_attention_tree(None, None, None, None, 16, 1.0, None, None, None)
