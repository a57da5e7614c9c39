"""Host-side refusals of the sublayer operators (no GPU): a status before anything is launched, and the
Python binding's checks of shapes, types and strides."""
import ctypes

import pytest

FAKE = ctypes.c_void_p(0x10000)      # 16-byte aligned, never dereferenced: validation fails first
FAKE_MIS = ctypes.c_void_p(0x10008)  # misaligned


@pytest.fixture(scope="module")
def lib():
    from dflash2_block_drafter_gb300 import _build
    import dflash2_block_drafter_gb300 as pkg
    _build.build()
    return pkg.library()


def test_kv4_page_bytes(lib):
    # per token, head and side: D / 2 bytes of codes and 4 bytes for each group of 64
    assert lib.dflash2_kv4_page_bytes(8, 128, 64) == 8 * 2 * 64 * (64 + 8)
    assert lib.dflash2_kv4_page_bytes(3, 64, 16) == 3 * 2 * 16 * (32 + 4)
    for heads, D, page in ((0, 128, 64), (513, 128, 64), (8, 96, 64), (8, 256, 64), (8, 128, 8), (8, 128, 48), (8, 128, 8192)):
        assert lib.dflash2_kv4_page_bytes(heads, D, page) == 0


def _append(lib, **kw):
    a = dict(k=FAKE, v=FAKE, ks=1024, vs=1024, slots=FAKE, T=4, heads=8, D=128, page=64, pages=4, dtype=0, cache=FAKE)
    a.update(kw)
    return lib.dflash2_kv4_append(a["k"], a["v"], a["ks"], a["vs"], a["slots"], a["T"], a["heads"], a["D"], a["page"],
                                  a["pages"], a["dtype"], a["cache"], None)


def test_kv4_append_rejects_bad_arguments(lib):
    assert _append(lib, dtype=1) == -2
    for bad in (dict(T=-1), dict(heads=0), dict(D=80), dict(page=100), dict(pages=0), dict(k=None), dict(v=None),
                dict(slots=None), dict(cache=None), dict(k=FAKE_MIS), dict(cache=FAKE_MIS), dict(ks=1016), dict(vs=1028),
                dict(ks=-1024)):
        assert _append(lib, **bad) == -1, bad
    assert _append(lib, T=0, k=None, v=None, slots=None) == 0  # no rows: nothing to do


def test_kv4_read_rejects_bad_arguments(lib):
    f = lambda **kw: (lambda a: lib.dflash2_kv4_read(a["cache"], a["slots"], a["T"], a["heads"], a["D"], a["page"],
                                                     a["pages"], a["dtype"], a["k"], a["v"], None))(
        dict(dict(cache=FAKE, slots=FAKE, T=4, heads=8, D=128, page=64, pages=4, dtype=0, k=FAKE, v=FAKE), **kw))
    assert f(dtype=1) == -2
    for bad in (dict(T=-1), dict(D=0), dict(page=15), dict(cache=None), dict(slots=None), dict(k=None), dict(v=FAKE_MIS)):
        assert f(**bad) == -1, bad
    assert f(T=0, k=None, v=None) == 0


def _attention(lib, **kw):
    a = dict(q=FAKE, qs=5120, cache=FAKE, table=FAKE, ctx=FAKE, kn=FAKE, vn=FAKE, ns=1024, B=2, G=16, Hq=40, Hkv=8, D=128,
             page=64, pages=10, width=4, causal=0, window=0, scale=0.1, dtype=0, out=FAKE, ws=None, wsb=0)
    a.update(kw)
    return lib.dflash2_kv4_attention(a["q"], a["qs"], a["cache"], a["table"], a["ctx"], a["kn"], a["vn"], a["ns"], a["B"],
                                     a["G"], a["Hq"], a["Hkv"], a["D"], a["page"], a["pages"], a["width"], a["causal"],
                                     a["window"], a["scale"], a["dtype"], a["out"], a["ws"], a["wsb"], None)


def test_kv4_attention_rejects_bad_arguments(lib):
    assert _attention(lib, dtype=1) == -2
    for bad in (dict(B=0), dict(G=0), dict(G=65), dict(Hq=41), dict(Hq=4), dict(Hq=8 * 65), dict(D=96), dict(page=24),
                dict(pages=0), dict(width=0), dict(width=2 ** 30), dict(q=None), dict(cache=None), dict(table=None),
                dict(ctx=None), dict(out=None), dict(kn=None), dict(vn=None), dict(q=FAKE_MIS), dict(kn=FAKE_MIS),
                dict(out=FAKE_MIS), dict(qs=5112), dict(qs=5124), dict(ns=1000), dict(window=-1), dict(causal=2),
                dict(scale=float("nan")), dict(scale=float("inf"))):
        assert _attention(lib, **bad) == -1, bad
    assert _attention(lib) == -4  # no workspace
    need = lib.dflash2_kv4_attention_workspace_bytes(2, 16, 40, 8, 128, 64, 4)
    assert need > 0 and _attention(lib, ws=FAKE, wsb=need - 1) == -4
    assert _attention(lib, ws=ctypes.c_void_p(0x10010), wsb=need) == -1  # not 256-byte aligned
    assert lib.dflash2_kv4_attention_workspace_bytes(2, 65, 40, 8, 128, 64, 4) == 0


def _ffn(lib, **kw):
    a = dict(x=FAKE, M=16, H=512, wg=FAKE, wu=FAKE, F=1024, act=0, dtype=0, h=FAKE, pre=None, ws=None, wsb=0)
    a.update(kw)
    return lib.dflash2_gated_ffn(a["x"], a["M"], a["H"], a["wg"], a["wu"], a["F"], a["act"], a["dtype"], a["h"], a["pre"],
                                 a["ws"], a["wsb"], None)


def test_gated_ffn_rejects_bad_arguments(lib):
    assert _ffn(lib, dtype=1) == -2
    for bad in (dict(M=-1), dict(H=0), dict(H=508), dict(F=4), dict(act=2), dict(act=-1), dict(x=None), dict(wg=None),
                dict(wu=None), dict(h=None), dict(x=FAKE_MIS), dict(pre=FAKE_MIS), dict(M=2 ** 31 - 1, F=2 ** 31 - 8)):
        assert _ffn(lib, **bad) == -1, bad
    assert _ffn(lib) == -4
    need = lib.dflash2_gated_ffn_workspace_bytes(16, 512, 1024, 0)
    assert _ffn(lib, ws=FAKE, wsb=need - 1) == -4
    assert _ffn(lib, ws=FAKE_MIS, wsb=need) == -1
    assert _ffn(lib, M=0, x=None, h=None) == 0


def test_gated_ffn_backward_rejects_bad_arguments(lib):
    def f(**kw):
        a = dict(dh=FAKE, pre=FAKE, x=FAKE, wg=FAKE, wu=FAKE, M=16, H=512, F=1024, act=1, dtype=0, dx=FAKE, dwg=FAKE,
                 dwu=FAKE, ws=None, wsb=0)
        a.update(kw)
        return lib.dflash2_gated_ffn_backward(a["dh"], a["pre"], a["x"], a["wg"], a["wu"], a["M"], a["H"], a["F"], a["act"],
                                              a["dtype"], a["dx"], a["dwg"], a["dwu"], a["ws"], a["wsb"], None)
    assert f(dtype=1) == -2
    for bad in (dict(dwg=None), dict(dwu=None), dict(dx=None, dwg=None, dwu=None), dict(dh=None), dict(pre=None),
                dict(x=None), dict(wg=None), dict(dh=FAKE_MIS), dict(dx=FAKE_MIS), dict(H=12)):
        assert f(**bad) == -1, bad
    assert f() == -4
    assert f(dx=None, wg=None, wu=None) == -4        # the weights only serve dx
    assert f(dwg=None, dwu=None, x=None) == -4       # x only serves the weights' gradients
    need = lib.dflash2_gated_ffn_workspace_bytes(16, 512, 1024, 1)
    assert need > lib.dflash2_gated_ffn_workspace_bytes(16, 512, 1024, 0)
    assert f(ws=FAKE, wsb=need - 1) == -4


def test_python_checks():
    torch = pytest.importorskip("torch")
    import dflash2_block_drafter_gb300 as d
    x = torch.zeros(4, 64, dtype=torch.bfloat16)
    w = torch.zeros(16, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="act"):
        d.dflash2_gated_ffn(x, w, w, act="relu")
    with pytest.raises(ValueError, match="CUDA"):
        d.dflash2_gated_ffn(x, w, w)
    with pytest.raises(ValueError, match="w_gate"):
        d.dflash2_gated_ffn(x, w, w[:8])
    with pytest.raises(ValueError, match="out holds"):
        d.dflash2_gated_ffn(x, w, w, out=torch.zeros(2, 16, dtype=torch.bfloat16))
    with pytest.raises(ValueError, match="pre"):
        d.dflash2_gated_ffn_backward(torch.zeros(4, 16, dtype=torch.bfloat16), w[:1], x, w, w)
    cache = torch.zeros(2, 1, 2, 1, 16 * 36, dtype=torch.uint8)
    k = torch.zeros(3, 1, 64, dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="cache must be"):
        d.dflash2_kv4_append(k, k, torch.zeros(3, dtype=torch.int64), cache, 32)
    with pytest.raises(ValueError, match="slots"):
        d.dflash2_kv4_append(k, k, torch.zeros(2, dtype=torch.int64), cache, 16)
    with pytest.raises(ValueError, match="heads"):
        d.dflash2_kv4_append(k.expand(3, 2, 64), k, torch.zeros(3, dtype=torch.int64), cache, 16)
    with pytest.raises(ValueError, match="bf16 CUDA"):
        d.dflash2_kv4_append(k, k, torch.zeros(3, dtype=torch.int64), cache, 16)
    with pytest.raises(ValueError, match="page_table"):
        d.dflash2_kv4_attention(torch.zeros(2, 1, 4, 64), cache, torch.zeros(1, 1, dtype=torch.int32),
                                torch.zeros(2, dtype=torch.int32), 16, 1.0)
