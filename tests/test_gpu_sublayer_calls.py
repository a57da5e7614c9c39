"""How the sublayer calls take workspaces: of any type, and made by the call for another stream."""
import pytest

from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _attention(torch, d):
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    cache = d.dflash2_kv4_cache(8, 2, 64, 16)
    d.dflash2_kv4_append(rnd(128, 2, 64), rnd(128, 2, 64), torch.arange(128, device="cuda"), cache, 16)
    q, table = rnd(1, 4, 8, 64), torch.arange(8, dtype=torch.int32, device="cuda")[None]
    ctx = torch.tensor([128], dtype=torch.int32, device="cuda")
    need = d.dflash2_kv4_attention_workspace_bytes(1, 4, 8, 2, 64, 16, 8)
    return need, lambda **kw: d.dflash2_kv4_attention(q, cache, table, ctx, 16, 0.125, **kw)


def test_an_attention_workspace_of_any_type(torch):
    import dflash2_block_drafter_gb300 as d
    need, call = _attention(torch, d)
    want = call()
    for dt in (torch.float32, torch.int64, torch.uint8):
        size = torch.empty(0, dtype=dt).element_size()
        assert torch.equal(want, call(workspace=torch.empty(-(-need // size), dtype=dt, device="cuda")))
    assert d.dflash2_poll_error() == 0


@pytest.mark.parametrize("handle", [False, True])
@pytest.mark.parametrize("which", ["attention", "ffn", "ffn backward", "read"])
def test_what_a_call_makes_belongs_to_its_stream(torch, which, handle, monkeypatch):
    """A call on a stream that was named: its workspace and results are no memory that the current stream still uses,
    and are not given out to the current stream while the named one is busy."""
    import dflash2_block_drafter_gb300 as d
    g = torch.Generator(device="cuda").manual_seed(0)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda", dtype=torch.float32).to(torch.bfloat16)
    if which == "attention":
        need, f = _attention(torch, d)
        names, call = ("workspace", "out"), lambda s: f(stream=s)
    elif which == "read":
        cache = d.dflash2_kv4_cache(256, 8, 128, 64)
        cache.zero_()
        slots = torch.arange(256 * 64, device="cuda")
        need = 2 * 256 * 64 * 8 * 128 * 2
        names, call = ("k", "v"), lambda s: d.dflash2_kv4_read(cache, slots, 128, 64, stream=s)
    else:
        M, H, F = 300, 256, 512
        x, wg, wu, dh = rnd(M, H), rnd(F, H), rnd(F, H), rnd(M, F)
        h, pre = d.dflash2_gated_ffn(x, wg, wu, want_pre=True)
        need = d.dflash2_gated_ffn_workspace_bytes(M, H, F, int(which == "ffn backward"))
        if which == "ffn":
            names, call = ("workspace", "out", "pre"), lambda s: d.dflash2_gated_ffn(x, wg, wu, want_pre=True, stream=s)
        else:
            names = "workspace", "dx", "dw_gate", "dw_up"
            call = lambda s: d.dflash2_gated_ffn_backward(dh, pre, x, wg, wu, stream=s)
    side = torch.cuda.Stream()
    stream = side.cuda_stream if handle else side
    used, dev = {}, d._dev

    def spy(t, name, *rest):
        if t is not None and name in names:
            used[name] = (t.data_ptr(), t.data_ptr() + t.numel() * t.element_size())
        return dev(t, name, *rest)

    monkeypatch.setattr(d, "_dev", spy)
    apart = lambda t: all(t.data_ptr() + t.numel() <= a or t.data_ptr() >= b for a, b in used.values())
    torch.cuda.synchronize()
    # the current stream's: freed, and still in use there
    torch.cuda._sleep(100_000_000)  # some 50 ms
    busy = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, need, 4096, 4096, 1 << 21)]
    spans = [(t.data_ptr(), t.numel()) for t in busy]
    del busy
    call(stream)
    assert sorted(used) == sorted(names) and not torch.cuda.current_stream().query()
    assert all(p + n <= a or p >= b for a, b in used.values() for p, n in spans)
    torch.cuda.synchronize()
    # the named stream's: the call before it is done
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
    call(stream)
    later = [torch.empty(n, dtype=torch.uint8, device="cuda") for n in (need, need, 4096, 4096, 1 << 21)]
    assert not side.query() and all(apart(t) for t in later)
    torch.cuda.synchronize()
    assert d.dflash2_poll_error() == 0
