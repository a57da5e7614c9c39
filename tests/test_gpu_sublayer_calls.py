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
