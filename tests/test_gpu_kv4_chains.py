"""GPU: pages, rows and attention behind one another with nothing waited for between: each call reads what the call in front
of it has just written (slots, lengths, page table, cache), not what stood there before."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu

STEPS = 10


@pytest.mark.parametrize("B,G,Hq,Hkv,D,page", [(1, 3, 2, 1, 64, 16), (4, 16, 10, 2, 128, 32), (40, 5, 4, 1, 128, 16)])
def test_rounds_behind_one_another(torch, B, G, Hq, Hkv, D, page):
    import dflash2_block_drafter_gb300 as d
    from dflash2_block_drafter_gb300.layer import ContextPages
    rng = np.random.default_rng(B)
    g = torch.Generator(device="cuda").manual_seed(B)
    rnd = lambda *s: torch.randn(*s, generator=g, device="cuda").to(torch.bfloat16)
    width = 2 + STEPS * G // page
    change = rng.integers(0, G + 1, (STEPS, B))
    change[:, 0] = G
    change[5, B // 2] = -change[:5, B // 2].sum()  # done: its pages go back
    place = np.where(np.arange(G) < change[..., None], np.arange(G), -1)
    i32 = lambda x: torch.tensor(x, dtype=torch.int32, device="cuda")
    ch, pl = i32(change), i32(place)
    q, k, v = (rnd(STEPS, B, G, h, D) for h in (Hq, Hkv, Hkv))
    ws = torch.empty(d.dflash2_kv4_attention_workspace_bytes(B, G, Hq, Hkv, D, page, width), dtype=torch.uint8, device="cuda")

    def run(wait):
        pages = ContextPages(B, B * width, width, page)
        cache = d.dflash2_kv4_cache(B * width, Hkv, D, page)
        cache.fill_(255)
        outs = []
        torch.cuda.synchronize()
        for i in range(STEPS):
            slots, _ = pages.gain(ch[i], place=pl[i])
            wait()
            d.dflash2_kv4_append(k[i].view(B * G, Hkv, D), v[i].view(B * G, Hkv, D), slots.view(-1), cache, page)
            wait()
            outs.append(d.dflash2_kv4_attention(q[i], cache, pages.table, pages.lengths, page, D ** -0.5, workspace=ws))
            wait()
        torch.cuda.synchronize()
        return torch.stack(outs), pages

    want, pages = run(torch.cuda.synchronize)
    np.testing.assert_array_equal(pages.lengths.cpu().numpy(), change.sum(0))
    assert want.isfinite().all() and want.any()
    for _ in range(5):
        got, pages = run(lambda: None)
        assert torch.equal(got, want)
        np.testing.assert_array_equal(pages.lengths.cpu().numpy(), change.sum(0))
    assert d.dflash2_poll_error() == 0
