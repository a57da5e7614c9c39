"""GPU: candidates one call behind the other in one workspace, nothing waited for between, each call naming other tokens: a
call's second kernel reads what its first has written, not what the call before left there."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)
from tests.test_gpu_logits_topk import _args, _case

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,rows,V,history,ragged", [(1, 1, 2000, 30, False), (3, 5, 1500, 400, True), (40, 4, 3000, 60, False),
                                                     (200, 3, 600, 40, True)])
def test_calls_behind_one_another_in_one_workspace(torch, captured, B, rows, V, history, ragged):
    import dflash2_block_drafter_gb300 as d
    K, calls = 8, []
    for i in range(6):
        c = _case(np.random.default_rng(i), B, rows, V, "bfloat16" if i % 2 else "float32", history, "tree", ragged, 3, 0.7)
        calls.append((c, *_args(torch, c)))
    size = max(d.dflash2_logits_topk_workspace_bytes(c["M"], V, B, c["ragged"], history, True, 3, K) for c, _, _ in calls)
    ws = torch.empty(size, dtype=torch.uint8, device="cuda")
    want = []
    for c, x, kw in calls:
        fresh = torch.empty(size, dtype=torch.uint8, device="cuda").fill_(255)
        torch.cuda.synchronize()
        want.append(d.dflash2_logits_topk(x, K, want_out=True, workspace=fresh, **kw))
        torch.cuda.synchronize()
    chain = lambda: [d.dflash2_logits_topk(x, K, want_out=True, workspace=ws, **kw) for _ in range(5) for _, x, kw in calls]
    if captured:
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            got = chain()
        for _ in range(10):
            graph.replay()
    else:
        got = chain()
    torch.cuda.synchronize()
    for i, g in enumerate(got):
        for x, y in zip(g, want[i % len(calls)]):
            assert torch.equal(x, y), f"call {i}"
    assert d.dflash2_poll_error() == 0


def test_spans_that_a_page_plan_has_just_written(torch):
    """The packed rows of each sequence's new tokens are its request's: row_offsets go from plan to candidates on the device."""
    import dflash2_block_drafter_gb300 as d
    from dflash2_block_drafter_gb300.layer import ContextPages
    rng = np.random.default_rng(2)
    B, G, V, K, steps = 30, 7, 3000, 4, 8
    M = B * G
    g = torch.Generator(device="cuda").manual_seed(1)
    x = torch.randn(M, V, generator=g, device="cuda")
    history = torch.randint(0, V, (B, 50), generator=g, device="cuda", dtype=torch.int32)
    full = torch.full((B,), 50, dtype=torch.int32, device="cuda")
    strong = torch.linspace(1.0, 3.0, B, device="cuda")
    gain = torch.tensor(rng.integers(0, G + 1, (steps, B)), dtype=torch.int32, device="cuda")

    def run(wait):
        pages = ContextPages(B, 40 * B, 40, 16)
        cand = torch.full((steps, M, K), -77, dtype=torch.int32, device="cuda")
        unary = torch.zeros(steps, M, K, device="cuda")
        torch.cuda.synchronize()
        for i in range(steps):
            pages.gain(gain[i], rows=M)
            wait()
            d.dflash2_logits_topk(x, K, requests=B, row_offsets=pages.offsets, history=history, history_len=full, repetition=strong,
                                  frequency=strong, cand=cand[i], unary=unary[i])
            wait()
        torch.cuda.synchronize()
        return cand, unary

    want = run(torch.cuda.synchronize)
    rows = gain.sum(1).tolist()
    for i, n in enumerate(rows):  # rows behind the last request are left as they were
        assert (want[0][i, :n] >= 0).all() and (want[0][i, n:] == -77).all()
    for _ in range(5):
        got = run(lambda: None)
        assert torch.equal(got[0], want[0]) and torch.equal(got[1], want[1])
    assert d.dflash2_poll_error() == 0
