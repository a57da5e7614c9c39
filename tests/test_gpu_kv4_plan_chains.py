"""GPU: page plans in place, one behind the other with nothing waited for between: lengths, free pages and their state are each
call's inputs and outputs. One CTA, and the cluster's eight."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)
from tests.test_gpu_kv4_plan import _case, _i32

pytestmark = pytest.mark.gpu

STEPS = 9


@pytest.mark.parametrize("captured", [False, True])
@pytest.mark.parametrize("B,page,rows,place", [(1, 16, 7, 0), (60, 32, 700, 0), (20, 16, 8000, 0), (3000, 16, 30000, 0),
                                               (8192, 64, 80000, 0), (64, 32, 0, 16), (900, 16, 0, 10)])
def test_a_chain_of_plans_in_place(torch, captured, B, page, rows, place):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(B + rows)
    grow = place or 9
    ctx, change, table, queue, state, pages = _case(rng, B, page, 60, grow, finish=0.0, spare=B * (1 + STEPS * grow // page))
    table = np.concatenate([table, np.full((B, 2 + STEPS * grow // page), -7)], 1)
    c, t, q, s = _i32(torch, ctx), _i32(torch, table), _i32(torch, queue), _i32(torch, state)
    # each step's change and places, and outputs
    changes, places, lengths = [], [], ctx.astype(int)
    for _ in range(STEPS):
        x = rng.integers(0, grow + 1, B)
        x = np.where(rng.random(B) < 0.3, -rng.integers(0, lengths + 1), x)
        lengths = lengths + x
        changes.append(x)
        keep = rng.random((B, place)) < 0.5
        places.append(np.where(keep, np.cumsum(keep, 1) - 1, -1) if place else None)
    ch = _i32(torch, np.stack(changes))
    pl = _i32(torch, np.stack(places)) if place else None
    shape = (STEPS, B, place) if place else (STEPS, rows)
    slots = torch.empty(shape, dtype=torch.int64, device="cuda")
    pos = torch.empty(shape, dtype=torch.int32, device="cuda")
    off = torch.empty((STEPS, B + 1), dtype=torch.int32, device="cuda")

    def chain():
        for i in range(STEPS):
            d.dflash2_kv4_plan(c, ch[i], t, q, s, page, pages, rows=rows, place=pl[i] if place else None, ctx_out=c, state_out=s,
                               offsets=off[i], slots=slots[i], positions=pos[i])

    if captured:
        start = [x.clone() for x in (c, t, q, s)]
        chain()
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            chain()
        for x, y in zip((c, t, q, s), start):
            x.copy_(y)
        graph.replay()
    else:
        chain()
    torch.cuda.synchronize()
    for i in range(STEPS):
        want = T.plan(ctx, changes[i], table, queue, state, page, pages, rows if not place else None, places[i])
        assert not want["bad"]
        for name, x in (("offsets", off[i]), ("slots", slots[i]), ("positions", pos[i])):
            np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=f"{name}, step {i}")
        ctx, table, queue, state = want["ctx"], want["table"], want["queue"], tuple(want["state"])
    for name, x in zip(("ctx", "state", "table", "queue"), (c, s, t, q)):
        np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=name)
    assert d.dflash2_poll_error() == 0


def test_gains_past_32_bits_together(torch):
    """Rows in places: each sequence's gain fits, all together pass what row_offsets can count, so the last is refused."""
    import dflash2_block_drafter_gb300 as d
    page, width, pages = 4096, 300000, 700000
    gain = [10 ** 9, 10 ** 9, 5 * 10 ** 8, 0, -3]
    ctx = _i32(torch, [0, 5, 7, 9, 4])
    table = torch.full((5, width), -7, dtype=torch.int32, device="cuda")
    table[:, 0] = _i32(torch, [0, 1, 2, 3, 4])
    queue = torch.arange(pages, dtype=torch.int32, device="cuda")
    place = _i32(torch, [[gain[0] - 1, 0], [0, gain[1] - 1], [0, 1], [0, 0], [0, 0]])
    before = table.clone()
    new, state, off, slots, pos = d.dflash2_kv4_plan(ctx, _i32(torch, gain), table, queue, _i32(torch, [5, pages - 5]), page, pages,
                                                     place=place)
    assert d.dflash2_poll_error() == 0
    assert new.tolist() == [10 ** 9, 10 ** 9 + 5, 7, 9, 1]
    assert off.tolist() == [0, 10 ** 9, 2 * 10 ** 9, 2 * 10 ** 9, 2 * 10 ** 9, 2 * 10 ** 9]
    need = [-(-10 ** 9 // page), -(-(10 ** 9 + 5) // page) - 1]
    assert state.tolist() == [5 + sum(need), pages - 5 - sum(need)]
    assert pos.tolist() == [[10 ** 9 - 1, 0], [5, 10 ** 9 + 4], [-1, -1], [-1, -1], [-1, -1]]
    last = lambda b, p: int(table[b, p // page]) * page + p % page
    assert slots.tolist() == [[last(0, 10 ** 9 - 1), last(0, 0)], [page + 5, last(1, 10 ** 9 + 4)], [-1, -1], [-1, -1], [-1, -1]]
    assert torch.equal(table[0, :need[0]], torch.arange(5, 5 + need[0], dtype=torch.int32, device="cuda"))
    assert torch.equal(table[2:], before[2:])
