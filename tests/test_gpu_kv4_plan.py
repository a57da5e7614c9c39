"""GPU parity of the page plan: every output, the page table and the ring of free pages, whole numbers throughout."""
import numpy as np
import pytest

from oracle import tree_oracle as T
from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


def _case(rng, B, page, ctx_max, grow, finish=0.2, short=1.0, spare=3):
    """(ctx, change, table, queue, state, pages): shuffled pages, a ring that starts anywhere."""
    ctx = rng.integers(0, ctx_max + 1, B)
    change = np.where(rng.random(B) < finish, -rng.integers(0, ctx + 1), rng.integers(0, grow + 1, B))
    used = -(-ctx // page)
    need = int(np.maximum(0, -(-(ctx + change) // page) - used).sum())
    pages = int(used.sum()) + need + spare
    order = rng.permutation(pages)
    width = -(-(ctx_max + grow) // page) + 1
    table = np.full((B, width), -7)
    at = 0
    for b, n in enumerate(used):
        table[b, :n] = order[at:at + n]
        at += n
    free = order[at:][:max(0, int((need + spare) * short))]
    Q = pages + int(rng.integers(0, 4))
    head = int(rng.integers(0, Q))
    queue = np.full(Q, -5)
    queue[(head + np.arange(free.size)) % Q] = free
    return ctx, change, table, queue, (head, free.size), pages


def _i32(torch, x):
    return torch.tensor(np.asarray(x), dtype=torch.int32, device="cuda")


def _check(torch, case, page, rows=None, place=None, in_place=False):
    import dflash2_block_drafter_gb300 as d
    ctx, change, table, queue, state, pages = case
    want = T.plan(ctx, change, table, queue, state, page, pages, rows, place)
    c, t, q, s = _i32(torch, ctx), _i32(torch, table), _i32(torch, queue), _i32(torch, state)
    kw = dict(ctx_out=c, state_out=s) if in_place else {}
    got = d.dflash2_kv4_plan(c, _i32(torch, change), t, q, s, page, pages, rows=rows or 0,
                             place=None if place is None else _i32(torch, place), **kw)
    err = d.dflash2_poll_error()
    assert (err == 0 and not want["bad"]) or err in want["bad"], (err, want["bad"])
    for name, x in zip(("ctx", "state", "offsets", "slots", "positions", "table", "queue"), got + (t, q)):
        np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=name)
    return want


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("B,page,ctx_max,grow,rows", [(1, 16, 0, 1, 1), (1, 64, 100, 5000, 5001), (3, 16, 40, 33, 80),
                                                      (64, 64, 900, 16, 1100), (1000, 32, 200, 7, 9000),
                                                      (1025, 16, 50, 3, 5000), (8192, 256, 600, 2, 20000)])
def test_packed_rows(torch, B, page, ctx_max, grow, rows, in_place):
    rng = np.random.default_rng(B + page)
    _check(torch, _case(rng, B, page, ctx_max, grow), page, rows, in_place=in_place)


@pytest.mark.parametrize("B,G", [(1, 1), (5, 16), (64, 64), (700, 13)])
def test_rows_in_places(torch, B, G):
    rng = np.random.default_rng(B * G)
    case = _case(rng, B, 32, 300, G)
    keep = rng.random((B, G)) < 0.5
    place = np.where(keep, np.cumsum(keep, 1) - 1, rng.integers(-3, 0, (B, G)))
    place[0, 0] = 2 ** 31 - 1  # behind what any sequence gains
    want = _check(torch, case, 32, place=place, in_place=True)
    assert B < 5 or (want["slots"] >= 0).any()


@pytest.mark.parametrize("short", [0.0, 0.3, 0.8])
def test_pages_run_short(torch, short):
    """From the first sequence that finds too few on, those that need pages are refused, and no others."""
    rng = np.random.default_rng(11)
    for B in (2, 40, 2000):
        case = _case(rng, B, 16, 100, 60, short=short)
        want = _check(torch, case, 16, rows=B * 60)
        assert B < 40 or (want["ctx"] == case[0])[case[1] > 16].any()


@pytest.mark.parametrize("rows", [0, 1, 57, 1500])
def test_rows_run_short(torch, rows):
    _check(torch, _case(np.random.default_rng(rows), 100, 16, 100, 40), 16, rows=rows)


def test_bad_lengths_states_and_pages_are_recorded(torch):
    rng = np.random.default_rng(5)
    base = _case(rng, 50, 16, 100, 40, finish=0.3)
    cap = base[2].shape[1] * 16
    for b, (L, c) in enumerate([(-1, 5), (cap + 1, 0), (5, -6), (cap - 3, 4), (2 ** 31 - 1, 2 ** 31 - 1), (-2 ** 31, -2 ** 31)]):
        ctx, change, *rest = (x.copy() if isinstance(x, np.ndarray) else x for x in base)
        ctx[7 * b], change[7 * b] = L, c
        want = _check(torch, (ctx, change, *rest), 16, rows=3000)
        assert -1 in want["bad"]
    Q = base[3].size
    for state in ((-1, 3), (Q, 3), (0, Q + 1), (3, -1)):
        want = _check(torch, (*base[:4], state, base[5]), 16, rows=3000)
        assert -1 in want["bad"] and (want["ctx"] == base[0]).all()
    # a ring without room for what comes back
    want = _check(torch, (np.array([40, 40]), np.array([-40, -8]), np.array([[1, 2, 3], [4, 5, 6]]), np.arange(4), (1, 1), 9),
                  16, rows=3)
    assert want["ctx"].tolist() == [0, 40] and -1 in want["bad"]
    # pages that the cache does not have, waiting or in a table
    want = _check(torch, (np.array([3, 20]), np.array([30, -20]), np.array([[1, 0, 0], [99, 2, 0]]), np.array([98, 4, 0, 0]),
                          (0, 2), 9), 16, rows=40)
    assert want["bad"] == {-6} and (want["slots"][:30] >= 0).sum() < 30


def test_a_captured_plan_steps_through_a_conversation(torch):
    """In place, replayed: lengths, pages and free pages go on from replay to replay, as the oracle's do."""
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(6)
    B, page, rows = 20, 16, 200
    ctx, change, table, queue, state, pages = _case(rng, B, page, 60, 9, finish=0.0, spare=150)
    table = np.concatenate([table, np.full((B, 40), -7)], 1)
    c, t, q, s = _i32(torch, ctx), _i32(torch, table), _i32(torch, queue), _i32(torch, state)
    ch = _i32(torch, change)
    off = torch.empty(B + 1, dtype=torch.int32, device="cuda")
    slots = torch.empty(rows, dtype=torch.int64, device="cuda")
    pos = torch.empty(rows, dtype=torch.int32, device="cuda")
    call = lambda: d.dflash2_kv4_plan(c, ch, t, q, s, page, pages, rows=rows, ctx_out=c, state_out=s, offsets=off,
                                      slots=slots, positions=pos)
    ch.zero_()
    call()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        call()
    for step in range(12):
        change = rng.integers(0, 10, B)
        change = np.where(rng.random(B) < 0.3, -rng.integers(0, ctx + 1), change)
        want = T.plan(ctx, change, table, queue, state, page, pages, rows)
        ch.copy_(_i32(torch, change))
        graph.replay()
        torch.cuda.synchronize()
        for name, x in zip(("ctx", "state", "offsets", "slots", "positions", "table", "queue"), (c, s, off, slots, pos, t, q)):
            np.testing.assert_array_equal(x.cpu().numpy(), want[name], err_msg=f"{name}, step {step}")
        ctx, table, queue, state = want["ctx"], want["table"], want["queue"], tuple(want["state"])
    assert d.dflash2_poll_error() == 0
