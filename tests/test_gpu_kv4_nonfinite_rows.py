"""Rows with a NaN or an infinity entering the 4-bit cache: their group reads as NaN, every other group exactly."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import S, _dev, _host, _rows, torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("bad", [float("nan"), float("inf"), -float("inf")])
@pytest.mark.parametrize("T,heads,D", [(5, 1, 64), (40, 3, 128)])
@pytest.mark.parametrize("channel", [0, 13, 63])
def test_groups_that_are_not_finite(torch, T, heads, D, bad, channel):
    import dflash2_block_drafter_gb300 as d
    rng = np.random.default_rng(channel)
    page = 16
    k, v = _rows(rng, T, heads, D), _rows(rng, T, heads, D)
    want = [S.bf16(S.kv4_values(x)) for x in (k, v)]
    for x, w, at in ((k, want[0], 1), (v, want[1], T - 1)):
        x[at, heads - 1, D - 64 + channel] = bad
        w[at, heads - 1, D - 64:] = np.nan
    pages = -(-T // page)
    cache = d.dflash2_kv4_cache(pages, heads, D, page)
    slots = torch.arange(T, device="cuda")
    d.dflash2_kv4_append(_dev(torch, k), _dev(torch, v), slots, cache, page)
    for got, w in zip(d.dflash2_kv4_read(cache, slots, D, page), want):
        np.testing.assert_array_equal(_host(got), w)
    assert d.dflash2_poll_error() == 0


def test_a_group_of_nothing_else(torch):
    import dflash2_block_drafter_gb300 as d
    k = torch.full((2, 1, 64), float("nan"), dtype=torch.bfloat16, device="cuda")
    v = torch.full((2, 1, 64), float("inf"), dtype=torch.bfloat16, device="cuda")
    cache = d.dflash2_kv4_cache(1, 1, 64, 16)
    slots = torch.tensor([3, 9], device="cuda")
    d.dflash2_kv4_append(k, v, slots, cache, 16)
    kr, vr = d.dflash2_kv4_read(cache, slots, 64, 16)
    assert bool(kr.isnan().all()) and bool(vr.isnan().all())


def test_a_range_past_fp32(torch):
    """(Both ends are finite, their difference is not.)"""
    import dflash2_block_drafter_gb300 as d
    k = torch.ones(1, 2, 64, dtype=torch.bfloat16, device="cuda")
    k[0, 0, 5], k[0, 0, 6] = 3e38, -3e38
    cache = d.dflash2_kv4_cache(1, 2, 64, 16)
    slots = torch.zeros(1, dtype=torch.int64, device="cuda")
    d.dflash2_kv4_append(k, k, slots, cache, 16)
    for got in d.dflash2_kv4_read(cache, slots, 64, 16):
        assert bool(got[0, 0].isnan().all()) and bool((got[0, 1] == 1.0).all())
