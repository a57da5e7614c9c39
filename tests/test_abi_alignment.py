"""Host: arrays that are not aligned to their element type are refused before anything is launched (no GPU). The kernels would
fault on them."""
import ctypes

import pytest

from tests.test_abi_sublayer import _append, _attention, lib  # noqa: F401 (fixture)
from tests.test_abi_trees import _pick, _plan, _tree


def _off(n):
    return ctypes.c_void_p(0x10000 + n)


@pytest.mark.parametrize("name", ["ctx", "change", "table", "queue", "state", "ctx_out", "state_out", "off", "pos", "place"])
def test_plan(lib, name):  # noqa: F811
    assert _plan(lib, **dict(dict(G=4) if name == "place" else {}, **{name: _off(2)})) == -1


def test_plan_slots_are_64_bits(lib):  # noqa: F811
    assert _plan(lib, slots=_off(4)) == -1


@pytest.mark.parametrize("name", ["table", "ctx"])
def test_attention(lib, name):  # noqa: F811
    assert _attention(lib, **{name: _off(2)}) == -1
    assert _tree(lib, **{name: _off(1)}) == -1
    assert _tree(lib, par=_off(2)) == -1


def test_cache_rows(lib):  # noqa: F811
    assert _append(lib, slots=_off(4)) == -1
    a = ctypes.c_void_p(0x10000)
    assert lib.dflash2_kv4_read(a, _off(4), 4, 8, 128, 64, 4, 0, a, a, None) == -1


@pytest.mark.parametrize("name", ["hist", "prompt", "length", "rep", "freq", "pres", "tokens", "parents", "ids", "bias", "mask",
                                  "cand", "unary", "off"])
def test_candidates(lib, name):  # noqa: F811
    assert _pick(lib, **{name: _off(2)}) == -1
