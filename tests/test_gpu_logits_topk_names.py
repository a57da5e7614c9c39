"""GPU parity of candidates whose requests name more tokens than a row's CTA keeps in shared memory (8 for each of its 1024, 512,
256 or 128 threads): those behind are computed again for each look, after part of `out` has been stored, which may be the
logits themselves. And rows where more reach the bound than can be ranked at once, with such names."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)
from tests.test_gpu_logits_topk import _case, _check

pytestmark = pytest.mark.gpu

# (requests, rows each, vocabulary, history): 1024, 512, 256 and 128 threads a row
SIZES = [(2, 3, 40000, 30000), (100, 2, 20011, 9000), (100, 5, 20011, 6000), (100, 5, 4000, 8000)]
KEPT = [8192, 4096, 2048, 1024]


def _named(rng, size, dtype, tokens="tree", **kw):
    """A case whose histories are drawn evenly over the vocabulary, full in every other request."""
    B, rows, V, n = size
    c = _case(rng, B, rows, V, dtype, n, tokens, False, 5, **kw)
    c["history"] = np.stack([rng.permutation(V)[:n] if n <= V else rng.integers(0, V, n) for _ in range(B)]).astype(np.int32)
    c["length"][::2] = n
    c["prompt"] = (c["length"] * rng.random(B)).astype(np.int32)
    return c


def _names(c, b):
    return len(np.unique(c["history"][b, :c["length"][b]]))


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size,kept", list(zip(SIZES, KEPT)))
def test_more_names_than_are_kept(torch, dtype, size, kept):
    rng = np.random.default_rng(kept)
    c = _named(rng, size, dtype, mask=0.8)
    assert _names(c, 0) > kept
    _check(torch, c, 16)
    _check(torch, c, 16, in_place=True)
    _check(torch, c, 5, want_out=False)
    _check(torch, c, 0)
    _check(torch, c, 0, in_place=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("size,kept", list(zip(SIZES, KEPT)))
def test_equal_values_and_more_names_than_are_kept(torch, dtype, size, kept):
    """Every token's value is the same, or one of three, or named tokens fall below the others: far more than 1024 tokens reach
    any bound."""
    rng = np.random.default_rng(kept + 1)
    c = _named(rng, size, dtype, mask=0.9)
    M, V = c["M"], c["V"]
    for k, still in (("rep", 1.0), ("freq", 0.0), ("pres", 0.0)):
        c[k][::4] = still
    c["freq"][2::4], c["pres"][2::4], c["rep"][2::4] = 0.0, 2.0, 1.5
    c["logits"][:] = 1.5
    c["logits"][1::3] = rng.integers(-1, 2, (len(c["logits"][1::3]), V))
    c["mask"][::7] = True
    _check(torch, c, 16)
    _check(torch, c, 16, in_place=True)
    _check(torch, c, 1, want_out=False)
    _check(torch, c, 4, in_place=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("V,n", [(32771, 30000), (50257, 32768)])
def test_long_generated_histories_under_strong_penalties(torch, dtype, V, n):
    """Lanes without a named token are few, and penalised tokens' own logits reach the weak bound that is left: more lanes, or
    more values, than are listed at once."""
    rng = np.random.default_rng(V)
    B = 6
    c = _case(rng, B, 3, V, dtype, n, None)
    c["length"][:], c["prompt"][:] = n, 0
    c["rep"][:], c["freq"][:], c["pres"][:] = 1.5, [1.0, 1.0, 2.0, 1.0, 0.5, 2.0], [1.0, 1.0, 2.0, 0.0, 0.5, 1.0]
    x = 2 * rng.standard_normal((c["M"], V)) - 0.4 * np.log1p(np.arange(V))  # (logits fall with the token, as its frequency does)
    c["logits"] = torch.from_numpy(x).to(getattr(torch, dtype)).float().numpy()
    _check(torch, c, 16, want_out=False)
    _check(torch, c, 16, in_place=True)
    _check(torch, c, 5)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_more_names_than_are_kept_over_a_vocabulary_of_two_windows(torch, dtype):
    rng = np.random.default_rng(3)
    c = _named(rng, (2, 2, 300001, 40000), dtype, mask=0.7)
    assert (c["history"][0] < 2 ** 18).sum() > 8192 and (c["history"][0] >= 2 ** 18).any()
    _check(torch, c, 16)
    _check(torch, c, 16, in_place=True)
    c["logits"][:] = -0.5
    c["rep"][0], c["freq"][0], c["pres"][0] = 1.0, 0.0, 0.0
    _check(torch, c, 16, in_place=True)
    _check(torch, c, 3)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_the_largest_vocabulary(torch, dtype):
    c = _case(np.random.default_rng(4), 2, 1, 1 << 22, dtype, 500, "tree", bias=40, mask=0.9)
    c["ids"][0, 0], c["bias"][0, 0] = (1 << 22) - 1, 30.0
    _check(torch, c, 16, pad=1, shift=3)
    _check(torch, c, 2, in_place=True)
