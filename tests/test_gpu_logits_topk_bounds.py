"""GPU parity of candidates in rows where more tokens reach the first bound than can be ranked: a nearer bound from 1024 shares
of them, more lanes than are listed, and tokens that fall into few shares."""
import numpy as np
import pytest

from tests.test_gpu_kv4 import torch  # noqa: F401 (fixture)
from tests.test_gpu_logits_topk import _case, _check

pytestmark = pytest.mark.gpu


def _share(tokens):
    """Which of the 1024 shares each token falls into (a product's upper ten bits)."""
    return (tokens.astype(np.uint32) * np.uint32(0x9e3779b1)) >> np.uint32(22)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
@pytest.mark.parametrize("M,V", [(3, 248320), (200, 20011), (500, 20011), (500, 4000), (2, 1 << 20)])
def test_rows_of_few_values(torch, dtype, M, V):
    """One value, two, or a thousand equal best ones among others."""
    rng = np.random.default_rng(V)
    c = _case(rng, M, 1, V, dtype, history=20, bias=2, mask=0.9)
    x = c["logits"]
    x[::3] = 1.5
    x[1::3] = rng.integers(0, 2, (len(x[1::3]), V))
    x[2::3, V // 2:V // 2 + 3000:2] = 40.0
    _check(torch, c, 16)
    _check(torch, c, 1, want_out=False)
    _check(torch, c, 4, in_place=True)
    _check(torch, c, 7, in_place=True)


@pytest.mark.parametrize("dtype", ["float32", "bfloat16"])
def test_tokens_of_few_shares(torch, dtype):
    """A mask that allows tokens of 1, 3, 15 and 17 shares only: with 16 wanted the first three give no nearer bound."""
    rng = np.random.default_rng(5)
    V, shares = 1 << 21, (1, 3, 15, 17)
    c = _case(rng, 8, 1, V, dtype, penalties=False, mask=0.0)
    at = _share(np.arange(V))
    for m in range(8):
        c["mask"][m] = at < shares[m % 4]
    assert c["mask"][0].sum() > 1500
    c["logits"][:4] = -2.0
    c["logits"][4:] = rng.integers(-3, 1, (4, V))
    _check(torch, c, 16, want_out=False)
    _check(torch, c, 3, in_place=True)
