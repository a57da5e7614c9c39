"""The gated feed-forward sublayer where x's rows are not whole lines of 128 bytes and the product is large enough
for them to be copied to ones that are; against float64, with the bounds of the other sizes."""
import pytest

from tests import test_gpu_ffn as T
from tests.test_gpu_ffn import torch  # noqa: F401 (fixture)

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("kind", ["silu", "gelu_tanh"])
@pytest.mark.parametrize("M,H,F", [(520, 1544, 4104), (1100, 2056, 2056)])
def test_rows_of_odd_pitch(torch, M, H, F, kind):
    T.test_forward(torch, M, H, F, kind)
    T.test_backward(torch, M, H, F, kind)


@pytest.mark.parametrize("M,H,F", [(300, 3136, 5120), (3600, 264, 520)])
def test_products_whose_last_round_is_cut_into_shares(torch, M, H, F):
    """80 tiles of 49 k-blocks (the round before is cut with the last four), 26 tiles of 160, 12 of 57."""
    T.test_forward(torch, M, H, F, "silu")
    T.test_backward(torch, M, H, F, "silu")
