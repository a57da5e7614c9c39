"""The sublayer calls' checks of shapes, before anything looks at a device (CPU only)."""
import pytest


def test_rows_of_other_dimensions_are_refused():
    """A tensor of more dimensions may walk its rows in any way (an expanded one holds fewer than it shows)."""
    torch = pytest.importorskip("torch")
    import dflash2_block_drafter_gb300 as d
    bf = torch.bfloat16
    cache = torch.zeros(2, 2, 2, 1, 16 * 36, dtype=torch.uint8)
    k, slots = torch.zeros(4, 2, 64, dtype=bf), torch.zeros(4, dtype=torch.int64)
    for v in (torch.zeros(1, 2, 64, dtype=bf).expand(1, 1, 4, 2, 64), torch.zeros(8, 64, dtype=bf), None):
        with pytest.raises(ValueError, match="v must be a tensor of 4 rows"):
            d._kv4_rows(v, "v", 4, 2, 64)
    with pytest.raises(ValueError, match="bf16 CUDA"):
        d.dflash2_kv4_append(k, k, slots, cache, 16)
    for t in (torch.zeros(3, 2, 2, 64, dtype=bf), torch.zeros(6, 1, 2, 64, dtype=bf), torch.zeros(1, 2, 3, 2, 64, dtype=bf)):
        with pytest.raises(ValueError, match=r"k_new must be a tensor of 6 rows of \[2, 64\] or \[2, 3\] of them"):
            d._kv4_rows(t, "k_new", 6, 2, 64, (2, 3))
    for t in (torch.zeros(6, 2, 64, dtype=bf), torch.zeros(2, 3, 2, 64, dtype=bf)):
        with pytest.raises(ValueError, match="bf16 CUDA"):  # (the shape is right)
            d._kv4_rows(t, "k_new", 6, 2, 64, (2, 3))
