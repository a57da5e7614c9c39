"""Sizes of the gated feed-forward near 2^31, as far as the host goes (CPU only)."""
import pytest


@pytest.fixture(scope="module")
def lib():
    from dflash2_block_drafter_gb300 import _build
    import dflash2_block_drafter_gb300 as pkg
    _build.build()
    return pkg.library()


def test_workspaces_of_the_largest_sizes(lib):
    size = lib.dflash2_gated_ffn_workspace_bytes
    up = lambda n, k: -(-n // k) * k
    fixed = size(1, 64, 64, 0)
    for M, H, F in ((2 ** 31 - 1, 8, 8), (2 ** 31 - 1, 64, 8), (1, 8, 2 ** 31 - 64), (1, 2 ** 31 - 64, 8), (5, 2 ** 30 + 8, 16)):
        x = 0 if H % 64 == 0 else up(M * up(H, 64) * 2, 256)
        assert size(M, H, F, 0) == fixed + x
        assert size(M, H, F, 1) == fixed + x + up(2 * M * up(F, 64) * 2, 256)
    for M, H, F in ((1, 8, 2 ** 31 - 8), (1, 2 ** 31 - 56, 8), (2 ** 31 - 1, 2 ** 31 - 64, 8)):
        assert size(M, H, F, 0) == 0 and size(M, H, F, 1) == 0
