"""Host side of the operators over pages (no GPU needed)."""
import pytest


@pytest.fixture(scope="module")
def hs():
    import __graft_entry__ as g
    g.build()
    import tiered_sparse_mla_gb300 as hs
    return hs


@pytest.mark.parametrize("B,T,H", [(1, 65536, 65536), (1, 65536, 65537), (1, 32768, 1), (1, 32767, 300), (65536, 1, 1),
                                   (65535, 1, 32769), (1, 1, 128 * 65535 + 1), (2 ** 31 - 1, 2 ** 31 - 1, 2 ** 31 - 1),
                                   (-1, 1, 1), (1, -5, 1), (1, 1, 0)])
def test_no_workspace_for_sizes_that_are_refused(hs, B, T, H):
    """Products of sizes past 32 bits are refused before a plan is made from them."""
    for N in (1, 64, 2 ** 31 - 1):
        assert hs.hs_page_decode_workspace_bytes(B, T, H, N) == 0


def test_workspace_of_the_largest_sizes(hs):
    for B, T, H in ((65535, 1, 32768), (1, 32767, 256), (255, 64, 128), (65535, 32767, 1)):
        for N in (1, 1000, 2 ** 31 - 1):
            n = hs.hs_page_decode_workspace_bytes(B, T, H, N)
            # partials of at most 128 splits of all rows
            assert 0 <= n <= 128 * (B * T * H * (512 * 4 + 4) + 512)
