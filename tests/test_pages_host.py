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


def test_kernels_launched_early_read_nothing_through_the_read_only_path():
    """A grid that may begin while the kernel before it still writes (it waits before it
    reads) must not read those writes through the read-only path, which may hold or fetch
    what was there before: const __restrict__ parameters, __ldg, ld.global.nc."""
    import glob
    import os
    import re
    import tiered_sparse_mla_gb300 as pkg
    found = 0
    for path in sorted(glob.glob(os.path.join(os.path.dirname(pkg.__file__), "csrc", "*.cu"))):
        with open(path) as f:
            text = re.sub(r"//[^\n]*", "", f.read())
        for kernel in text.split("__global__")[1:]:
            if "grid_dep_wait()" not in kernel:
                continue
            found += 1
            name = re.search(r"(\w+)\s*\((?!\()", re.sub(r"__launch_bounds__\([^;{]*?\)\s*\n?", "", kernel)).group(1)
            head = kernel[:kernel.index("{")]
            assert "__restrict__" not in head, f"{os.path.basename(path)}: {name}"
            assert not re.search(r"__ldg\(|ld_stream_v4\(|global\.nc", kernel), f"{os.path.basename(path)}: {name}"
    assert found >= 7
