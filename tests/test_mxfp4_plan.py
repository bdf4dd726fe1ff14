"""How the library plans MXFP4 products, asked of its internal planner (no GPU):
no launch that the argument checks let through is larger than a grid may be."""
import ctypes
import os

import pytest

gns = pytest.importorskip("gram_newton_schulz_amd")

pytestmark = pytest.mark.skipif(not os.path.exists(gns.LIB_PATH),
                                reason="libgns.so not built (run __graft_entry__.build())")

T256, T128, T64 = 0, 1, 2
TILES = {T256: (256, 256, 512), T128: (128, 128, 256), T64: (64, 256, 256)}      # rows, columns, threads


def plan(batch, m, n, k):
    """(tile, parts of the contraction) of gns::mx_plan."""
    f = gns.lib()["_ZN3gns7mx_planEllll"]
    f.restype, f.argtypes = ctypes.c_uint64, [ctypes.c_int64] * 4
    packed = f(batch, m, n, k)
    return packed & 0xffffffff, packed >> 32


def up(a, b):
    return -(-a // b)


def threads(batch, m, n, k):
    tile, parts = plan(batch, m, n, k)
    rows, cols, each = TILES[tile]
    return batch * up(m, rows) * up(n, cols) * parts * each


@pytest.mark.parametrize("m", [33, 64, 65, 100, 128, 129, 256, 257, 384, 385, 1000])
@pytest.mark.parametrize("n", [1, 64, 128, 129, 256, 257, 300, 385, 5000])
def test_grids_of_many_matrices(m, n):
    """The most matrices of a size that the calls take (fewer than 2^24 tiles of
    128 x 128), and numbers around the half of that."""
    most = ((1 << 24) - 1) // (up(m, 128) * up(n, 128))
    for batch in (most, most // 2, most // 2 + 1, most // 2 + 2, 1 << 20, 1 << 10):
        for k in (1, 128, 8192):
            if batch <= most:
                assert threads(batch, m, n, k) < 1 << 32, (batch, m, n, k)


def test_plans_of_ordinary_sizes():
    assert plan(1, 8192, 16384, 4096) == (T256, 1)
    assert plan(64, 48, 2048, 7168) == (T64, 1)
    tile, parts = plan(1, 48, 4096, 16384)
    assert tile == T128 and parts > 1


@pytest.mark.parametrize("m", [33, 40, 48, 63, 64])
def test_few_rows_never_run_in_the_largest_tiles(m):
    """Three quarters of whose rows they would waste: 192 tiles of 64 x 256 and
    more are taken, fewer are 128-edge ones."""
    for batch, n in [(1, 256 * t) for t in range(150, 300)] + [(1, 50257), (1, 63000), (28, 2048), (200, 100), (255, 256)]:
        tile, _ = plan(batch, m, n, 4096)
        assert tile == (T64 if batch * up(n, 256) >= 192 else T128), (batch, n)


@pytest.mark.parametrize("batch,m,n,k,in_the_product", [
    (1, 1, 4096, 16384, True), (1, 1, 131072, 4096, True), (64, 1, 2048, 2048, True), (1, 2, 65536, 4096, True),
    (1, 8, 4096, 4096, True), (1, 16, 4096, 1024, True), (1, 16, 4096, 4096, True), (1, 16, 131072, 4096, False), (1, 8, 16384, 4096, False),
    (1, 4, 16384, 16384, False), (1, 16, 4112, 4096, False), (64, 4, 1024, 2048, False), (1, 2, 131072, 4096, False)])
def test_rows_that_many_workgroups_would_quantise_are_quantised_once(batch, m, n, k, in_the_product):
    """... in the workspace, which only that needs at up to 16 rows."""
    need = gns.mxfp4_matmul_workspace_bytes(batch, m, n, k, quantized=False)
    assert (need == 0) == in_the_product
    assert gns.mxfp4_matmul_workspace_bytes(batch, m, n, k) == 0
