"""bench.py's timing of the layers' operators keeps their data out of the
last-level cache where it says so."""
import os
import sys

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, ROOT)
import bench  # noqa: E402


def test_copies_fill_the_cache_twice():
    for nbytes in (36e6, 37748736.0, 64 << 20, 200 << 20, 806e6):
        copies = bench.layer_copies(nbytes)
        assert 3 <= copies <= 16 and copies * nbytes >= 512 << 20
    # between two calls on the same copy all others' data has passed
    assert (bench.layer_copies(36e6) - 1) * 36e6 > 256 << 20


def test_small_calls_have_a_few_copies():
    assert bench.layer_copies(1.1e6) == bench.layer_copies(0) == 16
