"""Calls on lists of tensors that are refused before anything reaches the GPU
(none needed here)."""
import os

import pytest

gns = pytest.importorskip("gram_newton_schulz_amd")
from test_tensor_lists_host import BASE, E, F32, build, norm  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(gns.LIB_PATH),
                                reason="libgns.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("arrays", [4, 5])
def test_clip_in_place_of_a_gradient_that_is_other_memory_of_the_list(arrays):
    """Clipping in place would scale the parameter, a moment or the copy too."""
    for other in range(1, arrays):
        for shift in (0, 28):                      # the same memory, its last element only
            lists = [[(BASE + 4096 * a, 1, 8, 8, F32)] for a in range(arrays)]
            lists[other] = [(BASE + shift, 1, 8, 8, F32)]
            assert norm(build(lists)[1], clip=True) == E["ALIAS"], (other, shift)
