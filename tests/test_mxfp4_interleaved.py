"""Products whose matrices lie row by row beside one another ([rows, batch,
columns], as tokens by heads or by experts do), which overlap nowhere."""
import ctypes
import os

import pytest
import torch

gns = pytest.importorskip("gram_newton_schulz_amd")

from gpu_common import need_gpu, say  # noqa: E402
from gram_newton_schulz_amd.layers import Matrix  # noqa: E402

A, B, W = (0x100000000000 + i * 0x10000000000 for i in range(3))     # far apart, never dereferenced
SHAPE, ALIAS = 2, 7


@pytest.mark.skipif(not os.path.exists(gns.LIB_PATH), reason="libgns.so not built (run __graft_entry__.build())")
@pytest.mark.parametrize("linear", [False, True])
def test_what_overlaps_is_refused(linear):
    """Of 3 matrices of 40 x 70 results, over the factors' own memory: the
    layouts without overlaps are refused for that only."""
    a, b = (Matrix(at, at + (1 << 36), 3, rows, 200) for at, rows in ((A, 40), (B, 70)))

    def call(pitch, stride):
        tail = (B, 1, pitch, stride, 0, W, 1 << 40, None)
        if linear:
            return gns.lib().gns_mxfp4_linear(A, 1, 200, 8000, 40, ctypes.byref(b), *tail)
        return gns.lib().gns_mxfp4_matmul(ctypes.byref(a), ctypes.byref(b), *tail)

    for apart in ((70, 2800), (100, 3970), (210, 70), (211, 70), (212, 71), (300, 115)):
        assert call(*apart) == ALIAS, apart
    for overlapping in ((209, 70), (210, 69), (211, 71), (69, 2800), (70, 2799), (210, 0), (140, 70), (300, 116)):
        assert call(*overlapping) == SHAPE, overlapping


# of every kernel: few rows, 128-edge tiles and their parts, 64 x 256, 256-edge
@pytest.mark.gpu
@pytest.mark.parametrize("batch,m,n,k", [(3, 5, 70, 300), (3, 130, 77, 300), (2, 65, 70, 8192), (64, 40, 1000, 64),
                                         (2, 1900, 3333, 65)])
def test_interleaved_results(batch, m, n, k):
    need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(batch + m)
    x, w = (torch.empty(batch, rows, k, device="cuda").normal_(0.0, 1.0, generator=gen) for rows in (m, n))
    qx, qw = gns.mxfp4_quantize(x), gns.mxfp4_quantize(w)
    for dtype in (torch.float32, torch.bfloat16):
        for accumulate in (False, True):
            for a in (qx, x):
                say("interleaved results", batch, m, n, k, dtype, accumulate)
                buf = torch.full((m, batch, n + 3), 2.0, dtype=dtype, device="cuda")
                plain = torch.full((batch, m, n), 2.0, dtype=dtype, device="cuda")
                gns.mxfp4_matmul(a, qw, out=plain, accumulate=accumulate)
                out = buf[:, :, 1:n + 1].transpose(0, 1)
                assert gns.mxfp4_matmul(a, qw, out=out, accumulate=accumulate) is out
                assert torch.equal(out, plain)
                assert (buf[:, :, 0] == 2).all() and (buf[:, :, n + 1:] == 2).all()
