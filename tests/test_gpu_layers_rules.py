"""Products at the sizes between which the library's rules choose.  Tolerances
as in test_gpu_mxfp4.py."""
import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say
from test_gpu_mxfp4 import check_product, f64, rand

pytestmark = pytest.mark.gpu


# 191 to 256 tiles of 64 x 256
@pytest.mark.parametrize("batch,m,n,k", [(1, 48, 48896, 130), (1, 33, 48897, 64), (1, 64, 50257, 130), (28, 48, 2048, 200),
                                         (255, 40, 250, 65), (1, 63, 65281, 64)])
def test_few_rows_by_many(batch, m, n, k):
    gns = need_gpu()
    rng = np.random.default_rng(m + n)
    x, w = rand(rng, (batch, m, k), torch.bfloat16, wide=True), rand(rng, (batch, n, k), torch.float32)
    qx, qw = gns.mxfp4_quantize(x.cuda()), gns.mxfp4_quantize(w.cuda())
    vx, vw = (f64(gns.mxfp4_dequantize(q, dtype=torch.float32)) for q in (qx, qw))
    for dtype in (torch.float32, torch.bfloat16):
        say("few rows by many", batch, m, n, k, dtype)
        check_product(gns.mxfp4_matmul(qx, qw, dtype=dtype), vx, vw, k, dtype)
        old = rand(rng, (batch, m, n), dtype)
        check_product(gns.mxfp4_matmul(x.cuda(), qw, out=old.cuda(), accumulate=True), vx, vw, k, dtype, f64(old))


# quantised in the product, and before it, by the same sizes but for one
@pytest.mark.parametrize("batch,m,n,k", [(1, 2, 65536, 4096), (1, 2, 131072, 4096), (1, 8, 4096, 4096), (1, 8, 9000, 4090),
                                         (1, 16, 4096, 4096), (1, 16, 4097, 4096), (1, 16, 20000, 1000), (64, 4, 1024, 2048),
                                         (64, 1, 2048, 2048), (3, 5, 33000, 300)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_few_plain_rows_are_their_quantised_form(batch, m, n, k, dtype):
    gns = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(m + n)
    x = torch.empty(batch, m, k, device="cuda").normal_(0.0, 1.0, generator=gen).to(dtype)
    w = gns.mxfp4_quantize(torch.empty(batch, n, k, device="cuda").normal_(0.0, 1.0, generator=gen))
    say("few plain rows", batch, m, n, k, dtype)
    got = gns.mxfp4_matmul(x, w, dtype=torch.float32)
    assert torch.equal(got, gns.mxfp4_matmul(gns.mxfp4_quantize(x), w, dtype=torch.float32))
    rows = slice(n - 300, n)                     # of B, to the oracle's tolerance
    va, vb = (f64(gns.mxfp4_dequantize(q, dtype=torch.float32)) for q in (gns.mxfp4_quantize(x), w))
    check_product(got[:, :, rows], va, vb[:, rows], k, torch.float32)
