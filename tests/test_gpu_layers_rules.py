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
