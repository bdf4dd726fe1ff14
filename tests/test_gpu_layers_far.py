"""What lies beyond 2^32 elements, compared to the oracle element by element:
codes, scales, values back and products; and gradients of a million tokens.
Tolerances as in test_gpu_mxfp4.py and test_gpu_embedding.py."""
import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say
from oracle import layers
from test_gpu_mxfp4 import U, check_product, check_quantized, f64, rand

pytestmark = pytest.mark.gpu

ROWS, WIDTH, TAIL = 140000, 32768, 64           # whole blocks of 32 rows


@pytest.fixture(scope="module")
def far():
    """(matrix of zeros but for its last rows, those rows)"""
    need_gpu()
    rng = np.random.default_rng(60)
    tail = rand(rng, (TAIL, WIDTH), torch.bfloat16) * torch.exp2(torch.from_numpy(rng.integers(-9, 9, size=(TAIL, 1))).float())
    tail = tail.bfloat16()
    big = torch.zeros(ROWS, WIDTH, dtype=torch.bfloat16, device="cuda")
    big[-TAIL:] = tail.cuda()
    assert big.numel() > 1 << 32
    yield big, tail
    del big
    torch.cuda.empty_cache()


def test_far_rows(far):
    gns = need_gpu()
    big, tail = far
    say("far rows: quantise")
    q = gns.mxfp4_quantize(big)
    check_quantized(gns.MXFP4(q.codes[-TAIL:], q.scales[-TAIL // 32:], (TAIL, WIDTH)), f64(tail))
    assert not q.codes[:-TAIL].any() and not q.scales[:-TAIL // 32].any()
    want = layers.mxfp4_values(*layers.mxfp4_quantize(f64(tail)))
    say("far rows: back")
    back = gns.mxfp4_dequantize(q)
    assert np.array_equal(f64(back[-TAIL:]), want) and not back[:-TAIL].any()
    del back
    rng = np.random.default_rng(61)
    x = rand(rng, (70, WIDTH), torch.bfloat16)
    qx = gns.mxfp4_quantize(x.cuda())
    vx = f64(gns.mxfp4_dequantize(qx, dtype=torch.float32))
    for m in (1, 16, 33, 70):                   # the far rows are those of the second factor ...
        say("far rows: product", m)
        for a in (gns.mxfp4_quantize(x[:m].cuda()), x[:m].cuda()):
            y = gns.mxfp4_matmul(a, q, dtype=torch.float32)
            check_product(y[:, -TAIL:], vx[:m], want, WIDTH, torch.float32)
            assert not y[:, :-TAIL].any()
    say("far rows: product of far rows")        # ... and of the first
    for dtype in (torch.float32, torch.bfloat16):
        y = gns.mxfp4_matmul(q, qx, dtype=dtype)
        check_product(y[-TAIL:], want, vx, WIDTH, dtype)
        assert not y[:-TAIL].any()
        held = f64(y[-TAIL:])
        gns.mxfp4_matmul(q, qx, out=y, accumulate=True)
        check_product(y[-TAIL:], want, vx, WIDTH, dtype, held)


def test_far_columns(far):
    """The transpose: the far rows are the last blocks of every row of codes."""
    gns = need_gpu()
    big, tail = far
    codes, scales = layers.mxfp4_quantize(f64(tail).T)
    say("far columns: quantise")
    for t in (gns.mxfp4_quantize(big, transposed=True), gns.mxfp4_quantize_both(big)[1]):
        assert t.shape == (WIDTH, ROWS)
        first = (ROWS - TAIL) // 2
        packed = t.codes[:, first:].cpu().numpy()               # the last of them are padding
        got = np.stack([packed & 15, packed >> 4], -1).reshape(WIDTH, -1)
        assert np.array_equal(got[:, :TAIL], codes) and not got[:, TAIL:].any()
        assert not t.codes[:, :first].any()
        blocks = t.scales.permute(0, 2, 1, 3).reshape(WIDTH, -1).cpu().numpy()
        at = (ROWS - TAIL) // 32
        assert np.array_equal(blocks[:, at:at + TAIL // 32], scales)
        assert not blocks[:, :at].any() and not blocks[:, at + TAIL // 32:].any()
    say("far columns: back")
    back = gns.mxfp4_dequantize(t)
    assert np.array_equal(f64(back[:, -TAIL:]), layers.mxfp4_values(codes, scales)) and not back[:, :-TAIL].any()


# sorts whose digits' counts take more than one step of the scan, of one and of two digits
@pytest.mark.parametrize("count,vocab,width", [(1000003, 131072, 12), (1100000, 700, 5)])
def test_a_million_tokens(count, vocab, width):
    gns = need_gpu()
    rng = np.random.default_rng(62)
    tokens = torch.from_numpy(np.minimum((vocab ** rng.random(count)).astype(np.int64) - 1, vocab - 1))
    tokens[rng.random(count) < 0.2] = -1
    g = rand(rng, (count, width), torch.bfloat16)
    say("a million tokens", count, vocab, width)
    got = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.full((vocab, width), float("nan"), device="cuda"))
    t, x = tokens[tokens >= 0], g[tokens >= 0].double()
    ref = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, t, x)
    size = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, t, x.abs())
    n = torch.bincount(t, minlength=vocab).double()
    # an fp32 sum of n terms in some order, its scale and its rounding
    assert torch.all((got.cpu().double() - ref).abs() <= (n[:, None] + 4) * U * size)
    again = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.empty(vocab, width, device="cuda"))
    assert torch.equal(got, again)
