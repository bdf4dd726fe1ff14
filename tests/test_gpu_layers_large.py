"""Sizes from which the layers' kernels run in another form: matrices of many
tiles, matrices that fill the last-level cache, tables of which most rows are
cleared, and runs of many partial sums.

Codes, scales and bits are compared exactly, against the oracle or against the
same call on parts; sums have test_gpu_embedding.py's tolerance.
"""
import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say
from test_gpu_embedding import check_grad, ids
from test_gpu_mxfp4 import check_quantized, f64, rand

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("noisy", [False, True])
def test_fp32_matrices_of_many_tiles(noisy):
    """600 tiles of 128 x 128, rows and columns that end inside one."""
    gns = need_gpu()
    rng = np.random.default_rng(50 + noisy)
    rows, cols = 2999, 3130
    x = rand(rng, (rows, cols), torch.float32, wide=True)
    r = torch.from_numpy(rng.integers(0, 256, size=x.shape).astype(np.uint8)) if noisy else None
    dr = None if r is None else r.cuda()
    say("quantize many tiles", noisy)
    both = gns.mxfp4_quantize_both(x.cuda(), noise=dr)
    check_quantized(both[0], f64(x), None if r is None else r.numpy())
    check_quantized(both[1], f64(x).T, None if r is None else r.numpy().T)
    for turned in (False, True):
        one = gns.mxfp4_quantize(x.cuda(), transposed=turned, noise=dr)
        assert torch.equal(one.codes, both[turned].codes) and torch.equal(one.scales, both[turned].scales)


@pytest.mark.parametrize("dtype,rows,cols", [(torch.float32, 8197, 8330), (torch.bfloat16, 16389, 8330),
                                             (torch.float16, 8197, 16500)])
@pytest.mark.parametrize("noisy", [False, True])
def test_matrices_larger_than_the_cache(dtype, rows, cols, noisy):
    """A matrix is its parts: its rows in bands of 1024, which the other tests'
    forms take."""
    gns = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(51)
    x = (torch.empty(rows, cols, device="cuda").normal_(0.0, 1.0, generator=gen)
         * torch.exp2(torch.randint(-9, 9, (rows, 1), device="cuda", generator=gen).float())).to(dtype)
    assert x.numel() * x.element_size() > 256 << 20
    noise = torch.randint(0, 256, (rows, cols), dtype=torch.uint8, device="cuda", generator=gen) if noisy else None
    say("quantize large", dtype, noisy)
    a, t = gns.mxfp4_quantize_both(x, noise=noise)
    for r in range(0, rows, 1024):
        band = slice(r, min(r + 1024, rows))
        n = band.stop - r
        pa, pt = gns.mxfp4_quantize_both(x[band], noise=None if noise is None else noise[band])
        assert torch.equal(a.codes[band], pa.codes)
        assert torch.equal(a.scales[r // 32:r // 32 + pa.scales.shape[0]], pa.scales)
        wide = pt.codes.shape[-1]
        assert torch.equal(t.codes[:, r // 2:r // 2 + wide], pt.codes)
        assert torch.equal(t.scales[:, r // 128:r // 128 + pt.scales.shape[1]], pt.scales)
        assert n == 1024 or band.stop == rows
    for turned, whole in ((False, a), (True, t)):
        one = gns.mxfp4_quantize(x, transposed=turned, noise=noise)
        assert torch.equal(one.codes, whole.codes) and torch.equal(one.scales, whole.scales)


# few tokens of tables whose other rows are cleared: by 256 rows a workgroup, by some, by 8
@pytest.mark.parametrize("count,vocab,width", [(53, 56523, 81), (5, 70000, 1), (700, 9001, 300), (40, 3001, 5000),
                                               (4097, 30011, 33)])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_cleared_rows(count, vocab, width, dtype):
    gns = need_gpu()
    rng = np.random.default_rng(count + width)
    tokens = ids(rng, count, vocab, "padded")
    g = torch.from_numpy(rng.normal(size=(count, width))).to(dtype)
    say("cleared rows", count, vocab, width, dtype)
    got = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.full((vocab, width), float("nan"), dtype=dtype, device="cuda"))
    check_grad(got, tokens, g, vocab, 1.0, None, dtype)
    touched = torch.zeros(vocab, dtype=torch.bool)
    touched[tokens[(tokens >= 0) & (tokens < vocab)].long()] = True
    assert (got.cpu()[~touched] == 0).all()


# runs of 1 to 2000 partial sums, in rows of every number of threads
@pytest.mark.parametrize("width", [3, 20, 50, 122, 300, 1000])
@pytest.mark.parametrize("accumulate", [False, True])
def test_runs_of_every_length(width, accumulate):
    gns = need_gpu()
    rng = np.random.default_rng(width)
    lengths = [1, 2, 7, 8, 9, 15, 16, 17, 63, 64, 65, 100, 129, 500, 513, 600, 1100, 4200, 3, 5, 16000, 11]
    tokens = torch.from_numpy(rng.permutation(np.repeat(np.arange(len(lengths)) * 3 + 1, lengths)))
    vocab = 3 * len(lengths) + 4000
    g = torch.from_numpy(rng.normal(size=(len(tokens), width))).to(torch.bfloat16)
    old = torch.from_numpy(rng.normal(size=(vocab, width))).to(torch.float32) if accumulate else None
    into = torch.full((vocab, width), float("nan"), device="cuda") if old is None else old.cuda()
    say("runs", width, accumulate)
    got = gns.embedding_grad(tokens.cuda(), g.cuda(), into, scale=0.5, accumulate=accumulate)
    check_grad(got, tokens, g, vocab, 0.5, None if old is None else f64(old), torch.float32)


@pytest.mark.parametrize("dtype,m,n", [(torch.float32, 8200, 8211), (torch.bfloat16, 8199, 16401), (torch.float32, 4000, 4001)])
def test_accumulated_results_larger_than_the_cache(dtype, m, n):
    """The sum of what is there and the product's fp32 result, rounded once."""
    gns = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(52)
    a, b = (gns.mxfp4_quantize(torch.empty(rows, 65, device="cuda").normal_(0.0, 1.0, generator=gen)) for rows in (m, n))
    old = torch.empty(m, n + 3, device="cuda").normal_(0.0, 1.0, generator=gen).to(dtype)
    say("accumulate large", dtype, m, n)
    product = gns.mxfp4_matmul(a, b, dtype=torch.float32)
    into = old.clone()
    gns.mxfp4_matmul(a, b, out=into[:, 2:n + 2], accumulate=True)
    assert torch.equal(into[:, 2:n + 2], (old[:, 2:n + 2].float() + product).to(dtype))
    assert torch.equal(into[:, :2], old[:, :2]) and torch.equal(into[:, n + 2:], old[:, n + 2:])


# the numbers of tokens at which the sort has another form, and one more
@pytest.mark.parametrize("count", [1023, 1024, 1025, 2047, 2048, 2049, 4095, 4096, 4097, 6143, 6144, 6145, 8192, 8193])
@pytest.mark.parametrize("kind", ["zipf", "all", "padded"])
def test_sorts_of_every_length(count, kind):
    gns = need_gpu()
    rng = np.random.default_rng(count)
    vocab, width = 70001, 5
    tokens = ids(rng, count, vocab, kind)
    g = torch.from_numpy(rng.normal(size=(count, width))).to(torch.float32)
    say("sorts", count, kind)
    got = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.full((vocab, width), float("nan"), device="cuda"))
    check_grad(got, tokens, g, vocab, 1.0, None, torch.float32)
