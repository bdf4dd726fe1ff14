"""Token embedding and its gradient against the 64-bit oracle.

Tolerances, from u = 2^-24:
* a looked-up element is to the bit the fp32 product of the weight and scale,
  rounded to its type;
* a gradient element is a sum of n terms in fp32 in some order, times scale,
  plus what it held: at most (n + 3) u of the sum of the terms' magnitudes, and
  half a step of the type it is stored in.
"""
import math

import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say
from oracle import layers

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def rand(rng, shape, scale, dtype):
    return torch.from_numpy(np.asarray(rng.normal(size=shape) * scale)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def ids(rng, n, vocab, kind):
    if kind == "one":
        t = np.full(n, vocab // 2)
    elif kind == "all":
        t = rng.permutation(np.arange(n) % vocab)
    elif kind == "skewed":
        t = np.where(rng.random(n) < 0.6, vocab // 3, rng.integers(0, vocab, n))
    elif kind == "padded":
        t = np.where(rng.random(n) < 0.4, rng.choice([-1, vocab, -100, 2 ** 31 - 1]), rng.integers(0, vocab, n))
    elif kind == "only padding":
        t = np.full(n, -1)
    else:
        t = np.minimum((vocab ** rng.random(n)).astype(np.int64) - 1, vocab - 1)
    return torch.from_numpy(t.astype(np.int64))


SIZES = [(1, 1, 1), (1, 5, 3), (7, 3, 8), (16, 1000, 64), (63, 17, 65), (64, 300, 128), (65, 2, 129), (257, 40, 2048),
         (100, 70, 2049), (1000, 513, 100), (31, 9, 4100), (4096, 256, 128)]


@pytest.mark.parametrize("count,vocab,width", SIZES)
@pytest.mark.parametrize("kind", ["zipf", "padded"])
def test_lookup(count, vocab, width, kind):
    gns = need_gpu()
    rng = np.random.default_rng(count + width)
    tokens = ids(rng, count, vocab, kind)
    for wt in DTYPES:
        w = rand(rng, (vocab, width), 0.7, wt)
        for ot in DTYPES:
            for scale in (1.0, 11.3137):
                say(f"lookup {count}x{width} of {vocab} {kind} {wt} -> {ot}")
                got = gns.embedding(tokens.cuda(), w.cuda(), scale=scale, dtype=ot)
                real = (tokens >= 0) & (tokens < vocab)
                want = w[tokens.clamp(0, vocab - 1)].float() * torch.tensor(scale, dtype=torch.float32)
                want = torch.where(real[:, None], want, 0.0).to(ot)
                assert torch.equal(got.cpu(), want)
    got = gns.embedding(tokens.int().cuda().view(1, count, 1), w.cuda())
    assert got.shape == (1, count, 1, width) and got.dtype == w.dtype
    assert np.allclose(f64(got).reshape(count, width), layers.embedding(tokens.int().numpy(), f64(w)), rtol=0, atol=0)


def test_lookup_views():
    """Weights and outputs that are column slices, misaligned or repeated rows;
    what lies between is left alone."""
    gns = need_gpu()
    rng = np.random.default_rng(3)
    tokens = ids(rng, 200, 50, "padded")
    for dtype in DTYPES:
        base = rand(rng, (50, 301), 1.0, dtype).cuda()
        for lo, hi in ((0, 64), (1, 65), (8, 136), (100, 101), (3, 301)):
            w = base[:, lo:hi]
            buf = torch.full((200, 333), 7.0, dtype=dtype, device="cuda")
            say("lookup views", dtype, lo, hi)
            out = gns.embedding(tokens.cuda(), w, scale=2.0, out=buf[:, 5:5 + hi - lo])
            want = torch.full((200, 333), 7.0, dtype=dtype)
            want[:, 5:5 + hi - lo] = gns.embedding(tokens.cuda(), w.contiguous(), scale=2.0).cpu()
            assert torch.equal(buf.cpu(), want) and out.data_ptr() == buf[:, 5:].data_ptr()
        same = base[:1, :40].expand(50, 40)
        assert torch.equal(gns.embedding(tokens.cuda(), same).cpu(), gns.embedding(tokens.cuda(), same.contiguous()).cpu())


def check_grad(got, tokens, g, vocab, scale, old, dtype):
    sums, sizes, n = layers.embedding_grad(tokens.numpy(), f64(g), vocab, scale, old)
    tiny = float(torch.finfo(dtype).tiny) * float(torch.finfo(dtype).eps)
    tol = (n[:, None] + 3) * U * sizes
    tol = tol + (np.abs(sums) + tol) * (float(torch.finfo(dtype).eps) / 2) + tiny
    err = np.abs(f64(got) - sums)
    assert np.all(err <= tol), float(np.max(err / tol))
    return n


@pytest.mark.parametrize("count,vocab,width", SIZES)
@pytest.mark.parametrize("kind", ["zipf", "one", "all", "skewed", "padded", "only padding"])
def test_gradient(count, vocab, width, kind):
    gns = need_gpu()
    rng = np.random.default_rng(7 * count + width)
    tokens = ids(rng, count, vocab, kind)
    pairs = [(torch.bfloat16, torch.float32), (torch.float16, torch.bfloat16), (torch.float32, torch.float16)]
    for gt, wt in pairs + ([(d, d) for d in DTYPES] if count < 300 else []):
        g = rand(rng, (count, width), 0.3, gt)
        old = rand(rng, (vocab, width), 0.3, wt)
        for accumulate in (False, True):
            say(f"gradient {count}x{width} into {vocab} {kind} {gt} -> {wt} accumulate={accumulate}")
            into = old.cuda()
            got = gns.embedding_grad(tokens.cuda(), g.cuda(), into, scale=1.5, accumulate=accumulate)
            assert got.data_ptr() == into.data_ptr()
            n = check_grad(got, tokens, g, vocab, 1.5, f64(old) if accumulate else None, wt)
            if accumulate:                                  # rows of no token are not written
                untouched = torch.from_numpy(n == 0)
                assert torch.equal(got.cpu()[untouched], old[untouched])
            again = old.cuda()
            gns.embedding_grad(tokens.int().cuda(), g.cuda(), again, scale=1.5, accumulate=accumulate)
            if kind != "padded":                            # (int32 holds the same tokens)
                assert torch.equal(again.cpu(), got.cpu())


@pytest.mark.parametrize("count,vocab,width,kind", [
    (5000, 70000, 24, "zipf"), (20011, 131072, 16, "zipf"), (9001, 49999, 40, "skewed"), (70000, 3, 8, "all"),
    (33000, 1 << 20, 4, "all"), (40000, 5000, 12, "padded"), (66000, 2, 9, "one")])
def test_gradient_of_many_tokens(count, vocab, width, kind):
    """Sorts of several passes and of more than one tile; runs of one token
    longer than any piece of work."""
    gns = need_gpu()
    rng = np.random.default_rng(11)
    tokens = ids(rng, count, vocab, kind)
    g = rand(rng, (count, width), 0.3, torch.bfloat16)
    say("many tokens", count, vocab, width, kind)
    got = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.empty(vocab, width, device="cuda").fill_(math.nan))
    real = (tokens >= 0) & (tokens < vocab)
    t, x = tokens[real], g[real].double()
    ref = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, t, x)
    size = torch.zeros(vocab, width, dtype=torch.float64).index_add_(0, t, x.abs())
    n = torch.zeros(vocab, dtype=torch.float64).index_add_(0, t, torch.ones(len(t), dtype=torch.float64))
    assert torch.all((got.cpu().double() - ref).abs() <= (n[:, None] + 4) * U * size)
    again = gns.embedding_grad(tokens.cuda(), g.cuda(), torch.empty(vocab, width, device="cuda"))
    assert torch.equal(got, again)


def test_gradient_views():
    gns = need_gpu()
    rng = np.random.default_rng(4)
    tokens = ids(rng, 300, 60, "padded")
    for gt, wt in ((torch.bfloat16, torch.float32), (torch.float32, torch.bfloat16), (torch.float16, torch.float16)):
        base = rand(rng, (300, 301), 1.0, gt).cuda()
        for lo, hi in ((0, 64), (1, 65), (8, 136), (100, 101), (3, 301)):
            g = base[:, lo:hi]
            buf = torch.full((60, 333), 7.0, dtype=wt, device="cuda")
            say("gradient views", gt, wt, lo, hi)
            gns.embedding_grad(tokens.cuda(), g, buf[:, 5:5 + hi - lo])
            plain = torch.empty(60, hi - lo, dtype=wt, device="cuda")
            gns.embedding_grad(tokens.cuda(), g.contiguous(), plain)
            want = torch.full((60, 333), 7.0, dtype=wt)
            want[:, 5:5 + hi - lo] = plain.cpu()
            assert torch.equal(buf.cpu(), want)
            check_grad(plain, tokens, g.cpu(), 60, 1.0, None, wt)
        g = base[:1, :40].expand(300, 40)                   # one row for all, as of a sum's gradient
        plain = gns.embedding_grad(tokens.cuda(), g, torch.empty(60, 40, dtype=wt, device="cuda"))
        check_grad(plain, tokens, g.cpu(), 60, 1.0, None, wt)


def test_gradient_is_that_of_the_lookup():
    """<lookup(w + d) - lookup(w), g> = <d, gradient(g)> for fp32 values that
    leave both sides exact."""
    gns = need_gpu()
    rng = np.random.default_rng(5)
    tokens = ids(rng, 500, 30, "padded").cuda()
    w, d, g = (torch.from_numpy(rng.integers(-8, 9, size=s).astype(np.float32)).cuda()
               for s in ((30, 20), (30, 20), (500, 20)))
    say("adjoint")
    left = ((gns.embedding(tokens, w + d, scale=2.0) - gns.embedding(tokens, w, scale=2.0)).double() * g.double()).sum()
    grad = gns.embedding_grad(tokens, g, torch.empty_like(w), scale=2.0)
    assert float(left) == float((grad.double() * d.double()).sum())


def test_nonfinite_rows_stay_in_their_rows():
    gns = need_gpu()
    tokens = torch.tensor([2, 0, 2, 1, 5, -1], device="cuda")
    g = torch.ones(6, 33, device="cuda")
    g[2, 3], g[5] = math.nan, math.nan                       # the second is padding
    g[3, 4] = math.inf
    say("nonfinite")
    got = gns.embedding_grad(tokens, g, torch.empty(6, 33, device="cuda")).cpu()
    want = torch.zeros(6, 33)
    want[0], want[1], want[2], want[5] = 1, 1, 2, 1
    want[2, 3], want[1, 4] = math.nan, math.inf
    assert torch.equal(got.isnan(), want.isnan()) and torch.equal(got.nan_to_num(9.0), want.nan_to_num(9.0))


def test_nothing():
    gns = need_gpu()
    none = torch.empty(0, dtype=torch.int64, device="cuda")
    w = torch.ones(5, 4, device="cuda")
    say("nothing")
    assert gns.embedding(none, w).shape == (0, 4)
    assert gns.embedding(none.view(0, 3), w).shape == (0, 3, 4)
    assert gns.embedding(torch.tensor([1, 2], device="cuda"), w[:0]).tolist() == [[0.0] * 4] * 2
    assert gns.embedding(torch.tensor([1, 2], device="cuda"), w[:, :0]).shape == (2, 0)
    grad = torch.ones(5, 4, device="cuda")
    gns.embedding_grad(none, torch.empty(0, 4, device="cuda"), grad, accumulate=True)
    assert (grad == 1).all()
    gns.embedding_grad(none, torch.empty(0, 4, device="cuda"), grad)
    assert (grad == 0).all()
    gns.embedding_grad(torch.tensor([1], device="cuda"), torch.ones(1, 4, device="cuda"), grad[:0])
    gns.embedding_grad(torch.tensor([1], device="cuda"), torch.ones(1, 0, device="cuda"), grad[:, :0])


def test_streams_graphs_and_workspaces():
    """On another stream, in a graph replayed with new inputs beside eager
    calls, and with a workspace of the caller's that holds anything."""
    gns = need_gpu()
    rng = np.random.default_rng(9)
    count, vocab, width = 5000, 700, 96
    tokens = ids(rng, count, vocab, "skewed").cuda()
    w, g = rand(rng, (vocab, width), 1.0, torch.bfloat16).cuda(), rand(rng, (count, width), 1.0, torch.bfloat16).cuda()

    def both(t, x):
        return (gns.embedding(t, w, scale=3.0, dtype=torch.float32),
                gns.embedding_grad(t, x, torch.full((vocab, width), 2.0, device="cuda"), accumulate=True))

    want = both(tokens, g)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    say("embedding on another stream")
    got = (gns.embedding(tokens, w, scale=3.0, dtype=torch.float32, stream=side),
           gns.embedding_grad(tokens=tokens, grad=g, grad_weight=torch.full((vocab, width), 2.0, device="cuda"),
                              accumulate=True, stream=side.cuda_stream))
    side.synchronize()
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    ws = torch.randint(256, (gns.embedding_grad_workspace_bytes(count, vocab, width),), dtype=torch.uint8,
                       device="cuda")
    say("embedding, caller's workspace")
    for _ in range(2):
        got = gns.embedding_grad(tokens, g, torch.full((vocab, width), 2.0, device="cuda"), accumulate=True,
                                 workspace=ws)
        assert torch.equal(got, want[1])
    graph = torch.cuda.CUDAGraph()
    st, sg = tokens.clone(), g.clone()
    say("embedding captured")
    with torch.cuda.graph(graph):
        out = both(st, sg)
    for i in range(4):
        t2 = ids(rng, count, vocab, ["zipf", "padded", "one", "skewed"][i]).cuda()
        st.copy_(t2)
        sg.copy_(g.flip(0))
        graph.replay()
        eager = both(t2, g.flip(0).contiguous())
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
