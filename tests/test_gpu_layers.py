"""The embedding and MXFP4 layers together and in the places where calls can
go wrong: refusals of tensors, other streams and threads, arrays that
interleave, offsets beyond 32 bits, and a whole training step.

Tolerances as in test_gpu_mxfp4.py and test_gpu_embedding.py.
"""
import math
import os
import sys
import threading

import numpy as np
import pytest
import torch

from gpu_common import NS5, need_gpu, say
from oracle import layers
from test_gpu_embedding import check_grad, ids
from test_gpu_mxfp4 import DTYPES, U, check_product, check_quantized, f64, rand

sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))

pytestmark = pytest.mark.gpu


# every kernel of the products: 256-edge tiles with ragged edges, 64 x 256 ones, parts of a contraction, few rows
@pytest.mark.parametrize("batch,m,n,k", [(1, 3500, 3400, 130), (2, 1900, 3333, 65), (64, 40, 1000, 200), (70, 63, 777, 333),
                                         (1, 200, 300, 9000), (3, 65, 70, 8192), (1, 130, 130, 20000), (1, 3, 9000, 300),
                                         (2, 31, 600, 2100), (1, 16, 40, 4096), (1, 16, 40, 4097), (5, 2, 8300, 64)])
def test_products_of_every_kernel(batch, m, n, k):
    gns = need_gpu()
    rng = np.random.default_rng(m + n)
    x, w = rand(rng, (batch, m, k), torch.bfloat16, wide=True), rand(rng, (batch, n, k), torch.float32)
    qx, qw = gns.mxfp4_quantize(x.cuda()), gns.mxfp4_quantize(w.cuda())
    vx, vw = (f64(gns.mxfp4_dequantize(q, dtype=torch.float32)) for q in (qx, qw))
    for dtype in DTYPES:
        old = rand(rng, (batch, m, n), dtype)
        for a in (qx, x.cuda()):
            say(f"product {batch}x{m}x{n}x{k} {dtype} plain={a is not qx}")
            got = gns.mxfp4_matmul(a, qw, dtype=dtype)
            check_product(got, vx, vw, k, dtype)
            assert torch.equal(got, gns.mxfp4_matmul(a, qw, dtype=dtype))
            check_product(gns.mxfp4_matmul(a, qw, out=old.cuda(), accumulate=True), vx, vw, k, dtype, f64(old))


def test_nothing_but_the_result_is_written():
    """Products into the middle of larger buffers, of every kernel."""
    gns = need_gpu()
    rng = np.random.default_rng(40)
    for batch, m, n, k in ((1, 3500, 3400, 64), (64, 40, 1000, 64), (1, 130, 130, 20000), (2, 31, 600, 64), (1, 129, 257, 64)):
        qx = gns.mxfp4_quantize(rand(rng, (batch, m, k), torch.float32).cuda())
        qw = gns.mxfp4_quantize(rand(rng, (batch, n, k), torch.float32).cuda())
        for dtype in (torch.float32, torch.bfloat16):
            for accumulate in (False, True):
                say("canary", batch, m, n, k, dtype, accumulate)
                buf = torch.full((batch, m + 4, n + 9), 3.0, dtype=dtype, device="cuda")
                want = torch.full_like(buf, 3.0)
                plain = torch.full((batch, m, n), 3.0, dtype=dtype, device="cuda")
                gns.mxfp4_matmul(qx, qw, out=buf[:, 2:m + 2, 5:n + 5], accumulate=accumulate)
                want[:, 2:m + 2, 5:n + 5] = gns.mxfp4_matmul(qx, qw, out=plain, accumulate=accumulate)
                assert torch.equal(buf, want)


def test_arrays_that_interleave():
    """Column slices of one buffer as input and output of the same call."""
    gns = need_gpu()
    rng = np.random.default_rng(41)
    tokens = ids(rng, 70, 30, "zipf").cuda()
    for dtype in DTYPES:
        buf = rand(rng, (70, 96), dtype).cuda()
        keep = buf.clone()
        say("interleaved", dtype)
        w = gns.mxfp4_quantize(rand(rng, (32, 64), torch.float32).cuda())
        gns.mxfp4_matmul(buf[:, :64], w, out=buf[:, 64:])
        assert torch.equal(buf[:, :64], keep[:, :64])
        assert torch.equal(buf[:, 64:], gns.mxfp4_matmul(keep[:, :64].contiguous(), w))
        buf = keep.clone()
        table = gns.embedding_grad(tokens, buf[:, :40], torch.zeros(30, 96, dtype=dtype, device="cuda")[:, 40:80])
        assert torch.equal(table, gns.embedding_grad(tokens, keep[:, :40].contiguous(), torch.empty_like(table).contiguous()))
        gns.embedding(tokens % 30, keep[:30, :40].contiguous(), out=buf[:, 50:90])
        assert torch.equal(buf[:, :50], keep[:, :50]) and torch.equal(buf[:, 90:], keep[:, 90:])
        for call in (lambda: gns.mxfp4_matmul(buf[:, :64], w, out=buf[:, 63:95]),
                     lambda: gns.embedding(tokens, buf[:30, :40], out=buf[:, 39:79])):
            with pytest.raises(gns.GnsError) as e:
                call()
            assert e.value.name == "GNS_E_ALIAS"


def test_refusals():
    """Arguments that name no such arrays."""
    gns = need_gpu()
    t = torch.zeros(6, dtype=torch.int64, device="cuda")
    w, g = torch.zeros(10, 8, device="cuda"), torch.zeros(6, 8, device="cuda")
    q, q3 = gns.mxfp4_quantize(torch.zeros(10, 8, device="cuda")), gns.mxfp4_quantize(torch.zeros(2, 10, 8, device="cuda"))
    x = torch.zeros(4, 8, device="cuda")
    say("refusals")

    class Elsewhere:
        device, cuda_stream = torch.device("cuda", 1), 0

    cases = {
        "GNS_E_DTYPE": [lambda: gns.embedding(t.float(), w), lambda: gns.embedding(t, w.double()),
                        lambda: gns.embedding(t, w, dtype=torch.float64), lambda: gns.embedding(t, w, out=g.double()),
                        lambda: gns.embedding(t, w, out=g, dtype=torch.bfloat16), lambda: gns.embedding_grad(t, g.int(), w),
                        lambda: gns.mxfp4_quantize(w.double()), lambda: gns.mxfp4_dequantize(q, dtype=torch.int8),
                        lambda: gns.mxfp4_matmul(x.double(), q), lambda: gns.mxfp4_matmul(x, q, dtype=torch.float64),
                        lambda: gns.mxfp4_matmul(x, q, out=torch.zeros(4, 10, device="cuda"), dtype=torch.float16)],
        "GNS_E_SHAPE": [lambda: gns.embedding(t, w[0]), lambda: gns.embedding(t, w.t()), lambda: gns.embedding(t, w, out=g[:5]),
                        lambda: gns.embedding(t, w, out=torch.zeros(6, 9, device="cuda")),
                        lambda: gns.embedding(t.view(2, 3).t(), w), lambda: gns.embedding_grad(t, g[:5], w),
                        lambda: gns.embedding_grad(t, g, w[0]), lambda: gns.embedding_grad(t, g, w[:, :7]),
                        lambda: gns.embedding_grad(t, g, w[:1].expand(10, 8)),
                        lambda: gns.embedding(t, w, out=g[:1].expand(6, 8)),
                        lambda: gns.mxfp4_quantize(w[0]), lambda: gns.mxfp4_quantize(w.view(1, 1, 10, 8)),
                        lambda: gns.mxfp4_quantize(w[::2, ::2]), lambda: gns.mxfp4_quantize(w, noise=t),
                        lambda: gns.mxfp4_quantize(w, noise=torch.zeros(10, 16, dtype=torch.uint8, device="cuda")[:, ::2]),
                        lambda: gns.mxfp4_quantize(w, noise=torch.zeros(10, 8, device="cuda")),
                        lambda: gns.mxfp4_quantize(w, out=q3), lambda: gns.mxfp4_quantize(w, transposed=True, out=q),
                        lambda: gns.mxfp4_quantize(w, out=w), lambda: gns.mxfp4_dequantize(q, out=w[:, :7]),
                        lambda: gns.mxfp4_dequantize(q, out=w.t()), lambda: gns.mxfp4_matmul(x[:, :7], q),
                        lambda: gns.mxfp4_matmul(x, q3), lambda: gns.mxfp4_matmul(q, q3), lambda: gns.mxfp4_matmul(x[0, 0], q),
                        lambda: gns.mxfp4_matmul(x, q, out=torch.zeros(4, 9, device="cuda")),
                        lambda: gns.mxfp4_matmul(x, q, out=torch.zeros(4, 20, device="cuda")[:, ::2]),
                        lambda: gns.mxfp4_matmul(x, q, out=torch.zeros(1, 10, device="cuda").expand(4, 10)),
                        lambda: gns.mxfp4_matmul(torch.zeros(2, 3, 8, device="cuda").transpose(0, 1), q),
                        lambda: gns.MXFP4(q.codes, q.scales, (10, 300)), lambda: gns.MXFP4(q.codes, q.scales, (10,)),
                        lambda: gns.MXFP4(q.codes.int(), q.scales, (10, 8)), lambda: gns.mxfp4_empty((3,)), lambda: q[0]],
        "GNS_E_NULL": [lambda: gns.embedding(t, w.cpu()), lambda: gns.embedding(t, w, out=g.cpu()),
                       lambda: gns.embedding_grad(t, g.cpu(), w), lambda: gns.embedding_grad(t, g, w.cpu()),
                       lambda: gns.embedding(t, w.to_sparse()), lambda: gns.mxfp4_matmul(x, w), lambda: gns.mxfp4_matmul(x.cpu(), q),
                       lambda: gns.mxfp4_matmul(None, q), lambda: gns.mxfp4_matmul(x, q, accumulate=True),
                       lambda: gns.mxfp4_quantize(w, noise=torch.zeros(10, 8, dtype=torch.uint8)),
                       lambda: gns.mxfp4_matmul(x, q, workspace=torch.zeros(512, dtype=torch.uint8))],
        "GNS_E_PARAM": [lambda: gns.embedding(t, w, scale=math.inf), lambda: gns.embedding_grad(t, g, w, scale=math.nan),
                        lambda: gns.embedding(t, w, stream=Elsewhere()), lambda: gns.mxfp4_matmul(x, q, stream=Elsewhere()),
                        lambda: gns.mxfp4_quantize(w, stream=Elsewhere())],
        "GNS_E_WORKSPACE": [lambda: gns.embedding_grad(t.repeat(1000), g.repeat(1000, 1), torch.zeros(9000, 8, device="cuda"),
                                                       workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")),
                            lambda: gns.mxfp4_matmul(torch.zeros(20, 8, device="cuda"), q,
                                                     workspace=torch.zeros(512, dtype=torch.uint8, device="cuda")[::2])],
    }
    for name, calls in cases.items():
        for i, call in enumerate(calls):
            with pytest.raises(gns.GnsError) as e:
                call()
            assert e.value.name == name, (name, i)
    torch.cuda.synchronize()


def test_threads():
    """Threads with streams of their own share the weights."""
    gns = need_gpu()
    rng = np.random.default_rng(42)
    w = gns.mxfp4_quantize(rand(rng, (300, 512), torch.float32).cuda())
    table = rand(rng, (50, 512), torch.bfloat16).cuda()
    tokens = [ids(rng, 5000, 50, "skewed").cuda() for _ in range(3)]
    grads = [rand(rng, (5000, 512), torch.bfloat16).cuda() for _ in range(3)]

    def work(i):
        x = gns.embedding(tokens[i], table, scale=2.0)
        y = gns.mxfp4_matmul(x, w, dtype=torch.float32)
        z = gns.mxfp4_matmul(x[:4], w, dtype=torch.float32)
        q, t = gns.mxfp4_quantize_both(grads[i])
        return y, z, gns.mxfp4_matmul(t, t, dtype=torch.float32), gns.embedding_grad(
            tokens[i], grads[i], torch.ones(50, 512, device="cuda"), accumulate=True)

    want = [work(i) for i in range(3)]
    torch.cuda.synchronize()
    got = [None] * 3

    def thread(i):
        s = torch.cuda.Stream()
        with torch.cuda.stream(s):
            for _ in range(5):
                got[i] = work(i)
            s.synchronize()

    say("threads")
    threads = [threading.Thread(target=thread, args=(i,)) for i in range(3)]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    for a, b in zip(got, want):
        assert all(torch.equal(x, y) for x, y in zip(a, b))


def test_offsets_beyond_32_bits():
    """Arrays of more than 2^32 elements: what lies at their end."""
    gns = need_gpu()
    rng = np.random.default_rng(43)
    rows, width = 140000, 32768
    big = torch.zeros(rows, width, dtype=torch.bfloat16, device="cuda")
    tail = rand(rng, (40, width), torch.bfloat16)
    big[-40:] = tail.cuda()
    tokens = torch.tensor([rows - 1, rows - 40, 0, rows - 7, rows - 1, rows], device="cuda")
    say("far rows: lookup")
    got = gns.embedding(tokens, big).cpu()
    assert torch.equal(got[[0, 1, 3, 4]], tail[[39, 0, 33, 39]]) and not got[[2, 5]].any()
    say("far rows: quantize")
    q = gns.mxfp4_quantize(big)
    small = gns.mxfp4_quantize(tail.cuda())
    assert torch.equal(q.codes[-40:], small.codes) and not q.codes[:-40].any()
    x = rand(rng, (33, width), torch.bfloat16).cuda()
    want = gns.mxfp4_matmul(x, small, dtype=torch.float32)
    for m in (1, 20, 33):
        say("far rows: product", m)
        y = gns.mxfp4_matmul(x[:m], q, dtype=torch.float32)
        assert not y[:, :-40].any()
        ref = want[:m].double()
        assert torch.all((y[:, -40:].double() - ref).abs() <= 4 * width * U * ref.abs().max() * 40)
        assert torch.equal(y, gns.mxfp4_matmul(x[:m], q, dtype=torch.float32))
    del q, y
    say("far rows: transposed, dequantize")
    t = gns.mxfp4_quantize(big, transposed=True)
    values = gns.mxfp4_dequantize(t)
    assert not values[:, :-64].any()
    check_quantized(gns.mxfp4_quantize(tail.cuda(), transposed=True), f64(tail).T)
    del t, values
    say("far rows: gradient")
    g = rand(rng, (6, width), torch.bfloat16)
    gns.embedding_grad(tokens, g.cuda(), big)
    sums = torch.zeros(40, width)
    for i, row in ((0, 39), (1, 0), (3, 33), (4, 39)):
        sums[row] += g[i].float()
    assert torch.equal(big[-40:].cpu(), sums.bfloat16())
    assert torch.equal(big[0].cpu(), g[2]) and not big[1:-40].any()


def test_example_functions_have_the_formulas_gradients():
    """The example's autograd functions: the gradients of its layers are the
    formulas', and those of a sum of outputs agree with differences where the
    layer is linear (the embedding)."""
    gns = need_gpu()
    import train_step
    rng = np.random.default_rng(44)
    say("example functions")
    x = rand(rng, (300, 512), torch.bfloat16).cuda().requires_grad_()
    w = rand(rng, (384, 512), torch.bfloat16).cuda().requires_grad_()
    by_rows, by_columns = gns.mxfp4_quantize_both(w.detach())
    y = train_step.Linear4.apply(x, w, by_rows, by_columns)
    g = rand(rng, (300, 384), torch.bfloat16).cuda()
    y.backward(g)

    def q(t):
        return layers.mxfp4_values(*layers.mxfp4_quantize(t))

    fx, fw, fg = f64(x), f64(w), f64(g)
    check_product(y, q(fx), q(fw), 512, torch.bfloat16)
    check_product(x.grad, q(fg), q(fw.T), 384, torch.bfloat16)
    check_product(w.grad, q(fg.T), q(fx.T), 300, torch.bfloat16)
    tokens = ids(rng, 400, 60, "skewed")
    table = rand(rng, (60, 33), torch.float32).cuda().requires_grad_()
    out = train_step.Embedding.apply(tokens.cuda(), table)
    g = rand(rng, (400, 33), torch.float32)
    out.backward(g.cuda())
    check_grad(table.grad, tokens, g, 60, 1.0, None, torch.float32)
    step = torch.zeros_like(table)
    step[tokens[5], 7] = 0.5
    with torch.no_grad():
        up, down = ((train_step.Embedding.apply(tokens.cuda(), table.detach() + s * step).double() * g.cuda()).sum()
                    for s in (1, -1))
    # (the tables' sums are rounded to fp32: u of their size per looked-up element)
    assert abs(float(up - down) - float(table.grad[tokens[5], 7])) <= 2 * U * float(
        (out.detach().abs().double() * g.cuda().abs()).sum() + 400)


def test_a_training_step_of_them_together():
    """Lookup, a layer in 4 bits, its gradients into buckets that the norm is
    taken of, and the updates of all weights: each part against its oracle on
    what the parts before it gave."""
    gns = need_gpu()
    rng = np.random.default_rng(45)
    vocab, width, n = 300, 128, 256
    tokens = ids(rng, 2000, vocab, "padded")
    table, W = rand(rng, (vocab, width), torch.float32).cuda(), (rand(rng, (1, n, width), torch.float32) * 0.1).cuda()
    flat = torch.zeros(vocab * width + n * width, device="cuda")
    g_table, g_w = flat[:vocab * width].view(vocab, width), flat[vocab * width:].view(1, n, width)
    M, v = torch.zeros_like(W), torch.zeros(1, n, device="cuda")
    adam = gns.adamw_list([table], [g_table], [torch.zeros_like(table)], [torch.zeros_like(table)])
    grads = gns.tensor_list([g_w, g_table])
    count = torch.zeros(1, dtype=torch.int64, device="cuda")
    by_rows, by_columns = gns.mxfp4_quantize_both(W)
    target = rand(rng, (2000, n), torch.float32).cuda()
    for step in range(3):
        say("training step", step)
        for micro in range(2):                          # the second adds to the buckets
            x = gns.embedding(tokens.cuda(), table, scale=4.0, dtype=torch.bfloat16)
            y = gns.mxfp4_matmul(x, by_rows[0], dtype=torch.float32)
            gy = ((y - target) / 2000).bfloat16()
            q, qt = gns.mxfp4_quantize_both(gy)
            _, xt = gns.mxfp4_quantize_both(x)
            gx = gns.mxfp4_matmul(q, by_columns[0], dtype=torch.bfloat16)
            held = f64(g_w[0]), f64(g_table)
            gns.mxfp4_matmul(qt, xt, out=g_w[0], accumulate=micro > 0)
            gns.embedding_grad(tokens.cuda(), gx, g_table, scale=4.0, accumulate=micro > 0)
            values = [f64(gns.mxfp4_dequantize(m, dtype=torch.float32)) for m in (q, qt, xt, by_rows[0], by_columns[0])]
            check_product(y, layers.mxfp4_values(*layers.mxfp4_quantize(f64(x))), values[3], width, torch.float32)
            check_product(gx, values[0], values[4], n, torch.bfloat16)
            check_product(g_w[0], values[1], values[2], 2000, torch.float32, held[0] if micro else None)
            check_grad(g_table, tokens, gx.cpu(), vocab, 4.0, held[1] if micro else None, torch.float32)
        got = gns.grad_norm(grads, max_norm=0.1)
        norm = math.sqrt(float((flat.double() ** 2).sum()))
        assert abs(float(got.norm) - norm) <= 2 * U * norm
        before = table.clone()
        gns.dion3_step(W, g_w, M, v, 64, NS5, lr=0.01, grad_scale=got.clip)
        gns.adamw_step(adam, count=count, lr=0.01, grad_scale=got.clip)
        assert not torch.equal(before, table) and torch.isfinite(W).all()
        gns.mxfp4_quantize_both(W, out=(by_rows, by_columns))
        check_quantized(by_rows, f64(W))
        check_quantized(by_columns, np.swapaxes(f64(W), -1, -2))
    assert int(count) == 3


def test_example_runs_in_mxfp4():
    need_gpu()
    import train_step
    say("example --mxfp4")
    losses, norms = train_step.train(6, log=say, mxfp4=True)
    assert torch.isfinite(losses).all() and torch.isfinite(norms).all()


def test_captured_backward_pass():
    """The layers' gradients captured into a graph and replayed with new
    inputs, beside the program's eager calls."""
    gns = need_gpu()
    import train_step
    rng = np.random.default_rng(46)
    x0, w = rand(rng, (200, 256), torch.bfloat16).cuda(), rand(rng, (128, 256), torch.bfloat16).cuda()
    table = rand(rng, (90, 64), torch.bfloat16).cuda()
    tokens = ids(rng, 800, 90, "zipf").cuda()
    quantized = gns.mxfp4_quantize_both(w)

    def gradients(x, t):
        x, lw, lt = x.detach().requires_grad_(), w.detach().requires_grad_(), table.detach().requires_grad_()
        rows = train_step.Embedding.apply(t, lt).reshape(200, 256)
        y = train_step.Linear4.apply(x + rows, lw, *quantized)
        return torch.autograd.grad(y.float().square().mean(), (x, lw, lt))

    say("captured backward")
    sx, st = x0.clone(), tokens.clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        gradients(sx, st)
    torch.cuda.current_stream().wait_stream(side)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = gradients(sx, st)
    for i in range(4):
        x2, t2 = rand(rng, (200, 256), torch.bfloat16).cuda(), ids(rng, 800, 90, ["skewed", "one", "padded", "zipf"][i]).cuda()
        sx.copy_(x2)
        st.copy_(t2)
        graph.replay()
        eager = gradients(x2, t2)
        torch.cuda.synchronize()
        assert all(torch.equal(a, b) for a, b in zip(out, eager)), i
