"""Lists of tensors on every path that a call can take: skipped and unchanged
gradients through each number of launches, AdamW of large lists, in many
chunks, past 32-bit offsets, and what lies around its arrays.

Tolerances as in test_gpu_tensors.py: clipped elements to the bit; moments
6 u of |b1 m| + |(1 - b1) g|, parameters 4 u (|p| + |p'|) + 16 u of the update
term, u = 2^-24."""
import ctypes
import math

import numpy as np
import pytest
import torch

from gpu_common import need_gpu, say

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


def bits(t):
    return t.view(torch.int16 if t.element_size() == 2 else torch.int32)


def gradients(chunks, dtype):
    rng = np.random.default_rng(chunks)
    return torch.from_numpy(rng.normal(size=(chunks, 5)) * 0.5).to(dtype).cuda()


# one launch, one launch and a scaling that adds the partials up (two), three
CHUNKS = [4, 5, 512, 513, 4096, 4097]


@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("per_tensor", [False, True])
@pytest.mark.parametrize("into", [None, torch.float32])
@pytest.mark.parametrize("bad", [math.nan, -math.inf])
def test_nonfinite_on_every_path(chunks, per_tensor, into, bad):
    gns = need_gpu()
    for ord, at in ((2, chunks - 1), (math.inf, 0), (2, chunks // 2)):
        g = gradients(chunks, torch.bfloat16)
        g[at, 3] = bad
        before = g.clone()
        out = None if into is None else [torch.full((5,), 3.0, dtype=into, device="cuda") for _ in range(chunks)]
        lst = gns.tensor_list(list(g), out=out)
        assert lst.info.chunks == chunks
        say("nonfinite", chunks, per_tensor, into, bad, ord, at)
        got = gns.clip_grad_norm_(lst, 0.25, ord=ord, per_tensor=per_tensor)
        norm = float(got.norm)
        assert (math.isnan(norm) if math.isnan(bad) else norm == math.inf) and math.isnan(float(got.clip))
        assert torch.equal(bits(g), bits(before))
        if out is not None:
            assert bool((torch.stack(out) == 3.0).all())
        if per_tensor:
            finite = torch.isfinite(got.tensor_norms)
            assert not bool(finite[at]) and int(finite.sum()) == chunks - 1


@pytest.mark.parametrize("chunks", CHUNKS)
@pytest.mark.parametrize("per_tensor", [False, True])
def test_below_the_bound_on_every_path(chunks, per_tensor):
    """A factor of one: nothing changes in place, an output gets the gradients."""
    gns = need_gpu()
    g = gradients(chunks, torch.float16)
    before = g.clone()
    out = [torch.zeros(5, dtype=torch.float16, device="cuda") for _ in range(chunks)]
    say("below the bound", chunks, per_tensor)
    assert float(gns.clip_grad_norm_(list(g), 1e6, per_tensor=per_tensor).clip) == 1.0
    assert torch.equal(bits(g), bits(before))
    gns.clip_grad_norm_(gns.tensor_list(list(g), out=out), 1e6, per_tensor=per_tensor)
    assert torch.equal(bits(torch.stack(out)), bits(before)) and torch.equal(bits(g), bits(before))


@pytest.mark.parametrize("bad", [None, math.nan, math.inf])
def test_parts_of_chunks_that_write_nothing(bad):
    """A list beyond the last-level cache, whose chunks are cut into parts."""
    gns = need_gpu()
    g = torch.empty(150000001, device="cuda").normal_(0, 0.01).bfloat16()
    if bad is not None:
        g[150000000] = bad
    before, out = g.clone(), torch.full((g.numel(),), 3.0, dtype=torch.bfloat16, device="cuda")
    lst, into = gns.tensor_list([g]), gns.tensor_list([g], out=[out])
    assert lst.info.keep_from > 0 and lst.info.chunk_units > 1024
    say("parts that write nothing", bad)
    clip = float(gns.clip_grad_norm_(lst, 1e6).clip)
    assert clip == 1.0 if bad is None else math.isnan(clip)
    assert torch.equal(bits(g), bits(before))
    gns.clip_grad_norm_(into, 1e6)
    assert torch.equal(bits(out), bits(before)) if bad is None else bool((out == 3.0).all())


@pytest.mark.parametrize("copy", [None, torch.bfloat16])
def test_adamw_of_a_large_list(copy):
    """More than 2^27 elements: longer chunks, in more parts."""
    gns = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(94)
    sizes = (70000001, 77, 81234567)

    def arrays(scale):
        return [torch.empty(n, device="cuda").normal_(0, scale, generator=gen) for n in sizes]

    p, m, v = arrays(1.0), arrays(0.1), [t.square_() for t in arrays(0.1)]
    g = [t.bfloat16() for t in arrays(0.5)]
    c = None if copy is None else [torch.zeros(n, dtype=copy, device="cuda") for n in sizes]
    old = [[t.clone() for t in a] for a in (p, m, v)]
    lst = gns.adamw_list(p, g, m, v, copies=c)
    assert lst.info.chunk_units == 2048
    lr, b1, b2, eps, wd, t = 0.02, 0.9, 0.95, 1e-8, 0.3, 7
    scale = torch.tensor(0.37, device="cuda")
    say("large adamw", copy)
    gns.adamw_step(lst, t, lr=lr, betas=(b1, b2), eps=eps, weight_decay=wd, grad_scale=scale)
    for i in range(len(sizes)):
        gi = g[i].double() * scale.double()
        rm, rv = b1 * old[1][i].double() + (1 - b1) * gi, b2 * old[2][i].double() + (1 - b2) * gi * gi
        mag = b1 * old[1][i].double().abs() + (1 - b1) * gi.abs()
        del gi
        assert bool(((m[i].double() - rm).abs() <= 6 * U * mag + 2.0 ** -148).all())
        assert bool(((v[i].double() - rv).abs() <= 6 * U * rv + 2.0 ** -148).all())
        denom = (rv / (1 - b2 ** t)).sqrt_() + eps
        rp = old[0][i].double() * (1 - lr * wd) - lr / (1 - b1 ** t) * rm / denom
        bound = 4 * U * (old[0][i].double().abs() + rp.abs()) + 16 * U * lr / (1 - b1 ** t) * mag / denom
        assert bool(((p[i].double() - rp).abs() <= bound + 2.0 ** -148).all())
        if c is not None:
            assert torch.equal(c[i], p[i].to(copy))


def test_adamw_beyond_32_bits():
    """Elements past 2^31 and byte offsets past 2^33: a gradient here and there
    moves its own parameter by -lr g / (|g| + eps), and no other."""
    gns = need_gpu()
    n = (1 << 31) + 8195
    p, m, v = (torch.zeros(n, device="cuda") for _ in range(3))
    g, c = (torch.zeros(n, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    at = torch.tensor([0, 127, 8192, (1 << 30) - 1, 1 << 30, (1 << 31) - 1, 1 << 31, n - 4, n - 1], device="cuda")
    g[at] = torch.tensor([1.0, -2.0, 0.5, 3.0, -1.0, 0.25, -0.125, 8.0, -1.0], device="cuda").bfloat16()
    say("adamw beyond 32 bits")
    gns.adamw_step(gns.adamw_list([p], [g], [m], [v], copies=[c]), 1, lr=0.5, weight_decay=0.0)
    assert torch.allclose(p[at], -0.5 * torch.sign(g[at].float()), rtol=0, atol=1e-6)
    assert torch.equal(c[at], p[at].bfloat16())
    for t in (p, m, v, c):
        assert int(torch.count_nonzero(t)) == at.numel()


def test_most_tensors_of_a_list():
    """2^20 tensors, the most a list takes, and more chunks than their parts
    fit a grid whole: norm, clipping into another buffer and AdamW through the
    C ABI, on tensors packed behind one another."""
    gns = need_gpu()
    from gram_newton_schulz_amd import tensors as T
    count, last = 1 << 20, 3 * 8192
    sizes = np.full(count, 3, dtype=np.int64)
    sizes[-1] = last
    starts = np.concatenate([[0], np.cumsum(sizes)[:-1]])
    n = int(sizes.sum())
    gen = torch.Generator(device="cuda").manual_seed(95)
    flat = [torch.empty(n, device="cuda").normal_(0, s, generator=gen) for s in (0.5, 1.0, 0.1, 0.1)]
    flat[3].square_()
    old = [t.clone() for t in flat]
    out = torch.zeros(n, device="cuda")
    L = gns.lib()

    def build(buffers):
        e = np.zeros((len(buffers), count), dtype=T._ENTRY)
        for k, b in enumerate(buffers):
            e["data"][k] = b.data_ptr() + 4 * starts
            e["cols"][k] = e["pitch"][k] = sizes
        e["rows"] = 1
        nbytes = int(L.gns_tensor_list_bytes(e.ctypes.data, len(buffers), count))
        image, info = torch.empty(nbytes, dtype=torch.uint8, pin_memory=True), T.ListInfo()
        assert L.gns_tensor_list_build(e.ctypes.data, len(buffers), count, None, None, image.data_ptr(), nbytes,
                                       ctypes.byref(info)) == 0
        return info, image.cuda()

    stream = torch.cuda.current_stream().cuda_stream
    result, norms = torch.zeros(2, device="cuda"), torch.zeros(count, device="cuda")
    info, table = build([flat[0], out])
    assert info.chunks == count + 2
    ws = torch.zeros(int(L.gns_tensor_list_workspace_bytes(ctypes.byref(info))), dtype=torch.uint8, device="cuda")
    say("most tensors: clip")
    assert L.gns_grad_clip(ctypes.byref(info), table.data_ptr(), 0, 10.0, 1e-6, None, result.data_ptr(),
                           norms.data_ptr(), ws.data_ptr(), ws.numel(), stream) == 0
    norm = float(old[0].double().square().sum().sqrt())
    assert abs(float(result[0]) - norm) <= 1.01 * U * norm
    assert torch.equal(out, old[0] * result[1]) and torch.equal(flat[0], old[0])
    each = old[0][:3 * (count - 1)].view(-1, 3).double().square().sum(1).sqrt()
    assert bool(((norms[:-1].double() - each).abs() <= 1.01 * U * each).all())
    rest = float(old[0][3 * (count - 1):].double().square().sum().sqrt())
    assert abs(float(norms[-1]) - rest) <= 1.01 * U * rest
    info, table = build(flat)
    say("most tensors: adamw")
    assert L.gns_adamw_step(ctypes.byref(info), table.data_ptr(), 1, 0.02, 0.9, 0.95, 1e-8, 0.0, None, stream) == 0
    # one tensor of the same elements: the same arithmetic, element by element
    gns.adamw_step(gns.adamw_list(old[1:2], old[:1], old[2:3], old[3:]), 1, lr=0.02, betas=(0.9, 0.95), eps=1e-8,
                   weight_decay=0.0)
    assert all(torch.equal(a, b) for a, b in zip(flat, old))


@pytest.mark.parametrize("offset", [0, 1, 31, 64])
@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_adamw_writes_inside_its_arrays(offset, dtype):
    """What lies before and behind every array keeps its bits, and the
    gradients all of them."""
    gns = need_gpu()
    for n in (1, 5, 1023, 1024, 1025, 8192, 3 * 8192 + 1):
        held = [torch.full((n + 300,), 7.0, device="cuda") for _ in range(3)]
        held += [torch.full((n + 300,), 7.0, dtype=torch.bfloat16, device="cuda"),
                 torch.full((n + 300,), 7.0, dtype=dtype, device="cuda")]
        p, m, v, c, g = (t[offset:offset + n] for t in held)
        say("adamw inside", offset, dtype, n)
        gns.adamw_step(gns.adamw_list([p], [g], [m], [v], copies=[c]), 3, lr=0.5, weight_decay=0.1)
        for t in held:
            assert bool((t[:offset] == 7.0).all()) and bool((t[offset + n:] == 7.0).all())
        assert bool((g == 7.0).all())
        for t in (p, m, v, c):                         # every element alike, none left out
            assert bool((t == t[0]).all())
        # m = 0.9 * 7 + 0.1 * 7, v = 0.999 * 7 + 0.001 * 49
        assert math.isclose(float(m[0]), 7.0, rel_tol=12 * U) and math.isclose(float(v[0]), 7.042, rel_tol=12 * U)
        assert float(p[0]) < 7.0 and float(c[0]) == float(p[:1].bfloat16())
