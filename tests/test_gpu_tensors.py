"""Norm, clipping and AdamW over lists of tensors through the C ABI, against
the 64-bit oracle and, where the arithmetic is defined to the bit, against
plain fp32 torch.

Tolerances, from u = 2^-24, the unit roundoff of fp32:
* a norm and a clip factor are fp64 values rounded once: u, and half the
  smallest subnormal; the oracle's rounding is far below;
* a clipped element is to the bit the fp32 product of the gradient and the
  clip factor, rounded to its type;
* AdamW's moments: b1 m + (1 - b1) g with rounded b1, 1 - b1, g * scale,
  scale itself and two more operations: at most 6 u of |b1 m| + |(1 - b1) g|;
  its parameter: 4 u (|p| + |p'|) and, for the update term, whose numerator
  has those 6 u and whose denominator 3 u from v (the 6 u halved by the
  square root), with the root, the bias factors, the division and the rate:
  16 u of rate (|b1 m| + |(1 - b1) g|) / denominator.
"""
import math

import numpy as np
import pytest
import torch

import oracle
from gpu_common import NS5, need_gpu, say
from gram_newton_schulz_amd import synth

pytestmark = pytest.mark.gpu

U = 2.0 ** -24
TINY = 2.0 ** -150
DTYPES = [torch.float32, torch.bfloat16, torch.float16]


def rand(rng, shape, scale, dtype):
    return torch.from_numpy(np.asarray(rng.normal(size=shape) * scale)).to(dtype)


def f64(t):
    return t.detach().cpu().double().numpy()


def check_norm(got, grads, ord, max_norm, inv=1.0, eps=1e-6, each=None):
    norm, clip, norms = oracle.grad_norm([f64(g) for g in grads], ord, max_norm, eps, inv)
    assert abs(float(got.norm) - norm) <= 1.01 * U * norm + TINY
    assert abs(float(got.clip) - clip) <= 1.01 * U * abs(clip) + TINY
    if each is not None:
        for a, b in zip(each.tolist(), norms):
            assert abs(a - b) <= 1.01 * U * b + TINY
    return norm, clip


SIZES = [(1,), (7,), (8,), (9,), (63,), (2048,), (2049,), (8191,), (8192,), (8193,), (100003,), (0,), (3, 0),
         (5, 13), (1, 1), (129, 257), ()]


@pytest.mark.parametrize("dtype", DTYPES + ["mixed"])
@pytest.mark.parametrize("ord", [2, math.inf])
def test_norm_sizes(dtype, ord):
    gns = need_gpu()
    rng = np.random.default_rng(50)
    grads = [rand(rng, s, 10.0 ** rng.uniform(-3, 1), DTYPES[i % 3] if dtype == "mixed" else dtype)
             for i, s in enumerate(SIZES)]
    dev = [g.cuda() for g in grads]
    for max_norm in (0.5, 1e9, math.inf, 0.0):
        say(f"norm {dtype} ord={ord} max_norm={max_norm}")
        got = gns.grad_norm(dev, ord=ord, max_norm=max_norm, per_tensor=True)
        check_norm(got, grads, ord, max_norm, each=got.tensor_norms)
    for g, d in zip(grads, dev):                            # read only
        assert torch.equal(d.cpu(), g)
    for i in range(len(grads)):                             # each alone
        check_norm(gns.grad_norm(dev[i:i + 1], ord=ord, max_norm=0.1), grads[i:i + 1], ord, 0.1)


def test_norm_of_nothing():
    gns = need_gpu()
    for lst in ([], [torch.empty(0, device="cuda")], [torch.empty(0, 4, device="cuda")] * 3):
        say("norm of nothing", len(lst))
        got = gns.grad_norm(lst, max_norm=1.0, per_tensor=True)
        assert float(got.norm) == 0.0 and float(got.clip) == 1.0
        assert got.tensor_norms.tolist() == [0.0] * len(lst)
        got = gns.clip_grad_norm_(lst, 0.0)
        assert float(got.norm) == 0.0
    empty = gns.adamw_list([], [], [], [])
    gns.adamw_step(empty, 1, lr=0.1)
    torch.cuda.synchronize()


def test_norm_range():
    """Squares of the largest and of subnormal fp32 gradients neither overflow
    nor vanish on the way; only a norm beyond fp32 itself is infinite."""
    gns = need_gpu()
    for value, n in ((1e37, 64), (1e-30, 4096), (2.0 ** -149, 999), (3e38, 1)):
        g = torch.full((n,), value, dtype=torch.float32)
        say("norm range", value)
        check_norm(gns.grad_norm([g.cuda()], max_norm=1.0), [g], 2, 1.0)
    got = gns.grad_norm([torch.full((4,), 3e38, device="cuda")], max_norm=1.0)
    assert math.isinf(float(got.norm)) and 0 < float(got.clip) < 1e-38


VIEWS = {
    "offset": lambda b: [b[1:4098], b[4099:4100], b[5003:13196], b[13197:40000]],
    "columns": lambda b: [b[:39990].view(430, 93)[:, i:j] for i, j in ((0, 30), (30, 31), (31, 93))],
    "even columns": lambda b: [b[:38400].view(300, 128)[:, i:j] for i, j in ((0, 64), (64, 80), (80, 128))],
    "narrow": lambda b: [b[:39999].view(13333, 3)[:, 1:2], b[:39999].view(13333, 3)[:, 2:]],
    "transposed": lambda b: [b[:30000].view(100, 300).t(), b[30000:39000].view(90, 100)[:, 7:50].t()],
    "outer": lambda b: [b[:36000].view(12, 30, 100)[:, :, 3:71], b[36000:36600].view(6, 100)[::2]],
    "every second": lambda b: [b[:20000:2], b[20001:40000:2]],
}


@pytest.mark.parametrize("name", list(VIEWS))
@pytest.mark.parametrize("dtype", DTYPES)
def test_views(name, dtype):
    """Strided and misaligned views: their norms, and clipping in place that
    leaves everything between them alone."""
    gns = need_gpu()
    rng = np.random.default_rng(51)
    base = rand(rng, 40000, 0.3, dtype)
    cpu, dev = base.clone(), base.cuda()
    say("views", name, dtype)
    lst = gns.tensor_list(VIEWS[name](dev))
    for ord in (2, math.inf):
        got = gns.grad_norm(lst, ord=ord, max_norm=0.25, per_tensor=True)
        check_norm(got, VIEWS[name](base), ord, 0.25, each=got.tensor_norms)
    got = gns.clip_grad_norm_(lst, 0.25)
    clip = got.clip.cpu()
    for t in VIEWS[name](cpu):
        t.copy_((t.float() * clip).to(dtype))
    assert torch.equal(dev.cpu(), cpu)


def test_expanded_gradients():
    """Gradients that repeat one element or row, as the backward of a sum
    leaves: they have a norm and are refused where they would be written."""
    gns = need_gpu()
    row = torch.arange(1.0, 6.0)
    grads = [torch.tensor(0.5).expand(300, 7), row.expand(40, 5), row.unsqueeze(1).expand(5, 11)]
    dev = [torch.tensor(0.5).cuda().expand(300, 7), row.cuda().expand(40, 5), row.cuda().unsqueeze(1).expand(5, 11)]
    say("expanded")
    got = gns.grad_norm(dev, max_norm=1.0, per_tensor=True)
    check_norm(got, grads, 2, 1.0, each=got.tensor_norms)
    with pytest.raises(gns.GnsError) as e:
        gns.clip_grad_norm_(dev, 1.0)
    assert e.value.name == "GNS_E_ALIAS"
    out = [torch.empty(300, 7, device="cuda"), torch.empty(40, 5, device="cuda"), torch.empty(5, 11, device="cuda")]
    with pytest.raises(gns.GnsError):
        gns.tensor_list(dev[2:], out=out[2:])        # rows that have no common form with the output's
    got = gns.clip_grad_norm_(gns.tensor_list(dev[:2], out=out[:2]), 1.0)
    for o, g in zip(out, grads[:2]):
        assert torch.equal(o.cpu(), g * got.clip.cpu())


@pytest.mark.parametrize("src", DTYPES)
@pytest.mark.parametrize("dst", [None] + DTYPES)
def test_clip_types(src, dst):
    gns = need_gpu()
    rng = np.random.default_rng(52)
    grads = [rand(rng, s, 0.5, src) for s in SIZES]
    dev = [g.cuda() for g in grads]
    out = None if dst is None else [torch.full(g.shape, float("nan"), dtype=dst, device="cuda") for g in grads]
    inv = torch.tensor(0.125, device="cuda")
    say("clip", src, dst)
    got = gns.clip_grad_norm_(gns.tensor_list(dev, out=out), 3.0, inv_scale=inv, per_tensor=True)
    check_norm(got, grads, 2, 3.0, inv=0.125, each=got.tensor_norms)
    c32 = got.clip.cpu()
    for i, g in enumerate(grads):
        t = (dev if out is None else out)[i]
        assert torch.equal(t.cpu(), (g.float() * c32).to(t.dtype))
        if out is not None:
            assert torch.equal(dev[i].cpu(), g)


def test_clip_views_into_views():
    """Misaligned 16-bit slices clipped into slices of another pitch and type."""
    gns = need_gpu()
    rng = np.random.default_rng(53)
    src = rand(rng, (211, 150), 0.5, torch.bfloat16)
    dst = torch.full((211, 187), 7.0)
    cut = [(0, 33), (33, 34), (35, 150)]
    s, d = src.cuda(), dst.cuda()
    say("clip views into views")
    got = gns.clip_grad_norm_(gns.tensor_list([s[:, i:j] for i, j in cut], out=[d[:, i + 5:j + 5] for i, j in cut]),
                              0.5, ord=math.inf)
    check_norm(got, [src[:, i:j] for i, j in cut], math.inf, 0.5)
    for i, j in cut:
        dst[:, i + 5:j + 5] = src[:, i:j].float() * got.clip.cpu()
    assert torch.equal(d.cpu(), dst)


def test_clip_dense_into_slices_and_back():
    """Dense gradients into column slices, and slices into dense outputs."""
    gns = need_gpu()
    rng = np.random.default_rng(75)
    for src, dst in ((torch.bfloat16, torch.float32), (torch.float32, torch.float16)):
        g = rand(rng, (97, 45), 0.5, src)
        wide = torch.full((97, 60), 3.0, dtype=dst, device="cuda")
        say("dense into slices", src, dst)
        got = gns.clip_grad_norm_(gns.tensor_list([g.cuda()], out=[wide[:, 7:52]]), 0.5)
        want = (g.float() * got.clip.cpu()).to(dst)
        assert torch.equal(wide[:, 7:52].cpu(), want)
        assert bool((wide[:, :7] == 3.0).all()) and bool((wide[:, 52:] == 3.0).all())
        dense = torch.zeros(97, 45, dtype=dst, device="cuda")
        big = torch.zeros(97, 60, dtype=src, device="cuda")
        big[:, 7:52] = g.cuda()
        gns.clip_grad_norm_(gns.tensor_list([big[:, 7:52]], out=[dense]), 0.5)
        assert torch.equal(dense.cpu(), want)


@pytest.mark.parametrize("offset", [0, 1, 3, 31, 64])
@pytest.mark.parametrize("dtype", DTYPES)
def test_chunk_edges(offset, dtype):
    """Lengths around whole chunks, from starts of every alignment: each
    element is read and scaled exactly once, and nothing around it is."""
    gns = need_gpu()
    rng = np.random.default_rng(76)
    lengths = [8192 * k + d for k in (1, 2, 3) for d in (-65, -1, 0, 1, 63, 64)]
    flat = rand(rng, sum(lengths) + 200 * len(lengths), 0.5, dtype)
    dev, cpu = flat.cuda(), flat.clone()

    def views(base):
        out, at = [], 0
        for n in lengths:
            out.append(base[at + offset:at + offset + n])
            at += n + 200
        return out

    say("chunk edges", offset, dtype)
    got = gns.grad_norm(views(dev), max_norm=10.0, per_tensor=True)
    check_norm(got, views(cpu), 2, 10.0, each=got.tensor_norms)
    got = gns.clip_grad_norm_(views(dev), 10.0)
    for t in views(cpu):
        t.copy_((t.float() * got.clip.cpu()).to(dtype))
    assert torch.equal(dev.cpu(), cpu)
    for n in (8192 * 3 + 1, 5, 8192):
        p, m, v = (torch.zeros(n + 300, device="cuda") for _ in range(3))
        g = rand(rng, n, 0.5, dtype).cuda()
        view = [[t[offset:offset + n]] for t in (p, m, v)]
        gns.adamw_step(gns.adamw_list(view[0], [g], view[1], view[2]), 1, lr=0.5, weight_decay=0.0)
        # the first step from zero moves every parameter by -lr g / (|g| + eps)
        want = -0.5 * g.double() / (g.double().abs() + 1e-8)
        assert torch.allclose(p[offset:offset + n].double(), want, rtol=0, atol=1e-4)
        assert not p[:offset].any() and not p[offset + n:].any()
        assert not m[:offset].any() and not v[offset + n:].any()


@pytest.mark.parametrize("chunks", [3, 4, 5, 511, 512, 513, 4096, 4097])
@pytest.mark.parametrize("ord", [2, math.inf])
def test_number_of_chunks(chunks, ord):
    """Around the numbers of chunks at which the sum of the partials moves from
    one launch to another: `chunks` tensors of one chunk each."""
    gns = need_gpu()
    rng = np.random.default_rng(77)
    values = rand(rng, (chunks, 5), 0.5, torch.float32)
    dev = values.cuda()
    say("number of chunks", chunks, ord)
    lst = gns.tensor_list(list(dev))
    assert lst.info.chunks == chunks
    for per_tensor in (False, True):
        got = gns.grad_norm(lst, ord=ord, max_norm=1.0, per_tensor=per_tensor)
        check_norm(got, list(values), ord, 1.0, each=got.tensor_norms)
    got = gns.clip_grad_norm_(lst, 1.0, ord=ord)
    check_norm(got, list(values), ord, 1.0)
    assert torch.equal(dev.cpu(), values * got.clip.cpu())


def test_small_list_of_large_and_small_entries():
    """One launch, entries of one, of a few and of many chunks."""
    gns = need_gpu()
    rng = np.random.default_rng(79)
    sizes = [3, 8192 * 40 + 17, 0, 8192 * 3, 1, 8192 * 17, 8192 * 200 + 5, 8192 * 16 + 1, 9000]
    grads = [rand(rng, n, 0.1 * (i + 1), DTYPES[i % 3]) for i, n in enumerate(sizes)]
    dev = [g.cuda() for g in grads]
    for ord in (2, math.inf):
        say("large and small entries", ord)
        lst = gns.tensor_list(dev)
        assert 128 < lst.info.chunks <= 512
        for _ in range(3):
            got = gns.grad_norm(lst, ord=ord, max_norm=1.0, per_tensor=True)
            check_norm(got, grads, ord, 1.0, each=got.tensor_norms)


@pytest.mark.parametrize("count", [3, 600, 5000])
@pytest.mark.parametrize("clip", [False, True])
def test_writes_stay_inside(count, clip):
    """Result, tensor norms and workspace of exactly their sizes inside larger
    buffers, whose other bytes keep what they hold; the first 256 bytes of the
    workspace are zero again after every call."""
    gns = need_gpu()
    L = gns.lib()
    rng = np.random.default_rng(81)
    values = rand(rng, (count, 40), 0.5, torch.float32)
    dev = values.cuda()
    lst = gns.tensor_list(list(dev))
    need = lst.workspace_bytes
    arena = torch.full((1024 + need + 1024,), 77, dtype=torch.uint8, device="cuda")
    lo = -arena.data_ptr() % 256 + 256
    arena[lo:lo + 256] = 0
    floats = torch.full((count + 40,), 7.0, device="cuda")
    result, norms = floats[8:10], floats[20:20 + count]
    torch.cuda.synchronize()
    say("writes stay inside", count, clip)
    for _ in range(3):
        dev.copy_(values)
        st = (L.gns_grad_clip if clip else L.gns_grad_norm)(
            lst._info, lst._table, 0, 1.0, 1e-6, None, result.data_ptr(), norms.data_ptr(),
            arena.data_ptr() + lo, need, torch.cuda.current_stream().cuda_stream)
        assert st == 0
        norm, factor, each = oracle.grad_norm([f64(v) for v in values], 2, 1.0)
        assert abs(float(result[0]) - norm) <= 1.01 * U * norm and abs(float(result[1]) - factor) <= 1.01 * U * factor
        assert np.all(np.abs(f64(norms) - np.array(each)) <= 1.01 * U * np.array(each))
        assert not arena[lo:lo + 256].any()
    assert bool((arena[:lo] == 77).all()) and bool((arena[lo + need:] == 77).all())
    assert bool((floats[:8] == 7.0).all()) and bool((floats[10:20] == 7.0).all())
    assert bool((floats[20 + count:] == 7.0).all())


def test_list_beyond_the_cache():
    """More gradients than the last-level cache holds (loads of both kinds,
    chunks in parts), of odd sizes; against torch in fp64 and to the bit."""
    gns = need_gpu()
    gen = torch.Generator(device="cuda").manual_seed(78)
    for dtype, out_dtype in ((torch.bfloat16, torch.float32), (torch.bfloat16, None), (torch.float32, torch.bfloat16)):
        sizes = (70000001, 90000, 81234567) if dtype == torch.bfloat16 else (70000001, 90000, 3)
        g = [torch.empty(n, device="cuda").normal_(0, 0.01, generator=gen).to(dtype) for n in sizes]
        out = None if out_dtype is None else [torch.zeros(n, dtype=out_dtype, device="cuda") for n in sizes]
        lst = gns.tensor_list(g, out=out)
        assert lst.info.keep_from > 0
        norms = [float(t.double().square().sum().sqrt()) for t in g]
        norm = math.sqrt(sum(n * n for n in norms))
        say("beyond the cache", dtype, out_dtype)
        got = gns.grad_norm(lst, max_norm=1.0, per_tensor=True)
        assert abs(float(got.norm) - norm) <= 1.01 * U * norm
        for a, b in zip(got.tensor_norms.tolist(), norms):
            assert abs(a - b) <= 1.01 * U * b
        want = [(t.float() * got.clip).to(out_dtype or dtype) for t in g]
        gns.clip_grad_norm_(lst, 1.0)
        for a, b in zip(out or g, want):
            assert torch.equal(a, b)


def test_clip_below_the_bound_changes_nothing():
    gns = need_gpu()
    rng = np.random.default_rng(54)
    grads = [rand(rng, (300, 70), 0.5, torch.float16), rand(rng, 17, 0.5, torch.float32)]
    dev = [g.cuda() for g in grads]
    out = [torch.zeros_like(d) for d in dev]
    say("clip below the bound")
    got = gns.clip_grad_norm_(dev, 1e4)
    assert float(got.clip) == 1.0
    gns.clip_grad_norm_(gns.tensor_list(dev, out=out), 1e4)
    for g, d, o in zip(grads, dev, out):
        assert torch.equal(d.cpu(), g) and torch.equal(o.cpu(), g)
    got = gns.clip_grad_norm_(dev, 0.0)                     # bound zero
    assert float(got.clip) == 0.0 and all(not d.any() for d in dev)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("bad", [math.inf, -math.inf, math.nan])
@pytest.mark.parametrize("ord", [2, math.inf])
def test_nonfinite(dtype, bad, ord):
    """One Inf or NaN makes the norm so and the factor NaN; clipping and AdamW
    then write nothing."""
    gns = need_gpu()
    rng = np.random.default_rng(55)
    for at in (0, 777, 20010):
        grads = [rand(rng, 20011, 0.5, dtype), rand(rng, 64, 0.5, dtype)]
        grads[0][at] = bad
        dev = [g.cuda() for g in grads]
        say("nonfinite", dtype, bad, ord, at)
        got = gns.clip_grad_norm_(dev, 1.0, ord=ord, per_tensor=True)
        norm = float(got.norm)
        assert math.isnan(norm) if math.isnan(bad) else norm == math.inf
        assert math.isnan(float(got.clip)) and math.isfinite(float(got.tensor_norms[1]))
        for g, d in zip(grads, dev):
            assert torch.equal(d.cpu().view(torch.uint8), g.view(torch.uint8))
        out = [torch.full_like(d, 3.0) for d in dev]
        gns.clip_grad_norm_(gns.tensor_list(dev, out=out), 1.0, ord=ord)
        assert all(bool((o == 3.0).all()) for o in out)
        state = [[torch.rand(g.shape, device="cuda") for g in grads] for _ in range(3)]
        copies = [torch.full(g.shape, 9.0, dtype=torch.bfloat16, device="cuda") for g in grads]
        kept = [[t.clone() for t in a] for a in state]
        gns.adamw_step(gns.adamw_list(state[0], dev, state[1], state[2], copies=copies), 3, lr=0.1,
                       weight_decay=0.1, grad_scale=got.clip)
        for a, b in zip(state, kept):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        assert all(bool((c == 9.0).all()) for c in copies)


def adamw_case(gns, shapes, grad_dtype, copy_dtype, seed, scale=None, lr_scales=None, wd_scales=None, make=None,
               steps=1, first=1):
    rng = np.random.default_rng(seed)
    lr, betas, eps, wd = 0.02, (0.9, 0.95), 1e-8, 0.3
    cpu = {k: [rand(rng, s, sc, torch.float32) for s in shapes] for k, sc in (("p", 1.0), ("m", 0.1))}
    cpu["v"] = [rand(rng, s, 0.1, torch.float32).square() for s in shapes]
    cpu["g"] = [rand(rng, s, 0.5, DTYPES[i % 3] if grad_dtype == "mixed" else grad_dtype)
                for i, s in enumerate(shapes)]
    dev = {k: [make(k, t) if make else t.cuda() for t in v] for k, v in cpu.items()}
    copies = None
    if copy_dtype is not None:
        copies = [(make("c", t.to(copy_dtype)) if make else torch.zeros(t.shape, dtype=copy_dtype, device="cuda"))
                  for t in cpu["p"]]
    lst = gns.adamw_list(dev["p"], dev["g"], dev["m"], dev["v"], copies=copies, lr_scales=lr_scales,
                         wd_scales=wd_scales)
    gs = None if scale is None else torch.tensor(scale, device="cuda")
    s64 = 1.0 if scale is None else float(np.float32(scale))
    for step in range(first, first + steps):
        say("adamw", grad_dtype, copy_dtype, step)
        gns.adamw_step(lst, step, lr=lr, betas=betas, eps=eps, weight_decay=wd, grad_scale=gs)
        for i in range(len(shapes)):
            p, g, m, v = (f64(cpu[k][i]) for k in "pgmv")
            eta = lr * (lr_scales[i] if lr_scales else 1.0)
            decay = wd * (wd_scales[i] if wd_scales else 1.0)
            rp, rm, rv = oracle.adamw(p, g, m, v, step, eta, betas, eps, decay, s64)
            gp, gm, gv = (f64(dev[k][i]) for k in "pmv")
            mag = np.abs(betas[0] * m) + np.abs((1 - betas[0]) * g * s64)
            assert np.all(np.abs(gm - rm) <= 6 * U * mag + 2.0 ** -148)
            assert np.all(np.abs(gv - rv) <= 6 * U * rv + 2.0 ** -148)
            denom = np.sqrt(rv / (1 - betas[1] ** step)) + eps
            term = abs(eta) / (1 - betas[0] ** step) * mag / denom
            assert np.all(np.abs(gp - rp) <= 4 * U * (np.abs(p) + np.abs(rp)) + 16 * U * term + 2.0 ** -148)
            if copies is not None:
                assert torch.equal(copies[i].cpu(), dev["p"][i].cpu().to(copy_dtype))
            assert torch.equal(dev["g"][i].cpu(), cpu["g"][i])
            for k in "pmv":                                 # the next step starts from what the GPU has
                cpu[k][i] = dev[k][i].cpu().clone()
    return lst


@pytest.mark.parametrize("grad", DTYPES + ["mixed"])
@pytest.mark.parametrize("copy", [None] + DTYPES)
def test_adamw_sizes(grad, copy):
    gns = need_gpu()
    adamw_case(gns, SIZES, grad, copy, 60)


def test_adamw_scales_and_steps():
    """A clip factor, factors per tensor on rate and decay, several steps,
    and a late one."""
    gns = need_gpu()
    shapes = [(33, 65), (7,), (4096,)]
    adamw_case(gns, shapes, torch.float16, torch.bfloat16, 61, scale=0.037, lr_scales=[1.0, 0.25, 3.0],
               wd_scales=[1.0, 0.0, 2.0], steps=3)
    adamw_case(gns, shapes, torch.bfloat16, None, 62, scale=0.0, first=100000)


@pytest.mark.parametrize("pad", [1, 3, 8])
def test_adamw_views(pad):
    """Every array a column slice of a pitch of its own; the columns between
    keep what they held."""
    gns = need_gpu()
    held = []

    def make(kind, t):
        if t.dim() != 2:
            return t.cuda()
        extra = pad * (1 + "pgmvc".index(kind))
        base = torch.full((t.shape[0], t.shape[1] + extra), 5.0, dtype=t.dtype, device="cuda")
        view = base[:, extra // 2:extra // 2 + t.shape[1]]
        view.copy_(t)
        held.append((base, extra // 2, t.shape[1]))
        return view

    adamw_case(gns, [(33, 65), (128, 64), (50, 3), (17,)], torch.bfloat16, torch.float16, 63, scale=0.5, make=make)
    for base, lo, cols in held:
        assert bool((base[:, :lo] == 5.0).all()) and bool((base[:, lo + cols:] == 5.0).all())


def test_adamw_zero_state():
    """The first step from zero moments, where a zero gradient leaves 0 / eps."""
    gns = need_gpu()
    p, g = torch.full((9,), 2.0), torch.tensor([0.0, 1.0, -1.0, 1e-20, 3.0, -3.0, 0.0, 1e4, -1e-4])
    m, v = torch.zeros(9), torch.zeros(9)
    d = [t.cuda() for t in (p, g, m, v)]
    gns.adamw_step(gns.adamw_list([d[0]], [d[1]], [d[2]], [d[3]]), 1, lr=0.1, betas=(0.9, 0.999), eps=1e-8,
                   weight_decay=0.0)
    # v = (1 - b2) g^2 underflows at |g| = 1e-20 (1e-43 is a subnormal of 71 steps): its root is
    # good to 1 part in 140 and eps = 1e-8 swamps it, so the update is 1e-13
    want = 2.0 - 0.1 * g.double() / (g.double().abs() + 1e-8)
    assert torch.allclose(d[0].cpu().double(), want, rtol=0, atol=1e-6)


def test_many_tensors():
    """Thousands of small tensors in one call."""
    gns = need_gpu()
    rng = np.random.default_rng(64)
    grads = [rand(rng, int(n), 0.1, DTYPES[i % 3]) for i, n in enumerate(rng.integers(0, 300, 3000))]
    say("many tensors")
    got = gns.grad_norm([g.cuda() for g in grads], max_norm=1.0, per_tensor=True)
    check_norm(got, grads, 2, 1.0, each=got.tensor_norms)


def test_offsets_beyond_32_bits():
    """Element offsets past 2^32: a few rows very far apart, and one dense
    tensor of more than 2^31 elements."""
    gns = need_gpu()
    pitch = (1 << 31) + 40
    base = torch.zeros(2 * pitch + 1000, dtype=torch.bfloat16, device="cuda")
    view = base.as_strided((3, 701), (pitch, 1), 5)
    rng = np.random.default_rng(65)
    rows = rand(rng, (3, 701), 1.0, torch.bfloat16)
    view.copy_(rows)
    say("offsets beyond 32 bits: view")
    got = gns.clip_grad_norm_([view], 1.0)
    check_norm(got, [rows], 2, 1.0)
    want = (rows.float() * got.clip.cpu()).to(torch.bfloat16)
    assert torch.equal(view.cpu(), want)
    say("offsets beyond 32 bits: dense")
    got = gns.clip_grad_norm_([base[1:]], 0.5)
    check_norm(got, [want], 2, 0.5)
    assert torch.equal(view.cpu(), (want.float() * got.clip.cpu()).to(torch.bfloat16))
    assert int(torch.count_nonzero(base[5 + 701:5 + pitch])) == 0


def test_norm_of_shards():
    """Gradients in shards: the norm of the shards' norms is that of all of
    them (each rounded once, so two roundings), and a shard's NaN reaches it."""
    gns = need_gpu()
    rng = np.random.default_rng(80)
    shards = [[rand(rng, n, 0.3, torch.bfloat16) for n in sizes] for sizes in ((5000, 3), (70001,), (12, 9, 40000))]
    for ord in (2, math.inf):
        say("norm of shards", ord)
        parts = torch.stack([gns.grad_norm([g.cuda() for g in shard], ord=ord).norm for shard in shards])
        got = gns.grad_norm([parts], ord=ord, max_norm=1.0)
        norm, clip, _ = oracle.grad_norm([f64(g) for shard in shards for g in shard], ord, 1.0)
        assert abs(float(got.norm) - norm) <= 2.02 * U * norm
        assert abs(float(got.clip) - clip) <= 2.02 * U * clip
        parts[1] = math.nan
        assert math.isnan(float(gns.grad_norm([parts], ord=ord, max_norm=1.0).clip))


def test_repeats_are_identical():
    gns = need_gpu()
    rng = np.random.default_rng(66)
    dev = [rand(rng, n, 0.1, torch.bfloat16).cuda() for n in (300001, 17, 90000)]
    lst = gns.tensor_list(dev)
    say("repeats")
    first = gns.grad_norm(lst, max_norm=0.3).result.cpu()
    for _ in range(20):
        assert torch.equal(gns.grad_norm(lst, max_norm=0.3).result.cpu(), first)


def test_other_streams():
    """A list built on one stream and used on others, by object and by raw
    handle, with work queued on them before and after."""
    gns = need_gpu()
    rng = np.random.default_rng(67)
    g = rand(rng, 500003, 0.1, torch.float32)
    side = torch.cuda.Stream()
    dev = torch.zeros(500003, device="cuda")
    src = g.cuda()
    torch.cuda.synchronize()
    for stream in (side, side.cuda_stream):
        with torch.cuda.stream(side):
            dev.copy_(src)
        say("other streams")
        lst = gns.tensor_list([dev])                        # on the default stream
        got = gns.clip_grad_norm_(lst, 1.0, stream=stream)
        with torch.cuda.stream(side):
            after = dev * 2
            clip, norm = got.clip.clone(), got.norm.clone()
        side.synchronize()
        assert torch.equal(after.cpu(), g * clip.cpu() * 2)
        n64, _, _ = oracle.grad_norm([f64(g)])
        assert abs(float(norm) - n64) <= 1.01 * U * n64
    one_shot = gns.grad_norm([src], stream=side)
    side.synchronize()
    assert abs(float(one_shot.norm) - n64) <= 1.01 * U * n64


def test_list_of_a_side_stream():
    """A list built on a side stream, right behind the work that fills its
    tensors, and used on the default stream once that is ordered."""
    gns = need_gpu()
    rng = np.random.default_rng(82)
    g = rand(rng, 300001, 0.1, torch.float32)
    src = g.cuda()
    dev = torch.zeros(300001, device="cuda")
    torch.cuda.synchronize()
    side = torch.cuda.Stream()
    say("list of a side stream")
    with torch.cuda.stream(side):
        dev.copy_(src)
        lst = gns.tensor_list([dev])
        on_side = gns.grad_norm(lst).norm.clone()
    torch.cuda.current_stream().wait_stream(side)
    for stream in (None, 0, torch.cuda.default_stream()):
        got = gns.grad_norm(lst, max_norm=1.0, stream=stream)
        check_norm(got, [g], 2, 1.0)
        assert float(got.norm) == float(on_side)


def test_capture_by_stream_argument():
    """A call captured through its stream argument, from a list whose home is
    another stream."""
    gns = need_gpu()
    g = torch.full((5000,), 0.25, device="cuda")
    lst = gns.tensor_list([g])
    gns.grad_norm(lst)
    torch.cuda.synchronize()
    graph, stream = torch.cuda.CUDAGraph(), torch.cuda.Stream()
    say("capture by stream argument")
    with torch.cuda.graph(graph, stream=stream):
        got = gns.grad_norm(lst, max_norm=1.0, stream=stream)
    for value in (0.25, 2.0, 0.5):
        g.fill_(value)
        torch.cuda.synchronize()
        graph.replay()
        torch.cuda.synchronize()
        check_norm(got, [torch.full((5000,), value)], 2, 1.0)
        check_norm(gns.grad_norm(lst, max_norm=1.0), [torch.full((5000,), value)], 2, 1.0)


def test_graph_replay():
    """Norm, clip factor and AdamW captured into one graph; every replay equals
    the eager step bit for bit, with eager work between the replays."""
    gns = need_gpu()
    rng = np.random.default_rng(68)
    shapes = [(300, 70), (999,), (64, 64)]
    cpu = [[rand(rng, s, 0.5, torch.float32) for s in shapes] for _ in range(4)]
    cpu[3] = [t.square() for t in cpu[3]]
    dev = [[t.cuda() for t in a] for a in cpu]
    lst = gns.adamw_list(dev[0], dev[1], dev[2], dev[3])

    def reset():
        for a, b in zip(dev, cpu):
            for d, c in zip(a, b):
                d.copy_(c)

    def step():
        got = gns.grad_norm(lst, max_norm=0.5)
        gns.adamw_step(lst, 5, lr=0.1, weight_decay=0.1, grad_scale=got.clip)
        got = gns.clip_grad_norm_(lst, 0.25)
        return got.result

    say("graph eager")
    eager_result = step().clone()
    eager = [[t.clone() for t in a] for a in dev]
    reset()
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    say("graph capture")
    with torch.cuda.graph(graph):
        result = step()
        with pytest.raises(gns.GnsError):
            gns.tensor_list(dev[0])                         # building copies to the GPU
    for rep in range(4):
        reset()
        say("graph replay", rep)
        graph.replay()
        torch.cuda.synchronize()
        assert torch.equal(result, eager_result)
        for a, b in zip(dev, eager):
            assert all(torch.equal(x, y) for x, y in zip(a, b))
        reset()
        assert torch.equal(step(), eager_result)
        torch.cuda.synchronize()


def test_argument_errors():
    gns = need_gpu()
    g = torch.ones(8, device="cuda")
    lst = gns.tensor_list([g])

    def refuses(name, f):
        with pytest.raises(gns.GnsError) as e:
            f()
        assert e.value.name == name

    refuses("GNS_E_PARAM", lambda: gns.grad_norm(lst, ord=3))
    refuses("GNS_E_PARAM", lambda: gns.clip_grad_norm_(lst, -1.0))
    refuses("GNS_E_DTYPE", lambda: gns.grad_norm(lst, inv_scale=torch.ones(2, device="cuda")))
    refuses("GNS_E_DTYPE", lambda: gns.grad_norm(lst, inv_scale=torch.ones(1, device="cuda", dtype=torch.float64)))
    refuses("GNS_E_NULL", lambda: gns.grad_norm(lst, inv_scale=torch.ones(1)))
    refuses("GNS_E_WORKSPACE", lambda: gns.grad_norm(lst, workspace=torch.empty(4, dtype=torch.uint8, device="cuda")))
    refuses("GNS_E_DTYPE", lambda: gns.tensor_list([torch.ones(4, dtype=torch.int32, device="cuda")]))
    refuses("GNS_E_SHAPE", lambda: gns.adamw_step(lst, 1, lr=0.1))
    refuses("GNS_E_ALIAS", lambda: gns.clip_grad_norm_([g, g], 1.0))
    refuses("GNS_E_SHAPE", lambda: gns.tensor_list([torch.ones(4, 5, 6, device="cuda")[:, ::2, :3]]))
    half = [torch.ones(8, dtype=torch.bfloat16, device="cuda")]
    refuses("GNS_E_DTYPE", lambda: gns.adamw_step(gns.adamw_list(half, [g], [g.clone()], [g.clone()]), 1, lr=0.1))
    assert torch.equal(g.cpu(), torch.ones(8))


def test_timing_records():
    gns = need_gpu()
    g = torch.ones(1000, device="cuda")
    gns.timing_reset()
    gns.timing_enable(True)
    try:
        gns.grad_norm([g])
        gns.clip_grad_norm_([g], 1.0)
        names = [r[0] for r in gns.timing_read()]
    finally:
        gns.timing_enable(False)
        gns.timing_reset()
    assert names == ["grad_norm", "grad_clip"]
