"""Calls of the embedding and of MXFP4 layers that are refused before anything
reaches the GPU (none needed here; no pointer below is ever dereferenced)."""
import ctypes
import math
import os

import pytest
import torch

gns = pytest.importorskip("gram_newton_schulz_amd")
from gram_newton_schulz_amd.layers import Matrix  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(gns.LIB_PATH),
                                reason="libgns.so not built (run __graft_entry__.build())")

E = {"OK": 0, "NULL": 1, "SHAPE": 2, "DTYPE": 3, "ALIAS": 7, "WORKSPACE": 8, "PARAM": 11}
F32, BF16, F16, BF16X3 = 0, 1, 2, 3
A, B, C, D, W = (0x100000000000 + i * 0x10000000000 for i in range(5))     # far apart


def embedding(tokens=A, bits=64, count=10, weight=B, wt=BF16, vocab=100, width=16, pitch=16, scale=1.0, out=C, ot=F32,
              out_pitch=16):
    return gns.lib().gns_embedding(tokens, bits, count, weight, wt, vocab, width, pitch, scale, out, ot, out_pitch, None)


def gradient(tokens=A, bits=64, count=10, grad=B, gt=BF16, pitch=16, vocab=100, width=16, scale=1.0, into=C, wt=F32,
             into_pitch=16, accumulate=0, ws=W, ws_bytes=1 << 40):
    return gns.lib().gns_embedding_grad(tokens, bits, count, grad, gt, pitch, vocab, width, scale, into, wt, into_pitch,
                                        accumulate, ws, ws_bytes, None)


SIZES = [dict(count=-1), dict(count=(1 << 30) + 1), dict(vocab=-1), dict(vocab=1 << 31), dict(width=-1),
         dict(width=(1 << 24) + 1), dict(pitch=-1), dict(pitch=1 << 60), dict(count=1 << 30, width=1 << 20)]


@pytest.mark.parametrize("call", [embedding, gradient])
def test_embedding_arguments(call):
    for kw in SIZES:
        assert call(**kw) == E["SHAPE"], kw
    for kw in (dict(wt=BF16X3), dict(wt=7), dict(wt=-1), dict(**{"ot" if call is embedding else "gt": BF16X3})):
        assert call(**kw) == E["DTYPE"], kw
    for kw in (dict(bits=16), dict(bits=0), dict(scale=math.nan), dict(scale=math.inf), dict(scale=1e300),
               dict(tokens=A + 4), dict(bits=32, tokens=A + 2), dict(**{"out" if call is embedding else "into": C + 2}),
               dict(**{"weight" if call is embedding else "grad": B + 1})):
        assert call(**kw) == E["PARAM"], kw
    for name in ("tokens", "weight", "out") if call is embedding else ("tokens", "grad", "into"):
        assert call(**{name: None}) == E["NULL"], name


def test_embedding_written_rows_do_not_overlap():
    assert embedding(out_pitch=15) == E["SHAPE"] and embedding(out_pitch=0) == E["SHAPE"]
    assert gradient(into_pitch=15) == E["SHAPE"] and gradient(into_pitch=0) == E["SHAPE"]
    assert gradient(accumulate=2) == E["PARAM"]


def test_embedding_aliases():
    assert embedding(out=B, ot=BF16) == E["ALIAS"]
    assert embedding(out=B + 2 * 16 * 99 + 28) == E["ALIAS"]                # the last element of the last row
    assert embedding(out=A) == E["ALIAS"] and embedding(out=A + 72) == E["ALIAS"]
    assert embedding(out=B + 64, ot=BF16, out_pitch=64, pitch=64, width=40) == E["ALIAS"]  # slices that touch
    assert gradient(into=B) == E["ALIAS"] and gradient(into=A) == E["ALIAS"]
    assert gradient(count=20000, ws=C) == E["ALIAS"] and gradient(count=20000, ws=B) == E["ALIAS"]
    assert gradient(count=20000, ws=A + 256) == E["ALIAS"]


def test_embedding_workspace():
    need = gns.embedding_grad_workspace_bytes(20000, 100, 16)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=W + 128), dict(ws_bytes=need - 1)):
        assert gradient(count=20000, **kw) == E["WORKSPACE"], kw
    for kw in SIZES[:6]:
        z = dict(count=10, vocab=100, width=16)
        z.update(kw)
        assert gns.embedding_grad_workspace_bytes(z["count"], z["vocab"], z["width"]) == 0


def test_embedding_of_nothing():
    assert embedding(count=0, tokens=None, out=None) == E["OK"]
    assert embedding(width=0, tokens=None, out=None, weight=None) == E["OK"]
    assert gradient(vocab=0, into=None) == E["OK"] and gradient(width=0, grad=None, into=None) == E["OK"]
    assert gradient(count=0, tokens=None, grad=None, accumulate=1) == E["OK"]


def mx(codes=A, scales=A + (1 << 36), batch=2, rows=40, cols=200):
    return Matrix(codes, scales, batch, rows, cols)


def ref(m):
    return None if m is None else ctypes.byref(m)


def quantize(x=B, dtype=BF16, pitch=200, stride=8000, noise=None, rows=mx(), columns=None):
    return gns.lib().gns_mxfp4_quantize(x, dtype, pitch, stride, noise, ref(rows), ref(columns), None)


def test_sizes_of_mxfp4():
    L = gns.lib()
    assert L.gns_mxfp4_code_bytes(3, 5, 129) == 3 * 5 * 128 and L.gns_mxfp4_scale_bytes(3, 33, 129) == 3 * 2 * 2 * 128
    assert L.gns_mxfp4_code_bytes(0, 5, 5) == 0 and L.gns_mxfp4_scale_bytes(1, 0, 5) == 0
    for bad in ((-1, 5, 5), (1, -5, 5), (1, 5, -5), (1, (1 << 23) + 1, 5), (1, 5, (1 << 23) + 1), (1 << 41, 64, 64)):
        assert L.gns_mxfp4_code_bytes(*bad) == 0 and L.gns_mxfp4_scale_bytes(*bad) == 0
        assert L.gns_mxfp4_matmul_workspace_bytes(bad[0], bad[1], 5, bad[2]) == 0
        assert L.gns_mxfp4_linear_workspace_bytes(bad[0], 5, bad[1], bad[2]) == 0


def test_quantize_arguments():
    turned = mx(C, C + (1 << 36), rows=200, cols=40)
    assert quantize(rows=None) == E["NULL"] and quantize(x=None) == E["NULL"]
    assert quantize(rows=mx(codes=None)) == E["NULL"] and quantize(rows=mx(scales=None)) == E["NULL"]
    assert quantize(rows=None, columns=mx(C, None, rows=200, cols=40)) == E["NULL"]
    for kw in (dict(rows=mx(batch=-1)), dict(rows=mx(rows=-1)), dict(rows=mx(cols=(1 << 23) + 1)), dict(pitch=-1),
               dict(stride=-1), dict(pitch=1 << 60), dict(stride=1 << 60), dict(columns=mx(C, D, rows=200, cols=41)),
               dict(columns=mx(C, D, batch=3, rows=200, cols=40)), dict(columns=mx(C, D)),
               dict(rows=mx(batch=1, rows=1 << 23, cols=1 << 23))):
        assert quantize(**kw) == E["SHAPE"], kw
    for dtype in (BF16X3, -1, 9):
        assert quantize(dtype=dtype) == E["DTYPE"]
    for kw in (dict(x=B + 1), dict(dtype=F32, x=B + 2), dict(rows=mx(codes=A + 8)), dict(rows=mx(scales=C + 4)),
               dict(columns=mx(C + 1, D, rows=200, cols=40))):
        assert quantize(**kw) == E["PARAM"], kw
    for kw in (dict(rows=mx(codes=B)), dict(rows=mx(scales=B + 2 * 8000)), dict(rows=mx(A, A)),
               dict(noise=A), dict(noise=A + 100), dict(columns=mx(A, D, rows=200, cols=40)),
               dict(columns=mx(C, A + (1 << 36), rows=200, cols=40))):
        assert quantize(**kw) == E["ALIAS"], kw
    for empty in (dict(rows=mx(batch=0)), dict(rows=mx(rows=0)), dict(rows=mx(None, None, cols=0))):
        assert quantize(x=None, **empty) == E["OK"]
    assert turned.rows == 200


def test_dequantize_arguments():
    def call(q=mx(), out=B, dtype=BF16):
        return gns.lib().gns_mxfp4_dequantize(ref(q), out, dtype, None)

    assert call(q=None) == E["NULL"] and call(out=None) == E["NULL"] and call(q=mx(codes=None)) == E["NULL"]
    assert call(dtype=BF16X3) == E["DTYPE"] and call(q=mx(rows=-1)) == E["SHAPE"]
    assert call(out=B + 1) == E["PARAM"] and call(q=mx(codes=A + 1)) == E["PARAM"]
    assert call(out=A) == E["ALIAS"] and call(out=A + (1 << 36) + 100) == E["ALIAS"]
    assert call(q=mx(rows=0), out=None) == E["OK"]


def product(a=mx(), b=mx(B, B + (1 << 36), rows=70), out=C, dtype=BF16, pitch=70, stride=2800, accumulate=0, ws=W,
            ws_bytes=1 << 40):
    return gns.lib().gns_mxfp4_matmul(ref(a), ref(b), out, dtype, pitch, stride, accumulate, ws, ws_bytes, None)


def linear(x=A, xt=BF16, x_pitch=200, x_stride=8000, m=40, w=mx(B, B + (1 << 36), rows=70), out=C, dtype=BF16, pitch=70,
           stride=2800, accumulate=0, ws=W, ws_bytes=1 << 40):
    return gns.lib().gns_mxfp4_linear(x, xt, x_pitch, x_stride, m, ref(w), out, dtype, pitch, stride, accumulate, ws,
                                      ws_bytes, None)


@pytest.mark.parametrize("call", [product, linear])
def test_product_arguments(call):
    other = "b" if call is product else "w"
    for kw in (dict(pitch=69), dict(pitch=-1), dict(stride=2799), dict(stride=-1), dict(pitch=1 << 60),
               {other: mx(B, D, rows=-1)}, {other: mx(B, D, cols=1 << 24)}):
        assert call(**kw) == E["SHAPE"], kw
    for dtype in (BF16X3, -1, 4):
        assert call(dtype=dtype) == E["DTYPE"]
    for kw in (dict(accumulate=2), dict(accumulate=-1), dict(out=C + 1), dict(dtype=F32, out=C + 2, pitch=70),
               {other: mx(B + 4, D)}):
        assert call(**kw) == E["PARAM"], kw
    assert call(out=None) == E["NULL"] and call(**{other: None}) == E["NULL"]
    assert call(**{other: mx(None, D)}) == E["NULL"]
    for kw in (dict(out=B), dict(out=B + (1 << 36)), dict(out=A)):
        assert call(**kw) == E["ALIAS"], kw
    if call is linear:
        assert linear(xt=BF16X3) == E["DTYPE"] and linear(x=None) == E["NULL"] and linear(x=A + 1) == E["PARAM"]
        for kw in (dict(m=-1), dict(m=1 << 24), dict(x_pitch=-1), dict(x_stride=-1)):
            assert linear(**kw) == E["SHAPE"], kw
        need = gns.mxfp4_matmul_workspace_bytes(2, 40, 70, 200, quantized=False)
        assert need > 0
        for kw in (dict(ws=None), dict(ws=W + 16), dict(ws_bytes=need - 1)):
            assert linear(**kw) == E["WORKSPACE"], kw
        for at in (A, B, C):
            assert linear(ws=at) == E["ALIAS"]
    else:
        assert product(a=None) == E["NULL"] and product(a=mx(scales=None)) == E["NULL"]
        assert product(a=mx(cols=199)) == E["SHAPE"] and product(a=mx(batch=3)) == E["SHAPE"]


def test_product_in_parts_needs_its_workspace():
    a, b = mx(batch=1, rows=64, cols=1 << 16), mx(B, B + (1 << 36), batch=1, rows=64, cols=1 << 16)
    need = gns.mxfp4_matmul_workspace_bytes(1, 64, 64, 1 << 16)
    assert need > 0
    for kw in (dict(ws=None), dict(ws=W + 16), dict(ws_bytes=need - 1)):
        assert product(a=a, b=b, pitch=64, stride=0, **kw) == E["WORKSPACE"], kw
    for at in (A, B, C):
        assert product(a=a, b=b, pitch=64, stride=0, ws=at) == E["ALIAS"]


def test_products_of_nothing():
    assert product(a=mx(rows=0)) == E["OK"] and product(b=mx(B, D, rows=0)) == E["OK"]
    assert product(a=mx(cols=0), b=mx(B, D, cols=0, rows=70), accumulate=1) == E["OK"]
    assert linear(m=0, out=None, ws=None) == E["OK"] and linear(w=mx(batch=0), out=None, ws=None) == E["OK"]


def test_tensors_that_are_not_on_the_gpu():
    t, f = torch.zeros(3, dtype=torch.int64), torch.zeros(3, 4)
    for call in (lambda: gns.embedding(t, f), lambda: gns.embedding([1, 2], f), lambda: gns.embedding_grad(t, f, f),
                 lambda: gns.mxfp4_quantize(f), lambda: gns.mxfp4_quantize(f.numpy()), lambda: gns.mxfp4_quantize_both(f),
                 lambda: gns.mxfp4_quantize(f.to_sparse()), lambda: gns.mxfp4_dequantize(f), lambda: gns.mxfp4_matmul(f, f),
                 lambda: gns.MXFP4(f, f, (3, 4)), lambda: gns.mxfp4_empty((3, 4), "cpu"),
                 lambda: gns.mxfp4_quantize(f, stream=0), lambda: gns.embedding(tokens=t, weight=f, stream=0)):
        with pytest.raises(gns.GnsError) as e:
            call()
        assert e.value.name == "GNS_E_NULL"
