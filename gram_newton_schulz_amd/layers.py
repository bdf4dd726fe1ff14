"""Layers of the model whose parameters the library updates: the token
embedding with its gradient (gns_embedding, gns_embedding_grad) and products in
microscaled 4-bit floating point (gns_mxfp4_quantize, gns_mxfp4_dequantize,
gns_mxfp4_matmul, gns_mxfp4_linear).

The calls run on their tensors' device, whichever is current, on that device's
current stream or on ``stream``.  Like the other calls of this package they are
no autograd functions, and writing in place does not raise a tensor's version
counter.
"""
from __future__ import annotations

import contextlib
import ctypes
import functools
import math
from typing import Optional, Sequence, Tuple, Union

import torch

from .binding import GnsError, _DT, _check, _device_tensor, _workspace, lib
from .tensors import _current_device, _current_raw_stream

_TOKEN_BITS = {torch.int32: 32, torch.int64: 64}
_STRIDED = torch.strided


class Matrix(ctypes.Structure):
    """gns_mxfp4."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


# The calls of small problems take about as long as Python does around them (a
# launch is 3.3 us), so the checks below ask each question once, and in the
# form that costs least.

@contextlib.contextmanager
def _elsewhere(index: int, stream):
    """Makes the device, and the stream that a caller passed, current: what a
    call allocates then belongs to that stream."""
    device = torch.device("cuda", index)
    with torch.cuda.device(device), torch.cuda.stream(_stream_on(device, stream)):
        yield


def _stream_on(device: torch.device, stream) -> "torch.cuda.Stream":
    """A stream object of the device for what a caller may pass as ``stream``."""
    if stream is None:
        return torch.cuda.current_stream(device)
    if not isinstance(stream, int):
        on = getattr(stream, "device", device)      # (anything with a handle is taken)
        if on.index != device.index:
            raise GnsError(11, f"stream is on {on}, the tensors on {device}")
        if isinstance(stream, torch.cuda.Stream):
            return stream
        stream = stream.cuda_stream
    if stream == 0:
        return torch.cuda.default_stream(device)
    return torch.cuda.ExternalStream(stream, device=device)


def _index_of(name: str, t) -> int:
    """Device index of a dense tensor on a GPU."""
    if not isinstance(t, torch.Tensor) or t.layout is not _STRIDED:
        raise GnsError(1, f"{name} is not a dense tensor: {type(t).__name__}")
    if not t.is_cuda:
        _device_tensor(name, t, None)
    return t.get_device()


def _need(name: str, t, index: int) -> None:
    """Raise unless t is a dense tensor on that GPU."""
    if _index_of(name, t) != index:
        _device_tensor(name, t, torch.device("cuda", index))


def _type(name: str, t: torch.Tensor) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise GnsError(3, f"{name} has dtype {t.dtype}")
    return code


def _type_of(dtype) -> int:
    code = _DT.get(dtype)
    if code is None:
        raise GnsError(3, f"unsupported dtype {dtype}")
    return code


# ---------------------------------------------------------------------------
# token embedding
# ---------------------------------------------------------------------------
def _rows_of(name: str, t: torch.Tensor, lead: Sequence[int]) -> int:
    """Row pitch of a [*lead, width] tensor as one array of rows."""
    if tuple(t.shape[:-1]) != tuple(lead) or t.dim() != len(lead) + 1:
        raise GnsError(2, f"{name} has shape {tuple(t.shape)}, expected {tuple(lead)} rows")
    width = t.shape[-1]
    if t.numel() == 0 or t.is_contiguous():
        return width
    if width > 1 and t.stride(-1) != 1:
        raise GnsError(2, f"{name}: elements of a row must be consecutive (strides {t.stride()})")
    pitch = size = None
    for n, st in zip(reversed(t.shape[:-1]), reversed(t.stride()[:-1])):
        if n == 1:
            continue
        if pitch is None:
            pitch, size = st, n
        elif st == pitch * size:
            size *= n
        else:
            raise GnsError(2, f"{name}: strides {t.stride()} are not rows at equal distances")
    return width if pitch is None else pitch


def _tokens(tokens) -> int:
    bits = _TOKEN_BITS.get(tokens.dtype)
    if bits is None:
        raise GnsError(3, f"tokens have dtype {tokens.dtype}: int32 or int64 is needed")
    if not tokens.is_contiguous():
        raise GnsError(2, "tokens must be contiguous")
    return bits


def _table(name: str, t: torch.Tensor, index: int):
    """(vocab, width, pitch, type) of a table."""
    _need(name, t, index)
    shape = t.shape
    if len(shape) != 2:
        raise GnsError(2, f"{name} must be [vocab, width], got {tuple(shape)}")
    vocab, width = shape
    return vocab, width, width if t.is_contiguous() else _rows_of(name, t, (vocab,)), _type(name, t)


def embedding(tokens: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``scale * weight[tokens]`` in one pass (gns_embedding): tokens (int32 or
    int64, any shape) into rows of weight ([vocab, width]), in ``dtype``
    (weight's by default) or into ``out`` ([*tokens.shape, width]).  A token
    outside the vocabulary is padding and gives a row of zeros.  No graph is
    recorded: the gradient is :func:`embedding_grad`."""
    index = _index_of("tokens", tokens)
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return embedding(tokens, weight, scale=scale, dtype=dtype, out=out)
    bits = _tokens(tokens)
    vocab, width, pitch, code = _table("weight", weight, index)
    if out is None:
        dtype = dtype or weight.dtype
        out_code, out_pitch = _type_of(dtype), width
        out = torch.empty((*tokens.shape, width), dtype=dtype, device=tokens.device)
    else:
        _need("out", out, index)
        if out.dim() == 0 or out.shape[-1] != width:
            raise GnsError(2, f"out has shape {tuple(out.shape)}, rows of weight have {width}")
        if dtype is not None and out.dtype != dtype:
            raise GnsError(3, f"out has dtype {out.dtype}, dtype is {dtype}")
        out_code, out_pitch = _type("out", out), _rows_of("out", out, tokens.shape)
    _check(lib().gns_embedding(tokens.data_ptr(), bits, tokens.numel(), weight.data_ptr(), code, vocab, width, pitch,
                               float(scale), out.data_ptr(), out_code, out_pitch, _current_raw_stream(index)))
    return out


@functools.lru_cache(maxsize=1024)
def embedding_grad_workspace_bytes(count: int, vocab: int, width: int) -> int:
    return int(lib().gns_embedding_grad_workspace_bytes(count, vocab, width))


def embedding_grad(tokens: torch.Tensor, grad: torch.Tensor, grad_weight: torch.Tensor, *, scale: float = 1.0,
                   accumulate: bool = False, workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """The gradient of :func:`embedding` with respect to its weight
    (gns_embedding_grad): row v of grad_weight ([vocab, width], written in
    place) becomes ``scale`` times the sum of the rows of grad
    ([*tokens.shape, width]) whose token is v, or with ``accumulate`` grows by
    it.  The sums are fp32 in an order that the tokens alone decide, rounded
    once; the three may have different types.  Padding tokens are left out.
    grad_weight may be a slice of a gradient bucket, ready for grad_norm and
    adamw_step.  Returns grad_weight."""
    index = _index_of("tokens", tokens)
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return embedding_grad(tokens, grad, grad_weight, scale=scale, accumulate=accumulate, workspace=workspace)
    bits = _tokens(tokens)
    _need("grad", grad, index)
    vocab, width, pitch, code = _table("grad_weight", grad_weight, index)
    if grad.dim() == 0 or grad.shape[-1] != width:
        raise GnsError(2, f"grad has shape {tuple(grad.shape)}, rows of grad_weight have {width}")
    grad_pitch, count = _rows_of("grad", grad, tokens.shape), tokens.numel()
    if workspace is None:
        room = embedding_grad_workspace_bytes(count, vocab, width)
        ws = torch.empty(room, dtype=torch.uint8, device=tokens.device) if room else None
    else:
        ws = _workspace(0, tokens.device, workspace)
        room = ws.numel() * ws.element_size()
    _check(lib().gns_embedding_grad(tokens.data_ptr(), bits, count, grad.data_ptr(), _type("grad", grad), grad_pitch,
                                    vocab, width, float(scale), grad_weight.data_ptr(), code, pitch, 1 if accumulate else 0,
                                    None if ws is None else ws.data_ptr(), room, _current_raw_stream(index)))
    return grad_weight


# ---------------------------------------------------------------------------
# MXFP4
# ---------------------------------------------------------------------------
class MXFP4:
    """A matrix, or a batch of matrices, in blocks of 32 4-bit floats along the
    rows with a power of two each (gns_mxfp4).  ``shape`` is that of the values,
    ``codes`` ([..., rows, K / 2], K the columns rounded up to 128) and
    ``scales`` ([..., row blocks, K / 128, 32, 4]) are uint8.  Index a batch for
    one of its matrices."""
    __slots__ = ("shape", "_codes", "_scales", "_room", "_index", "_c", "_ref", "_dims")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape: Sequence[int]):
        shape = torch.Size(shape)
        lead, rows, cols = _sizes(shape)
        groups = -(-cols // 128)
        wanted = {"codes": (*lead, rows, groups * 64), "scales": (*lead, -(-rows // 32), groups, 32, 4)}
        index = _index_of("codes", codes)
        _need("scales", scales, index)
        for name, t in (("codes", codes), ("scales", scales)):
            if t.dtype != torch.uint8 or tuple(t.shape) != wanted[name] or not t.is_contiguous():
                raise GnsError(2, f"{name} must be contiguous uint8 {wanted[name]}, got {t.dtype} {tuple(t.shape)}")
        self._set(shape, codes.data_ptr(), scales.data_ptr(), index)
        self._codes, self._scales = codes, scales

    def _set(self, shape, codes: int, scales: int, index: int) -> None:
        self.shape, self._index = shape, index
        self._dims = batch, rows, cols = (1, *shape) if len(shape) == 2 else tuple(shape)
        self._codes = self._scales = self._room = None
        self._c = Matrix(codes, scales, batch, rows, cols)
        self._ref = ctypes.byref(self._c)

    def _view(self, offset: int, shape) -> torch.Tensor:
        n = math.prod(shape)
        return self._room[offset:offset + n].view(shape)

    @property
    def codes(self) -> torch.Tensor:
        if self._codes is None:
            lead, rows, cols = _sizes(self.shape)
            self._codes = self._view(self._c.codes - self._room.data_ptr() if self._c.codes else 0,
                                     (*lead, rows, -(-cols // 128) * 64))
        return self._codes

    @property
    def scales(self) -> torch.Tensor:
        if self._scales is None:
            lead, rows, cols = _sizes(self.shape)
            self._scales = self._view(self._c.scales - self._room.data_ptr() if self._c.scales else 0,
                                      (*lead, -(-rows // 32), -(-cols // 128), 32, 4))
        return self._scales

    @property
    def device(self) -> torch.device:
        return torch.device("cuda", self._index)

    @property
    def nbytes(self) -> int:
        return self.codes.numel() + self.scales.numel()

    def __getitem__(self, i: int) -> "MXFP4":
        if len(self.shape) != 3:
            raise GnsError(2, "only a batch of matrices is indexed")
        return MXFP4(self.codes[i], self.scales[i], self.shape[1:])

    def __len__(self) -> int:
        return self.shape[0]

    def __repr__(self) -> str:
        return f"MXFP4({tuple(self.shape)}, device={str(self.device)!r})"


def _sizes(shape):
    if len(shape) == 2:
        return (), *shape
    if len(shape) == 3:
        return shape[:1], *shape[1:]
    raise GnsError(2, f"shape must be [rows, cols] or [batch, rows, cols], got {tuple(shape)}")


def _rooms(shapes, index: int):
    """MXFP4 objects of the shapes in one allocation, each array on 256 bytes."""
    at, places = 0, []
    for shape in shapes:
        lead, rows, cols = _sizes(shape)
        batch, groups = lead[0] if lead else 1, -(-cols // 128)
        scales = at + (batch * rows * groups * 64 + 255) // 256 * 256
        places.append((shape, at, scales))
        at = scales + (batch * -(-rows // 32) * groups * 128 + 255) // 256 * 256
    room = torch.empty(at, dtype=torch.uint8, device=torch.device("cuda", index))
    base, made = room.data_ptr(), []
    for shape, codes, scales in places:
        q = object.__new__(MXFP4)
        q._set(shape, base + codes, base + scales, index)
        q._room = room
        made.append(q)
    return made


def mxfp4_empty(shape: Sequence[int], device=None) -> MXFP4:
    """Room for a matrix or a batch of matrices (the ``out`` of
    :func:`mxfp4_quantize`)."""
    device = torch.device("cuda" if device is None else device)
    if device.type != "cuda":
        raise GnsError(1, f"device must be a GPU, got {device}")
    return _rooms([torch.Size(shape)], torch.cuda.current_device() if device.index is None else device.index)[0]


def _matrix(x: torch.Tensor):
    """(batch, rows, cols, pitch, batch stride) of a [rows, cols] or
    [batch, rows, cols] tensor whose rows' elements are consecutive, or None."""
    shape = x.shape
    if len(shape) == 2:
        batch, (rows, cols) = 1, shape
    else:
        batch, rows, cols = shape
    if x.is_contiguous():
        return batch, rows, cols, cols, rows * cols
    st = x.stride()
    if cols > 1 and st[-1] != 1 and x.numel():
        return None
    return batch, rows, cols, st[-2] if rows > 1 and cols else cols, st[0] if batch > 1 and len(shape) == 3 else 0


def _quantize(x, noise, straight, turned, index: int) -> None:
    """Q(x) into ``straight`` and Q(x^T) into ``turned`` (either may be None:
    not wanted)."""
    code = _type("x", x)
    form = _matrix(x)
    if form is None:
        form = _matrix(x.mT)
        if form is None:
            raise GnsError(2, f"x: elements of a row or of a column must be consecutive (strides {x.stride()})")
        straight, turned = turned, straight
        noise = None if noise is None else noise.mT
    if noise is not None:
        _need("noise", noise, index)
        if noise.dtype != torch.uint8 or not noise.is_contiguous():
            raise GnsError(2, "noise must be uint8, contiguous in x's order")
    _check(lib().gns_mxfp4_quantize(x.data_ptr(), code, form[3], form[4], None if noise is None else noise.data_ptr(),
                                    None if straight is None else straight._ref,
                                    None if turned is None else turned._ref, _current_raw_stream(index)))


def _quantize_shape(x, noise):
    shape = x.shape
    if len(shape) not in (2, 3):
        raise GnsError(2, f"x must be [rows, cols] or [batch, rows, cols], got {tuple(shape)}")
    if noise is not None and (not isinstance(noise, torch.Tensor) or noise.shape != shape):
        raise GnsError(2, "noise must have x's shape")
    return shape, torch.Size((*shape[:-2], shape[-1], shape[-2]))


def _check_room(q, shape, index: int) -> None:
    if not isinstance(q, MXFP4) or q.shape != shape:
        raise GnsError(2, f"out must be an MXFP4 of shape {tuple(shape)}, got {q!r}")
    if q._index != index:
        raise GnsError(1, f"out is on {q.device}, x on cuda:{index}")


def mxfp4_quantize(x: torch.Tensor, *, transposed: bool = False, noise: Optional[torch.Tensor] = None,
                   out: Optional[MXFP4] = None, stream=None) -> MXFP4:
    """x ([rows, cols] or [batch, rows, cols]; fp32, bf16 or fp16; rows or
    columns of consecutive elements) in MXFP4 with blocks along its rows, or
    with ``transposed`` its transpose, with blocks along its columns
    (gns_mxfp4_quantize).  Values are rounded to nearest, or with ``noise``
    (random bytes of x's shape) up or down with their probability and nothing
    cut off."""
    index = _index_of("x", x)
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return mxfp4_quantize(x, transposed=transposed, noise=noise, out=out)
    shape = _quantize_shape(x, noise)[1 if transposed else 0]
    if out is None:
        out, = _rooms((shape,), index)
    else:
        _check_room(out, shape, index)
    _quantize(x, noise, None if transposed else out, out if transposed else None, index)
    return out


def mxfp4_quantize_both(x: torch.Tensor, *, noise: Optional[torch.Tensor] = None,
                        out: Optional[Tuple[MXFP4, MXFP4]] = None, stream=None) -> Tuple[MXFP4, MXFP4]:
    """:func:`mxfp4_quantize` of x and of its transpose in one pass over x: what
    the products of the forward and the backward pass take."""
    index = _index_of("x", x)
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return mxfp4_quantize_both(x, noise=noise, out=out)
    shapes = _quantize_shape(x, noise)
    if out is None:
        a, b = _rooms(shapes, index)
    else:
        a, b = out
        _check_room(a, shapes[0], index)
        _check_room(b, shapes[1], index)
    _quantize(x, noise, a, b, index)
    return a, b


def mxfp4_dequantize(q: MXFP4, *, dtype: Optional[torch.dtype] = None, out: Optional[torch.Tensor] = None,
                     stream=None) -> torch.Tensor:
    """The values that q stands for, in ``dtype`` (bf16 by default) or into
    ``out`` (gns_mxfp4_dequantize): exact in fp32 and bf16."""
    if not isinstance(q, MXFP4):
        raise GnsError(1, f"q is not an MXFP4: {type(q).__name__}")
    index = q._index
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return mxfp4_dequantize(q, dtype=dtype, out=out)
    if out is None:
        dtype = dtype or torch.bfloat16
        code = _type_of(dtype)
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    else:
        _need("out", out, index)
        code = _type("out", out)
        if out.shape != q.shape or not out.is_contiguous():
            raise GnsError(2, f"out must be contiguous {tuple(q.shape)}")
        if dtype is not None and out.dtype != dtype:
            raise GnsError(3, f"out has dtype {out.dtype}, dtype is {dtype}")
    _check(lib().gns_mxfp4_dequantize(q._ref, out.data_ptr(), code, _current_raw_stream(index)))
    return out


@functools.lru_cache(maxsize=1024)
def mxfp4_matmul_workspace_bytes(batch: int, m: int, n: int, k: int, quantized: bool = True) -> int:
    """Bytes that :func:`mxfp4_matmul` needs for [batch, m, k] by [batch, n, k]
    (``quantized``: whether its first factor is)."""
    L = lib()
    return int((L.gns_mxfp4_matmul_workspace_bytes if quantized else L.gns_mxfp4_linear_workspace_bytes)(batch, m, n, k))


def mxfp4_matmul(a: Union[MXFP4, torch.Tensor], b: MXFP4, *, out: Optional[torch.Tensor] = None,
                 dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                 workspace: Optional[torch.Tensor] = None, stream=None) -> torch.Tensor:
    """``a @ b^T`` ([m, k] by [n, k], or batches of them), with sums in fp32
    (gns_mxfp4_matmul), in ``dtype`` (a's, or bf16) or into ``out``;
    ``accumulate`` adds to ``out``.  A plain tensor ``a`` is quantised on the
    way (gns_mxfp4_linear); with one matrix b it may have any leading axes.  No
    graph is recorded: a layer's gradients are two more products, of its
    factors quantised along the other axis."""
    if not isinstance(b, MXFP4):
        raise GnsError(1, f"b is not an MXFP4: {type(b).__name__}")
    index = b._index
    if stream is not None or index != _current_device():
        with _elsewhere(index, stream):
            return mxfp4_matmul(a, b, out=out, dtype=dtype, accumulate=accumulate, workspace=workspace)
    batch, n, k = b._dims
    batched = len(b.shape) == 3
    quantized = isinstance(a, MXFP4)
    shape = a.shape if quantized else None
    if quantized:
        if a._index != index:
            raise GnsError(1, f"a is on {a.device}, b on {b.device}")
        if shape[-1] != k or len(shape) != len(b.shape) or a._dims[0] != batch:
            raise GnsError(2, f"a is {tuple(shape)}, b {tuple(b.shape)}")
        m = a._dims[1]
    else:
        _need("a", a, index)
        shape = a.shape
        if len(shape) == 0 or shape[-1] != k or (batched and (len(shape) != 3 or shape[0] != batch)):
            raise GnsError(2, f"a is {tuple(shape)}, b {tuple(b.shape)}")
        code = _type("a", a)
        if batched:
            form = _matrix(a)
            if form is None:
                raise GnsError(2, f"a: elements of a row must be consecutive (strides {a.stride()})")
            _, m, _, pitch, batch_stride = form
        else:
            m = math.prod(shape[:-1])
            pitch, batch_stride = _rows_of("a", a, shape[:-1]), 0
    made = (*shape[:-1], n)
    if out is None:
        if accumulate:
            raise GnsError(1, "accumulate needs out")
        dtype = dtype or (torch.bfloat16 if quantized else a.dtype)
        out_code, out_pitch, out_stride = _type_of(dtype), n, m * n
        out = torch.empty(made, dtype=dtype, device=b.device)
    else:
        _need("out", out, index)
        out_code = _type("out", out)
        if tuple(out.shape) != made:
            raise GnsError(2, f"out has shape {tuple(out.shape)}, the product {made}")
        if dtype is not None and out.dtype != dtype:
            raise GnsError(3, f"out has dtype {out.dtype}, dtype is {dtype}")
        if batched:
            form = _matrix(out)
            if form is None:
                raise GnsError(2, f"out: elements of a row must be consecutive (strides {out.stride()})")
            out_pitch, out_stride = form[3:]
        else:
            out_pitch, out_stride = _rows_of("out", out, made[:-1]), 0
    if workspace is None:
        room = mxfp4_matmul_workspace_bytes(batch, m, n, k, quantized)
        ws = torch.empty(room, dtype=torch.uint8, device=b.device) if room else None
    else:
        ws = _workspace(0, b.device, workspace)
        room = ws.numel() * ws.element_size()
    tail = (out.data_ptr(), out_code, out_pitch, out_stride, 1 if accumulate else 0,
            None if ws is None else ws.data_ptr(), room, _current_raw_stream(index))
    if quantized:
        _check(lib().gns_mxfp4_matmul(a._ref, b._ref, *tail))
    else:
        _check(lib().gns_mxfp4_linear(a.data_ptr(), code, pitch, batch_stride, m, b._ref, *tail))
    return out
