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

import ctypes
import functools
from typing import Optional, Sequence, Tuple, Union

import torch

from .binding import GnsError, _DT, _check, _device_tensor, _dtype_code, _ptr, _workspace, lib
from .tensors import _current_device, _current_raw_stream

_TOKEN_BITS = {torch.int32: 32, torch.int64: 64}


class Matrix(ctypes.Structure):
    """gns_mxfp4."""
    _fields_ = [("codes", ctypes.c_void_p), ("scales", ctypes.c_void_p), ("batch", ctypes.c_int64),
                ("rows", ctypes.c_int64), ("cols", ctypes.c_int64)]


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


def _placed(position: int, name: str):
    """Runs a call on the device of the named argument and on ``stream``, with
    both current: what it allocates belongs to that stream."""
    def wrap(fn):
        @functools.wraps(fn)
        def call(*args, stream=None, **kwargs):
            device = getattr(args[position] if len(args) > position else kwargs.get(name), "device", None)
            if device is None or device.type != "cuda":
                return fn(*args, **kwargs)                       # (which raises)
            if stream is None and device.index == _current_device():
                return fn(*args, **kwargs)
            with torch.cuda.device(device), torch.cuda.stream(_stream_on(device, stream)):
                return fn(*args, **kwargs)
        return call
    return wrap


def _need(name: str, t, device=None) -> None:
    if not isinstance(t, torch.Tensor) or t.layout is not torch.strided:
        raise GnsError(1, f"{name} is not a dense tensor: {type(t).__name__}")
    _device_tensor(name, t, device)


def _type(name: str, t: torch.Tensor) -> int:
    code = _DT.get(t.dtype)
    if code is None:
        raise GnsError(3, f"{name} has dtype {t.dtype}")
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
    _need("tokens", tokens)
    if tokens.dtype not in _TOKEN_BITS:
        raise GnsError(3, f"tokens have dtype {tokens.dtype}: int32 or int64 is needed")
    if not tokens.is_contiguous():
        raise GnsError(2, "tokens must be contiguous")
    return _TOKEN_BITS[tokens.dtype]


@_placed(0, "tokens")
def embedding(tokens: torch.Tensor, weight: torch.Tensor, *, scale: float = 1.0, dtype: Optional[torch.dtype] = None,
              out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``scale * weight[tokens]`` in one pass (gns_embedding): tokens (int32 or
    int64, any shape) into rows of weight ([vocab, width]), in ``dtype``
    (weight's by default) or into ``out`` ([*tokens.shape, width]).  A token
    outside the vocabulary is padding and gives a row of zeros."""
    bits = _tokens(tokens)
    device = tokens.device
    _need("weight", weight, device)
    if weight.dim() != 2:
        raise GnsError(2, f"weight must be [vocab, width], got {tuple(weight.shape)}")
    vocab, width = weight.shape
    if out is None:
        out = torch.empty(*tokens.shape, width, dtype=dtype or weight.dtype, device=device)
    else:
        _need("out", out, device)
        if out.dim() == 0 or out.shape[-1] != width:
            raise GnsError(2, f"out has shape {tuple(out.shape)}, rows of weight have {width}")
        if dtype is not None and out.dtype != dtype:
            raise GnsError(3, f"out has dtype {out.dtype}, dtype is {dtype}")
    _check(lib().gns_embedding(tokens.data_ptr(), bits, tokens.numel(), weight.data_ptr(), _type("weight", weight),
                               vocab, width, _rows_of("weight", weight, (vocab,)), float(scale), out.data_ptr(),
                               _type("out", out), _rows_of("out", out, tokens.shape),
                               _current_raw_stream(device.index)))
    return out


def embedding_grad_workspace_bytes(count: int, vocab: int, width: int) -> int:
    return int(lib().gns_embedding_grad_workspace_bytes(count, vocab, width))


@_placed(0, "tokens")
def embedding_grad(tokens: torch.Tensor, grad: torch.Tensor, grad_weight: torch.Tensor, *, scale: float = 1.0,
                   accumulate: bool = False, workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The gradient of :func:`embedding` with respect to its weight
    (gns_embedding_grad): row v of grad_weight ([vocab, width], written in
    place) becomes ``scale`` times the sum of the rows of grad
    ([*tokens.shape, width]) whose token is v, or with ``accumulate`` grows by
    it.  The sums are fp32 in an order that the tokens alone decide, rounded
    once; the three may have different types.  Padding tokens are left out.
    grad_weight may be a slice of a gradient bucket, ready for grad_norm and
    adamw_step.  Returns grad_weight."""
    bits = _tokens(tokens)
    device = tokens.device
    _need("grad", grad, device)
    _need("grad_weight", grad_weight, device)
    if grad_weight.dim() != 2:
        raise GnsError(2, f"grad_weight must be [vocab, width], got {tuple(grad_weight.shape)}")
    vocab, width = grad_weight.shape
    if grad.dim() == 0 or grad.shape[-1] != width:
        raise GnsError(2, f"grad has shape {tuple(grad.shape)}, rows of grad_weight have {width}")
    L, count = lib(), tokens.numel()
    ws = _workspace(0 if workspace is not None else L.gns_embedding_grad_workspace_bytes(count, vocab, width), device,
                    workspace)
    _check(L.gns_embedding_grad(tokens.data_ptr(), bits, count, grad.data_ptr(), _type("grad", grad),
                                _rows_of("grad", grad, tokens.shape), vocab, width, float(scale),
                                grad_weight.data_ptr(), _type("grad_weight", grad_weight),
                                _rows_of("grad_weight", grad_weight, (vocab,)), 1 if accumulate else 0, ws.data_ptr(),
                                ws.numel() * ws.element_size(), _current_raw_stream(device.index)))
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
    __slots__ = ("codes", "scales", "shape", "_c", "_ref")

    def __init__(self, codes: torch.Tensor, scales: torch.Tensor, shape: Sequence[int]):
        shape = torch.Size(shape)
        if len(shape) not in (2, 3):
            raise GnsError(2, f"shape must be [rows, cols] or [batch, rows, cols], got {tuple(shape)}")
        lead, (rows, cols) = shape[:-2], shape[-2:]
        groups = -(-cols // 128)
        wanted = {"codes": (*lead, rows, groups * 64), "scales": (*lead, -(-rows // 32), groups, 32, 4)}
        for name, t in (("codes", codes), ("scales", scales)):
            _need(name, t, codes.device)
            if t.dtype != torch.uint8 or tuple(t.shape) != wanted[name] or not t.is_contiguous():
                raise GnsError(2, f"{name} must be contiguous uint8 {wanted[name]}, got {t.dtype} {tuple(t.shape)}")
        self.codes, self.scales, self.shape = codes, scales, shape
        self._c = Matrix(codes.data_ptr(), scales.data_ptr(), lead[0] if lead else 1, rows, cols)
        self._ref = ctypes.byref(self._c)

    @property
    def device(self) -> torch.device:
        return self.codes.device

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


def mxfp4_empty(shape: Sequence[int], device=None) -> MXFP4:
    """Room for a matrix or a batch of matrices (the ``out`` of
    :func:`mxfp4_quantize`)."""
    shape = torch.Size(shape)
    if len(shape) not in (2, 3):
        raise GnsError(2, f"shape must be [rows, cols] or [batch, rows, cols], got {tuple(shape)}")
    lead, (rows, cols) = shape[:-2], shape[-2:]
    groups = -(-cols // 128)
    device = torch.device("cuda") if device is None else device
    return MXFP4(torch.empty(*lead, rows, groups * 64, dtype=torch.uint8, device=device),
                 torch.empty(*lead, -(-rows // 32), groups, 32, 4, dtype=torch.uint8, device=device), shape)


def _matrix(name: str, x: torch.Tensor):
    """(batch, rows, cols, pitch, batch stride) of a [rows, cols] or
    [batch, rows, cols] tensor whose rows' elements are consecutive, or None."""
    shape, st = x.shape, x.stride()
    rows, cols = shape[-2:]
    if cols > 1 and st[-1] != 1 and x.numel():
        return None
    pitch = st[-2] if rows > 1 and cols else cols
    if len(shape) == 2:
        return 1, rows, cols, pitch, 0
    return shape[0], rows, cols, pitch, st[0] if shape[0] > 1 else 0


def _quantize(x, noise, straight, turned):
    """Q(x) into ``straight`` and Q(x^T) into ``turned`` (either may be None:
    not wanted)."""
    device = x.device
    code = _type("x", x)
    form = _matrix("x", x)
    if form is None:
        form = _matrix("x", x.mT)
        if form is None:
            raise GnsError(2, f"x: elements of a row or of a column must be consecutive (strides {x.stride()})")
        straight, turned = turned, straight
        noise = None if noise is None else noise.mT
    if noise is not None:
        _need("noise", noise, device)
        if noise.dtype != torch.uint8 or not noise.is_contiguous():
            raise GnsError(2, "noise must be uint8, contiguous in x's order")
    batch, rows, cols, pitch, batch_stride = form
    _check(lib().gns_mxfp4_quantize(x.data_ptr(), code, pitch, batch_stride, _ptr(noise),
                                    None if straight is None else straight._ref,
                                    None if turned is None else turned._ref, _current_raw_stream(device.index)))


def _quantize_args(x, noise):
    _need("x", x)
    if x.dim() not in (2, 3):
        raise GnsError(2, f"x must be [rows, cols] or [batch, rows, cols], got {tuple(x.shape)}")
    if noise is not None and (not isinstance(noise, torch.Tensor) or noise.shape != x.shape):
        raise GnsError(2, "noise must have x's shape")


def _quantized_out(out, shape, device) -> MXFP4:
    if out is None:
        return mxfp4_empty(shape, device)
    if not isinstance(out, MXFP4) or out.shape != shape:
        raise GnsError(2, f"out must be an MXFP4 of shape {tuple(shape)}, got {out!r}")
    _device_tensor("out", out.codes, device)
    return out


@_placed(0, "x")
def mxfp4_quantize(x: torch.Tensor, *, transposed: bool = False, noise: Optional[torch.Tensor] = None,
                   out: Optional[MXFP4] = None) -> MXFP4:
    """x ([rows, cols] or [batch, rows, cols]; fp32, bf16 or fp16; rows or
    columns of consecutive elements) in MXFP4 with blocks along its rows, or
    with ``transposed`` its transpose, with blocks along its columns
    (gns_mxfp4_quantize).  Values are rounded to nearest, or with ``noise``
    (random bytes of x's shape) up or down with their probability and nothing
    cut off."""
    _quantize_args(x, noise)
    shape = x.mT.shape if transposed else x.shape
    out = _quantized_out(out, shape, x.device)
    _quantize(x, noise, None if transposed else out, out if transposed else None)
    return out


@_placed(0, "x")
def mxfp4_quantize_both(x: torch.Tensor, *, noise: Optional[torch.Tensor] = None,
                        out: Optional[Tuple[MXFP4, MXFP4]] = None) -> Tuple[MXFP4, MXFP4]:
    """:func:`mxfp4_quantize` of x and of its transpose in one pass over x: what
    the products of the forward and the backward pass take."""
    _quantize_args(x, noise)
    a, b = (None, None) if out is None else out
    a, b = _quantized_out(a, x.shape, x.device), _quantized_out(b, x.mT.shape, x.device)
    _quantize(x, noise, a, b)
    return a, b


@_placed(0, "q")
def mxfp4_dequantize(q: MXFP4, *, dtype: torch.dtype = torch.bfloat16,
                     out: Optional[torch.Tensor] = None) -> torch.Tensor:
    """The values that q stands for (gns_mxfp4_dequantize): exact in fp32 and
    bf16."""
    if not isinstance(q, MXFP4):
        raise GnsError(1, f"q is not an MXFP4: {type(q).__name__}")
    if out is None:
        out = torch.empty(q.shape, dtype=dtype, device=q.device)
    else:
        _need("out", out, q.device)
        if out.shape != q.shape or not out.is_contiguous():
            raise GnsError(2, f"out must be contiguous {tuple(q.shape)}")
    _check(lib().gns_mxfp4_dequantize(q._ref, out.data_ptr(), _type("out", out), _current_raw_stream(q.device.index)))
    return out


def mxfp4_matmul_workspace_bytes(batch: int, m: int, n: int, k: int, quantized: bool = True) -> int:
    """Bytes that :func:`mxfp4_matmul` needs for [batch, m, k] by [batch, n, k]
    (``quantized``: whether its first factor is)."""
    L = lib()
    return int((L.gns_mxfp4_matmul_workspace_bytes if quantized else L.gns_mxfp4_linear_workspace_bytes)(batch, m, n, k))


@_placed(1, "b")
def mxfp4_matmul(a: Union[MXFP4, torch.Tensor], b: MXFP4, *, out: Optional[torch.Tensor] = None,
                 dtype: Optional[torch.dtype] = None, accumulate: bool = False,
                 workspace: Optional[torch.Tensor] = None) -> torch.Tensor:
    """``a @ b^T`` ([m, k] by [n, k], or batches of them), with sums in fp32
    (gns_mxfp4_matmul), in ``dtype`` (a's, or bf16) or into ``out``;
    ``accumulate`` adds to ``out``.  A plain tensor ``a`` is quantised on the
    way (gns_mxfp4_linear); with one matrix b it may have any leading axes."""
    if not isinstance(b, MXFP4):
        raise GnsError(1, f"b is not an MXFP4: {type(b).__name__}")
    device = b.device
    n, k = b.shape[-2:]
    quantized = isinstance(a, MXFP4)
    if quantized:
        _device_tensor("a", a.codes, device)
        m = a.shape[-2]
        if a.shape[-1] != k or a.shape[:-2] != b.shape[:-2]:
            raise GnsError(2, f"a is {tuple(a.shape)}, b {tuple(b.shape)}")
        shape = (*a.shape[:-1], n)
    else:
        _need("a", a, device)
        if a.dim() == 0 or a.shape[-1] != k or (len(b.shape) == 3 and (a.dim() != 3 or a.shape[0] != b.shape[0])):
            raise GnsError(2, f"a is {tuple(a.shape)}, b {tuple(b.shape)}")
        shape = (*a.shape[:-1], n)
        code = _type("a", a)
        if len(b.shape) == 3:
            form = _matrix("a", a)
            if form is None:
                raise GnsError(2, f"a: elements of a row must be consecutive (strides {a.stride()})")
            _, m, _, pitch, batch_stride = form
        else:
            m = 1
            for s in a.shape[:-1]:
                m *= s
            pitch, batch_stride = _rows_of("a", a, a.shape[:-1]), 0
    batch = b._c.batch
    if out is None:
        if accumulate:
            raise GnsError(1, "accumulate needs out")
        out = torch.empty(shape, dtype=dtype or (torch.bfloat16 if quantized else a.dtype), device=device)
    else:
        _need("out", out, device)
        if tuple(out.shape) != tuple(shape):
            raise GnsError(2, f"out has shape {tuple(out.shape)}, the product {tuple(shape)}")
        if dtype is not None and out.dtype != dtype:
            raise GnsError(3, f"out has dtype {out.dtype}, dtype is {dtype}")
    if len(b.shape) == 3:
        form = _matrix("out", out)
        if form is None:
            raise GnsError(2, f"out: elements of a row must be consecutive (strides {out.stride()})")
        out_pitch, out_stride = form[3:]
    else:
        out_pitch, out_stride = _rows_of("out", out, shape[:-1]), 0
    L = lib()
    if workspace is None:
        need = (L.gns_mxfp4_matmul_workspace_bytes if quantized else L.gns_mxfp4_linear_workspace_bytes)(batch, m, n, k)
        ws = torch.empty(need, dtype=torch.uint8, device=device) if need else None
    else:
        ws = _workspace(0, device, workspace)
    at, room = (None, 0) if ws is None else (ws.data_ptr(), ws.numel() * ws.element_size())
    tail = (out.data_ptr(), _type("out", out), out_pitch, out_stride, 1 if accumulate else 0, at, room,
            _current_raw_stream(device.index))
    if quantized:
        _check(L.gns_mxfp4_matmul(a._ref, b._ref, *tail))
    else:
        _check(L.gns_mxfp4_linear(a.data_ptr(), code, pitch, batch_stride, m, b._ref, *tail))
    return out
