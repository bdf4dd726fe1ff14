"""Lists of tensors: global gradient norm, clipping and AdamW over every
tensor of a model in a few launches (the C ABI's gns_tensor_list,
gns_grad_norm, gns_grad_clip, gns_adamw_step and gns_adamw_step_counted).

A :class:`TensorList` names its tensors once and is then passed to the calls,
which take no per-tensor arguments and run on the tensors' device, whichever
is current.  It holds their addresses, so it serves while the tensors keep
their memory: build it again after anything that replaces a ``.grad`` or a
parameter.
"""
from __future__ import annotations

import contextlib
import ctypes
import math
import threading
from typing import Optional, Sequence, Union

import numpy as np
import torch

from .binding import GnsError, _DT, _check, _device_tensor, _dtype_code, _ptr, _scalar_ptr, _workspace, lib

NORM_L2, NORM_MAX = 0, 1
_NORMS = {2: NORM_L2, math.inf: NORM_MAX}
ADAMW_WORKSPACE_BYTES = 256

# the current stream's handle without the Stream object around it, which costs
# 1.8 us of a call that takes 6
_current_raw_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (
    lambda index: torch.cuda.current_stream(index).cuda_stream)
_current_device = getattr(torch._C, "_cuda_getDevice", None) or torch.cuda.current_device


class Tensor(ctypes.Structure):
    """gns_tensor."""
    _fields_ = [("data", ctypes.c_void_p), ("rows", ctypes.c_int64), ("cols", ctypes.c_int64),
                ("pitch", ctypes.c_int64), ("dtype", ctypes.c_int)]


# the same, for filling many at once
_ENTRY = np.dtype([("data", np.uint64), ("rows", np.int64), ("cols", np.int64), ("pitch", np.int64),
                   ("dtype", np.int32), ("_pad", np.int32)])
assert _ENTRY.itemsize == ctypes.sizeof(Tensor)


class ListInfo(ctypes.Structure):
    """gns_tensor_list."""
    _fields_ = [("arrays", ctypes.c_int), ("count", ctypes.c_int64), ("elements", ctypes.c_int64),
                ("chunks", ctypes.c_int64), ("chunk_units", ctypes.c_int64), ("keep_from", ctypes.c_int64),
                ("table_bytes", ctypes.c_size_t),
                ("dtypes", ctypes.c_uint * 5), ("bytes", ctypes.c_double * 5), ("overlaps", ctypes.c_uint)]


def _rows(group: Sequence[torch.Tensor]):
    """Common rows x cols form of tensors of one shape: (rows, cols, pitches),
    or None when their strides have none."""
    if all(t.is_contiguous() for t in group):
        n = group[0].numel()
        return 1, n, [n] * len(group)
    strides = [t.stride() for t in group]
    dims = sorted((d for d, size in enumerate(group[0].shape) if size != 1),
                  key=lambda d: [-s[d] if s[d] else -math.inf for s in strides])   # repeated dimensions outermost
    merged = []                       # (size, strides), outermost first
    for d in dims:
        size, st = group[0].shape[d], [s[d] for s in strides]
        if merged and all(a == b * size for a, b in zip(merged[-1][1], st)):
            merged[-1] = (merged[-1][0] * size, st)
        else:
            merged.append((size, st))
    if len(merged) == 1:
        size, st = merged[0]
        return (1, size, [size] * len(group)) if all(s == 1 for s in st) else (size, 1, st)
    if len(merged) == 2 and all(s == 1 for s in merged[1][1]):
        return merged[0][0], merged[1][0], merged[0][1]
    return None


class TensorList:
    """Arrays of tensors of the same shapes, ready for the calls on them (see
    :func:`tensor_list` and :func:`adamw_list`).  Keeps the tensors alive.
    Build it before a graph capture that uses it, and keep it as long as the
    graph is replayed."""

    def __init__(self, arrays: Sequence[Sequence[torch.Tensor]], names: Sequence[str],
                 lr_scales: Optional[Sequence[float]] = None, wd_scales: Optional[Sequence[float]] = None):
        if torch.cuda.is_available() and torch.cuda.is_current_stream_capturing():
            raise GnsError(10, "build the list of tensors before the capture (its table is copied to the GPU)")
        arrays = [list(a) for a in arrays]
        count = len(arrays[0])
        for name, a in zip(names, arrays):
            if len(a) != count:
                raise GnsError(2, f"{len(a)} {name}, {count} {names[0]}")
        for name, scales in (("lr_scales", lr_scales), ("wd_scales", wd_scales)):
            if scales is not None and len(scales) != count:
                raise GnsError(2, f"{len(scales)} {name}, {count} {names[0]}")
        self.arrays, self.tensors, self.device = len(arrays), arrays, None
        # column by column: a list is built again whenever a program replaces
        # its gradients, and may have thousands of them
        entries = np.zeros((self.arrays, max(1, count)), dtype=_ENTRY)
        shapes = None
        dense = [True] * count
        for k, (name, a) in enumerate(zip(names, arrays)):
            if not all(isinstance(t, torch.Tensor) and t.layout is torch.strided for t in a):
                i = next(i for i in range(count)
                         if not isinstance(a[i], torch.Tensor) or a[i].layout is not torch.strided)
                raise GnsError(1, f"{name}[{i}] is not a dense tensor: {type(a[i]).__name__}")
            mine = [t.shape for t in a]
            shapes = shapes or mine
            if mine != shapes:
                i = next(i for i in range(count) if mine[i] != shapes[i])
                raise GnsError(2, f"{name}[{i}] has shape {tuple(mine[i])}, "
                                  f"{names[0]}[{i}] has {tuple(shapes[i])}")
            if count == 0:
                continue
            if {t.get_device() for t in a} != {arrays[0][0].get_device()} or not arrays[0][0].is_cuda:
                for i, t in enumerate(a):
                    _device_tensor(f"{name}[{i}]", t, arrays[0][0].device if k or i else None)
            entries["data"][k] = [t.data_ptr() for t in a]
            entries["dtype"][k] = [_DT[t.dtype] if t.dtype in _DT else _dtype_code(t.dtype) for t in a]
            dense = [d and t.is_contiguous() for d, t in zip(dense, a)]
        if count:
            self.device = arrays[0][0].device
            entries["rows"] = 1
            entries["cols"] = entries["pitch"] = [t.numel() for t in arrays[0]]
        for i in (i for i, d in enumerate(dense) if not d):
            group = [a[i] for a in arrays]
            form = _rows(group) if group[0].numel() else (1, 0, [0] * self.arrays)
            if form is None:
                raise GnsError(2, f"{names[0]}[{i}]: strides {[t.stride() for t in group]} are not rows of "
                                  "consecutive elements that are the same for every array")
            entries["rows"][:, i], entries["cols"][:, i], entries["pitch"][:, i] = form
        L = lib()
        nbytes = int(L.gns_tensor_list_bytes(entries.ctypes.data, self.arrays, count))
        self.info = ListInfo()
        image = torch.empty(max(nbytes, 16), dtype=torch.uint8, device="cpu", pin_memory=self.device is not None)
        as_floats = [None if s is None else (ctypes.c_float * max(1, count))(*s) for s in (lr_scales, wd_scales)]
        _check(L.gns_tensor_list_build(entries.ctypes.data, self.arrays, count, *as_floats, image.data_ptr(),
                                       image.numel(), ctypes.byref(self.info)))
        self.count = count
        self.workspace_bytes = int(L.gns_tensor_list_workspace_bytes(ctypes.byref(self.info)))
        self._info = ctypes.byref(self.info)
        self._workspaces = {}
        self._lock = threading.RLock()
        if self.device is None:
            self.device = torch.device("cuda", torch.cuda.current_device())
        self._index = self.device.index
        self._others = torch.cuda.device_count() > 1    # asking which is current takes 0.2 us
        # the copy runs on the current stream; calls on other streams wait for it
        home = torch.cuda.current_stream(self.device)
        self._home = home.cuda_stream
        self.table = image.to(self.device, non_blocking=True)
        self._ready = torch.cuda.Event()
        self._ready.record(home)
        self._table = self.table.data_ptr()

    def __len__(self) -> int:
        return self.count

    def _workspace(self, raw: int) -> torch.Tensor:
        """The workspace of calls on one stream (those of different streams may
        overlap in time).  A captured call has one of its own: its graph may be
        replayed beside other calls.  Taken and used under the list's lock: a
        call's launches hand partials over in it, and the library's call lets
        other threads run."""
        if torch.cuda.is_current_stream_capturing():
            return torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        ws = self._workspaces.get(raw)
        if ws is None:
            ws = self._workspaces[raw] = torch.zeros(self.workspace_bytes, dtype=torch.uint8, device=self.device)
        return ws

    def _stream(self, raw: int):
        """A stream object for a raw stream."""
        if raw == 0:
            return torch.cuda.default_stream(self.device)
        return torch.cuda.ExternalStream(raw, device=self.device)

    def _on(self, stream) -> int:
        """The raw stream a call runs on, ordered after the table's copy.  (A
        raw handle is taken for one of the list's device.)"""
        if stream is None:
            raw = _current_raw_stream(self._index)
        elif isinstance(stream, int):
            raw = stream
        else:
            device = getattr(stream, "device", self.device)     # (anything with a handle is taken)
            if device.index != self._index:
                raise GnsError(11, f"stream is on {device}, the list on {self.device}")
            raw = stream.cuda_stream
        if raw != self._home:
            with torch.cuda.stream(self._stream(raw)):
                # (a capture begins after everything before it has ended)
                if not torch.cuda.is_current_stream_capturing():
                    self._ready.wait()
                self.table.record_stream(torch.cuda.current_stream(self.device))
        return raw


def tensor_list(grads: Sequence[torch.Tensor], out: Optional[Sequence[torch.Tensor]] = None) -> TensorList:
    """A list of gradients, and where clipping writes them when ``out`` is
    given (any mix of fp32, bf16 and fp16 in both).  Strided views are taken
    where they are rows of consecutive elements."""
    if out is None:
        return TensorList([grads], ["grads"])
    return TensorList([grads, out], ["grads", "out"])


def adamw_list(params: Sequence[torch.Tensor], grads: Sequence[torch.Tensor],
               exp_avgs: Sequence[torch.Tensor], exp_avg_sqs: Sequence[torch.Tensor], *,
               copies: Optional[Sequence[torch.Tensor]] = None,
               lr_scales: Optional[Sequence[float]] = None,
               wd_scales: Optional[Sequence[float]] = None) -> TensorList:
    """A list for :func:`adamw_step` (and the norm of its gradients): fp32
    parameters and moments, gradients of any type, and optionally 16-bit
    ``copies`` that every step refreshes.  ``lr_scales`` and ``wd_scales`` are
    factors per tensor on the learning rate and the weight decay."""
    arrays, names = [grads, params, exp_avgs, exp_avg_sqs], ["grads", "params", "exp_avgs", "exp_avg_sqs"]
    if copies is not None:
        arrays, names = arrays + [copies], names + ["copies"]
    return TensorList(arrays, names, lr_scales, wd_scales)


class GradNorm:
    """What a norm or a clipping call leaves on the GPU: ``norm`` and ``clip``
    (the factor to pass as ``grad_scale``) as float32 scalars, and with
    ``per_tensor`` every tensor's norm."""
    __slots__ = ("result", "tensor_norms")

    def __init__(self, result: torch.Tensor, tensor_norms: Optional[torch.Tensor]):
        self.result, self.tensor_norms = result, tensor_norms

    @property
    def norm(self) -> torch.Tensor:
        return self.result[0]

    @property
    def clip(self) -> torch.Tensor:
        return self.result[1]


def _norm_call(fn, grads, max_norm, ord, eps, inv_scale, per_tensor, workspace, stream) -> GradNorm:
    lst = grads if isinstance(grads, TensorList) else tensor_list(grads)
    if ord not in _NORMS:
        raise GnsError(11, f"ord must be 2 or inf, got {ord}")
    # the library launches on the current device, where handle 0 is another stream
    if lst._others and _current_device() != lst._index:
        with torch.cuda.device(lst.device):
            return _norm_call(fn, lst, max_norm, ord, eps, inv_scale, per_tensor, workspace, stream)
    s = lst._on(stream)
    scale = None if inv_scale is None else _scalar_ptr("inv_scale", inv_scale, lst.device)

    def buffers():
        return (torch.empty(2, dtype=torch.float32, device=lst.device),
                torch.empty(lst.count, dtype=torch.float32, device=lst.device) if per_tensor else None,
                lst._workspace(s) if workspace is None else _workspace(0, lst.device, workspace))

    with lst._lock:
        if stream is None:
            result, norms, ws = buffers()
        else:                                  # allocated for the stream that the call runs on
            with torch.cuda.stream(lst._stream(s)):
                result, norms, ws = buffers()
        _check(fn(lst._info, lst._table, _NORMS[ord], float(max_norm), float(eps), scale, result.data_ptr(),
                  _ptr(norms), ws.data_ptr(), ws.numel(), s))
    return GradNorm(result, norms)


def grad_norm(grads: Union[TensorList, Sequence[torch.Tensor]], *, ord: float = 2, max_norm: float = math.inf,
              eps: float = 1e-6, inv_scale: Optional[torch.Tensor] = None, per_tensor: bool = False,
              workspace: Optional[torch.Tensor] = None, stream=None) -> GradNorm:
    """Norm of all gradients as one vector (``ord`` 2 or inf, over the
    gradients times ``inv_scale``) and the factor that unscales them and clips
    them to ``max_norm`` (gns_grad_norm).  Nothing synchronises: pass the
    result's ``clip`` to :func:`adamw_step` and ``dion3_step`` as
    ``grad_scale``, which then clip while they read the gradients.  When a
    gradient is not finite, ``clip`` is NaN and those steps change nothing.
    With gradients sharded over ranks, gather the ranks' norms (taken with
    ``inv_scale``) and call this on them as one tensor: its norm and ``clip``
    are those of all gradients (times ``inv_scale`` once more for ``clip``).
    The list keeps a workspace for every stream it is used on, and threads may
    share the list; ``workspace`` (uint8, ``workspace_bytes`` of the list, its
    first 256 bytes zero before the first use) takes its place."""
    return _norm_call(lib().gns_grad_norm, grads, max_norm, ord, eps, inv_scale, per_tensor, workspace, stream)


def clip_grad_norm_(grads: Union[TensorList, Sequence[torch.Tensor]], max_norm: float, *, ord: float = 2,
                    eps: float = 1e-6, inv_scale: Optional[torch.Tensor] = None, per_tensor: bool = False,
                    workspace: Optional[torch.Tensor] = None, stream=None) -> GradNorm:
    """:func:`grad_norm`, then the gradients times its ``clip``: in place, or
    into the outputs of a list built with ``out`` (gns_grad_clip).  Gradients
    whose norm is not finite are left as they are.  ``inv_scale`` and
    ``workspace`` must not be memory that is written."""
    return _norm_call(lib().gns_grad_clip, grads, max_norm, ord, eps, inv_scale, per_tensor, workspace, stream)


def adamw_step(tensors: TensorList, step: Optional[int] = None, *, lr: float, betas: Sequence[float] = (0.9, 0.999),
               eps: float = 1e-8, weight_decay: float = 0.01, grad_scale: Optional[torch.Tensor] = None,
               count: Optional[torch.Tensor] = None, stream=None) -> None:
    """One AdamW update of every parameter of an :func:`adamw_list`, the
    ``step``-th (from 1), with decoupled weight decay (gns_adamw_step).
    ``grad_scale`` (a float32 on the GPU, not memory of the list) multiplies
    the gradients; when it is not finite nothing changes.

    A step that was skipped so is no update, which the program does not learn
    without waiting for the GPU.  ``count`` (one int64 on the GPU, zero before
    the first update) takes the place of ``step``: the updates made so far,
    counted up by every call that is not skipped (gns_adamw_step_counted).
    Save it with the moments.  In a captured graph every replay is then the
    next update; ``step``, ``lr`` and the other numbers are replayed as they
    were captured.

    Like all calls of this package that write in place, it does not raise the
    tensors' version counters: autograd does not notice that a parameter was
    updated between a forward pass and its backward pass."""
    if (step is None) is (count is None):
        raise GnsError(11, "either step or count")
    if tensors._others and _current_device() != tensors._index:
        with torch.cuda.device(tensors.device):
            return adamw_step(tensors, step, lr=lr, betas=betas, eps=eps, weight_decay=weight_decay,
                              grad_scale=grad_scale, count=count, stream=stream)
    s = tensors._on(stream)
    scale = None if grad_scale is None else _scalar_ptr("grad_scale", grad_scale, tensors.device)
    if count is None:
        _check(lib().gns_adamw_step(tensors._info, tensors._table, int(step), float(lr), float(betas[0]),
                                    float(betas[1]), float(eps), float(weight_decay), scale, s))
        return
    with contextlib.nullcontext() if stream is None else torch.cuda.stream(tensors._stream(s)):
        ws = torch.empty(ADAMW_WORKSPACE_BYTES, dtype=torch.uint8, device=tensors.device)
    _check(lib().gns_adamw_step_counted(tensors._info, tensors._table,
                                        _scalar_ptr("count", count, tensors.device, torch.int64), float(lr),
                                        float(betas[0]), float(betas[1]), float(eps), float(weight_decay), scale,
                                        ws.data_ptr(), ws.numel(), s))
