"""Lists of tensors on the host (no GPU needed): the device table covers every
element once, overlaps are found, bad arguments are refused with the
documented status before anything is enqueued, and the oracle agrees with
torch's own optimiser."""
import ctypes
import math
import os
import struct

import numpy as np
import pytest
import torch

import oracle

gns = pytest.importorskip("gram_newton_schulz_amd")
from gram_newton_schulz_amd import tensors as T  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(gns.LIB_PATH),
                                reason="libgns.so not built (run __graft_entry__.build())")

BASE = 0x10000000  # never dereferenced
WS = 0x7f0000000000
E = {"OK": 0, "NULL": 1, "SHAPE": 2, "DTYPE": 3, "ALIAS": 7, "WORKSPACE": 8, "PARAM": 11}
F32, BF16, F16 = gns.GNS_F32, gns.GNS_BF16, gns.GNS_F16
ENTRY = struct.Struct("<5Q5qqqqII2f5B11x")


def make(arrays):
    """arrays: per array a list of (address, rows, cols, pitch, dtype)."""
    flat = [T.Tensor(*t) for a in arrays for t in a]
    return (T.Tensor * max(1, len(flat)))(*flat), len(arrays), len(arrays[0])


def build(arrays, short=0):
    L = gns.lib()
    ent, n, count = make(arrays)
    nbytes = L.gns_tensor_list_bytes(ent, n, count)
    table = np.zeros(max(nbytes, 16) // 8 + 2, dtype=np.uint64)
    info = T.ListInfo()
    at = (table.ctypes.data + 15) // 16 * 16
    st = L.gns_tensor_list_build(ent, n, count, None, None, at, nbytes - short, ctypes.byref(info))
    raw = ctypes.string_at(at, nbytes) if st == 0 else b""
    return st, info, raw


def parse(info, raw):
    entries = [ENTRY.unpack_from(raw, ENTRY.size * i) for i in range(info.count)]
    chunks = [struct.unpack_from("<II", raw, ENTRY.size * info.count + 8 * c) for c in range(info.chunks)]
    return entries, chunks


def overlaps(info, a, b):
    return bool(info.overlaps >> (5 * min(a, b) + max(a, b)) & 1)


@pytest.mark.parametrize("sizes", [[1], [7, 8, 9], [8192, 8191, 8193, 1], [0, 5, 0], [], [1 << 27, 3, 40001]])
def test_chunks_cover_every_unit_once(sizes):
    at, lst = BASE, []
    for n in sizes:
        lst.append((at if n else None, 1, n, n, BF16))
        at += 2 * n
    st, info, raw = build([lst])
    assert st == 0 and info.elements == sum(sizes) and info.overlaps == 0
    entries, chunks = parse(info, raw)
    seen = {}
    for entry, index in chunks:
        units = entries[entry][12]
        lo = index * info.chunk_units
        assert 0 <= lo < units
        assert seen.get(entry, 0) == lo                    # in order, no gap
        seen[entry] = min(units, lo + info.chunk_units)
    for i, n in enumerate(sizes):
        assert entries[i][12] == -(-n // 8) and seen.get(i, 0) == entries[i][12]
        assert entries[i][14] == -(-entries[i][12] // info.chunk_units)
    starts = [e[13] for e in entries]
    assert starts == [sum(e[14] for e in entries[:i]) for i in range(len(entries))]


def test_strided_entries_count_units_by_row():
    st, info, raw = build([[(BASE, 5, 13, 40, F32), (BASE + 4 * 13, 5, 13, 40, F32), (BASE + 4 * 400, 4, 6, 6, F16)]])
    assert st == 0 and info.overlaps == 0 and info.elements == 5 * 13 * 2 + 24
    entries, _ = parse(info, raw)
    assert [e[11] for e in entries] == [2, 2, 3] and [e[12] for e in entries] == [10, 10, 3]
    assert [e[10] for e in entries] == [13, 13, 24]          # the dense one is a single row
    # an entry that is dense in one array only keeps its rows in all of them
    st, info, raw = build([[(BASE, 4, 6, 9, F32)], [(BASE + 4096, 4, 6, 6, BF16)]])
    entries, _ = parse(info, raw)
    assert st == 0 and entries[0][10] == 6 and entries[0][5:7] == (9, 6) and entries[0][12] == 4


def test_overlaps():
    a = (BASE, 1, 100, 100, F32)
    assert build([[a, (BASE + 400, 1, 5, 5, F32)]])[1].overlaps == 0
    info = build([[a, (BASE + 396, 1, 5, 5, F32)]])[1]
    assert overlaps(info, 0, 0)
    info = build([[a], [(BASE + 200, 1, 100, 100, F32)]])[1]
    assert overlaps(info, 0, 1) and not overlaps(info, 0, 0) and not overlaps(info, 1, 1)
    # column slices of one matrix touch nothing of each other, until one is a column too wide
    cols = [(BASE + 4 * c, 7, w, 30, F32) for c, w in ((0, 10), (10, 15), (25, 5))]
    assert build([cols])[1].overlaps == 0
    assert overlaps(build([[cols[0], (BASE + 4 * 9, 7, 5, 30, F32)]])[1], 0, 0)
    assert overlaps(build([[cols[2], (BASE + 4 * 26, 7, 10, 30, F32)]])[1], 0, 0)   # wraps into the next row
    assert overlaps(build([[cols[0], (BASE + 4 * 15, 1, 16, 16, F32)]])[1], 0, 0)
    assert build([[cols[0], (BASE + 4 * 15, 1, 15, 15, F32)]])[1].overlaps == 0
    # rows that repeat
    assert overlaps(build([[(BASE, 4, 8, 0, F32)]])[1], 0, 0)
    # different pitches count as shared
    assert overlaps(build([[(BASE, 4, 2, 8, F32), (BASE + 16, 4, 2, 10, F32)]])[1], 0, 0)


def test_build_refusals():
    ok = (BASE, 2, 3, 3, F32)
    for bad, want in [((BASE, -1, 3, 3, F32), "SHAPE"), ((BASE, 2, -3, 3, F32), "SHAPE"),
                      ((BASE, 2, 3, -1, F32), "SHAPE"), ((None, 2, 3, 3, F32), "NULL"),
                      ((BASE, 2, 3, 3, gns.GNS_BF16X3), "DTYPE"), ((BASE, 2, 3, 3, 9), "DTYPE"),
                      ((BASE + 2, 2, 3, 3, F32), "PARAM"), ((BASE + 1, 2, 3, 3, BF16), "PARAM"),
                      ((BASE, 1 << 40, 1 << 30, 1 << 30, F32), "SHAPE"),
                      ((BASE, 4, 3, 1 << 62, F32), "SHAPE")]:
        ent, n, count = make([[ok, bad]])
        assert gns.lib().gns_tensor_list_bytes(ent, n, count) == 0
        info, buf = T.ListInfo(), np.zeros(64, dtype=np.uint64)
        assert gns.lib().gns_tensor_list_build(ent, n, count, None, None, buf.ctypes.data, 512,
                                               ctypes.byref(info)) == E[want], bad
    L, info = gns.lib(), T.ListInfo()
    ent, _, _ = make([[ok], [ok]])
    buf = np.zeros(64, dtype=np.uint64)
    call = lambda n, count, lr=None, table=buf.ctypes.data, size=512, out=ctypes.byref(info): \
        L.gns_tensor_list_build(ent, n, count, lr, None, table, size, out)   # noqa: E731
    assert call(3, 1) == E["SHAPE"] and call(0, 1) == E["SHAPE"] and call(1, -1) == E["SHAPE"]
    assert call(1, (1 << 20) + 1) == E["SHAPE"]
    assert call(1, 1, table=None) == E["NULL"] and call(1, 1, out=None) == E["NULL"]
    assert call(1, 1, size=100) == E["WORKSPACE"] and call(1, 1, table=buf.ctypes.data + 4) == E["WORKSPACE"]
    assert call(1, 1, lr=(ctypes.c_float * 1)(math.nan)) == E["PARAM"]
    assert L.gns_tensor_list_build(None, 1, 1, None, None, buf.ctypes.data, 512, ctypes.byref(info)) == E["NULL"]
    # arrays whose entries differ in shape
    ent, n, count = make([[ok], [(BASE + 64, 3, 2, 2, F32)]])
    assert L.gns_tensor_list_bytes(ent, n, count) == 0
    assert build([[ok, ok]], short=8)[0] == E["WORKSPACE"]


def norm(info, clip=False, kind=0, max_norm=1.0, eps=1e-6, table=BASE, result=BASE + 4096, ws=WS, ws_bytes=1 << 20):
    f = gns.lib().gns_grad_clip if clip else gns.lib().gns_grad_norm
    return f(ctypes.byref(info) if info is not None else None, table, kind, max_norm, eps, None, result, None,
             ws, ws_bytes, None)


def test_norm_and_clip_refusals():
    _, info, _ = build([[(BASE, 2, 3, 3, F32)]])
    assert gns.lib().gns_tensor_list_workspace_bytes(ctypes.byref(info)) == 256 + 8
    assert gns.lib().gns_tensor_list_workspace_bytes(None) == 0
    for clip in (False, True):
        assert norm(None, clip) == E["NULL"]
        assert norm(info, clip, kind=2) == E["PARAM"]
        assert norm(info, clip, max_norm=-1.0) == E["PARAM"] and norm(info, clip, max_norm=math.nan) == E["PARAM"]
        assert norm(info, clip, eps=-1e-9) == E["PARAM"] and norm(info, clip, eps=math.inf) == E["PARAM"]
        assert norm(info, clip, table=None) == E["NULL"] and norm(info, clip, result=None) == E["NULL"]
        assert norm(info, clip, ws=None) == E["WORKSPACE"] and norm(info, clip, ws=WS + 8) == E["WORKSPACE"]
        assert norm(info, clip, ws_bytes=4) == E["WORKSPACE"]
    broken = T.ListInfo.from_buffer_copy(info)
    broken.chunks += 1                                     # not what the build left
    assert norm(broken) == E["SHAPE"]
    # written memory that is other memory of the list too
    same = (BASE, 1, 8, 8, F32)
    assert norm(build([[same, same]])[1], True) == E["ALIAS"]
    assert norm(build([[(BASE, 4, 8, 0, F32)]])[1], True) == E["ALIAS"]
    assert norm(build([[same], [same]])[1], True) == E["ALIAS"]
    out = (BASE + 64, 1, 8, 8, F32)
    assert norm(build([[same, same], [out, out]])[1], True) == E["ALIAS"]


def adamw(info, step=1, lr=0.1, b1=0.9, b2=0.99, eps=1e-8, wd=0.0, table=BASE):
    return gns.lib().gns_adamw_step(ctypes.byref(info) if info is not None else None, table, step, lr, b1, b2, eps,
                                    wd, None, None)


def test_adamw_refusals():
    def lst(grad=F32, moment=F32, shift=(0, 1, 2, 3), n=4):
        arrays = [[(BASE + 4096 * shift[a], 1, 8, 8, grad if a == 0 else moment if a == 3 else F32)]
                  for a in range(4)]
        return build(arrays[:n])[1]
    assert adamw(None) == E["NULL"]
    assert adamw(build([[(BASE, 1, 8, 8, F32)]])[1]) == E["SHAPE"]
    assert adamw(lst(moment=BF16)) == E["DTYPE"]
    assert adamw(lst(), table=None) == E["NULL"]
    for kw in ({"step": 0}, {"lr": math.inf}, {"b1": 1.0}, {"b1": -0.1}, {"b2": math.nan}, {"eps": 0.0},
               {"eps": math.inf}, {"wd": math.nan}):
        assert adamw(lst(), **kw) == E["PARAM"], kw
    assert adamw(lst(shift=(0, 1, 1, 3))) == E["ALIAS"]
    assert adamw(lst(shift=(2, 1, 2, 3))) == E["ALIAS"]
    # an empty list has nothing to do
    assert adamw(build([[], [], [], []])[1], table=None) == E["OK"]


def test_binding_refuses_cpu_tensors_and_mismatches():
    with pytest.raises(gns.GnsError) as e:
        gns.tensor_list([torch.zeros(3)])
    assert e.value.name == "GNS_E_NULL"
    with pytest.raises(gns.GnsError) as e:
        gns.tensor_list([torch.zeros(3)], out=[])
    assert e.value.name == "GNS_E_SHAPE"
    with pytest.raises(gns.GnsError):
        gns.tensor_list([None])
    with pytest.raises(gns.GnsError):
        gns.adamw_list([torch.zeros(3)], [torch.zeros(4)], [torch.zeros(3)], [torch.zeros(3)])
    with pytest.raises(gns.GnsError):
        gns.adamw_list([], [], [], [], lr_scales=[1.0])


def strided(shape, strides, dtype=torch.float32):
    n = 1 + sum((s - 1) * t for s, t in zip(shape, strides))
    return torch.zeros(n, dtype=dtype).as_strided(shape, strides)


@pytest.mark.parametrize("shape,strides,want", [
    ((4, 6), (6, 1), (1, 24, [24])),            # dense
    ((4, 6), (1, 4), (1, 24, [24])),            # transposed: the same memory
    ((4, 6), (10, 1), (4, 6, [10])),            # column slice
    ((6, 4), (1, 10), (4, 6, [10])),            # its transpose
    ((2, 3, 5), (15, 5, 1), (1, 30, [30])),
    ((2, 3, 5), (30, 10, 1), (6, 5, [10])),     # two outer dimensions that merge
    ((2, 5, 3), (15, 1, 5), (1, 30, [30])),
    ((2, 3, 5), (31, 10, 1), None),             # three that do not
    ((4, 6), (12, 2), (24, 1, [2])),            # every second element
    ((4, 6), (13, 2), None),
    ((4, 6), (0, 1), (4, 6, [0])),              # an expanded row
    ((4, 6), (0, 0), (24, 1, [0])),             # an expanded scalar
    ((4, 6), (1, 0), (6, 4, [0])),          # a repeated column
    ((), (), (1, 1, [1])),
    ((1, 6), (99, 1), (1, 6, [6])),
    ((6, 1), (3, 1), (6, 1, [3])),
])
def test_row_forms(shape, strides, want):
    assert T._rows([strided(shape, strides)]) == want


def test_row_forms_of_groups():
    a, b = strided((4, 6), (6, 1)), strided((4, 6), (9, 1))
    assert T._rows([a, b]) == (4, 6, [6, 9])
    assert T._rows([a, strided((4, 6), (1, 4))]) is None        # one transposed, one not
    t = strided((4, 6), (1, 4))
    assert T._rows([t, t]) == (1, 24, [24, 24])


def test_oracle_adamw_matches_torch():
    """The oracle's update against torch.optim.AdamW on the CPU in 64 bits."""
    rng = np.random.default_rng(3)
    p = rng.normal(size=37)
    param = torch.nn.Parameter(torch.from_numpy(p.copy()))
    opt = torch.optim.AdamW([param], lr=0.02, betas=(0.9, 0.95), eps=1e-8, weight_decay=0.3)
    m = v = np.zeros_like(p)
    for step in range(1, 5):
        g = rng.normal(size=37)
        param.grad = torch.from_numpy(g.copy())
        opt.step()
        p, m, v = oracle.adamw(p, g, m, v, step, 0.02, (0.9, 0.95), 1e-8, 0.3)
        assert np.allclose(param.detach().numpy(), p, rtol=1e-13, atol=1e-15)


def test_oracle_norm_matches_torch():
    rng = np.random.default_rng(4)
    gs = [rng.normal(size=(3, 5)), rng.normal(size=11)]
    for ord in (2, math.inf):
        params = [torch.nn.Parameter(torch.zeros(g.shape, dtype=torch.float64)) for g in gs]
        for q, g in zip(params, gs):
            q.grad = torch.from_numpy(g.copy())
        want = torch.nn.utils.clip_grad_norm_(params, 0.7, norm_type=ord)
        norm, clip, _ = oracle.grad_norm(gs, ord, 0.7)
        assert abs(norm - float(want)) <= 1e-14 * norm
        for q, g in zip(params, gs):
            assert np.allclose(q.grad.numpy(), g * clip, rtol=1e-13)
