"""Calls on lists of tensors that are refused before anything reaches the GPU
(none needed here)."""
import ctypes
import os
import threading

import pytest
import torch

gns = pytest.importorskip("gram_newton_schulz_amd")
from gram_newton_schulz_amd import binding, tensors as T  # noqa: E402
from test_tensor_lists_host import BASE, E, F32, WS, adamw, build, norm  # noqa: E402

pytestmark = pytest.mark.skipif(not os.path.exists(gns.LIB_PATH),
                                reason="libgns.so not built (run __graft_entry__.build())")


@pytest.mark.parametrize("arrays", [4, 5])
def test_clip_in_place_of_a_gradient_that_is_other_memory_of_the_list(arrays):
    """Clipping in place would scale the parameter, a moment or the copy too."""
    for other in range(1, arrays):
        for shift in (0, 28):                      # the same memory, its last element only
            lists = [[(BASE + 4096 * a, 1, 8, 8, F32)] for a in range(arrays)]
            lists[other] = [(BASE + shift, 1, 8, 8, F32)]
            assert norm(build(lists)[1], clip=True) == E["ALIAS"], (other, shift)


@pytest.mark.parametrize("workspace,name", [
    (torch.zeros(4096, dtype=torch.uint8), "GNS_E_NULL"),
    (torch.zeros(4096, dtype=torch.uint8, device="meta"), "GNS_E_NULL"),
    (torch.zeros(1, dtype=torch.uint8).expand(4096), "GNS_E_WORKSPACE"),
    (torch.zeros(8192, dtype=torch.uint8)[::2], "GNS_E_WORKSPACE")], ids=["host", "meta", "expanded", "strided"])
def test_workspace_that_is_not_the_memory_it_names(workspace, name, monkeypatch):
    """The library takes a workspace's address and its number of bytes: a host
    tensor, or one that has other memory than that, is refused before."""
    if name == "GNS_E_WORKSPACE":                  # its device is not what is wrong with it
        monkeypatch.setattr(binding, "_device_tensor", lambda *a: None)
    lst = object.__new__(T.TensorList)
    lst.__dict__.update(device=torch.device("cuda", 0), _index=0, _others=True, count=1, _info=None, _table=0, _home=0,
                        _lock=threading.RLock())
    monkeypatch.setattr(T, "_current_device", lambda: 0)
    monkeypatch.setattr(T, "_current_raw_stream", lambda index: 0)
    real = torch.empty
    monkeypatch.setattr(torch, "empty", lambda *a, device=None, **kw: real(*a, **kw))
    for call in (lambda: binding._workspace(16, torch.device("cuda", 0), workspace),
                 lambda: T._norm_call(lambda *a: 0, lst, 1.0, 2, 1e-6, None, False, workspace, None)):
        with pytest.raises(gns.GnsError) as e:
            call()
        assert e.value.name == name


def test_adamw_eps_is_checked_as_it_is_used():
    """eps goes into the update in fp32, where anything up to 2^-150 is zero
    and an element without a gradient would be 0 / 0."""
    info = build([[(BASE + 4096 * a, 1, 8, 8, F32)] for a in range(4)])[1]
    for eps in (2.0 ** -150, 1e-46, 1e-300, 0.0, -1e-8):
        assert adamw(info, eps=eps) == E["PARAM"], eps
    # the smallest that is one of fp32 passes this check (and stops at the table)
    assert adamw(info, eps=2.0 ** -149, table=None) == E["NULL"]


def test_counted_adamw_refusals():
    info = build([[(BASE + 4096 * a, 1, 8, 8, F32)] for a in range(4)])[1]

    def call(info=info, count=WS, eps=1e-8, b1=0.9, table=None, ws=WS + 4096, ws_bytes=T.ADAMW_WORKSPACE_BYTES):
        return gns.lib().gns_adamw_step_counted(ctypes.byref(info), table, count, 0.1, b1, 0.99, eps, 0.0, None, ws,
                                                ws_bytes, None)

    assert call() == E["NULL"] and call(count=None) == E["NULL"]
    assert call(count=WS + 4) == E["PARAM"] and call(eps=0.0) == E["PARAM"] and call(b1=1.0) == E["PARAM"]
    for kw in ({"ws": None}, {"ws": WS + 16}, {"ws_bytes": 255}):
        assert call(**kw) == E["WORKSPACE"], kw
    assert call(info=build([[(BASE, 1, 8, 8, F32)]])[1]) == E["SHAPE"]
    shared = build([[(BASE + 4096 * min(a, 2), 1, 8, 8, F32)] for a in range(4)])[1]
    assert call(info=shared, table=BASE) == E["ALIAS"]
