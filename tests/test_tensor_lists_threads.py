"""Host threads that share one list of tensors (no GPU needed: the library's
call is a stand-in that takes a while)."""
import threading
import time

import pytest
import torch

gns = pytest.importorskip("gram_newton_schulz_amd")
from gram_newton_schulz_amd import tensors as T  # noqa: E402


@pytest.fixture
def one_list(monkeypatch):
    """A list on the CPU, whose calls see stream 0, no capture."""
    lst = object.__new__(T.TensorList)
    lst.__dict__.update(device=torch.device("cpu"), _index=None, _others=True, count=1,
                        workspace_bytes=1024, _info=None, _table=0, _home=0, _workspaces={}, _lock=threading.RLock())
    monkeypatch.setattr(T, "_current_device", lambda: None)
    monkeypatch.setattr(T, "_current_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    return lst


def test_calls_on_one_stream_do_not_mix_their_launches(one_list):
    """A norm of many chunks is two launches that hand the partials over in
    the workspace: while one call is between them, no other call may use it."""
    inside, mixed, seen = {}, [], []
    guard = threading.Lock()

    def call(info, table, kind, max_norm, eps, inv_scale, result, norms, workspace, nbytes, stream):
        with guard:
            inside[workspace] = inside.get(workspace, 0) + 1
            seen.append(workspace)
            if inside[workspace] > 1:
                mixed.append(workspace)
        time.sleep(0.005)                          # releases the interpreter lock, as the library's call does
        with guard:
            inside[workspace] -= 1
        return 0

    start = threading.Barrier(4)

    def worker(ord):
        start.wait()
        for _ in range(10):
            T._norm_call(call, one_list, 1.0, ord, 1e-6, None, False, None, None)

    threads = [threading.Thread(target=worker, args=(o,)) for o in (2, float("inf"), 2, float("inf"))]
    for t in threads:
        t.start()
    for t in threads:
        t.join()
    assert len(seen) == 40 and not mixed
