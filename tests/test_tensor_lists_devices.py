"""Lists of tensors on a device that is not the current one (no GPU needed:
device handling and the library's calls are stand-ins)."""
import threading
from types import SimpleNamespace

import pytest
import torch

gns = pytest.importorskip("gram_newton_schulz_amd")
from gram_newton_schulz_amd import tensors as T  # noqa: E402


class Second:
    """Stands for cuda:1 where only its index is looked at."""
    type, index = "cuda", 1


@pytest.fixture
def machine(monkeypatch):
    """Two devices, the first current; the calls that reach the library are
    recorded with the device that was current then."""
    state = SimpleNamespace(current=0, calls=[])

    class Device:
        def __init__(self, device):
            self.index = device.index

        def __enter__(self):
            self.before, state.current = state.current, self.index

        def __exit__(self, *exc):
            state.current = self.before

    def call(*args):
        state.calls.append((state.current, args[-1]))
        return 0

    monkeypatch.setattr(T, "_current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", Device)
    monkeypatch.setattr(T, "_current_raw_stream", lambda index: 0)
    monkeypatch.setattr(torch.cuda, "is_current_stream_capturing", lambda: False)
    monkeypatch.setattr(T, "lib", lambda: SimpleNamespace(gns_grad_norm=call, gns_grad_clip=call, gns_adamw_step=call))
    real = torch.empty, torch.zeros                    # (allocations on cuda:1 come from the CPU)
    for f in real:
        monkeypatch.setattr(torch, f.__name__, lambda *a, _f=f, device=None, **kw: _f(*a, **kw))
    return state


def on(device):
    lst = object.__new__(T.TensorList)
    lst.__dict__.update(device=device, _index=device.index, _others=True, count=1,
                        workspace_bytes=1024, _info=None, _table=0, _home=0, _workspaces={}, _lock=threading.RLock())
    return lst


def test_calls_run_on_the_device_of_the_list(machine):
    """Stream 0 is each device's own default stream, so the call has to be
    made with the list's device current."""
    lst = on(Second())
    gns.grad_norm(lst)
    gns.clip_grad_norm_(lst, 1.0)
    gns.adamw_step(lst, 1, lr=0.1)
    assert machine.calls == [(1, 0)] * 3 and machine.current == 0
    machine.current = 1                                # current already
    gns.grad_norm(lst)
    assert machine.calls[-1] == (1, 0) and machine.current == 1


def test_streams_of_another_device_are_refused(machine):
    lst = on(Second())
    stream = SimpleNamespace(device=SimpleNamespace(type="cuda", index=0), cuda_stream=0)
    for f in (lambda: gns.grad_norm(lst, stream=stream), lambda: gns.clip_grad_norm_(lst, 1.0, stream=stream),
              lambda: gns.adamw_step(lst, 1, lr=0.1, stream=stream)):
        with pytest.raises(gns.GnsError) as e:
            f()
        assert e.value.name == "GNS_E_PARAM"
    assert not machine.calls and machine.current == 0


def test_any_object_with_a_handle_is_a_stream(machine):
    lst = on(Second())
    gns.adamw_step(lst, 1, lr=0.1, stream=SimpleNamespace(cuda_stream=0))
    assert machine.calls == [(1, 0)]
