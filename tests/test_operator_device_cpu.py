"""The calls made through ctypes run on the device of their tensors, whichever
device is current: against a stand-in for the library, with tensors that have
no memory, on a machine without a GPU."""
import contextlib
import types

import pytest
import torch
from torch._subclasses.fake_tensor import FakeTensorMode

from sparse_moe_expert_gb300 import binding


@pytest.fixture()
def machine(monkeypatch):
    """Two devices, 0 current, each with its current stream (handle 100 +
    device); calls[i] = (name, current device, stream handle)."""
    state = types.SimpleNamespace(current=0, calls=[])

    @contextlib.contextmanager
    def device(d):
        before, state.current = state.current, torch.device(d).index
        yield
        state.current = before

    class Lib:
        def __getattr__(self, name):
            def call(*args):
                state.calls.append((name, state.current, args[-1].value))
                return 0
            return call

    monkeypatch.setattr(torch.cuda, "current_device", lambda: state.current)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda d=None: types.SimpleNamespace(
        cuda_stream=100 + (state.current if d is None else torch.device(d).index)))
    monkeypatch.setattr(binding, "lib", lambda: Lib())
    monkeypatch.setattr(binding, "_p", lambda t: None)
    with FakeTensorMode():
        yield state


@pytest.mark.parametrize("index", [0, 1])
def test_router_logits_run_on_their_device(machine, index):
    d = f"cuda:{index}"
    out = binding.moe_router_logits(torch.empty((4, 64), dtype=torch.bfloat16, device=d),
                                    torch.empty((8, 64), device=d))
    assert out.device.index == index
    assert machine.calls == [("moe_router_logits", index, 100 + index)] and machine.current == 0


@pytest.mark.parametrize("index", [0, 1])
def test_grouping_runs_on_its_device(machine, index):
    d = f"cuda:{index}"
    out = binding.moe_permute_masked(torch.empty((4, 2), dtype=torch.int32, device=d),
                                     torch.empty(1, dtype=torch.int32, device=d), 8)
    assert all(t.device.index == index for t in out)
    assert machine.calls == [("moe_permute_masked", index, 100 + index)] and machine.current == 0
