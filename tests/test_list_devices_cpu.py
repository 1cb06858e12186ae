"""Devices of the tensor lists in the binding (no GPU): the device a list is
given, and the one a call launches on."""
import pytest
import torch

import quantized_momentum_newton_amd as q


def adamw_entry(n=8):
    return (torch.zeros(n), torch.zeros(n), q.AdamWState(n, device="cpu"), None, 1.0, 0.0)


@pytest.mark.parametrize("device", [None, "cpu", torch.device("cpu")])
def test_device_in_any_form(device):
    for plan in (q.GradPlan([torch.zeros(8)], device=device), q.AdamWPlan([adamw_entry()], device=device)):
        assert plan.device == torch.device("cpu") and plan.dev.device == plan.device
    plan = q.GradPlan([torch.zeros(8)], device=device)
    with pytest.raises(ValueError, match="elements"):
        q.grad_scale(plan, torch.zeros(2))       # past the check of its device


def test_unindexed_device_is_the_current_one(monkeypatch):
    monkeypatch.setattr(torch.cuda, "current_device", lambda: 3)
    home = torch.device("cuda", 3)
    assert q._plan_device("cuda", home) == home and q._plan_device(torch.device("cuda"), home).index == 3
    assert q._plan_device("cuda:3", home) == home
    with pytest.raises(ValueError, match="cuda:1"):
        q._plan_device("cuda", torch.device("cuda", 1))


def test_a_list_lives_where_its_tensors_are():
    with pytest.raises(ValueError, match="cpu"):
        q.GradPlan([torch.zeros(8)], device="meta")
    with pytest.raises(ValueError, match="cpu"):
        q.AdamWPlan([adamw_entry()], device="meta")


CALLS = {"grad_norm": lambda p, s: q.grad_norm(p, stream=s), "grad_scale": lambda p, s: q.grad_scale(p, torch.zeros(1), stream=s),
         "adamw_step": lambda p, s: q.adamw_step(p, 1, stream=s), "adamw_read_state": lambda p, s: q.adamw_read_state(p, stream=s)}


class FakeStream:
    def __init__(self, index, handle):
        self.device, self.cuda_stream = torch.device("cuda", index), handle


@pytest.fixture
def two_devices(monkeypatch):
    """Stand-ins for the runtime's current device and streams, and for the
    library: what a call launches on, as (entry, current device, queue)."""
    now, seen = [0], []

    class device:
        def __init__(self, index):
            self.index = index

        def __enter__(self):
            self.before, now[0] = now[0], self.index

        def __exit__(self, *a):
            now[0] = self.before

    monkeypatch.setattr(torch._C, "_cuda_getDevice", lambda: now[0], raising=False)
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 1000 + index, raising=False)
    monkeypatch.setattr(torch.cuda, "device", device)
    monkeypatch.setattr(q, "_new", lambda count, dtype, plan, stream: torch.zeros(count, dtype=dtype))
    monkeypatch.setattr(q, "_require", lambda *a, **k: None)

    class Lib:
        def __getattr__(self, name):
            if name == "grad_norm_workspace_bytes":
                return lambda plan: 8

            def entry(*args):
                seen.append((name, now[0], args[-1]))
                return 0
            return entry

    monkeypatch.setattr(q, "_LIB", Lib())
    return now, seen


@pytest.mark.parametrize("name", list(CALLS))
@pytest.mark.parametrize("current", [0, 1])
def test_calls_run_on_the_lists_device(request, name, current):
    plan = q.GradPlan([torch.zeros(8)]) if name.startswith("grad") else q.AdamWPlan([adamw_entry()])
    plan.device = torch.device("cuda", 1)
    now, seen = request.getfixturevalue("two_devices")
    now[0] = current
    CALLS[name](plan, None)
    CALLS[name](plan, FakeStream(1, 77))
    assert seen == [(name, 1, 1001), (name, 1, 77)] and now[0] == current
    with pytest.raises(ValueError, match="stream"):
        CALLS[name](plan, FakeStream(0, 78))
    assert len(seen) == 2
