"""A list dropped while a call on another stream is pending (no GPU): its
device copy is recorded on every queue it is used on."""
import pytest
import torch

import quantized_momentum_newton_amd as q
from test_list_devices_cpu import CALLS, FakeStream, adamw_entry, two_devices  # noqa: F401


class FakeCopy:
    """Stands for the device copy: which streams it was recorded on."""

    def __init__(self):
        self.on = []

    def record_stream(self, stream):
        self.on.append(stream.cuda_stream)


@pytest.mark.parametrize("name", list(CALLS))
def test_the_device_copy_is_recorded_on_other_queues(request, monkeypatch, name):
    plan = q.GradPlan([torch.zeros(8)]) if name.startswith("grad") else q.AdamWPlan([adamw_entry()])
    plan.device, plan.dev, plan.queues = torch.device("cuda", 1), FakeCopy(), {1001}
    now, seen = request.getfixturevalue("two_devices")
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: FakeStream(index, 1000 + index))
    CALLS[name](plan, None)                       # the queue it was made on
    assert plan.dev.on == []
    for _ in range(2):
        CALLS[name](plan, FakeStream(1, 77))
    assert plan.dev.on == [77]
    monkeypatch.setattr(torch._C, "_cuda_getCurrentRawStream", lambda index: 2000 + index)
    monkeypatch.setattr(torch.cuda, "current_stream", lambda index: FakeStream(index, 2000 + index))
    CALLS[name](plan, None)                       # another current stream
    assert plan.dev.on == [77, 2001] and len(seen) == 4
