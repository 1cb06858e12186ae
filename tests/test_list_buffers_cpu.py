"""Buffers that the gradient-norm and AdamW calls are given next to their list
(no GPU): workspace and outputs."""
import pytest
import torch

import quantized_momentum_newton_amd as q


@pytest.mark.parametrize("ws", [torch.empty(4096, dtype=torch.uint8, device="meta"), torch.zeros(8192, dtype=torch.uint8)[::2],
                                "4096", 4096])
def test_workspace_is_a_contiguous_tensor_on_the_lists_device(ws):
    """A workspace in host memory would be written by the device."""
    plan = q.GradPlan([torch.zeros(8)])
    with pytest.raises((ValueError, TypeError), match="ws"):
        q.grad_norm(plan, ws=ws)


def test_workspace_size_is_in_bytes(monkeypatch):
    plan = q.GradPlan([torch.zeros(8)])
    got = []
    monkeypatch.setattr(q, "_launch", lambda plan, stream, entry, *args: got.append(args[-1]))
    q.grad_norm(plan, ws=torch.zeros(4, dtype=torch.float64))
    assert got == [32]
