"""Buffers that the gradient-norm and AdamW calls are given next to their list
(no GPU): workspace and outputs."""
import ctypes

import pytest
import torch

import quantized_momentum_newton_amd as q
from test_adamw_cpu import ARG, BASE, DEV, LIB, _adamw, _encode, _grads


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


def test_outputs_may_not_share_memory():
    """Both outputs of a call are written by it, in no order."""
    a, g = _encode(_adamw([(1024, 8), (100, 32)])), _encode(_grads([(1024, 0)]))
    span = 4 * 256 * 5
    for lo, hi in ((0, 0), (0, span - 16), (64, 48)):
        at = [ctypes.c_void_p(BASE + x) for x in (lo, hi)]
        assert LIB.adamw_read_state(a[1], DEV, *at, None) == ARG and b"overlap" in LIB.qm_last_error()
        assert LIB.adamw_read_state(a[1], DEV, *at[::-1], None) == ARG and b"overlap" in LIB.qm_last_error()
    at = ctypes.c_void_p(BASE + 4096)
    assert LIB.grad_norm(g[1], DEV, 1.0, 1e-6, at, at, DEV, 4096, None) == ARG and b"share" in LIB.qm_last_error()
