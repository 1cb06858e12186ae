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
