"""The training example's step without a GPU: which operators a batch whose
norm is not finite reaches."""
import importlib.util
import os

import pytest
import torch

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def load_example():
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    return mod


@pytest.mark.parametrize("coef,calls", [(float("nan"), []), (0.5, ["grad_scale", "muon_step", "adamw_step"])])
def test_a_norm_that_is_not_finite_stops_every_operator_that_writes(monkeypatch, coef, calls):
    mod = load_example()
    seen = []
    for name in ("grad_scale", "muon_step", "adamw_step"):
        monkeypatch.setattr(mod.q, name, lambda *a, _name=name, **k: seen.append(_name))
    monkeypatch.setattr(mod.q, "grad_norm", lambda *a, coef, norm, _c=coef_value(coef), **k: coef.copy_(_c))
    opt = mod.Optimizer.__new__(mod.Optimizer)
    opt.steps, opt.max_norm, opt.lr_adamw = 4, 1.0, 1e-3
    opt.all_grads = opt.muon_grads = opt.muon_plan = opt.mats = opt.muon_hp = opt.muon_ws = opt.adamw_plan = opt.ws = None
    opt.norm, opt.coef = torch.zeros(1), torch.zeros(1)
    done = opt.step()
    assert seen == calls and bool(done) == bool(calls) and opt.steps == 4 + bool(calls)


def coef_value(c):
    return torch.full((1,), c)
