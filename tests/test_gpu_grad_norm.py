"""Global gradient norm, clip factor and scaling on the GPU against fp64.

The norm is summed in fp64, whose error over 10^9 terms stays far below fp32's
half step, so norm and factor may be off by their rounding to fp32 alone
(2^-24 relative; 2^-23 allowed for a value next to a border of the sum's own
rounding).  The scaled gradients are one fp32 product rounded once more to
their type: bit for bit."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from harness import inputs as H
from oracle import adamw as A

pytestmark = pytest.mark.gpu
DEV = "cuda"
REL = 2.0 ** -23
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def host(t):
    return t.detach().double().cpu().numpy()


def check(grads, max_norm, eps=1e-6):
    before = [g.detach().clone() for g in grads]
    norm, coef = A.norm_and_coef([host(g) for g in grads], max_norm, eps)
    plan = q.GradPlan(grads)
    n, c = q.grad_norm(plan, max_norm, eps)
    q.grad_scale(plan, c)
    torch.cuda.synchronize()
    say("norm", n.item(), norm, "coef", c.item(), coef)
    assert abs(n.item() - norm) <= REL * norm
    assert abs(c.item() - coef) <= REL * coef
    for g, b in zip(grads, before):
        assert torch.equal(g.cpu(), (b.float().cpu() * c.cpu()).to(g.dtype))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("sizes", [[1], [0, 3], [255, 256, 257], [1023, 1024, 1025, 1], [70001, 5, 333 * 1001],
                                   [8192 * 1024 + 77]])
def test_sizes(dt, sizes):
    grads = []
    for i, n in enumerate(sizes):
        room = torch.full((n + 16,), 3.0, dtype=dt, device=DEV)
        room[8 + i % 3:8 + i % 3 + n] = H.grad((n,), dt, DEV, 40 + i, n, std=1e-1)
        grads.append(room[8 + i % 3:8 + i % 3 + n])
    check(grads, 0.05)
    check(grads, 1e6)


@pytest.mark.parametrize("cols,ld", [(8, 8), (256, 300), (7, 9), (1, 2), (1001, 1003)])
def test_views_and_mixed_types(cols, ld):
    wide = [torch.full((41, ld), 5.0, dtype=dt, device=DEV) for dt in TYPES]
    grads = [w[:, :cols] for w in wide]
    for i, g in enumerate(grads):
        g.copy_(H.grad((41, cols), g.dtype, DEV, 60 + i, cols, std=0.3))
    grads.append(H.grad((33,), torch.bfloat16, DEV, 70, 1))
    check(grads, 0.2)
    for w in wide:
        assert torch.all(w[:, cols:] == 5.0)


def test_squares_past_fp32():
    """Gradients whose squares leave fp32's range have a finite norm."""
    g = [torch.full((1000,), 1e30, device=DEV), torch.full((10,), 1e-30, device=DEV)]
    plan = q.GradPlan(g)
    n, c = q.grad_norm(plan, 1.0)
    assert abs(n.item() / (1e30 * 1000 ** 0.5) - 1) < 1e-6 and 0 < c.item() < 1e-30
    plan = q.GradPlan([torch.full((1000,), 1e-30, device=DEV)])
    assert abs(q.grad_norm(plan)[0].item() / (1e-30 * 1000 ** 0.5) - 1) < 1e-6


def test_zero_gradients_and_no_limit():
    plan = q.GradPlan([torch.zeros(300, device=DEV)])
    n, c = q.grad_norm(plan, 1.0)
    assert n.item() == 0.0 and c.item() == 1.0
    n, c = q.grad_norm(plan, 1.0, eps=0.0)          # max_norm / 0
    assert n.item() == 0.0 and c.item() == 1.0
    n, c = q.grad_norm(q.GradPlan([torch.ones(4, device=DEV)]))
    assert n.item() == 2.0 and c.item() == 1.0
    n, c = q.grad_norm(q.GradPlan([torch.zeros(0, device=DEV)]), 1.0)
    assert n.item() == 0.0 and c.item() == 1.0


@pytest.mark.parametrize("bad", [float("nan"), float("inf")])
def test_non_finite_gradients(bad):
    g = torch.ones(5000, device=DEV, dtype=torch.bfloat16)
    g[4321] = bad
    plan = q.GradPlan([g])
    before = g.clone()
    n, c = q.grad_norm(plan, 1.0)
    q.grad_scale(plan, c)
    torch.cuda.synchronize()
    assert not np.isfinite(n.item()) and np.isnan(c.item())
    assert torch.equal(g.view(torch.int16), before.view(torch.int16))


def test_repeats_bit_for_bit_with_a_dirty_workspace():
    g = H.grad((3_000_001,), torch.float32, DEV, 9, 9)
    plan = q.GradPlan([g, H.grad((77,), torch.bfloat16, DEV, 9, 10)])
    ws, got = plan.workspace(), []
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got.append(q.grad_norm(plan, 0.1, ws=ws))
    torch.cuda.synchronize()
    assert all(torch.equal(a[0], got[0][0]) and torch.equal(a[1], got[0][1]) for a in got)
