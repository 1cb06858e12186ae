"""Strided gradients whose rows end inside a task, in every way the kernels
address them: AdamW's loads, the norm's and the scaling's loads and stores,
with what lies between two rows untouched.  Bounds as in tests/test_gpu_adamw.py
and tests/test_gpu_grad_norm.py."""
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from harness import inputs as H
from test_gpu_adamw import DEV, DTYPES, HP, Param
from test_gpu_grad_norm import TYPES, check

pytestmark = pytest.mark.gpu

# columns >= 1024 in multiples of 8 with row ends inside tasks, then rows shorter than a task, rows whose
# length is a multiple of 4 or of nothing
VIEWS = [(1032, 1040), (1288, 1300), (1536, 1544), (1544, 1551), (2056, 2100), (3000, 3007), (8, 9), (1016, 1019),
         (1028, 1030), (1001, 1003), (2047, 2048)]


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("cols,ld", VIEWS)
def test_adamw_views(cols, ld, bits, wdt):
    ps = [Param(rows * cols, bits, DTYPES[wdt], gdt, 2000 + cols + 13 * k, cols=cols, ld=ld)
          for k, (rows, gdt) in enumerate([(37, torch.bfloat16), (9, torch.float32), (5, torch.float16), (1, torch.float32)])]
    plan = q.AdamWPlan([p.tuple() for p in ps])
    say("adamw views", bits, wdt, cols, ld)
    q.adamw_step(plan, 3, **HP)
    torch.cuda.synchronize()
    for i, p in enumerate(ps):
        p.check(i, 3)


@pytest.mark.parametrize("cols,ld", VIEWS)
def test_norm_and_scaling_of_views(cols, ld):
    wide = [torch.full((41, ld), 5.0, dtype=dt, device=DEV) for dt in TYPES]
    grads = [w[:, :cols] for w in wide]
    for i, g in enumerate(grads):
        g.copy_(H.grad((41, cols), g.dtype, DEV, 80 + i, cols, std=0.3))
    check(grads, 0.2)
    for w in wide:
        assert torch.all(w[:, cols:] == 5.0)


@pytest.mark.parametrize("gap", [(1 << 28) - 8, 1 << 28, (1 << 28) + 8])
def test_rows_far_apart(gap):
    """Jumps below, at and above the limit of the 32-bit offsets, two rows that
    end inside a task."""
    cols, rows = 1288, 3
    say("rows", gap, "elements apart")
    room = torch.zeros((rows - 1) * (cols + gap) + cols, dtype=torch.float32, device=DEV)
    g = room.as_strided((rows, cols), (cols + gap, 1))
    g.copy_(H.grad((rows, cols), torch.float32, DEV, 91, 1, std=1e-2))
    nonzero = int(torch.count_nonzero(g))
    p = Param(rows * cols, 32, torch.float32, torch.float32, 92)
    p.grad = g
    p.snapshot()
    plan = q.AdamWPlan([p.tuple()])
    q.adamw_step(plan, 3, **HP)
    torch.cuda.synchronize()
    p.check(0, 3)
    check([g], 0.05)
    assert sum(int(torch.count_nonzero(c)) for c in room.split(1 << 28)) == nonzero
