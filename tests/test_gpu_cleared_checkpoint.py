"""A checkpoint in cleared buffers stands for zeros, wherever it is read."""
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def cleared(rows, cols):
    ld, groups = -(-cols // 16) * 16, -(-rows // 32)
    return q.ActCheckpoint(rows, cols, data=torch.zeros(rows, ld, dtype=torch.uint8, device=DEV),
                           scale=torch.zeros(groups, ld, dtype=torch.uint8, device=DEV))


@pytest.mark.parametrize("dt", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("rows,cols", [(40, 100), (70, 600), (5000, 300)])
def test_zeros(dt, rows, cols):
    c = cleared(rows, cols)
    assert torch.all(q.act_read(c, dtype=dt) == 0) and torch.all(q.act_read(c, dtype=torch.float32) == 0)
    x = torch.randn(rows, cols, generator=torch.Generator().manual_seed(1)).to(dt).to(DEV)
    assert torch.all(q.weight_grad(x, c, torch.ones(cols, cols, device=DEV)) == 0)
    for act in ("silu", "gelu"):
        for y in q.gated_act_backward(c, cleared(rows, cols), x, recompute=True, act=act):
            assert torch.all(y == 0)
