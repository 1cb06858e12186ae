"""Embedding lookup on the GPU: tokens outside the table under any scale."""
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("scale", [-1.5, 0.0, float("inf"), float("-inf"), float("nan"), 1e30])
@pytest.mark.parametrize("tt", TYPES)
@pytest.mark.parametrize("ot", TYPES)
def test_padding_gives_zeros_whatever_the_scale(tt, ot, scale):
    """A token outside the table: a row of positive zeros."""
    table = torch.randn(20, 33, generator=torch.Generator().manual_seed(1)).to(tt).to(DEV)
    tok = torch.tensor([3, -1, 20, 7, -2 ** 40, 2 ** 40, 19], device=DEV)
    out = q.embedding_lookup(tok, table, scale, dtype=ot)
    inside = (tok >= 0) & (tok < 20)
    assert torch.all(out[~inside] == 0) and not torch.any(torch.signbit(out[~inside]))
    want = (table[tok[inside]].float() * torch.tensor(scale, device=DEV)).to(ot)
    assert torch.equal(out[inside].isnan(), want.isnan())
    assert torch.equal(out[inside].nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
