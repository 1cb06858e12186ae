"""Results in 16 bits are the fp32 results, rounded: not an exact product or
sum rounded once, which differs next to the borders of f16.  Bit for bit."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
@pytest.mark.parametrize("shape", ["whole tasks", "blocks", "rows", "short rows"])
def test_scaling_of_every_16_bit_number(dt, shape):
    """Every number of the type times 60 factors of all magnitudes, in whole
    tasks, single blocks and strided rows."""
    bits = torch.arange(65536, dtype=torch.int32).to(torch.int16).view(dt)
    x = bits[torch.isfinite(bits.float())]
    if shape == "blocks":
        x = x[:-1]                                       # ragged
    rng = np.random.default_rng(12)
    factors = [0.0018759474623948336, 1.0, 0.0, 2.0 ** -10, 3.0] + (np.exp2(rng.uniform(-9, 4, 55))).astype(np.float32).tolist()
    for c in factors:
        c = torch.tensor([c], dtype=torch.float32)
        if shape == "whole tasks":
            parts = [torch.cat([x, x.new_zeros(-x.numel() % 1024)]).to(DEV)]
        elif shape == "blocks":
            parts = [p.clone().to(DEV) for p in x.split(997)]
        else:
            cols = 1032 if shape == "rows" else 31
            n = x.numel() // cols * cols
            room = torch.zeros(n // cols, cols + 8, dtype=dt, device=DEV)
            room[:, :cols] = x[:n].view(-1, cols).to(DEV)
            parts = [room[:, :cols]]
        before = [p.cpu().clone() for p in parts]
        q.grad_scale(q.GradPlan(parts), c.to(DEV))
        torch.cuda.synchronize()
        for p, b in zip(parts, before):
            want = (b.float() * c).to(dt)
            got = p.cpu()
            bad = (got.contiguous().view(torch.int16) != want.contiguous().view(torch.int16)).nonzero()
            assert bad.numel() == 0, (c.item(), bad.shape[0], b[tuple(bad[0])], got[tuple(bad[0])], want[tuple(bad[0])])


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("dt", [torch.float16, torch.bfloat16])
def test_16_bit_weights_and_copies_are_the_fp32_weight_rounded(dt, bits, rounding):
    """The same step on fp32 weights that hold the 16-bit ones' values: its
    weights rounded are the 16-bit weights, and its copies, in both types."""
    n = (1 << 20) + 77
    g = torch.Generator(device=DEV)
    g.manual_seed(44)
    start = torch.randn(n, generator=g, device=DEV).to(dt)
    grad = torch.randn(n, generator=g, device=DEV)

    def step(weight, copy):
        c = torch.zeros(n, dtype=copy, device=DEV)
        q.adamw_step(q.AdamWPlan([(weight, grad, q.AdamWState(n, bits), c, 1.0, 0.1)]), 1, lr=1e-2, rounding=rounding, seed=1)
        torch.cuda.synchronize()
        return c

    for copy in (torch.float16, torch.bfloat16):
        say("16-bit weights", dt, bits, rounding, copy)
        wide, narrow = start.float(), start.clone()
        for c in (step(wide, copy), step(narrow, copy)):
            assert torch.equal(c, wide.to(copy))
        assert torch.equal(narrow, wide.to(dt))
