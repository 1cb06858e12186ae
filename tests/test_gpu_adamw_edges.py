"""8-bit AdamW states at the ends of fp32's range and next to the borders of
their coding, in every form of the step: whole tasks and single blocks, fp32
and 16-bit weights, nearest and stochastic codes.  Codes and block maxima bit
for bit with the oracle; weights within the bounds of tests/test_gpu_adamw.py."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from oracle import adamw as A
from test_adamw_borders_cpu import border_gradients
from test_gpu_adamw import DEV, DTYPES, Param

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("wdt", list(DTYPES))
@pytest.mark.parametrize("beta1", [0.9, 0.995, 0.999])
def test_largest_finite_maxima(beta1, wdt, rounding):
    """Blocks of m whose 128th code would lie past fp32's largest number
    (beta1 above 127/128), next to ordinary ones and to both sides of that
    border."""
    top = float(np.finfo(np.float32).max)
    border = top * 127 / (128 * beta1)
    p = Param(3 * 1024 + 257, 8, DTYPES[wdt], torch.float32, 1200)
    absmax = [3.4e38, top, 1e-2, min(border * (1 - 2.0 ** -20), top), min(border * (1 + 2.0 ** -20), top), 3.0e38,
              1e-2, 1e-2, 1e-2, 1e-2, 1e-2, 3.4e38, top, 3.4e38]
    p.state.m_absmax.copy_(torch.tensor(absmax))
    p.grad[:1024] = 0
    p.snapshot()
    plan = q.AdamWPlan([p.tuple()])
    hp = dict(lr=1e-37, betas=(beta1, 0.99), eps=1.0)
    for step in (1, 2):
        say("largest maxima", beta1, wdt, rounding, "step", step)
        q.adamw_step(plan, step, **hp, rounding=rounding, seed=21)
        torch.cuda.synchronize()
        p.check(0, step, rounding=rounding, seed=21, hp=hp)
        assert torch.isfinite(p.state.m_absmax).all()
        p.snapshot()


@pytest.mark.parametrize("wdt", ["f32", "bf16"])
def test_stochastic_codes_of_m_on_both_sides_of_their_borders(wdt):
    """Every element's m one fp32 step below, on, or one above the border that
    its random number sets."""
    n, seed, step = 256 * 4 * 50 + 3 * 256 + 77, (9 << 32) + 5, 3
    word = A.words(n, seed, step, 0)
    g, want = border_gradients(word)
    p = Param(n, 8, DTYPES[wdt], torch.float32, 1300, zero=True)
    p.grad.copy_(torch.from_numpy(g))
    plan = q.AdamWPlan([p.tuple()])
    q.adamw_step(plan, step, lr=1e-3, betas=(0.0, 0.9), eps=1e-8, rounding="stochastic", seed=seed)
    torch.cuda.synchronize()
    got = p.state.m.cpu().numpy()
    bad = np.nonzero(got != want)[0]
    assert bad.size == 0, (bad[:5], got[bad[:5]], want[bad[:5]], g[bad[:5]])
