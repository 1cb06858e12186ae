"""8-bit AdamW states at the ends of fp32's range and next to the borders of
their coding, in every form of the step: whole tasks and single blocks, fp32
and 16-bit weights, nearest and stochastic codes.  Codes and block maxima bit
for bit with the oracle; weights within the bounds of tests/test_gpu_adamw.py."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from harness import inputs as H
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


EDGES = ["zero", "tiny", "inf", "nan", "both", "spread", "large", "ordinary"]


def edge_block(kind):
    g = torch.zeros(256)
    if kind == "tiny":
        g[0], g[100] = 1e-31, 3e-32
    elif kind == "inf":
        g[17], g[18] = float("inf"), 1.0
    elif kind == "nan":
        g[255] = float("nan")
    elif kind == "both":
        g[0], g[1] = float("nan"), -float("inf")
    elif kind == "spread":
        g = torch.logspace(-20, 18, 256)
    elif kind == "large":
        g[:] = 3.0e38
    elif kind == "ordinary":
        g = torch.linspace(-1e-2, 1e-2, 256)
    return g


@pytest.mark.parametrize("rounding", ["nearest", "stochastic"])
@pytest.mark.parametrize("wdt", list(DTYPES))
def test_edge_blocks_in_every_form(wdt, rounding):
    """Each kind of block in each place of a whole task, and as a block of its
    own at the tensor's end: codes and maxima bit for bit over three steps,
    the ordinary blocks' weights as if they stood alone."""
    order = [EDGES[(t + b * (t % 3 + 1)) % 8] for t in range(24) for b in range(4)] + EDGES
    n = 256 * len(order) - 100                       # ends inside an ordinary block
    g = torch.cat([edge_block(k) for k in order])[:n]
    p = Param(n, 8, DTYPES[wdt], torch.float32, 1400, zero=True)
    alone = Param(n, 8, DTYPES[wdt], torch.float32, 1400, zero=True)
    p.grad.copy_(g)
    ordinary = torch.tensor([k == "ordinary" for k in order]).repeat_interleave(256)[:n]
    alone.grad.copy_(torch.where(ordinary, g, 0.0))
    p.snapshot()
    plans = [q.AdamWPlan([x.tuple()]) for x in (p, alone)]
    seed = (3 << 32) + 1
    for step in (1, 2, 3):
        say("edge blocks", wdt, rounding, "step", step)
        for plan in plans:
            q.adamw_step(plan, step, lr=2e-3, betas=(0.9, 0.99), eps=1e-8, rounding=rounding, seed=seed)
        torch.cuda.synchronize()
        word = A.words(n, seed, step, 0) if rounding == "stochastic" else None
        with np.errstate(all="ignore"):
            want = A.coded_states(p.h["m"], p.h["v"], p.h["m_absmax"], p.h["v_absmax"], p.h["g"], 0.9, 0.99, word)
        for k, x in zip(("m", "v", "m_absmax", "v_absmax"), want):
            got = getattr(p.state, k).cpu().numpy()
            assert np.array_equal(got, x, equal_nan=x.dtype.kind == "f"), (k, step)
        p.snapshot()
    w = p.weight.cpu()
    assert torch.equal(w[ordinary], alone.weight.cpu()[ordinary]) and torch.isfinite(w[ordinary].float()).all()
    poisoned = torch.tensor([k in ("inf", "nan", "both") for k in order]).repeat_interleave(256)[:n]
    assert torch.isnan(w[poisoned].float()).all()    # their states decode to NaN from the second step on


def test_codes_past_32_bit_offsets():
    """8-bit states of 2^32 + 300 elements: every code and maximum around 2^31
    and 2^32 against the oracle, whose random words count from the tensor's
    start."""
    n, seed, step = (1 << 32) + 300, 2, 5
    say("adamw codes past 2^32 elements")
    w = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    g = torch.zeros(n, dtype=torch.bfloat16, device=DEV)
    state = q.AdamWState(n, 8, DEV)
    spots = [slice(0, 512), slice((1 << 31) - 512, (1 << 31) + 512), slice((1 << 32) - 1024, n)]
    for k, s in enumerate(spots):
        g[s] = H.grad((s.stop - s.start,), torch.bfloat16, DEV, 610, k, std=1e-2)
    q.adamw_step(q.AdamWPlan([(w, g, state, None, 1.0, 0.1)]), step, lr=2e-3, betas=(0.9, 0.99), eps=1e-8,
                 rounding="stochastic", seed=seed)
    torch.cuda.synchronize()
    for s in spots:
        size = s.stop - s.start
        nb = -(-size // 256)
        zero = (np.zeros(size, np.int8), np.zeros(size, np.uint8), np.zeros(nb, np.float32), np.zeros(nb, np.float32))
        word = A.words(size, seed, step, 0, first=s.start)
        want = A.coded_states(*zero, g[s].float().cpu().numpy(), 0.9, 0.99, word)
        blocks = slice(s.start // 256, s.start // 256 + nb)
        for got, x in zip((state.m[s], state.v[s], state.m_absmax[blocks], state.v_absmax[blocks]), want):
            assert np.array_equal(got.cpu().numpy(), x), s
