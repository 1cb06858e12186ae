"""Infinities and NaN through the gated activation on the GPU.

The forward pass is compared with the definition in 64 bits, element by
element; the backward pass with the definition at the kept values, where a
group of 32 rows of a column that holds a bad element is NaN as a whole: every
result that the definition makes NaN or infinite is that, and every other one
has the bits that it has without the bad elements."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from oracle import gradients as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
NAN, INF = float("nan"), float("inf")


def h64(t):
    return t.detach().cpu().double().numpy()


def check(got, want, clean, what):
    """want: the definition in 64 bits; clean: the result without bad elements."""
    g = h64(got)
    assert np.array_equal(np.isnan(g), np.isnan(want)), (what, "NaN")
    inf = np.isinf(want)
    assert np.array_equal(np.isinf(g), inf) and np.array_equal(g[inf], want[inf]), (what, "infinities")
    rest = torch.tensor(np.isfinite(want), device=DEV)
    assert torch.equal(got[rest], clean[rest]), what


def matrices(rows, cols, dt):
    gen = torch.Generator().manual_seed(rows + cols)
    new = lambda: torch.randn(rows, cols, generator=gen).clamp(-4, 4)
    # no zeros: 0 times an infinity is tested at places of its own
    gate, up, dh = (torch.where(x.abs() < 2.0 ** -6, torch.ones_like(x), x).to(dt).to(DEV) for x in (new(), new(), new()))
    return gate, up, dh


# rows behind a whole group, narrow patches, wide ones, a last patch of few columns
@pytest.mark.parametrize("rows,cols", [(3, 5), (70, 130), (70, 600), (33, 1025)])
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", TYPES)
def test_bad_elements_show_where_the_definition_has_them(dt, act, rows, cols):
    clean = matrices(rows, cols, dt)
    clean[1][1, 1] = 0                                # beside an infinite gate
    if cols > 8:
        clean[1][1, 10] = 0                           # beside an infinite dh
    gate, up, dh = (x.clone() for x in clean)
    gate[0, 0], gate[1, 1], gate[2, 2] = NAN, INF, -INF
    up[rows - 1, 3], up[0, 4] = NAN, INF
    gate[rows - 1, cols - 1] = NAN
    if cols > 8:
        up[rows - 1, cols - 2], up[0, cols - 3] = -INF, NAN
        gate[0, cols - 3] = -INF                      # both bad
        dh[0, 8], dh[rows - 1, 9], dh[1, 10] = NAN, INF, -INF

    with np.errstate(all="ignore"):
        a = O.act(h64(gate), act)[0]
        check(q.gated_act_forward(gate, up, act=act, keep=False)[0], a * h64(up),
              q.gated_act_forward(*clean[:2], act=act, keep=False)[0], "h")
        _, g8, u8 = q.gated_act_forward(gate, up, act=act)
        g, u, d = O.decode(*O.encode(h64(gate))), O.decode(*O.encode(h64(up))), h64(dh)
        a, slope = O.act(g, act)[:2]
        # the same call where bad elements are ordinary ones: other groups keep their bits
        _, cg8, cu8 = q.gated_act_forward(torch.where(gate.isfinite(), gate, clean[0]), torch.where(up.isfinite(), up, clean[1]), act=act)
        want = q.gated_act_backward(cg8, cu8, torch.where(dh.isfinite(), dh, clean[2]), recompute=True, act=act)
        got = q.gated_act_backward(g8, u8, dh, recompute=True, act=act)
        for x, w, c, what in zip(got, (d * u * slope, d * a, a * u), want, ("dgate", "dup", "h again")):
            check(x, w, c, what)


@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [NAN, INF, -INF])
def test_a_bad_gate_makes_its_group_nan(dt, act, bad):
    """One bad gate among 32 rows: the group's dgate, dup and h are NaN, and
    nothing else is."""
    gate, up, dh = matrices(96, 520, dt)
    gate[40, 515] = bad
    _, g8, u8 = q.gated_act_forward(gate, up, act=act)
    want = torch.zeros(96, 520, dtype=torch.bool, device=DEV)
    want[32:64, 515] = True
    for x in q.gated_act_backward(g8, u8, dh, recompute=True, act=act):
        assert torch.equal(x.isnan(), want)
        assert torch.all(x[~want].isfinite())
