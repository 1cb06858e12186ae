"""Shapes of an AdamW list's tensors (no GPU): weight, gradient and copy are
taken element by element in row-major order, so their shapes have to agree on
it."""
import pytest
import torch

import quantized_momentum_newton_amd as q


def plan(weight, grad, copy=None):
    w, g = torch.zeros(weight), torch.zeros(grad)
    c = torch.zeros(copy, dtype=torch.bfloat16) if copy is not None else None
    return q.AdamWPlan([(w, g, q.AdamWState(w.numel(), device="cpu"), c, 1.0, 0.0)])


@pytest.mark.parametrize("weight,grad", [((4, 8), (8, 4)), ((2, 3, 4), (3, 2, 4)), ((6, 4), (3, 8)),
                                         ((4, 8), (2, 16))])
def test_other_orders_are_refused(weight, grad):
    with pytest.raises(ValueError, match="grad 0"):
        plan(weight, grad)
    with pytest.raises(ValueError, match="copy 0"):
        plan(weight, weight, grad)


@pytest.mark.parametrize("weight,grad", [((4, 8), (4, 8)), ((32,), (4, 8)), ((4, 8), (32,)), ((2, 3, 4), (2, 12)),
                                         ((2, 3, 4), (6, 4)), ((1, 8), (8,)), ((8, 1), (8,)), ((1,), ()), ((0, 5), (0,))])
def test_merged_dimensions_are_the_same_order(weight, grad):
    assert plan(weight, grad, weight).numels == [torch.zeros(weight).numel()]


def test_a_matrix_view_of_a_stack():
    w, wide = torch.zeros(5, 3, 4), torch.zeros(5, 20)
    q.AdamWPlan([(w, wide[:, :12], q.AdamWState(60, device="cpu"), None, 1.0, 0.0)])
    with pytest.raises(ValueError, match="grad 0"):
        q.AdamWPlan([(w, torch.zeros(12, 8)[:, :5], q.AdamWState(60, device="cpu"), None, 1.0, 0.0)])
