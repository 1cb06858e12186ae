"""A list that is dropped while its call is pending on another stream."""
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


@pytest.mark.parametrize("given", [True, False])
def test_a_list_dropped_while_a_side_stream_uses_it(given):
    """The memory of its device copy is not given out before the call has
    run: norm and step are right although tensors of its size are made and
    written at once.  (Without the record the allocator would hand them that
    memory; the new tensors hold a copy of the same bytes, so that even then
    every read would stay in bounds.)"""
    n, count = 300, 40
    grads = [torch.full((n,), 0.5, device=DEV) for _ in range(count)]
    weights = [torch.ones(n, device=DEV) for _ in range(count)]
    states = [q.AdamWState(n, 32) for _ in range(count)]
    side = torch.cuda.Stream()
    q.grad_norm(q.GradPlan(grads))                # loads the kernels, which takes longer than a sleep
    q.adamw_step(q.AdamWPlan([(torch.ones(n, device=DEV), grads[0], q.AdamWState(n, 32), None, 1.0, 0.0)]), 1)
    torch.cuda.synchronize()
    side.wait_stream(torch.cuda.current_stream())
    plans = [q.GradPlan(grads), q.AdamWPlan([(w, g, s, None, 1.0, 0.0) for w, g, s in zip(weights, grads, states)])]
    copies = [p.dev.clone() for p in plans]
    at = [p.dev.data_ptr() for p in plans]
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)
        if not given:
            norm, coef = q.grad_norm(plans[0], 1.0)
            q.adamw_step(plans[1], 1, lr=0.1)
    if given:
        norm, coef = q.grad_norm(plans[0], 1.0, stream=side)
        q.adamw_step(plans[1], 1, lr=0.1, stream=side)
    del plans
    later = [c.clone() for c in copies for _ in range(8)]
    assert not side.query()                       # still asleep
    assert not {t.data_ptr() for t in later} & set(at)
    torch.cuda.synchronize()
    assert abs(norm.item() - 0.5 * (n * count) ** 0.5) < 1e-4
    for w in weights:
        assert torch.allclose(w, torch.full_like(w, 0.9), rtol=0, atol=1e-6)
