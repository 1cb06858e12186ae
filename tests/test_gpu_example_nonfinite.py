"""The training example meets one batch whose gradients are not finite."""
import pytest
import torch

from test_example_cpu import load_example

pytestmark = pytest.mark.gpu


@pytest.mark.parametrize("name", ["up0", "head", "gain1"])
@pytest.mark.parametrize("bad", [float("inf"), float("nan")])
def test_a_bad_batch_leaves_weights_and_states_as_they_are(name, bad):
    """Wherever the infinity or NaN is: in a Muon matrix, in an 8-bit or in a
    32-bit AdamW tensor.  The step after it goes on."""
    mod = load_example()
    model = mod.Model("cuda")
    opt = mod.Optimizer(model)
    gen = torch.Generator(device="cuda")
    gen.manual_seed(3)
    live = [p.detach() for p in model.weights.values()] + [t for t in opt.muon_plan._keep[0::3] + opt.muon_plan._keep[1::3]]
    live += [t for s in opt.adamw_plan._keep if isinstance(s, mod.q.AdamWState) for t in s.tensors()]

    def batch():
        tokens = torch.randint(0, mod.VOCAB, (mod.BATCH,), generator=gen, device="cuda")
        for p in model.weights.values():
            p.grad.zero_()
        loss = model.loss(tokens, tokens.flip(0))
        loss.backward()
        return loss.item()

    batch()
    assert opt.step() is True
    batch()
    model.weights[name].grad.view(-1)[77] = bad
    before = [t.clone() for t in live]
    assert opt.step() is False and opt.steps == 1
    torch.cuda.synchronize()
    for a, b in zip(before, live):
        assert torch.equal(a, b)
    batch()
    assert opt.step() is True and opt.steps == 2
    torch.cuda.synchronize()
    assert all(torch.isfinite(t.float()).all() for t in live)
    assert not all(torch.equal(a, b) for a, b in zip(before, live))
