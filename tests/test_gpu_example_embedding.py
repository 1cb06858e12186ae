"""The example's embedding: its rows, and its gradient added to the table's
buffer, against torch's indexing in 64 bits.  Sums of at most 1024 fp32 numbers
are off by at most 1024 * 2^-24 of the sum of magnitudes."""
import importlib.util
import os

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_embedding_rows_and_gradient():
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    model = mod.Model("cuda")
    table = model.weights["embedding"]
    tokens = torch.randint(0, mod.VOCAB, (mod.BATCH,), generator=torch.Generator("cuda").manual_seed(1), device="cuda")
    r = torch.randn(mod.BATCH, mod.WIDTH, generator=torch.Generator("cuda").manual_seed(2), device="cuda")
    table.grad.fill_(0.25)
    x = mod.Embedding.apply(table, tokens)
    assert torch.equal(x, table.detach()[tokens])
    (x * r).sum().backward()
    exact = table.detach().double().requires_grad_()
    (exact[tokens] * r.double()).sum().backward()
    size = torch.zeros_like(exact).index_add_(0, tokens, r.double().abs()) + 0.25
    off = (table.grad.double() - 0.25 - exact.grad).abs()
    assert torch.all(off <= 1026 * 2.0 ** -24 * size)
    model.loss(tokens, tokens).backward()
    assert all(torch.isfinite(w.grad).all() and w.grad.abs().sum() > 0 for w in model.weights.values())
