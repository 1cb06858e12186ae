"""Embedding gradient on the GPU: every pair of types in rows of every length,
against the oracle in 64 bits."""
import pytest
import torch

import quantized_momentum_newton_amd as q
from oracle import gradients as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("dt,gt", [(d, g) for d in TYPES for g in TYPES])
@pytest.mark.parametrize("cols,extra", [(257, 0), (513, 1), (1024, 0), (1031, 2), (2050, 0), (3001, 7)])
def test_rows_of_every_length_in_every_type(dt, gt, acc, cols, extra):
    """Empty rows, single tokens, rows of 32, 33 and many, in rows of the table
    that one and several units of columns take, at any address.  Whole numbers
    whose sums stay below 2^8 hold in 16 bits: bit for bit."""
    vocab = 60
    gen = torch.Generator().manual_seed(cols)
    counts = torch.zeros(vocab, dtype=torch.int64)
    counts[1], counts[2], counts[5], counts[6], counts[7], counts[30], counts[59] = 1, 2, 32, 33, 100, 64, 31
    tok = torch.repeat_interleave(torch.arange(vocab), counts)
    tok = torch.cat([tok, torch.tensor([-1, vocab])])[torch.randperm(len(tok) + 2, generator=gen)]
    dy = torch.randint(-1, 2, (len(tok), cols + extra), generator=gen).to(dt).to(DEV)[:, :cols]
    want = torch.tensor(O.embedding_grad(tok.numpy(), dy.float().cpu().numpy(), vocab, 2.0), device=DEV)
    assert want.abs().max() < 250
    room = torch.full((vocab, cols + extra + 1), 5.0, dtype=gt, device=DEV)
    grad = room[:, 1:1 + cols]
    q.embedding_grad(tok.to(DEV), dy, grad, 2.0, accumulate=acc)
    assert torch.equal(grad.double(), want + 5 * acc)
    assert torch.all(room[:, 0] == 5) and torch.all(room[:, 1 + cols:] == 5)
    # whole rows at aligned addresses
    grad = torch.full((vocab, cols), 5.0, dtype=gt, device=DEV)
    q.embedding_grad(tok.to(DEV), dy.contiguous(), grad, 2.0, accumulate=acc)
    assert torch.equal(grad.double(), want + 5 * acc)
