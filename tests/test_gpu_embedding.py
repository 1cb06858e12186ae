"""Embedding lookup and gradient on the GPU against the oracle in 64 bits.

The lookup is one fp32 product rounded to its type, bit for bit.  The gradient
of small whole numbers is exact (every partial sum is); of real numbers each
addition is off by at most 2^-24 of the sum of magnitudes so far: with n tokens
in a row (n + 2) 2^-24 times that sum, and one rounding."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from oracle import gradients as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]


def tokens(kind, n, vocab, seed, dt=torch.int64):
    gen = torch.Generator().manual_seed(seed)
    if kind == "spread":
        t = torch.randint(0, vocab, (n,), generator=gen)
    elif kind == "one":
        t = torch.full((n,), vocab - 1)
    elif kind == "few":                     # long rows next to one another
        t = torch.randint(0, min(3, vocab), (n,), generator=gen)
    elif kind == "skewed":
        t = (torch.rand(n, generator=gen) ** 6 * vocab).long()
    else:                                   # padding: outside on both sides
        t = torch.randint(-2, vocab + 2, (n,), generator=gen)
        if dt == torch.int64 and n > 3:
            t[1], t[2] = 2 ** 32, -2 ** 63
    return t.to(dt).to(DEV)


@pytest.mark.parametrize("tt", TYPES)
@pytest.mark.parametrize("ot", TYPES)
@pytest.mark.parametrize("n,vocab,cols,pitch", [(1, 1, 1, 0), (7, 10, 8, 0), (100, 50, 33, 40), (64, 300, 520, 0), (3, 20, 2049, 2050)])
def test_lookup(tt, ot, n, vocab, cols, pitch):
    wide = torch.randn(vocab, pitch or cols, generator=torch.Generator().manual_seed(n)).to(tt).to(DEV)
    table = wide[:, :cols]
    tok = tokens("padded", n, vocab, n, torch.int32)
    room = torch.full((n, cols + 2), 9.0, dtype=ot, device=DEV)
    q.embedding_lookup(tok, table, 1.7, out=room[:, 1:1 + cols])
    inside = (tok >= 0) & (tok < vocab)
    want = (table[tok.clamp(0, vocab - 1).long()].float() * torch.tensor(1.7, device=DEV)).to(ot)
    want[~inside] = 0
    assert torch.equal(room[:, 1:1 + cols], want)
    assert torch.all(room[:, 0] == 9) and torch.all(room[:, 1 + cols] == 9)


def test_tokens_of_any_shape_and_types_of_the_result():
    table = torch.randn(9, 12, device=DEV)
    tok = tokens("spread", 24, 9, 1).view(2, 3, 4)
    assert torch.equal(q.embedding_lookup(tok, table), table[tok.view(-1)])
    assert q.embedding_lookup(tok, table, dtype=torch.bfloat16).dtype == torch.bfloat16
    assert q.embedding_lookup(tok[:0], table).shape == (0, 12)


@pytest.mark.parametrize("kind", ["spread", "one", "few", "skewed", "padded"])
@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (5, 3, 40), (64, 7, 64), (65, 7, 100), (129, 2000, 129), (1000, 40, 256),
                                          (3000, 300, 513), (5000, 70000, 24), (20000, 600, 72), (700, 300000, 8)])
def test_whole_numbers_are_exact(kind, n, vocab, cols):
    dt = torch.int32 if n % 2 else torch.int64
    tok = tokens(kind, n, vocab, n + cols, dt)
    gen = torch.Generator(device=DEV).manual_seed(n)
    dy = torch.randint(-3, 4, (n, cols), generator=gen, device=DEV).to(torch.bfloat16)
    want = torch.tensor(O.embedding_grad(tok.cpu().numpy(), dy.float().cpu().numpy(), vocab, 2.0), device=DEV)
    room = torch.full((vocab, cols + 2), 9.0, device=DEV)
    grad = room[:, 1:1 + cols]
    q.embedding_grad(tok, dy, grad, 2.0)
    assert torch.equal(grad.double(), want)
    q.embedding_grad(tok, dy, grad, 2.0, accumulate=True)
    assert torch.equal(grad.double(), 2 * want)
    assert torch.all(room[:, 0] == 9) and torch.all(room[:, 1 + cols] == 9)


@pytest.mark.parametrize("kind", ["spread", "few", "padded"])
@pytest.mark.parametrize("n,vocab,cols,dt", [(32768, 500, 24, torch.int64), (32769, 500, 24, torch.int32), (70000, 900, 40, torch.int64),
                                             (140000, 50000, 16, torch.int32)])
def test_more_tokens_than_a_wave_holds(kind, n, vocab, cols, dt):
    """Up to 32768 tokens stay in registers between the two looks at them."""
    tok = tokens(kind, n, vocab, n, dt)
    dy = torch.randint(-3, 4, (n, cols), generator=torch.Generator(device=DEV).manual_seed(n), device=DEV).to(torch.bfloat16)
    want = torch.tensor(O.embedding_grad(tok.cpu().numpy(), dy.float().cpu().numpy(), vocab, 1.0), device=DEV)
    assert torch.equal(q.embedding_grad(tok, dy, torch.empty(vocab, cols, device=DEV)).double(), want)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("gt", TYPES)
@pytest.mark.parametrize("acc", [False, True])
def test_real_numbers(dt, gt, acc):
    n, vocab, cols, scale = 900, 200, 70, 0.3
    tok = tokens("skewed", n, vocab, 5)
    dy = torch.randn(n, cols, generator=torch.Generator().manual_seed(6)).to(dt).to(DEV)
    start = torch.randn(vocab, cols, generator=torch.Generator().manual_seed(7)).to(gt).to(DEV)
    t, d = tok.cpu().numpy(), dy.double().cpu().numpy()
    want = O.embedding_grad(t, d, vocab, np.float32(scale)) + (start.double().cpu().numpy() if acc else 0)
    size = O.embedding_grad(t, np.abs(d), vocab, scale) + (np.abs(start.double().cpu().numpy()) if acc else 0)
    count = np.bincount(t, minlength=vocab)[:, None]
    grad = start.clone()
    q.embedding_grad(tok, dy, grad, scale, accumulate=acc)
    bound = (count + 2) * 2.0 ** -24 * size * (1 + 1e-6) + torch.finfo(gt).eps / 2 * np.abs(want) * (1 + 2.0 ** -20)
    bound += {torch.float16: 2.0 ** -25}.get(gt, 0)
    off = np.abs(grad.double().cpu().numpy() - want)
    assert np.all(off <= bound), float((off - bound).max())
    if acc:      # rows without tokens keep their bits
        rest = torch.tensor(count[:, 0] == 0, device=DEV)
        assert torch.equal(grad[rest], start[rest])


def test_the_gradient_is_the_lookups():
    """<dy, lookup(T)> = <grad, T> for whole numbers: exact."""
    tok = tokens("padded", 500, 40, 8)
    table = torch.randint(-3, 4, (40, 16), device=DEV).float()
    dy = torch.randint(-3, 4, (500, 16), device=DEV).float()
    out = q.embedding_lookup(tok, table, 2.0)
    grad = q.embedding_grad(tok, dy, torch.empty_like(table), 2.0)
    assert (out * dy).double().sum().item() == (grad * table).double().sum().item()


def test_no_tokens():
    tok, dy = torch.zeros(0, dtype=torch.int64, device=DEV), torch.zeros(0, 24, device=DEV)
    grad = torch.ones(30, 24, device=DEV)
    q.embedding_grad(tok, dy, grad, accumulate=True)
    assert torch.all(grad == 1)
    q.embedding_grad(tok, dy, grad)
    assert torch.all(grad == 0)


def test_nan_stays_in_its_row():
    tok = tokens("skewed", 2000, 50, 9)
    dy = torch.ones(2000, 40, dtype=torch.bfloat16, device=DEV)
    dy[1234, 5] = float("nan")
    grad = q.embedding_grad(tok, dy, torch.empty(50, 40, device=DEV))
    want = torch.zeros(50, 40, dtype=torch.bool, device=DEV)
    want[tok[1234], 5] = True
    assert torch.equal(grad.isnan(), want)


def test_repeats_bit_for_bit_with_a_dirty_workspace():
    tok = tokens("skewed", 30000, 5000, 10)
    dy = torch.randn(30000, 300, device=DEV).to(torch.bfloat16)
    grad = torch.empty(5000, 300, device=DEV)
    ws, got = q.embedding_grad_workspace(tok, dy, grad), []
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got.append(q.embedding_grad(tok, dy, torch.empty_like(grad), 0.1, ws=ws))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    say("dirty workspace: ok")
