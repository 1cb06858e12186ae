"""The order in which the embedding gradient adds a row's tokens, bit for bit."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"


def ordered_sum(tok, dy, vocab):
    """The sum in fp32 as it is defined: tokens sorted by value, equal ones by
    position; a row of up to 32 tokens one after the other; a longer one in parts
    that end where multiples of 32 positions of the order lie, the parts in
    eight contiguous shares, each added up in order, then the shares."""
    grad = np.zeros((vocab, dy.shape[1]), np.float32)
    order = np.argsort(tok, kind="stable")
    order = order[(tok[order] >= 0) & (tok[order] < vocab)]
    # padding sorts outside: positions of the order count the tokens inside
    values = tok[order]

    def add(rows):
        acc = np.zeros(dy.shape[1], np.float32)
        for r in rows:
            acc = acc + r
        return acc

    for v in np.unique(values):
        s, e = np.searchsorted(values, v), np.searchsorted(values, v, side="right")
        if e - s <= 32:
            grad[v] = add(dy[order[s:e]])
            continue
        cuts = [s] + list(range((s // 32 + 1) * 32, e, 32)) + [e]
        parts = [add(dy[order[a:b]]) for a, b in zip(cuts, cuts[1:])]
        each = -(-len(parts) // 8)
        grad[v] = add([add(parts[min(w * each, len(parts)):min((w + 1) * each, len(parts))]) for w in range(8)])
    return grad


@pytest.mark.parametrize("n,vocab,kind", [(31, 4, "few"), (64, 1, "one"), (1024, 3, "few"), (1025, 700, "spread"), (4096, 5, "few"),
                                          (5000, 2000, "skewed"), (3000, 300, "padded"), (40000, 7, "few"), (34000, 1, "one"),
                                          (33000, 5000, "skewed"), (6000, 64, "turns"), (6000, 9, "turns")])
def test_the_sum_has_its_order(n, vocab, kind):
    """Numbers of sizes far apart: any other order of a row's tokens gives other
    bits."""
    rng = np.random.default_rng(n + vocab)
    if kind == "few":
        tok = rng.integers(0, vocab, n)
    elif kind == "one":
        tok = np.full(n, vocab - 1)
    elif kind == "skewed":
        tok = (rng.random(n) ** 6 * vocab).astype(np.int64)
    elif kind == "turns":             # one value through neighbouring positions, then the next
        tok = np.arange(n) // 48 % vocab
    elif kind == "padded":
        tok = rng.integers(-2, vocab + 2, n)
    else:
        tok = rng.integers(0, vocab, n)
    dy = (rng.standard_normal((n, 8)) * 2.0 ** rng.integers(-12, 12, (n, 1))).astype(np.float32)
    want = ordered_sum(tok, dy, vocab)
    for dt in (np.int64, np.int32):
        got = q.embedding_grad(torch.tensor(tok.astype(dt), device=DEV), torch.tensor(dy, device=DEV), torch.full((vocab, 8), 9.0, device=DEV))
        assert np.array_equal(got.cpu().numpy().view(np.uint32), want.view(np.uint32))
