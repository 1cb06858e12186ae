"""Every operator that makes gradients reads its inputs on the stream that it is
given: they are written there behind a delay, over other values, so a launch on
another stream reads those."""
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
B = torch.bfloat16
ROWS, COLS, VOCAB = 300, 96, 50


def late(pairs, call):
    """call(stream) where each buffer of `pairs` gets its values on the stream,
    late."""
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(40_000_000)
        for buffer, value in pairs:
            buffer.copy_(value)
    out = call(side)
    side.synchronize()
    return out


def new(seed, *shape):
    return torch.randn(*shape, generator=torch.Generator().manual_seed(seed)).to(B).to(DEV)


def copies(*tensors):
    """(buffer that holds zeros, value) of each."""
    return [(torch.zeros_like(t), t) for t in tensors]


def checkpoint(x):
    c = q.act_pack(x)
    return c, copies(c.data, c.scale)


def same(got, want):
    assert all(torch.equal(a, b) for a, b in zip(got, want))
    # the values behind the delay differ from what was there before
    assert any(torch.any(w != 0) for w in want)


def test_pack_and_read():
    x = new(1, ROWS, COLS)
    want = q.act_pack(x)
    pairs = copies(x)
    got = late(pairs, lambda s: q.act_pack(pairs[0][0], stream=s))
    same([got.data, got.scale], [want.data, want.scale])
    value = q.act_read(want)
    kept = copies(want.data, want.scale)
    c = q.ActCheckpoint(ROWS, COLS, data=kept[0][0], scale=kept[1][0])
    same([late(kept, lambda s: q.act_read(c, stream=s))], [value])


def test_gated_activation():
    gate, up, dh = new(2, ROWS, COLS), new(3, ROWS, COLS), new(4, ROWS, COLS)
    h, g8, u8 = q.gated_act_forward(gate, up)
    pairs = copies(gate, up)
    got = late(pairs, lambda s: q.gated_act_forward(pairs[0][0], pairs[1][0], stream=s))
    same([got[0], got[1].data, got[2].data], [h, g8.data, u8.data])
    want = q.gated_act_backward(g8, u8, dh, recompute=True)
    pairs = copies(g8.data, g8.scale, u8.data, u8.scale, dh)
    g, u = (q.ActCheckpoint(ROWS, COLS, data=pairs[i][0], scale=pairs[i + 1][0]) for i in (0, 2))
    same(late(pairs, lambda s: q.gated_act_backward(g, u, pairs[4][0], recompute=True, stream=s)), want)


@pytest.mark.parametrize("rows", [60, 5000])     # without and with parts
@pytest.mark.parametrize("kept", [False, True])
def test_weight_grad(rows, kept):
    dy, x = new(5, rows, COLS), new(6, rows, COLS)
    arg = q.act_pack(x) if kept else x
    want = q.weight_grad(dy, arg, torch.empty(COLS, COLS, device=DEV))
    start = torch.full((COLS, COLS), 2.0, device=DEV)
    added = q.weight_grad(dy, arg, start.clone(), accumulate=True)
    pairs = copies(dy, start, *((arg.data, arg.scale) if kept else (x,)))
    src = q.ActCheckpoint(rows, COLS, data=pairs[2][0], scale=pairs[3][0]) if kept else pairs[2][0]
    out = torch.empty(COLS, COLS, device=DEV)
    same([late(pairs, lambda s: q.weight_grad(pairs[0][0], src, out, stream=s))], [want])
    for buffer, _ in pairs:
        buffer.zero_()
    same([late(pairs, lambda s: q.weight_grad(pairs[0][0], src, pairs[1][0], accumulate=True, stream=s))], [added])


@pytest.mark.parametrize("n", [40, ROWS])        # without and with parts
@pytest.mark.parametrize("acc", [False, True])
def test_embedding(n, acc):
    tok = torch.randint(0, 5, (n,), generator=torch.Generator().manual_seed(7)).to(DEV) + 3
    table, dy = new(8, VOCAB, COLS), new(9, n, COLS)
    want = q.embedding_lookup(tok, table)
    pairs = copies(tok, table)
    same([late(pairs, lambda s: q.embedding_lookup(pairs[0][0], pairs[1][0], stream=s))], [want])
    start = torch.full((VOCAB, COLS), 2.0, device=DEV)
    want = q.embedding_grad(tok, dy, start.clone(), accumulate=acc)
    pairs = copies(tok, dy, start)
    same([late(pairs, lambda s: q.embedding_grad(pairs[0][0], pairs[1][0], pairs[2][0], accumulate=acc, stream=s))], [want])
