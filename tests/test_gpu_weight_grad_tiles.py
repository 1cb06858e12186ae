"""The weight gradient on the GPU in tiles of 256 x 256: written by the tiles
themselves, in parts that are joined, and both in one launch; aligned panels and
panels at any address; both types, kept input, results of every type.

Whole numbers: every partial sum is below 2^24, so fp32 sums are exact, and a
result of up to 2^8 in bf16, 2^11 in f16 is rounded at most once."""
import pytest
import torch

import quantized_momentum_newton_amd as q

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, F = torch.bfloat16, torch.float16, torch.float32


def whole(gen, rows, cols, dt, extra=0):
    wide = torch.full((rows, cols + extra), float("nan"), dtype=dt, device=DEV)
    wide[:, :cols] = torch.randint(-2, 3, (rows, cols), generator=gen, device=DEV, dtype=torch.int32)
    return wide[:, :cols]


# (rows, n, k), and what the rule for tiles makes of them
SIZES = [
    (200, 4096, 4096),       # 256 tiles, one round, no parts
    (237, 4090, 4095),       # the same, panels at any address
    (400, 6145, 4097),       # a round and more, no parts, any address
    (5001, 2560, 2048),      # parts only
    (5001, 2559, 2047),      # parts only, any address
    (2000, 4096, 4352),      # a round of whole tiles, the rest in parts
    (2500, 4343, 4095),      # the same, any address
    (130, 4096, 4352),       # 128 tiles: two rounds and more, no parts
]


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("kept", [False, True])
@pytest.mark.parametrize("rows,n,k", SIZES)
def test_whole_numbers_in_large_tiles(rows, n, k, kept, dt):
    gen = torch.Generator(device=DEV).manual_seed(rows + n)
    odd = n % 8 != 0
    dy, x = whole(gen, rows, n, dt, 3 * odd), whole(gen, rows, k, dt, odd)
    want = dy.float().t() @ x.float()          # exact: below 2^24
    arg = q.act_pack(x) if kept else x
    for out_t, acc in ((F, False), (F, True), (B, False), (B, True), (H, True)):
        room = torch.full((n, k + 1 + odd), 3.0, dtype=out_t, device=DEV)
        out = room[:, :k] if odd else torch.full((n, k), 3.0, dtype=out_t, device=DEV)
        q.weight_grad(dy, arg, out, accumulate=acc)
        assert torch.equal(out, (want + 3 * acc).to(out_t)), (out_t, acc)
        assert torch.all(room[:, k:] == 3)


def test_a_layers_matrix():
    """Three rounds of whole tiles and half a round in parts, added to what is
    there, from kept input."""
    rows, n, k = 8192, 14336, 4096
    gen = torch.Generator(device=DEV).manual_seed(7)
    dy, x = whole(gen, rows, n, B), whole(gen, rows, k, B)
    want = dy.float().t() @ x.float()
    out = torch.full((n, k), 3.0, device=DEV)
    q.weight_grad(dy, q.act_pack(x), out, accumulate=True)
    assert torch.equal(out, want + 3)
    assert torch.equal(q.weight_grad(dy, x, out), want)


def test_a_dirty_workspace_changes_nothing():
    gen = torch.Generator(device=DEV).manual_seed(8)
    dy = torch.randn(2500, 4343, generator=gen, device=DEV).to(B)
    x = torch.randn(2500, 4095, generator=gen, device=DEV).to(B)
    out = torch.empty(4343, 4095, device=DEV)
    ws, got = q.weight_grad_workspace(dy, x, out), []
    assert ws.numel() > 0
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got.append(q.weight_grad(dy, x, torch.empty_like(out), ws=ws))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])


def test_f16_operands_past_the_largest():
    """Kept bytes of f16 numbers from 63488 on stand for 65536, which is an
    infinity in f16: in the product as in what act_read gives."""
    x = torch.ones(40, 24, dtype=H, device=DEV)
    x[3, 5], x[7, 6], x[9, 7], x[39, 8] = 65504.0, -63488.0, 63456.0, 61440.0
    c = q.act_pack(x)
    v = q.act_read(c, dtype=H)
    assert v[3, 5] == float("inf") and v[7, 6] == float("-inf") and v[9, 7] == 61440 and v[39, 8] == 61440
    assert q.act_read(c, dtype=F)[3, 5] == 65536
    dy = torch.zeros(40, 4, dtype=H, device=DEV)
    dy[3, 0], dy[7, 1], dy[9, 2], dy[39, 3] = 1, 1, 1, 1
    out = q.weight_grad(dy, c, torch.empty(4, 24, device=DEV))
    want = (dy.double().cpu()[:, :, None] * v.double().cpu()[:, None, :]).sum(0)
    assert torch.equal(out.cpu().isnan(), want.isnan())
    assert torch.equal(out.cpu().double().nan_to_num(nan=0.0), want.nan_to_num(nan=0.0))
