"""The weight gradient on the GPU against 64 bits.

With small whole numbers as inputs every partial sum is a whole number below
2^24, so fp32 sums are exact and the result is bit for bit: this covers every
place of every tile.  With real numbers each of the sums a result passes
through (a matrix instruction adds at least 8 products to the accumulator; the
parts of a split product; what is added to) is off by at most 2^-23 of the sum
of magnitudes: (rows / 8 + 64) 2^-23 times that, and one rounding."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say

pytestmark = pytest.mark.gpu
DEV = "cuda"
B, H, F = torch.bfloat16, torch.float16, torch.float32


def whole(gen, rows, cols, dt, pitch=0, shift=0):
    x = torch.randint(-2, 3, (rows, cols), generator=gen, device=DEV, dtype=torch.int32)
    pitch = pitch or cols
    room = torch.full((rows * pitch + shift + 16,), float("nan"), dtype=dt, device=DEV)
    view = room[shift:shift + rows * pitch].view(rows, pitch)[:, :cols]
    view.copy_(x)
    return view


def product(dy, x):
    """dy^T x exactly, on the CPU in 64 bits."""
    return torch.from_numpy(dy.cpu().double().numpy().T @ x.cpu().double().numpy())


SIZES = [(1, 1, 1), (1, 40, 24), (3, 17, 129), (31, 64, 64), (64, 128, 128), (65, 130, 257), (100, 300, 40), (129, 256, 256),
         (512, 8, 1000), (1000, 520, 264), (2049, 72, 96), (700, 1025, 511)]


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("rows,n,k", SIZES)
@pytest.mark.parametrize("kept", [True, False])
def test_whole_numbers_are_exact(dt, rows, n, k, kept):
    gen = torch.Generator(device=DEV).manual_seed(rows * n + k)
    dy, x = whole(gen, rows, n, dt), whole(gen, rows, k, dt)
    want = product(dy, x)
    arg = q.act_pack(x) if kept else x
    room = torch.full((n, k + 3), -1.0, device=DEV)
    out = q.weight_grad(dy, arg, room[:, 1:1 + k])
    assert torch.equal(out.cpu().double(), want)
    assert torch.all(room[:, :1] == -1) and torch.all(room[:, 1 + k:] == -1)
    q.weight_grad(dy, arg, out, accumulate=True)
    assert torch.equal(out.cpu().double(), 2 * want)


@pytest.mark.parametrize("rows,n,k,extra,shift", [(200, 96, 72, 31, 0), (200, 96, 72, 32, 1), (130, 33, 31, 0, 1),
                                                 (70, 264, 270, 28, 0), (513, 130, 136, 8, 8), (64, 1, 8, 1, 3)])
def test_any_pitch_and_alignment(rows, n, k, extra, shift):
    """Columns of wider buffers whose other elements are NaN, at any element."""
    gen = torch.Generator(device=DEV).manual_seed(extra + n)
    dy, x = whole(gen, rows, n, B, n + extra, shift), whole(gen, rows, k, B, k + extra, shift)
    want = product(dy, x)
    assert torch.equal(q.weight_grad(dy, x, torch.empty(n, k, device=DEV)).cpu().double(), want)
    kept = q.act_pack(x)
    assert torch.equal(q.weight_grad(dy, kept, torch.empty(n, k, device=DEV)).cpu().double(), want)


@pytest.mark.parametrize("rows,n,k", [(4096, 128, 256), (8192, 512, 768), (5000, 2560, 2048), (64, 4096, 4352), (100000, 40, 24)])
def test_larger(rows, n, k):
    """Split over the rows and whole, several rounds of tiles."""
    gen = torch.Generator(device=DEV).manual_seed(rows)
    dy, x = whole(gen, rows, n, B), whole(gen, rows, k, B)
    want = (dy.float().t() @ x.float()).double()      # exact as well
    for arg in (x, q.act_pack(x)):
        assert torch.equal(q.weight_grad(dy, arg, torch.empty(n, k, device=DEV)).double(), want)


@pytest.mark.parametrize("acc", [False, True])
@pytest.mark.parametrize("rows,n,k", [(2, 257, 129), (1, 1000, 400), (66, 129, 513), (6000, 2047, 1001), (4096, 1001, 130), (40000, 129, 255),
                                      (3000, 2049, 1283), (9000, 511, 3001), (5001, 7, 1300)])
def test_last_panels_that_start_early(rows, n, k, acc):
    """Sides that are no multiple of a tile, at odd addresses, whole and split:
    overlapping tiles add what they share once, to f32 and to 16-bit results in
    rows of any pitch."""
    gen = torch.Generator(device=DEV).manual_seed(rows + k)
    dy, x = whole(gen, rows, n, B, n + 3, 1), whole(gen, rows, k, B)
    want = (dy.float().t() @ x.float()).double()      # exact as well
    kept = q.act_pack(x)
    for arg in (x, kept):
        for extra in (0, 1):
            room = torch.full((n, k + extra), 3.0, device=DEV)
            out = q.weight_grad(dy, arg, room[:, :k], accumulate=acc)
            assert torch.equal(out.double(), want + 3 * acc)
            assert torch.all(room[:, k:] == 3)
        out = q.weight_grad(dy, arg, torch.full((n, k), 3.0, dtype=B, device=DEV), accumulate=acc)
        assert torch.equal(out, (want + 3 * acc).float().to(B))


@pytest.mark.parametrize("dt", [B, H])
@pytest.mark.parametrize("out_t", [F, B, H])
@pytest.mark.parametrize("rows,n,k,kept", [(500, 136, 264, True), (500, 136, 264, False), (3000, 64, 50, True), (77, 70, 33, False)])
def test_real_numbers(dt, out_t, rows, n, k, kept):
    gen = torch.Generator(device=DEV).manual_seed(rows + n)
    dy = (torch.randn(rows, n, generator=gen, device=DEV) * 0.1).to(dt)
    x = (torch.randn(rows, k, generator=gen, device=DEV) * torch.exp(torch.randn(k, generator=gen, device=DEV))).to(dt)
    start = torch.randn(n, k, generator=gen, device=DEV).to(out_t)
    arg = q.act_pack(x) if kept else x
    if kept:
        x = q.act_read(arg, dtype=dt)
    exact = product(dy, x).numpy()
    size = product(dy.abs(), x.abs()).numpy()
    for acc in (False, True):
        out = start.clone()
        q.weight_grad(dy, arg, out, accumulate=acc)
        want = exact + (start.cpu().double().numpy() if acc else 0)
        bound = (rows / 8 + 64) * 2.0 ** -23 * (size + np.abs(want)) + torch.finfo(out_t).eps / 2 * np.abs(want)
        off = np.abs(out.cpu().double().numpy() - want)
        assert np.all(off <= bound * (1 + 1e-6)), float((off - bound).max())


def test_f16_takes_kept_values_rounded():
    """Values that f16 does not hold: small ones at its subnormals."""
    x = torch.full((32, 16), 2.0 ** -20, device=DEV)
    x[0] = 17 * 2.0 ** -24
    x[1] = 1.5 * 2.0 ** -24          # kept exactly (a power of two times 1.5), half a step in f16
    c = q.act_pack(x)
    v = q.act_read(c, dtype=torch.float16)
    dy = torch.zeros(32, 8, dtype=H, device=DEV)
    for r in range(8):
        dy[r, r] = 1
    out = q.weight_grad(dy, c, torch.empty(8, 16, device=DEV))
    assert torch.equal(out, v[:8].float())


def test_no_rows():
    dy, x = torch.zeros(0, 20, dtype=B, device=DEV), torch.zeros(0, 24, dtype=B, device=DEV)
    out = torch.ones(20, 24, device=DEV)
    q.weight_grad(dy, x, out, accumulate=True)
    assert torch.all(out == 1)
    q.weight_grad(dy, x, out)
    assert torch.all(out == 0)
    out.fill_(1)
    q.weight_grad(dy, q.act_pack(x), out)
    assert torch.all(out == 0)


def test_bad_elements_reach_their_row_and_column_only():
    gen = torch.Generator(device=DEV).manual_seed(1)
    dy, x = whole(gen, 100, 140, B), whole(gen, 100, 150, B)
    dy[50, 33] = float("nan")
    x[70, 149] = float("nan")
    for arg in (x, q.act_pack(x)):
        out = q.weight_grad(dy, arg, torch.empty(140, 150, device=DEV))
        want = torch.zeros(140, 150, dtype=torch.bool, device=DEV)
        want[33] = True
        want[:, 149] = True
        assert torch.equal(out.isnan(), want)


def test_repeats_bit_for_bit_with_a_dirty_workspace():
    gen = torch.Generator(device=DEV).manual_seed(2)
    dy = torch.randn(6000, 200, generator=gen, device=DEV).to(B)
    x = q.act_pack(torch.randn(6000, 300, generator=gen, device=DEV).to(B))
    out = torch.empty(200, 300, device=DEV)
    ws, got = q.weight_grad_workspace(dy, x, out), []
    assert ws.numel() > 0
    for fill in (0, 255, 127):
        ws.fill_(fill)
        got.append(q.weight_grad(dy, x, torch.empty_like(out), ws=ws))
    assert torch.equal(got[0], got[1]) and torch.equal(got[0], got[2])
    say("dirty workspace: ok")
