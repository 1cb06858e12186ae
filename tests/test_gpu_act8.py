"""Activations in 8 bits and the gated activation on the GPU against the
oracle in 64 bits.

Bytes and scales are defined by exact steps (a power of two, one rounding to
nearest even): bit for bit, as are the values in fp32 and bf16.  The gated
activation is fp32 arithmetic rounded once to its type.  Its sigmoid s(z):
exp(-z) is off by the rounding of its argument, |z| 2^-23 relative, and an ulp
each for exponential, sum and reciprocal, so s by (|z| + 4) 2^-23; four more
products: (|z| + 8) 2^-23 = K of h and dup.  The slope s + g s (1 - s) z' has
1 - s with the absolute error of s, so its error is K s (1 + |g| z').  Results
below the type's smallest normal number lose bits to its subnormals: half their
step, and exp(-z) past 2^126 ends the sigmoid at 0: |g u| 2^-126."""
import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from gpu_util import say
from oracle import gradients as O

pytestmark = pytest.mark.gpu
DEV = "cuda"
TYPES = [torch.float32, torch.bfloat16, torch.float16]
SUBNORMAL = {torch.float32: 2.0 ** -150, torch.bfloat16: 2.0 ** -134, torch.float16: 2.0 ** -25}


def h64(t):
    return t.detach().cpu().double().numpy()


def inputs(rows, cols, dt, seed, pitch=0, shift=0):
    """Columns of sizes from tiny to large, some zeros, in a buffer of 7s."""
    gen = torch.Generator().manual_seed(seed)
    size = torch.exp2(torch.randint(-12, 9, (cols,), generator=gen).float())
    x = torch.randn(rows, cols, generator=gen) * size * (torch.rand(rows, cols, generator=gen) > 0.05)
    pitch = pitch or cols
    room = torch.full((rows * pitch + shift + 8,), 7.0, dtype=dt, device=DEV)
    view = room[shift:shift + rows * pitch].view(rows, pitch)[:, :cols]
    view.copy_(x)
    return room, view


def check_codes(x, c, rows, cols):
    data, scale = O.encode(h64(x))
    got, got_scale = c.data.cpu().numpy()[:, :cols], c.scale.cpu().numpy()[:, :cols]
    assert np.array_equal(got_scale, scale)
    assert np.array_equal(got, data)
    return O.decode(data, scale)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols,pitch,shift", [
    (1, 1, 0, 0), (1, 130, 0, 1), (31, 127, 0, 0), (32, 128, 0, 0), (33, 129, 131, 3), (64, 8, 0, 0), (5, 1000, 1003, 1),
    (100, 512, 0, 0), (257, 264, 320, 0), (128, 4096, 0, 0)])
def test_bytes_scales_and_values(dt, rows, cols, pitch, shift):
    room, x = inputs(rows, cols, dt, rows * cols, pitch, shift)
    before = room.clone()
    c = q.ActCheckpoint(rows, cols, device=DEV)
    c.data.fill_(0xA5)
    q.act_pack(x, c)
    assert torch.equal(room, before)
    v = check_codes(x, c, rows, cols)
    for out_t in TYPES:
        wide = torch.full((rows, cols + 5), 3.0, dtype=out_t, device=DEV)
        q.act_read(c, wide[:, 2:2 + cols])
        want = torch.tensor(v, device=DEV).to(torch.float32).to(out_t)
        assert torch.equal(wide[:, 2:2 + cols], want)
        assert torch.all(wide[:, :2] == 3) and torch.all(wide[:, 2 + cols:] == 3)
    assert torch.equal(q.act_read(c).double(), torch.tensor(v, device=DEV))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("rows,cols,ld", [(33, 511, 512), (40, 512, 512), (40, 513, 528), (65, 700, 704), (100, 1025, 1152), (8, 516, 640),
                                          (130, 2047, 2048)])
def test_narrow_and_wide_patches_and_any_row_length(dt, rows, cols, ld):
    """Both ways over a matrix, rows of kept bytes on and off cache lines."""
    _, x = inputs(rows, cols, dt, rows + cols)
    groups = -(-rows // 32)
    c = q.ActCheckpoint(rows, cols, data=torch.zeros(rows, ld, dtype=torch.uint8, device=DEV),
                        scale=torch.zeros(groups, ld, dtype=torch.uint8, device=DEV))
    q.act_pack(x, c)
    v = torch.tensor(check_codes(x, c, rows, cols), device=DEV)
    for out_t in TYPES:
        assert torch.equal(q.act_read(c, dtype=out_t), v.to(torch.float32).to(out_t))
    up = x.flip(0).contiguous()
    h, g8, u8 = q.gated_act_forward(x, up, gate_ckpt=c)
    check_codes(up, u8, rows, cols)
    assert torch.equal(q.act_read(g8), v.to(torch.bfloat16))
    whole = q.gated_act_forward(x, up, keep=False)[0]
    assert torch.equal(h, whole)
    parts = torch.cat([q.gated_act_forward(x[:, k:k + 100], up[:, k:k + 100], keep=False)[0] for k in range(0, cols, 100)], 1)
    assert torch.equal(h, parts)
    wide = q.gated_act_backward(g8, u8, h, recompute=True)
    for k in range(0, cols, 100):
        part = [q.ActCheckpoint(rows, min(100, cols - k), device=DEV) for _ in range(2)]
        for p, s in zip(part, (x, up)):
            q.act_pack(s[:, k:k + 100], p)
        narrow = q.gated_act_backward(*part, h[:, k:k + 100], recompute=True)
        for a, b in zip(wide, narrow):
            assert torch.equal(a[:, k:k + 100], b)


def test_rows_behind_the_last_are_left_as_they_were():
    """A checkpoint inside larger buffers: only its rows are written."""
    data = torch.full((70, 64), 0x11, dtype=torch.uint8, device=DEV)
    scale = torch.full((4, 64), 0x22, dtype=torch.uint8, device=DEV)
    _, x = inputs(40, 50, torch.bfloat16, 3)
    q.act_pack(x, q.ActCheckpoint(40, 50, data=data[:40], scale=scale[:2]))
    assert torch.all(data[40:] == 0x11) and torch.all(scale[2:] == 0x22)
    assert torch.all(data[:40, 56:] == 0x11)


def test_ends_of_the_range():
    x = torch.zeros(64, 16, device=DEV)
    x[0, 0], x[1, 0], x[2, 0] = 448, 17, 19
    x[0, 1] = 2.0 ** 127 * 1.99
    x[0, 2] = 2.0 ** -140
    x[0, 3] = 448.0001
    x[40, 4] = -3.4e38
    x[:, 5] = torch.arange(64, device=DEV) * 2.0 ** -104      # subnormal codes at the lowest scale
    x[:, 6] = -0.0
    c = q.act_pack(x)
    check_codes(x, c, 64, 16)


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("bad", [float("nan"), float("inf"), float("-inf")])
def test_a_group_with_a_bad_element_is_nan_and_no_other(dt, bad):
    _, x = inputs(70, 40, dt, 4)
    x[35, 7] = bad
    x[69, 39] = bad
    v = q.act_read(q.act_pack(x), dtype=torch.float32)
    want = torch.zeros(70, 40, dtype=torch.bool, device=DEV)
    want[32:64, 7] = True
    want[64:, 39] = True
    assert torch.equal(v.isnan(), want)


def gate_inputs(rows, cols, dt, seed, fused):
    gen = torch.Generator().manual_seed(seed)
    # gates from far negative to far positive, a part of them next to the slope's zeros
    g = torch.randn(rows, cols, generator=gen) * 3
    g[::3] = torch.linspace(-30, 30, cols) if cols > 1 else -1.25
    u = torch.randn(rows, cols, generator=gen) * 2
    wide = torch.cat([g, u], 1).to(dt).to(DEV)
    return (wide[:, :cols], wide[:, cols:]) if fused else (wide[:, :cols].clone(), wide[:, cols:].clone())


def close(got, want, rel, what):
    """|got - want| within rel (an array of absolute bounds) and one rounding."""
    got = h64(got) if isinstance(got, torch.Tensor) else got
    off = np.abs(got - want) - rel
    assert np.all(np.isfinite(got)), what
    assert np.all(off <= 0), (what, float(off.max()), np.unravel_index(off.argmax(), off.shape))


@pytest.mark.parametrize("dt", TYPES)
@pytest.mark.parametrize("act", ["silu", "gelu"])
@pytest.mark.parametrize("rows,cols,fused", [(1, 1, False), (33, 130, True), (100, 512, True), (64, 257, False), (7, 1000, True)])
def test_gated_activation(dt, act, rows, cols, fused):
    gate, up = gate_inputs(rows, cols, dt, rows + cols, fused)
    h, g8, u8 = q.gated_act_forward(gate, up, act=act)
    g, u = h64(gate), h64(up)
    half = torch.finfo(dt).eps / 2

    def bounds(g, z):
        return (np.abs(z) + 8) * 2.0 ** -23

    value, _, s, z, _ = O.act(g, act)
    y = value * u
    tiny = SUBNORMAL[dt] + np.abs(g * u) * 2.0 ** -126
    close(h, y, (half + bounds(g, z)) * np.abs(y) + tiny, "h")
    g, u = check_codes(gate, g8, rows, cols), check_codes(up, u8, rows, cols)

    dh = (torch.randn(rows, cols, generator=torch.Generator().manual_seed(9)) * 0.1).to(dt).to(DEV)
    wide = torch.full((rows, 2 * cols + 3), 5.0, dtype=dt, device=DEV)
    dg, du, again = q.gated_act_backward(g8, u8, dh, wide[:, :cols], wide[:, cols:2 * cols], recompute=True, act=act)
    assert torch.all(wide[:, 2 * cols:] == 5)
    d = h64(dh)
    value, slope, s, z, dz = O.act(g, act)
    k = bounds(g, z)
    # every factor's size, for what underflows on the way
    tiny = SUBNORMAL[dt] + (np.abs(g) + 1) * (np.abs(u) + np.abs(d) + 1) ** 2 * 2.0 ** -125
    close(again, value * u, (half + k) * np.abs(value * u) + tiny, "h again")
    close(du, d * value, (half + k) * np.abs(d * value) + tiny, "dup")
    y = d * u * slope
    close(dg, y, half * np.abs(y) * (1 + k) + 2 * k * np.abs(d * u) * s * (1 + np.abs(g) * dz) + tiny, "dgate")
    two = q.gated_act_backward(g8, u8, dh, act=act)
    assert two[2] is None and torch.equal(two[0], dg) and torch.equal(two[1], du)


@pytest.mark.parametrize("act", ["silu", "gelu"])
def test_gradients_are_the_differences(act):
    """dgate and dup against central differences of the forward in fp32, at
    values that 8 bits hold exactly (an odd number of sixteenths below 2, where
    the largest of a column is 1.875).  The difference over 2^-6 is off by its
    third-order term, step^2 / 6 times the third derivative (below 1), and by
    fp32 roundings of h over the step: 2^-12 / 6 + 4 * 2^-24 * 2^6 < 1e-4."""
    rows, cols = 32, 30
    g = (torch.arange(rows * cols).view(rows, cols) % 15 + 1) / 8.0 * torch.where(torch.arange(cols) % 2 == 0, 1.0, -1.0)
    u = g.flip(0).contiguous().roll(1, 1)
    g[0], u[0] = 1.875, 1.875
    g, u, e = g.to(DEV), u.to(DEV), 2.0 ** -6
    _, g8, u8 = q.gated_act_forward(g, u, act=act)
    assert torch.equal(q.act_read(g8, dtype=torch.float32), g) and torch.equal(q.act_read(u8, dtype=torch.float32), u)
    dg, du, _ = q.gated_act_backward(g8, u8, torch.ones_like(g), act=act)
    f = lambda a, b: q.gated_act_forward(a, b, act=act, keep=False)[0]
    assert torch.allclose(dg, (f(g + e, u) - f(g - e, u)) / (2 * e), rtol=0, atol=2e-4)
    assert torch.allclose(du, (f(g, u + e) - f(g, u - e)) / (2 * e), rtol=0, atol=1e-4)


def test_large_gates():
    """Gates whose powers leave fp32's range: value 0 or g, slope 0 or 1."""
    g = torch.tensor([[3e38, -3e38, 1e20, -1e20, 200.0, -200.0, 90.0, -110.0]], device=DEV)
    u = torch.full_like(g, 0.5)
    for act in ("silu", "gelu"):
        h, g8, u8 = q.gated_act_forward(g, u, act=act)
        assert torch.allclose(h, g.clamp(min=0) * 0.5, rtol=1e-6, atol=1e-30)
        dg, du, _ = q.gated_act_backward(g8, u8, torch.ones_like(g), act=act)
        v = q.act_read(g8, dtype=torch.float32)
        assert torch.allclose(dg, (v > 0).float() * 0.5, rtol=1e-6, atol=1e-30), dg
        assert torch.allclose(du, v.clamp(min=0), rtol=1e-6, atol=1e-30)


def test_no_rows():
    x = torch.zeros(0, 20, device=DEV, dtype=torch.bfloat16)
    c = q.act_pack(x)
    assert q.act_read(c).shape == (0, 20)
    h, g8, u8 = q.gated_act_forward(x, x.clone())
    assert h.shape == (0, 20) and q.gated_act_backward(g8, u8, x)[0].shape == (0, 20)
    say("no rows: ok")
