"""Activations in 8 bits, weight gradients, gated activations and embeddings
without a GPU: the oracle's pins and every refusal before a launch."""
import ctypes

import numpy as np
import pytest
import torch

import quantized_momentum_newton_amd as q
from oracle import gradients as O
from quantized_momentum_newton_amd import _lib as L

LIB = q._LIB
BASE = 0x7f0000000000     # fake device addresses: only alignment and overlap are looked at
ARG, ALIGN, DTYPE, SHAPE, WORKSPACE, UNSUPPORTED = 1, 2, 3, 4, 5, 7


# ------------------------------------------------------------------ oracle

def test_bytes_are_the_e4m3_format():
    want = torch.arange(256, dtype=torch.uint8).view(torch.float8_e4m3fn).double().numpy()
    assert np.array_equal(O.e4m3_values(), want, equal_nan=True)


@pytest.mark.parametrize("rows", [1, 31, 32, 33, 70])
def test_codes_are_the_nearest_and_the_scale_the_smallest(rows):
    rng = np.random.default_rng(rows)
    x = rng.standard_normal((rows, 9)) * 10.0 ** rng.integers(-9, 9, 9)
    x[:, 3] = 0
    data, scale = O.encode(x)
    v, table = O.decode(data, scale), O.e4m3_values()
    for g in range(scale.shape[0]):
        part, unit = x[32 * g:32 * g + 32], 2.0 ** (scale[g].astype(float) - 127)
        top = np.abs(part).max(0)
        assert np.all(top <= 448 * unit)
        assert np.all((top > 224 * unit) | (scale[g] == O.LOW + 127))
        for r in range(part.shape[0]):
            for c in range(9):
                err = abs(v[32 * g + r, c] - part[r, c])
                assert err <= np.nanmin(np.abs(table * unit[c] - part[r, c]))
                assert err <= max(abs(part[r, c]) / 16, 2.0 ** -10 * unit[c])     # what the header states


def test_ties_go_to_the_even_byte_and_ends_of_the_range():
    x = np.zeros((32, 4))
    x[0, 0], x[1, 0], x[2, 0] = 448, 17, 19        # 17 between 16 and 18, 19 between 18 and 20
    x[0, 1] = 2.0 ** 127 * 1.99                    # its exponent would be 120: 448 * 2^119 is what is kept
    x[0, 2] = 2.0 ** -140
    x[0, 3] = 448.0001
    data, scale = O.encode(x)
    v = O.decode(data, scale)
    assert v[1, 0] == 16 and v[2, 0] == 20
    assert v[0, 1] == 448 * 2.0 ** 119
    assert v[0, 2] == 0 and scale[0, 2] == 32
    assert scale[0, 3] == 128


def test_activations_and_their_slopes():
    g = np.linspace(-12, 12, 241)
    silu = torch.nn.functional.silu(torch.tensor(g)).numpy()
    gelu = torch.nn.functional.gelu(torch.tensor(g), approximate="tanh").numpy()
    assert np.allclose(O.act(g, "silu")[0], silu, rtol=1e-12, atol=1e-300)
    assert np.allclose(O.act(g, "gelu")[0], gelu, rtol=1e-9, atol=1e-14)
    for kind in ("silu", "gelu"):
        h = 1e-6
        diff = (O.act(g + h, kind)[0] - O.act(g - h, kind)[0]) / (2 * h)
        assert np.allclose(O.act(g, kind)[1], diff, rtol=1e-7, atol=1e-9)


def test_embedding_gradient_is_the_lookups():
    """<dy, lookup(table)> = <grad, table> for any table."""
    rng = np.random.default_rng(1)
    tokens = np.array([3, 0, 3, -1, 9, 3, 12])
    table, dy = rng.standard_normal((10, 5)), rng.standard_normal((7, 5))
    a = (O.embedding_lookup(tokens, table, 1.7) * dy).sum()
    assert np.isclose(a, (O.embedding_grad(tokens, dy, 10, 1.7) * table).sum(), rtol=1e-13)


# --------------------------------------------------------- refusals, C ABI

def kept(rows=64, cols=40, ld=48, data=BASE, scale=BASE + (1 << 30)):
    return L.Act8(data, scale, rows, cols, ld)


X = BASE + (2 << 30)
Y = BASE + (3 << 30)
Z = BASE + (4 << 30)


def pack(x=X, dtype=L.QM_BF16, ld=40, k=None):
    return LIB.act_pack(x, dtype, ld, kept() if k is None else k, None)


@pytest.mark.parametrize("status,call", [
    (ARG, lambda: LIB.act_pack(X, 1, 40, None, None)),
    (ARG, lambda: pack(x=None)),
    (ARG, lambda: pack(k=kept(data=None))),
    (ARG, lambda: pack(k=kept(scale=None))),
    (ARG, lambda: pack(x=BASE + 64)),                          # inside the data
    (ARG, lambda: pack(k=kept(scale=BASE + 64 * 48 - 16))),     # scales inside the data
    (ALIGN, lambda: pack(x=X + 1)),
    (ALIGN, lambda: pack(x=X + 2, dtype=0)),
    (ALIGN, lambda: pack(k=kept(data=BASE + 8))),
    (ALIGN, lambda: pack(k=kept(scale=Z + 8))),
    (DTYPE, lambda: pack(dtype=3)),
    (SHAPE, lambda: pack(ld=39)),
    (SHAPE, lambda: pack(ld=1 << 24)),
    (SHAPE, lambda: pack(k=kept(ld=40))),
    (SHAPE, lambda: pack(k=kept(ld=32))),
    (SHAPE, lambda: pack(k=kept(rows=-1))),
    (SHAPE, lambda: pack(k=kept(cols=-1))),
    (SHAPE, lambda: pack(k=kept(rows=1 << 31))),
    (UNSUPPORTED, lambda: pack(ld=128, k=kept(rows=(1 << 30) + 64, cols=128, ld=128, scale=BASE + (1 << 40)), x=BASE + (1 << 42))),
    (ARG, lambda: LIB.act_read(kept(), BASE + 32, 1, 40, None)),
    (ARG, lambda: LIB.act_read(kept(), None, 1, 40, None)),
    (ARG, lambda: LIB.act_read(None, X, 1, 40, None)),
    (DTYPE, lambda: LIB.act_read(kept(), X, -1, 40, None)),
])
def test_pack_and_read_refuse(status, call):
    assert call() == status
    assert LIB.qm_last_error()


def weight(dy=X, dtype=1, ld_dy=64, x=Y, ld_x=40, k8=None, rows=64, n=64, k=40, out=Z, out_dtype=0, ld_out=40, acc=1,
           ws=None, nws=0):
    return LIB.weight_grad(dy, dtype, ld_dy, x, ld_x, k8, rows, n, k, out, out_dtype, ld_out, acc, ws, nws, None)


@pytest.mark.parametrize("status,call", [
    (DTYPE, lambda: weight(dtype=0)),
    (DTYPE, lambda: weight(out_dtype=5)),
    (ARG, lambda: weight(x=None)),
    (ARG, lambda: weight(k8=kept())),                           # x and kept
    (ARG, lambda: weight(dy=None)),
    (ARG, lambda: weight(out=None)),
    (ARG, lambda: weight(acc=2)),
    (ARG, lambda: weight(out=X + 64)),
    (ARG, lambda: weight(out=Y + 64)),
    (SHAPE, lambda: weight(ld_dy=63)),
    (SHAPE, lambda: weight(ld_x=39)),
    (SHAPE, lambda: weight(ld_out=39)),
    (SHAPE, lambda: weight(x=None, k8=kept(cols=41))),
    (SHAPE, lambda: weight(x=None, k8=kept(rows=63))),
    (SHAPE, lambda: weight(rows=-1)),
    (SHAPE, lambda: weight(rows=1 << 30)),
    (ALIGN, lambda: weight(dy=X + 1)),
    (ALIGN, lambda: weight(out=Z + 2)),
    (WORKSPACE, lambda: weight(rows=4096)),
    (WORKSPACE, lambda: weight(rows=4096, ws=BASE, nws=LIB.weight_grad_workspace_bytes(4096, 64, 40) - 1)),
    (ALIGN, lambda: weight(rows=4096, ws=BASE + 8, nws=1 << 30)),
    (ARG, lambda: weight(rows=4096, ws=X + 4096, nws=1 << 30)),
    (SHAPE, lambda: weight(ld_out=1 << 21)),
    (UNSUPPORTED, lambda: weight(rows=1, n=1 << 18, k=1 << 18, ld_dy=1 << 18, ld_x=1 << 18, ld_out=1 << 18)),
])
def test_weight_grad_refuses(status, call):
    assert call() == status


def forward(gate=X, ldg=128, up=X + 80, ldu=128, dtype=1, rows=64, cols=40, act=0, h=Y, ldh=40, g8=None, u8=None):
    return LIB.gated_act_forward(gate, ldg, up, ldu, dtype, rows, cols, act, h, ldh, g8, u8, None)


def backward(g8=None, u8=None, dh=X, ldd=40, dtype=1, act=0, dg=Y, ldg=80, du=Y + 80, ldu=80, h=None, ldh=0):
    g8 = kept() if g8 is None else g8
    u8 = kept(data=Z, scale=Z + (1 << 20)) if u8 is None else u8
    return LIB.gated_act_backward(g8, u8, dh, ldd, dtype, act, dg, ldg, du, ldu, h, ldh, None)


@pytest.mark.parametrize("status,call", [
    (ARG, lambda: forward(act=2)),
    (ARG, lambda: forward(g8=kept())),                          # one checkpoint of two
    (ARG, lambda: forward(g8=kept(), u8=kept())),               # the same one twice
    (ARG, lambda: forward(h=X)),
    (ARG, lambda: forward(h=X + 80, ldh=128)),                  # h where up is
    (ARG, lambda: forward(gate=None)),
    (DTYPE, lambda: forward(dtype=9)),
    (SHAPE, lambda: forward(ldu=39)),
    (SHAPE, lambda: forward(g8=kept(), u8=kept(cols=39, data=Z, scale=Z + (1 << 20)))),
    (ALIGN, lambda: forward(up=X + 81)),
    (ARG, lambda: backward(act=-1)),
    (ARG, lambda: LIB.gated_act_backward(None, kept(), X, 40, 1, 0, Y, 40, Z, 40, None, 0, None)),
    (ARG, lambda: LIB.gated_act_backward(kept(), None, X, 40, 1, 0, Y, 40, Z, 40, None, 0, None)),
    (ARG, lambda: backward(dg=X)),                              # dgate over dh
    (ARG, lambda: backward(du=Y + 78)),                         # dup's rows over dgate's
    (ARG, lambda: backward(dg=BASE, ldg=40)),                   # over the checkpoint
    (ARG, lambda: backward(h=Y, ldh=80)),
    (SHAPE, lambda: backward(u8=kept(rows=65, data=Z, scale=Z + (1 << 20)))),
    (SHAPE, lambda: backward(h=BASE + (6 << 30), ldh=39)),
])
def test_gated_activation_refuses(status, call):
    assert call() == status


def lookup(tok=X, bits=64, n=100, table=Y, tt=0, ldt=40, vocab=50, cols=40, out=Z, ot=1, ldo=40):
    return LIB.embedding_lookup(tok, bits, n, table, tt, ldt, vocab, cols, 1.0, out, ot, ldo, None)


def grad(tok=X, bits=64, n=100, dy=Y, dt=1, ldd=40, g=Z, gt=0, ldg=40, vocab=50, cols=40, acc=0, ws=BASE, nws=None):
    nws = LIB.embedding_grad_workspace_bytes(n, vocab, cols) if nws is None else nws
    return LIB.embedding_grad(tok, bits, n, dy, dt, ldd, g, gt, ldg, vocab, cols, 1.0, acc, ws, nws, None)


@pytest.mark.parametrize("status,call", [
    (DTYPE, lambda: lookup(bits=16)),
    (DTYPE, lambda: lookup(tt=4)),
    (DTYPE, lambda: lookup(ot=4)),
    (ARG, lambda: lookup(tok=None)),
    (ARG, lambda: lookup(table=None)),
    (ARG, lambda: lookup(out=None)),
    (ARG, lambda: lookup(out=Y + 160)),
    (ARG, lambda: lookup(out=X)),
    (ALIGN, lambda: lookup(tok=X + 4)),
    (SHAPE, lambda: lookup(ldt=39)),
    (SHAPE, lambda: lookup(n=-1)),
    (SHAPE, lambda: lookup(n=1 << 30)),
    (SHAPE, lambda: lookup(vocab=1 << 30)),
    (DTYPE, lambda: grad(bits=8)),
    (ARG, lambda: grad(acc=3)),
    (ARG, lambda: grad(g=Y + 80)),
    (ARG, lambda: grad(g=X, ldg=40)),
    (ARG, lambda: grad(ws=Z)),
    (ARG, lambda: grad(dy=None)),
    (SHAPE, lambda: grad(ldg=39)),
    (SHAPE, lambda: grad(vocab=-1, nws=0)),
    (WORKSPACE, lambda: grad(ws=None)),
    (WORKSPACE, lambda: grad(nws=100)),
    (ALIGN, lambda: grad(ws=BASE + 8)),
    (ALIGN, lambda: grad(g=Z + 2)),
])
def test_embedding_refuses(status, call):
    assert call() == status


def test_nothing_to_do_is_no_error():
    """Matrices without elements: no launch, null pointers allowed."""
    empty = kept(rows=0, data=None, scale=None)
    assert LIB.act_pack(None, 1, 0, empty, None) == 0
    assert LIB.act_read(empty, None, 1, 0, None) == 0
    assert weight(rows=0, dy=None, x=None, acc=1) == 0
    assert weight(n=0, dy=None, out=None) == 0
    assert weight(k=0, x=None, out=None) == 0
    assert forward(rows=0, gate=None, up=None, h=None) == 0
    assert LIB.gated_act_backward(empty, empty, None, 0, 1, 0, None, 0, None, 0, None, 0, None) == 0
    assert lookup(n=0, tok=None, out=None) == 0
    assert grad(n=0, tok=None, dy=None, acc=1) == 0
    assert grad(vocab=0, g=None, nws=0) == 0


def test_workspace_queries():
    w = LIB.weight_grad_workspace_bytes
    assert w(-1, 4, 4) == 0 and w(1 << 30, 4, 4) == 0
    assert w(64, 64, 64) == 0                       # one step of rows cannot be split
    assert w(65536, 64, 64) > 0
    assert w(65536, 64, 64) <= 64 << 20
    e = LIB.embedding_grad_workspace_bytes
    assert e(-1, 4, 4) == 0 and e(4, 1 << 30, 4) == 0
    # the order (8 bytes a token), the starts of vocab + 1 rows
    assert e(64, 100, 8) >= 64 * 8 + 101 * 4
    # two fp32 rows for every 64 positions
    assert e(6400, 100, 9) >= 6400 * 8 + 101 * 4 + 100 * 4 + 100 * 2 * 16 * 4


# --------------------------------------------------------- refusals, binding

B, F = torch.bfloat16, torch.float32


def test_checkpoint_buffers():
    c = q.ActCheckpoint(70, 33, device="cpu")
    assert c.data.shape == (70, 48) and c.scale.shape == (3, 48) and c.shape == (70, 33)
    assert c.nbytes == 73 * 48
    c = q.ActCheckpoint(70, 33, data=torch.zeros(70, 64, dtype=torch.uint8))
    assert c.scale.shape == (3, 64)
    for bad in (dict(data=torch.zeros(70, 40, dtype=torch.uint8)), dict(data=torch.zeros(70, 32, dtype=torch.uint8)),
                dict(data=torch.zeros(69, 48, dtype=torch.uint8)), dict(scale=torch.zeros(2, 48, dtype=torch.uint8)),
                dict(data=torch.zeros(70, 48, dtype=torch.uint8), scale=torch.zeros(3, 64, dtype=torch.uint8)),
                dict(data=torch.zeros(70, 96, dtype=torch.uint8)[:, :48])):
        with pytest.raises(ValueError):
            q.ActCheckpoint(70, 33, **bad)
    with pytest.raises(TypeError):
        q.ActCheckpoint(70, 33, data=torch.zeros(70, 48, dtype=torch.int8))
    with pytest.raises(ValueError):
        q.ActCheckpoint(-1, 33, device="cpu")


def c8(rows=8, cols=6):
    return q.ActCheckpoint(rows, cols, device="cpu")


@pytest.mark.parametrize("error,call", [
    (TypeError, lambda: q.act_pack([1.0])),
    (TypeError, lambda: q.act_pack(torch.zeros(4, 4, dtype=torch.float64))),
    (ValueError, lambda: q.act_pack(torch.zeros(4))),
    (ValueError, lambda: q.act_pack(torch.zeros(4, 4, 4))),
    (ValueError, lambda: q.act_pack(torch.zeros(4, 4).t()[:, :3].t()[:, ::2])),
    (ValueError, lambda: q.act_pack(torch.zeros(1, 4).expand(4, 4))),
    (ValueError, lambda: q.act_pack(torch.zeros(8, 5), ckpt=c8())),
    (TypeError, lambda: q.act_pack(torch.zeros(8, 6), ckpt=3)),
    (ValueError, lambda: q.act_pack(torch.zeros(8, 6))),                     # not on a GPU
    (TypeError, lambda: q.act_read(torch.zeros(4, 4))),
    (ValueError, lambda: q.act_read(c8(), out=torch.zeros(8, 5))),
    (TypeError, lambda: q.act_read(c8(), dtype=torch.int32)),
    (TypeError, lambda: q.weight_grad(torch.zeros(8, 4), c8(), torch.zeros(4, 6))),          # fp32 dy
    (TypeError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), torch.zeros(8, 6), torch.zeros(4, 6))),
    (ValueError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), c8(9), torch.zeros(4, 6))),
    (ValueError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), torch.zeros(9, 6, dtype=B), torch.zeros(4, 6))),
    (ValueError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), c8(), torch.zeros(6, 4))),
    (ValueError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), c8(), torch.zeros(6, 4).t())),
    (ValueError, lambda: q.weight_grad(torch.zeros(8, 4, dtype=B), c8(), torch.zeros(4, 6), ws=3)),
    (ValueError, lambda: q.gated_act_forward(torch.zeros(8, 6), torch.zeros(8, 5))),
    (TypeError, lambda: q.gated_act_forward(torch.zeros(8, 6), torch.zeros(8, 6, dtype=B))),
    (ValueError, lambda: q.gated_act_forward(torch.zeros(8, 6), torch.zeros(8, 6), gate_ckpt=c8(), keep=False)),
    (KeyError, lambda: q.gated_act_forward(torch.zeros(8, 6), torch.zeros(8, 6), act="relu")),
    (TypeError, lambda: q.gated_act_backward(None, c8(), torch.zeros(8, 6))),
    (TypeError, lambda: q.gated_act_backward(c8(), torch.zeros(8, 6), torch.zeros(8, 6))),
    (ValueError, lambda: q.gated_act_backward(c8(), c8(9), torch.zeros(8, 6))),
    (TypeError, lambda: q.gated_act_backward(c8(), c8(), torch.zeros(8, 6), dgate=torch.zeros(8, 6, dtype=B))),
    (TypeError, lambda: q.embedding_lookup(torch.zeros(3), torch.zeros(5, 4))),
    (TypeError, lambda: q.embedding_lookup(torch.zeros(3, dtype=torch.int16), torch.zeros(5, 4))),
    (ValueError, lambda: q.embedding_lookup(torch.zeros(6, dtype=torch.int64)[::2], torch.zeros(5, 4))),
    (ValueError, lambda: q.embedding_lookup(torch.zeros(3, dtype=torch.int64), torch.zeros(5, 4), out=torch.zeros(3, 5))),
    (ValueError, lambda: q.embedding_grad(torch.zeros(3, dtype=torch.int64), torch.zeros(4, 4), torch.zeros(5, 4))),
    (ValueError, lambda: q.embedding_grad(torch.zeros(3, dtype=torch.int64), torch.zeros(3, 4), torch.zeros(5, 5))),
])
def test_binding_refuses(error, call):
    with pytest.raises(error):
        call()


def test_rows_of_one_element_and_one_row_have_any_stride():
    """What numbers no second element is not looked at."""
    assert q._matrix(torch.zeros(4, 8)[:, :1], "x")[2] == 8
    assert q._matrix(torch.zeros(1, 5), "x")[2] == 5
    assert ctypes.sizeof(L.Act8) == 40
