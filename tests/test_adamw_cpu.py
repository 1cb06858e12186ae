"""AdamW and gradient-norm lists without a GPU: the oracle's pins, the list
encoder's rules, and every refusal before a launch."""
import ctypes
import math

import numpy as np
import pytest
import torch

import oracle
import quantized_momentum_newton_amd as q
from oracle import adamw as A
from quantized_momentum_newton_amd import _lib as L

LIB = q._LIB
BASE = 0x7f0000000000     # fake device addresses: only alignment and overlap are looked at
ARG, ALIGN, DTYPE, SHAPE, WORKSPACE, UNSUPPORTED, PLAN = 1, 2, 3, 4, 5, 7, 8


# ------------------------------------------------------------------ oracle

def test_adamw_first_step_closed_form():
    """From zero states the first step moves every weight by lr sign(g)
    (eps -> 0) after the decay."""
    g = np.array([1e-3, -2.0, 5e-2])
    m, v = A.moments(np.zeros(3), np.zeros(3), g, 0.9, 0.999)
    w = A.weight(np.array([1.0, -1.0, 0.5]), m, v, 1, 0.01, 0.9, 0.999, 0.0, 0.1)
    assert np.allclose(w, np.array([1.0, -1.0, 0.5]) * (1 - 0.001) - 0.01 * np.sign(g), rtol=1e-14, atol=0)


def test_adamw_matches_torch_in_64_bits():
    torch.manual_seed(3)
    p = torch.randn(300, dtype=torch.float64, requires_grad=True)
    opt = torch.optim.AdamW([p], lr=3e-3, betas=(0.8, 0.97), eps=1e-7, weight_decay=0.05, foreach=False, fused=False)
    w, m, v = p.detach().numpy().copy(), np.zeros(300), np.zeros(300)
    for t in range(1, 8):
        g = torch.randn(300, dtype=torch.float64) * 10.0 ** (-t)
        p.grad = g
        opt.step()
        m, v = A.moments(m, v, g.numpy(), 0.8, 0.97)
        w = A.weight(w, m, v, t, 3e-3, 0.8, 0.97, 1e-7, 0.05)
        assert np.allclose(p.detach().numpy(), w, rtol=1e-12, atol=1e-15)


def test_words_are_the_scalar_generator():
    w = A.words(23, 0x123456789ABCDEF, 77, 5)
    for e in range(23):
        ref = oracle.philox4x32_10([e // 4, 0, 77, 5], [0x89ABCDEF, 0x1234567])
        assert w[e] == ref[e % 4]


def _random_state(n, rng):
    nb = -(-n // 256)
    return (rng.integers(-127, 128, n).astype(np.int8), rng.integers(0, 256, n).astype(np.uint8),
            rng.uniform(1e-4, 1e-2, nb).astype(np.float32), rng.uniform(1e-7, 1e-5, nb).astype(np.float32))


def test_codes_decode_near_their_values():
    """m within half a step of its block; v's code is the one whose square is
    nearest, so |v - decoded| <= (k + 1/2) steps at root k; never 0 where v > 0."""
    rng = np.random.default_rng(1)
    n = 256 * 40 + 77
    st = _random_state(n, rng)
    g = (rng.standard_normal(n) * 1e-3).astype(np.float32)
    cm, cv, tm, tv = A.coded_states(*st, g, 0.9, 0.999)
    m, v = A.moments(*A.decode(*st), g, 0.9, 0.999)
    dm, dv = A.decode(cm, cv, tm, tv)
    blk = np.arange(n) // 256
    assert np.all(np.abs(dm - m) <= (tm / 127)[blk] * (0.5 + 127 * 2.0 ** -20))
    root = np.sqrt(v / (tv.astype(np.float64) / 65025)[blk])
    bound = np.where(root < 1, 1.0, np.floor(root) + 0.5) * (1 + 2.0 ** -10)
    assert np.all(np.abs(dv - v) <= bound * (tv / 65025)[blk])
    assert np.all(cv[v > 0] >= 1)
    # brute force over all codes
    y = v / (tv.astype(np.float64) / 65025)[blk]
    near = np.abs(np.arange(256)[None, :] ** 2 - y[:, None])
    best, got = near.min(1), np.abs(cv.astype(np.float64) ** 2 - y)
    assert np.all((got <= best + 1e-2) | (cv == 1))


def test_codes_of_squares_and_of_the_values_next_to_midpoints():
    """With beta2 = 0 and a block maximum of 65025, y = v = g^2: whole g code
    as themselves, g one part in 1e4 either side of sqrt(k^2 + k + 1/2) as k
    and k + 1."""
    z = (np.zeros(256, np.int8), np.zeros(256, np.uint8), np.zeros(1, np.float32), np.zeros(1, np.float32))
    g = np.arange(256).astype(np.float32)
    assert np.array_equal(A.coded_states(*z, g, 0.0, 0.0)[1], np.arange(256))
    k = np.arange(255)
    mid = np.sqrt(k * k + k + 0.5)
    for f, want in ((1 - 1e-4, k), (1 + 1e-4, k + 1)):
        g = np.append(mid * f, 255.0).astype(np.float32)
        assert np.array_equal(A.coded_states(*z, g, 0.0, 0.0)[1][:255], np.maximum(want, 1))


def test_edge_blocks():
    n = 256 * 5
    z = (np.zeros(n, np.int8), np.zeros(n, np.uint8), np.zeros(5, np.float32), np.zeros(5, np.float32))
    g = np.zeros(n, np.float32)
    g[256] = 1e-31                  # below the smallest block maximum: a block of zeros
    g[512], g[513] = np.inf, 1.0
    g[768], g[769] = np.nan, np.inf
    g[1024], g[1025] = 1.0, 1e-18   # v tiny next to its block: code 1, not 0
    cm, cv, tm, tv = A.coded_states(*z, g, 0.9, 0.999)
    assert np.all(cm[:256 * 4] == 0) and np.all(cv[:256 * 4] == 0)
    assert tm[0] == 0 and tm[1] == 0 and np.isinf(tm[2]) and np.isnan(tm[3])
    assert cm[1024] == 127 and cv[1024] == 255 and cv[1025] == 1 and cm[1025] == 0
    dm, dv = A.decode(cm, cv, tm, tv)
    assert np.all(np.isnan(dm[512:1024])) and np.all(np.isnan(dv[512:1024]))
    assert np.all(dm[:512] == 0)


def test_stochastic_codes_keep_the_mean():
    """A constant gradient over 60 steps: nearest holds v's codes still where
    stochastic rounding carries the mean of v to the fp64 average within 6
    standard errors (over 64 blocks)."""
    nb, n = 64, 64 * 256
    top = np.full(nb, 1.0, np.float32)
    v0 = np.full(n, 100, np.uint8)
    v0.reshape(nb, 256)[:, 0] = 255
    st = (np.zeros(n, np.int8), v0, np.zeros(nb, np.float32), top)
    g = np.full(n, math.sqrt(3.0 * (100 / 255) ** 2), np.float32)
    g.reshape(nb, 256)[:, 0] = 1.0        # keeps each block's maximum at 1
    near, stoch = st, st
    exact = A.decode(*st)[1].astype(np.float64)
    for t in range(60):
        near = A.coded_states(*near, g, 0.9, 0.999)
        stoch = A.coded_states(*stoch, g, 0.9, 0.999, A.words(n, 9, t, 0))
        exact = 0.999 * exact + 0.001 * g.astype(np.float64) ** 2
    body = np.arange(n) % 256 != 0
    dn, ds = A.decode(*near)[1][body], A.decode(*stoch)[1][body].astype(np.float64)
    assert np.all(near[1][body] == 100)                              # each step changes v by less than half a code
    e = exact[body][0]
    assert e > 1.1 * dn[0]
    assert abs(ds.mean() - e) < 6 * ds.std() / math.sqrt(ds.size) + 1e-6


# ----------------------------------------------------------------- encoder

def _grads(specs):
    arr = (L.GradTensor * len(specs))()
    at = BASE
    for i, (n, dt) in enumerate(specs):
        arr[i] = L.GradTensor(at, n, 0, 0, dt, 0)
        at += (n * 4 + 4095) // 4096 * 4096
    return arr


def _adamw(specs):
    arr = (L.AdamWTensor * len(specs))()
    at = [BASE]

    def take(count):
        a = at[0]
        at[0] += (count + 4096) // 4096 * 4096
        return a
    for i, (n, bits) in enumerate(specs):
        nb = -(-n // 256)
        ssz = 4 if bits == 32 else 1
        arr[i] = L.AdamWTensor(take(4 * n), take(4 * n), take(ssz * n), take(ssz * n),
                               take(4 * nb) if bits == 8 else None, take(4 * nb) if bits == 8 else None, take(2 * n),
                               n, 0, 0, L.QM_F32, L.QM_BF16, L.QM_BF16, bits, 1.0, 0.1)
    return arr


def _encode(arr):
    fn = LIB.qm_grad_plan_encode if isinstance(arr[0], L.GradTensor) else LIB.qm_adamw_plan_encode
    size = ctypes.c_size_t(0)
    st = fn(arr, len(arr), None, ctypes.byref(size))
    if st != 0:
        return st, None
    buf = (ctypes.c_uint64 * ((size.value + 7) // 8))()
    st = fn(arr, len(arr), ctypes.cast(buf, ctypes.c_void_p), ctypes.byref(size))
    return st, ctypes.cast(buf, ctypes.c_void_p) if st == 0 else None, buf, size.value


def test_lists_encode():
    r = _encode(_adamw([(1, 32), (0, 8), (257, 8), (5000, 32), (1024, 8)]))
    assert r[0] == 0
    assert LIB.qm_list_blocks(r[1]) == 1 + 0 + 2 + 20 + 4
    r = _encode(_grads([(7, L.QM_F32), (0, L.QM_F16), (4096, L.QM_BF16)]))
    assert r[0] == 0 and LIB.qm_list_blocks(r[1]) == 17
    assert LIB.grad_norm_workspace_bytes(r[1]) >= 8


@pytest.mark.parametrize("change,status", [
    (dict(weight=None), ARG), (dict(grad=None), ARG), (dict(m=None), ARG), (dict(v=None), ARG),
    (dict(m_absmax=None), ARG), (dict(v_absmax=None), ARG), (dict(numel=-1), ARG),
    (dict(weight_dtype=9), DTYPE), (dict(grad_dtype=3), DTYPE), (dict(copy_dtype=L.QM_F32), DTYPE),
    (dict(state_bits=16), DTYPE), (dict(lr_scale=float("nan")), ARG), (dict(weight_decay=float("inf")), ARG),
    (dict(weight="+2"), ALIGN), (dict(grad="+1"), ALIGN), (dict(m_absmax="+2"), ALIGN), (dict(copy="+1"), ALIGN),
    (dict(grad_cols=3, grad_ld=4), SHAPE), (dict(grad_cols=8, grad_ld=4), SHAPE), (dict(grad_cols=-8, grad_ld=8), SHAPE),
    (dict(grad_cols=8, grad_ld=1 << 60), SHAPE), (dict(numel=1 << 45), UNSUPPORTED),
    (dict(numel=1 << 33, grad_cols=8, grad_ld=16), UNSUPPORTED),
    (dict(numel=1 << 36, grad=1 << 44, weight=1 << 45, m=1 << 43, v=1 << 42, m_absmax=1 << 41, v_absmax=3 << 40,
          copy=1 << 46), UNSUPPORTED),
    (dict(weight="grad"), ARG), (dict(m="v"), ARG), (dict(copy="m_absmax"), ARG),
])
def test_adamw_list_refusals(change, status):
    arr = _adamw([(1024, 8)])
    for k, v in change.items():
        if isinstance(v, str):
            v = getattr(arr[0], k) + int(v) if v[0] == "+" else getattr(arr[0], v)
        setattr(arr[0], k, v)
    assert _encode(arr)[0] == status, LIB.qm_last_error()
    assert LIB.qm_last_error()


def test_adamw_list_refuses_scales_of_32_bit_states_and_shared_buffers():
    arr = _adamw([(1024, 32)])
    arr[0].m_absmax = BASE + (1 << 30)
    assert _encode(arr)[0] == ARG
    arr = _adamw([(1024, 32), (1024, 8)])
    arr[1].weight = arr[0].weight + 4 * 1023
    assert _encode(arr)[0] == ARG


@pytest.mark.parametrize("change,status", [
    (dict(grad=None), ARG), (dict(numel=-5), ARG), (dict(dtype=7), DTYPE), (dict(reserved=1), ARG),
    (dict(grad="+2"), ALIGN), (dict(cols=7, ld=9), SHAPE), (dict(cols=16, ld=8), SHAPE),
])
def test_grad_list_refusals(change, status):
    arr = _grads([(1024, L.QM_F32)])
    for k, v in change.items():
        setattr(arr[0], k, arr[0].grad + int(v) if isinstance(v, str) else v)
    assert _encode(arr)[0] == status, LIB.qm_last_error()


def test_interleaved_column_slices_are_not_an_overlap():
    arr = _grads([(64 * 8, L.QM_F16), (64 * 8, L.QM_F16)])
    for i in range(2):
        arr[i].cols, arr[i].ld = 8, 16
        arr[i].grad = BASE + 16 * i
    assert _encode(arr)[0] == 0, LIB.qm_last_error()
    arr[1].grad = BASE + 14
    assert _encode(arr)[0] == ARG


def test_empty_and_bad_lists():
    size = ctypes.c_size_t(0)
    assert LIB.qm_adamw_plan_encode(None, 1, None, ctypes.byref(size)) == ARG
    assert LIB.qm_adamw_plan_encode(_adamw([(4, 32)]), 0, None, ctypes.byref(size)) == ARG
    assert LIB.qm_grad_plan_encode(_grads([(4, 0)]), 1, None, None) == ARG
    buf = (ctypes.c_uint64 * 8)()
    p = ctypes.cast(buf, ctypes.c_void_p)
    size.value = 8
    assert LIB.qm_grad_plan_encode(_grads([(4, 0)]), 1, p, ctypes.byref(size)) == ARG      # too small
    assert LIB.qm_list_blocks(p) == -1 and LIB.qm_list_blocks(None) == -1
    assert LIB.grad_norm_workspace_bytes(p) == 0


# ------------------------------------------------------------- step refusals

def _hp(**kw):
    d = dict(lr=1e-3, beta1=0.9, beta2=0.999, eps=1e-8, step=1, rounding=0, offset=0, seed=0)
    d.update(kw)
    return L.AdamWHparams(*d.values())


DEV = ctypes.c_void_p(BASE)


@pytest.mark.parametrize("kw", [dict(lr=float("nan")), dict(lr=float("inf")), dict(beta1=1.0), dict(beta1=-0.1),
                                dict(beta2=1.0), dict(beta2=float("nan")), dict(eps=0.0), dict(eps=-1e-8),
                                dict(eps=float("inf")), dict(eps=1e-60), dict(step=0), dict(step=-3),
                                dict(rounding=2)])
def test_adamw_step_refuses_hyperparameters(kw):
    r = _encode(_adamw([(1024, 8)]))
    assert LIB.adamw_step(r[1], DEV, ctypes.byref(_hp(**kw)), None, None) == ARG
    assert LIB.qm_last_error()


def test_step_refusals():
    a, g = _encode(_adamw([(1024, 8)])), _encode(_grads([(1024, 0)]))
    hp = ctypes.byref(_hp())
    assert LIB.adamw_step(None, DEV, hp, None, None) == ARG
    assert LIB.adamw_step(a[1], None, hp, None, None) == ARG
    assert LIB.adamw_step(a[1], DEV, None, None, None) == ARG
    assert LIB.adamw_step(g[1], DEV, hp, None, None) == PLAN
    assert LIB.adamw_step(a[1], ctypes.c_void_p(BASE + 8), hp, None, None) == ALIGN
    assert LIB.adamw_step(a[1], DEV, hp, ctypes.c_void_p(BASE + 2), None) == ALIGN
    assert LIB.adamw_step(ctypes.c_void_p(a[1].value + 4), DEV, hp, None, None) == ALIGN
    assert LIB.adamw_read_state(a[1], DEV, None, DEV, None) == ARG
    assert LIB.adamw_read_state(a[1], DEV, DEV, ctypes.c_void_p(BASE + 4), None) == ALIGN
    assert LIB.adamw_read_state(g[1], DEV, DEV, DEV, None) == PLAN
    assert LIB.grad_scale(g[1], DEV, None, None) == ARG
    assert LIB.grad_scale(a[1], DEV, DEV, None) == PLAN
    assert LIB.grad_scale(g[1], DEV, ctypes.c_void_p(BASE + 1), None) == ALIGN
    n = LIB.grad_norm_workspace_bytes(g[1])

    def norm(plan=g[1], dev=DEV, mx=1.0, eps=1e-6, out=DEV, coef=DEV, ws=DEV, nb=n):
        return LIB.grad_norm(plan, dev, mx, eps, out, coef, ws, nb, None)
    assert norm(plan=a[1]) == PLAN and norm(dev=None) == ARG
    assert norm(mx=0.0) == ARG and norm(mx=float("nan")) == ARG and norm(mx=-1.0) == ARG
    assert norm(eps=-1.0) == ARG and norm(eps=float("inf")) == ARG
    assert norm(out=None) == ARG and norm(coef=None) == ARG and norm(coef=ctypes.c_void_p(BASE + 2)) == ALIGN
    assert norm(ws=None) == WORKSPACE and norm(nb=n - 1) == WORKSPACE and norm(ws=ctypes.c_void_p(BASE + 4)) == ALIGN


def test_lists_of_empty_tensors_launch_nothing():
    a = _encode(_adamw([(0, 8), (0, 32)]))
    assert LIB.adamw_step(a[1], DEV, ctypes.byref(_hp()), None, None) == 0
    assert LIB.adamw_read_state(a[1], DEV, None, None, None) == 0
    g = _encode(_grads([(0, 0)]))
    assert LIB.grad_scale(g[1], DEV, DEV, None) == 0


# ------------------------------------------------------------------ binding

def test_binding_refusals():
    w, g = torch.zeros(8), torch.zeros(8)
    st = q.AdamWState(8, device="cpu")
    with pytest.raises(ValueError):
        q.AdamWState(8, bits=16, device="cpu")
    with pytest.raises(ValueError):
        q.AdamWState(8, bits=32, m_absmax=torch.zeros(1))
    with pytest.raises(TypeError):
        q.AdamWState(8, bits=8, m=torch.zeros(8))
    with pytest.raises(ValueError):
        q.AdamWState(8, bits=8, m=torch.zeros(7, dtype=torch.int8))
    with pytest.raises(ValueError):
        q.AdamWPlan([])
    with pytest.raises(ValueError):
        q.AdamWPlan([(torch.zeros(7), g, st, None, 1.0, 0.0)])
    with pytest.raises(ValueError):
        q.AdamWPlan([(w, torch.zeros(7), st, None, 1.0, 0.0)])
    with pytest.raises(ValueError):
        q.AdamWPlan([(torch.zeros(8, 2)[:, 0], g, st, None, 1.0, 0.0)])
    with pytest.raises(TypeError):
        q.AdamWPlan([(w, g.double(), st, None, 1.0, 0.0)])
    with pytest.raises(ValueError):
        q.AdamWPlan([(w, torch.zeros(1).expand(8), st, None, 1.0, 0.0)])
    with pytest.raises(ValueError):
        q.AdamWPlan([(w, torch.zeros(1, 4).expand(2, 4), st, None, 1.0, 0.0)])
    with pytest.raises(q.QmuonError) as e:
        q.AdamWPlan([(w, g, st, torch.zeros(8), 1.0, 0.0)])      # an fp32 copy
    assert e.value.status == DTYPE
    with pytest.raises(q.QmuonError) as e:
        q.AdamWPlan([(w, w, st, None, 1.0, 0.0)])                # weight and grad the same buffer
    assert e.value.status == ARG
    with pytest.raises(ValueError):
        q.GradPlan([])
    with pytest.raises(ValueError):
        q.GradPlan([torch.zeros(4, 4).t()])
    with pytest.raises(TypeError):
        q.GradPlan([torch.zeros(4, dtype=torch.int32)])
    p = q.AdamWPlan([(w, g, st, None, 1.0, 0.0)])
    with pytest.raises(KeyError):
        q.adamw_step(p, 1, rounding="up")
    with pytest.raises(TypeError):
        q.adamw_step(p, 1, grad_scale=torch.zeros(1, dtype=torch.float64))
    with pytest.raises(ValueError):
        q.adamw_read_state(p, m=torch.zeros(8))
    with pytest.raises(ValueError):
        q.grad_scale(q.GradPlan([g]), torch.zeros(2))
