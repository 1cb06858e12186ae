"""AdamW over one tensor, and the global gradient norm: plain numpy.

TEST INFRASTRUCTURE ONLY (see the package).  Weights and 32-bit states are
computed in fp64 without intermediate roundings.  The codes and block maxima
of 8-bit states are defined by binary32 operations in a stated order;
`coded_states` does exactly those, one numpy fp32 operation per rounding.
"""
import numpy as np

from . import philox4x32_10  # noqa: F401  (the scalar form, for pins of `words`)

BLOCK = 256
TINY = np.float32(2.0 ** -100)
F = np.float32


def _blocks(x, dtype):
    """[numel] -> [blocks, 256], zero-padded."""
    n = x.size
    nb = -(-n // BLOCK)
    out = np.zeros(nb * BLOCK, dtype=dtype)
    out[:n] = x
    return out.reshape(nb, BLOCK)


def decode(m_code, v_code, m_absmax, v_absmax):
    """Values (fp32) of 8-bit states."""
    n = m_code.size
    c = _blocks(v_code, F)
    with np.errstate(invalid="ignore"):
        m = _blocks(m_code, F) * (m_absmax / F(127))[:, None]
        v = (c * c) * (v_absmax / F(65025))[:, None]
    return m.reshape(-1)[:n], v.reshape(-1)[:n]


def moments(m0, v0, g, beta1, beta2):
    """New (m, v) in fp64."""
    g = g.astype(np.float64)
    return (beta1 * m0.astype(np.float64) + (1 - beta1) * g,
            beta2 * v0.astype(np.float64) + (1 - beta2) * g * g)


def weight(w0, m, v, step, lr, beta1, beta2, eps, weight_decay):
    """New weight in fp64 from the new moments."""
    hat = (m / (1 - beta1 ** step)) / (np.sqrt(v / (1 - beta2 ** step)) + eps)
    w0 = w0.astype(np.float64)
    return w0 - lr * weight_decay * w0 - lr * hat


def words(numel, seed, offset, tensor, first=0):
    """32-bit random word of every element from `first` (a multiple of 4) on:
    Philox4x32-10, counter (element / 4 as two words, offset, tensor), key
    seed."""
    mask, n4 = np.uint64(0xFFFFFFFF), -(-numel // 4)
    q = np.arange(first // 4, first // 4 + n4, dtype=np.uint64)
    sh = np.uint64(32)
    c = [q & mask, q >> sh, np.full(n4, offset, np.uint64), np.full(n4, tensor, np.uint64)]
    k0, k1 = seed & 0xFFFFFFFF, seed >> 32
    for _ in range(10):
        p0, p1 = np.uint64(0xD2511F53) * c[0], np.uint64(0xCD9E8D57) * c[2]
        c = [(p1 >> sh) ^ c[1] ^ np.uint64(k0), p1 & mask, (p0 >> sh) ^ c[3] ^ np.uint64(k1), p0 & mask]
        k0, k1 = (k0 + 0x9E3779B9) & 0xFFFFFFFF, (k1 + 0xBB67AE85) & 0xFFFFFFFF
    return np.stack(c, axis=1).reshape(-1)[:numel].astype(np.uint32)


def coded_states(m_code, v_code, m_absmax, v_absmax, g, beta1, beta2, word=None):
    """New 8-bit states.  g: fp32 [numel], already times the clip factor (one
    fp32 product).  word: random words for stochastic rounding, None: nearest.
    Returns (m_code, v_code, m_absmax, v_absmax)."""
    n = m_code.size
    b1, a1, b2, a2 = F(beta1), F(1.0 - beta1), F(beta2), F(1.0 - beta2)
    with np.errstate(all="ignore"):
        g = _blocks(g, F)
        step_m, step_v = (m_absmax / F(127)) * b1, (v_absmax / F(65025)) * b2
        c = _blocks(v_code, F)
        m = _blocks(m_code, F) * step_m[:, None] + a1 * g
        v = (c * c) * step_v[:, None] + a2 * (g * g)
        inside = np.arange(m.size).reshape(m.shape) < n
        m, v = np.where(inside, m, F(0)), np.where(inside, v, F(0))
        top_m, top_v = np.max(np.abs(m), axis=1), np.max(v, axis=1)       # NaN if any is
        top_m, top_v = np.where(top_m < TINY, F(0), top_m), np.where(top_v < TINY, F(0), top_v)
        ok_m, ok_v = np.isfinite(top_m), np.isfinite(top_v)
        inv_m = np.where(ok_m & (top_m > 0), F(127) / top_m, F(0)).astype(F)
        inv_v = np.where(ok_v & (top_v > 0), F(65025) / top_v, F(0)).astype(F)
        x, y = m * inv_m[:, None], v * inv_v[:, None]
        x = np.where(ok_m[:, None], x, F(0))
        y = np.where(ok_v[:, None], y, F(0)).astype(np.float64)
        k = np.floor(np.sqrt(y))                     # y has 24 bits: its fp64 root never rounds up to a whole number
        above = y - k * k                            # exact
        if word is None:
            cm = np.rint(x)
            up = above > k + 0.5
        else:
            r = _blocks(word, np.uint32)
            cm = np.floor(x).astype(np.float64)
            cm = cm + ((r >> np.uint32(16)).astype(np.float64) * 2.0 ** -16 < x - cm)     # exact
            up = above > (r & np.uint32(0x7FFF)).astype(np.float64) * 2.0 ** -15 * (2 * k + 1)
        cm = np.clip(cm, -127, 127)
        cv = np.where((v > 0) & (ok_v & (top_v > 0))[:, None], np.clip(k + up, 1, 255), 0)
    return (cm.astype(np.int8).reshape(-1)[:n], cv.astype(np.uint8).reshape(-1)[:n],
            top_m.astype(F), top_v.astype(F))


def norm_and_coef(grads, max_norm, eps):
    """(norm, coef) in fp64 of a list of arrays."""
    s = sum(float(np.sum(np.square(g.astype(np.float64)))) for g in grads)
    if not np.isfinite(s):
        return float(np.sqrt(s)), float("nan")
    norm = float(np.sqrt(s))
    return norm, min(1.0, max_norm / (norm + eps)) if norm + eps > 0 else 1.0
