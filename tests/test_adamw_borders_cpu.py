"""The coding of 8-bit AdamW states next to its borders, in the oracle: what
the definition in include/qmuon.h says there, without a GPU."""
import numpy as np
import pytest

import oracle
from oracle import adamw as A


def border_gradients(word):
    """Per element (none of them a block's first) a gradient that lies, by its
    place modulo 3, one fp32 step below, on or one above the border of its
    random number u = word >> 16, where floor(x) + u / 2^16 = x, in [0, 1) for
    u below 2^15 and in (-1, 0) else; a block's first is 127, so that with
    beta1 = 0 and zero states x is the gradient itself.  Returns (gradients,
    expected codes of m)."""
    n = word.size
    e = np.arange(n)
    u = (word >> np.uint32(16)).astype(np.float64)
    down = np.where(u < 32768, 0.0, -1.0)
    on = (down + u / 65536).astype(np.float32)              # exact: 16 bits
    side = e % 3 - 1
    g = np.where(side < 0, np.nextafter(on, np.float32(-np.inf)), np.where(side > 0, np.nextafter(on, np.float32(np.inf)), on))
    codes = np.where(side > 0, down + 1, down)
    # one step below a whole number is the interval under it, and its fraction is above any u
    codes = np.where((side < 0) & (u == 0), down, codes)
    first = e % 256 == 0
    return np.where(first, np.float32(127), g).astype(np.float32), np.where(first, 127, codes).astype(np.int8)


def zero_state(n):
    nb = -(-n // 256)
    return np.zeros(n, np.int8), np.zeros(n, np.uint8), np.zeros(nb, np.float32), np.zeros(nb, np.float32)


def test_stochastic_code_of_m_compares_exactly():
    """floor(x) + 1 if u / 2^16 < x - floor(x): the difference is not rounded.
    It has more than 24 bits for x in (-1/2, 0)."""
    z = zero_state(256)
    for x, u, want in ((-(0.5 - 2.0 ** -25), 32768, 0), (-(2.0 ** -16 - 2.0 ** -40), 65535, 0), (-(2.0 ** -16), 65535, -1),
                       (-0.5, 32768, -1), (-(2.0 ** -60), 65535, 0), (2.0 ** -60, 0, 1), (0.25, 16384, 0), (0.0, 0, 0)):
        g = np.zeros(256, np.float32)
        g[0], g[1] = 127.0, x
        assert g[1] == x
        word = np.full(256, u << 16, np.uint32)
        assert A.coded_states(*z, g, 0.0, 0.9, word)[0][1] == want, (x, u)


@pytest.mark.parametrize("seed", [2, 77])
def test_stochastic_codes_of_m_on_both_sides_of_their_borders(seed):
    n = 256 * 64
    word = A.words(n, seed, 3, 0)
    g, want = border_gradients(word)
    assert np.array_equal(A.coded_states(*zero_state(n), g, 0.0, 0.9, word)[0], want)


@pytest.mark.parametrize("y", [1e-6, 0.1, 0.5, 0.99, 1.0, 1.01, 1.5, 2.5, 3.99, 4.0, 50.3, 1000.7, 64000.0])
def test_mean_of_the_square_of_stochastic_codes_of_v(y):
    """E[code^2] = y from y = 1 on (within 6 standard errors); below, the code
    is 1 always, so a decoded v is at least one code of its block: more than v
    by the factor 1 / y."""
    n = 256 * 1000
    g = np.full(n, np.sqrt(np.float32(y)), np.float32)
    g[::256] = 255.0                      # every block's maximum: 65025, so that y = v = g * g
    code = A.coded_states(*zero_state(n), g, 0.9, 0.0, A.words(n, 13, 1, 0))[1].astype(np.float64)
    assert np.all(code[::256] == 255)
    body = code[np.arange(n) % 256 != 0]
    exact = float(g[1]) ** 2
    if y < 1:
        assert np.all(body == 1)
    else:
        k = np.floor(np.sqrt(exact))
        assert np.all((body == k) | (body == k + 1))
        spread = np.sqrt(max((exact - k * k) * ((k + 1) ** 2 - exact), 0.0) / body.size)
        # the random number has 15 bits: its mean threshold is half a step (2k + 1) 2^-16 low
        assert abs((body ** 2).mean() - exact) <= 6 * spread + (2 * k + 1) * 2.0 ** -16 + 2.0 ** -22 * exact


def test_words_from_an_element_on():
    """The counter's second word is used from element 2^34 on."""
    assert np.array_equal(A.words(100, 5, 6, 7)[40:], A.words(60, 5, 6, 7, first=40))
    for first in (1 << 32, (1 << 34) - 4, 1 << 34):
        w = A.words(8, (3 << 32) + 9, 77, 5, first=first)
        for e in range(8):
            group = (first + e) // 4
            ref = oracle.philox4x32_10([group & 0xFFFFFFFF, group >> 32, 77, 5], [9, 3])
            assert w[e] == ref[e % 4]
