"""Plain definitions, in 64 bits, of the operators that make the gradients:
activations in 8 bits, weight gradients, gated activations, embeddings.  Shares
no code with the library."""
import numpy as np

GROUP = 32
LOW, HIGH = -95, 119


def e4m3_values():
    """The number each byte stands for: 1 sign bit, 4 exponent bits biased by
    7, 3 mantissa bits, subnormals, 0x7f and 0xff NaN."""
    out = np.empty(256)
    for b in range(256):
        e, m = (b >> 3) & 15, b & 7
        v = (1 + m / 8) * 2.0 ** (e - 7) if e else m * 2.0 ** -9
        out[b] = np.nan if b & 127 == 127 else (-v if b & 128 else v)
    return out


def group_exponent(top):
    """The smallest integer e with top <= 448 * 2^e, between LOW and HIGH."""
    for e in range(LOW, HIGH + 1):
        if top <= 448 * 2.0 ** e:
            return e
    return HIGH


def encode(x):
    """(bytes, scale bytes) of a rows x cols matrix; scale bytes one per group
    of 32 rows and column.  A group with an infinity or a NaN: bytes 0x7f."""
    x = np.asarray(x, dtype=np.float64)
    rows, cols = x.shape
    values = e4m3_values()[:127]                       # not negative, ascending
    middle = (values[1:] + values[:-1]) / 2
    data = np.zeros((rows, cols), dtype=np.uint8)
    scale = np.zeros((-(-rows // GROUP), cols), dtype=np.uint8)
    for g in range(scale.shape[0]):
        part = x[g * GROUP:(g + 1) * GROUP]
        bad = ~np.isfinite(part).all(0)
        top = np.abs(np.where(bad, 0, part)).max(0)
        e = np.array([group_exponent(t) for t in top])
        y = np.minimum(np.abs(np.where(bad, 0, part)) * 2.0 ** -e.astype(np.float64), 448.0)
        k = np.searchsorted(middle, y)                 # first middle >= y: rounds down, ties too
        tie = (k < 126) & (y == middle[np.minimum(k, 125)])
        k = k + (tie & (k % 2 == 1))                   # ties to the even byte
        code = (k + 128 * np.signbit(part)).astype(np.uint8)
        data[g * GROUP:(g + 1) * GROUP] = np.where(bad, 0x7f, code)
        scale[g] = np.where(bad, 255, e + 127)         # the scale of a bad group is not defined
    return data, scale


def decode(data, scale):
    unit = 2.0 ** (scale.astype(np.float64) - 127)
    return e4m3_values()[data] * np.repeat(unit, GROUP, axis=0)[:data.shape[0]]


def sigmoid(z):
    return np.exp(-np.logaddexp(0.0, -z))


GELU = 2 * np.sqrt(2 / np.pi)


def act(g, kind):
    """(value, slope, s, z, dz/dg): act = g s, s = sigmoid(z)."""
    g = np.asarray(g, dtype=np.float64)
    if kind == "silu":
        z, dz = g, np.ones_like(g)
    else:
        z, dz = GELU * (g + 0.044715 * g ** 3), GELU * (1 + 3 * 0.044715 * g ** 2)
    s = sigmoid(z)
    return g * s, s + g * s * sigmoid(-z) * dz, s, z, dz


def weight_grad(dy, x):
    return np.asarray(dy, dtype=np.float64).T @ np.asarray(x, dtype=np.float64)


def embedding_lookup(tokens, table, scale):
    out = np.zeros((len(tokens), table.shape[1]))
    for i, t in enumerate(tokens):
        if 0 <= t < len(table):
            out[i] = scale * np.asarray(table[t], dtype=np.float64)
    return out


def embedding_grad(tokens, dy, vocab, scale):
    grad = np.zeros((vocab, dy.shape[1]))
    inside = (tokens >= 0) & (tokens < vocab)
    np.add.at(grad, tokens[inside], np.asarray(dy, dtype=np.float64)[inside])
    return scale * grad
