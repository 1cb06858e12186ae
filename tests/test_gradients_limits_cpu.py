"""The embedding's largest launches, refused on the host (addresses are made up:
nothing is launched)."""
import quantized_momentum_newton_amd as q

LIB = q._LIB
UNSUPPORTED = 7
TOKENS, ROWS, TABLE, SPACE = (k << 44 for k in (1, 2, 3, 4))


def test_gradient_past_the_largest_launch():
    n = vocab = 1 << 28
    ws = LIB.embedding_grad_workspace_bytes(n, vocab, 8)
    assert LIB.embedding_grad(TOKENS, 32, n, ROWS, 1, 8, TABLE, 1, 8, vocab, 8, 1.0, 0, SPACE, ws, None) == UNSUPPORTED
    assert b"2^31 threads" in LIB.qm_last_error()


def test_lookup_past_the_largest_launch():
    n = 1 << 29      # times 32 pieces of 8 columns
    assert LIB.embedding_lookup(TOKENS, 32, n, TABLE, 1, 256, 10, 256, 1.0, ROWS, 1, 256, None) == UNSUPPORTED
    assert b"2^34 pieces" in LIB.qm_last_error()
