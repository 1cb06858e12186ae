"""Workspace of the embedding gradient: every array that the call lays out in
it, counted from the layout's definition."""
import pytest

import quantized_momentum_newton_amd as q


def up(n):
    return -(-n // 256) * 256


@pytest.mark.parametrize("n,vocab,cols", [(1, 1, 1), (32, 100, 8), (33, 100, 8), (64, 100, 9), (6400, 100, 9), (6401, 50257, 2048),
                                          (131072, 130000, 33), (0, 40, 8)])
def test_embedding_grad_workspace(n, vocab, cols):
    """The order (token and position, 8 bytes), the starts of vocab + 1 rows, and
    for every 32 positions, where there are more, the long row that starts there
    and two fp32 rows of columns rounded up to 8."""
    chunks = -(-n // 32) if n > 32 else 0
    part = chunks * 2 * (-(-cols // 8) * 8) * 4
    assert q.embedding_grad_workspace_bytes(n, vocab, cols) == up(up(up(n * 8) + up((vocab + 1) * 4)) + up(chunks * 4)) + up(part)
