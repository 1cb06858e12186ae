"""Limits of the tensor lists, by fake device addresses (no GPU): the largest
list a launch can cover."""
import ctypes

import pytest

import quantized_momentum_newton_amd as q
from quantized_momentum_newton_amd import _lib as L

LIB = q._LIB
UNSUPPORTED = 7
LAST = 2 ** 25 - 4      # tasks: 2 * ceil(LAST / 4) workgroups of 256 threads stay below 2^32


def adamw(numel, cols=0, ld=0, state_bits=8):
    size = ctypes.c_size_t(0)
    at = [(k + 1) << 46 for k in range(6)]
    m_top, v_top = (at[4], at[5]) if state_bits == 8 else (None, None)
    t = L.AdamWTensor(at[0], at[1], at[2], at[3], m_top, v_top, None, numel, cols, ld, L.QM_BF16, L.QM_BF16, 0,
                      state_bits, 1.0, 0.0)
    return LIB.qm_adamw_plan_encode((L.AdamWTensor * 1)(t), 1, None, ctypes.byref(size)), size.value


@pytest.mark.parametrize("bits", [8, 32])
@pytest.mark.parametrize("tasks,status", [(LAST, 0), (LAST + 1, UNSUPPORTED), (LAST + 3, UNSUPPORTED), (LAST + 4, UNSUPPORTED),
                                          (LAST + 5, UNSUPPORTED)])
def test_largest_list(tasks, status, bits):
    assert 2 * -(-LAST // 4) * 256 < 2 ** 32 <= 2 * -(-(LAST + 1) // 4) * 256
    assert adamw(tasks * 1024, state_bits=bits)[0] == status, LIB.qm_last_error()


def test_largest_list_of_gradients():
    for tasks, status in ((LAST, 0), (LAST + 1, UNSUPPORTED)):
        size = ctypes.c_size_t(0)
        g = (L.GradTensor * 1)(L.GradTensor(1 << 40, tasks * 1024, 0, 0, L.QM_BF16, 0))
        assert LIB.qm_grad_plan_encode(g, 1, None, ctypes.byref(size)) == status
