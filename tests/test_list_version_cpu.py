"""A list blob of another layout or kind is refused by every entry point that
reads one, before any launch (no GPU).  A library that took another layout's
blob would read its table offsets from the wrong fields."""
import ctypes

import pytest

from quantized_momentum_newton_amd import _lib as L
from test_adamw_cpu import ALIGN, DEV, LIB, PLAN, _adamw, _encode, _grads, _hp

WORDS = {"magic": 0, "version": 1, "kind": 2}       # 32-bit words of the header


@pytest.mark.parametrize("word,value", [("version", 0), ("version", 1), ("version", 3), ("version", 2 ** 32 - 1),
                                        ("magic", 0), ("magic", 0x54534c50), ("kind", 0), ("kind", 3)])
@pytest.mark.parametrize("grads", [False, True])
def test_blobs_of_another_layout_are_refused(word, value, grads):
    status, plan, buf, size = _encode(_grads([(1024, L.QM_F32)]) if grads else _adamw([(1024, 8)]))
    assert status == 0 and LIB.qm_list_blocks(plan) == 4
    head = ctypes.cast(buf, ctypes.POINTER(ctypes.c_uint32))
    assert head[WORDS["version"]] == 2 and head[WORDS["magic"]] == 0x54534c51
    head[WORDS[word]] = value
    assert LIB.qm_list_blocks(plan) == -1 and LIB.qm_last_error()
    if grads:
        assert LIB.grad_norm_workspace_bytes(plan) == 0
        assert LIB.grad_norm(plan, DEV, 1.0, 1e-6, DEV, DEV, DEV, 1 << 20, None) == PLAN
        assert LIB.grad_scale(plan, DEV, DEV, None) == PLAN
    else:
        assert LIB.adamw_step(plan, DEV, ctypes.byref(_hp()), None, None) == PLAN
        assert LIB.adamw_read_state(plan, DEV, DEV, DEV, None) == PLAN
    assert LIB.qm_last_error()


def test_host_blob_alignment():
    plan = _encode(_adamw([(1024, 8)]))[1]
    assert LIB.adamw_read_state(ctypes.c_void_p(plan.value + 4), DEV, DEV, DEV, None) == ALIGN
    assert LIB.qm_list_blocks(ctypes.c_void_p(plan.value + 4)) == -1
