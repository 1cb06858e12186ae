"""Hyperparameters of the AdamW step that fp32 cannot hold (no GPU)."""
import ctypes

import pytest

from test_adamw_cpu import ARG, DEV, LIB, _adamw, _encode, _hp


@pytest.mark.parametrize("kw", [dict(lr=1e39), dict(lr=-1e39), dict(lr=3e38, beta1=0.9, step=1)])
def test_step_sizes_past_fp32_are_refused(kw):
    """lr or lr / (1 - beta1^t) as an infinity would turn every weight whose
    moment or decay is 0 into a NaN."""
    plan = _encode(_adamw([(0, 8), (0, 32)]))[1]       # nothing to launch
    assert LIB.adamw_step(plan, DEV, ctypes.byref(_hp(**kw)), None, None) == ARG and b"lr" in LIB.qm_last_error()
    assert LIB.adamw_step(plan, DEV, ctypes.byref(_hp(lr=3e38, beta1=0.9, step=10 ** 6)), None, None) == 0
