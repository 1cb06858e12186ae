"""The training example: every optimizer operator in one program."""
import importlib.util
import math
import os

import pytest

from gpu_util import say

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))


def test_example_learns():
    """From a loss near log(vocabulary) to a tenth of it, without a step that
    is not finite."""
    spec = importlib.util.spec_from_file_location("train_lm", os.path.join(ROOT, "examples", "train_lm.py"))
    mod = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(mod)
    losses = mod.main(120, report=say)
    assert all(math.isfinite(x) for x in losses)
    assert abs(losses[0] - math.log(mod.VOCAB)) < 1.0
    assert losses[-1] < 0.1 * losses[0]
