"""The serving operators together, as the example runs them: verified windows of a hybrid model give
the logits of the same tokens run one at a time."""
import importlib.util
import os

import pytest

pytestmark = pytest.mark.gpu

PATH = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples",
                    "hybrid_verify.py")


def test_windows_equal_single_tokens():
    """Both runs do the same sums in another order and round activations to bf16 (2^-8) a few times
    a layer; a page's scale may also have been raised by a drafted token that was refused, which
    moves codes by at most one step of the 8-bit format below its normal range. The logits stay
    within 2^-4 of the largest one."""
    spec = importlib.util.spec_from_file_location("hybrid_verify", PATH)
    example = importlib.util.module_from_spec(spec)
    spec.loader.exec_module(example)
    rows, worst = example.check()
    assert all(7 <= len(r) <= 25 for r in rows)   # six steps of 1 .. 4 tokens after the first
    assert worst < 2.0 ** -4, worst
