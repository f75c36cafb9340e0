"""The limits that the header states, at their borders."""
import ctypes

import pytest

import mixture_experts_layer_logits_amd as m
from test_abi import LIB, MOE_EINVAL, MOE_OK, Shape


@pytest.mark.parametrize("k,E,code", [(1, 1, MOE_OK), (32, 32, MOE_OK), (32, 1024, MOE_OK), (33, 64, MOE_EINVAL),
                                      (2, 1, MOE_EINVAL), (1, 1025, MOE_EINVAL)])
def test_choices_a_token(k, E, code):
    lib = ctypes.CDLL(LIB)
    s = Shape(0, 64, 64, E, k, m.MOE_BF16, m.MOE_BF16, 0)  # an empty batch: nothing is launched
    assert lib.moe_combine(ctypes.byref(s), *[None] * 6) == code
