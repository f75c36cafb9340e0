"""Rules that the kernels' sources keep and that no run can show."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixture_experts_layer_logits_amd",
                    "csrc")


@pytest.mark.parametrize("name", ["balance.hip", "route.hip"])
def test_lds_exchanges_inside_a_wave_are_fenced(name):
    """A wave barrier alone orders scheduling, not memory: lanes that hand values on through LDS
    without a workgroup barrier use lanes.h's wave_lds_fence."""
    text = open(os.path.join(CSRC, name)).read()
    assert "wave_lds_fence()" in text and not re.search(r"__builtin_amdgcn_wave_barrier", text)


def test_the_wave_fence_is_one():
    text = open(os.path.join(CSRC, "lanes.h")).read()
    body = re.search(r"void wave_lds_fence\(\) \{(.*?)\n\}", text, re.S).group(1)
    calls = re.findall(r"__builtin_amdgcn_(\w+)\((.*)\);", body)
    assert calls == [("fence", '__ATOMIC_RELEASE, "wavefront"'), ("wave_barrier", ""),
                     ("fence", '__ATOMIC_ACQUIRE, "wavefront"')]
