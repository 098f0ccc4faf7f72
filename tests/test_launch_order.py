"""A kernel that lets the next one begin before it has itself waited for the one before lets that next kernel run beside
the one before: a projection launched early (LORA_OPT_PDL) requests its W before it waits. Read from the sources."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "mixed_lora_projection_gb300", "csrc")


@pytest.mark.parametrize("name", ["layer_ops.cu", "attn_decode.cu", "attn_prompt.cu"])
def test_operators_wait_before_they_let_the_next_kernel_begin(name):
    src = re.sub(r"//[^\n]*", "", open(os.path.join(CSRC, name)).read())
    kernels = re.split(r"__global__", src)[1:]
    assert kernels
    for k in kernels:
        calls = re.findall(r"griddep_(wait|launch_dependents)\(\)", k)
        assert calls == ["wait", "launch_dependents"], (name, calls)
