"""Source check: kernels that may start while the one before them in the stream still runs do not read what that
kernel may be writing through the non-coherent path, which takes its data as constant for the kernel's whole life
(the compiler may move such a load above the wait, and it may find a line that an earlier load left in L1)."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "int8_mixed_precision_rowwise_b200",
                    "csrc")
# Constant for a program's life: the norm's weight and the slopes of the position biases.
CONSTANT = ("p.w ", "p.w)", "p.slopes")


@pytest.mark.parametrize("name", ["norm.cu", "kvcache.cu", "kvcache.cuh", "attention.cuh", "attention.cu",
                                  "attn_decode.cu", "attn_prefill.cu"])
def test_no_non_coherent_loads_of_what_a_kernel_before_writes(name):
    with open(os.path.join(CSRC, name)) as f:
        text = re.sub(r"//[^\n]*", "", f.read())
    loads = [text[m.end():m.end() + 60].split("\n")[0] for m in re.finditer(r"\b(?:__ldg|ld\.global\.nc)\b\(?", text)]
    assert not [a for a in loads if not a.startswith(CONSTANT)]
    assert "__restrict__" not in text  # with it, plain loads take that path as well
