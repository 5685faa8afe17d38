"""What the kernels' sources promise where no output can show it."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "grpo_loss_gb300", "csrc")


def code(name):
    """A source without its comments."""
    with open(os.path.join(CSRC, name)) as f:
        return re.sub(r"//[^\n]*|/\*.*?\*/", " ", f.read(), flags=re.S)


@pytest.mark.parametrize("name", ["adamw.cu", "norm.cu"])
def test_in_place_kernels_have_no_read_only_loads(name):
    """Their outputs may be their inputs, and a read-only load is defined only for
    memory that the kernel does not write."""
    assert not re.findall(r"__ldg\b|__restrict__|ld\.global\.nc", code(name))
