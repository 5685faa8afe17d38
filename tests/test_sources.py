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


def arguments(text, call):
    """The arguments of each ``call(...)`` in the text."""
    for m in re.finditer(r"\b%s\(" % call, text):
        depth, args = 1, [""]
        for c in text[m.end():]:
            depth += (c == "(") - (c == ")")
            if depth == 0:
                break
            if c == "," and depth == 1:
                args.append("")
            else:
                args[-1] += c
        yield [a.strip() for a in args]


def test_weights_have_no_sums_that_may_be_fused():
    """The assembler may round a packed product and its sum at once in one inlined copy
    and not in another. A row's sums and its draw use several copies of the weights,
    which have to agree bit by bit: no packed sum takes a packed product."""
    text = code("sample.cu")
    text = text[text.index("void weight2("):text.index("uint64_t weight(Weigher")]
    products = set(re.findall(r"(\w+) = mul2\(", text))
    assert products
    for args in arguments(text, "add2"):
        for a in args:
            assert a not in products and not a.startswith("mul2("), args
