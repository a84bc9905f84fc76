"""The 8-bit chain without a GPU: what its sources and entry points have to keep to."""
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "signed_gradient_rounding_b200", "csrc")


def code(name):
    with open(os.path.join(CSRC, name)) as f:
        text = f.read()
    return re.sub(r"//[^\n]*|/\*.*?\*/", "", text, flags=re.S)


@pytest.mark.parametrize("name", ["scaled_rows.cu", "scaled_product.cu"])
def test_overlapped_launches_read_nothing_as_constant(name):
    """A launch of the chain begins while the one before it still writes: no load may go through the
    read-only path, and every kernel waits before anything else it does to memory."""
    text = code(name)
    assert not re.findall(r"__ldg\w*|\.nc\b|__restrict__", text)
    kernels = re.findall(r"__global__ void.*?\n}\n", text, flags=re.S)
    assert kernels and all(len(re.findall(r"\bchain_wait\(\)", k)) == 1 for k in kernels)
