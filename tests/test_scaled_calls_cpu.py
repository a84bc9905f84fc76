"""The 8-bit chain without a GPU: what its sources and entry points have to keep to."""
import ctypes
import os
import re

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "signed_gradient_rounding_b200", "csrc")

P = ctypes.c_void_p(4096)      # never dereferenced: every call here is refused first
EUNSUPPORTED = 2


@pytest.fixture(scope="module")
def ar():
    import signed_gradient_rounding_b200 as ar
    return ar


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


@pytest.mark.parametrize("out", [1 << 31, 1 << 54, (1 << 54) + 8, 1 << 62])
@pytest.mark.parametrize("experts", [1, 2, 1024])
def test_sizes_whose_product_overflows_are_refused(ar, out, experts):
    """experts * out past 64 bits: 1024 * 2^54 is 0 there."""
    assert ar.lib.ar_grouped_linear(P, 256, 4, 256, P, experts, P, None, 256, out, P, out, None, None) == EUNSUPPORTED
    assert ar.lib.ar_grouped_linear_scaled(P, 256, P, 4, 256, P, experts, P, 256, P, out, P, out, None, None) == EUNSUPPORTED
    assert ar.lib.ar_linear_scaled(P, 256, P, 4, 256, P, 256, P, out, None, 0, P, out, None, None) == EUNSUPPORTED


def test_row_quantisers_refuse_what_no_grid_holds(ar):
    """2^35 blocks of columns, at 16 a CTA: one CTA more than a grid has."""
    rows = 1 << 30
    assert ar.lib.ar_quant_scaled(P, 1, 1, 32, rows, 1, 1, P, 1, P, None) == EUNSUPPORTED
    assert ar.lib.ar_quant_scaled(P, 1, 4096, 1, rows, 4096, 1, P, 4096, P, None) == EUNSUPPORTED
    assert ar.lib.ar_silu_mul_scaled(P, 4095, P, 4095, rows, 4095, P, 4095, P, None) == EUNSUPPORTED
