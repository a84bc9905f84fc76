"""GPU tests of single calls of the 8-bit chain: values at the ends of the range, empty and
overlapping tensors, the memory of calls on a given stream.  Formulas in 64 bits, roundings in
units u = 2^-24 as in test_gpu_scaled.py.
"""
import pytest
import torch

pytestmark = pytest.mark.gpu

U = 2.0 ** -24


@pytest.fixture(scope="module")
def ar():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import signed_gradient_rounding_b200 as ar
    return ar


def bf16_between(lo, hi):
    """Every bf16 number from lo to hi, [n, 1]."""
    bits = torch.arange(1 << 16, dtype=torch.int32, device="cuda").to(torch.int16)
    x = bits.view(torch.bfloat16)
    return x[(x >= lo) & (x <= hi)][:, None]


@pytest.mark.parametrize("cols", [8, 1])  # 16-byte accesses, and columns one by one
def test_silu_mul_scaled_over_its_range(ar, cols):
    """Rows of one value each: the row's scale is |silu(a) b| / 448, so it shows the value itself in fp32.

    u-units: the argument f log2(e) - 7 rounded once (at most (|f| log2(e) + 7) ln 2 < |f| + 5), log2(e)
    itself |f| / 2, the exponential 4, the sum 1, the reciprocal 2, three products 3, the scale's
    division 1: 16 + 1.5 |f|.  A silu below the smallest normal number, 2^-126, may come out as 0."""
    a = bf16_between(-300.0, 300.0)
    b = torch.where(a < 0, 2.0 ** 100, -1.0).to(torch.bfloat16)  # (so that the scale is a normal number)
    q, s = ar.silu_mul_scaled(a.expand(-1, cols).contiguous(), b.expand(-1, cols).contiguous())
    silu = a.double() * torch.sigmoid(a.double())
    v = silu * b.double()
    zero = (q.float() == 0).all(1, keepdim=True)
    got = torch.where(zero, 0.0, s.double() * 448)
    off = (got - v.abs()).abs() - v.abs() * (16 + 1.5 * a.double().abs()) * U
    off = torch.where(silu.abs() < 2.0 ** -126, (got - v.abs()).abs() - 2.0 ** -126 * b.double().abs(), off)
    # (values whose scale is not a normal number are left out: near 0, v / 448 below 2^-126)
    off = off[v.abs() / 448 >= 2.0 ** -126]
    assert off.numel() > 30000 and (off <= 0).all(), (int((off > 0).sum()), a[v.abs() / 448 >= 2.0 ** -126][off.argmax()].item())
    sign = torch.sign(q.float()) * torch.sign(v).float()
    assert ((sign >= 0) & ((sign > 0) | zero)).all()


def test_silu_left_end_in_a_block_of_its_own(ar):
    """A block that holds nothing but the far left of silu, with large and small gates."""
    a = torch.linspace(-88.5, -87.5, 128, device="cuda").to(torch.bfloat16).repeat(2, 1)
    b = torch.full_like(a, 1.0)
    b[1] = 1e38
    q, s = ar.silu_mul_scaled(a, b)
    v = a.double() * torch.sigmoid(a.double()) * b.double()
    top = v.abs().amax(1, keepdim=True) / 448
    # row 0: v / 448 is subnormal, a multiple of 2^-149
    assert ((s.double() - top).abs() <= top * 150 * U + 2.0 ** -149).all()
    u = v / s.double()
    assert ((q.double() - u).abs() <= u.abs() * (2.0 ** -4 + 300 * U)).all()


@pytest.mark.parametrize("rows,cols", [(0, 512), (3, 0), (0, 0)])
def test_empty_batches(ar, rows, cols):
    """No rows or no columns: every call returns at once, the norm with the residual in place among them."""
    x, r = (torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for sum_out in (None, r, torch.empty_like(r)):
        y, q, s, h = ar.rms_norm(x, None, 1e-6, residual=r, want_scaled=True, sum_out=sum_out)
        assert y.shape == q.shape == h.shape == (rows, cols) and s.shape == (rows, (cols + 127) // 128)
        assert sum_out is None or h is sum_out
    for block_rows in (1, 128):
        q, s = ar.quant_scaled(x, block_rows)
        assert q.shape == (rows, cols) and s.shape == (-(-rows // block_rows), (cols + 127) // 128)
    assert ar.silu_mul_scaled(x, r)[0].shape == (rows, cols)


def test_products_of_no_rows(ar):
    w = torch.ones(2, 24, 512, dtype=torch.bfloat16, device="cuda")
    wq, ws = ar.quant_scaled(w, 128)
    x = torch.empty(0, 512, dtype=torch.bfloat16, device="cuda")
    q, s = ar.quant_scaled(x)
    offsets = torch.zeros(3, dtype=torch.int32, device="cuda")
    add, out = (torch.empty(0, 24, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for o in (None, out):
        assert ar.linear_scaled(q, s, wq[0], ws[0], out=o).shape == (0, 24)
        assert ar.linear_scaled(q, s, wq[0], ws[0], add=add, out=o).shape == (0, 24)
        assert ar.grouped_linear(x, offsets, w, out=o).shape == (0, 24)
        assert ar.grouped_linear_scaled(q, s, offsets, wq, ws, out=o).shape == (0, 24)
    assert ar.linear_scaled(q, s, wq[0], ws[0], add=add, out=add) is add
