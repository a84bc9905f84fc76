"""GPU parity of the 8-bit chain (rms_norm, quant_scaled, silu_mul_scaled, linear_scaled,
grouped_linear, grouped_linear_scaled) against the formulas in 64 bits.

Tolerances, from the roundings alone (u = 2^-24, half a step of fp32):
  * a value rounded once to bf16: 2^-8 of it; to e4m3: 2^-4 of it, or half the
    subnormal step, 2^-10;
  * RMS norm: a thread's chain of at most 32 squares, 10 shuffle additions, then the mean, eps,
    a square root, a division and two products: under 64 u = 2^-18 of each value, with the
    root halving the sum's share;
  * silu(a) * b: exp(-a) = 2^(-a log2(e)) with the argument rounded once and log2(e) rounded once:
    |a| log2(e) (u + u/2) ln 2 < 2 |a| u relative; the hardware's 2^x, the sum, the
    reciprocal and the two products are off by less than 8 u = 2^-21 (each of the first and
    the third within 2 units);
  * products: each block of 128 on the tensor cores within 2^-19 of the sum of its |terms|
    (the bound this library's other products are held to), and one fp32 operation per
    block of K and per share of K: at most (blocks + 16) u of that sum.
"""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu

BF16, E4M3, SUB = 2.0 ** -8, 2.0 ** -4, 2.0 ** -10
U = 2.0 ** -24
NORM_EPS, SILU_EPS = 2.0 ** -18, 2.0 ** -21
TINY = 2.0 ** -133                # half the smallest bf16 step


@pytest.fixture(scope="module")
def ar():
    assert torch.cuda.is_available(), "GPU tests need a CUDA device"
    import signed_gradient_rounding_b200 as ar
    return ar


def rand(seed, *shape, std=1.0, dtype=torch.bfloat16):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x = torch.randn(*shape, generator=gen, device="cuda") * std
    if shape[-1] >= 8:
        x[..., torch.randint(shape[-1], (1 + shape[-1] // 100,), generator=gen, device="cuda")] *= 20
    return x.to(dtype)


def pitched(x, pad):
    """The same matrix as a slice of wider rows (whose other columns are NaN)."""
    wide = torch.full((*x.shape[:-1], x.shape[-1] + pad), float("nan"), dtype=torch.float32, device="cuda").to(x.dtype)
    wide[..., :x.shape[-1]] = x
    return wide[..., :x.shape[-1]]


def nblk(n):
    return (n + 127) // 128


def block_amax(v, block_rows):
    rows, cols = v.shape
    pad = torch.nn.functional.pad(v.abs(), (0, -cols % 128, 0, -rows % block_rows))
    return pad.view(pad.shape[0] // block_rows, block_rows, nblk(cols), 128).amax((1, 3))


def spread(s, block_rows, rows, cols):
    return s.repeat_interleave(block_rows, 0)[:rows].repeat_interleave(128, 1)[:, :cols]


def plain_quant(x, block_rows=1):
    """The definition in fp32, on the CPU (IEEE operations): bit-exact."""
    x = x.float().cpu()
    s = block_amax(x, block_rows) / torch.tensor(448.0)
    s = torch.where(s == 0, torch.ones_like(s), s)
    u = x / spread(s, block_rows, *x.shape)
    return u.clamp(-448, 448).to(torch.float8_e4m3fn), s


def same(a, b):
    """Equal values, NaN in the same places."""
    return torch.allclose(a.double().cpu(), b.double().cpu(), rtol=0, atol=0, equal_nan=True)


def check_scaled(q, scale, v64, rel):
    """(q, scale) of values known in 64 bits, themselves off by at most `rel` in the kernel."""
    s64 = block_amax(v64, 1) / 448
    s64[s64 == 0] = 1
    assert ((scale.double() - s64).abs() <= s64 * (rel + 2 * U)).all()
    u = v64 / spread(s64, 1, *v64.shape)
    off = (q.double() - u).abs() - (u.abs() * (E4M3 + 4 * rel + 8 * U) + SUB)
    assert (off <= 0).all(), f"{int((off > 0).sum())} codes off, worst by {off.max().item()}"


# ---------------------------------------------------------------------------
# Quantisers
# ---------------------------------------------------------------------------

@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (3, 127), (5, 129), (7, 1000), (33, 4096), (129, 11008), (2, 29568)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
@pytest.mark.parametrize("pad", [0, 3, 8])
def test_quant_rows_bit_exact(ar, rows, cols, dtype, pad):
    x = pitched(rand(rows + cols, rows, cols, dtype=dtype), pad) if pad else rand(rows + cols, rows, cols, dtype=dtype)
    q, s = ar.quant_scaled(x)
    qr, sr = plain_quant(x)
    assert torch.equal(s.cpu(), sr)
    assert torch.equal(q.float().cpu(), qr.float())


@pytest.mark.parametrize("shape", [(1, 1), (128, 128), (130, 300), (256, 4096), (77, 129), (3, 64, 256), (5, 200, 130)])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float32])
def test_quant_tiles_bit_exact(ar, shape, dtype):
    x = rand(sum(shape), *shape, std=0.02, dtype=dtype)
    q, s = ar.quant_scaled(x, block_rows=128)
    assert q.shape == x.shape and s.shape == (*shape[:-2], nblk(shape[-2]), nblk(shape[-1]))
    for m in range(shape[0] if len(shape) == 3 else 1):
        pick = (lambda t: t[m]) if len(shape) == 3 else (lambda t: t)
        qr, sr = plain_quant(pick(x), 128)
        assert torch.equal(pick(s).cpu(), sr)
        assert torch.equal(pick(q).float().cpu(), qr.float())


def test_quant_many_scales(ar):
    """A million blocks whose maxima spread over the whole range: every scale and code against torch's
    division (correctly rounded)."""
    gen = torch.Generator(device="cuda").manual_seed(5)
    x = torch.randn(1 << 13, 1 << 14, generator=gen, device="cuda")
    size = torch.exp2(torch.rand(1 << 13, 1 << 7, 1, generator=gen, device="cuda") * 220 - 120)
    x = (x.view(1 << 13, 1 << 7, 128) * size).reshape(x.shape)
    q, s = ar.quant_scaled(x)
    top = x.view(1 << 13, 1 << 7, 128).abs().amax(2)
    assert torch.equal(s, top / torch.full_like(top, 448.0))
    u = x.view(1 << 13, 1 << 7, 128) / s[..., None]
    assert torch.equal(q.float().view_as(u), u.clamp(-448, 448).to(torch.float8_e4m3fn).float())


@pytest.mark.parametrize("block_rows", [1, 128])
def test_quant_special_values(ar, block_rows):
    """Zero, denormal and huge blocks, ties, a NaN (stays in its place) and an infinity."""
    x = rand(1, 4, 1024, dtype=torch.float32)
    x[:, 0:128] = 0
    x[:, 128:256] *= 1e-40
    x[:, 256:384] *= 1e37
    x[:, 384:512] = torch.arange(128, device="cuda") * 0.25      # amax 31.75
    x[:, 511] = 448.0                                            # scale 1: many exact ties
    x[:, 512:640] *= 2.0 ** -85                                  # around the fast division's border
    x[:, 640:768] *= 1e-30
    x[1, 770] = float("nan")
    q, s = ar.quant_scaled(x, block_rows)
    clean = x.clone()
    clean[1, 770] = 0
    qr, sr = plain_quant(clean, block_rows)     # (one value of the huge blocks is an infinity already)
    assert same(s, sr)
    got = q.float()
    assert torch.isnan(got[1, 770])
    got[1, 770] = 0
    assert same(got, qr)
    x[1, 770] = float("-inf")
    q, s = ar.quant_scaled(x, block_rows)
    assert torch.isinf((s[1] if block_rows == 1 else s[0])[6])
    assert torch.isnan(q.double()[1, 768:896] * spread(s, block_rows, 4, 1024).double()[1, 768:896]).all()
    assert same(q[:, :768], qr[:, :768]) and same(q[:, 896:], qr[:, 896:]) and same(s[:, :6], sr[:, :6])


@pytest.mark.parametrize("rows,cols", [(1, 8), (7, 11008), (3, 130), (65, 4096), (2, 77)])
@pytest.mark.parametrize("fused", [False, True])
def test_silu_mul_scaled(ar, rows, cols, fused):
    a, b = rand(cols, rows, cols, std=3.0), rand(cols + 1, rows, cols)
    if fused:  # the two halves of one gate-and-up output
        both = torch.cat([a, b], 1)
        a, b = both[:, :cols], both[:, cols:]
    q, s = ar.silu_mul_scaled(a, b)
    # an element's own |a| counts; the block's scale is its largest element's
    check_scaled(q, s, a.double() * torch.sigmoid(a.double()) * b.double(), SILU_EPS + 2 * a.abs().max().item() * U)


def test_silu_far_ends(ar):
    """silu at the ends of the range: -0 to the left, the value itself to the right."""
    a = torch.tensor([[-1e38, -200.0, -90.0, -88.5, -80.0, 0.0, 88.0, 200.0]], device="cuda").to(torch.bfloat16)
    b = torch.ones_like(a)
    q, s = ar.silu_mul_scaled(a, b)
    check_scaled(q, s, a.double() * torch.sigmoid(a.double()), SILU_EPS + 2 * 200 * U)  # (past 200, exp is 0 or infinite)


# ---------------------------------------------------------------------------
# RMS norm
# ---------------------------------------------------------------------------

def check_norm(ar, x, r, w, eps, inplace=False):
    h64 = x.double() if r is None else x.double() + r.double()
    v64 = h64 / (h64.square().mean(1, keepdim=True) + eps).sqrt()
    if w is not None:
        v64 = v64 * w.double()
    y, q, s, h = ar.rms_norm(x, w, eps, residual=r, want_scaled=True, sum_out=r if inplace else None)
    assert ((y.double() - v64).abs() <= v64.abs() * (BF16 + NORM_EPS) + TINY).all()
    check_scaled(q, s, v64, NORM_EPS)
    if r is None:
        assert h is None
    elif r.dtype == torch.bfloat16:
        assert ((h.double() - h64).abs() <= h64.abs() * (BF16 + 2 * U) + TINY).all()
    else:
        assert ((h.double() - h64).abs() <= h64.abs() * U).all()
    if inplace:
        assert h is r


@pytest.mark.parametrize("rows,cols", [(1, 1), (1, 128), (2, 100), (9, 256), (3, 257), (5, 1024), (4, 1032), (1, 4096), (300, 4096),
                                       (2, 8192), (3, 8200), (2, 11008), (2, 11264), (3, 11272), (2, 16384), (2, 29568), (1, 32768),
                                       (2, 32767), (500, 12000)])
@pytest.mark.parametrize("res", [None, torch.bfloat16, torch.float32])
@pytest.mark.parametrize("xt", [torch.bfloat16, torch.float32])
def test_rms_norm(ar, rows, cols, res, xt):
    x = rand(1, rows, cols, dtype=xt)
    r = None if res is None else rand(2, rows, cols, std=4.0, dtype=res)
    w = (1 + 0.2 * torch.randn(cols, device="cuda")).to(torch.bfloat16)
    check_norm(ar, x, r, w, 1e-5)


@pytest.mark.parametrize("cols", [256, 4096, 4100])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_rms_norm_pitches_weights_in_place(ar, cols, res):
    x, r = pitched(rand(3, 5, cols), 8), pitched(rand(4, 5, cols, dtype=res), 5)
    check_norm(ar, x, r, None, 0.0)
    w = 1 + 0.2 * torch.randn(cols, device="cuda")
    check_norm(ar, x, r, w, 1e-6)
    check_norm(ar, x, r, w, 1e-6, inplace=True)


def test_rms_norm_rows_of_zeros_and_outputs(ar):
    x = torch.zeros(3, 512, dtype=torch.bfloat16, device="cuda")
    x[1] = rand(1, 512)
    y, q, s, h = ar.rms_norm(x, None, 1e-6, want_scaled=True)
    assert h is None and (y[0] == 0).all() and (q[2].float() == 0).all() and (s[0] == 1).all()
    y, q, s, h = ar.rms_norm(x, None, 1e-6, residual=x, want_bf16=False)
    assert y is None and q is None and s is None and torch.equal(h, x + x)
    with pytest.raises(ar.ArError):
        ar.rms_norm(x, None, 1e-6, want_bf16=False)
    y, q, s, h = ar.rms_norm(x[:0], None, 1e-6, want_scaled=True)
    assert y.shape == (0, 512) and s.shape == (0, 4)


# ---------------------------------------------------------------------------
# Products
# ---------------------------------------------------------------------------

def scaled_operands(ar, n, inn, out, seed, experts=None):
    xq, xs = ar.quant_scaled(rand(seed, n, inn))
    w = rand(seed + 1, *((out, inn) if experts is None else (experts, out, inn)), std=0.02)
    wq, ws = ar.quant_scaled(w, block_rows=128)
    return xq, xs, wq, ws


def read_rows(q, s):
    return q.double() * spread(s.double(), 1, *q.shape)


def read_tiles(q, s):
    return q.double() * spread(s.double(), 128, *q.shape)


def check_product(Y, x64, w64, nb, add=None):
    ref = x64 @ w64.T
    terms = x64.abs() @ w64.abs().T
    if add is not None:
        ref = ref + add.double()
        terms = terms + add.double().abs()
    off = (Y.double() - ref).abs() - (ref.abs() * BF16 + terms * (2.0 ** -19 + (nb + 16) * U) + TINY)
    assert (off <= 0).all(), f"{int((off > 0).sum())} of {off.numel()} off, worst by {off.max().item()}"


@pytest.mark.parametrize("n", [1, 3, 8, 9, 17, 33, 64, 65, 130, 257, 600])
@pytest.mark.parametrize("inn,out", [(16, 8), (128, 128), (272, 129), (1040, 1), (4096, 384), (400, 77), (11008, 264)])
def test_linear_scaled(ar, n, inn, out):
    xq, xs, wq, ws = scaled_operands(ar, n, inn, out, n + inn)
    add = rand(5, n, out) if (n + out) % 2 else None
    Y = ar.linear_scaled(xq, xs, wq, ws, add=add)
    check_product(Y, read_rows(xq, xs), read_tiles(wq, ws), nblk(inn), add)
    assert torch.equal(Y, ar.linear_scaled(xq, xs, wq, ws, add=add))


@pytest.mark.parametrize("n,inn,out", [(1, 29568, 8192), (300, 29568, 1000), (5000, 4096, 1032), (2100, 512, 4096),
                                       (40, 4096, 4096), (128, 4096, 4096), (1000, 4096, 4096)])
def test_linear_scaled_large(ar, n, inn, out):
    xq, xs, wq, ws = scaled_operands(ar, n, inn, out, n)
    Y = ar.linear_scaled(xq, xs, wq, ws)
    check_product(Y, read_rows(xq, xs), read_tiles(wq, ws), nblk(inn))


@pytest.mark.parametrize("n", [2, 20, 200])
@pytest.mark.parametrize("out", [136, 131])
def test_linear_scaled_pitches(ar, n, out):
    """Operands, residual and output as slices of wider rows; the columns beside the output stay."""
    xq, xs, wq, ws = scaled_operands(ar, n, 528, out, 9)
    add = pitched(rand(6, n, out), 13)
    wide = torch.full((n, out + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    Y = ar.linear_scaled(pitched(xq, 32), xs, pitched(wq, 16), ws, add=add, out=wide[:, 8:8 + out])
    check_product(Y, read_rows(xq, xs), read_tiles(wq, ws), nblk(528), add)
    assert (wide[:, :8] == 7).all() and (wide[:, 8 + out:] == 7).all()
    # the residual stream updated in place
    stream = add.clone()
    ar.linear_scaled(xq, xs, wq, ws, add=stream, out=stream)
    assert torch.equal(stream, Y)


@pytest.mark.parametrize("n,inn", [(3, 1040), (200, 1040), (200, 1152), (600, 144), (70, 4112)])
def test_linear_scaled_slice_of_a_batch(ar, n, inn):
    """Some rows of a batch: scales that start on any of the 4-byte places of a 16-byte unit."""
    xq, xs, wq, ws = scaled_operands(ar, n + 3, inn, 264, 3)
    for first in range(4):
        rows = slice(first, first + n - 1)
        Y = ar.linear_scaled(xq[rows], xs[rows], wq, ws)
        check_product(Y, read_rows(xq[rows], xs[rows]), read_tiles(wq, ws), nblk(inn))


COUNTS = {
    "one": [5],
    "decode": [0, 1, 0, 3, 1, 0, 0, 2, 9],
    "empty": [0, 0, 0],
    "ragged": [1, 0, 130, 17, 128, 0, 300, 64, 5],
    "skewed": [700, 0, 1, 2],
    "many": [(7 * i) % 5 for i in range(70)],
}


def offsets_of(counts):
    return torch.tensor([0] + counts, device="cuda").cumsum(0).to(torch.int32)


@pytest.mark.parametrize("kind", ["bf16", "pair", "scaled"])
@pytest.mark.parametrize("counts", list(COUNTS))
@pytest.mark.parametrize("inn,out,pad", [(16, 8, 0), (272, 131, 3), (1040, 256, 200), (2048, 129, 1)])
def test_grouped(ar, kind, counts, inn, out, pad):
    """Every expert's rows against its own weight; the rows behind the last expert's stay."""
    counts = COUNTS[counts]
    rows, experts = sum(counts), len(counts)
    n = rows + pad
    offsets = offsets_of(counts)
    Y = torch.full((n, out), 3.0, dtype=torch.bfloat16, device="cuda")
    if kind == "scaled":
        xq, xs, wq, ws = scaled_operands(ar, n, inn, out, rows, experts)
        got = ar.grouped_linear_scaled(xq, xs, offsets, wq, ws, out=Y)
        x64 = read_rows(xq, xs)
    else:
        x, w = rand(rows, n, inn), rand(rows + 1, experts, out, inn, std=0.02, dtype=torch.float32)
        hi = w.to(torch.bfloat16)
        lo = (w - hi.float()).to(torch.bfloat16) if kind == "pair" else None
        got = ar.grouped_linear(x, offsets, hi, lo, out=Y)
        x64 = x.double()
    assert got is Y and (Y[rows:] == 3).all()
    at = 0
    for e, c in enumerate(counts):
        if kind == "scaled":
            w64 = read_tiles(wq[e], ws[e])
        else:
            w64 = hi[e].double() + (lo[e].double() if lo is not None else 0)
        check_product(Y[at:at + c], x64[at:at + c], w64, nblk(2 * inn) * 2)
        at += c


@pytest.mark.parametrize("kind", ["bf16", "scaled"])
def test_grouped_pitches(ar, kind):
    counts = [40, 0, 90, 3]
    n, inn, out = sum(counts), 272, 136
    offsets = offsets_of(counts)
    wide = torch.full((n, out + 24), 7.0, dtype=torch.bfloat16, device="cuda")
    if kind == "scaled":
        xq, xs, wq, ws = scaled_operands(ar, n, inn, out, 3, len(counts))
        ref = ar.grouped_linear_scaled(xq, xs, offsets, wq, ws)
        Y = ar.grouped_linear_scaled(pitched(xq, 16), xs, offsets, pitched(wq, 32), ws, out=wide[:, 5:5 + out])
    else:
        x, w = rand(1, n, inn), rand(2, len(counts), out, inn, std=0.02)
        ref = ar.grouped_linear(x, offsets, w)
        Y = ar.grouped_linear(pitched(x, 8), offsets, pitched(w, 16), out=wide[:, 5:5 + out])
    assert torch.equal(Y, ref)
    assert (wide[:, :5] == 7).all() and (wide[:, 5 + out:] == 7).all()


@pytest.mark.parametrize("n", [16, 400])
def test_grouped_same_as_dense(ar, n):
    """One expert with all rows is the dense product, to the bit."""
    xq, xs, wq, ws = scaled_operands(ar, n, 1024, 264, 4)
    dense = ar.linear_scaled(xq, xs, wq, ws)
    grouped = ar.grouped_linear_scaled(xq, xs, offsets_of([n]), wq[None], ws[None])
    assert torch.equal(dense, grouped)


def test_products_keep_nonfinite_values_to_their_rows(ar):
    """A NaN or an infinity in a row of X reaches that row of Y alone (of its own expert's weight)."""
    counts = [3, 150, 60]
    x, w = rand(1, sum(counts), 256), rand(2, 3, 200, 256, std=0.02)
    offsets = offsets_of(counts)
    ref = ar.grouped_linear(x, offsets, w)
    bad = x.clone()
    bad[2, 17] = float("nan")
    bad[160, 3] = float("inf")
    Y = ar.grouped_linear(bad, offsets, w)
    keep = torch.ones(sum(counts), dtype=torch.bool, device="cuda")
    keep[[2, 160]] = False
    assert torch.equal(Y[keep], ref[keep]) and torch.isnan(Y[2]).all() and not torch.isfinite(Y[160]).any()
    w2 = w.clone()
    w2[1] = float("nan")
    Y = ar.grouped_linear(x, offsets, w2)
    assert torch.equal(Y[:3], ref[:3]) and torch.equal(Y[153:], ref[153:]) and torch.isnan(Y[3:153]).all()


# ---------------------------------------------------------------------------
# Long tensors: element offsets past 32 bits
# ---------------------------------------------------------------------------

def test_offsets_past_32_bits(ar):
    n, inn, out = 70001, 16, 32768                      # Y: 2.3e9 elements
    xq, xs, wq, ws = scaled_operands(ar, n, inn, out, 1)
    Y = ar.linear_scaled(xq, xs, wq, ws)
    check_product(Y[-130:], read_rows(xq[-130:], xs[-130:]), read_tiles(wq, ws), 1)
    q, s = ar.silu_mul_scaled(Y, Y)
    y64 = Y[-3:].double()
    check_scaled(q[-3:], s[-3:], y64 * torch.sigmoid(y64) * y64, SILU_EPS + 2 * y64.abs().max().item() * U)
    del q, s
    v, _, _, _ = ar.rms_norm(Y, None, 1e-6)
    v64 = y64 / (y64.square().mean(1, keepdim=True) + 1e-6).sqrt()
    assert ((v[-3:].double() - v64).abs() <= v64.abs() * (BF16 + NORM_EPS) + TINY).all()


# ---------------------------------------------------------------------------
# Together: a decoder layer's MLP, dense and by expert
# ---------------------------------------------------------------------------

def layer(ar, x, stream, w):
    """norm (residual in place) -> gate-and-up by expert -> silu*mul -> down by expert -> dense output + residual."""
    _, q, s, h = ar.rms_norm(x, w["norm"], 1e-6, residual=stream, want_bf16=False, want_scaled=True)
    gu = ar.grouped_linear_scaled(q, s, w["offsets"], *w["gate_up"])
    half = gu.shape[1] // 2
    q2, s2 = ar.silu_mul_scaled(gu[:, :half], gu[:, half:])
    d = ar.grouped_linear_scaled(q2, s2, w["offsets"], *w["down"])
    q3, s3 = ar.quant_scaled(d)
    return ar.linear_scaled(q3, s3, *w["o"], add=h), (q, s, gu, q2, s2, d, q3, s3, h)


def layer_weights(ar, hidden, inter, counts):
    return dict(norm=(1 + 0.1 * torch.randn(hidden, device="cuda")).to(torch.bfloat16), offsets=offsets_of(counts),
                gate_up=ar.quant_scaled(rand(1, len(counts), 2 * inter, hidden, std=0.02), 128),
                down=ar.quant_scaled(rand(2, len(counts), hidden, inter, std=0.02), 128),
                o=ar.quant_scaled(rand(3, hidden, hidden, std=0.02), 128))


@pytest.mark.parametrize("counts", [[1, 0, 2, 1], [100, 3, 0, 61], [300, 200, 1, 99]])
def test_layer_together(ar, counts):
    hidden, inter, n = 512, 384, sum(counts)
    w = layer_weights(ar, hidden, inter, counts)
    x, r = rand(7, n, hidden), rand(8, n, hidden)
    y, (q, s, gu, q2, s2, d, q3, s3, h) = layer(ar, x, r, w)
    # every step against its formula on the bytes the step before it gave
    h64 = x.double() + r.double()
    v64 = h64 / (h64.square().mean(1, keepdim=True) + 1e-6).sqrt() * w["norm"].double()
    check_scaled(q, s, v64, NORM_EPS)
    at = 0
    for e, c in enumerate(counts):
        rows = slice(at, at + c)
        check_product(gu[rows], read_rows(q[rows], s[rows]), read_tiles(w["gate_up"][0][e], w["gate_up"][1][e]), 4)
        check_product(d[rows], read_rows(q2[rows], s2[rows]), read_tiles(w["down"][0][e], w["down"][1][e]), 3)
        at += c
    g64 = gu[:, :inter].double()
    check_scaled(q2, s2, g64 * torch.sigmoid(g64) * gu[:, inter:].double(), SILU_EPS + 2 * g64.abs().max().item() * U)
    check_product(y, read_rows(q3, s3), read_tiles(*w["o"]), 4, h)


def test_layer_captured_and_on_another_stream(ar):
    """A captured layer replays to the same bits on new inputs in its buffers; so does a run on a side stream."""
    counts = [30, 0, 5, 200]
    w = layer_weights(ar, 512, 256, counts)
    x, r = rand(1, sum(counts), 512), rand(2, sum(counts), 512)
    x2, r2 = rand(3, sum(counts), 512), rand(4, sum(counts), 512)
    want, want2 = layer(ar, x, r, w)[0].clone(), layer(ar, x2, r2, w)[0].clone()
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        got = layer(ar, x, r, w)[0]
    torch.cuda.current_stream().wait_stream(side)
    assert torch.equal(got, want)
    xb, rb = x.clone(), r.clone()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = layer(ar, xb, rb, w)[0]
    graph.replay()
    assert torch.equal(out, want)
    xb.copy_(x2)
    rb.copy_(r2)
    graph.replay()
    assert torch.equal(out, want2)


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("n,inn,out", [(2048, 128, 2300), (1100, 256, 3901), (2000, 1152, 301), (150, 8192, 603), (600, 2176, 1502),
                                       (150, 8192, 2)])
def test_rows_of_the_output_at_every_offset(ar, n, inn, out, kind):
    """Y and the residual at any distance from a 16-byte boundary, over the tiles' shapes and splits: the
    values of an aligned call, and nothing beside the rows."""
    wide = (out + 7) // 8 * 8
    x, w, res = rand(1, n, inn), rand(2, wide, inn, std=0.05), rand(3, n, wide)
    if kind == "scaled":
        xq, wq = ar.quant_scaled(x), ar.quant_scaled(w, 128)
        ws = wq[1][:(out + 127) // 128]

        def run(o, **kw):
            return ar.linear_scaled(*xq, wq[0][:o], wq[1] if o == wide else ws, **kw)
    else:
        offsets = torch.tensor([0, n], dtype=torch.int32, device="cuda")

        def run(o, add=None, **kw):
            return ar.grouped_linear(x, offsets, w[None, :o], **kw)
    plain, added = run(wide), run(wide, add=res)
    for y_off, add_off, gap in [(0, 1, 3), (1, 0, 0), (3, 3, 8), (7, 2, 1), (2, 7, 2), (4, 5, 4), (5, 4, 16), (6, 6, 9), (1, None, 5)]:
        buf = torch.full((n * (out + gap) + 16,), 7.0, dtype=torch.bfloat16, device="cuda")
        y = buf[y_off:].as_strided((n, out), (out + gap, 1))
        add = None
        if add_off is not None:
            add = torch.zeros(n * (out + 3) + 16, dtype=torch.bfloat16, device="cuda")[add_off:].as_strided((n, out), (out + 3, 1))
            add.copy_(res[:, :out])
        run(out, add=add, out=y)
        assert torch.equal(y, (plain if add is None else added)[:, :out]), (y_off, add_off, gap)
        y.fill_(7.0)
        assert bool((buf == 7.0).all()), (y_off, add_off, gap)


def test_launches_in_a_row_are_ordered(ar):
    """Layers back to back, each over the buffers of the one before: as with a synchronisation between
    them, in a stream and in a graph (the launches overlap their starts)."""
    counts = [300, 0, 17, 99]
    w = layer_weights(ar, 512, 256, counts)
    xs, rs = [rand(i, sum(counts), 512) for i in range(6)], [rand(9 + i, sum(counts), 512) for i in range(6)]
    want = []
    for x, r in zip(xs, rs):
        torch.cuda.synchronize()
        want.append(layer(ar, x, r, w)[0])
    torch.cuda.synchronize()
    xb, rb = torch.empty_like(xs[0]), torch.empty_like(rs[0])

    def chain():
        out = []
        for x, r in zip(xs, rs):
            xb.copy_(x)
            rb.copy_(r)
            out.append(layer(ar, xb, rb, w)[0])
        return out

    for _ in range(20):
        assert all(torch.equal(a, b) for a, b in zip(chain(), want))
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        out = chain()
    for _ in range(10):
        for y in out:
            y.zero_()
        graph.replay()
        assert all(torch.equal(a, b) for a, b in zip(out, want))


def test_launches_on_a_forked_stream_in_a_graph(ar):
    """A captured launch whose result two streams read, joined again: the overlapped starts keep both orders."""
    x, w = rand(3, 64, 512), rand(4, 512)
    want_v = ar.rms_norm(x, w)[0]
    want_q = ar.quant_scaled(want_v)[0]
    want_z = ar.rms_norm(want_v, w)[0]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        v = ar.rms_norm(x, w)[0]
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        with torch.cuda.stream(side):
            q = ar.quant_scaled(v)[0]
        z = ar.rms_norm(v, w)[0]
        here.wait_stream(side)
        last = ar.quant_scaled(z)[0]
    for _ in range(5):
        for t in (v, z):
            t.zero_()
        q.view(torch.uint8).zero_()
        last.view(torch.uint8).zero_()
        graph.replay()
        assert torch.equal(v, want_v) and torch.equal(z, want_z)
        assert torch.equal(q.view(torch.uint8), want_q.view(torch.uint8))
        assert torch.equal(last.view(torch.uint8), ar.quant_scaled(want_z)[0].view(torch.uint8))


def test_graph_with_other_offsets(ar):
    """The offsets are read on the device: a captured product follows them."""
    x, w = rand(1, 300, 256), rand(2, 4, 136, 256, std=0.02)
    offsets = offsets_of([100, 0, 150, 50])
    Y = torch.zeros(300, 136, dtype=torch.bfloat16, device="cuda")
    ar.grouped_linear(x, offsets, w, out=Y)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        ar.grouped_linear(x, offsets, w, out=Y)
    for counts in ([0, 300, 0, 0], [10, 20, 30, 40], [0, 0, 0, 0]):
        offsets.copy_(offsets_of(counts))
        Y.fill_(3.0)
        graph.replay()
        at = 0
        for e, c in enumerate(counts):
            check_product(Y[at:at + c], x[at:at + c].double(), w[e].double(), 4)
            at += c
        assert (Y[at:] == 3).all()


FIRST_IN_CAPTURE = """
import torch
import signed_gradient_rounding_b200 as ar
x = torch.randn(300, 512, device="cuda").bfloat16()
w = torch.randn(2, 136, 512, device="cuda").bfloat16()
offsets = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()
with torch.cuda.graph(graph):
    y, q, s, h = ar.rms_norm(x, None, want_scaled=True)
    wq, ws = ar.quant_scaled(w, 128)
    big = ar.grouped_linear_scaled(q, s, offsets, wq, ws)
    one = ar.linear_scaled(q[:1], s[:1], wq[0], ws[0])
    mid = ar.linear_scaled(q, s, wq[1], ws[1])
    half = ar.grouped_linear(y, offsets, w)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in (big, one, mid, half)]
y, q, s, h = ar.rms_norm(x, None, want_scaled=True)
want = (ar.grouped_linear_scaled(q, s, offsets, wq, ws), ar.linear_scaled(q[:1], s[:1], wq[0], ws[0]),
        ar.linear_scaled(q, s, wq[1], ws[1]), ar.grouped_linear(y, offsets, w))
assert all(torch.equal(a, b) for a, b in zip(got, want))
print("captured first")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of every entry point is captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("n", [40, 400])
@pytest.mark.parametrize("offsets", [[0, 10, 5, 30], [-7, 3, 1 << 30, 20], [25, 12, 3, 0], [1 << 30] * 4, [-(1 << 31), -1, 0, 0]])
def test_offsets_that_break_the_rules_stay_inside(ar, n, offsets):
    """Offsets out of range or decreasing: the rows around X and Y are neither read into Y nor written."""
    inn, out = 256, 136
    wide_x = torch.full((n + 256, inn), float("nan"), dtype=torch.bfloat16, device="cuda")
    wide_x[128:128 + n] = rand(1, n, inn)
    wide_y = torch.full((n + 256, out), 3.0, dtype=torch.bfloat16, device="cuda")
    w = rand(2, 3, out, inn, std=0.02)
    ar.grouped_linear(wide_x[128:128 + n], torch.tensor(offsets, dtype=torch.int32, device="cuda"), w,
                      out=wide_y[128:128 + n])
    assert (wide_y[:128] == 3).all() and (wide_y[128 + n:] == 3).all() and torch.isfinite(wide_y).all()


def test_two_calls_at_once(ar):
    """Calls on two streams at once do not disturb each other."""
    a, b = scaled_operands(ar, 300, 2048, 520, 1), scaled_operands(ar, 5, 2048, 520, 2)
    want = ar.linear_scaled(*a), ar.linear_scaled(*b)
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    got = [[], []]
    torch.cuda.synchronize()
    for _ in range(10):
        for i, ops in enumerate((a, b)):
            got[i].append(ar.linear_scaled(*ops, stream=streams[i]))
    torch.cuda.synchronize()
    for i in range(2):
        assert all(torch.equal(y, want[i]) for y in got[i])


def test_stream_argument_keeps_memory(ar):
    """Operands and results of a call on a given stream may be dropped at once: their memory is not
    handed out again while that stream still works on them."""
    ops = scaled_operands(ar, 2000, 4096, 4096, 1)
    want = ar.linear_scaled(*ops)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    results = []
    for _ in range(6):
        copies = [t.clone() for t in ops]
        side.wait_stream(torch.cuda.current_stream())
        for _ in range(3):
            y = ar.linear_scaled(*copies, stream=side)
        results.append(y)
        del copies, y
        for t in ops:  # takes the copies' memory, if it is free
            torch.zeros_like(t, dtype=torch.uint8 if t.dtype == torch.float8_e4m3fn else t.dtype).fill_(127)
    torch.cuda.synchronize()
    assert all(torch.equal(y, want) for y in results)


def test_status_word_stays_zero(ar):
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    ops = scaled_operands(ar, 300, 1024, 520, 1)
    ar.linear_scaled(*ops, status=status)
    assert status.item() == 0


def test_binding_refusals(ar):
    xq, xs, wq, ws = scaled_operands(ar, 8, 256, 64, 1)
    bf = torch.zeros(8, 256, dtype=torch.bfloat16, device="cuda")
    offsets = offsets_of([8])
    bad = [
        lambda: ar.linear_scaled(bf, xs, wq, ws), lambda: ar.linear_scaled(xq, xs[:4], wq, ws),
        lambda: ar.linear_scaled(xq, xs.double(), wq, ws), lambda: ar.linear_scaled(xq, xs, wq[:, :128], ws),
        lambda: ar.linear_scaled(xq, xs, wq, ws[:, :1]), lambda: ar.linear_scaled(xq, xs, wq, ws, add=bf),
        lambda: ar.linear_scaled(xq, xs, wq, ws, out=bf), lambda: ar.linear_scaled(xq.T, xs, wq, ws),
        lambda: ar.linear_scaled(xq, xs, wq, ws, status=bf), lambda: ar.linear_scaled(xq, xs, wq[0], ws),
        lambda: ar.grouped_linear(bf, offsets.long(), bf[None]), lambda: ar.grouped_linear(bf, offsets_of([4, 4]), bf[None]),
        lambda: ar.grouped_linear(bf, offsets, bf), lambda: ar.grouped_linear(bf, offsets, bf[None], bf[None, :4]),
        lambda: ar.grouped_linear_scaled(xq, xs, offsets, wq[None], ws), lambda: ar.rms_norm(bf, bf[0, :128]),
        lambda: ar.rms_norm(bf, None, residual=bf[:4]), lambda: ar.rms_norm(bf, None, sum_out=bf),
        lambda: ar.rms_norm(bf, None, residual=bf, sum_out=bf.float()), lambda: ar.rms_norm(bf, None, residual=bf, sum_out=bf),
        lambda: ar.grouped_linear(bf, offsets, bf[None].repeat(1, 32, 1), out=bf), lambda: ar.rms_norm(bf.half(), None),
        lambda: ar.quant_scaled(bf.half()), lambda: ar.silu_mul_scaled(bf, bf[:, :128]),
        lambda: ar.silu_mul_scaled(bf.float(), bf.float()), lambda: ar.quant_scaled(bf[0]),
    ]
    for i, call in enumerate(bad):
        with pytest.raises(ValueError):
            call()
            pytest.fail(f"call {i} was not refused")
    for call in (lambda: ar.linear_scaled(xq[:, :24], xs[:, :1].contiguous(), wq[:, :24], ws[:, :1].contiguous()),
                 lambda: ar.linear_scaled(xq[:, 8:136], xs[:, :1].contiguous(), wq[:, :128], ws[:, :1].contiguous()),
                 lambda: ar.quant_scaled(bf, block_rows=64), lambda: ar.rms_norm(bf, None, -1.0),
                 lambda: ar.rms_norm(bf[:, :1].expand(8, 256).contiguous()[:1].expand(8, 256), None)):
        with pytest.raises(ar.ArError):
            call()
