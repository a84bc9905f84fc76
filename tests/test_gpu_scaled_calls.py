"""GPU tests of single calls of the 8-bit chain: values at the ends of the range, empty and
overlapping tensors, the memory of calls on a given stream.  Formulas in 64 bits, roundings in
units u = 2^-24 as in test_gpu_scaled.py.
"""
import random

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


def calls_on(ar, seed=1, rows=300, cols=512, out=264):
    """Every entry point as a function of a stream, its operands in hand; each returns its new tensors."""
    gen = torch.Generator(device="cuda").manual_seed(seed)
    x, r = (torch.randn(rows, cols, generator=gen, device="cuda").to(torch.bfloat16) for _ in range(2))
    w = torch.randn(2, out, cols, generator=gen, device="cuda").to(torch.bfloat16)
    xq, xs = ar.quant_scaled(x)
    wq, ws = ar.quant_scaled(w, 128)
    offsets = torch.tensor([0, 100, rows], dtype=torch.int32, device="cuda")
    return dict(rms_norm=lambda s: ar.rms_norm(x, None, residual=r, want_scaled=True, stream=s),
                quant_scaled=lambda s: ar.quant_scaled(x, stream=s),
                silu_mul_scaled=lambda s: ar.silu_mul_scaled(x, r, stream=s),
                linear_scaled=lambda s: (ar.linear_scaled(xq, xs, wq[0], ws[0], stream=s),),
                grouped_linear=lambda s: (ar.grouped_linear(x, offsets, w, stream=s),),
                grouped_linear_scaled=lambda s: (ar.grouped_linear_scaled(xq, xs, offsets, wq, ws, stream=s),))


NAMES = ["rms_norm", "quant_scaled", "silu_mul_scaled", "linear_scaled", "grouped_linear", "grouped_linear_scaled"]


@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_a_given_stream_take_no_memory_still_in_use(ar, name):
    """A call on a stream that need not wait for the current one, while the current one still reads a
    tensor that was just dropped: the call's outputs must not get that memory."""
    call = calls_on(ar)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for like in want:
        held = [torch.full_like(like, 3.0, dtype=torch.float32 if like.dtype == torch.float32 else torch.uint8).view(-1)
                if like.dtype.itemsize == 1 or like.dtype == torch.float32 else torch.full_like(like, 3.0).view(-1)
                for _ in range(4)]
        places = {t.data_ptr() for t in held}
        torch.cuda._sleep(20_000_000)         # (about 10 ms)
        copies = [t + 0 for t in held]        # queued behind it
        del held
        got = call(side)
        assert not places & {t.data_ptr() for t in got}
        torch.cuda.synchronize()
        assert all((c == 3).all() for c in copies)
        for g, w in zip(got, want):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_outputs_on_a_given_stream_may_be_dropped_by_the_current_one(ar, name):
    """The current stream reads a call's outputs (after waiting for the call's stream) and drops them: the
    next call on that stream does not write over them before they are read."""
    call = calls_on(ar)[name]
    want = call(None)
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    for _ in range(3):
        got = call(side)
        places = {t.data_ptr() for t in got}
        torch.cuda.current_stream().wait_stream(side)
        torch.cuda._sleep(100_000_000)        # (about 50 ms)
        copies = [g.view(torch.uint8) + 0 for g in got]
        del got
        again = {t.data_ptr() for t in call(side)}
        assert not torch.cuda.current_stream().query(), "the outputs were read before the next call"
        assert not places & again
        torch.cuda.synchronize()
        for c, w in zip(copies, want):
            assert torch.equal(c, w.view(torch.uint8))


@pytest.mark.parametrize("name", ["linear_scaled", "grouped_linear", "grouped_linear_scaled"])
def test_status_word_is_kept_for_a_given_stream(ar, name):
    """A status word that is dropped while its call waits on a given stream is not handed out again."""
    x = torch.randn(300, 512, device="cuda").to(torch.bfloat16)
    w = torch.randn(2, 264, 512, device="cuda").to(torch.bfloat16)
    (xq, xs), (wq, ws) = ar.quant_scaled(x), ar.quant_scaled(w, 128)
    offsets = torch.tensor([0, 100, 300], dtype=torch.int32, device="cuda")
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    call = {"linear_scaled": lambda t: ar.linear_scaled(xq, xs, wq[0], ws[0], status=t, stream=side),
            "grouped_linear": lambda t: ar.grouped_linear(x, offsets, w, status=t, stream=side),
            "grouped_linear_scaled": lambda t: ar.grouped_linear_scaled(xq, xs, offsets, wq, ws, status=t, stream=side)}[name]
    call(None)  # (the first call of a kernel loads it, which takes longer than the wait below)
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    place = status.data_ptr()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        torch.cuda._sleep(100_000_000)  # (about 50 ms)
    call(status)
    del status
    places = [torch.empty(1, dtype=torch.int32, device="cuda").data_ptr() for _ in range(4)]
    assert not side.query(), "the call's stream was done before the word was asked for"
    assert place not in places
    torch.cuda.synchronize()


def refused(call):
    try:
        call()
    except ValueError:
        return True
    return False


def view(buf, first, rows, cols, pitch):
    return buf[first:].as_strided((rows, cols), (pitch, 1))


def elements(first, rows, cols, pitch):
    return {first + r * pitch + c for r in range(rows) for c in range(cols)}


def test_outputs_over_inputs_are_refused(ar):
    """out beside, between or over the rows of add, sum_out of x and the residual: refused exactly where
    an element is shared, unless it is the input itself."""
    rng = random.Random(3)
    buf = torch.zeros(4096, dtype=torch.bfloat16, device="cuda")
    seen = {True: 0, False: 0}
    for i in range(400):
        rows, cols = rng.randint(1, 6), rng.randint(1, 12)
        xq, xs = ar.quant_scaled(torch.ones(rows, 16, dtype=torch.bfloat16, device="cuda"))
        wq, ws = ar.quant_scaled(torch.ones(cols, 16, dtype=torch.bfloat16, device="cuda"), 128)
        x = torch.ones(rows, cols, dtype=torch.bfloat16, device="cuda")
        p1 = cols + rng.choice([0, 1, 5, 13, 40])
        p2 = rng.choice([p1, p1, cols + rng.choice([0, 1, 7, 30])])
        o1 = rng.randint(0, 200)
        o2 = o1 + rng.choice([0, 0, 1, cols, -cols, p1, rng.randint(-60, 60), rng.randint(-200, 200)])
        if o2 < 0:
            continue
        a, b = view(buf, o1, rows, cols, p1), view(buf, o2, rows, cols, p2)
        shared = bool(elements(o1, rows, cols, p1) & elements(o2, rows, cols, p2))
        itself = o1 == o2 and (p1 == p2 or rows == 1)
        seen[shared] += 1
        assert refused(lambda: ar.linear_scaled(xq, xs, wq, ws, add=a, out=b)) == (shared and not itself)
        assert refused(lambda: ar.rms_norm(x, None, residual=a, sum_out=b)) == (shared and not itself)
        assert refused(lambda: ar.rms_norm(a, None, residual=x, sum_out=b)) == shared
        weight = view(buf, o1, 1, cols, cols)[0]
        assert refused(lambda: ar.rms_norm(x, weight, residual=x.clone(), sum_out=b)) == bool(
            elements(o1, 1, cols, cols) & elements(o2, rows, cols, p2))
    assert min(seen.values()) > 50


def test_product_outputs_over_operands_are_refused(ar):
    """out in the memory of any operand of the three products."""
    n, inn, out = 8, 256, 128
    raw = torch.zeros(1 << 20, dtype=torch.uint8, device="cuda")
    Y = raw[:n * out * 2].view(torch.bfloat16).view(n, out)   # 2048 bytes
    x = torch.ones(n, inn, dtype=torch.bfloat16, device="cuda")
    w = torch.ones(2, out, inn, dtype=torch.bfloat16, device="cuda")
    (xq, xs), (wq, ws) = ar.quant_scaled(x), ar.quant_scaled(w, 128)
    offsets = torch.tensor([0, 4, n], dtype=torch.int32, device="cuda")

    def placed(t, at):  # a copy of t from byte `at` of raw on
        size = t.numel() * t.element_size()
        raw[at:at + size].copy_(t.contiguous().view(torch.uint8).view(-1) if t.dtype.itemsize > 1 else t.view(torch.uint8).view(-1))
        return raw[at:at + size].view(t.dtype).view(t.shape)

    for at, bad in ((1024, True), (2032, True), (2048, False), (4096, False)):
        for i in range(4):
            o = [xq, xs, wq[0], ws[0]]
            o[i] = placed(o[i], at)
            assert refused(lambda: ar.linear_scaled(*o, out=Y)) == bad, (at, i)
        for i in range(4):
            o = [x, offsets, w, w]
            o[i] = placed(o[i], at)
            assert refused(lambda: ar.grouped_linear(*o, out=Y)) == bad, (at, i)
        for i in range(5):
            o = [xq, xs, offsets, wq, ws]
            o[i] = placed(o[i], at)
            assert refused(lambda: ar.grouped_linear_scaled(*o, out=Y)) == bad, (at, i)
    # rows that overlap one another, as in an expanded tensor, are the library's to refuse
    with pytest.raises(ar.ArError):
        ar.linear_scaled(xq, xs, wq[0], ws[0], add=Y[:1].expand(n, out), out=Y)
    with pytest.raises(ar.ArError):
        ar.linear_scaled(xq, xs, wq[0], ws[0], add=torch.zeros_like(Y), out=Y[:1].expand(n, out))


@pytest.mark.parametrize("block_rows", [0, -1, 2, 127, 129, 1 + (1 << 32), 128 + (1 << 32), 1 - (1 << 32), (1 << 63) - 1])
def test_quant_scaled_refuses_other_blocks(ar, block_rows):
    """Numbers that are 1 or 128 in their low 32 bits among them: the scales would have another shape."""
    with pytest.raises(ar.ArError):
        ar.quant_scaled(torch.ones(300, 256, dtype=torch.bfloat16, device="cuda"), block_rows)


@pytest.mark.parametrize("rows", [1, 3, 297, 700])
@pytest.mark.parametrize("cols", [1024, 1032, 4096, 4104, 8192, 8200, 12288, 12296])
@pytest.mark.parametrize("res", [torch.bfloat16, torch.float32])
def test_rms_norm_where_the_threads_share_of_a_row_changes(ar, rows, cols, res):
    """Widths and row counts on both sides of each rule of the norm's launch.  Tolerances as in test_gpu_scaled.py:
    the norm within 2^-18, its one rounding to bf16 2^-8, to e4m3 2^-4 or half the subnormal step."""
    gen = torch.Generator(device="cuda").manual_seed(cols)
    x = torch.randn(rows, cols, generator=gen, device="cuda").to(torch.bfloat16)
    r = (4 * torch.randn(rows, cols, generator=gen, device="cuda")).to(res)
    w = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
    y, q, s, h = ar.rms_norm(x, w, 1e-5, residual=r, want_scaled=True)
    h64 = x.double() + r.double()
    v = h64 / (h64.square().mean(1, keepdim=True) + 1e-5).sqrt() * w.double()
    assert ((y.double() - v).abs() <= v.abs() * (2.0 ** -8 + 2.0 ** -18) + 2.0 ** -133).all()
    assert ((h.double() - h64).abs() <= h64.abs() * (2.0 ** -8 + 2 * U if res == torch.bfloat16 else U) + 2.0 ** -133).all()
    top = torch.nn.functional.pad(v.abs(), (0, -cols % 128)).view(rows, -1, 128).amax(2) / 448
    assert ((s.double() - top).abs() <= top * (2.0 ** -18 + 2 * U)).all()
    u = v / top.repeat_interleave(128, 1)[:, :cols]
    assert ((q.double() - u).abs() <= u.abs() * (2.0 ** -4 + 2.0 ** -16 + 8 * U) + 2.0 ** -10).all()


@pytest.mark.parametrize("name", NAMES)
def test_given_stream_inside_a_capture(ar, name):
    """A call on a stream that a capture has forked to, joined again: replays give the same bits, and the
    graph's memory stays its own."""
    call = calls_on(ar)[name]
    want = [t.clone() for t in call(None)]
    side = torch.cuda.Stream()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        here = torch.cuda.current_stream()
        side.wait_stream(here)
        got = call(side)
        here.wait_stream(side)
        again = call(None)
    noise = [call(side) for _ in range(3)]
    for _ in range(3):
        for t in (*got, *again):
            t.view(torch.uint8).zero_()
        graph.replay()
        torch.cuda.synchronize()
        for g, a, w in zip(got, again, want):
            assert torch.equal(g.view(torch.uint8), w.view(torch.uint8)) and torch.equal(a.view(torch.uint8), w.view(torch.uint8))
    torch.cuda.synchronize()
    for ts in noise:
        for t, w in zip(ts, want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))


@pytest.mark.parametrize("name", NAMES)
def test_default_and_current_stream_as_the_given_one(ar, name):
    call = calls_on(ar)[name]
    want = call(None)
    for stream in (torch.cuda.default_stream(), torch.cuda.current_stream()):
        for t, w in zip(call(stream), want):
            assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
    side = torch.cuda.Stream()
    torch.cuda.synchronize()
    with torch.cuda.stream(side):
        got = call(torch.cuda.default_stream())
    torch.cuda.synchronize()
    for t, w in zip(got, want):
        assert torch.equal(t.view(torch.uint8), w.view(torch.uint8))
