"""The products of the 8-bit chain on every form of the tile kernel: 128 x 128 tiles (alone, and with K
shared by 2 or 4 CTAs), 128 x 256, and pairs of CTAs on 256 x 256, for aligned and unaligned rows of Y;
dense and by expert, e4m3, bf16 and a hi + lo pair.  Each test checks that the kernel it is about is the
one that ran.  Tolerances as in test_gpu_scaled.py.
"""
import ctypes
import os
import re
import subprocess
import sys

import pytest
import torch

from tests.test_gpu_scaled import (ar, check_product, layer, layer_weights, nblk, offsets_of, pitched, rand,  # noqa: F401
                                   read_rows, read_tiles, scaled_operands)

pytestmark = pytest.mark.gpu


def launched(call, path):
    """The kernels that `call` launches, as (name, template arguments, CTAs), from a graph that captures it."""
    call()  # (not the first call in a capture: that has a test of its own)
    graph = torch.cuda.CUDAGraph(keep_graph=True)
    with torch.cuda.graph(graph):
        call()
    dot = os.path.join(str(path), "graph.dot")
    assert ctypes.CDLL("libcuda.so.1").cuGraphDebugDotPrint(ctypes.c_void_p(graph.raw_cuda_graph()), dot.encode(), 1) == 0
    with open(dot) as f:
        text = f.read()
    names = re.findall(r"(tile|skinny|rms_norm|row_quant|tile_quant|tile_quant_async)_kernelI?((?:L[bi]\d+E)*)E.*?\\<\\<\\<\{?(\d+)", text)
    return [(n, tuple(int(v) for v in re.findall(r"L[bi](\d+)E", t)), int(ctas)) for n, t, ctas in names]


def check_tile(call, kind, pair, bn, whole, path):
    """`call` launches one kernel, this form of the tile kernel; returns its CTAs."""
    kernels = launched(call, path)
    assert [k[:2] for k in kernels] == [("tile", (int(kind == "scaled"), int(pair), bn, int(whole)))], kernels
    return kernels[0][2]


# rows per expert (experts without rows, with one, with a block to the row, a row more, and so many that a
# CTA works for several experts), columns of K (no multiple of 128), columns of Y
GROUPED = {
    "128 split 4": (False, 128, [1, 0, 130, 17, 100], 8208, 264),
    "128 split 2": (False, 128, [300, 0, 1, 128, 60, 5], 2064, 776),
    "128": (False, 128, [300, 0, 1, 128, 460, 11], 1040, 1032),
    "256": (False, 256, [700, 0, 1, 129, 1200, 256, 3], 1040, 2056),
    "pair": (True, 256, [2700, 1, 129, 2200], 1040, 2056),
}
DENSE = {
    "128 split 4": (False, 128, 250, 4112, 520),
    "128 split 2": (False, 128, 600, 2064, 904),
    "128": (False, 128, 1100, 1040, 1032),
    "256": (False, 256, 1100, 1040, 4088),
    "pair": (True, 256, 2043, 1040, 2056),
}
KINDS = ["scaled", "bf16", "hi + lo"]


def split_of(form, ctas, units):
    want = int(form.split()[-1]) if "split" in form else 1
    return want == 1 or ctas == want * units


class Experts:
    """Operands of a product by expert, and the call."""

    def __init__(self, ar, kind, counts, inn, out, pad=0, seed=1):
        self.ar, self.kind, self.counts, self.out = ar, kind, counts, out
        self.n = sum(counts) + pad
        self.offsets = offsets_of(counts)
        self.experts = len(counts)
        if kind == "scaled":
            self.X, self.xs, self.W, self.ws = scaled_operands(ar, self.n, inn, out, seed, self.experts)
            self.x64, self.W_lo = read_rows(self.X, self.xs), None
        else:
            self.X = rand(seed, self.n, inn)
            w = rand(seed + 1, self.experts, out, inn, std=0.02, dtype=torch.float32)
            self.W = w.to(torch.bfloat16)
            self.W_lo = (w - self.W.float()).to(torch.bfloat16) if kind == "hi + lo" else None
            self.x64 = self.X.double()

    def w64(self, e):
        if self.kind == "scaled":
            return read_tiles(self.W[e], self.ws[e])
        return self.W[e].double() + (0 if self.W_lo is None else self.W_lo[e].double())

    def __call__(self, out=None, X=None, xs=None, W=None, W_lo=None, offsets=None, **kw):
        X, W = self.X if X is None else X, self.W if W is None else W
        offsets = self.offsets if offsets is None else offsets
        if self.kind == "scaled":
            return self.ar.grouped_linear_scaled(X, self.xs if xs is None else xs, offsets, W, self.ws, out=out, **kw)
        return self.ar.grouped_linear(X, offsets, W, self.W_lo if W_lo is None else W_lo, out=out, **kw)

    def check(self, Y, counts=None, keep=None):
        """Every expert's rows against the formula (keep: those rows alone)."""
        at = 0
        for e, c in enumerate(counts or self.counts):
            rows = torch.arange(at, at + c, device="cuda")
            if keep is not None:
                rows = rows[keep[at:at + c]]
            check_product(Y[rows], self.x64[rows], self.w64(e), nblk(2 * self.X.shape[1]) * 2)
            at += c


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("kind", KINDS)
@pytest.mark.parametrize("form", list(GROUPED))
def test_by_expert(ar, form, kind, odd, tmp_path):  # noqa: F811
    pair, bn, counts, inn, out = GROUPED[form]
    out -= 5 * odd
    pad = 0 if form == "128 split 2" else 77
    p = Experts(ar, kind, counts, inn, out, pad)
    Y = torch.full((p.n, out), 3.0, dtype=torch.bfloat16, device="cuda")
    ctas = check_tile(lambda: p(Y), "scaled" if kind == "scaled" else "bf16", pair, bn, not odd, tmp_path)
    assert split_of(form, ctas, (-(-p.n // 128) + len(counts) - 1) * -(-out // 128))
    Y.fill_(3.0)
    assert p(Y) is Y and (Y[sum(counts):] == 3).all()
    p.check(Y)
    for _ in range(3):
        Z = torch.full_like(Y, 3.0)
        assert torch.equal(p(Z), Y)
    # operands and output as slices of wider rows: the same values, and nothing beside them
    el = 16 if kind == "scaled" else 8
    wide = torch.full((p.n, out + 29), 7.0, dtype=torch.bfloat16, device="cuda")
    wide[:, 11:11 + out] = 3.0
    lo = None if p.W_lo is None else pitched(p.W_lo, el)
    p(wide[:, 11:11 + out], X=pitched(p.X, 2 * el), W=pitched(p.W, el), W_lo=lo)
    assert torch.equal(wide[:, 11:11 + out], Y) and (wide[:, :11] == 7).all() and (wide[:, 11 + out:] == 7).all()


@pytest.mark.parametrize("odd", [False, True])
@pytest.mark.parametrize("form", list(DENSE))
def test_dense(ar, form, odd, tmp_path):  # noqa: F811
    """With the residual, in place too; some rows of a batch, whose scales start at any of the 4-byte places
    of a 16-byte unit; operands, residual and output as slices of wider rows."""
    pair, bn, n, inn, out = DENSE[form]
    out -= 3 * odd
    xq, xs, wq, ws = scaled_operands(ar, n, inn, out, 5)
    x64, w64, nb = read_rows(xq, xs), read_tiles(wq, ws), nblk(inn)
    add = rand(6, n, out)
    for res in (None, add):
        ctas = check_tile(lambda: ar.linear_scaled(xq, xs, wq, ws, add=res), "scaled", pair, bn, not odd, tmp_path)
        assert split_of(form, ctas, -(-n // 128) * -(-out // 128))
        Y = ar.linear_scaled(xq, xs, wq, ws, add=res)
        check_product(Y, x64, w64, nb, res)
        assert torch.equal(Y, ar.linear_scaled(xq, xs, wq, ws, add=res))
    stream = add.clone()
    assert ar.linear_scaled(xq, xs, wq, ws, add=stream, out=stream) is stream and torch.equal(stream, Y)
    wide, res = torch.full((n, out + 24), 7.0, dtype=torch.bfloat16, device="cuda"), pitched(add, 13)
    ar.linear_scaled(pitched(xq, 32), xs, pitched(wq, 16), ws, add=res, out=wide[:, 9:9 + out])
    assert torch.equal(wide[:, 9:9 + out], Y) and (wide[:, :9] == 7).all() and (wide[:, 9 + out:] == 7).all()
    for first in range(4):
        rows = slice(first, first + n - 4)
        call = lambda: ar.linear_scaled(xq[rows], xs[rows], wq, ws, add=add[rows])  # noqa: E731
        check_tile(call, "scaled", pair, bn, not odd, tmp_path)
        check_product(call(), x64[rows], w64, nb, add[rows])
        base = torch.cat([xs.new_zeros(first), xs.reshape(-1)])[first:].view_as(xs)  # the same scales at another place
        assert base.data_ptr() % 16 == 4 * first
        assert torch.equal(ar.linear_scaled(xq, base, wq, ws, add=add), Y)


BROKEN = [[0, 10, 5, 30], [-7, 3, 1 << 30, 20], [900, 12, 3, 0], [1 << 30] * 4, [-(1 << 31), -1, 0, 0], [0, 1 << 30, 0, 1 << 30],
          [(1 << 31) - 1, -(1 << 31), (1 << 31) - 1, -(1 << 31)]]


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("form", list(GROUPED))
def test_offsets_that_break_the_rules_stay_inside(ar, form, kind, tmp_path):  # noqa: F811
    """Offsets out of range or decreasing: the rows around X are not read into Y, those around Y not written."""
    pair, bn, counts, inn, out = GROUPED[form]
    p = Experts(ar, kind, counts, inn, out)
    n = p.n
    if kind == "scaled":
        wide = torch.full((n + 512, inn), 0x7F, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)  # NaN
        wide.view(torch.uint8)[256:256 + n] = p.X.view(torch.uint8)
    else:
        wide = torch.full((n + 512, inn), float("nan"), dtype=torch.bfloat16, device="cuda")
        wide[256:256 + n] = p.X
    X = wide[256:256 + n]
    Y = torch.full((n + 512, out), 3.0, dtype=torch.bfloat16, device="cuda")
    check_tile(lambda: p(Y[256:256 + n], X=X), kind, pair, bn, True, tmp_path)
    for broken in BROKEN:
        Y.fill_(3.0)
        offsets = (broken * (len(counts) // len(broken) + 1))[:len(counts) + 1]
        offsets += offsets[:1] * (len(counts) + 1 - len(offsets))
        p(Y[256:256 + n], X=X, offsets=torch.tensor(offsets, dtype=torch.int32, device="cuda"))
        assert (Y[:256] == 3).all() and (Y[256 + n:] == 3).all() and torch.isfinite(Y).all(), broken


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("form", list(GROUPED))
def test_graph_with_other_offsets(ar, form, kind, tmp_path):  # noqa: F811
    """The offsets are read on the device: a captured product follows them, to none, all or a few rows each."""
    pair, bn, counts, inn, out = GROUPED[form]
    p = Experts(ar, kind, counts, inn, out, 20)
    Y = torch.zeros(p.n, out, dtype=torch.bfloat16, device="cuda")
    check_tile(lambda: p(Y), kind, pair, bn, True, tmp_path)
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        p(Y)
    E, n = len(counts), p.n
    for other in ([0] * E, [n] + [0] * (E - 1), [0] * (E - 1) + [n - 3], [7 * e + 1 for e in range(E)], counts[::-1]):
        p.offsets.copy_(offsets_of(other))
        Y.fill_(3.0)
        graph.replay()
        p.check(Y, other)
        assert (Y[sum(other):] == 3).all()


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("form", list(GROUPED))
def test_nonfinite_values_keep_to_their_rows(ar, form, kind, tmp_path):  # noqa: F811
    """A NaN or an infinity in a row of X or its scales reaches that row of Y alone, one in a weight its
    expert's rows (columns) alone."""
    pair, bn, counts, inn, out = GROUPED[form]
    p = Experts(ar, kind, counts, inn, out)
    ref = p()
    check_tile(p, kind, pair, bn, True, tmp_path)
    first = [sum(counts[:e]) for e in range(len(counts))]
    big = max(range(len(counts)), key=lambda e: counts[e])
    rows = [first[big], first[big] + counts[big] - 1, first[big] + counts[big] // 2]
    keep = torch.ones(p.n, dtype=torch.bool, device="cuda")
    keep[rows] = False
    X, xs = p.X.clone(), None
    if kind == "scaled":
        xs = p.xs.clone()
        X.view(torch.uint8)[rows[0], 17] = 0x7F
        xs[rows[1], 0] = float("inf")
        xs[rows[2], -1] = float("nan")
    else:
        X[rows[0], 17] = float("nan")
        X[rows[1], 0] = float("inf")
        X[rows[2], -1] = float("-inf")
    Y = p(X=X, xs=xs)
    assert torch.equal(Y[keep], ref[keep]) and not torch.isfinite(Y[~keep]).any()
    W = p.W.clone()
    if kind == "scaled":
        W.view(torch.uint8)[big, 5] = 0x7F
    else:
        W[big, 5] = float("nan")
    Y = p(W=W)
    inside = torch.zeros_like(Y, dtype=torch.bool)
    inside[first[big]:first[big] + counts[big], 5] = True
    assert torch.isnan(Y[inside]).all() and torch.equal(Y[~inside], ref[~inside])


# A layer whose three products run on the tile kernel.
COUNTS = [900, 0, 300, 1, 700]
HIDDEN, INTER = 1024, 768


def check_layer_runs_on_tiles(call, path):
    names = [k[0] for k in launched(call, path)]
    assert names.count("tile") == 3 and "skinny" not in names, names


def test_launches_in_a_row_are_ordered(ar, tmp_path):  # noqa: F811
    """Layers back to back, each over the buffers of the one before: as with a synchronisation between
    them, in a stream and in a graph (the launches overlap their starts)."""
    w = layer_weights(ar, HIDDEN, INTER, COUNTS)
    n = sum(COUNTS)
    xs, rs = [rand(i, n, HIDDEN) for i in range(5)], [rand(9 + i, n, HIDDEN) for i in range(5)]
    check_layer_runs_on_tiles(lambda: layer(ar, xs[0], rs[0], w), tmp_path)
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


@pytest.mark.parametrize("kind", KINDS)
def test_products_in_a_row_are_ordered(ar, kind, tmp_path):  # noqa: F811
    """Products of several tile shapes, each on what a norm made of the one before, with few-row products
    between them: as with a synchronisation after each."""
    width = 1040
    ops = [Experts(ar, kind, GROUPED[f][2], width, width, seed=7 + i) for i, f in enumerate(GROUPED)]
    small = [Experts(ar, kind, [1, 2, 0, 3], width, width, seed=50 + i) for i in range(5)]
    n = max(p.n for p in ops)
    first = rand(3, n, width)

    def chain(sync):
        """Every product on the rows of the one before (normed, so that they stay in range)."""
        v, outs = first, []
        for p, s in zip(ops, small):
            for q in (p, s):
                if sync:
                    torch.cuda.synchronize()
                y = torch.zeros(n, width, dtype=torch.bfloat16, device="cuda")
                v, xq, xs, _ = ar.rms_norm(v, None, 1e-6, residual=first, want_scaled=True)
                q(y[:q.n], X=(xq if kind == "scaled" else v)[:q.n], xs=xs[:q.n])
                v = y
                outs.append(y)
        return outs

    want = chain(True)
    assert all(torch.isfinite(y).all() for y in want)
    for _ in range(10):
        assert all(torch.equal(a, b) for a, b in zip(chain(False), want))
    forms = {k[1] for k in launched(lambda: chain(False), tmp_path) if k[0] == "tile"}
    assert len(forms) >= 2, forms


def test_layer_captured_and_on_another_stream(ar, tmp_path):  # noqa: F811
    """A captured layer replays to the same bits on new inputs in its buffers; so does a run on a side stream."""
    w = layer_weights(ar, HIDDEN, INTER, COUNTS)
    n = sum(COUNTS)
    x, r, x2, r2 = (rand(i, n, HIDDEN) for i in range(1, 5))
    check_layer_runs_on_tiles(lambda: layer(ar, x, r, w), tmp_path)
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


def test_two_calls_at_once(ar):  # noqa: F811
    """Calls of every form on two streams at once, and two replays of graphs, do not disturb each other."""
    ops = [scaled_operands(ar, *DENSE[f][2:], seed=i) for i, f in enumerate(DENSE)]
    want = [ar.linear_scaled(*o) for o in ops]
    streams = torch.cuda.Stream(), torch.cuda.Stream()
    torch.cuda.synchronize()
    got = []
    for turn in range(10):
        for i in range(len(ops)):
            for k, s in enumerate(streams):
                j = (i * (k + 1) + turn) % len(ops)
                got.append((j, ar.linear_scaled(*ops[j], stream=s)))
    torch.cuda.synchronize()
    assert all(torch.equal(y, want[j]) for j, y in got)
    graphs = []
    for i in range(2):
        g = torch.cuda.CUDAGraph()
        with torch.cuda.graph(g):
            ys = [ar.linear_scaled(*o) for o in (ops if i else ops[::-1])]
        graphs.append((g, ys if i else ys[::-1]))
    for _ in range(5):
        for _, ys in graphs:
            for y in ys:
                y.zero_()
        torch.cuda.synchronize()
        for (g, _), s in zip(graphs, streams):
            with torch.cuda.stream(s):
                g.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(y, w) for _, ys in graphs for y, w in zip(ys, want))


FIRST_IN_CAPTURE = """
import torch
import signed_gradient_rounding_b200 as ar
x = torch.randn(2043, 1040, device="cuda").bfloat16()
w = torch.randn(2, 2056, 1040, device="cuda").bfloat16()
offsets = torch.tensor([0, 1000, 2043], dtype=torch.int32, device="cuda")
few = torch.tensor([0, 300, 600], dtype=torch.int32, device="cuda")
graph = torch.cuda.CUDAGraph()


def calls(q, s, wq, ws, y):
    return (ar.grouped_linear_scaled(q, s, offsets, wq, ws), ar.linear_scaled(q, s, wq[0], ws[0]),
            ar.linear_scaled(q[:1100], s[:1100], wq[1][:1032], ws[1][:9]), ar.linear_scaled(q[:250], s[:250], wq[1], ws[1]),
            ar.grouped_linear(y, offsets, w), ar.grouped_linear(y[:600], few, w[:, :2051].contiguous()))


with torch.cuda.graph(graph):
    y, q, s, h = ar.rms_norm(x, None, want_scaled=True)
    wq, ws = ar.quant_scaled(w, 128)
    got = calls(q, s, wq, ws, y)
graph.replay()
torch.cuda.synchronize()
got = [t.clone() for t in got]
y, q, s, h = ar.rms_norm(x, None, want_scaled=True)
assert all(torch.equal(a, b) for a, b in zip(got, calls(q, s, wq, ws, y)))
print("captured first")
"""


def test_first_calls_inside_a_capture():
    """A process whose first call of every kernel is captured."""
    root = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
    r = subprocess.run([sys.executable, "-c", FIRST_IN_CAPTURE], cwd=root, capture_output=True, text=True, timeout=300)
    assert r.returncode == 0 and "captured first" in r.stdout, r.stderr[-2000:]


@pytest.mark.parametrize("form", list(GROUPED))
def test_status_word_stays_zero(ar, form, tmp_path):  # noqa: F811
    for kind in ("scaled", "bf16"):
        pair, bn, counts, inn, out = GROUPED[form]
        p = Experts(ar, kind, counts, inn, out)
        status = torch.zeros(1, dtype=torch.int32, device="cuda")
        check_tile(lambda: p(status=status), kind, pair, bn, True, tmp_path)
        p(status=status)
        assert status.item() == 0


@pytest.mark.parametrize("n", [3, 40, 700])
def test_from_tuned_layers(ar, n):  # noqa: F811
    """Two layers tuned by this library, dequantised to a hi + lo pair and multiplied by expert; and their
    weight quantised again, as scaled tensors."""
    inn, out, group = 512, 264, 64
    x = rand(4, 1024, inn)
    tuned = []
    for seed in (1, 2):
        W = rand(seed, out, inn, std=0.02)
        p = ar.make_params(bits=4, group_size=group, iters=5, batch_rows=512)
        res = ar.tune_layer(W, x, p)
        tuned.append((res.codes, res.scale, res.zero_point, *ar.dequant(res.codes, res.scale, res.zero_point, group, want_f32=True)))
    exact = [(c.double() - z.double().repeat_interleave(group, 1)) * s.double().repeat_interleave(group, 1)
             for c, s, z, *_ in tuned]
    hi, lo = torch.stack([t[3] for t in tuned]), torch.stack([t[4] for t in tuned])
    counts = [n // 3, n - n // 3]
    X = x[:n]
    Y = ar.grouped_linear(X, offsets_of(counts), hi, lo)
    at = 0
    for c, w64, h, l in zip(counts, exact, hi, lo):
        rows = slice(at, at + c)
        check_product(Y[rows], X[rows].double(), h.double() + l.double(), nblk(2 * inn) * 2)
        # hi + lo carries the weight to 2^-17 of it (two roundings to bf16, and one to fp32 before)
        assert ((h.double() + l.double() - w64).abs() <= w64.abs() * (2.0 ** -16 + 2.0 ** -23)).all()
        at += c
    xq, xs = ar.quant_scaled(X)
    wq, ws = ar.quant_scaled(torch.stack([t[5] for t in tuned]), 128)
    Y = ar.grouped_linear_scaled(xq, xs, offsets_of(counts), wq, ws)
    at = 0
    for e, c in enumerate(counts):
        rows = slice(at, at + c)
        check_product(Y[rows], read_rows(xq[rows], xs[rows]), read_tiles(wq[e], ws[e]), nblk(inn))
        dense = ar.linear_scaled(xq[rows], xs[rows], wq[e], ws[e])
        check_product(dense, read_rows(xq[rows], xs[rows]), read_tiles(wq[e], ws[e]), nblk(inn))
        # the quantised weight is the dequantised one to a half step of e4m3
        w = read_tiles(wq[e], ws[e])
        step = exact[e].abs() * 2.0 ** -4 + ws[e].double().repeat_interleave(128, 0)[:out].repeat_interleave(128, 1)[:, :inn] * 2.0 ** -10
        assert ((w - exact[e]).abs() <= step * (1 + 2.0 ** -18)).all()
        at += c


@pytest.mark.parametrize("kind", ["scaled", "bf16"])
@pytest.mark.parametrize("form", list(GROUPED))
def test_waits_that_run_out_end_the_call(ar, form, kind, tmp_path, monkeypatch):  # noqa: F811
    """No operands ever come: every role gives up, the status word says so, nothing is written, and the calls
    behind it in the stream and after it are as ever."""
    pair, bn, counts, inn, out = GROUPED[form]
    p = Experts(ar, kind, counts, inn, out, 7)
    want = torch.full((p.n, out), 3.0, dtype=torch.bfloat16, device="cuda")
    check_tile(lambda: p(want), kind, pair, bn, True, tmp_path)
    want.fill_(3.0)
    p(want)
    buf = torch.full((p.n + 200, out), 3.0, dtype=torch.bfloat16, device="cuda")
    Y, after = buf[100:100 + p.n], torch.full_like(want, 3.0)
    status, clean = (torch.zeros(1, dtype=torch.int32, device="cuda") for _ in range(2))
    torch.cuda.synchronize()
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    monkeypatch.setenv("AR_FAULT", "wait")
    p(Y, status=status)
    p(Y)  # without a word
    monkeypatch.delenv("AR_FAULT")
    end.record()
    p(after, status=clean)
    torch.cuda.synchronize()
    assert status.item() == ar.AR_ETIMEOUT and (buf == 3).all() and 4 <= begin.elapsed_time(end) < 500
    assert clean.item() == 0 and torch.equal(after, want)


@pytest.mark.parametrize("form", list(DENSE))
def test_waits_that_run_out_leave_the_residual(ar, form, monkeypatch):  # noqa: F811
    """The dense product with its residual in place, aligned and not."""
    pair, bn, n, inn, out = DENSE[form]
    for odd in (0, 3):
        ops = scaled_operands(ar, n, inn, out - odd, 5)
        add = rand(6, n, out - odd)
        stream, status = add.clone(), torch.zeros(1, dtype=torch.int32, device="cuda")
        monkeypatch.setenv("AR_FAULT", "wait")
        ar.linear_scaled(*ops, add=stream, out=stream, status=status)
        monkeypatch.delenv("AR_FAULT")
        assert status.item() == ar.AR_ETIMEOUT and torch.equal(stream, add)
        ar.linear_scaled(*ops, add=stream, out=stream)
        assert torch.equal(stream, ar.linear_scaled(*ops, add=add))


def test_sums_longer_than_a_second(ar, tmp_path):  # noqa: F811
    """So many columns that one accumulator takes more than a second: the waits for it do not run out.
    Rows of +1, -1, ... whose last elements leave small whole numbers: every partial sum is exact."""
    n, inn = 17, 6 << 27
    torch.cuda.empty_cache()
    X = torch.ones(n, inn, dtype=torch.bfloat16, device="cuda")
    X *= torch.arange(1, n + 1, device="cuda", dtype=torch.bfloat16)[:, None]
    hi, lo = (torch.ones(1, 1, inn, dtype=torch.bfloat16, device="cuda") for _ in range(2))
    for w, last in ((hi, 3.0), (lo, 9.0)):
        w[..., 1::2] = -1.0
        w[..., -1] = last
    status = torch.zeros(1, dtype=torch.int32, device="cuda")
    offsets = offsets_of([n])
    small = slice(0, 1 << 20)
    check_tile(lambda: ar.grouped_linear(X[:, small], offsets, hi[..., small], lo[..., small]), "bf16", False, 128, False, tmp_path)
    begin, end = (torch.cuda.Event(enable_timing=True) for _ in range(2))
    begin.record()
    Y = ar.grouped_linear(X, offsets, hi, lo, status=status)
    end.record()
    torch.cuda.synchronize()
    del X, hi, lo
    torch.cuda.empty_cache()
    want = torch.arange(1, n + 1, device="cuda")[:, None] * (1.0 + 3.0 + 1.0 + 9.0)  # (at most 238: exact in bf16)
    assert status.item() == 0 and torch.equal(Y.float(), want)
    assert begin.elapsed_time(end) > 1000
