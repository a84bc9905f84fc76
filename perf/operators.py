"""The 8-bit chain of a decoder layer, in plain torch and through the library.

Four operators, in the order a layer runs them:

* ``norm``: root-mean-square norm with the residual's addition, output in bf16 and in e4m3 with one
  scale per row and block of 128 columns;
* ``quant``: e4m3 with a scale per block of 128 columns (activations, or silu(a) * b of a gated MLP)
  or per 128 x 128 block (weights);
* ``linear``: matrix product of two such tensors, with an optional residual;
* ``grouped``: the products of tokens sorted by expert with their experts' weights, bf16 or e4m3.

``run`` computes them with elementary torch operations in 32 bits, or, where ``own`` is true, calls
the library.
"""
from __future__ import annotations

import math

import torch

own = False

BLOCK = 128
E4M3_MAX = 448.0


# ---------------------------------------------------------------------------
# Cases
# ---------------------------------------------------------------------------

def listed():
    return [
        # One token of a decoding request in front of q/k/v: latency.
        dict(name="norm_token", op="norm", rows=1, cols=4096, res="bf16", y=False, q=True),
        # A calibration block (8 samples x 2048 tokens) in front of an MLP with a bf16 router beside it.
        dict(name="norm_prefill", op="norm", rows=16384, cols=4096, res="bf16", y=True, q=True),
        # An odd number of tokens of the wider model, with the residual stream held in fp32.
        dict(name="norm_f32_stream", op="norm", rows=2049, cols=8192, res="f32", y=True, q=False),
        # gate_proj's weight, quantised once at load.
        dict(name="quant_weight", op="quant", kind="weight", rows=11008, cols=4096),
        # The gated MLP's input of down_proj for a few decoding requests: latency.
        dict(name="quant_gated_tokens", op="quant", kind="gated", rows=7, cols=11008),
        # The same for a calibration block.
        dict(name="quant_gated_prefill", op="quant", kind="gated", rows=16384, cols=11008),
        # gate_proj for one token: the weight's bytes.
        dict(name="linear_token", op="linear", n=1, inn=4096, out=11008, add=False),
        # The wide model's down_proj on a ragged batch, with the residual.
        dict(name="linear_ragged", op="linear", n=333, inn=29568, out=8192, add=True),
        # gate_proj of a calibration block: the tensor cores.
        dict(name="linear_prefill", op="linear", n=16384, inn=4096, out=11008, add=False),
        # Eight tokens of 8 experts each out of 64 in a decoding step, in a buffer padded to 96 rows.
        dict(name="grouped_decode", op="grouped", kind="scaled", experts=64, rows=64, pad=32, inn=4096, out=2048,
             skew=0.3),
        # Calibration tokens through bf16 experts of uneven popularity, some of them idle.
        dict(name="grouped_bf16", op="grouped", kind="bf16", experts=16, rows=8191, pad=0, inn=2048, out=4096, skew=1.0),
        # Prefill through 8-bit experts.
        dict(name="grouped_prefill", op="grouped", kind="scaled", experts=32, rows=16384, pad=77, inn=4096, out=2816,
             skew=0.7),
    ]


def _log(rng, lo, hi):
    return int(round(math.exp(rng.uniform(math.log(lo), math.log(hi)))))


def draw(rng):
    op = rng.choice(["norm", "quant", "linear", "linear", "grouped", "grouped"])
    if op in ("norm", "quant"):
        # Any width for the norm and the quantiser: the model's own, or odd ones.
        cols = rng.choice([4096, 11008, 8192, 29568, _log(rng, 64, 16384), _log(rng, 64, 16384) // 8 * 8])
        rows = min(_log(rng, 1, 16384), 16384 * 11008 // cols)
        if op == "norm":
            y, q = rng.choice([(False, True), (True, True), (True, False)])
            return dict(op=op, rows=rows, cols=cols, res=rng.choice(["bf16", "bf16", "f32", "none"]), y=y, q=q)
        return dict(op=op, kind=rng.choice(["weight", "rows", "gated"]), rows=rows, cols=cols)
    if op == "linear":
        inn, out = rng.choice([(4096, 4096), (4096, 11008), (11008, 4096), (29568, 8192),
                               (_log(rng, 8, 688) * 16, _log(rng, 64, 11008)), (_log(rng, 8, 688) * 16, _log(rng, 64, 11008))])
        n = min(_log(rng, 1, 16384), 16384 * 4096 * 11008 // (inn * out))
        return dict(op=op, n=n, inn=inn, out=out, add=rng.random() < 0.4)
    kind = rng.choice(["bf16", "scaled"])
    experts = _log(rng, 2, 64)
    inn, out = _log(rng, 16, 256) * 16, _log(rng, 128, 4096)
    rows = _log(rng, 1, 16384)
    return dict(op=op, kind=kind, experts=experts, rows=rows, pad=rng.choice([0, 0, rng.randint(1, 200)]), inn=inn, out=out,
                skew=rng.choice([0.0, 0.5, 1.0]))


# ---------------------------------------------------------------------------
# Inputs
# ---------------------------------------------------------------------------

def _blocks(n):
    return -(-n // BLOCK)


def _activations(rows, cols, gen):
    """Tokens whose channels differ in spread, one channel in a hundred 20 times larger."""
    sigma = torch.exp(0.5 * torch.randn(cols, generator=gen, device="cuda"))
    sigma[torch.randperm(cols, generator=gen, device="cuda")[:round(0.01 * cols)]] *= 20
    x = torch.randn(rows, cols, generator=gen, device="cuda")
    return x.mul_(sigma)


def _to_e4m3(x, s):
    """x / s in e4m3, round to nearest even; x, s fp32 of the same shape or broadcast."""
    return (x / s).clamp_(-E4M3_MAX, E4M3_MAX).to(torch.float8_e4m3fn)


def _row_scale(x):
    """max |x| / 448 per row and block of 128 columns (1 where that is 0): [rows, blocks], and the same per column."""
    rows, cols = x.shape
    nb = _blocks(cols)
    padded = torch.nn.functional.pad(x, (0, nb * BLOCK - cols))
    s = padded.view(rows, nb, BLOCK).abs().amax(2) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    return s, s.repeat_interleave(BLOCK, 1)[:, :cols]


def _tile_scale(w):
    """The same per 128 x 128 block of the last two axes of w [..., rows, cols]."""
    rows, cols = w.shape[-2:]
    rb, cb = _blocks(rows), _blocks(cols)
    padded = torch.nn.functional.pad(w, (0, cb * BLOCK - cols, 0, rb * BLOCK - rows))
    s = padded.view(*w.shape[:-2], rb, BLOCK, cb, BLOCK).abs().amax((-3, -1)) / E4M3_MAX
    s = torch.where(s == 0, torch.ones_like(s), s)
    return s, _spread(s, rows, cols)


def _spread(s, rows, cols):
    """A scale per 128 x 128 block [..., rb, cb] as one per element [..., rows, cols]."""
    return s.repeat_interleave(BLOCK, -2)[..., :rows, :].repeat_interleave(BLOCK, -1)[..., :cols]


def _counts(case, seed):
    """Rows per expert: popularity falls off as a power of a shuffled rank."""
    gen = torch.Generator().manual_seed(seed * 7 + 3)
    weight = (1.0 + torch.randperm(case["experts"], generator=gen).double()) ** -case["skew"]
    picked = torch.multinomial(weight, case["rows"], replacement=True, generator=gen)
    return torch.bincount(picked, minlength=case["experts"])


def prepare(case, seed):
    gen = torch.Generator(device="cuda").manual_seed(seed)
    op = case["op"]
    state = dict(case=case)
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        state["x"] = _activations(rows, cols, gen).to(torch.bfloat16)
        if case["res"] != "none":
            state["r"] = _activations(rows, cols, gen).to(torch.float32 if case["res"] == "f32" else torch.bfloat16)
        state["w"] = (1 + 0.2 * torch.randn(cols, generator=gen, device="cuda")).to(torch.bfloat16)
        state["eps"] = 1e-5
    elif op == "quant":
        rows, cols = case["rows"], case["cols"]
        if case["kind"] == "weight":
            state["x"] = (0.02 * torch.randn(rows, cols, generator=gen, device="cuda")).to(torch.bfloat16)
        else:
            state["x"] = _activations(rows, cols, gen).to(torch.bfloat16)
        if case["kind"] == "gated":
            state["b"] = _activations(rows, cols, gen).to(torch.bfloat16)
    elif op == "linear":
        n, inn, out = case["n"], case["inn"], case["out"]
        x = _activations(n, inn, gen).to(torch.bfloat16).float()
        state["xs"], full = _row_scale(x)
        state["xq"] = _to_e4m3(x, full)
        w = (0.02 * torch.randn(out, inn, generator=gen, device="cuda")).to(torch.bfloat16).float()
        state["ws"], full = _tile_scale(w)
        state["wq"] = _to_e4m3(w, full)
        if case["add"]:
            state["add"] = _activations(n, out, gen).to(torch.bfloat16)
    else:
        experts, inn, out = case["experts"], case["inn"], case["out"]
        counts = _counts(case, seed)
        state["offsets"] = torch.cat([torch.zeros(1, dtype=torch.int64), counts.cumsum(0)]).to(torch.int32).cuda()
        state["most"] = int(counts.max())  # the longest run of rows, known where the batch is built
        x = _activations(case["rows"] + case["pad"], inn, gen).to(torch.bfloat16)
        w = (0.02 * torch.randn(experts, out, inn, generator=gen, device="cuda")).to(torch.bfloat16)
        if case["kind"] == "scaled":
            x = x.float()
            state["xs"], full = _row_scale(x)
            state["xq"] = _to_e4m3(x, full)
            w = w.float()
            state["ws"], full = _tile_scale(w)
            state["wq"] = _to_e4m3(w, full)
        else:
            state["x"], state["w"] = x, w
        # The batch's output buffer; its rows behind the last expert's belong to somebody else.
        state["out"] = torch.randn(case["rows"] + case["pad"], out, generator=gen, device="cuda").to(torch.bfloat16)
    return state


# ---------------------------------------------------------------------------
# One pass
# ---------------------------------------------------------------------------

def run(state):
    op = state["case"]["op"]
    if op == "norm":
        return _norm(state)
    if op == "quant":
        return _quant(state)
    if op == "linear":
        return _linear(state)
    return _grouped(state)


def _norm(state):
    case, x, w, eps = state["case"], state["x"], state["w"], state["eps"]
    r = state.get("r")
    if own:
        import signed_gradient_rounding_b200 as ar
        y, q, scale, h = ar.rms_norm(x, w, eps, residual=r, want_bf16=case["y"], want_scaled=case["q"])
    else:
        f = x.float() if r is None else x.float() + r.float()
        h = None if r is None else f.to(r.dtype)
        f = f * torch.rsqrt(f.square().mean(1, keepdim=True) + eps) * w.float()
        y = f.to(torch.bfloat16) if case["y"] else None
        q = scale = None
        if case["q"]:
            scale, full = _row_scale(f)
            q = _to_e4m3(f, full)
    return {k: v for k, v in dict(y=y, q=q, scale=scale, h=h).items() if v is not None}


def _quant(state):
    case, x = state["case"], state["x"]
    if own:
        import signed_gradient_rounding_b200 as ar
        if case["kind"] == "gated":
            q, scale = ar.silu_mul_scaled(x, state["b"])
        else:
            q, scale = ar.quant_scaled(x, block_rows=BLOCK if case["kind"] == "weight" else 1)
    else:
        f = x.float()
        if case["kind"] == "gated":
            f = f / (1 + torch.exp(-f)) * state["b"].float()
        scale, full = _tile_scale(f) if case["kind"] == "weight" else _row_scale(f)
        q = _to_e4m3(f, full)
    return dict(q=q, scale=scale)


def _linear(state):
    case = state["case"]
    add = state.get("add")
    if own:
        import signed_gradient_rounding_b200 as ar
        return ar.linear_scaled(state["xq"], state["xs"], state["wq"], state["ws"], add=add)
    x = state["xq"].float() * state["xs"].repeat_interleave(BLOCK, 1)[:, :case["inn"]]
    w = state["wq"].float() * _spread(state["ws"], case["out"], case["inn"])
    y = x @ w.T
    if add is not None:
        y += add.float()
    return y.to(torch.bfloat16)


def _grouped(state):
    case, out = state["case"], state["out"]
    scaled = case["kind"] == "scaled"
    if own:
        import signed_gradient_rounding_b200 as ar
        if scaled:
            return ar.grouped_linear_scaled(state["xq"], state["xs"], state["offsets"], state["wq"], state["ws"], out=out)
        return ar.grouped_linear(state["x"], state["offsets"], state["w"], out=out)
    if scaled:
        x = state["xq"].float() * state["xs"].repeat_interleave(BLOCK, 1)[:, :case["inn"]]
        w = state["wq"].float() * _spread(state["ws"], case["out"], case["inn"])
    else:
        x, w = state["x"].float(), state["w"].float()
    # Each expert's rows in a padded slot of their own, one batched product, and the rows back in place.
    offsets = state["offsets"].long()
    row = torch.arange(case["rows"], device=x.device)
    expert = torch.searchsorted(offsets[1:], row, right=True)
    slot = row - offsets[expert]
    padded = torch.zeros(case["experts"], state["most"], case["inn"], device=x.device)
    padded[expert, slot] = x[:case["rows"]]
    y = torch.bmm(padded, w.transpose(1, 2))
    out[:case["rows"]] = y[expert, slot].to(out.dtype)
    return out


# ---------------------------------------------------------------------------
# What a pass cannot do without, and its value in 64 bits
# ---------------------------------------------------------------------------

def work(case):
    op = case["op"]
    if op == "norm":
        rows, cols = case["rows"], case["cols"]
        res = dict(none=0, bf16=4, f32=8)[case["res"]]
        b = rows * cols * (2 + res + 2 * case["y"] + case["q"]) + 2 * cols + 4 * rows * _blocks(cols) * case["q"]
        return dict(bytes=b, flops=5 * rows * cols)
    if op == "quant":
        rows, cols = case["rows"], case["cols"]
        groups = _blocks(cols) * (_blocks(rows) if case["kind"] == "weight" else rows)
        gated = case["kind"] == "gated"
        return dict(bytes=rows * cols * (5 if gated else 3) + 4 * groups, flops=rows * cols * (6 if gated else 2))
    if op == "linear":
        n, inn, out = case["n"], case["inn"], case["out"]
        b = (n + out) * inn + 4 * _blocks(inn) * (n + _blocks(out)) + 2 * n * out * (2 if case["add"] else 1)
        return dict(bytes=b, flops=2 * n * inn * out)
    rows, inn, out = case["rows"], case["inn"], case["out"]
    active = int((_counts(case, 1) > 0).sum())  # experts with rows: their weights are read
    size = 1 if case["kind"] == "scaled" else 2
    b = size * inn * (rows + active * out) + 2 * rows * out
    if case["kind"] == "scaled":
        b += 4 * _blocks(inn) * (rows + active * _blocks(out))
    return dict(bytes=b, flops=2 * rows * inn * out)


def _wide(x, scale, block_rows):
    """An e4m3 tensor with its scales as numbers in 64 bits: one block of columns at a time."""
    v = x.double()
    for k in range(scale.shape[-1]):
        s = scale[..., k].double()
        if block_rows > 1:
            s = s.repeat_interleave(block_rows, -1)[..., :x.shape[-2]]
        v[..., k * BLOCK:(k + 1) * BLOCK] *= s.unsqueeze(-1)
    return v


def _exact_q(v, block_rows):
    """The quotients that e4m3 rounds, and the scales."""
    rows, cols = v.shape
    q = torch.empty_like(v)
    scale = torch.empty(-(-rows // block_rows), _blocks(cols), dtype=torch.float64, device=v.device)
    pad = -rows % block_rows
    for k in range(scale.shape[1]):
        part = v[:, k * BLOCK:(k + 1) * BLOCK]
        top = torch.cat([part.abs().amax(1), part.new_zeros(pad)]).view(-1, block_rows).amax(1) / E4M3_MAX
        top[top == 0] = 1
        scale[:, k] = top
        q[:, k * BLOCK:(k + 1) * BLOCK] = part / top.repeat_interleave(block_rows)[:rows, None]
    return q, scale


def exact(case, seed):
    state = prepare(case, seed)
    op = case["op"]
    if op == "norm":
        v = state["x"].double()
        got = {}
        if "r" in state:
            v += state["r"].double()
            got["h"] = v.clone()
        rms = ((v * v).sum(1) / case["cols"] + state["eps"]).sqrt()
        v /= rms[:, None]
        v *= state["w"].double()
        if case["q"]:
            got["q"], got["scale"] = _exact_q(v, 1)
        if case["y"]:
            got["y"] = v
        return got
    if op == "quant":
        v = state["x"].double()
        if case["kind"] == "gated":
            v = v * torch.sigmoid(v) * state["b"].double()
        q, scale = _exact_q(v, BLOCK if case["kind"] == "weight" else 1)
        return dict(q=q, scale=scale)
    if op == "linear":
        y = _wide(state["xq"], state["xs"], 1) @ _wide(state["wq"], state["ws"], BLOCK).T
        return y + state["add"].double() if case["add"] else y
    y = state["out"].double()
    ends = state["offsets"].tolist()
    for e in range(case["experts"]):
        a, b = ends[e], ends[e + 1]
        if b > a and case["kind"] == "scaled":
            y[a:b] = _wide(state["xq"][a:b], state["xs"][a:b], 1) @ _wide(state["wq"][e], state["ws"][e], BLOCK).T
        elif b > a:
            y[a:b] = state["x"][a:b].double() @ state["w"][e].double().T
    return y
