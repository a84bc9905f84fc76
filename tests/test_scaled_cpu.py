"""The 8-bit chain without a GPU: what its entry points refuse, in the C ABI and in
the binding, before any CUDA call."""
import ctypes

import pytest
import torch

P = ctypes.c_void_p(4096)      # never dereferenced: every call here is refused first
ODD = ctypes.c_void_p(4097)
OFF8 = ctypes.c_void_p(4104)
EINVAL, EUNSUPPORTED, OK, ECUDA = 1, 2, 0, 4


@pytest.fixture(scope="module")
def ar():
    import signed_gradient_rounding_b200 as ar
    return ar


NORM = dict(x=P, x_dtype=1, ldx=256, rows=4, cols=256, residual=P, r_dtype=1, ldr=256, weight=P, w_dtype=1, eps=1e-6,
            sum=P, lds=256, y=P, ldy=256, q=P, ldq=256, scale=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(x_dtype=2), EINVAL), (dict(r_dtype=7), EINVAL),
    (dict(w_dtype=-1), EINVAL), (dict(eps=-1e-6), EINVAL), (dict(eps=float("nan")), EINVAL),
    (dict(eps=float("inf")), EINVAL), (dict(x=None), EINVAL), (dict(residual=None), EINVAL), (dict(scale=None), EINVAL),
    (dict(sum=None, y=None, q=None), EINVAL), (dict(ldx=255), EINVAL), (dict(ldr=255), EINVAL), (dict(lds=255), EINVAL),
    (dict(ldy=255), EINVAL), (dict(ldq=255), EINVAL), (dict(x=ODD), EINVAL), (dict(residual=ODD), EINVAL),
    (dict(sum=ODD), EINVAL), (dict(weight=ODD), EINVAL), (dict(y=ODD), EINVAL),
    (dict(cols=32769, ldx=1 << 16, ldr=1 << 16, lds=1 << 16, ldy=1 << 16, ldq=1 << 16), EUNSUPPORTED),
    (dict(rows=(1 << 30) + 1), EUNSUPPORTED), (dict(rows=0, x=None), OK), (dict(cols=0, x=None), OK)])
def test_rms_norm_refusals(ar, change, status):
    assert ar.lib.ar_rms_norm(*{**NORM, **change}.values()) == status


QUANT = dict(x=P, x_dtype=1, ldx=256, count=2, rows=4, cols=256, block_rows=1, q=P, ldq=256, scale=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(count=-1), EINVAL), (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(x_dtype=3), EINVAL),
    (dict(block_rows=2), EINVAL), (dict(block_rows=0), EINVAL), (dict(x=None), EINVAL), (dict(q=None), EINVAL),
    (dict(scale=None), EINVAL), (dict(ldx=255), EINVAL), (dict(ldq=255), EINVAL), (dict(x=ODD), EINVAL),
    (dict(scale=ODD), EINVAL), (dict(rows=(1 << 30) + 1), EUNSUPPORTED),
    (dict(rows=1 << 30, cols=1 << 20, ldx=1 << 20, ldq=1 << 20), EUNSUPPORTED),
    (dict(rows=1 << 30, cols=1 << 16, ldx=1 << 16, ldq=1 << 16, block_rows=128), EUNSUPPORTED),
    (dict(count=0, x=None), OK), (dict(rows=0, x=None), OK), (dict(cols=0, x=None), OK)])
def test_quant_refusals(ar, change, status):
    assert ar.lib.ar_quant_scaled(*{**QUANT, **change}.values()) == status


SILU = dict(a=P, lda=256, b=P, ldb=256, rows=4, cols=256, q=P, ldq=256, scale=P, stream=None)


@pytest.mark.parametrize("change,status", [
    (dict(rows=-1), EINVAL), (dict(cols=-1), EINVAL), (dict(a=None), EINVAL), (dict(b=None), EINVAL),
    (dict(q=None), EINVAL), (dict(scale=None), EINVAL), (dict(lda=255), EINVAL), (dict(ldb=255), EINVAL),
    (dict(ldq=255), EINVAL), (dict(a=ODD), EINVAL), (dict(b=ODD), EINVAL), (dict(rows=(1 << 30) + 1), EUNSUPPORTED),
    (dict(rows=0, a=None), OK), (dict(cols=0, a=None), OK)])
def test_silu_refusals(ar, change, status):
    assert ar.lib.ar_silu_mul_scaled(*{**SILU, **change}.values()) == status


LINEAR = dict(X=P, ldx=256, xs=P, n=4, inn=256, W=P, ldw=256, ws=P, out=64, add=P, ldadd=64, Y=P, ldy=64, status=None,
              stream=None)
OPERANDS = [
    (dict(n=-1), EINVAL), (dict(inn=0), EINVAL), (dict(out=0), EINVAL), (dict(inn=252), EINVAL), (dict(ldx=260), EINVAL),
    (dict(ldw=260), EINVAL), (dict(ldx=240), EINVAL), (dict(ldw=240), EINVAL), (dict(ldy=63), EINVAL),
    (dict(X=None), EINVAL), (dict(W=None), EINVAL), (dict(Y=None), EINVAL), (dict(W=OFF8), EINVAL), (dict(X=OFF8), EINVAL),
    (dict(Y=ODD), EINVAL), (dict(n=(1 << 30) + 1), EUNSUPPORTED), (dict(out=1 << 31, ldy=1 << 31), EUNSUPPORTED),
    (dict(n=0, X=None, Y=None), OK)]
SCALES = [(dict(xs=None), EINVAL), (dict(ws=None), EINVAL), (dict(xs=ODD), EINVAL), (dict(ws=ODD), EINVAL)]


@pytest.mark.parametrize("change,status", OPERANDS + SCALES + [(dict(ldadd=63), EINVAL), (dict(add=ODD), EINVAL)])
def test_linear_refusals(ar, change, status):
    args = {**LINEAR, **change}
    if "out" in change and change["out"] > 1 << 30:
        args["ldadd"] = change["out"]
    assert ar.lib.ar_linear_scaled(*args.values()) == status


GROUPED = dict(X=P, ldx=256, n=4, inn=256, offsets=P, experts=3, W=P, W_lo=None, ldw=256, out=64, Y=P, ldy=64,
               status=None, stream=None)
GROUPED_SCALED = dict(X=P, ldx=256, xs=P, n=4, inn=256, offsets=P, experts=3, W=P, ldw=256, ws=P, out=64, Y=P, ldy=64,
                      status=None, stream=None)
EXPERTS = [(dict(experts=0), EINVAL), (dict(experts=-1), EINVAL), (dict(offsets=None), EINVAL), (dict(offsets=ODD), EINVAL),
           (dict(experts=1025), EUNSUPPORTED), (dict(experts=1024, out=(1 << 20) + 1, ldy=1 << 21), EUNSUPPORTED)]


@pytest.mark.parametrize("change,status", OPERANDS + EXPERTS + [(dict(W_lo=OFF8), EINVAL)])
def test_grouped_refusals(ar, change, status):
    assert ar.lib.ar_grouped_linear(*{**GROUPED, **change}.values()) == status


@pytest.mark.parametrize("change,status", OPERANDS + EXPERTS + SCALES)
def test_grouped_scaled_refusals(ar, change, status):
    assert ar.lib.ar_grouped_linear_scaled(*{**GROUPED_SCALED, **change}.values()) == status


def test_fault_hook(ar, monkeypatch):
    calls = [(ar.lib.ar_rms_norm, NORM), (ar.lib.ar_quant_scaled, QUANT), (ar.lib.ar_silu_mul_scaled, SILU),
             (ar.lib.ar_linear_scaled, LINEAR), (ar.lib.ar_grouped_linear, GROUPED),
             (ar.lib.ar_grouped_linear_scaled, GROUPED_SCALED)]
    for kind, status in (("param", EINVAL), ("launch", ECUDA)):
        monkeypatch.setenv("AR_FAULT", kind)
        for fn, args in calls:
            assert fn(*args.values()) == status


def test_binding_refuses_host_tensors(ar):
    x = torch.zeros(4, 256, dtype=torch.bfloat16)
    q, s = torch.zeros(4, 256, dtype=torch.float8_e4m3fn), torch.ones(4, 2)
    w, ws = torch.zeros(3, 64, 256, dtype=torch.float8_e4m3fn), torch.ones(3, 1, 2)
    offsets = torch.zeros(4, dtype=torch.int32)
    for call in (lambda: ar.rms_norm(x, None), lambda: ar.quant_scaled(x), lambda: ar.silu_mul_scaled(x, x),
                 lambda: ar.linear_scaled(q, s, w[0], ws[0]), lambda: ar.grouped_linear(x, offsets, w.to(torch.bfloat16)),
                 lambda: ar.grouped_linear_scaled(q, s, offsets, w, ws)):
        with pytest.raises(ValueError):
            call()
