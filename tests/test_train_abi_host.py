"""Refusals of the norm, gradient-norm and AdamW entry points on the host,
before any CUDA call, and the exports' workspace sizes."""
import ctypes

import pytest

from vocab_sharded_lm_gb300 import _build, vpce

FAKE = 0x7F0000000000  # a 256-byte aligned "device" address, never dereferenced on the host
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return vpce.load_library()


def _norm(lib, codes=False, **kw):
    a = dict(x=FAKE, dtype=1, ld_x=0, res=FAKE, rdtype=1, ld_res=0, w=FAKE, wdtype=1, eps=1e-6, s=4, h=64, group=0,
             res_out=FAKE, ld_ro=0, out=FAKE, ld_out=0, scale=FAKE, rstd=FAKE)
    a.update(kw)
    head = [a[k] for k in ("x", "dtype", "ld_x", "res", "rdtype", "ld_res", "w", "wdtype", "eps", "s", "h")]
    tail = [a[k] for k in ("res_out", "ld_ro", "out", "ld_out")]
    if codes:
        return lib.vpce_rmsnorm_quantized_forward(*head, a["group"], *tail, a["scale"], a["rstd"], None)
    return lib.vpce_rmsnorm_forward(*head, *tail, a["rstd"], None)


@pytest.mark.parametrize("codes", [False, True])
@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(rdtype=-1), 3), (dict(wdtype=7), 3),
    (dict(dtype=0, rdtype=1), 3),                     # a bf16 stream beside fp32 rows
    (dict(s=-1), 1), (dict(s=(1 << 31) + 1), 1),
    (dict(h=0), 1), (dict(h=vpce.VPCE_MAX_NORM_COLUMNS + 1), 1),
    (dict(eps=-1.0), 1), (dict(eps=NAN), 1), (dict(eps=INF), 1),
    (dict(x=None), 1), (dict(w=None), 1), (dict(out=None), 1),
    (dict(res_out=None), 1), (dict(res=None), 1),     # a sum without a residual, or the other way round
    (dict(ld_x=63), 1), (dict(ld_res=-1), 1), (dict(ld_ro=1), 1), (dict(ld_out=63), 1), (dict(ld_x=1 << 60), 1),
    (dict(x=FAKE + 1), 2), (dict(res=FAKE + 1), 2), (dict(res_out=FAKE + 1), 2), (dict(w=FAKE + 1), 2),
    (dict(rstd=FAKE + 2), 2), (dict(rdtype=0, res=FAKE + 2), 2),
])
def test_norm_refuses(lib, codes, kw, code):
    assert _norm(lib, codes, **kw) == code


@pytest.mark.parametrize("kw,code", [
    (dict(group=-16), 1), (dict(group=8), 1), (dict(group=100), 1), (dict(scale=None), 1), (dict(scale=FAKE + 2), 2),
])
def test_quantized_norm_refuses(lib, kw, code):
    assert _norm(lib, True, **kw) == code


def test_norm_of_bf16_rows_off_their_elements(lib):
    assert _norm(lib, False, out=FAKE + 1) == 2


def _norm_bwd(lib, **kw):
    a = dict(dy=FAKE, gdtype=1, ld_g=0, x=FAKE, xdtype=1, ld_x=0, w=FAKE, wdtype=0, rstd=FAKE, dres=FAKE, ld_r=0, s=4,
             h=64, dx=FAKE, ld_dx=0, dw=FAKE, acc=0, ws=FAKE, wsb=4 * 64 * 4)
    a.update(kw)
    return lib.vpce_rmsnorm_backward(*a.values(), None)


@pytest.mark.parametrize("kw,code", [
    (dict(gdtype=2), 3), (dict(xdtype=2), 3), (dict(wdtype=2), 3), (dict(gdtype=0), 3),
    (dict(s=-1), 1), (dict(s=1 << 40), 1), (dict(h=0), 1), (dict(h=1 << 20), 1), (dict(acc=2), 1),
    (dict(dy=None), 1), (dict(x=None), 1), (dict(w=None), 1), (dict(rstd=None), 1), (dict(dx=None), 1),
    (dict(dw=None), 1), (dict(ws=None), 1),
    (dict(ld_g=63), 1), (dict(ld_x=63), 1), (dict(ld_r=63), 1), (dict(ld_dx=63), 1),
    (dict(dy=FAKE + 1), 2), (dict(x=FAKE + 1), 2), (dict(dres=FAKE + 1), 2), (dict(dx=FAKE + 1), 2),
    (dict(w=FAKE + 2), 2), (dict(rstd=FAKE + 2), 2), (dict(dw=FAKE + 2), 2), (dict(ws=FAKE + 16), 2),
    (dict(wsb=4 * 64 * 4 - 1), 4),
])
def test_norm_backward_refuses(lib, kw, code):
    assert _norm_bwd(lib, **kw) == code


def test_norm_workspace_bytes(lib):
    f = lib.vpce_rmsnorm_backward_workspace_bytes
    assert f(4, 64) == 4 * 64 * 4 and f(1 << 31, 64) == f(1 << 20, 64) > 0 and f(0, 1) > 0
    assert f(-1, 64) == 0 and f(4, 0) == 0 and f(4, 32769) == 0


def _tensors(**kw):
    a = dict(param=FAKE, grad=FAKE, copy=None, exp_avg=FAKE, exp_avg_sq=FAKE, exp_avg_scale=None,
             exp_avg_sq_scale=None, n=100, weight_decay=0.1)
    a.update(kw)
    return (vpce._AdamWTensor * 1)(vpce._AdamWTensor(*a.values()))


def _adamw(lib, t=None, **kw):
    a = dict(tensors=_tensors(**(t or {})), n=1, pdtype=0, gdtype=0, bits=32, step=FAKE, lr=1e-3, lr_dev=None, b1=0.9,
             b2=0.999, eps=1e-8, scale=None, rng=None)
    a.update(kw)
    return lib.vpce_adamw_step(*a.values(), None)


EIGHT = dict(exp_avg_scale=FAKE, exp_avg_sq_scale=FAKE)


@pytest.mark.parametrize("t,kw,code", [
    ({}, dict(pdtype=2), 3), ({}, dict(gdtype=-1), 3),
    ({}, dict(bits=16), 1), ({}, dict(bits=0), 1),
    ({}, dict(n=-1), 1), ({}, dict(tensors=None), 1),
    ({}, dict(step=None), 1), ({}, dict(step=FAKE + 4), 2),
    ({}, dict(lr=-1.0), 1), ({}, dict(lr=NAN), 1), ({}, dict(lr=INF), 1), ({}, dict(lr_dev=FAKE + 2), 2),
    ({}, dict(b1=1.0), 1), ({}, dict(b1=-0.1), 1), ({}, dict(b2=1.0), 1), ({}, dict(b2=NAN), 1),
    ({}, dict(eps=-1e-8), 1), ({}, dict(eps=INF), 1), ({}, dict(eps=1e-39), 1), ({}, dict(scale=FAKE + 1), 2),
    (dict(n=-1), {}, 1), (dict(n=1 << 35), {}, 1),
    (dict(param=None), {}, 1), (dict(grad=None), {}, 1), (dict(exp_avg=None), {}, 1), (dict(exp_avg_sq=None), {}, 1),
    (dict(weight_decay=INF), {}, 1), (dict(weight_decay=NAN), {}, 1),
    (dict(param=FAKE + 2), {}, 2), (dict(grad=FAKE + 1), dict(gdtype=1), 2), (dict(copy=FAKE + 1), {}, 2),
    (dict(exp_avg=FAKE + 1), {}, 2), (dict(exp_avg_sq=FAKE + 2), {}, 2),
    (dict(copy=FAKE), dict(pdtype=1), 1),             # a bf16 copy of bf16 weights
    (EIGHT, {}, 1),                                   # scales beside fp32 states
    ({}, dict(bits=8, rng=FAKE), 1),                  # 8-bit states without scales
    (EIGHT, dict(bits=8), 1),                         # ... or without random words
    (EIGHT, dict(bits=8, rng=FAKE + 4), 2),
    (dict(EIGHT, exp_avg_scale=FAKE + 2), dict(bits=8, rng=FAKE), 2),
])
def test_adamw_refuses(lib, t, kw, code):
    assert _adamw(lib, t, **kw) == code


def test_a_list_past_the_runs_that_are_counted_is_refused(lib):
    n = 40
    big = (vpce._AdamWTensor * n)(*[_tensors(n=(1 << 35) - 1)[0] for _ in range(n)])
    assert _adamw(lib, tensors=big, n=n) == 1
    assert lib.vpce_grad_norm(big, n, 0, 1.0, FAKE, FAKE, FAKE, 1 << 30, None) == 1


def _grad_norm(lib, t=None, **kw):
    a = dict(tensors=_tensors(**(t or {})), n=1, gdtype=0, most=1.0, norm=FAKE, scale=FAKE, ws=FAKE, wsb=1 << 20)
    a.update(kw)
    return lib.vpce_grad_norm(*a.values(), None)


@pytest.mark.parametrize("t,kw,code", [
    ({}, dict(gdtype=3), 3), ({}, dict(n=-1), 1), ({}, dict(tensors=None), 1),
    ({}, dict(most=0.0), 1), ({}, dict(most=-1.0), 1), ({}, dict(most=NAN), 1),
    ({}, dict(norm=None, scale=None), 1), ({}, dict(ws=None), 1),
    ({}, dict(norm=FAKE + 2), 2), ({}, dict(scale=FAKE + 1), 2), ({}, dict(ws=FAKE + 4), 2), ({}, dict(wsb=16), 4),
    (dict(grad=None), {}, 1), (dict(grad=FAKE + 2), {}, 2), (dict(n=-3), {}, 1),
])
def test_grad_norm_refuses(lib, t, kw, code):
    assert _grad_norm(lib, t, **kw) == code


def test_grad_norm_workspace_bytes(lib):
    f = lib.vpce_grad_norm_workspace_bytes
    assert f(1) == f(440) < f(441) and f(-1) == 0 and f(1 << 31) == 0


def test_the_c_structure_is_the_headers(lib):
    assert ctypes.sizeof(vpce._AdamWTensor) == 72 and vpce._AdamWTensor.n.offset == 56
