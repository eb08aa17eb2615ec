"""What the Python forms of the norm, the gradient norm and the AdamW step ask
of their operands before the library is called, and what they hand to it."""
import contextlib
import types

import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

from _fake_cuda import Fake0, Fake1, fake, install

S, H = 4, 32
F32, BF16, I64, F8 = torch.float32, torch.bfloat16, torch.int64, torch.float8_e4m3fn


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch, vpce)


def new(*shape, dtype=F32, index=0):
    return fake(torch.zeros(shape, dtype=dtype), index)


def _placed(k, *operands):
    """The operands, the k-th of them on another device."""
    return [o.as_subclass(Fake1) if i == k else o for i, o in enumerate(operands)]


def _norm(k, **kw):
    x, w, r, o, ro, rs = _placed(k, new(S, H), new(H), new(S, H), new(S, H), new(S, H), new(S))
    vpce.vpce_rmsnorm_forward(x, w, r, out=o, residual_out=ro, rstd_out=rs, **kw)


def _norm8(k, **kw):
    x, w, r, q, sc, ro, rs = _placed(k, new(S, H), new(H), new(S, H), new(S, H, dtype=F8), new(S, 2), new(S, H),
                                     new(S))
    vpce.vpce_rmsnorm_quantized_forward(x, w, r, group=16, q_out=q, scale_out=sc, residual_out=ro, rstd_out=rs, **kw)


def _norm_grad(k, **kw):
    g, x, w, rs, gr, gi, gw, ws = _placed(k, new(S, H), new(S, H), new(H), new(S), new(S, H), new(S, H), new(H),
                                          new(4096, dtype=torch.uint8))
    vpce.vpce_rmsnorm_backward(g, x, w, rs, grad_residual=gr, grad_in=gi, grad_weight=gw, workspace=ws, **kw)


def _grad_norm(k, **kw):
    g0, g1, n, sc, ws = _placed(k, new(5), new(7), new(1), new(1), new(4096, dtype=torch.uint8))
    vpce.vpce_grad_norm([g0, g1], 1.0, norm_out=n, scale_out=sc, workspace=ws, **kw)


def _adamw(k, **kw):
    p0, p1, g0, g1, c0, c1, m0, m1, v0, v1, t, lr, sc, rng = _placed(
        k, new(5), new(7), new(5), new(7), new(5, dtype=BF16), new(7, dtype=BF16), new(5), new(7), new(5), new(7),
        new(1, dtype=I64), new(1), new(1), new(2, dtype=I64))
    plan = vpce.vpce_adamw_plan([p0, p1], [g0, g1], copies=[c0, c1], exp_avg=[m0, m1], exp_avg_sq=[v0, v1])
    vpce.vpce_adamw_step(plan, t, lr=lr, grad_scale=sc, rng=rng, **kw)


CALLS = {_norm: 6, _norm8: 7, _norm_grad: 8, _grad_norm: 5, _adamw: 14}


@pytest.fixture
def devices(monkeypatch):
    seen = []

    @contextlib.contextmanager
    def device(index):
        seen.append(index)
        yield

    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


@pytest.mark.parametrize("call,k", [(c, k) for c, n in CALLS.items() for k in range(n)],
                         ids=lambda v: getattr(v, "__name__", v))
def test_an_operand_on_another_device_is_refused(lib, devices, call, k):
    with pytest.raises(ValueError):
        call(k)
    assert lib.calls == []


def _everywhere(call, index, monkeypatch, **kw):
    monkeypatch.setitem(globals(), "_placed", lambda k, *operands: [o.as_subclass((Fake0, Fake1)[index])
                                                                    for o in operands])
    call(-1, **kw)


@pytest.mark.parametrize("call", CALLS, ids=lambda v: v.__name__)
def test_a_call_is_made_on_its_operands_device(lib, devices, monkeypatch, call):
    _everywhere(call, 0, monkeypatch)
    assert devices == [] and len(lib.calls) == 1
    _everywhere(call, 1, monkeypatch)
    assert set(devices) == {1} and len(lib.calls) == 2


@pytest.mark.parametrize("call", CALLS, ids=lambda v: v.__name__)
def test_a_stream_of_another_device_is_refused(lib, devices, monkeypatch, call):
    stream = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    with pytest.raises(ValueError, match="stream"):
        _everywhere(call, 1, monkeypatch, stream=stream)
    assert lib.calls == []


def shared(rows, cols, dtype=F32):
    return fake(torch.zeros(1, cols, dtype=dtype)).expand(rows, cols)


REFUSED = {
    "x over one row": lambda: vpce.vpce_rmsnorm_forward(shared(S, H), new(H), out=new(S, H), rstd_out=new(S)),
    "residual over one row": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), shared(S, H), out=new(S, H),
                                                               residual_out=new(S, H), rstd_out=new(S)),
    "out over one row": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), out=shared(S, H), rstd_out=new(S)),
    "columns apart": lambda: vpce.vpce_rmsnorm_forward(new(S, 2 * H)[:, ::2], new(H), out=new(S, H), rstd_out=new(S)),
    "out of another shape": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), out=new(S, H + 1), rstd_out=new(S)),
    "out of another type": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), out=new(S, H, dtype=BF16),
                                                             rstd_out=new(S)),
    "weight of another size": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H + 1), out=new(S, H),
                                                                rstd_out=new(S)),
    "weight apart": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(2 * H)[::2], out=new(S, H), rstd_out=new(S)),
    "half precision": lambda: vpce.vpce_rmsnorm_forward(new(S, H, dtype=torch.float16), new(H)),
    "3-D": lambda: vpce.vpce_rmsnorm_forward(new(1, S, H), new(H)),
    "not on a GPU": lambda: vpce.vpce_rmsnorm_forward(torch.zeros(S, H), torch.zeros(H)),
    "a bf16 stream beside fp32": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), new(S, H, dtype=BF16)),
    "a sum without a residual": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), residual_out=new(S, H)),
    "rstd apart": lambda: vpce.vpce_rmsnorm_forward(new(S, H), new(H), out=new(S, H), rstd_out=new(2 * S)[::2]),
    "an odd group": lambda: vpce.vpce_rmsnorm_quantized_forward(new(S, H), new(H), group=24),
    "scales of another shape": lambda: vpce.vpce_rmsnorm_quantized_forward(
        new(S, H), new(H), group=16, q_out=new(S, H, dtype=F8), scale_out=new(S, 1), rstd_out=new(S)),
    "codes as bytes": lambda: vpce.vpce_rmsnorm_quantized_forward(
        new(S, H), new(H), q_out=new(S, H, dtype=torch.uint8), scale_out=new(S, 1), rstd_out=new(S)),
    "gradient accumulated into nothing": lambda: vpce.vpce_rmsnorm_backward(
        new(S, H), new(S, H), new(H), new(S), grad_in=new(S, H), accumulate=True),
    "a bf16 sum beside fp32 gradients": lambda: vpce.vpce_rmsnorm_backward(
        new(S, H), new(S, H, dtype=BF16), new(H), new(S)),
    "gradient of another shape": lambda: vpce.vpce_rmsnorm_backward(new(S, H), new(S + 1, H), new(H), new(S)),
    "weight gradient in bf16": lambda: vpce.vpce_rmsnorm_backward(
        new(S, H), new(S, H), new(H), new(S), grad_in=new(S, H), grad_weight=new(H, dtype=BF16)),
    "grad_in over one row": lambda: vpce.vpce_rmsnorm_backward(new(S, H), new(S, H), new(H), new(S),
                                                               grad_in=shared(S, H)),
    "no gradients": lambda: vpce.vpce_grad_norm([]),
    "gradients of two types": lambda: vpce.vpce_grad_norm([new(4), new(4, dtype=BF16)]),
    "a gradient apart": lambda: vpce.vpce_grad_norm([new(8)[::2]]),
    "norm into many": lambda: vpce.vpce_grad_norm([new(8)], norm_out=new(2)),
    "no parameters": lambda: vpce.vpce_adamw_plan([], []),
    "a gradient too few": lambda: vpce.vpce_adamw_plan([new(4), new(4)], [new(4)]),
    "sizes apart": lambda: vpce.vpce_adamw_plan([new(4)], [new(5)]),
    "parameters of two types": lambda: vpce.vpce_adamw_plan([new(4), new(4, dtype=BF16)], [new(4), new(4)]),
    "a parameter apart": lambda: vpce.vpce_adamw_plan([new(8)[::2]], [new(4)]),
    "copies of bf16 parameters": lambda: vpce.vpce_adamw_plan([new(4, dtype=BF16)], [new(4)],
                                                              copies=[new(4, dtype=BF16)]),
    "16-bit states": lambda: vpce.vpce_adamw_plan([new(4)], [new(4)], state_bits=16),
    "scales of fp32 states": lambda: vpce.vpce_adamw_plan([new(4)], [new(4)], exp_avg=[new(4)], exp_avg_sq=[new(4)],
                                                          exp_avg_scale=[new(1)]),
    "states of another type": lambda: vpce.vpce_adamw_plan([new(4)], [new(4)], state_bits=8, exp_avg=[new(4)]),
    "decays too few": lambda: vpce.vpce_adamw_plan([new(4), new(4)], [new(4), new(4)], weight_decay=[0.1],
                                                   exp_avg=[new(4), new(4)], exp_avg_sq=[new(4), new(4)]),
}


@pytest.mark.parametrize("call", REFUSED.values(), ids=REFUSED)
def test_refused(lib, call):
    with pytest.raises((ValueError, TypeError)):
        call()
    assert lib.calls == []


def _states(n, bits=32):
    if bits == 32:
        return dict(exp_avg=[new(n)], exp_avg_sq=[new(n)])
    k = -(-n // 256)
    return dict(state_bits=8, exp_avg=[new(n, dtype=F8)], exp_avg_sq=[new(n, dtype=F8)], exp_avg_scale=[new(k)],
                exp_avg_sq_scale=[new(k)])


def test_memory_that_a_step_writes_twice_is_refused(lib):
    flat, g = new(100), new(50)
    for a, b in (((0, 50), (0, 50)), ((0, 50), (49, 99)), ((10, 60), (0, 50))):
        with pytest.raises(ValueError, match="share memory"):
            vpce.vpce_adamw_plan([flat[a[0]:a[1]], flat[b[0]:b[1]]], [g, g], exp_avg=[new(50), new(50)],
                                 exp_avg_sq=[new(50), new(50)])
    with pytest.raises(ValueError, match="share memory"):
        vpce.vpce_adamw_plan([flat[:50]], [flat[25:75]], **_states(50))       # a parameter that is a gradient
    m = new(50)
    with pytest.raises(ValueError, match="share memory"):
        vpce.vpce_adamw_plan([new(50)], [g], exp_avg=[m], exp_avg_sq=[m])
    # neighbours, and one gradient for two parameters, are fine
    vpce.vpce_adamw_plan([flat[:50], flat[50:]], [g, g], exp_avg=[new(50), new(50)], exp_avg_sq=[new(50), new(50)])


@pytest.mark.parametrize("step", [None, lambda: new(2, dtype=I64), lambda: new(1)])
def test_step_number(lib, step):
    plan = vpce.vpce_adamw_plan([new(4)], [new(4)], **_states(4))
    with pytest.raises(ValueError):
        vpce.vpce_adamw_step(plan, None if step is None else step(), lr=1e-3)


def test_eight_bit_states_need_random_words_and_plans_come_from_the_library(lib):
    plan = vpce.vpce_adamw_plan([new(300)], [new(300)], **_states(300, 8))
    with pytest.raises(ValueError, match="rng"):
        vpce.vpce_adamw_step(plan, new(1, dtype=I64), lr=1e-3)
    with pytest.raises(TypeError):
        vpce.vpce_adamw_step([new(4)], new(1, dtype=I64), lr=1e-3)
    assert lib.calls == []


def test_what_the_library_gets(lib):
    p, g, t = new(300), new(300, dtype=BF16), new(1, dtype=I64)
    st = _states(300, 8)
    plan = vpce.vpce_adamw_plan([p], [g], weight_decay=[0.25], **st)
    vpce.vpce_adamw_step(plan, t, lr=1e-3, betas=(0.8, 0.9), eps=1e-6, rng=new(2, dtype=I64))
    name, args = lib.calls[-1]
    row = args[0][0]
    assert name == "vpce_adamw_step" and args[1:5] == (1, vpce.VPCE_FP32, vpce.VPCE_BF16, 8)
    assert (row.param, row.grad, row.copy, row.n, row.weight_decay) == (p.data_ptr(), g.data_ptr(), None, 300, 0.25)
    assert row.exp_avg_sq_scale == st["exp_avg_sq_scale"][0].data_ptr()
    assert args[5:11] == (t.data_ptr(), 1e-3, None, 0.8, 0.9, 1e-6)
    x, w = new(2 * S, H)[::2], new(H, dtype=BF16)
    out = new(S, H)
    r = vpce.vpce_rmsnorm_forward(x, w, eps=1e-5, out=out, rstd_out=new(S))
    args = lib.calls[-1][1]
    assert args[1:6] == (vpce.VPCE_FP32, 2 * H, None, vpce.VPCE_FP32, 0) and args[7:11] == (vpce.VPCE_BF16, 1e-5, S, H)
    assert r.residual is x and args[11] is None


def test_expanded_gradients_are_read_through_a_dense_copy(lib):
    seen = {}

    def look(name, args):
        import ctypes
        seen["dy"] = list((ctypes.c_float * (S * H)).from_address(args[0]))

    lib.at_call = look
    row = torch.arange(H, dtype=F32)
    dy = fake(row.clone()[None]).expand(S, H)
    vpce.vpce_rmsnorm_backward(dy, new(S, H), new(H), new(S), grad_in=new(S, H), grad_weight=new(H),
                               workspace=new(4096, dtype=torch.uint8))
    assert lib.calls[-1][1][2] == H and seen["dy"] == row.tolist() * S


def test_workspaces_are_contiguous_memory(lib):
    ws = new(8192, dtype=torch.uint8)[::2]
    with pytest.raises(ValueError):
        vpce.vpce_rmsnorm_backward(new(S, H), new(S, H), new(H), new(S), grad_in=new(S, H), grad_weight=new(H),
                                   workspace=ws)
    with pytest.raises(ValueError):
        vpce.vpce_grad_norm([new(4)], norm_out=new(1), scale_out=new(1), workspace=ws)
