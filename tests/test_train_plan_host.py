"""An AdamW plan writes at the addresses of its making: a tensor of any of its
lists that is elsewhere by the time of a step is refused, and what the plan's
addresses point at stays allocated as long as the plan lives."""
import pytest
import torch
from torch.multiprocessing.reductions import StorageWeakRef

from vocab_sharded_lm_gb300 import vpce

from _fake_cuda import Fake0, install

F32, BF16, I64, F8 = torch.float32, torch.bfloat16, torch.int64, torch.float8_e4m3fn
SIZES = (300, 5, 1000)
LISTS = ["params", "grads", "copies", "exp_avg", "exp_avg_sq", "exp_avg_scale", "exp_avg_sq_scale"]


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch, vpce)


def new(n, dtype=F32):
    # (not a view, which would keep its base's memory)
    return torch.Tensor._make_subclass(Fake0, torch.zeros(n, dtype=dtype))


def _plan(bits, copies=True):
    per = lambda dtype, d=1: [new(-(-n // d), dtype) for n in SIZES]  # noqa: E731
    kw = dict(exp_avg=per(F32), exp_avg_sq=per(F32)) if bits == 32 else \
        dict(exp_avg=per(F8), exp_avg_sq=per(F8), exp_avg_scale=per(F32, 256), exp_avg_sq_scale=per(F32, 256))
    return vpce.vpce_adamw_plan(per(F32), per(F32), copies=per(BF16) if copies else None, state_bits=bits, **kw)


def _step(plan):
    vpce.vpce_adamw_step(plan, new(1, I64), lr=1e-3, rng=new(2, I64))


def _elsewhere(x):
    """The tensor's values in other memory, as a module's conversion, a load or an
    offload and its return leave them."""
    x.data = x.data.clone()


@pytest.mark.parametrize("which", range(len(SIZES)))
@pytest.mark.parametrize("bits,name", [(b, n) for b in (32, 8) for n in LISTS if b == 8 or "scale" not in n])
def test_a_step_with_moved_memory_is_refused(lib, bits, name, which):
    plan = _plan(bits)
    _step(plan)
    assert len(lib.calls) == 1
    x = getattr(plan, name)[which]
    held = x.data
    _elsewhere(x)
    with pytest.raises(ValueError, match="moved"):
        _step(plan)
    assert len(lib.calls) == 1
    x.data = held
    _step(plan)
    assert len(lib.calls) == 2


@pytest.mark.parametrize("name", LISTS)
def test_a_replaced_entry_is_refused(lib, name):
    plan = _plan(8)
    xs = getattr(plan, name)
    xs[1] = xs[1].clone()
    with pytest.raises(ValueError, match="moved"):
        _step(plan)
    assert lib.calls == []


def test_the_gradient_norm_asks_for_the_gradients_alone(lib):
    kw = dict(norm_out=new(1), scale_out=new(1), workspace=new(4096, torch.uint8))
    plan = _plan(32)
    _elsewhere(plan.params[0])
    vpce.vpce_grad_norm(plan, 1.0, **kw)
    assert len(lib.calls) == 1
    _elsewhere(plan.grads[2])
    with pytest.raises(ValueError, match="moved"):
        vpce.vpce_grad_norm(plan, 1.0, **kw)
    assert len(lib.calls) == 1


@pytest.mark.parametrize("name", LISTS)
def test_the_plan_keeps_the_memory_that_it_points_at(lib, name):
    plan = _plan(8)
    x = getattr(plan, name)[2]
    memory = StorageWeakRef(x.untyped_storage())
    x.data = torch.zeros(0, dtype=x.dtype)
    assert not memory.expired()
    del plan, x
    assert memory.expired()


def test_lists_without_copies_and_with_empty_tensors(lib):
    _step(_plan(32, copies=False))
    plan = vpce.vpce_adamw_plan([new(0), new(4)], [new(0), new(4)], exp_avg=[new(0), new(4)], exp_avg_sq=[new(0), new(4)])
    _step(plan)
    assert len(lib.calls) == 2
