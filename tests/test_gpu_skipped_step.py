"""A step that is skipped because its gradients are not finite is not counted:
the bias corrections 1 - beta^t of later steps are those of the updates that m
and v have had."""
import os
import sys

import numpy as np
import pytest
import torch

from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


@pytest.mark.parametrize("bits", [32, 8])
def test_the_example_does_not_count_a_skipped_step(monkeypatch, bits):
    import policy_step as E

    inner, step, numbers, moved = E.policy_step, vpce.vpce_adamw_step, [], []

    def policy_step(table, grads, *args, **kw):
        result = inner(table, grads, *args, **kw)
        if len(numbers) in (0, 2):
            grads[0][0, 0] = float("inf")
        return result

    def adamw_step(plan, number, **kw):
        before = plan.params[0].clone()
        step(plan, number, **kw)
        numbers.append(number.item())
        moved.append(not torch.equal(before, plan.params[0]))

    monkeypatch.setattr(E, "policy_step", policy_step)
    monkeypatch.setattr(vpce, "vpce_adamw_step", adamw_step)
    E.main(["--steps", "5", "--tokens", "64", "--vocab", "500", "--hidden", "64", "--shards", "2", "--optimizer",
            "adamw", "--state-bits", str(bits)])
    assert moved == [False, True, False, True, True]
    assert numbers == [0, 1, 1, 2, 3]


def test_an_update_after_a_skipped_step_is_the_formulas():
    # p, m and v after steps 1 and 2 with a skipped one between them; tolerances:
    # an update is within 40 roundings of it, two of them, p's own 4 roundings
    n, lr, eps, rg = 1000, 1e-2, 1e-8, np.random.default_rng(0)
    g = [rg.normal(size=n).astype(np.float32) for _ in range(3)]
    p = torch.zeros(n, device="cuda")
    grad, number = torch.zeros(n, device="cuda"), torch.zeros(1, dtype=torch.int64, device="cuda")
    plan = vpce.vpce_adamw_plan([p], [grad], weight_decay=0.0)
    for k in range(3):
        grad.copy_(torch.from_numpy(g[k]))
        if k == 1:
            grad[7] = float("nan")
        _, scale = vpce.vpce_grad_norm(plan)
        number += scale != 0
        vpce.vpce_adamw_step(plan, number, lr=lr, betas=(0.9, 0.95), eps=eps, grad_scale=scale)
    want, m, v = np.zeros(n), np.zeros(n), np.zeros(n)
    for t, k in ((1, 0), (2, 2)):
        want, m, v = T.adamw(want, g[k].astype(np.float64), m, v, t, float(np.float32(lr)), 0.9, 0.95,
                             float(np.float32(eps)), 0.0)
    # (an update is at most lr (1 - beta1) / sqrt(1 - beta2) and some: 3 lr bounds it here)
    assert np.all(np.abs(p.double().cpu().numpy() - want) <= 2 * 3 * lr * 40 * 2.0 ** -24)
    assert number.item() == 2
