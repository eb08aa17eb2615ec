"""The policy-gradient example runs the scores and the embedding together:
its table gradient against fp64 autograd of the same model, and a few steps
that raise the rewarded tokens' probability."""
import math
import os
import sys

import numpy as np
import pytest
import torch

from oracle import scores_oracle as S

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
sys.path.insert(0, os.path.join(ROOT, "examples"))

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build, vpce

    _build.build()
    vpce.load_library()


def test_gradient_matches_autograd():
    import policy_step as E

    V, h, s, p, T, beta = 700, 64, 96, 0.25, 1.3, 0.05
    vs = [0, 250, 700]
    r = np.random.default_rng(3)
    table = torch.from_numpy(r.normal(size=(V, h)) / math.sqrt(h)).to(torch.bfloat16)
    ids, y = torch.from_numpy(r.integers(0, V, s)), torch.from_numpy(r.integers(0, V, s))
    y[::7] = -100
    ids[3] = 5                                     # the padding id
    adv = torch.from_numpy(r.normal(size=s)).float()
    rng = torch.tensor([77, 3], dtype=torch.int64, device="cuda")
    shards = [table[vs[i]:vs[i + 1]].cuda() for i in range(2)]
    grads = [torch.empty(w.shape, device="cuda") for w in shards]
    obj, scores = E.policy_step(shards, grads, ids.cuda(), y.cuda(), adv.cuda(), vs, beta=beta, p=p, rng=rng,
                                padding_id=5, top=3, temperature=T)
    # the same in fp64, with the hidden states and logits rounded to bf16 where the model keeps them
    w = table.double().requires_grad_()
    keep = torch.from_numpy(S.keep_mask(77, 3, s, h, p)).double()
    drop = S.drop_threshold(p)
    x = w[ids] * (math.sqrt(h) * 65536 / (65536 - drop)) * keep * (ids != 5).double()[:, None]
    x = x + (x.detach().to(torch.bfloat16).double() - x.detach())
    z = x @ w.T
    z = z + (z.detach().to(torch.bfloat16).double() - z.detach())
    lp = torch.log_softmax(z / T, 1)
    live = y != -100
    pick = lp.gather(1, y.clamp(min=0)[:, None])[:, 0]
    ent = -(lp.exp() * lp).sum(1)
    ref = -((adv.double() * pick + beta * ent)[live]).sum() / live.sum()
    ref.backward()
    # bf16 logits round at a different place in the two products (half an ulp
    # of logits below 16 is 2^-5), dlogits and dhidden round to bf16 (2^-9
    # each), and so does the product with the hidden states
    assert abs(obj.item() - ref.item()) <= 2.0 ** -5
    got = torch.cat(grads).double().cpu()
    err = (got - w.grad).norm() / w.grad.norm()
    assert err <= 2e-2, err
    assert scores.top_ids.shape == (s, 3)


def test_steps_raise_the_rewarded_tokens():
    import policy_step as E

    history = E.main(["--steps", "8", "--tokens", "256", "--vocab", "2000", "--hidden", "128", "--shards", "3"])
    assert history[-1] > history[0] + 0.05
