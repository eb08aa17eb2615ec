"""The pieces of a training step run together: lookup with dropout into a
residual stream, the norm with the residual's addition, the LM head's one-call
training step, the norm's gradient, the table's gradient, the norm of all
gradients and the AdamW step of table, head and gain with bf16 copies, which
the next step reads.  Gradients against fp64 autograd of the same model, the
update against the fp64 formula, eager steps against a captured one."""
import math

import numpy as np
import pytest
import torch

from oracle import scores_oracle as S
from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
V, H, ROWS, VS, P, EPS = 700, 128, 192, [0, 250, 700], 0.25, 1e-5


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


class Ends:
    """The two ends of a model; what lies between is a fixed branch."""

    def __init__(self, bits, seed=3):
        r = np.random.default_rng(seed)
        dev = lambda x, dt: torch.from_numpy(x).to(dt).cuda()  # noqa: E731
        table, head = r.normal(size=(V, H)) / math.sqrt(H), r.normal(size=(V, H)) / math.sqrt(H)
        f32, b16 = torch.float32, torch.bfloat16
        split = lambda x, dt: [dev(x[VS[i]:VS[i + 1]], dt) for i in range(2)]  # noqa: E731
        self.master = split(table, f32) + split(head, f32) + [dev(1 + 0.1 * r.normal(size=H), f32)]
        self.live = [w.to(b16) for w in self.master]
        self.grads = [torch.zeros_like(w) for w in self.master]
        self.branch = dev(r.normal(size=(ROWS, H)), b16)
        self.ids, self.targets = dev(r.integers(0, V, ROWS), torch.int64), dev(r.integers(0, V, ROWS), torch.int64)
        self.targets[::7] = -100
        self.rng = torch.tensor([77, 3], dtype=torch.int64, device="cuda")
        self.step = torch.tensor([1], dtype=torch.int64, device="cuda")
        self.plan = vpce.vpce_adamw_plan(self.master, self.grads, copies=self.live, state_bits=bits,
                                         weight_decay=[0.1] * 4 + [0.0])
        self.ws = torch.empty(vpce.vpce_lmhead_forward_backward_workspace_bytes(ROWS, V, H), dtype=torch.uint8,
                              device="cuda")
        self.loss = torch.zeros((), device="cuda")

    def backward(self):
        """Loss and gradients, into ``grads``."""
        for g in self.grads[2:4]:
            g.zero_()                                          # the head's are accumulated
        table, head, gain = self.live[:2], self.live[2:4], self.live[4]
        stream = vpce.vpce_embedding_dropout_forward(table, self.ids, VS, scale=math.sqrt(H), p=P, rng=self.rng)
        n = vpce.vpce_rmsnorm_forward(self.branch, gain, stream, eps=EPS, residual_out=stream)
        _, dx, _ = vpce.vpce_lmhead_forward_backward(n.out, head, self.targets, VS, loss_out=self.loss,
                                                     grad_weight_shards=self.grads[2:4], workspace=self.ws)
        dstream, _ = vpce.vpce_rmsnorm_backward(dx, n.residual, gain, n.rstd, grad_weight=self.grads[4])
        vpce.vpce_embedding_dropout_backward(dstream, self.ids, self.grads[:2], VS, scale=math.sqrt(H), p=P,
                                             rng=self.rng, accumulate=False)

    def update(self):
        self.norm, scale = vpce.vpce_grad_norm(self.plan, 0.5)
        vpce.vpce_adamw_step(self.plan, self.step, lr=1e-2, betas=(0.9, 0.95), grad_scale=scale, rng=self.rng)

    def train(self):
        self.backward()
        self.update()
        self.step += 1
        self.rng[1] += 1

    def all(self):
        xs = self.master + self.live + self.plan.exp_avg + self.plan.exp_avg_sq + [self.loss]
        return [x.view(torch.uint8).clone() if x.dtype == torch.float8_e4m3fn else x.clone() for x in xs]


def _rounded(x):
    """x as bf16 holds it, its gradient passed on."""
    return x + (x.detach().to(torch.bfloat16).double() - x.detach())


def test_gradients_match_autograd():
    m = Ends(32)
    m.backward()
    table, head, gain = (torch.cat([w.double().cpu() for w in ws]).requires_grad_()
                         for ws in (m.live[:2], m.live[2:4], m.live[4:]))
    ids, y = m.ids.cpu(), m.targets.cpu()
    keep = torch.from_numpy(S.keep_mask(77, 3, ROWS, H, P)).double()
    x = _rounded(table[ids] * (math.sqrt(H) * 65536 / (65536 - S.drop_threshold(P))) * keep)
    r = m.branch.double().cpu() + x
    out = _rounded(r * (r.pow(2).mean(1, keepdim=True) + EPS).rsqrt() * gain)
    loss = torch.nn.functional.cross_entropy(out @ head.T, y, ignore_index=-100)
    loss.backward()
    assert abs(m.loss.item() - loss.item()) <= 1e-5 * loss.item()
    # dlogits, their product dX and the stream's gradient are held in bf16
    # (2^-8 of an element each at most), the stored sum too: 1.5% of the norm
    # covers the four of them without any averaging
    for got, want in ((m.grads[:2], table.grad), (m.grads[2:4], head.grad), (m.grads[4:], gain.grad)):
        got = torch.cat([g.double().cpu() for g in got])
        assert (got - want).norm() <= 2.0 ** -6 * want.norm()


@pytest.mark.parametrize("bits", [32, 8])
def test_update_matches_the_formula(bits):
    m = Ends(bits)
    m.backward()
    grads = [g.double().cpu().numpy() for g in m.grads]
    before = [w.double().cpu().numpy() for w in m.master]
    m.update()
    norm, scale = T.grad_norm(grads, 0.5)
    assert norm > 0.5 and abs(m.norm.item() - norm) <= 1e-5 * norm
    for i, (w, g) in enumerate(zip(before, grads)):
        p, _, _ = T.adamw(w, g, 0 * w, 0 * w, 1, float(np.float32(1e-2)), 0.9, 0.95, float(np.float32(1e-8)),
                          float(np.float32(m.plan._table[i].weight_decay)), scale)
        # in the first step the update is lr g / (|g| + eps): 40 roundings of it,
        # the clipping factor's error (2e-5) only where |g| is near eps
        tol = 1e-2 * (40 * 2.0 ** -24 + 2e-5 * 1e-8 / (np.abs(g * scale) + 1e-8)) + 4 * 2.0 ** -24 * np.abs(w)
        assert np.all(np.abs(m.master[i].double().cpu().numpy() - p) <= tol)
        assert torch.equal(m.live[i], m.master[i].to(torch.bfloat16))


@pytest.mark.parametrize("bits", [32, 8])
def test_a_captured_step_goes_on_as_eager_ones_do(bits):
    a, b = Ends(bits), Ends(bits)
    for _ in range(4):
        a.train()
    b.train()                                                  # set-up, and the first step
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        b.train()
    for _ in range(3):
        graph.replay()
    torch.cuda.synchronize()
    assert b.step.item() == a.step.item() == 5
    assert all(torch.equal(x, y) for x, y in zip(a.all(), b.all()))


@pytest.mark.parametrize("bits", [32, 8])
def test_the_policy_example_runs_with_adamw(bits):
    import os
    import sys

    sys.path.insert(0, os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "examples"))
    import policy_step as E

    history = E.main(["--steps", "4", "--tokens", "256", "--vocab", "2000", "--hidden", "128", "--shards", "3",
                      "--optimizer", "adamw", "--state-bits", str(bits)])
    assert len(history) == 4 and all(math.isfinite(x) for x in history)
