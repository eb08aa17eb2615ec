"""Token scores of long rows against fp64 on the device, with the error that
the sums' own structure gives (eps = 2^-24).

A row of V columns is cut into at most 40 pieces whose length doubles from 512
16-byte vectors on, so a piece has at most V / (20 E) + 512 vectors (E columns
each).  A lane takes a 32nd of them into four running sums, V / 2560 + 4 E
additions each; every 256 vectors the four are added and may be moved to a new
offset, at most 5 roundings; the warp's tree and the fold of the pieces add 12.
An exponential carries at most 8 eps in all.  So S is within
    A = V / 2560 + 4 E + 5 (V / (5120 E) + 2) + 12 + 8
roundings, ln S within A eps absolutely, logp within that and 4 eps of its value
(difference, quotient, subtraction).  U's terms carry the same relative errors,
and |U| / S <= 1 + ln V: the entropy is within A eps (2 + ln V)."""
import math

import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
EPS = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


@pytest.mark.parametrize("s,V,t,dtype", [(64, 128256, 8, "bf16"), (64, 152064, 8, "fp32"), (1, 256000, 16, "bf16"),
                                         (3, 1 << 20, 1, "bf16"), (17, 50259, 3, "fp32")])
def test_sums_are_as_good_as_their_structure(s, V, t, dtype):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(2 * V + s)
    dt, E = (torch.bfloat16, 8) if dtype == "bf16" else (torch.float32, 4)
    z = torch.empty(s, V, dtype=dt, device="cuda").normal_(0, 2, generator=gen)
    vs = [i * (V // t) for i in range(t)] + [V]
    y = torch.randint(0, V, (s,), device="cuda", generator=gen)
    r = vpce.vpce_logprob_forward([z[:, vs[i]:vs[i + 1]].contiguous() for i in range(t)], y, vs)
    lp = torch.log_softmax(z.double(), 1)
    want = lp.gather(1, y[:, None])[:, 0]
    A = V / 2560 + 4 * E + 5 * (V / (5120 * E) + 2) + 12 + 8
    err = (r.logp.double() - want).abs()
    assert bool((err <= EPS * (A + 4 * want.abs())).all()), float((err / EPS).max())
    ent = -(lp.exp() * lp).sum(1)
    err = (r.entropy.double() - ent).abs()
    assert float(err.max()) <= EPS * A * (2 + math.log(V)), float((err / EPS).max())
