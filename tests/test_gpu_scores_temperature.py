"""Token scores at the ends of the accepted temperatures, where (largest logit)
/ T is too large for sums relative to a common offset, and just below that.

Tolerances: those of test_gpu_logprob.py hold unchanged.  The exponent of a
column is (z - max) / T with the same three roundings whatever T is, whether it
is formed by subtraction or by one fused multiply-add from the rounded offset
(whose rounding is added back to ln S and cancels in the entropy), and |u| e^u
<= 1 / e bounds what they do to the sums.  The outputs are fp32: a log
probability below its range (a column at the type's lowest value, divided by a
small temperature) is -inf."""
import numpy as np
import pytest
import torch

from oracle import scores_oracle as S
from vocab_sharded_lm_gb300 import vpce

from test_gpu_logprob import LOW, _built, _check_backward, _check_forward, _place  # noqa: F401

pytestmark = pytest.mark.gpu
V, VS, ROWS, TOP = 2049, [0, 700, 1333, 2049], 40, 9


def _logits(kind, dtype, T):
    """[ROWS, V] fp64 of representable values.  near x: a distribution of
    several likely columns around x at this temperature."""
    r = np.random.default_rng(11)
    if kind == "spread":
        x = r.normal(0, 3, (ROWS, V))
    else:
        x = float(kind.split()[1]) + r.normal(0, 1.5, (ROWS, V)) * T
    z = torch.from_numpy(x).to(torch.bfloat16 if dtype == "bf16" else torch.float32).double().numpy()
    z[3, ::2] = -np.inf
    z[4] = LOW[dtype]
    z[5] = -np.inf
    z[6, 1:] = LOW[dtype]
    return z


CASES = [(T, dtype, kind) for T in (1e-30, 1e-5, 3e-4, 1e30) for dtype in ("bf16", "fp32")
         for kind in ("spread", "near 5", "near 20") if T < 1 or kind == "spread"]


@pytest.mark.parametrize("T,dtype,kind", CASES)
def test_forward(T, dtype, kind):
    T = float(np.float32(T))
    z = _logits(kind, dtype, T)
    y = np.random.default_rng(12).integers(0, V, ROWS)
    y[7], y[6] = -100, 0
    flag = torch.full((1,), 3, dtype=torch.int32, device="cuda")
    r = vpce.vpce_logprob_forward(_place(z, VS, dtype, "columns"), torch.from_numpy(y).cuda(), VS, top=TOP,
                                  temperature=T, flag=flag)
    assert flag.item() == 0
    ref = S.token_scores(z, y, TOP, T)
    for name in ("logp", "top_logp"):
        ref[name] = np.where(ref[name] < -np.finfo(np.float32).max, -np.inf, ref[name])
    _check_forward(r, ref, V)


@pytest.mark.parametrize("T,dtype,kind", CASES)
def test_backward(T, dtype, kind):
    T = float(np.float32(T))
    z = _logits(kind, dtype, T)
    r = np.random.default_rng(13)
    y = r.integers(0, V, ROWS)
    y[7], y[3] = -100, 1
    ids = S.token_scores(z, y, 3, T)["top_ids"]
    _check_backward(z, y, VS, dtype, "dense", T, r.normal(size=ROWS), r.normal(size=ROWS), ids,
                    r.normal(size=(ROWS, 3)), False)
