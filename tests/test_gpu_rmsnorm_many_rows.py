"""The norm and its gradient over so many rows that every team of threads takes
several, each with other values, against the fp64 oracle: rows' slots in shared
memory are filled again, the two halves of the reductions' words take turns, and
a group's words belong to one row after another.

The rows that a launch holds at once are its CTAs times the teams of a CTA, and
its slots are that times the rows of a ring.  With 152 SMs, from the launches'
own rules: 64 CTAs an SM without a ring (four rows each up to 1024 columns), one
an SM with one, of 512 threads' worth of teams and at most 3 rows (gradient in
vectors: 8 in bf16 up to 256 columns, 4 up to 8192)."""
import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

import test_gpu_rmsnorm as R
from test_gpu_rmsnorm import _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
SMS = 152

FORWARD = [
    # s, h, x, residual, weight, pad, misalign; rows at once (with their slots)
    ((40001, 64, "bf16", "bf16", "bf16", 0, 0), 64 * 4),
    ((40001, 256, "fp32", None, "bf16", 0, 0), 64 * 4),
    ((10001, 1032, "bf16", "fp32", "bf16", 0, 0), 64),
    ((10001, 2048, "bf16", "bf16", "fp32", 0, 0), 64),
    ((700, 8200, "bf16", "bf16", "bf16", 0, 0), 4),
    ((500, 8200, "fp32", "fp32", "fp32", 0, 0), 2),
    ((700, 16384, "bf16", "fp32", "bf16", 0, 0), 3),
    ((10001, 131, "fp32", "fp32", "fp32", 0, 0), 16 * 4),
    ((2501, 1031, "bf16", "bf16", "bf16", 1, 3), 4 * 4),
    ((700, 8199, "bf16", None, "fp32", 0, 0), 4),
    ((500, 17001, "bf16", "fp32", "bf16", 0, 0), 3),
]
BACKWARD = [
    ((22001, 72, "bf16", "bf16", "bf16", 0, 0), 16 * 9),
    ((12501, 256, "fp32", "fp32", "fp32", 0, 0), 16 * 5),
    ((1601, 4096, "bf16", "bf16", "bf16", 0, 0), 2 * 5),
    ((1001, 4104, "bf16", "fp32", "bf16", 0, 0), 3),
    ((1001, 4096, "fp32", None, "fp32", 0, 0), 2 * 3),
    ((700, 16384, "bf16", "bf16", "fp32", 0, 0), 3),
    ((500, 9000, "bf16", "fp32", "bf16", 0, 0), 2),
    ((500, 17008, "bf16", "bf16", "bf16", 0, 0), 2),
    ((10001, 131, "fp32", "fp32", "fp32", 0, 0), 16 * 4),
    ((2501, 1031, "bf16", "bf16", "bf16", 1, 3), 4 * 4),
    ((700, 8199, "bf16", None, "fp32", 0, 0), 4),
    ((500, 17001, "bf16", "fp32", "bf16", 0, 0), 3),
]


def _several_each(s, at_once):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    assert s > sms * at_once or sms > SMS, "rows for every team to come round again"


@pytest.mark.parametrize("case,at_once", FORWARD, ids=lambda v: f"{v[0]}x{v[1]}-{v[2]}-{v[3]}" if type(v) is tuple else "")
def test_forward(case, at_once):
    _several_each(case[0], at_once)
    R.test_forward_matches_the_oracle(*case)


@pytest.mark.parametrize("group", [0, 48, 128])
@pytest.mark.parametrize("case,at_once", FORWARD, ids=lambda v: f"{v[0]}x{v[1]}-{v[2]}-{v[3]}" if type(v) is tuple else "")
def test_quantized_forward(case, at_once, group):
    R.test_quantized_forward_matches_the_oracle(*case, group)


@pytest.mark.parametrize("case,at_once", BACKWARD, ids=lambda v: f"{v[0]}x{v[1]}-{v[2]}-{v[3]}" if type(v) is tuple else "")
def test_backward(case, at_once):
    _several_each(case[0], at_once)
    R.test_backward_matches_the_oracle(*case, False)


@pytest.mark.parametrize("s,h", [(40001, 64), (10001, 1032), (10001, 131), (2501, 1031), (700, 8200), (700, 8199),
                                 (500, 17001)])
def test_in_place(s, h):
    # rows that are written while others are on their way: the bits of the calls
    # into other memory, which the tests above compare with the oracle
    xs, _ = R._rows(1, s, h, "bf16")
    rs, _ = R._rows(2, s, h, "bf16", 2.0)
    w, _ = R._rows(3, 1, h, "bf16")
    ref = vpce.vpce_rmsnorm_forward(xs, w[0], rs)
    dx, dw = vpce.vpce_rmsnorm_backward(xs, ref.residual, w[0], ref.rstd, grad_residual=rs)
    x2, r2 = xs.clone(), rs.clone()
    vpce.vpce_rmsnorm_forward(x2, w[0], r2, out=x2, residual_out=r2)
    assert torch.equal(x2, ref.out) and torch.equal(r2, ref.residual)
    for k in range(3):
        a, b, c = xs.clone(), ref.residual.clone(), rs.clone()
        dx2, dw2 = vpce.vpce_rmsnorm_backward(a, b, w[0], ref.rstd, grad_residual=c, grad_in=(a, b, c)[k])
        assert torch.equal(dx2, dx) and torch.equal(dw2, dw)
