"""Every width of rows off 16 bytes can be the first that a process asks for:
what a launch needs beyond a kernel's defaults (shared memory above 48 KB, the
kernel's static memory among it) does not come from an earlier, wider call."""
import os
import subprocess
import sys

import pytest
import torch

pytestmark = pytest.mark.gpu
ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

# widths go up, and with them every kernel's shared memory: no call is helped by
# the one before.  (16 columns apart: a row's place in the ring grows by 16 bytes
# of shared memory for every 4 or 8 columns, and each window in which static
# memory decides is 85 bytes of a row or more.)
SWEEP = """
import sys
import torch
from vocab_sharded_lm_gb300 import vpce
residual, kind = sys.argv[1] == "residual", sys.argv[2]
refused = []
for h in range(3, 17000, 16):
    for x, r in (("bf16", "bf16"), ("fp32", "fp32")) + ((("bf16", "fp32"),) if residual else ()):
        dt = {"bf16": torch.bfloat16, "fp32": torch.float32}
        a, w = torch.ones(2, h, dtype=dt[x], device="cuda"), torch.ones(h, device="cuda")
        b = torch.ones(2, h, dtype=dt[r], device="cuda") if residual else None
        try:
            if kind == "plain":
                y = vpce.vpce_rmsnorm_forward(a, w, b, eps=0.0).out
            elif kind == "gradient":
                y = 1 + vpce.vpce_rmsnorm_backward(a, a.to(dt[r]), w, torch.ones(2, device="cuda"), grad_residual=b)[0]
                y = y - 1 if residual else y
            else:
                q = vpce.vpce_rmsnorm_quantized_forward(a, w, b, eps=0.0, group=int(kind))
                y = q.q.float() * q.scale[:, :1]
            assert bool(((y.float() - 1).abs() < 1e-3).all()), (h, x, r)
        except vpce.VPCEError as e:
            refused.append((h, x, r, str(e)))
assert not refused, refused[:5]
"""


@pytest.mark.parametrize("kind", ["plain", "0", "64", "128", "gradient"])
@pytest.mark.parametrize("residual", ["residual", "none"])
def test_widths_going_up(residual, kind):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    r = subprocess.run([sys.executable, "-c", SWEEP, residual, kind], cwd=ROOT, capture_output=True, text=True,
                       timeout=300)
    assert r.returncode == 0, r.stderr[-2000:]
