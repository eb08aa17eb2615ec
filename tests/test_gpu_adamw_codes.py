"""The 8-bit codes of m are those of a plain fp32 evaluation where the scale is
next to fp32's smallest numbers too, as in rows of a table that have had no
gradient for long.  The values are made so that a quotient that is one ulp off
takes the other code: bit for bit, no tolerance."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
f32 = np.float32


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


def _place(q, u):
    """Whether the code above is taken: the 20 bits below e4m3's against 2^20 (u + 1/2) / 2^16."""
    return (np.asarray(q, f32).view(np.int32) & 0xFFFFF) > 16 * u + 8


def _one_ulp_off(x, s):
    """x (1 / s) with one residual step in fp32: what the residual's underflow leaves."""
    inv = f32(1) / s
    q = x * inv
    r = (x.astype(np.float64) - q.astype(np.float64) * np.float64(s)).astype(f32)
    return (q.astype(np.float64) + r.astype(np.float64) * np.float64(inv)).astype(f32)


def _block(s_exponent, u, r, smallest):
    """256 values whose largest sets a scale of about 2^s_exponent, and how many
    of them lie where a quotient one ulp off takes the other code."""
    while True:
        top = f32(r.uniform(1, 2) * 448 * 2.0 ** s_exponent)
        s = top * f32(1 / 448)
        if top / s <= 448:
            break
    x = np.full(256, top, f32)
    edges = 0
    for k in range(1, 256):
        for _ in range(8):
            # the code's own bits, and the last place below the border or the first above it
            code = r.integers(smallest, 0x7E)
            word = (code << 20) + (960 << 20) | int(16 * u[k] + 8 + r.integers(0, 2))
            x[k] = np.array([word], np.int32).view(f32)[0] * s
            near = (x[k:k + 1].view(np.int32) + np.arange(-4, 5)).astype(np.int32).view(f32)
            near = near[near < top]
            at = np.flatnonzero(_place(near / s, u[k]) != _place(_one_ulp_off(near, s), u[k]))
            if at.size:
                x[k] = near[at[0]]
                edges += 1
                break
    return x, edges


@pytest.mark.parametrize("v0", [0.0, 1.0], ids=["v zero", "v ordinary"])
@pytest.mark.parametrize("smallest", [0x08, 0x38], ids=["from 2^-6", "from 1"])
@pytest.mark.parametrize("misalign", [0, 1])
def test_codes_of_m_at_the_smallest_scales(misalign, smallest, v0):
    # beta1 = 0: m is the gradient.  A whole number of turns of 2048 elements: the
    # vector path is the one through shared memory; and one element by itself
    blocks, r = 24, np.random.default_rng(7 + smallest)
    n = blocks * 256
    u = T.random_halves(n, 0, 5, 9)
    made = [_block(-108 - b % 18, u[b * 256:(b + 1) * 256], r, smallest) for b in range(blocks)]
    assert sum(e for _, e in made) >= 40               # (the test would say nothing otherwise)
    x = np.concatenate([m for m, _ in made]) * np.where(r.random(n) < 0.5, f32(-1), f32(1))
    flat = torch.zeros(n + misalign, device="cuda")
    g = flat[misalign:]
    g.copy_(torch.from_numpy(x))
    p = torch.zeros(n + misalign, device="cuda")[misalign:]
    codes = [torch.zeros(n + misalign, dtype=torch.float8_e4m3fn, device="cuda")[misalign:] for _ in range(2)]
    codes[1].copy_(torch.full((n,), v0, device="cuda"))
    scales = [torch.full((blocks,), 1.0, device="cuda") for _ in range(2)]
    plan = vpce.vpce_adamw_plan([p], [g], weight_decay=0.0, state_bits=8, exp_avg=[codes[0]], exp_avg_sq=[codes[1]],
                                exp_avg_scale=[scales[0]], exp_avg_sq_scale=[scales[1]])
    vpce.vpce_adamw_step(plan, torch.ones(1, dtype=torch.int64, device="cuda"), lr=1e-3, betas=(0.0, 0.9),
                         rng=torch.tensor([5, 9], dtype=torch.int64, device="cuda"))
    m = np.abs(x).reshape(blocks, 256)
    s = m.max(axis=1) * f32(1 / 448)
    assert np.array_equal(scales[0].cpu().numpy(), s)
    q = (m / s[:, None]).reshape(-1)
    word = q.view(np.int32)
    want = ((word >> 20) - 960 + _place(q, u)).clip(max=0x7E) | np.where(x < 0, 0x80, 0)
    got = codes[0].view(torch.uint8).cpu().numpy().astype(np.int64)
    assert np.array_equal(got, want), (got != want).sum()
