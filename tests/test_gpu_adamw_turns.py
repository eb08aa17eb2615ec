"""AdamW over tensors so long that a CTA takes several turns of 2048 elements:
the slots of the 8-bit step's ring are filled again, and a block's scales are
handed on from turn to turn.  Gradients without a period, every element against
the path that takes tensors element by element, some whole runs against the
fp64 oracle (with the tolerances of tests/test_gpu_adamw.py)."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

import test_gpu_adamw as A
from test_gpu_adamw import _built  # noqa: F401  (the fixture)

pytestmark = pytest.mark.gpu
TURN, RUNS_AN_SM = 2048, 32     # elements of a turn; runs an SM that the launch aims at


def _long(x, misalign):
    flat = torch.empty(x.numel() + misalign, dtype=x.dtype, device="cuda")
    flat[misalign:].copy_(x)
    return flat[misalign:]


def _random(n, gen, std, dtype):
    return torch.empty(n, device="cuda").normal_(0.0, std, generator=gen).to(dtype)


@pytest.mark.parametrize("param,grad,copy", [("fp32", "fp32", True), ("fp32", "bf16", False), ("bf16", "bf16", False)])
@pytest.mark.parametrize("bits,turns", [(8, 3), (8, 4), (8, 10), (32, 4)])
def test_runs_of_several_turns(bits, turns, param, grad, copy):
    sms = torch.cuda.get_device_properties(0).multi_processor_count
    n = TURN * sms * RUNS_AN_SM * turns + 777
    run = TURN * turns
    gen = torch.Generator(device="cuda")
    gen.manual_seed(turns)
    dt = {"fp32": torch.float32, "bf16": torch.bfloat16}
    p, g = _random(n, gen, 1.0, dt[param]), _random(n, gen, 1e-2, dt[grad])
    if bits == 32:
        m, v = _random(n, gen, 3e-3, torch.float32), _random(n, gen, 1e-2, torch.float32).square_()
        scales = [None, None]
    else:
        m = torch.randint(0, 255, (n,), device="cuda", generator=gen, dtype=torch.uint8)
        v = torch.randint(1, 127, (n,), device="cuda", generator=gen, dtype=torch.uint8)
        m[m == 127] = 0                               # (a NaN's code)
        m, v = m.view(torch.float8_e4m3fn), v.view(torch.float8_e4m3fn)
        scales = [torch.rand(-(-n // 256), device="cuda", generator=gen).add_(1.0).mul_(k) for k in (1e-5, 3e-5)]
    lr, t, b1, b2, eps, factor, words = 1e-2, 7, 0.9, 0.95, 1e-8, 0.5, (17, (1 << 33) + 3)
    out = []
    for misalign in (0, 1):
        a = [_long(x, misalign) for x in (p, g)]
        a += [_long(x.view(torch.uint8), misalign).view(x.dtype) if bits == 8 else _long(x, misalign) for x in (m, v)]
        kw = {} if bits == 32 else dict(exp_avg_scale=[scales[0].clone()], exp_avg_sq_scale=[scales[1].clone()])
        c = [_long(p.to(torch.bfloat16), misalign)] if copy else None
        plan = vpce.vpce_adamw_plan([a[0]], [a[1]], copies=c, weight_decay=0.1, state_bits=bits, exp_avg=[a[2]],
                                    exp_avg_sq=[a[3]], **kw)
        vpce.vpce_adamw_step(plan, A._step(t), lr=lr, betas=(b1, b2), eps=eps,
                             grad_scale=torch.tensor([factor], device="cuda"), rng=A._words(*words))
        xs = [a[0], a[2], a[3]] + [xs[0] for xs in (plan.copies, plan.exp_avg_scale, plan.exp_avg_sq_scale) if xs]
        out.append([x.view(torch.uint8) if x.dtype == torch.float8_e4m3fn else x for x in xs])
    for x, y in zip(*out):
        assert torch.equal(x, y)
    # whole runs: the first, some in between, the last whole one, and what is left
    runs = -(-n // run)
    some = [0, 1, 2, runs // 3, runs // 2, runs - 2, runs - 1]
    k = np.concatenate([np.arange(i * run, min((i + 1) * run, n)) for i in some])
    kt = torch.from_numpy(k).cuda()
    bt = torch.from_numpy(np.unique(k // 256)).cuda()
    per = np.searchsorted(np.unique(k // 256), k // 256)
    f64 = lambda x, at: x[at].double().cpu().numpy() if x.dtype != torch.float8_e4m3fn else \
        x.view(torch.uint8)[at].view(torch.float8_e4m3fn).float().double().cpu().numpy()  # noqa: E731
    p0, g0, m0, v0 = (f64(x, kt) for x in (p, g, m, v))
    if bits == 8:
        m0, v0 = m0 * f64(scales[0], bt)[per], (v0 * f64(scales[1], bt)[per]) ** 2
    U, F32 = A.U, A.F32
    rp, rm, rv = T.adamw(p0, g0, m0, v0, t, F32(lr), b1, b2, F32(eps), F32(0.1), factor)
    mag_m = b1 * np.abs(m0) + (1 - b1) * np.abs(g0 * factor)
    update = F32(lr) / (1 - b1 ** t) / (np.sqrt(rv / (1 - b2 ** t)) + F32(eps))
    tol = update * mag_m * 4 * U + update * np.abs(rm) * 32 * U + 3 * U * np.abs(p0)
    half = 2.0 ** -8 if param == "bf16" else U
    got = [f64(x.view(torch.float8_e4m3fn) if x.dtype == torch.uint8 else x, kt) for x in out[0][:3]]
    assert np.all(np.abs(got[0] - rp) <= tol + half * np.abs(rp) + 1e-38)
    if copy:
        assert torch.equal(out[0][3], out[0][0].to(torch.bfloat16))
    if bits == 32:
        assert np.all(np.abs(got[1] - rm) <= 4 * U * mag_m + 1e-45)
        assert np.all(np.abs(got[2] - rv) <= 6 * U * rv + 1e-45)
        return
    kk = k.astype(np.uint64)
    halves = T.philox4x32_10((kk // 8 & 0xFFFFFFFF, 0 * kk, 0 * kk + (words[1] & 0xFFFFFFFF), 0 * kk + (words[1] >> 32)),
                             (words[0] & 0xFFFFFFFF, words[0] >> 32))
    halves = np.stack([w >> np.uint64(16 * i) & np.uint64(0xFFFF) for w in halves for i in (0, 1)], axis=1)
    u = halves[np.arange(k.size), k % 8].astype(np.int64)
    for x, codes, scale, sq in ((rm, got[1], out[0][-2], False), (np.sqrt(rv), got[2], out[0][-1], True)):
        edges = np.flatnonzero(np.diff(per, prepend=-1))
        ref = np.maximum(np.maximum.reduceat(np.abs(x), edges) / 448.0, T.TINY)
        slack = 0 if sq else np.maximum.reduceat(mag_m, edges) / 448 * 4 * U
        assert np.all(np.abs(f64(scale, bt) - ref) <= 8 * U * ref + slack + 1e-45)
        want, far = T.stochastic_codes(x, ref[per], u, sq)
        off = codes != want
        grow = 1.0 if sq else np.maximum(1.0, mag_m / np.maximum(np.abs(rm), 1e-300))
        assert np.all((far <= 2.0 * grow)[off]) and off.mean() < 1e-2
