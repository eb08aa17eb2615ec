"""GPU parity of the AdamW step and the gradient norm with the fp64 oracle.

With u = 2^-24 (half a step of fp32):
* m: two products and a sum, beta and 1 - beta rounded once each: 4 u of the
  terms' magnitudes; v: 6 u of v (three products).
* the update lr m / den: m's own error over den, and 32 u of the update for
  the roots, the bias corrections (each within 2 ulp of a value that an error
  u of t ln(beta) moves by at most u), the quotient (2 ulp) and the rates.
* param: 3 u of the old one besides, and half a step of its type.
* 8-bit states: scales within 8 u of the exact ones; a code differs from the
  exact arithmetic's only where the random number lies within 2 units of 2^-16
  of the border: a value known within 8 u moves the border's place by at most
  16 x 8 u (a step of e4m3 is at least 1/16 of a normal value), 0.5 units,
  squares by twice that."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
U = 2.0 ** -24
F32 = lambda v: float(np.float32(v))  # noqa: E731


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


def _words(seed, offset):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


def _step(t):
    return torch.tensor([t], dtype=torch.int64, device="cuda")


def _on_gpu(x, dtype, misalign=0):
    """A contiguous copy, `misalign` elements past 512 bytes."""
    flat = torch.empty(x.size + misalign, dtype=dtype, device="cuda")
    v = flat[misalign:]
    v.copy_(torch.from_numpy(np.ascontiguousarray(x)).to(torch.float32))
    return v


def _np(x):
    return x.float().double().cpu().numpy() if x.dtype != torch.float64 else x.cpu().numpy()


class Model:
    """Tensors of some sizes with gradients and states."""

    def __init__(self, sizes, param="fp32", grad="fp32", copy=False, bits=32, misalign=0, seed=0, zero=False):
        r = np.random.default_rng(seed)
        self.sizes = sizes
        self.params = [_on_gpu(r.normal(size=n), DT[param], misalign) for n in sizes]
        self.grads = [_on_gpu(r.normal(size=n) * 1e-2, DT[grad], misalign) for n in sizes]
        self.copies = [_on_gpu(r.normal(size=n), torch.bfloat16, misalign) for n in sizes] if copy else None
        self.decays = [0.1 * (i % 3) for i in range(len(sizes))]
        self.bits = bits
        kw = {}
        if not zero:
            m = [r.normal(size=n) * 3e-3 for n in sizes]
            v = [r.uniform(0.01, 2, size=n) * 1e-4 for n in sizes]
            if bits == 32:
                kw = dict(exp_avg=[_on_gpu(x, torch.float32, misalign) for x in m],
                          exp_avg_sq=[_on_gpu(x, torch.float32, misalign) for x in v])
            else:
                grid = T.e4m3_grid()
                code = lambda n, low: grid[r.integers(low, 127, n)]  # noqa: E731
                sign = [np.where(r.random(n) < 0.5, -1.0, 1.0) for n in sizes]
                kw = dict(exp_avg=[_on_gpu(code(n, 0) * s, torch.float8_e4m3fn, misalign)
                                   for n, s in zip(sizes, sign)],
                          exp_avg_sq=[_on_gpu(code(n, 1), torch.float8_e4m3fn, misalign) for n in sizes],
                          exp_avg_scale=[_on_gpu(r.uniform(1, 2, -(-n // 256)) * 1e-5, torch.float32) for n in sizes],
                          exp_avg_sq_scale=[_on_gpu(r.uniform(1, 2, -(-n // 256)) * 3e-5, torch.float32)
                                            for n in sizes])
        self.plan = vpce.vpce_adamw_plan(self.params, self.grads, copies=self.copies, weight_decay=self.decays,
                                         state_bits=bits, **kw)

    def states(self, i):
        m, v = _np(self.plan.exp_avg[i]), _np(self.plan.exp_avg_sq[i])
        if self.bits == 8:
            n = self.sizes[i]
            m = m * np.repeat(_np(self.plan.exp_avg_scale[i]), 256)[:n]
            v = (v * np.repeat(_np(self.plan.exp_avg_sq_scale[i]), 256)[:n]) ** 2
        return m, v

    def snapshot(self):
        return [(_np(p), _np(g), *self.states(i)) for i, (p, g) in enumerate(zip(self.params, self.grads))]

    def everything(self):
        lists = [self.params, self.plan.exp_avg, self.plan.exp_avg_sq, self.copies or [],
                 self.plan.exp_avg_scale or [], self.plan.exp_avg_sq_scale or []]
        return [x.view(torch.uint8).clone() if x.dtype == torch.float8_e4m3fn else x.clone()
                for xs in lists for x in xs]


def _check(model, before, t, lr, b1, b2, eps, scale, words=(0, 0)):
    for i, (p, g, m, v) in enumerate(before):
        if p.size == 0:
            continue
        wd = F32(model.decays[i])
        rp, rm, rv = T.adamw(p, g, m, v, max(t, 1), F32(lr), b1, b2, F32(eps), wd, scale)
        mag_m = b1 * np.abs(m) + (1 - b1) * np.abs(g * scale)
        den = np.sqrt(rv / (1 - b2 ** max(t, 1))) + F32(eps)
        update = F32(lr) / (1 - b1 ** max(t, 1)) / den
        tol = update * mag_m * 4 * U + update * np.abs(rm) * 32 * U + 3 * U * np.abs(p)
        got = _np(model.params[i])
        half = 2.0 ** -8 if model.params[i].dtype == torch.bfloat16 else U
        assert np.all(np.abs(got - rp) <= tol + half * np.abs(rp) + 1e-38), i
        if model.copies:
            assert torch.equal(model.copies[i], model.params[i].to(torch.bfloat16))
        if model.bits == 32:
            assert np.all(np.abs(_np(model.plan.exp_avg[i]) - rm) <= 4 * U * mag_m + 1e-45)
            assert np.all(np.abs(_np(model.plan.exp_avg_sq[i]) - rv) <= 6 * U * rv + 1e-45)
            continue
        u = T.random_halves(p.size, i, *words)
        for x, codes, scales, sq in ((rm, model.plan.exp_avg[i], model.plan.exp_avg_scale[i], False),
                                     (np.sqrt(rv), model.plan.exp_avg_sq[i], model.plan.exp_avg_sq_scale[i], True)):
            ref, each = T.block_scales(x)
            # (m's error is relative to its terms, so the scales of m may be
            # off by 4 u of the largest terms of the block)
            edges = list(range(0, p.size, 256))
            slack = 0 if sq else np.maximum.reduceat(mag_m, edges) / 448 * 4 * U
            assert np.all(np.abs(_np(scales) - ref) <= 8 * U * ref + slack + 1e-45)
            want, far = T.stochastic_codes(x, each, u, sq)
            got = _np(codes)
            off = got != want
            # where m's terms cancel, its relative error, and so the border's, grows
            grow = 1.0 if sq else np.maximum(1.0, mag_m / np.maximum(np.abs(rm), 1e-300))
            near = far <= 2.0 * grow
            assert np.all(near[off]), (i, sq, far[off].max())
            grid = np.append(T.e4m3_grid(), 480.0)
            at = np.searchsorted(grid, np.abs(want[off]))
            assert np.all((np.abs(got[off]) >= grid[np.maximum(at - 1, 0)]) & (np.abs(got[off]) <= grid[at + 1]))
            assert off.mean() < 1e-2


SIZES = [
    [1],
    [0, 7, 8, 9, 0],
    [255, 256, 257, 4096],
    [5000, 1, 70001, 2048, 0, 333],
    [300 + i for i in range(40)],
]
TYPES = [("fp32", "fp32", False), ("fp32", "fp32", True), ("fp32", "bf16", True), ("bf16", "bf16", False),
         ("bf16", "fp32", False)]


@pytest.mark.parametrize("bits", [32, 8])
@pytest.mark.parametrize("param,grad,copy", TYPES)
@pytest.mark.parametrize("misalign", [0, 1, 4, 8])
@pytest.mark.parametrize("sizes", SIZES, ids=lambda s: f"{len(s)}x{max(s)}")
def test_step_matches_the_oracle(sizes, param, grad, copy, bits, misalign):
    model = Model(sizes, param, grad, copy, bits, misalign, seed=len(sizes) + misalign)
    words = ((1 << 63) + 99, (5 << 40) + 1)
    for t, b2, scale in ((1, 0.999, None), (1000, 0.95, 0.25)):
        before = model.snapshot()
        vpce.vpce_adamw_step(model.plan, _step(t), lr=1e-2, betas=(0.9, b2), eps=1e-8,
                             grad_scale=None if scale is None else torch.tensor([scale], device="cuda"),
                             rng=_words(*words) if bits == 8 else None)
        _check(model, before, t, 1e-2, 0.9, b2, 1e-8, 1.0 if scale is None else scale, words)


@pytest.mark.parametrize("bits,param,grad", [(32, "fp32", "fp32"), (8, "fp32", "fp32"), (8, "bf16", "bf16"),
                                             (8, "fp32", "bf16")])
def test_tensors_of_many_turns(bits, param, grad):
    # 12 M elements: a CTA takes several turns of 2048 elements
    model = Model([9000001, 6144, 3000000], param, grad, param == "fp32", bits, seed=11)
    words = (17, (1 << 33) + 3)
    before = model.snapshot()
    vpce.vpce_adamw_step(model.plan, _step(7), lr=1e-2, betas=(0.9, 0.95), grad_scale=torch.tensor([0.5], device="cuda"),
                         rng=_words(*words))
    _check(model, before, 7, 1e-2, 0.9, 0.95, 1e-8, 0.5, words)


def test_blocks_of_every_kind_in_vectors_and_element_by_element():
    # blocks of zeros, with a tiny m, a tiny v, of one value, denormal squares:
    # against the oracle, and the same bits off 16 bytes, where another path runs
    n, r = 40 * 256, np.random.default_rng(3)
    g = r.normal(size=(40, 256)) * 1e-2
    g[0:4] = 0
    g[4, 3:] = 0                                  # one element of the block
    g[5:9, ::17] = 1e-9                           # m below e4m3's normal values, v too
    g[9] = 0.25
    g[10:14] *= 1e-17                             # squares below fp32's normal numbers
    g[14, 100] = 1e4                              # all others small beside it
    g[15:17] *= 1e15
    out = []
    for misalign in (0, 1):
        p = _on_gpu(r.normal(size=n) if not misalign else out[0][0], torch.float32, misalign)
        start = p.clone()
        model_g = _on_gpu(g.reshape(-1), torch.float32, misalign)
        codes = [torch.zeros(n + misalign, dtype=torch.float8_e4m3fn, device="cuda")[misalign:] for _ in range(2)]
        plan = vpce.vpce_adamw_plan([p], [model_g], weight_decay=0.1, state_bits=8, exp_avg=[codes[0]],
                                    exp_avg_sq=[codes[1]])
        for t in (1, 2, 3):
            vpce.vpce_adamw_step(plan, _step(t), lr=1e-2, betas=(0.9, 0.95), rng=_words(5, t))
        states = [plan.exp_avg[0].view(torch.uint8), plan.exp_avg_sq[0].view(torch.uint8), plan.exp_avg_scale[0],
                  plan.exp_avg_sq_scale[0], p]
        out.append((start.double().cpu().numpy(), [x.clone() for x in states]))
    assert all(torch.equal(a, b) for a, b in zip(out[0][1], out[1][1]))
    m8, v8, ms, vs, p = out[0][1]
    assert not m8[: 4 * 256].any() and not v8[: 4 * 256].any() and bool((ms[:4] == T.TINY).all())
    keep = (1 - F32(1e-2) * F32(0.1)) ** 3
    assert np.allclose(p[: 4 * 256].double().cpu().numpy(), out[0][0][: 4 * 256] * keep, rtol=1e-6)
    assert bool(p.isfinite().all()) and bool(vs.isfinite().all())


def test_more_than_31_bits_of_elements():
    n = (1 << 31) + 4099
    p = torch.zeros(n, dtype=torch.bfloat16, device="cuda")
    g = torch.ones(n, dtype=torch.bfloat16, device="cuda")
    plan = vpce.vpce_adamw_plan([p], [g], weight_decay=0.0, state_bits=8)
    norm, scale = vpce.vpce_grad_norm(plan, 1.0)
    assert abs(norm.item() / n ** 0.5 - 1) <= 1e-5 and abs(scale.item() * n ** 0.5 - 1) <= 1e-5
    vpce.vpce_adamw_step(plan, _step(1), lr=0.5, rng=_words(1, 1))
    assert bool((p == -0.5).all())
    for codes, scales in ((plan.exp_avg[0], plan.exp_avg_scale[0]), (plan.exp_avg_sq[0], plan.exp_avg_sq_scale[0])):
        assert bool((codes.view(torch.uint8) == 0x7E).all()) and bool((scales == scales[0]).all())
    # the last elements' random words
    g.mul_(torch.linspace(0.1, 1.0, 1024, device="cuda", dtype=torch.bfloat16).repeat(n // 1024 + 1)[:n])
    tail = slice(n - n % 256 - 512, n)
    before = [_np(x) for x in (plan.exp_avg[0][tail], plan.exp_avg_sq[0][tail])]
    sc = [scales[0].double().item() for scales in (plan.exp_avg_scale[0], plan.exp_avg_sq_scale[0])]
    vpce.vpce_adamw_step(plan, _step(2), lr=0.5, rng=_words(9, 10))
    m = 0.9 * before[0] * sc[0] + 0.1 * _np(g[tail])
    v = 0.999 * (before[1] * sc[1]) ** 2 + 0.001 * _np(g[tail]) ** 2
    k = np.arange(tail.start, n)
    words = T.philox4x32_10((k // 8 & 0xFFFFFFFF, 0 * k, 0 * k + 10, 0 * k), (9, 0))
    half = np.stack([w >> np.uint64(16 * i) & np.uint64(0xFFFF) for w in words for i in (0, 1)], axis=1)
    u = half[np.arange(k.size), k % 8].astype(np.int64)
    for x, codes, sq in ((m, plan.exp_avg[0], False), (np.sqrt(v), plan.exp_avg_sq[0], True)):
        _, each = T.block_scales(x)
        want, far = T.stochastic_codes(x, each, u, sq)
        off = _np(codes[tail]) != want
        assert np.all(far[off] <= 2.0) and off.mean() < 1e-2


def test_more_tensors_than_a_launch_holds():
    for bits in (32, 8):
        model = Model([17 + i % 300 for i in range(1000)], bits=bits, seed=3)
        before = model.snapshot()
        vpce.vpce_adamw_step(model.plan, _step(3), lr=1e-2, rng=_words(4, 5))
        _check(model, before, 3, 1e-2, 0.9, 0.999, 1e-8, 1.0, (4, 5))
        norm, scale = vpce.vpce_grad_norm(model.plan, 0.5)
        want, ws = T.grad_norm([b[1] for b in before], 0.5)
        assert abs(norm.item() - want) <= 1e-6 * want and abs(scale.item() - ws) <= 1e-6 * ws


@pytest.mark.parametrize("bits", [32, 8])
def test_states_from_zero_over_some_steps(bits):
    # state dequantized before each step is the next one's input
    model = Model([700, 4097], copy=True, bits=bits, zero=True, seed=9)
    for t in range(1, 6):
        before = model.snapshot()
        if t == 1:
            assert not before[0][2].any() and not before[1][3].any()
        vpce.vpce_adamw_step(model.plan, _step(t), lr=1e-3, rng=_words(1, t))
        _check(model, before, t, 1e-3, 0.9, 0.999, 1e-8, 1.0, (1, t))


def test_rate_and_step_on_the_device_and_odd_hyperparameters():
    lr = torch.tensor([3e-3], device="cuda")
    for t, betas, eps in ((0, (0.9, 0.999), 1e-8), (-5, (0.9, 0.999), 1e-8), (10 ** 12, (0.9, 0.999), 1e-8),
                          (2, (0.0, 0.0), 1e-3), (2, (0.5, 0.0), 1e-3), (1, (0.9, 0.99999), 0.0)):
        model = Model([1000], seed=4)
        before = model.snapshot()
        vpce.vpce_adamw_step(model.plan, _step(t), lr=lr, betas=betas, eps=eps)
        _check(model, before, t, 3e-3, *betas, eps, 1.0)


@pytest.mark.parametrize("bits", [32, 8])
def test_a_grad_scale_of_zero_skips_the_step(bits):
    model = Model([1000, 77], copy=True, bits=bits, seed=5)
    model.grads[0][3] = float("nan")
    norm, scale = vpce.vpce_grad_norm(model.plan, 1.0)
    assert norm.isnan() and scale.item() == 0
    before = model.everything()
    vpce.vpce_adamw_step(model.plan, _step(2), lr=1e-2, grad_scale=scale, rng=_words(1, 1))
    assert all(torch.equal(a, b) for a, b in zip(before, model.everything()))


def test_what_is_not_finite_stays_in_its_place():
    for bits in (32, 8):
        model = Model([1024], bits=bits, seed=6)
        model.grads[0][300] = float("nan")
        model.grads[0][700] = float("inf")
        vpce.vpce_adamw_step(model.plan, _step(2), lr=1e-2, rng=_words(1, 1))
        bad = ~model.params[0].isfinite().cpu().numpy()
        assert list(np.flatnonzero(bad)) == [300, 700]
        m = model.plan.exp_avg[0].float()
        assert bool(m[300].isnan())
        if bits == 8:
            assert bool(model.plan.exp_avg_scale[0][1].isnan()) and bool(model.plan.exp_avg_scale[0][2].isinf())
            assert bool(model.plan.exp_avg_scale[0][[0, 3]].isfinite().all())
        else:
            assert bool(m[700].isinf()) and bool(m[:300].isfinite().all())


def test_small_values_of_eight_bit_states():
    # the rest of a block 1e-7 of its largest element: v takes the least code, m may take 0
    n = 512
    g = torch.full((n,), 1e-6, device="cuda")
    g[0] = 10.0
    p = torch.zeros(n, device="cuda")
    plan = vpce.vpce_adamw_plan([p], [g], weight_decay=0.0, state_bits=8)
    vpce.vpce_adamw_step(plan, _step(1), lr=1.0, rng=_words(1, 2))
    assert torch.allclose(p, torch.full_like(p, -1.0), rtol=2e-2)     # the update itself is not quantized (eps 1e-8)
    codes = plan.exp_avg_sq[0].float()
    assert codes[0] == 448 and bool((codes[1:256] == 2.0 ** -9).all()) and bool((codes[256:] == 448).all())
    g.zero_()
    before = p.clone()
    vpce.vpce_adamw_step(plan, _step(2), lr=1.0, rng=_words(1, 3))
    # m decays against a v that is not 0: no step is longer than lr (0.9 m / 0.19) / sqrt(v)
    assert float((p - before).abs().max()) < 2.0


def test_rounding_keeps_the_expectation():
    # one value between two codes, 2^18 elements: the mean of m and of v after
    # a step from states of 0 within five standard deviations
    n = 1 << 18
    p, g = torch.zeros(n, device="cuda"), torch.zeros(n, device="cuda")
    for sq, a in ((False, 1.05), (True, 1.05), (False, 0.0107), (True, 0.0107)):
        # g sets the value: m = 0.5 g, v = 0.5 g^2 from states of 0, the block's largest element 448
        g.fill_(a * 2 if not sq else a * 2 ** 0.5)
        g[::256] = 448.0 * 2 if not sq else 448.0 * 2 ** 0.5
        plan = vpce.vpce_adamw_plan([p], [g], state_bits=8)
        vpce.vpce_adamw_step(plan, _step(1), lr=0.0, betas=(0.5, 0.5), rng=_words(11, 3 + sq))
        q = (plan.exp_avg_sq if sq else plan.exp_avg)[0].float().double().view(-1, 256)[:, 1:]
        lo, hi = q.min().item(), q.max().item()
        assert lo < a < hi
        x = q * q if sq else q
        dev = x.std().item() / q.numel() ** 0.5
        assert abs(x.mean().item() - (a * a if sq else a)) <= 5 * dev + 1e-5 * a


@pytest.mark.parametrize("grad", ["fp32", "bf16"])
@pytest.mark.parametrize("sizes", SIZES + [[1 << 20, 123457]], ids=lambda s: f"{len(s)}x{max(s)}")
@pytest.mark.parametrize("misalign", [0, 1])
def test_grad_norm(sizes, grad, misalign):
    # squares (u), eight sums of at most 4 n / (grid 4096) + 12 terms each: all
    # positive, so within (terms + 12) u; n / 2^16 + 64 covers every size here
    model = Model(sizes, grad=grad, misalign=misalign, seed=1)
    want, _ = T.grad_norm([_np(g) for g in model.grads])
    tol = (sum(sizes) / 65536 + 64) * U
    for src in (model.plan, model.grads):
        norm, scale = vpce.vpce_grad_norm(src)
        assert abs(norm.item() - want) <= tol * want and scale.item() == 1.0
        for most in (want * 2, want / 3):
            norm, scale = vpce.vpce_grad_norm(src, most)
            ref = min(1.0, F32(most) / want)
            assert abs(scale.item() - ref) <= 2 * tol * ref
    assert torch.equal(vpce.vpce_grad_norm(model.plan)[0], vpce.vpce_grad_norm(model.grads)[0])


def test_grad_norm_of_zeros_and_of_what_is_not_finite():
    g = [torch.zeros(1000, device="cuda"), torch.zeros(5, device="cuda")]
    ws = torch.full((vpce.load_library().vpce_grad_norm_workspace_bytes(2),), 0xFF, dtype=torch.uint8, device="cuda")
    out = [torch.full((1,), 7.0, device="cuda") for _ in range(2)]
    vpce.vpce_grad_norm(g, 1.0, norm_out=out[0], scale_out=out[1], workspace=ws)
    assert out[0].item() == 0 and out[1].item() == 1
    for bad in (float("inf"), float("nan"), 1e30):
        g[1][2] = bad
        norm, scale = vpce.vpce_grad_norm(g, 1.0)
        assert not norm.isfinite() and scale.item() == 0
    assert vpce.vpce_grad_norm([torch.zeros(0, device="cuda")])[0].item() == 0


def test_tensors_between_others_are_left_alone():
    for bits in (32, 8):
        flat = torch.zeros(4096, device="cuda")
        grads = torch.ones(4096, device="cuda")
        spans = [(3, 100), (200, 456), (1000, 1255)]
        params, gs = [flat[a:b] for a, b in spans], [grads[a:b] for a, b in spans]
        plan = vpce.vpce_adamw_plan(params, gs, state_bits=bits)
        vpce.vpce_adamw_step(plan, _step(1), lr=1.0, rng=_words(0, 0))
        inside = torch.zeros(4096, dtype=torch.bool, device="cuda")
        for a, b in spans:
            inside[a:b] = True
        assert bool((flat[inside] != 0).all()) and not flat[~inside].any()


def test_same_bits_again_on_another_stream_and_in_a_graph():
    for bits in (32, 8):
        def fresh():
            return Model([5000, 300, 70000], copy=True, bits=bits, seed=7)

        a, b, c = fresh(), fresh(), fresh()
        words = [_words(3, k) for k in range(3)]
        for k in range(3):
            _, scale = vpce.vpce_grad_norm(a.plan, 0.5)
            vpce.vpce_adamw_step(a.plan, _step(k + 1), lr=1e-2 * (k + 1), grad_scale=scale, rng=words[k])
        side = torch.cuda.Stream()
        side.wait_stream(torch.cuda.current_stream())
        for k in range(3):
            with torch.cuda.stream(side):
                t = _step(k + 1)
            _, scale = vpce.vpce_grad_norm(b.plan, 0.5, stream=side)
            vpce.vpce_adamw_step(b.plan, t, lr=1e-2 * (k + 1), grad_scale=scale, rng=words[k], stream=side)
        side.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.everything(), b.everything()))
        # captured: step, rate and random words change between the replays
        t, lr, rng = _step(1), torch.tensor([1e-2], device="cuda"), _words(3, 0)
        torch.cuda.synchronize()
        graph = torch.cuda.CUDAGraph()
        with torch.cuda.graph(graph):
            _, scale = vpce.vpce_grad_norm(c.plan, 0.5)
            vpce.vpce_adamw_step(c.plan, t, lr=lr, grad_scale=scale, rng=rng)
            t += 1
        for k in range(3):
            lr.fill_(1e-2 * (k + 1))
            rng[1] = k
            graph.replay()
        torch.cuda.synchronize()
        assert all(torch.equal(x, y) for x, y in zip(a.everything(), c.everything()))


def test_two_plans_at_once_on_two_streams():
    a, b, a2, b2 = (Model([100000, 999], bits=8, seed=k) for k in (1, 2, 1, 2))
    for m in (a2, b2):
        vpce.vpce_adamw_step(m.plan, _step(1), lr=1e-2, grad_scale=vpce.vpce_grad_norm(m.plan, 0.5)[1],
                             rng=_words(1, 1))
    torch.cuda.synchronize()
    s1, s2, w, t = torch.cuda.Stream(), torch.cuda.Stream(), _words(1, 1), _step(1)
    torch.cuda.synchronize()
    for m, s in ((a, s1), (b, s2)):
        vpce.vpce_adamw_step(m.plan, t, lr=1e-2, grad_scale=vpce.vpce_grad_norm(m.plan, 0.5, stream=s)[1], rng=w,
                             stream=s)
    torch.cuda.synchronize()
    for m, r in ((a, a2), (b, b2)):
        assert all(torch.equal(x, y) for x, y in zip(m.everything(), r.everything()))


def test_moved_memory_is_refused():
    model = Model([100], seed=1)
    model.params[0].data = torch.zeros(100, device="cuda")
    with pytest.raises(ValueError, match="moved"):
        vpce.vpce_adamw_step(model.plan, _step(1), lr=1e-2)
