"""GPU parity of the token scores (vpce_logprob_forward / _backward) with the
fp64 oracle.

Tolerances (rows of at most 5000 columns; eps = 2^-24):
* an exponential's argument u = (z - max)/T carries 2 eps |u| and the
  exponential itself at most 4 eps, and |u| e^u <= 1/e, so S is off by less
  than 8 eps relatively, plus eps per addition: a lane adds at most 5000 / 32
  terms in sequence, the merges a few more, under 200 in all.  ln S and logp
  are then within 210 eps = 1.3e-5 absolutely (plus 4 eps of their value):
  2e-5 max(1, |value|).
* entropy = ln S - U / S: U's terms carry the same relative errors weighted by
  |u|, so U / S is within 1.3e-5 * (2 + ln V) (U / S <= 1 + ln V), in all
  2e-5 (2 + ln V).
* alternatives are exact.
* gradient: p is within 3e-5 relatively (its exponent is logp's error), the
  bracket within 2e-5 of its terms; so |error| T <= p (5e-5 (|w| + |g_H| (|ln p|
  + H)) + 5e-5 |g_H| (2 + ln V)) + 4 eps sum |g|, and one rounding to the
  output type (2^-8 of the value for bf16, 2^-23 for fp32).
"""
import ctypes

import numpy as np
import pytest
import torch

from oracle import scores_oracle as S
from oracle import vpce_oracle as O
from vocab_sharded_lm_gb300 import vpce

from _parity import from_device, to_device

pytestmark = pytest.mark.gpu
LOW = {"bf16": float(torch.finfo(torch.bfloat16).min), "fp32": float(torch.finfo(torch.float32).min)}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


def _logits(seed, s, V, dtype, sigma=3.0):
    """Random logits as stored ([s, V] fp64 of exactly representable values)."""
    x = torch.from_numpy(np.random.default_rng(seed).normal(0, sigma, (s, V)))
    return x.to(torch.bfloat16 if dtype == "bf16" else torch.float32).double().numpy()


def _place(z, vs, dtype, layout, misalign=0):
    """The shards on the GPU: dense, padded rows, or column blocks."""
    tt = torch.from_numpy(z).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    parts = [tt[:, vs[i]:vs[i + 1]] for i in range(len(vs) - 1)]
    if layout == "dense":
        out = []
        for q in parts:
            flat = torch.empty(q.numel() + misalign, dtype=q.dtype, device="cuda")
            v = flat[misalign:].view(q.shape)
            v.copy_(q)
            out.append(v)
        return out
    if layout == "columns":
        full = tt.cuda()
        return list(full.split([q.shape[1] for q in parts], dim=1))
    ld = max(q.shape[1] for q in parts) + 5
    out = []
    for q in parts:
        b = torch.full((q.shape[0], ld), float("nan"), dtype=q.dtype, device="cuda")
        b[:, :q.shape[1]] = q.cuda()
        out.append(b[:, :q.shape[1]])
    return out


def _check_forward(r, ref, V):
    """r: LogprobResult, ref: the oracle's."""
    def close(got, want, tol):
        got = got.cpu().numpy().astype(np.float64)
        assert np.array_equal(np.isnan(got), np.isnan(want))
        assert np.array_equal(got[np.isinf(want)], want[np.isinf(want)])
        f = np.isfinite(want)
        assert np.all(np.isfinite(got[f]))
        err = np.abs(got[f] - want[f])
        bound = np.broadcast_to(tol(want), want.shape)[f]
        assert np.all(err <= bound), float((err / bound).max())

    if r.logp is not None:
        close(r.logp, ref["logp"], lambda w: 2e-5 * np.maximum(1, np.abs(w)))
    close(r.entropy, ref["entropy"], lambda w: np.full(w.shape, 2e-5 * (2 + np.log(V))))
    close(r.stats, ref["stats"], lambda w: np.full(w.shape, 2e-5 * (2 + np.log(V))))
    st = r.stats.cpu().numpy().astype(np.float64)
    assert np.array_equal(st[:, 0], ref["stats"][:, 0], equal_nan=True)   # the largest logit is a copy
    if r.top_ids is not None:
        np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ref["top_ids"])
        close(r.top_logp, ref["top_logp"], lambda w: 2e-5 * np.maximum(1, np.abs(w)))


CASES = [
    # s, V, vs, dtype, layout, top, T
    (1, 1, [0, 1], "bf16", "dense", 1, 1.0),
    (1, 31, [0, 31], "fp32", "dense", 31, 1.0),
    (3, 33, [0, 1, 2, 33], "bf16", "dense", 32, 0.5),
    (5, 129, [0, 64, 129], "fp32", "columns", 5, 1.0),
    (64, 1000, [0, 500, 1000], "fp32", "dense", 8, 1.0),
    (37, 2049, [0, 7, 1024, 2049], "bf16", "columns", 20, 1.7),
    (9, 4097, [0, 4097], "bf16", "padded", 32, 1.0),
    (200, 4999, [0, 1, 2, 3, 1000, 2500, 4000, 4998, 4999], "bf16", "columns", 5, 1.0),
    (31, 4999, [0, 2500, 4999], "fp32", "padded", 20, 0.3),
    (700, 1537, [0, 800, 1537], "bf16", "dense", 3, 1.0),
    (30, 64 * 31, [31 * i for i in range(65)], "fp32", "dense", 32, 1.0),   # as many shards as there can be
    (30, 64 * 31, [31 * i for i in range(65)], "bf16", "columns", 8, 1.0),
]


@pytest.mark.parametrize("s,V,vs,dtype,layout,top,T", CASES)
def test_forward_matches_the_oracle(s, V, vs, dtype, layout, top, T):
    z = _logits(s * 7 + V, s, V, dtype)
    rng = np.random.default_rng(V)
    y = rng.integers(0, V, s)
    if s > 4:
        y[1], y[s // 2] = -100, -100
        y[2], y[3] = 0, V - 1
    shards = _place(z, vs, dtype, layout)
    r = vpce.vpce_logprob_forward(shards, torch.from_numpy(y).cuda(), vs, top=top, temperature=T)
    _check_forward(r, S.token_scores(z, y, top, T), V)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("misalign", [1, 3, 5])
def test_forward_off_16_bytes(dtype, misalign):
    V, vs = 777, [0, 5, 400, 777]
    z = _logits(misalign, 12, V, dtype)
    y = np.arange(12) * 60
    r = vpce.vpce_logprob_forward(_place(z, vs, dtype, "dense", misalign), torch.from_numpy(y).cuda(), vs, top=6)
    _check_forward(r, S.token_scores(z, y, 6), V)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("s", [11, 400])
def test_forward_masks_infinities_and_ties(dtype, s):
    V, vs, top = 3001, [0, 1500, 3001], 32
    z = _logits(5, s, V, dtype)
    rng = np.random.default_rng(6)
    z[0] = -np.inf                                   # nothing left
    z[1] = -np.inf
    z[1, 17] = 2.0                                   # one column left
    z[2] = LOW[dtype]                                # a mask of the lowest value everywhere: uniform
    z[3, rng.random(V) < 0.99] = LOW[dtype]
    z[4, 40] = np.inf
    z[5, [7, 2000]] = np.nan
    z[6] = 1.25                                      # all equal
    z[7] = np.round(z[7] / 4) * 4                    # many ties at the boundary
    z[8, rng.random(V) < 0.999] = -np.inf
    z[9, :50] = 30.0
    z[10, ::3], z[10, 1::3], z[10, 2::3] = 0.0, -0.0, -1.0   # signed zeros are equal
    y = rng.integers(0, V, s)
    y[1], y[8] = 17, int(np.nonzero(np.isfinite(z[8]))[0][0])
    r = vpce.vpce_logprob_forward(_place(z, vs, dtype, "dense"), torch.from_numpy(y).cuda(), vs, top=top)
    _check_forward(r, S.token_scores(z, y, top), V)


def test_forward_sorted_rows_and_large_logits():
    # ascending rows put every alternative at the end, descending ones at the start
    V, vs = 4500, [0, 1111, 4500]
    z = np.sort(_logits(8, 6, V, "fp32", 100.0), axis=1)
    z[3:] = z[3:, ::-1]
    z[1] += 3e4
    z[4] *= 1e30
    z = z.astype(np.float32).astype(np.float64)
    y = np.array([V - 1, 0, 5, 0, 1, 2])
    r = vpce.vpce_logprob_forward(_place(z, vs, "fp32", "dense"), torch.from_numpy(y).cuda(), vs, top=32)
    ref = S.token_scores(z, y, 32)
    np.testing.assert_array_equal(r.top_ids.cpu().numpy(), ref["top_ids"])
    got, want = r.logp.cpu().numpy(), ref["logp"]
    assert np.all(np.abs(got - want) <= 2e-5 * np.maximum(1, np.abs(want)))


def test_forward_outputs_are_optional_and_without_targets():
    V, vs = 900, [0, 900]
    z = _logits(9, 20, V, "bf16")
    sh = _place(z, vs, "bf16", "dense")
    ref = S.token_scores(z, None, 4)
    r = vpce.vpce_logprob_forward(sh, None, vs, top=4)
    assert r.logp is None
    _check_forward(r, ref, V)
    r0 = vpce.vpce_logprob_forward(sh, None, vs)
    assert r0.top_ids is None and torch.equal(r0.entropy, r.entropy)
    # each output alone, through the C entry
    lib = vpce.load_library()
    ptrs, starts = vpce._ptr_array([sh[0].data_ptr()]), vpce._i64_array(vs)
    ent = torch.full((20,), -1.0, device="cuda")
    ids = torch.full((20, 2), -7, dtype=torch.int64, device="cuda")
    st = torch.cuda.current_stream().cuda_stream
    assert lib.vpce_logprob_forward(ptrs, 1, 1, 20, starts, 0, None, -100, 1.0, 0, None, ent.data_ptr(), None, None,
                                    None, None, st) == 0
    assert lib.vpce_logprob_forward(ptrs, 1, 1, 20, starts, 0, None, -100, 1.0, 2, None, None, ids.data_ptr(), None,
                                    None, None, st) == 0
    assert torch.equal(ent, r.entropy) and torch.equal(ids, r.top_ids[:, :2])


def test_bad_targets_raise_the_flag():
    V, vs = 300, [0, 100, 300]
    z = _logits(10, 6, V, "fp32")
    y = np.array([0, V, -1, -100, 5, 2 ** 40])
    flag = torch.full((1,), 77, dtype=torch.int32, device="cuda")
    r = vpce.vpce_logprob_forward(_place(z, vs, "fp32", "dense"), torch.from_numpy(y).cuda(), vs, top=2, flag=flag)
    ref = S.token_scores(z, y, 2)
    _check_forward(r, ref, V)
    assert flag.item() == vpce.VPCE_FLAG_BAD_TARGET and ref["bad"]
    vpce.vpce_logprob_forward(_place(z, vs, "fp32", "dense"), torch.from_numpy(y % V).cuda(), vs, flag=flag)
    assert flag.item() == 0


@pytest.mark.parametrize("dtype,V", [("bf16", 40), ("bf16", 5000), ("fp32", 257)])
def test_many_short_rows(dtype, V):
    # every CTA works through some hundred rows of one to three pieces
    s, top = 40000, 4
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V)
    z = torch.randn(s, V, device="cuda", generator=gen).mul_(3).to(torch.bfloat16 if dtype == "bf16" else torch.float32)
    y = torch.randint(0, V, (s,), device="cuda", generator=gen)
    y[::5] = -100
    r = vpce.vpce_logprob_forward([z], y, top=top)
    lp = torch.log_softmax(z.double(), 1)
    live = y != -100
    want = lp.gather(1, y.clamp(min=0)[:, None])[:, 0]
    assert float((r.logp.double() - want)[live].abs().max()) <= 2e-5 * float(want.abs().max())
    ent = -(lp.exp() * lp).sum(1)
    assert float((r.entropy.double() - ent)[live].abs().max()) <= 2e-5 * (2 + np.log(V))
    order = torch.argsort(z.double(), dim=1, descending=True, stable=True)[:, :top]
    assert torch.equal(r.top_ids[live], order[live])
    assert not r.logp[~live].any() and bool((r.top_ids[~live] == -1).all())


def test_empty_batch():
    z = torch.empty(0, 64, dtype=torch.bfloat16, device="cuda")
    r = vpce.vpce_logprob_forward([z], torch.empty(0, dtype=torch.int64, device="cuda"), top=3)
    assert r.logp.shape == (0,) and r.top_ids.shape == (0, 3)
    g = vpce.vpce_logprob_backward([z], torch.empty(0, dtype=torch.int64, device="cuda"), r.stats,
                                   grad_entropy=torch.empty(0, device="cuda"))
    assert g[0].shape == (0, 64)


def _stats_of(z, y, T):
    return torch.from_numpy(S.token_scores(z, y, 0, T)["stats"]).float().cuda()


def _check_backward(z, y, vs, dtype, layout, T, gl, ge, ids, gt, in_place, misalign=0):
    shards = _place(z, vs, dtype, layout, misalign)
    yd = torch.from_numpy(y).cuda() if y is not None else None
    fwd = vpce.vpce_logprob_forward(shards, yd, vs, temperature=T)
    f32 = lambda a: None if a is None else torch.from_numpy(a.astype(np.float32)).cuda()  # noqa: E731
    keep = [sh.clone() for sh in shards]
    idd = None if ids is None else torch.from_numpy(ids).cuda()
    out = vpce.vpce_logprob_backward(shards, yd, fwd.stats, vs, temperature=T, grad_logp=f32(gl),
                                     grad_entropy=f32(ge), top_ids=idd, grad_top_logp=f32(gt),
                                     grad_shards=shards if in_place else None)
    if not in_place:
        assert all(torch.equal(a.view(torch.int16 if dtype == "bf16" else torch.int32),
                               b.view(torch.int16 if dtype == "bf16" else torch.int32))
                   for a, b in zip([sh.contiguous() for sh in shards], [k.contiguous() for k in keep]))
    got = np.concatenate([o.double().cpu().numpy() for o in out], axis=1)
    r32 = lambda a: None if a is None else a.astype(np.float32).astype(np.float64)  # noqa: E731
    ref = S.token_scores_backward(z, y, r32(gl), r32(ge), ids, r32(gt), T)
    assert np.array_equal(np.isnan(got), np.isnan(ref))
    s, V = z.shape
    with np.errstate(all="ignore"):
        m = z.max(1, keepdims=True)
        lp = (z - m) / T - np.log(np.exp((z - m) / T).sum(1, keepdims=True))
        p = np.exp(lp)
        H = -np.where(p > 0, p * lp, 0).sum(1, keepdims=True)
        one = lambda a: np.zeros((s, 1)) if a is None else np.abs(r32(a))[:, None]  # noqa: E731
        tops = np.zeros((s, 1)) if gt is None else np.abs(r32(gt)).sum(1, keepdims=True)
        w, gh = one(gl) + tops, one(ge)
        bound = (np.where(p > 0, p * (5e-5 * (w + gh * (np.abs(lp) + H)) + 5e-5 * gh * (2 + np.log(V))), 0)
                 + 2.0 ** -22 * w) / T + np.abs(ref) * (2.0 ** -8 if dtype == "bf16" else 2.0 ** -23) + 1e-38
        f = ~np.isnan(ref)
        assert np.all(np.abs(got - ref)[f] <= bound[f]), float(np.nanmax((np.abs(got - ref) / bound)[f]))
    return out


BWD = [
    (1, 1, [0, 1], "fp32", "dense", 1.0, 0),
    (1, 40, [0, 13, 40], "bf16", "dense", 1.0, 5),
    (7, 513, [0, 3, 256, 513], "bf16", "columns", 0.7, 32),
    (33, 1000, [0, 500, 1000], "fp32", "dense", 1.0, 8),
    (20, 4999, [0, 1, 2500, 4999], "fp32", "columns", 1.6, 3),
    (40, 2050, [0, 1024, 2050], "bf16", "padded", 1.0, 0),
    (3, 4800, [0, 4800], "bf16", "dense", 1.0, 20),
]


@pytest.mark.parametrize("in_place", [False, True])
@pytest.mark.parametrize("s,V,vs,dtype,layout,T,top", BWD)
def test_backward_matches_the_oracle(s, V, vs, dtype, layout, T, top, in_place):
    z = _logits(s + V, s, V, dtype)
    r = np.random.default_rng(s)
    y = r.integers(0, V, s)
    if s > 4:
        y[1], y[3], y[4] = -100, V - 1, 0
    ids = gt = None
    if top:
        ids = S.token_scores(z, y, top)["top_ids"]
        gt = r.normal(size=(s, top))
        if s > 4:
            ids[0, 0] = y[0]                     # the target among the alternatives
            ids[2, -1] = -1                      # skipped
            ids[4, 1] = ids[4, 0]                # counted twice
    _check_backward(z, y, vs, dtype, layout, T, r.normal(size=s), r.normal(size=s), ids, gt, in_place)


@pytest.mark.parametrize("which", ["logp", "entropy", "top"])
def test_backward_of_one_output(which):
    V, vs, s = 700, [0, 350, 700], 9
    z = _logits(3, s, V, "fp32")
    r = np.random.default_rng(4)
    y = r.integers(0, V, s) if which == "logp" else None
    ids = S.token_scores(z, None, 4)["top_ids"] if which == "top" else None
    _check_backward(z, y, vs, "fp32", "dense", 1.0, r.normal(size=s) if which == "logp" else None,
                    r.normal(size=s) if which == "entropy" else None, ids,
                    r.normal(size=(s, 4)) if which == "top" else None, False)


@pytest.mark.parametrize("dtype", ["bf16", "fp32"])
@pytest.mark.parametrize("misalign", [0, 1, 5])
def test_backward_masks_and_bad_rows(dtype, misalign):
    V, vs, s = 1111, [0, 300, 1111], 9
    z = _logits(12, s, V, dtype)
    r = np.random.default_rng(13)
    z[0] = -np.inf
    z[1] = -np.inf
    z[1, 9] = 1.0
    z[2, r.random(V) < 0.9] = -np.inf
    z[3, 5] = np.nan
    z[4] = LOW[dtype]
    z[5, r.random(V) < 0.5] = LOW[dtype]
    z[6, 8] = np.inf
    y = r.integers(0, V, s)
    y[1], y[7], y[8] = 9, -100, V + 3             # an ignored row, a target out of range
    y[2] = int(np.nonzero(np.isfinite(z[2]))[0][0])
    _check_backward(z, y, vs, dtype, "dense", 1.0, r.normal(size=s), r.normal(size=s), None, None, False, misalign)


def test_backward_matches_differences_of_the_forward():
    # fp32 central differences of the library's own forward: with a step of
    # 0.25 the third-order term is below 0.25^2 / 6 < 0.011 |g| sum and the
    # forward's error adds 2e-5 (2 + ln V) 2 / 0.5 < 1e-3
    V, vs, s = 60, [0, 25, 60], 4
    z = _logits(20, s, V, "fp32", 1.0)
    y = np.array([3, 59, 24, 25])
    yd = torch.from_numpy(y).cuda()
    gl, ge = np.array([1.0, -0.5, 0.25, 2.0]), np.array([0.5, 1.0, -1.0, 0.25])

    def value(zz):
        r = vpce.vpce_logprob_forward(_place(zz, vs, "fp32", "dense"), yd, vs)
        return (r.logp.double().cpu().numpy() * gl + r.entropy.double().cpu().numpy() * ge)

    sh = _place(z, vs, "fp32", "dense")
    st = vpce.vpce_logprob_forward(sh, yd, vs).stats
    d = vpce.vpce_logprob_backward(sh, yd, st, vs, grad_logp=torch.from_numpy(gl).float().cuda(),
                                   grad_entropy=torch.from_numpy(ge).float().cuda())
    d = torch.cat(d, 1).double().cpu().numpy()
    for k in (0, 3, 24, 25, 59):
        e = np.zeros_like(z)
        e[:, k] = 0.25
        num = (value(z + e) - value(z - e)) / 0.5
        assert np.all(np.abs(num - d[:, k]) <= 0.02 * (np.abs(gl) + np.abs(ge)) + 1e-3)


def test_results_repeat_and_hold_on_another_stream():
    V, vs, s = 3000, [0, 1500, 3000], 500
    z = _logits(30, s, V, "bf16")
    y = torch.from_numpy(np.random.default_rng(1).integers(0, V, s)).cuda()
    sh = _place(z, vs, "bf16", "dense")
    a = vpce.vpce_logprob_forward(sh, y, vs, top=20)
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        b = vpce.vpce_logprob_forward(sh, y, vs, top=20)
    c = vpce.vpce_logprob_forward(sh, y, vs, top=20, stream=side)
    side.synchronize()
    for o in (b, c):
        assert all(torch.equal(p, q) for p, q in zip(a, o))
    g = torch.linspace(-1, 1, s, device="cuda")
    d1 = vpce.vpce_logprob_backward(sh, y, a.stats, vs, grad_logp=g, grad_entropy=g)
    d2 = vpce.vpce_logprob_backward(sh, y, a.stats, vs, grad_logp=g, grad_entropy=g)
    assert all(torch.equal(p, q) for p, q in zip(d1, d2))


def test_graph_replay_follows_the_inputs():
    V, vs, s = 2000, [0, 900, 2000], 64
    z1, z2 = _logits(40, s, V, "bf16"), _logits(41, s, V, "bf16")
    sh, other = _place(z1, vs, "bf16", "dense"), _place(z2, vs, "bf16", "dense")
    y = torch.from_numpy(np.random.default_rng(2).integers(0, V, s)).cuda()
    g = torch.linspace(-1, 1, s, device="cuda")
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    grads = [torch.empty_like(q) for q in sh]
    out = vpce.vpce_logprob_forward(sh, y, vs, top=5, flag=flag)
    bufs = dict(logp_out=out.logp, entropy_out=out.entropy, top_ids_out=out.top_ids, top_logp_out=out.top_logp,
                stats_out=out.stats)

    def step():
        r = vpce.vpce_logprob_forward(sh, y, vs, top=5, flag=flag, **bufs)
        vpce.vpce_logprob_backward(sh, y, r.stats, vs, grad_logp=g, grad_entropy=g, grad_shards=grads)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for a, b in zip(sh, other):
        a.copy_(b)
    graph.replay()
    torch.cuda.synchronize()
    want = vpce.vpce_logprob_forward(other, y, vs, top=5)
    wg = vpce.vpce_logprob_backward(other, y, want.stats, vs, grad_logp=g, grad_entropy=g)
    assert all(torch.equal(p, q) for p, q in zip(out, want)) and all(torch.equal(p, q) for p, q in zip(grads, wg))


def test_offsets_past_32_bits():
    # one shard of 70000 x 65536 bf16: 9.2 GB, the last rows start past 2^32 elements
    s, V = 70000, 65536
    z = torch.zeros(s, V, dtype=torch.bfloat16, device="cuda")
    rows = [0, 32767, 65535, 65536, 69999]
    for i, r in enumerate(rows):
        z[r, 100 * i + 7] = 8.0
    y = torch.full((s,), -100, dtype=torch.int64, device="cuda")
    y[rows] = torch.tensor([100 * i + 7 for i in range(len(rows))], device="cuda")
    r = vpce.vpce_logprob_forward([z], y, top=2)
    lp = 8.0 - np.log(np.exp(8.0) + V - 1)
    assert np.all(np.abs(r.logp[rows].cpu().numpy() - lp) <= 2e-5 * abs(lp))
    assert r.top_ids[rows].tolist() == [[100 * i + 7, 0] for i in range(len(rows))]
    vpce.vpce_logprob_backward([z], y, r.stats, grad_logp=torch.ones(s, device="cuda"), grad_shards=[z])
    assert int((z != 0).any(1).sum()) == len(rows)
    got = z[rows, [100 * i + 7 for i in range(len(rows))]].float().cpu().numpy()
    want = 1 - np.exp(lp)
    assert np.all(np.abs(got - want) <= want * 2.0 ** -8 + 5e-5)


@pytest.mark.parametrize("s,V,t,dtype,top", [(64, 128256, 8, "bf16", 20), (700, 152064, 8, "fp32", 32),
                                             (1, 256000, 16, "bf16", 5), (3, 1 << 20, 1, "bf16", 32)])
def test_long_rows_against_fp64_on_the_device(s, V, t, dtype, top):
    gen = torch.Generator(device="cuda")
    gen.manual_seed(V + s)
    dt = torch.bfloat16 if dtype == "bf16" else torch.float32
    z = torch.empty(s, V, dtype=dt, device="cuda").normal_(0, 3, generator=gen)
    vs = [i * (V // t) for i in range(t)] + [V]
    shards = [z[:, vs[i]:vs[i + 1]].contiguous() for i in range(t)]
    y = torch.randint(0, V, (s,), device="cuda", generator=gen)
    r = vpce.vpce_logprob_forward(shards, y, vs, top=top)
    lp = torch.log_softmax(z.double(), 1)
    # rows this long are split over 8 warps of partials: under 1100 sequential
    # additions a lane, 1110 eps = 6.7e-5
    assert float((r.logp.double() - lp.gather(1, y[:, None])[:, 0]).abs().max()) <= 8e-5
    ent = -(lp.exp() * lp).sum(1)
    assert float((r.entropy.double() - ent).abs().max()) <= 8e-5 * (2 + np.log(V))
    zf = z.double()
    for row in range(0, s, max(1, s // 16)):
        order = np.lexsort((np.arange(V), -zf[row].cpu().numpy()))[:top]
        assert r.top_ids[row].tolist() == order.tolist()
