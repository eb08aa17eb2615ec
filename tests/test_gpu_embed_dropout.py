"""GPU parity of the scaled embedding with dropout (vpce_embedding_dropout_*)
with the fp64 oracle.

* Forward: the factor is rounded to fp32 and the product once more (2^-23 of
  the value in all), then to the output type: 2^-22 |value| for fp32,
  2^-8 |value| for bf16.  Dropped, padded and out-of-range elements are 0
  exactly.
* Backward: a table element is an fp32 sum of count products: within
  (count + 3) 2^-24 of the sum of the terms' magnitudes (any order)."""
import numpy as np
import pytest
import torch

from oracle import scores_oracle as S
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


def _table(seed, V, h, dtype):
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=(V, h))).to(DT[dtype])
    return x, x.double().numpy()


def _rng(seed, offset):
    wrap = lambda v: v - (1 << 64) if v >= 1 << 63 else v  # noqa: E731
    return torch.tensor([wrap(seed), wrap(offset)], dtype=torch.int64, device="cuda")


def _shards(x, vs, pad=0, misalign=0):
    """The table's shards; pad: extra columns a row, misalign: elements past 16 bytes."""
    out = []
    for i in range(len(vs) - 1):
        q = x[vs[i]:vs[i + 1]]
        ld = q.shape[1] + pad
        flat = torch.full((q.shape[0] * ld + misalign,), float("nan"), dtype=x.dtype, device="cuda")
        v = flat[misalign:].view(q.shape[0], ld)[:, :q.shape[1]]
        v.copy_(q)
        out.append(v)
    return out


FWD = [
    # V, vs, h, s, table, out, p, pad, misalign
    (10, [0, 10], 1, 1, "fp32", "fp32", 0.0, 0, 0),
    (10, [0, 3, 10], 7, 40, "bf16", "bf16", 0.5, 0, 0),
    (1000, [0, 1, 2, 500, 1000], 64, 300, "bf16", "bf16", 0.1, 0, 0),
    (1000, [0, 400, 1000], 264, 111, "bf16", "fp32", 0.25, 8, 0),
    (300, [0, 300], 515, 70, "fp32", "bf16", 0.3, 1, 0),
    (300, [0, 100, 300], 1032, 33, "fp32", "fp32", 0.9, 0, 1),
    (300, [0, 100, 300], 136, 65, "bf16", "bf16", 0.2, 0, 3),
    (64, [0, 64], 4096, 20, "fp32", "bf16", 0.0, 0, 0),
]


@pytest.mark.parametrize("V,vs,h,s,table,out,p,pad,misalign", FWD)
def test_forward_matches_the_oracle(V, vs, h, s, table, out, p, pad, misalign):
    x, xd = _table(V + h, V, h, table)
    r = np.random.default_rng(s)
    ids = r.integers(0, V, s)
    padding = V // 2
    if s > 8:
        ids[[0, 1, 2, 3, 4]] = [0, V - 1, -1, V, padding]
    seed, offset = (1 << 63) + 12345, (3 << 40) + 9
    scale = 22.627417
    flag = torch.full((1,), 5, dtype=torch.int32, device="cuda")
    buf = torch.full((s, h + pad), -3.0, dtype=DT[out], device="cuda")
    got = vpce.vpce_embedding_dropout_forward(_shards(x, vs, pad, misalign), torch.from_numpy(ids).cuda(), vs,
                                              scale=scale, p=p, rng=_rng(seed, offset) if p else None,
                                              padding_id=padding, out=buf[:, :h], flag=flag)
    ref, bad = S.embedding_dropout_forward(xd, ids, float(np.float32(scale)), p, seed, offset, padding)
    g = got.double().cpu().numpy()
    assert np.array_equal(g == 0, ref == 0)
    assert np.all(np.abs(g - ref) <= np.abs(ref) * (2.0 ** -8 if out == "bf16" else 2.0 ** -22))
    assert bool(flag.item() & vpce.VPCE_FLAG_BAD_TARGET) == bad
    if pad:
        assert bool((buf[:, h:] == -3.0).all())


def test_forward_default_output_type_scale_one_is_a_copy():
    x, _ = _table(3, 50, 48, "bf16")
    ids = torch.arange(49, -1, -1, device="cuda")
    out = vpce.vpce_embedding_dropout_forward([x.cuda()], ids)
    assert out.dtype == torch.bfloat16 and torch.equal(out, x.cuda().flip(0))
    assert vpce.vpce_embedding_dropout_forward([x.cuda()], ids, out_dtype=torch.float32).dtype == torch.float32


def test_padding_outside_the_vocabulary_and_dropped_infinities():
    x, xd = _table(4, 20, 32, "fp32")
    x[5], xd[5] = float("inf"), np.inf
    ids = np.array([-7, 5, 3, -7])
    flag = torch.zeros(1, dtype=torch.int32, device="cuda")
    out = vpce.vpce_embedding_dropout_forward([x.cuda()], torch.from_numpy(ids).cuda(), p=0.5, rng=_rng(1, 2),
                                              padding_id=-7, flag=flag)
    keep = S.keep_mask(1, 2, 4, 32, 0.5)
    assert flag.item() == 0 and not out[0].any() and not out[3].any()
    assert np.array_equal(np.isinf(out[1].cpu().numpy()), keep[1]) and bool((out[1][~torch.from_numpy(keep[1])] == 0).all())


BWD = [
    # V, vs, h, s, grad, p, kind, pad, misalign
    (1, [0, 1], 1, 1, "fp32", 0.0, "uniform", 0, 0),
    (10, [0, 3, 10], 7, 40, "bf16", 0.5, "uniform", 0, 0),
    (2000, [0, 1, 999, 2000], 64, 3000, "bf16", 0.1, "zipf", 0, 0),
    (2000, [0, 1, 999, 2000], 64, 3000, "fp32", 0.0, "uniform", 0, 0),
    (900, [0, 450, 900], 515, 2500, "fp32", 0.25, "zipf", 0, 0),
    (900, [0, 450, 900], 516, 2500, "bf16", 0.25, "zipf", 4, 0),
    (900, [0, 450, 900], 264, 700, "bf16", 0.0, "zipf", 0, 3),
    (40, [0, 40], 1100, 3000, "bf16", 0.1, "zipf", 0, 0),
    (3, [0, 3], 40, 5000, "fp32", 0.1, "uniform", 0, 0),
    (262143, [0, 100000, 262143], 16, 20000, "bf16", 0.1, "uniform", 0, 0),
    (5000, [0, 2500, 5000], 24, 70001, "bf16", 0.1, "zipf", 0, 0),
    (1 << 22, [0, 1 << 22], 4, 300, "fp32", 0.0, "uniform", 0, 0),
]


def _ids(kind, s, V, seed):
    r = np.random.default_rng(seed)
    if kind == "uniform":
        return r.integers(0, V, s)
    w = np.cumsum(np.arange(1, V + 1) ** -1.1)
    return np.minimum(np.searchsorted(w, r.random(s) * w[-1]), V - 1)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("V,vs,h,s,grad,p,kind,pad,misalign", BWD)
def test_backward_matches_the_oracle(V, vs, h, s, grad, p, kind, pad, misalign, accumulate):
    ids = _ids(kind, s, V, V + s)
    padding = 1 if V > 1 else None
    if s > 20:
        ids[[0, 7, 8, 9]] = [-1, V, V - 1, -(1 << 60)]
    g, gd = _table(s, s, h, grad)
    seed, offset, scale = 77, (1 << 63) + 5, 3.5
    base = [torch.full((vs[i + 1] - vs[i], h + pad), 0.25, device="cuda") for i in range(len(vs) - 1)]
    init = 0.25 if accumulate else 0.0
    gs = [b[:, :h] for b in base]
    gx = _shards(g, [0, s], pad, misalign)[0]
    ws = torch.full((vpce.vpce_embedding_dropout_backward_workspace_bytes(s, V, h),), 0xA5, dtype=torch.uint8,
                    device="cuda")
    call = dict(scale=scale, p=p, rng=_rng(seed, offset) if p else None, padding_id=padding, accumulate=accumulate)
    vpce.vpce_embedding_dropout_backward(gx, torch.from_numpy(ids).cuda(), gs, vs, workspace=ws, **call)
    got = np.concatenate([q.double().cpu().numpy() for q in gs])
    ref, mag, count = S.embedding_dropout_backward(gd, ids, V, scale, p, seed, offset, padding)
    assert np.all(np.abs(got - ref - init) <= (count[:, None] + 3) * 2.0 ** -24 * (mag + init))
    if pad:
        assert all(bool((b[:, h:] == 0.25).all()) for b in base)
    again = [torch.full_like(q, 0.25) for q in gs]
    vpce.vpce_embedding_dropout_backward(gx, torch.from_numpy(ids).cuda(), again, vs, **call)
    assert all(torch.equal(a, b) for a, b in zip(gs, again))     # the same bits


@pytest.mark.parametrize("s", [300, 40000])
def test_backward_of_one_id_and_of_nothing(s):
    V, h, vs = 70, 72, [0, 30, 70]
    g, gd = _table(s, s, h, "bf16")
    for ids in (np.full(s, 31), np.full(s, 5), np.full(s, -1)):
        gs = [torch.full((30, h), 9.0, device="cuda"), torch.full((40, h), 9.0, device="cuda")]
        vpce.vpce_embedding_dropout_backward(g.cuda(), torch.from_numpy(ids).cuda(), gs, vs, padding_id=5, p=0.1,
                                             rng=_rng(3, 4), accumulate=False)
        ref, mag, count = S.embedding_dropout_backward(gd, ids, V, 1.0, 0.1, 3, 4, 5)
        got = torch.cat(gs).double().cpu().numpy()
        assert np.all(np.abs(got - ref) <= (count[:, None] + 3) * 2.0 ** -24 * mag)


def test_backward_empty_batch():
    g = torch.empty(0, 16, device="cuda")
    ids = torch.empty(0, dtype=torch.int64, device="cuda")
    gs = [torch.full((8, 16), 2.0, device="cuda")]
    vpce.vpce_embedding_dropout_backward(g, ids, gs)
    assert bool((gs[0] == 2.0).all())
    vpce.vpce_embedding_dropout_backward(g, ids, gs, accumulate=False)
    assert not gs[0].any()


def test_forward_and_backward_are_adjoint_on_the_device():
    # <out, g> = <E, dE>, as sums of fp32 products: 1e-4 of the sum of magnitudes
    V, h, s, vs = 500, 200, 900, [0, 123, 500]
    x, xd = _table(9, V, h, "fp32")
    g, gd = _table(10, s, h, "fp32")
    ids = torch.from_numpy(_ids("zipf", s, V, 2)).cuda()
    kw = dict(scale=2.0, p=0.35, rng=_rng(5, 6), padding_id=0)
    out = vpce.vpce_embedding_dropout_forward(_shards(x, vs), ids, vs, **kw)
    gs = [torch.empty(vs[i + 1] - vs[i], h, device="cuda") for i in range(2)]
    vpce.vpce_embedding_dropout_backward(g.cuda(), ids, gs, vs, accumulate=False, **kw)
    a = (out.double() * g.cuda().double()).sum().item()
    b = (torch.cat(gs).double() * x.cuda().double()).sum().item()
    assert abs(a - b) <= 1e-4 * float((out.double() * g.cuda().double()).abs().sum())


def test_another_stream_gives_the_same_bits():
    V, h, s, vs = 400, 264, 900, [0, 150, 400]
    x, _ = _table(13, V, h, "bf16")
    g, _ = _table(14, s, h, "bf16")
    tab, gx, ids = _shards(x, vs), g.cuda(), torch.from_numpy(_ids("zipf", s, V, 4)).cuda()
    kw = dict(p=0.2, rng=_rng(8, 9))
    out = vpce.vpce_embedding_dropout_forward(tab, ids, vs, **kw)
    gs = [torch.zeros(vs[i + 1] - vs[i], h, device="cuda") for i in range(2)]
    vpce.vpce_embedding_dropout_backward(gx, ids, gs, vs, **kw)
    gs2 = [torch.zeros_like(q) for q in gs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    out2 = vpce.vpce_embedding_dropout_forward(tab, ids, vs, stream=side, **kw)
    vpce.vpce_embedding_dropout_backward(gx, ids, gs2, vs, stream=side, **kw)
    junk = torch.full((1 << 22,), 7, dtype=torch.uint8, device="cuda")   # the workspace is not up for reuse here
    side.synchronize()
    assert torch.equal(out, out2) and all(torch.equal(a, b) for a, b in zip(gs, gs2)) and junk[0] == 7


def test_graph_replay_draws_a_new_mask():
    V, h, s, vs = 200, 96, 50, [0, 90, 200]
    x, xd = _table(11, V, h, "bf16")
    tab = _shards(x, vs)
    ids_h = _ids("uniform", s, V, 3)
    ids = torch.from_numpy(ids_h).cuda()
    rng = _rng(21, 0)
    out = torch.empty(s, h, dtype=torch.bfloat16, device="cuda")
    gs = [torch.empty(vs[i + 1] - vs[i], h, device="cuda") for i in range(2)]
    ws = torch.empty(vpce.vpce_embedding_dropout_backward_workspace_bytes(s, V, h), dtype=torch.uint8, device="cuda")

    def step():
        vpce.vpce_embedding_dropout_forward(tab, ids, vs, p=0.5, rng=rng, out=out)
        vpce.vpce_embedding_dropout_backward(out, ids, gs, vs, p=0.5, rng=rng, accumulate=False, workspace=ws)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for offset in (1, 2):
        rng[1] = offset
        graph.replay()
        torch.cuda.synchronize()
        ref, _ = S.embedding_dropout_forward(xd, ids_h, 1.0, 0.5, 21, offset)
        got = out.double().cpu().numpy()
        assert np.array_equal(got == 0, ref == 0)
        d, mag, count = S.embedding_dropout_backward(got, ids_h, V, 1.0, 0.5, 21, offset)
        assert np.all(np.abs(torch.cat(gs).double().cpu().numpy() - d) <= (count[:, None] + 3) * 2.0 ** -24 * mag)
