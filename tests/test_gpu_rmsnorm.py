"""GPU parity of the norm with residual (vpce_rmsnorm_*) with the fp64 oracle.

With u = 2^-24 (half a step of fp32):
* rstd: a sum of squares in at most 32 steps a thread and 10 of a tree is
  within 45 u, its root within 23 u; the mean, eps and the square root's 2 ulp
  add 7 u: 32 u in all, 2^-19.
* out: that, the sum's rounding (1 u) and two products: 2^-18 of the value in
  fp32; half a step of bf16, 2^-8, more in bf16.
* scale: as the largest out, with one division: 2^-18.
* codes: the nearest value of out / scale, which the kernel knows within
  2^-17: another one only within that distance of a midpoint.
* gradient: every term is a product of at most five rounded factors, the row's
  mean adds 45 u of its terms' magnitudes: 64 u of the magnitudes' sum; the
  weight's terms add up in some order: (s + 8) u of theirs."""
import numpy as np
import pytest
import torch

from oracle import train_oracle as T
from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu
DT = {"bf16": torch.bfloat16, "fp32": torch.float32}
HALF = {"bf16": 2.0 ** -8, "fp32": 0.0}
U = 2.0 ** -24


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


def _rows(seed, s, h, dtype, std=1.0, pad=0, misalign=0):
    """[s, h] on the GPU in rows of h + pad elements, `misalign` elements past
    16 bytes, NaN around it; and its values in fp64."""
    x = torch.from_numpy(np.random.default_rng(seed).normal(size=(s, h)) * std).to(DT[dtype])
    flat = torch.full((s * (h + pad) + misalign,), float("nan"), dtype=DT[dtype], device="cuda")
    v = flat[misalign:].view(s, h + pad)[:, :h]
    v.copy_(x)
    return v, x.double().numpy()


CASES = [
    # s, h, x, residual, weight, pad, misalign
    (1, 1, "fp32", None, "fp32", 0, 0),
    (3, 7, "bf16", "bf16", "fp32", 0, 0),
    (50, 1, "fp32", "fp32", "fp32", 0, 2),
    (50, 1, "bf16", "bf16", "bf16", 0, 5),
    (40, 3, "bf16", "fp32", "fp32", 0, 3),
    (5, 8, "bf16", "fp32", "bf16", 0, 0),
    (9, 256, "bf16", "bf16", "bf16", 8, 0),
    (9, 264, "fp32", "fp32", "bf16", 0, 0),
    (6, 1024, "bf16", None, "bf16", 0, 0),
    (6, 1024, "bf16", "fp32", "fp32", 0, 1),
    (33, 515, "fp32", "fp32", "fp32", 0, 0),
    (33, 515, "bf16", "bf16", "bf16", 1, 3),
    (4, 1032, "bf16", "bf16", "bf16", 0, 0),
    (2, 2049, "fp32", None, "bf16", 0, 0),
    (700, 136, "bf16", "fp32", "bf16", 0, 0),
    (3, 8192, "bf16", "bf16", "bf16", 0, 0),
    (400, 4096, "bf16", "bf16", "fp32", 64, 0),
    (2, 8200, "fp32", "fp32", "fp32", 0, 0),
    (2, 16392, "bf16", "bf16", "bf16", 0, 0),
    (2, 17001, "bf16", "fp32", "bf16", 0, 0),
    (2, 32768, "fp32", "fp32", "bf16", 0, 0),
    (1, 32767, "bf16", "bf16", "bf16", 0, 0),
]


def _inputs(s, h, x, residual, weight, pad, misalign):
    xs, xd = _rows(s + h, s, h, x, 1.0, pad, misalign)
    rs, rd = (None, None) if residual is None else _rows(s * h + 1, s, h, residual, 2.0, pad, misalign)
    w, wd = _rows(h, 1, h, weight, 1.0)
    return xs, xd, rs, rd, w[0], wd[0]


@pytest.mark.parametrize("s,h,x,residual,weight,pad,misalign", CASES)
def test_forward_matches_the_oracle(s, h, x, residual, weight, pad, misalign):
    xs, xd, rs, rd, w, wd = _inputs(s, h, x, residual, weight, pad, misalign)
    out = torch.full((s, h + pad), -3.0, dtype=DT[x], device="cuda")
    got = vpce.vpce_rmsnorm_forward(xs, w, rs, eps=1e-5, out=out[:, :h])
    y, r, rstd = T.rmsnorm(xd, wd, rd, float(np.float32(1e-5)))
    assert np.all(np.abs(got.rstd.double().cpu().numpy() - rstd) <= 2.0 ** -19 * rstd)
    assert np.all(np.abs(got.out.double().cpu().numpy() - y) <= (2.0 ** -18 + HALF[x]) * np.abs(y))
    if residual is None:
        assert got.residual is xs
    else:
        assert np.all(np.abs(got.residual.double().cpu().numpy() - r) <= (U + HALF[residual]) * np.abs(r))
    if pad:
        assert bool((out[:, h:] == -3.0).all())
    again = vpce.vpce_rmsnorm_forward(xs, w, rs, eps=1e-5)
    assert torch.equal(again.out, got.out) and torch.equal(again.rstd, got.rstd)


@pytest.mark.parametrize("group", [0, 16, 64, 128, 48, 1024])
@pytest.mark.parametrize("s,h,x,residual,weight,pad,misalign", CASES)
def test_quantized_forward_matches_the_oracle(s, h, x, residual, weight, pad, misalign, group):
    xs, xd, rs, rd, w, wd = _inputs(s, h, x, residual, weight, pad, misalign)
    q = torch.full((s, h + pad), 0x55, dtype=torch.uint8, device="cuda").view(torch.float8_e4m3fn)
    got = vpce.vpce_rmsnorm_quantized_forward(xs, w, rs, eps=1e-5, group=group, q_out=q[:, :h])
    y, r, rstd = T.rmsnorm(xd, wd, rd, float(np.float32(1e-5)))
    scale, each = T.group_scales(y, group)
    assert np.all(np.abs(got.rstd.double().cpu().numpy() - rstd) <= 2.0 ** -19 * rstd)
    gs = got.scale.double().cpu().numpy()
    assert gs.shape == scale.shape and np.all(np.abs(gs - scale) <= 2.0 ** -18 * scale)
    a = y / each
    want, near = T.nearest_e4m3(np.clip(a, -448, 448))
    codes = got.q.float().double().cpu().numpy()
    other = codes != want
    assert np.all(near[other] <= 2.0 ** -17 * np.abs(a[other]))
    assert np.all(np.abs(codes - a) <= 2.0 ** -4 * (1 + 2.0 ** -12) * np.abs(a) + 2.0 ** -10)
    if residual is not None:
        assert np.all(np.abs(got.residual.double().cpu().numpy() - r) <= (U + HALF[residual]) * np.abs(r))
    if pad:
        assert bool((q.view(torch.uint8)[:, h:] == 0x55).all())
    # the quantized form's sum and rstd are the other form's
    plain = vpce.vpce_rmsnorm_forward(xs, w, rs, eps=1e-5)
    assert torch.equal(plain.rstd, got.rstd)


@pytest.mark.parametrize("accumulate", [False, True])
@pytest.mark.parametrize("s,h,x,residual,weight,pad,misalign", CASES)
def test_backward_matches_the_oracle(s, h, x, residual, weight, pad, misalign, accumulate):
    rt = residual or x
    r, rd = _rows(s + h, s, h, rt, 2.0, pad, misalign)
    dy, dyd = _rows(s * h + 3, s, h, x, 1e-2, pad, misalign)
    dres, dresd = (None, None) if residual is None else _rows(s * h + 5, s, h, rt, 1e-2, pad, misalign)
    w, wd = _rows(h, 1, h, weight, 1.0)
    rstd = torch.from_numpy(1 / np.sqrt((rd ** 2).mean(1) + 1e-5)).float().cuda()
    dw = torch.full((h,), 0.25, device="cuda")
    dx = torch.full((s, h + pad), -3.0, dtype=DT[rt], device="cuda")
    ws = torch.full((vpce.vpce_rmsnorm_backward_workspace_bytes(s, h),), 0xFF, dtype=torch.uint8, device="cuda")
    call = dict(grad_residual=dres, accumulate=accumulate)
    vpce.vpce_rmsnorm_backward(dy, r, w[0], rstd, grad_in=dx[:, :h], grad_weight=dw, workspace=ws, **call)
    ref, refw, mag, magw = T.rmsnorm_backward(dyd, rd, wd[0], rstd.double().cpu().numpy(), dresd)
    err = np.abs(dx[:, :h].double().cpu().numpy() - ref)
    assert np.all(err <= 64 * U * mag + HALF[rt] * np.abs(ref))
    base = 0.25 if accumulate else 0.0
    assert np.all(np.abs(dw.double().cpu().numpy() - refw - base) <= (s + 8) * U * (magw + base))
    if pad:
        assert bool((dx[:, h:] == -3.0).all())
    dw2 = torch.full((h,), 0.25, device="cuda")
    dx2, _ = vpce.vpce_rmsnorm_backward(dy, r, w[0], rstd, grad_weight=dw2, **call)
    assert torch.equal(dx2, dx[:, :h]) and torch.equal(dw2, dw)   # the same bits


@pytest.mark.parametrize("residual", [False, True])
@pytest.mark.parametrize("x,r", [("bf16", "bf16"), ("bf16", "fp32"), ("fp32", "fp32")])
@pytest.mark.parametrize("s,h", [(9, 256), (170, 512), (9, 1024), (330, 2048), (6, 5120), (4, 8192), (3, 16384)])
def test_rows_that_fill_their_threads(s, h, x, r, residual):
    # every thread's columns are all of the row's: forms without the branches of
    # other rows, with and without a residual
    if r != x and not residual:
        pytest.skip("the residual's type without a residual")
    case = (s, h, x, r if residual else None, "bf16", 0, 0)
    test_forward_matches_the_oracle(*case)
    for group in (0, 48, 128):
        test_quantized_forward_matches_the_oracle(*case, group)
    test_backward_matches_the_oracle(*case, False)


def test_backward_of_many_rows_adds_every_row():
    # 20000 rows of equal terms: each column's sum is exact in fp32
    s, h = 20000, 72
    r = torch.ones(s, h, device="cuda")
    dy = torch.full((s, h), 0.5, device="cuda")
    rstd = torch.full((s,), 2.0, device="cuda")
    _, dw = vpce.vpce_rmsnorm_backward(dy, r, torch.zeros(h, device="cuda"), rstd)
    assert bool((dw == float(s)).all())


@pytest.mark.parametrize("x,residual", [("fp32", None), ("fp32", "fp32")])
def test_gradient_against_differences(x, residual):
    # central differences of L = sum(out * c) along random directions; fp32
    # rounding of L's terms (2^-18 each, as above) over the step's length
    s, h = 4, 40
    xs, _ = _rows(1, s, h, x)
    rs = None if residual is None else _rows(2, s, h, residual)[0]
    w, _ = _rows(3, 1, h, "fp32")
    c, cd = _rows(4, s, h, "fp32")
    f = vpce.vpce_rmsnorm_forward(xs, w[0], rs)
    dx, dw = vpce.vpce_rmsnorm_backward(c, f.residual, w[0], f.rstd)
    step = 2.0 ** -6

    def loss(xx, ww):
        y = vpce.vpce_rmsnorm_forward(xx, ww, rs).out.double().cpu().numpy()
        return (y * cd).sum(), (np.abs(y * cd)).sum()

    for k in range(3):
        dir_x, dir_w = _rows(10 + k, s, h, "fp32")[0], _rows(20 + k, 1, h, "fp32")[0][0]
        for a, b, want in ((dir_x, 0 * dir_w, (dx.double() * dir_x.double()).sum().item()),
                           (0 * dir_x, dir_w, (dw.double() * dir_w.double()).sum().item())):
            up, mag = loss(xs + step * a, w[0] + step * b)
            down, _ = loss(xs - step * a, w[0] - step * b)
            # the third derivative's term is step^2 / 6 of a value of the size of
            # the loss' terms along a direction of length about sqrt(s h)
            assert abs((up - down) / (2 * step) - want) <= mag * 2.0 ** -18 / step + step ** 2 * mag * 4


@pytest.mark.parametrize("h", [520, 515, 4097, 8200])
def test_in_place_and_empty(h):
    s = 337
    xs, _ = _rows(1, s, h, "bf16")
    rs, _ = _rows(2, s, h, "bf16", 2.0)
    w, _ = _rows(3, 1, h, "bf16")
    ref = vpce.vpce_rmsnorm_forward(xs, w[0], rs)
    x2, r2 = xs.clone(), rs.clone()
    got = vpce.vpce_rmsnorm_forward(x2, w[0], r2, out=x2, residual_out=r2)
    assert got.out is x2 and got.residual is r2
    assert torch.equal(x2, ref.out) and torch.equal(r2, ref.residual)
    x3 = xs.clone()
    assert torch.equal(vpce.vpce_rmsnorm_forward(x3, w[0], rs, residual_out=x3).residual, ref.residual)
    dy, _ = _rows(4, s, h, "bf16")
    dr, _ = _rows(5, s, h, "bf16")
    dx, dw = vpce.vpce_rmsnorm_backward(dy, ref.residual, w[0], ref.rstd, grad_residual=dr)
    for k in range(3):
        a, b, c = dy.clone(), ref.residual.clone(), dr.clone()
        into = (a, b, c)[k]
        dx2, dw2 = vpce.vpce_rmsnorm_backward(a, b, w[0], ref.rstd, grad_residual=c, grad_in=into)
        assert dx2 is into and torch.equal(into, dx) and torch.equal(dw2, dw)
    none = xs[:0]
    f = vpce.vpce_rmsnorm_forward(none, w[0])
    assert f.out.shape == (0, h)
    assert vpce.vpce_rmsnorm_quantized_forward(none, w[0], group=64).scale.shape == (0, -(-h // 64))
    g = torch.full((h,), 2.0, device="cuda")
    vpce.vpce_rmsnorm_backward(none, none, w[0], f.rstd, grad_weight=g, accumulate=True)
    assert bool((g == 2.0).all())
    vpce.vpce_rmsnorm_backward(none, none, w[0], f.rstd, grad_weight=g)
    assert not g.any()


@pytest.mark.parametrize("h", [256, 512, 1024, 8192, 16384])
def test_in_place_in_rows_that_fill_their_threads(h):
    test_in_place_and_empty(h)


@pytest.mark.parametrize("h,group", [(512, 128), (515, 64), (2048, 0)])
def test_rows_of_zeros_and_of_what_is_not_finite(h, group):
    x = torch.ones(6, h, device="cuda")
    x[0] = 0.0
    x[1, 3] = float("nan")
    x[2, 5] = float("inf")
    x[3] = 1e25          # squares past fp32
    x[4] = 1e-30         # squares below it: eps alone
    w = torch.ones(h, device="cuda")
    f = vpce.vpce_rmsnorm_forward(x, w, eps=1e-6)
    q = vpce.vpce_rmsnorm_quantized_forward(x, w, eps=1e-6, group=group)
    assert not f.out[0].any() and not q.q[0].float().any() and bool((q.scale[0] == T.TINY).all())
    assert bool(f.out[1].isnan().all()) and bool(q.q[1].float().isnan().all()) and bool(q.scale[1].isnan().all())
    assert bool(f.out[2, 5].isnan()) and not f.out[2, :5].any() and bool(q.q[2, 5].float().isnan())
    assert not f.out[3].any() and f.rstd[3] == 0
    assert torch.allclose(f.out[4], torch.full_like(x[4], 1e-27), rtol=1e-6, atol=0)
    assert torch.allclose(f.out[5], torch.full_like(x[5], (1 + 1e-6) ** -0.5), rtol=1e-6)
    # an infinite weight: its group alone
    w[1] = float("inf")
    q = vpce.vpce_rmsnorm_quantized_forward(torch.ones(1, h, device="cuda"), w, group=group)
    assert bool(q.scale[0, 0].isinf()) and bool(q.q[0, 1].float().isnan())
    if group:
        assert bool(q.scale[0, 1:].isfinite().all()) and bool((q.q[0, group:].float() == 448).all())
    # eps 0 and a row of zeros: 0 / 0
    assert bool(vpce.vpce_rmsnorm_forward(x[:1], torch.ones(h, device="cuda"), eps=0.0).out.isnan().all())


def test_offsets_past_32_bits():
    # rows 2^31 elements apart
    s, h, ld = 3, 264, 1 << 31
    big = torch.empty((s - 1) * ld + h, dtype=torch.bfloat16, device="cuda")
    x = big.as_strided((s, h), (ld, 1))
    dense, _ = _rows(1, s, h, "bf16")
    x.copy_(dense)
    w, _ = _rows(2, 1, h, "bf16")
    f, fd = vpce.vpce_rmsnorm_forward(x, w[0]), vpce.vpce_rmsnorm_forward(dense, w[0])
    assert torch.equal(f.out, fd.out)
    q, qd = (vpce.vpce_rmsnorm_quantized_forward(v, w[0], group=16) for v in (x, dense))
    assert torch.equal(q.q.view(torch.uint8), qd.q.view(torch.uint8)) and torch.equal(q.scale, qd.scale)
    a, b = (vpce.vpce_rmsnorm_backward(v, v, w[0], f.rstd, grad_residual=v) for v in (x, dense))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])
    x = big[1:].as_strided((s, h - 1), (ld - 1, 1))          # and off 16 bytes
    x.copy_(dense[:, 1:])
    odd = dense[:, 1:].contiguous()
    f, fd = vpce.vpce_rmsnorm_forward(x, w[0][1:]), vpce.vpce_rmsnorm_forward(odd, w[0][1:])
    assert torch.equal(f.out, fd.out)
    a, b = (vpce.vpce_rmsnorm_backward(v, v, w[0][1:], f.rstd, grad_residual=v) for v in (x, odd))
    assert torch.equal(a[0], b[0]) and torch.equal(a[1], b[1])


def test_another_stream_gives_the_same_bits():
    s, h = 900, 1032
    x, _ = _rows(1, s, h, "bf16")
    r, _ = _rows(2, s, h, "bf16")
    w, _ = _rows(3, 1, h, "bf16")
    side = torch.cuda.Stream()

    def all_of(**kw):
        f = vpce.vpce_rmsnorm_forward(x, w[0], r, **kw)
        q = vpce.vpce_rmsnorm_quantized_forward(x, w[0], r, group=128, **kw)
        return [*f, q.q.view(torch.uint8), q.scale, *vpce.vpce_rmsnorm_backward(x, f.residual, w[0], f.rstd,
                                                                                grad_residual=r, **kw)]

    a = all_of()
    side.wait_stream(torch.cuda.current_stream())
    b = all_of(stream=side)
    side.synchronize()
    assert all(torch.equal(p, q) for p, q in zip(a, b))


def test_graph_replay_follows_its_inputs():
    s, h = 300, 2048
    x, _ = _rows(1, s, h, "bf16")
    r, _ = _rows(2, s, h, "bf16")
    w, _ = _rows(3, 1, h, "bf16")
    dw = torch.zeros(h, device="cuda")
    state = {}

    def step():
        f = vpce.vpce_rmsnorm_forward(x, w[0], r)
        q = vpce.vpce_rmsnorm_quantized_forward(x, w[0], r, group=128)
        dx, _ = vpce.vpce_rmsnorm_backward(x, f.residual, w[0], f.rstd, grad_residual=r, grad_weight=dw)
        state.update(out=f.out, q=q.q, scale=q.scale, dx=dx)

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    torch.cuda.current_stream().wait_stream(side)
    torch.cuda.synchronize()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    held = dict(state)
    for k in range(3):
        x.copy_(_rows(50 + k, s, h, "bf16")[0])
        graph.replay()
        torch.cuda.synchronize()
        got = {n: t.clone() for n, t in held.items()} | {"dw": dw.clone()}
        step()
        torch.cuda.synchronize()
        for n in ("out", "scale", "dx"):
            assert torch.equal(got[n], state[n]), n
        assert torch.equal(got["q"].view(torch.uint8), state["q"].view(torch.uint8)) and torch.equal(got["dw"], dw)
