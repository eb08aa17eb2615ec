"""Refusals of the token-score and embedding-dropout entry points on the host,
before any CUDA call, and the exports' workspace sizes."""
import ctypes

import pytest

from vocab_sharded_lm_gb300 import _build, vpce

FAKE = 0x7F0000000000  # a 256-byte aligned "device" address, never dereferenced on the host
NAN, INF = float("nan"), float("inf")


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return vpce.load_library()


def _arr(v):
    return None if v is None else vpce._ptr_array(v)


def _fwd(lib, **kw):
    a = dict(shards=[FAKE, FAKE + 4096], dtype=1, t=2, s=4, vs=[0, 8, 48], ld=0, y=FAKE, ig=-100, T=1.0, top=4,
             logp=FAKE, ent=FAKE, ids=FAKE, tl=FAKE, stats=FAKE, flag=FAKE)
    a.update(kw)
    return lib.vpce_logprob_forward(_arr(a["shards"]), a["dtype"], a["t"], a["s"],
                                    vpce._i64_array(a["vs"]) if a["vs"] else None, a["ld"], a["y"], a["ig"], a["T"],
                                    a["top"], a["logp"], a["ent"], a["ids"], a["tl"], a["stats"], a["flag"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3),
    (dict(t=0), 1),
    (dict(s=-1), 1),
    (dict(shards=None), 1),
    (dict(shards=[FAKE, 0]), 1),
    (dict(shards=[FAKE + 1, FAKE]), 2),
    (dict(vs=None), 1),
    (dict(vs=[1, 8, 48]), 1),
    (dict(vs=[0, 8, 8]), 1),
    (dict(ld=39), 1),
    (dict(y=None), 1),                                # logp without targets
    (dict(y=FAKE + 4), 2),
    (dict(T=0.0), 1), (dict(T=-1.0), 1), (dict(T=NAN), 1), (dict(T=INF), 1), (dict(T=1e-40), 1),
    (dict(top=-1), 1), (dict(top=33), 1),
    (dict(top=10, vs=[0, 1, 9]), 1),                  # more alternatives than columns
    (dict(ids=None), 1),
    (dict(top=0), 1),                                 # top outputs without top
    (dict(top=0, ids=None, tl=None, logp=None, ent=None, stats=None), 1),
    (dict(logp=FAKE + 2), 2), (dict(ent=FAKE + 1), 2), (dict(ids=FAKE + 4), 2), (dict(tl=FAKE + 2), 2),
    (dict(stats=FAKE + 8), 2), (dict(flag=FAKE + 2), 2),
])
def test_logprob_forward_refuses(lib, kw, code):
    assert _fwd(lib, **kw) == code


def _bwd(lib, **kw):
    a = dict(shards=[FAKE, FAKE + 4096], dtype=0, t=2, s=4, vs=[0, 8, 48], ld=0, y=FAKE, ig=-100, T=1.0, stats=FAKE,
             gl=FAKE, ge=FAKE, top=4, ids=FAKE, gt=FAKE, grads=[FAKE, FAKE + 4096], ldg=0)
    a.update(kw)
    return lib.vpce_logprob_backward(_arr(a["shards"]), a["dtype"], a["t"], a["s"],
                                     vpce._i64_array(a["vs"]) if a["vs"] else None, a["ld"], a["y"], a["ig"], a["T"],
                                     a["stats"], a["gl"], a["ge"], a["top"], a["ids"], a["gt"], _arr(a["grads"]),
                                     a["ldg"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=9), 3),
    (dict(y=None), 1),
    (dict(stats=None), 1),
    (dict(stats=FAKE + 4), 2),
    (dict(gl=None, ge=None, top=0), 1),
    (dict(ids=None), 1), (dict(gt=None), 1), (dict(top=33), 1), (dict(top=-2), 1),
    (dict(gl=FAKE + 2), 2), (dict(ge=FAKE + 3), 2), (dict(ids=FAKE + 4), 2), (dict(gt=FAKE + 1), 2),
    (dict(grads=None), 1), (dict(grads=[FAKE, 0]), 1), (dict(grads=[FAKE + 2, FAKE]), 2),
    (dict(ldg=39), 1),
    (dict(ldg=64), 1),                                # in place with another stride
    (dict(T=0.0), 1), (dict(T=NAN), 1),
    (dict(vs=[0, 0, 48]), 1),
])
def test_logprob_backward_refuses(lib, kw, code):
    assert _bwd(lib, **kw) == code


def _efwd(lib, **kw):
    a = dict(tab=[FAKE, FAKE + 4096], dtype=1, t=2, vs=[0, 8, 16], h=24, ldt=0, ids=FAKE, s=4, pad=-1, scale=1.0,
             p=0.1, rng=FAKE, out=FAKE, od=1, ldo=0, flag=None)
    a.update(kw)
    return lib.vpce_embedding_dropout_forward(_arr(a["tab"]), a["dtype"], a["t"],
                                              vpce._i64_array(a["vs"]) if a["vs"] else None, a["h"], a["ldt"],
                                              a["ids"], a["s"], a["pad"], a["scale"], a["p"], a["rng"], a["out"],
                                              a["od"], a["ldo"], a["flag"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=2), 3), (dict(od=-1), 3),
    (dict(t=0), 1), (dict(t=65), 1), (dict(s=-1), 1), (dict(h=0), 1), (dict(h=1 << 31), 1),
    (dict(vs=None), 1), (dict(vs=[0, 8, 8]), 1), (dict(vs=[1, 8, 16]), 1), (dict(vs=[0, 8, 1 << 31]), 1),
    (dict(tab=None), 1), (dict(tab=[FAKE, 0]), 1), (dict(tab=[FAKE + 1, FAKE]), 2),
    (dict(ldt=23), 1), (dict(ldo=23), 1),
    (dict(ids=None), 1), (dict(ids=FAKE + 4), 2),
    (dict(scale=NAN), 1), (dict(scale=INF), 1), (dict(scale=3e38, p=0.9), 1),
    (dict(p=-0.1), 1), (dict(p=1.0), 1), (dict(p=NAN), 1),
    (dict(rng=None), 1), (dict(rng=FAKE + 4), 2),
    (dict(out=None), 1), (dict(out=FAKE + 1), 2), (dict(flag=FAKE + 2), 2),
])
def test_embedding_dropout_forward_refuses(lib, kw, code):
    assert _efwd(lib, **kw) == code


def _ebwd(lib, **kw):
    a = dict(g=FAKE, dtype=1, ldg=0, ids=FAKE, s=4, pad=-1, scale=1.0, p=0.1, rng=FAKE, tab=[FAKE, FAKE + 4096], t=2,
             vs=[0, 8, 16], h=23, ldt=0, acc=0, ws=FAKE, nb=1 << 30)
    a.update(kw)
    return lib.vpce_embedding_dropout_backward(a["g"], a["dtype"], a["ldg"], a["ids"], a["s"], a["pad"], a["scale"],
                                               a["p"], a["rng"], _arr(a["tab"]), a["t"],
                                               vpce._i64_array(a["vs"]) if a["vs"] else None, a["h"], a["ldt"],
                                               a["acc"], a["ws"], a["nb"], None)


@pytest.mark.parametrize("kw,code", [
    (dict(dtype=5), 3),
    (dict(t=0), 1), (dict(s=-1), 1), (dict(h=0), 1), (dict(vs=None), 1), (dict(vs=[0, 9, 8]), 1),
    (dict(tab=None), 1), (dict(tab=[FAKE, 0]), 1), (dict(tab=[FAKE + 2, FAKE]), 2),
    (dict(ldg=22), 1), (dict(ldt=22), 1), (dict(acc=2), 1),
    (dict(g=None), 1), (dict(g=FAKE + 1), 2), (dict(ids=None), 1), (dict(ids=FAKE + 1), 2),
    (dict(scale=NAN), 1), (dict(p=1.5), 1), (dict(rng=None), 1), (dict(rng=FAKE + 1), 2),
    (dict(ws=None), 1), (dict(ws=FAKE + 64), 2), (dict(nb=1), 4),
])
def test_embedding_dropout_backward_refuses(lib, kw, code):
    assert _ebwd(lib, **kw) == code


def test_workspace_sizes(lib):
    f = lib.vpce_embedding_dropout_backward_workspace_bytes
    assert f(-1, 10, 10) == 0 and f(1, 0, 10) == 0 and f(1, 10, 0) == 0 and f(1, 1 << 31, 10) == 0
    for s, V, h in ((0, 1, 1), (8192, 128256, 8192), (1 << 20, 256000, 64)):
        assert f(s, V, h) > 0 and f(s, V, h) % 256 == 0


def test_valid_calls_without_a_gpu_report_a_cuda_error(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the host-only path")
    assert _fwd(lib) == 5 and _bwd(lib) == 5 and _efwd(lib) == 5 and _ebwd(lib) == 5
    assert _fwd(lib, y=None, logp=None) == 5                # targets are optional without logp
    assert _fwd(lib, top=0, ids=None, tl=None) == 5
    assert _efwd(lib, p=0.0, rng=None) == 5                 # no generator without dropout
    assert _bwd(lib, gl=None, y=None, top=0, ids=None, gt=None) == 5


def test_python_refusals():
    """The torch forms check shapes and types before the library is called."""
    import torch

    cpu = torch.zeros(2, 8)
    with pytest.raises(ValueError):
        vpce.vpce_logprob_forward([cpu])                    # not CUDA
    with pytest.raises(ValueError):
        vpce.vpce_logprob_forward([])
    with pytest.raises(TypeError):
        vpce.vpce_logprob_forward([cpu.double()])
    with pytest.raises(ValueError):
        vpce.vpce_embedding_dropout_forward([cpu], torch.zeros(3, dtype=torch.int64))
