"""What the Python forms ask of their operands before the library is called:
workspaces, and one device for all of them, on which the call is made."""
import contextlib
import types

import pytest
import torch

from vocab_sharded_lm_gb300 import distributed, vpce

from _fake_cuda import Fake0, Fake1, fake, install

S, H, V = 4, 16, 24
F32, BF16, I64, U8 = torch.float32, torch.bfloat16, torch.int64, torch.uint8


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch, vpce)


def new(*shape, dtype=F32, index=0):
    return fake(torch.zeros(shape, dtype=dtype), index)


def ids():
    return new(S, dtype=I64)


def bf(*shape):
    return new(*shape, dtype=BF16)


# every call that takes a workspace
WITH_WORKSPACE = {
    "vpce_embedding_dropout_backward": lambda ws: vpce.vpce_embedding_dropout_backward(
        new(S, H), ids(), [new(V, H)], workspace=ws),
    "vpce_embedding_backward": lambda ws: vpce.vpce_embedding_backward(new(S, H), ids(), [new(V, H)], workspace=ws),
    "vpce_forward": lambda ws: vpce.vpce_forward([new(S, V)], ids(), loss_out=new(), workspace=ws),
    "vpce_backward": lambda ws: vpce.vpce_backward([new(S, V)], ids(), ws),
    "vpce_backward_rows": lambda ws: vpce.vpce_backward([new(S, V)], ids(), ws, grad_rows=new(S)),
    "vpce_forward_backward": lambda ws: vpce.vpce_forward_backward([new(S, V)], ids(), loss_out=new(), workspace=ws),
    "vpce_forward_backward_rows": lambda ws: vpce.vpce_forward_backward(
        [new(S, V)], ids(), grad_rows=new(S), loss_out=new(), workspace=ws),
    "vpce_lmhead_forward": lambda ws: vpce.vpce_lmhead_forward(
        bf(S, H), [bf(V, H)], ids(), loss_out=new(), workspace=ws),
    "vpce_lmhead_backward": lambda ws: vpce.vpce_lmhead_backward(
        bf(S, H), [bf(V, H)], ids(), new(256, dtype=U8), grad_hidden=bf(S, H), grad_weight_shards=[new(V, H)],
        workspace=ws),
    "vpce_lmhead_backward, the forward's": lambda ws: vpce.vpce_lmhead_backward(
        bf(S, H), [bf(V, H)], ids(), ws, grad_hidden=bf(S, H), grad_weight_shards=[new(V, H)],
        workspace=new(256, dtype=U8)),
    "vpce_lmhead_forward_backward": lambda ws: vpce.vpce_lmhead_forward_backward(
        bf(S, H), [bf(V, H)], ids(), loss_out=new(), grad_hidden=bf(S, H), grad_weight_shards=[new(V, H)],
        workspace=ws),
}


@pytest.mark.parametrize("name", WITH_WORKSPACE)
def test_a_workspace_is_contiguous_cuda_memory_and_counted_in_bytes(lib, name):
    call = WITH_WORKSPACE[name]
    with pytest.raises(ValueError, match="workspace"):
        call(torch.zeros(1 << 12, dtype=U8))                  # host memory
    with pytest.raises(ValueError, match="workspace"):
        call(new(1, dtype=U8).expand(1 << 12))                # one byte
    assert lib.calls == []
    ws = new(64, dtype=F32)
    call(ws)
    (_, args), = lib.calls
    at = [getattr(a, "value", a) for a in args].index(ws.data_ptr())
    assert args[at + 1] == 256


# every call, with operand k moved to another device (k < 0: none)
def _placed(k, *operands):
    return [o.as_subclass(Fake1) if i == k else o for i, o in enumerate(operands)]


def _score(k, **kw):
    z0, z1, y, lp, en, ids_, tl, st, fl = _placed(k, new(S, V), new(S, V), ids(), new(S), new(S),
                                                  new(S, 2, dtype=I64), new(S, 2), new(S, 4), new(1, dtype=torch.int32))
    vpce.vpce_logprob_forward([z0, z1], y, top=2, logp_out=lp, entropy_out=en, top_ids_out=ids_, top_logp_out=tl,
                              stats_out=st, flag=fl, **kw)


def _score_grad(k, **kw):
    z, y, st, gl, ge, ti, gt, g = _placed(k, new(S, V), ids(), new(S, 4), new(S), new(S), new(S, 2, dtype=I64),
                                          new(S, 2), new(S, V))
    vpce.vpce_logprob_backward([z], y, st, grad_logp=gl, grad_entropy=ge, top_ids=ti, grad_top_logp=gt,
                               grad_shards=[g], **kw)


def _lookup_dropout(k, **kw):
    e0, e1, i, r, o, f = _placed(k, new(V, H), new(V, H), ids(), new(2, dtype=I64), new(S, H),
                                 new(1, dtype=torch.int32))
    vpce.vpce_embedding_dropout_forward([e0, e1], i, p=0.5, rng=r, out=o, flag=f, **kw)


def _lookup_dropout_grad(k, **kw):
    g, i, e0, e1, r, w = _placed(k, new(S, H), ids(), new(V, H), new(V, H), new(2, dtype=I64), new(256, dtype=U8))
    vpce.vpce_embedding_dropout_backward(g, i, [e0, e1], p=0.5, rng=r, workspace=w, **kw)


def _lookup(k, **kw):
    e0, e1, i, o, f = _placed(k, new(V, H), new(V, H), ids(), new(S, H), new(1, dtype=torch.int32))
    vpce.vpce_embedding_forward([e0, e1], i, out=o, flag=f, **kw)


def _lookup_grad(k, **kw):
    g, i, e0, e1, w = _placed(k, new(S, H), ids(), new(V, H), new(V, H), new(256, dtype=U8))
    vpce.vpce_embedding_backward(g, i, [e0, e1], workspace=w, **kw)


def _loss(k, **kw):
    z0, z1, y, lo, ro, w = _placed(k, new(S, V), new(S, V), ids(), new(), new(S), new(256, dtype=U8))
    vpce.vpce_forward([z0, z1], y, loss_out=lo, row_loss_out=ro, workspace=w, **kw)


def _loss_grad(k, **kw):
    z, y, w, g = _placed(k, new(S, V), ids(), new(256, dtype=U8), new(S))
    vpce.vpce_backward([z], y, w, grad_rows=g, **kw)


def _fused(k, **kw):
    z, y, lo, ro, g, w = _placed(k, new(S, V), ids(), new(), new(S), new(S), new(256, dtype=U8))
    vpce.vpce_forward_backward([z], y, loss_out=lo, row_loss_out=ro, grad_rows=g, workspace=w, **kw)


def _static(k, **kw):
    z, y, lo, ro = _placed(k, new(S, V), ids(), new(), new(S))
    vpce.vpce_forward_static([z], y, lo, row_loss_out=ro, **kw)


def _head(k, **kw):
    x, w0, w1, y, lo, ro, w = _placed(k, bf(S, H), bf(V, H), bf(V, H), ids(), new(), new(S), new(256, dtype=U8))
    vpce.vpce_lmhead_forward(x, [w0, w1], y, loss_out=lo, row_loss_out=ro, workspace=w, **kw)


def _head_grad(k, **kw):
    x, w0, y, f, g, gx, gw, w = _placed(k, bf(S, H), bf(V, H), ids(), new(256, dtype=U8), new(S), bf(S, H), new(V, H),
                                        new(256, dtype=U8))
    vpce.vpce_lmhead_backward(x, [w0], y, f, grad_rows=g, grad_hidden=gx, grad_weight_shards=[gw], workspace=w, **kw)


def _head_step(k, **kw):
    x, w0, y, lo, ro, g, gx, gw, w = _placed(k, bf(S, H), bf(V, H), ids(), new(), new(S), new(S), bf(S, H), new(V, H),
                                             new(256, dtype=U8))
    vpce.vpce_lmhead_forward_backward(x, [w0], y, loss_out=lo, row_loss_out=ro, grad_rows=g, grad_hidden=gx,
                                      grad_weight_shards=[gw], workspace=w, **kw)


CALLS = {_score: 9, _score_grad: 8, _lookup_dropout: 6, _lookup_dropout_grad: 6, _lookup: 5, _lookup_grad: 5,
         _loss: 6, _loss_grad: 4, _fused: 6, _static: 4, _head: 7, _head_grad: 8, _head_step: 9}


@pytest.fixture
def devices(monkeypatch):
    """The devices that calls make current."""
    seen = []

    @contextlib.contextmanager
    def device(index):
        seen.append(index)
        yield

    monkeypatch.setattr(torch.cuda, "device", device)
    return seen


@pytest.mark.parametrize("call,k", [(c, k) for c, n in CALLS.items() for k in range(n)],
                         ids=lambda v: getattr(v, "__name__", v))
def test_an_operand_on_another_device_is_refused(lib, devices, call, k):
    with pytest.raises(ValueError):
        call(k)
    assert lib.calls == []


def _everywhere(call, index, monkeypatch, **kw):
    """The call with every operand on one device."""
    monkeypatch.setitem(globals(), "_placed", lambda k, *operands: [o.as_subclass((Fake0, Fake1)[index])
                                                                    for o in operands])
    call(-1, **kw)


@pytest.mark.parametrize("call", CALLS, ids=lambda v: v.__name__)
def test_a_call_is_made_on_its_operands_device(lib, devices, monkeypatch, call):
    _everywhere(call, 0, monkeypatch)
    assert devices == [] and len(lib.calls) == 1      # current already
    _everywhere(call, 1, monkeypatch)
    assert devices == [1] and len(lib.calls) == 2


@pytest.mark.parametrize("call", CALLS, ids=lambda v: v.__name__)
def test_a_stream_of_another_device_is_refused(lib, devices, monkeypatch, call):
    stream = types.SimpleNamespace(device=torch.device("cuda", 0), cuda_stream=7)
    with pytest.raises(ValueError, match="stream"):
        _everywhere(call, 1, monkeypatch, stream=stream)
    assert lib.calls == []


def test_local_steps_of_the_process_group_run_on_their_operands_device(lib, devices):
    """The rank's kernels, called while another device is current."""
    be = distributed.CudaBackend()
    with pytest.raises(ValueError):
        be.partials([new(S, V)], None, new(S, dtype=I64, index=1), -100, new(256, dtype=U8))
    with pytest.raises(ValueError):
        be.combine(new(1, S, 2), new(S), V, ids(), -100, "mean", 1, new(256, dtype=U8, index=1))
    assert lib.calls == [] and devices == []


@pytest.mark.parametrize("call", CALLS, ids=lambda v: v.__name__)
@pytest.mark.parametrize("how", ["one word for all", "every second word"])
def test_targets_and_ids_are_consecutive_words(lib, monkeypatch, call, how):
    """The kernels read s words from the address on."""
    bad = new(1, dtype=I64).expand(S) if how == "one word for all" else new(2 * S, dtype=I64)[::2]
    monkeypatch.setitem(globals(), "ids", lambda: bad)
    with pytest.raises(ValueError):
        call(-1)
    assert lib.calls == []
