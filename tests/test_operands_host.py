"""What the Python forms ask of their operands before the library is called:
workspaces."""
import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

from _fake_cuda import fake, install

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
