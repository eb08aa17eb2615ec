"""What the Python forms make of tensors whose rows share memory.  The C
entries read a row stride of 0 as "dense", so an expanded tensor must be read
through a dense copy (gradients, which autograd expands) or refused (logits,
tables and whatever is written)."""
import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

from _fake_cuda import fake, floats_at, install

S, H, V = 4, 16, 24
F32, BF16, I64 = torch.float32, torch.bfloat16, torch.int64


@pytest.fixture
def lib(monkeypatch):
    return install(monkeypatch, vpce)


def new(*shape, dtype=F32):
    return fake(torch.zeros(shape, dtype=dtype))


def shared(rows, cols, dtype=F32):
    """[rows, cols] over the memory of one row."""
    x = fake(torch.zeros(1, cols, dtype=dtype)).expand(rows, cols)
    assert x.stride() == (0, 1)
    return x


def ids():
    return new(S, dtype=I64)


def ws(n=256):
    return new(n, dtype=torch.uint8)


def scores_out():
    return dict(logp_out=new(S), entropy_out=new(S), stats_out=new(S, 4))


REFUSED = {
    "score logits": lambda: vpce.vpce_logprob_forward([new(S, V), shared(S, V)], ids(), **scores_out()),
    "score gradient's logits": lambda: vpce.vpce_logprob_backward(
        [shared(S, V)], ids(), new(S, 4), grad_logp=new(S), grad_shards=[new(S, V)]),
    "score gradient": lambda: vpce.vpce_logprob_backward(
        [new(S, V)], ids(), new(S, 4), grad_logp=new(S), grad_shards=[shared(S, V)]),
    "dropout table": lambda: vpce.vpce_embedding_dropout_forward([shared(V, H)], ids(), out=new(S, H)),
    "dropout out": lambda: vpce.vpce_embedding_dropout_forward([new(V, H)], ids(), out=shared(S, H)),
    "dropout gradient table": lambda: vpce.vpce_embedding_dropout_backward(
        new(S, H), ids(), [new(V, H), shared(V, H)], workspace=ws()),
    "loss logits": lambda: vpce.vpce_forward([shared(S, V)], ids(), loss_out=new(), workspace=ws()),
    "loss gradient": lambda: vpce.vpce_backward([shared(S, V)], ids(), ws()),
    "fused loss": lambda: vpce.vpce_forward_backward([shared(S, V)], ids(), loss_out=new(), workspace=ws()),
    "static loss": lambda: vpce.vpce_forward_static([shared(S, V)], ids(), new()),
    "head hidden": lambda: vpce.vpce_lmhead_forward(
        shared(S, H, BF16), [new(V, H, dtype=BF16)], ids(), loss_out=new(), workspace=ws()),
    "head weight": lambda: vpce.vpce_lmhead_forward(
        new(S, H, dtype=BF16), [shared(V, H, BF16)], ids(), loss_out=new(), workspace=ws()),
    "head gradient's hidden": lambda: vpce.vpce_lmhead_backward(
        shared(S, H, BF16), [new(V, H, dtype=BF16)], ids(), ws(), grad_hidden=new(S, H, dtype=BF16),
        grad_weight_shards=[new(V, H)], workspace=ws()),
    "head hidden gradient": lambda: vpce.vpce_lmhead_backward(
        new(S, H, dtype=BF16), [new(V, H, dtype=BF16)], ids(), ws(), grad_hidden=shared(S, H, BF16),
        grad_weight_shards=[new(V, H)], workspace=ws()),
    "head weight gradient": lambda: vpce.vpce_lmhead_forward_backward(
        new(S, H, dtype=BF16), [new(V, H, dtype=BF16)], ids(), loss_out=new(), grad_hidden=new(S, H, dtype=BF16),
        grad_weight_shards=[shared(V, H)], workspace=ws()),
    "head weight gradients of two strides": lambda: vpce.vpce_lmhead_backward(
        new(S, H, dtype=BF16), [new(V, H, dtype=BF16)] * 2, ids(), ws(), grad_hidden=new(S, H, dtype=BF16),
        grad_weight_shards=[new(V, H), new(V, H + 8)[:, :H]], workspace=ws()),
    "lookup table": lambda: vpce.vpce_embedding_forward([shared(V, H)], ids(), out=new(S, H)),
    "lookup out": lambda: vpce.vpce_embedding_forward([new(V, H)], ids(), out=shared(S, H)),
    "lookup gradient table": lambda: vpce.vpce_embedding_backward(new(S, H), ids(), [shared(V, H)], workspace=ws()),
}


@pytest.mark.parametrize("name", REFUSED)
def test_shared_rows_are_refused(lib, name):
    with pytest.raises(ValueError, match="row stride"):
        REFUSED[name]()
    assert lib.calls == []


@pytest.mark.parametrize("call,entry", [
    (vpce.vpce_embedding_dropout_backward, "vpce_embedding_dropout_backward"),
    (vpce.vpce_embedding_backward, "vpce_embedding_backward"),
])
def test_an_expanded_gradient_is_read_as_its_rows(lib, call, entry):
    """The gradient of x.sum(0) reaches the call with strides (0, 1)."""
    x = torch.zeros(S, H, requires_grad=True)
    seen = []
    x.register_hook(seen.append)
    (x.sum(0) * torch.arange(1.0, H + 1)).sum().backward()
    grad = fake(seen[0])
    assert grad.stride() == (0, 1)
    read = []

    def look(name, args):
        ld = args[2] or H
        read.extend(floats_at(getattr(args[0], "value", args[0]), (S - 1) * ld + H)[r * ld:r * ld + H]
                    for r in range(S))

    lib.at_call = look
    call(grad, ids(), [new(V, H)], workspace=ws())
    assert [name for name, _ in lib.calls] == [entry]
    assert read == [[float(c + 1) for c in range(H)]] * S


def test_one_row_and_padded_rows_pass_as_before(lib):
    one = fake(torch.zeros(1, V)).expand(1, V)
    vpce.vpce_logprob_forward([one], new(1, dtype=I64), logp_out=new(1), entropy_out=new(1), stats_out=new(1, 4))
    vpce.vpce_logprob_forward([new(S, V + 3)[:, :V]], ids(), **scores_out())
    padded = new(S, H + 5)[:, :H]
    vpce.vpce_embedding_dropout_backward(padded, ids(), [new(V, H + 2)[:, :H]], workspace=ws())
    vpce.vpce_embedding_dropout_forward([new(1, H).expand(1, H)], ids(), out=padded)
    (_, a), (_, b), (_, c), (_, d) = lib.calls
    assert a[5] == 0 and b[5] == V + 3
    assert c[2] == H + 5 and c[0] == padded.data_ptr() and c[13] == H + 2
    assert d[5] == H and d[14] == H + 5
