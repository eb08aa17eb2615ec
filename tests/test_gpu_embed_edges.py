"""Edges of the scaled embedding with dropout on the GPU: ids of the padding
sentinel's value, and gradients whose rows share memory."""
import numpy as np
import pytest
import torch

from vocab_sharded_lm_gb300 import vpce

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _built():
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    _build.build()
    vpce.load_library()


@pytest.mark.parametrize("padding_id,bad", [(None, True), (3, True), (-(1 << 63) + 1, False)])
def test_an_id_of_the_sentinels_value_is_out_of_range(padding_id, bad):
    """Without padding (INT64_MIN in the C call) no id is padding."""
    table = torch.arange(1.0, 81.0, device="cuda").view(10, 8)
    low = -(1 << 63) + (0 if bad else 1)
    ids = torch.tensor([2, low, 3, 9], dtype=torch.int64, device="cuda")
    flag = torch.full((1,), 9, dtype=torch.int32, device="cuda")
    out = vpce.vpce_embedding_dropout_forward([table], ids, padding_id=padding_id, flag=flag)
    assert flag.item() == (vpce.VPCE_FLAG_BAD_TARGET if bad else 0)
    want = torch.stack([table[2], torch.zeros(8, device="cuda"),
                        torch.zeros(8, device="cuda") if padding_id == 3 else table[3], table[9]])
    assert torch.equal(out, want)


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16])
def test_the_gradient_of_a_sum_over_rows(dtype):
    """It arrives with row stride 0 and gives what its dense copy gives, bit
    for bit (with dropout: the mask differs from row to row)."""
    s, h, V = 300, 40, 50
    x = torch.zeros(s, h, dtype=dtype, device="cuda", requires_grad=True)
    seen = []
    x.register_hook(seen.append)
    (x.sum(0) * torch.linspace(-1, 2, h, device="cuda").to(dtype)).sum().backward()
    grad = seen[0]
    assert grad.stride() == (0, 1)
    ids = torch.from_numpy(np.random.default_rng(1).integers(0, V, s)).cuda()
    rng = torch.tensor([3, 4], dtype=torch.int64, device="cuda")

    def tables():
        return [torch.ones(20, h, device="cuda"), torch.ones(V - 20, h, device="cuda")]

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    for stream in (None, side):
        a = vpce.vpce_embedding_dropout_backward(grad, ids, tables(), p=0.3, rng=rng, stream=stream)
        b = vpce.vpce_embedding_dropout_backward(grad.contiguous(), ids, tables(), p=0.3, rng=rng)
        torch.cuda.synchronize()
        assert all(torch.equal(p, q) for p, q in zip(a, b))
        # the plain lookup's adjoint adds in any order: counts times the row
        c = vpce.vpce_embedding_backward(grad, ids, tables(), stream=stream)
        torch.cuda.synchronize()
        count = torch.bincount(ids, minlength=V).double()[:, None]
        want = 1 + count * grad[0].double()
        got = torch.cat(c).double()
        assert bool(((got - want).abs() <= (count + 3) * 2.0 ** -24 * (1 + count * grad[0].double().abs())).all())
