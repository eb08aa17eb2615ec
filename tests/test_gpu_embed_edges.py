"""Edges of the scaled embedding with dropout on the GPU: ids of the padding
sentinel's value."""
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
