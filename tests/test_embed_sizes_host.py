"""Row counts past 32 bits of the scaled embedding with dropout are refused on
the host.  Positions of the table gradient's sort and sum are 32-bit, and so
is the lookup's number of CTAs; 2^31 rows of one column fit the card."""
import pytest

from vocab_sharded_lm_gb300 import _build, vpce

FAKE = 0x7F0000000000  # a 256-byte aligned "device" address, never dereferenced on the host
MOST = (1 << 31) - 4096


@pytest.fixture(scope="module")
def lib():
    _build.build()
    return vpce.load_library()


def _gradient(lib, s, h):
    return lib.vpce_embedding_dropout_backward(FAKE, 1, 0, FAKE, s, -1, 1.0, 0.1, FAKE, vpce._ptr_array([FAKE]), 1,
                                               vpce._i64_array([0, 16]), h, 0, 0, FAKE, 1 << 60, None)


def _lookup(lib, s, h):
    return lib.vpce_embedding_dropout_forward(vpce._ptr_array([FAKE]), 1, 1, vpce._i64_array([0, 16]), h, 0, FAKE, s,
                                              -1, 1.0, 0.1, FAKE, FAKE, 1, 0, None, None)


def test_table_gradient(lib):
    nbytes = lib.vpce_embedding_dropout_backward_workspace_bytes
    for s in (MOST + 1, (1 << 31) - 64, 1 << 31):
        assert nbytes(s, 16, 1) == 0
        assert _gradient(lib, s, 1) == 1
    assert nbytes(MOST, 16, 1) > 0


def test_lookup(lib):
    for s, h in ((1 << 31, 8193), (1 << 31, (1 << 31) - 1), (1 << 20, (1 << 31) - 1)):
        assert _lookup(lib, s, h) == 1


def test_the_largest_sizes_pass_the_checks(lib):
    import torch

    if torch.cuda.is_available():
        pytest.skip("a GPU is present; this checks the host-only path")
    assert _gradient(lib, MOST, 1) == 5          # a CUDA error: past the checks
    assert _lookup(lib, 1 << 31, 1) == 5 and _lookup(lib, 1 << 21, 8193) == 5
