"""The roots and quotients behind the e4m3 codes are correctly rounded: roots of
every fp32 value in their range, quotients of random and of neighbouring values
by scales of every exponent."""
import os
import subprocess

import pytest
import torch

pytestmark = pytest.mark.gpu
HERE = os.path.dirname(os.path.abspath(__file__))


def test_roots_and_quotients_are_correctly_rounded(tmp_path):
    if not torch.cuda.is_available():
        pytest.skip("needs a GPU")
    from vocab_sharded_lm_gb300 import _build

    program = str(tmp_path / "rounding_check")
    subprocess.run([_build._nvcc(), *_build.ARCH, *_build.NVCC_FLAGS, "-I", _build.CSRC,
                    os.path.join(HERE, "rounding_check.cu"), "-o", program], check=True, capture_output=True)
    roots, quotients, pairs, ulps, seen = map(int, subprocess.run([program], check=True, capture_output=True, text=True,
                                                                  timeout=120).stdout.split())
    assert seen > 100_000_000 and (roots, quotients, pairs) == (0, 0, 0)
    # by scales below 2^-95 the residual may be lost: then x inv is what is left, of
    # two roundings of 2^-24 each, and 2^-23 of a value is at most two of its ulps
    # (an ulp is 2^-24 of it or more) from the exact quotient, 2.5 from the rounded one
    assert ulps <= 2
