"""Host checks of limits that a value, not a size, breaks (placeholder device addresses: where no GPU is visible)."""

import ctypes
import math

import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding
from speculative_decoding_verification_82_gb300.build import build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device addresses: run without a GPU")
P = ctypes.c_void_p


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.library()


@host_only
def test_an_attention_scale_whose_factor_overflows(lib):
    """Scores are multiplied by scale log2(e): a scale of 3e38 is finite and the factor is not.  (With no tokens, a scale that
    passes returns before anything is looked up on a device.)"""

    def f(scale):
        return lib.spec_attention(P(1 << 20), 1, 1024, 2, 0, 8, 2, 128, P(2 << 20), P(3 << 20), 1, None, None, 10, 16, P(4 << 20), 4,
                                  P(5 << 20), None, None, scale, P(6 << 20), None, None, P(1 << 30), 1 << 40, None)

    largest = float(torch.finfo(torch.float32).max) * math.log(2)
    for scale in (2.0**-149, 1.0, largest * (1 - 2.0**-20)):
        assert f(scale) == binding.SPEC_OK, scale
    for scale in (largest * (1 + 2.0**-20), 3e38, math.inf, 0.0, -1.0, math.nan):
        assert f(scale) == binding.SPEC_ERR_INVALID_ARG, scale
