"""spec_attention over an e4m3 cache where a query's size times a K scale leaves 32-bit floats' range, and the scores do not:
the large parts of queries and keys do not meet."""

import pytest
import torch

import test_gpu_attention as base
from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G,tree", [(1, 8, False), (6, 8, False), (61, 4, True), (300, 1, False)])
def test_large_queries_orthogonal_to_large_keys(T, G, tree, D):
    """Keys of 2^120 in the first half of the elements; every second query of 2^120 in the other half (its scores are 0:
    the mean of V), the others of 2^-121 in the first (scores of a few units)."""
    c = base.make(60 + T, 3, T, 2, G, D, [300, 77, 0], 16, e4m3=True, tree=tree)
    unused = c["k_cache"].view(torch.uint8) == 0x7F
    codes = (torch.randn(c["k_cache"].shape, generator=base.gen(61), device="cuda") * 2.0**-1).to(base.E4M3)
    codes.view(torch.uint8)[..., D // 2 :] = 0
    c["k_cache"] = torch.where(unused, c["k_cache"].view(torch.uint8), codes.view(torch.uint8)).view(base.E4M3)
    c["k_scale"] = torch.exp2(torch.randint(118, 121, c["k_scale"].shape, generator=base.gen(62), device="cuda").float())
    q = torch.randn(c["q"].shape, generator=base.gen(63), device="cuda").double()
    first = torch.arange(D, device="cuda") < D // 2
    large = (torch.arange(2 * G, device="cuda") + torch.arange(T, device="cuda")[:, None]) % 2 == 0
    c["q"] = torch.where(large[..., None], q * ~first * 2.0**120, q * first * 2.0**-121).to(torch.bfloat16)
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda")
    r = base.call(c, lse=lse)
    assert r["err_flags"].tolist() == [0] * 3
    assert torch.isfinite(r["out"]).all() and torch.isfinite(lse).all()
    base.check(c, r)
