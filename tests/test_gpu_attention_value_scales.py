"""spec_attention over e4m3 caches whose V scales lie as far apart, in one request, as the header allows: the sum of the
weights, which is kept in units of those scales, loses nothing.

A partial sum joins the others by a factor of 2^(m - M), zero below 2^-126.  m is at least its largest score plus V exponent
less 15, M at most theirs less 7: with V exponents 80 apart what is lost weighs at most 2^-38 of the rest a position, nothing
beside the bounds' 2^-13 up to 2^25 positions."""

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


@pytest.mark.parametrize("low,high", [(-60, 20), (20, 100)])
@pytest.mark.parametrize("order", ["low first", "high first", "by turns", "mixed"])
@pytest.mark.parametrize("T,G,tree,D", [(1, 8, False, 128), (6, 8, False, 64), (61, 2, True, 128), (300, 1, False, 128)])
def test_value_scales_at_both_ends(T, G, tree, D, order, low, high):
    lens = [700, 90, 33]
    c = base.make(70 + T, len(lens), T, 2, G, D, lens, 32, e4m3=True, tree=tree)
    scale = c["v_scale"].view(-1, 2)
    for b, n in enumerate(lens):
        at = torch.arange(n + T, device="cuda")
        high = {"low first": at >= n // 2, "high first": at < n // 2, "by turns": at // 32 % 2 == 0, "mixed": at % 2 == 0}[order]
        slot = c["page_table"][b].long()[at // 32] * 32 + at % 32
        scale[slot] = torch.where(high, 2.0**high, 2.0**low).float()[:, None]
    lse = torch.full(c["q"].shape[:3], 7.0, device="cuda")
    r = base.call(c, lse=lse)
    assert torch.isfinite(r["out"]).all() and torch.isfinite(lse).all()
    base.check(c, r)
