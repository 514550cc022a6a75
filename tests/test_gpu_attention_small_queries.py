"""spec_attention on queries that are small or zero, and on scores whose factors leave 32-bit floats' range, over 8- and
16-bit caches: hidden positions count for nothing whatever the size of the query, and no output is NaN where the
definition is finite."""

import math

import numpy as np
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


def check(c, scale=None):
    """The bounds of the definition's tests, and no NaN: those hold for a NaN (which compares false) too."""
    r = base.call(c, lse=torch.full(c["q"].shape[:3], 7.0, device="cuda"), **({} if scale is None else dict(scale=scale)))
    assert torch.isfinite(r["out"]).all() and torch.isfinite(r["lse"]).all()
    base.check(c, r, scale=scale)
    return r


def lens_for(T):
    """Context lengths whose last position lies in each quarter of a tile, and the shortest one."""
    return [128 * 3 + x - T % 128 for x in (10, 40, 70, 100, 128)] + [0]


@pytest.mark.parametrize("kind", ["bf16-e4m3", "f16-e4m3", "bf16", "f16"])
@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T,G,tree", [(1, 8, False), (6, 8, False), (61, 8, True), (61, 2, True), (300, 2, False)])
def test_small_and_zero_queries_among_usual_ones(T, G, tree, D, kind):
    lens = lens_for(T)
    dtype = torch.bfloat16 if kind.startswith("bf16") else torch.float16
    c = base.make(T + D, len(lens), T, 2, G, D, lens, 16, dtype, kind.endswith("e4m3"), tree)
    small = torch.tensor([0.0, 1.0, 2.0**-7, 2.0**-8, 2.0**-20, 2.0**-100, 2.0**-126, 1.0])
    pick = torch.from_numpy(np.random.default_rng(D + G).integers(0, len(small), c["q"].shape[:3]))
    c["q"] = (c["q"].double() * small[pick].double().cuda()[..., None]).to(dtype)
    check(c)
    c["q"].zero_()  # the mean of V
    r = check(c)
    n = c["context_len"][:, None].double() + (torch.arange(T, device="cuda") + 1 if not tree else torch.stack(
        [base.sees(T, 0, p.tolist()).sum(-1) for p in c["parents"]]))
    assert ((r["lse"].double() - torch.log(n)[..., None]).abs() <= 2.0**-13 * (1 + torch.log(n)[..., None])).all()


@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
@pytest.mark.parametrize("T", [2, 40])
def test_zero_keys_and_values_as_written(T, dtype):
    """All-zero K and V rows, which spec_kv_write gives the smallest scale there is, among usual ones: a whole cache,
    some pages and the chunk's last tokens."""
    lens = lens_for(T)
    B, H, D, page = len(lens), 2, 128, 16
    c = base.make(50, B, T, H, 4, D, lens, page, dtype, True)
    g = base.gen(51)
    pages = c["k_cache"].shape[0]
    for name in ("k", "v"):
        x = torch.randn((1, pages * page, H, D), generator=g, device="cuda").to(dtype)
        x.view(pages, page, H, D)[torch.rand((pages,), generator=g, device="cuda") < 0.3] = 0
        for b in range(B):
            at = torch.arange(lens[b] + T // 2, lens[b] + T, device="cuda") if b else torch.arange(lens[b] + T, device="cuda")
            x[0, c["page_table"][b].long()[at // page] * page + at % page] = 0
        c["x" + name] = x
    slots = torch.arange(pages * page, dtype=torch.int32, device="cuda")[None]
    binding.spec_kv_write(c["xk"], c["xv"], c["k_cache"], c["v_cache"], slots, k_scale=c["k_scale"], v_scale=c["v_scale"])
    check(c)
    c["q"] = c["q"] * 2.0**-9
    check(c)


@pytest.mark.parametrize("kind", ["f16-e4m3", "bf16-e4m3", "f16", "bf16"])
def test_the_smallest_scales(kind):
    """A caller's scale down to the smallest normal: scores vanish against 1, and nothing else changes."""
    dtype = torch.bfloat16 if kind.startswith("bf16") else torch.float16
    c = base.make(52, 3, 5, 2, 4, 64, [200, 37, 0], 16, dtype, kind.endswith("e4m3"))
    for scale in (2.0**-24, 1e-10, 2.0**-126):
        check(c, scale)
