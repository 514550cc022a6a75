"""The cases of test_gpu_attention once more, under a check that a NaN cannot pass: there an output counts as bad when
its distance from the reference is above a bound, which is false for a NaN.  Here every output has to be a number
where the definition gives one, and every call hands in `lse`, whose values are held to the definition too."""

import pytest
import torch

import test_gpu_attention as base
from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu
bounds, call = base.check, base.call


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def call_with_lse(c, **kw):
    kw.setdefault("lse", torch.full(c["q"].shape[:3], 7.0, device="cuda"))
    return call(c, **kw)


def check(c, r, rows=None, scale=None):
    bounds(c, r, rows, scale)
    B, T = c["q"].shape[:2]
    for b in range(B):
        n = int(c["chunk_len"][b]) if c.get("chunk_len") is not None else T
        if n == 0:
            continue
        out, _, lse, _ = base.reference(c, b, scale)
        keep = list(range(n)) if rows is None else [t for t in rows[b] if t < n]
        assert torch.isfinite(out).all() and torch.isfinite(lse).all()
        assert torch.isfinite(r["out"][b, keep]).all()
        if r.get("lse") is not None:
            assert torch.isfinite(r["lse"][b, keep]).all()


@pytest.fixture(autouse=True)
def _strict(monkeypatch):
    monkeypatch.setattr(base, "check", check)
    monkeypatch.setattr(base, "call", call_with_lse)


@pytest.mark.parametrize("kind", ["bf16", "f16", "bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("shape", base.SHAPES, ids=lambda s: "-".join(map(str, s[:5])))
def test_against_the_definition(shape, kind):
    base.test_against_the_definition(shape, kind)


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("log2", [127, 126, -126])
def test_scales_at_the_ends_of_their_range(T, log2):
    base.test_scales_at_the_ends_of_their_range(T, log2)


@pytest.mark.parametrize("T,G", [(2, 4), (40, 8)])
def test_values_near_the_ends_of_their_range(T, G):
    base.test_values_near_the_ends_of_their_range(T, G)


@pytest.mark.parametrize("T,G,tree", [(6, 8, False), (61, 4, True), (300, 2, False)])
def test_ragged_chunks(T, G, tree):
    base.test_ragged_chunks_leave_the_rows_behind_them(T, G, tree)


def test_large_and_flat_scores():
    base.test_large_and_flat_scores()


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("dtype", [torch.bfloat16, torch.float16])
def test_large_and_flat_scores_over_codes(dtype, D):
    c = base.make(12, 2, 6, 2, 4, D, [400, 31], 16, dtype, True)
    for factor in (64, 0):
        c["q"].mul_(factor)
        check(c, call_with_lse(c))
    c = base.make(13, 2, 6, 2, 4, D, [400, 31], 16, dtype, True)
    check(c, call_with_lse(c, scale=0.3), scale=0.3)


def test_strided_queries_and_shared_pages():
    base.test_strided_queries_and_shared_pages()


def test_streams_graphs_and_two_workspaces():
    base.test_streams_graphs_and_two_workspaces()


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_beyond_32_bit_offsets(e4m3):
    base.test_pages_beyond_32_bit_offsets(e4m3)


def test_the_verification_step_end_to_end():
    base.test_the_verification_step_end_to_end()
