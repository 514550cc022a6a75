"""spec_logits_process in place against the call into another buffer, bit for bit: every token's rules are applied
once, wherever the token lies in the blocks' chunks of the vocabulary (1,024, 2,048 or 4,096 tokens, by the
number of rows and requests)."""

import numpy as np
import pytest
import torch

import test_gpu_logits as base
from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def at_the_borders(c, V, seed):
    """The case's history, biases and drafted tokens, all within 8 tokens of a multiple of 1,024 of a vocabulary of V."""
    rng = np.random.default_rng(seed)
    spots = np.arange(0, V, 1024)[:, None] + np.arange(-8, 8)
    spots = spots[(spots >= 0) & (spots < V)]
    for k in ("history", "bias_tokens", "draft_tokens", "node_tokens"):
        if c.get(k) is not None:
            c[k] = spots[rng.integers(0, len(spots), c[k].shape)].astype(np.int32)
    return c


@pytest.mark.parametrize("mask", [False, True])
@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,R,V,kind", [
    (3, 4, 8192, "chain"),      # chunks of 1,024
    (160, 3, 8192, "chain"),    # of 2,048
    (310, 2, 8192, "chain"),    # of 4,096
    (2, 61, 128256, "tree"),    # of 1,024
    (12, 6, 128256, "chain"),   # of 2,048
    (20, 61, 128256, "tree"),   # of 4,096, several times the blocks that fit at once
    (3, 5, 8191, "chain"),      # misaligned rows
])
def test_in_place_equals_out_of_place(B, R, V, kind, dtype, mask):
    c = at_the_borders(base.case(B + R, B, R, 50, kind, dtype, 300, 20, False), V, B)
    g = torch.Generator(device="cuda").manual_seed(R)  # the logits and masks of a full vocabulary: on the device
    x = torch.randn((B, R, V), generator=g, device="cuda").mul(4).to(base.DT[dtype])
    if mask:
        words = torch.randint(-(2**31), 2**31 - 1, (2, B, R, (V + 31) // 32), generator=g, device="cuda", dtype=torch.int32)
        c["allowed"] = (words[0] | words[1]).cpu().numpy()
    want = base.run(c, logits=x)["logits"]
    assert not torch.equal(want, x)
    for _ in range(3):
        y = x.clone()
        r = base.run(c, logits=y, out=dict(logits=y))
        assert r["logits"].data_ptr() == y.data_ptr() and int(r["err_flags"].abs().sum()) == 0
        assert torch.equal(y, want)


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_in_place_against_the_definition(dtype):
    """Also in numbers: a repetition penalty of 2 on a logit of 8 leaves 4, not 2."""
    c = at_the_borders(base.case(7, 3, 4, 8192, "chain", dtype, 300, 20, True), 8192, 8)
    x = c["logits"].cuda()
    base.check(c, base.run(c, logits=x, out=dict(logits=x))["logits"])
    V, step = 16384, 1024
    x = torch.full((2, 2, V), 8.0, dtype=base.DT[dtype], device="cuda")
    h = torch.arange(0, V, step, dtype=torch.int32, device="cuda").repeat(2, 1)
    n = torch.full((2,), h.shape[1], dtype=torch.int32, device="cuda")
    r = binding.spec_logits_process(x, history=h, history_len=n, prompt_len=n, repetition=torch.full((2,), 2.0, device="cuda"),
                                    out=dict(logits=x))["logits"]
    assert (r[:, :, ::step] == 4).all() and int((r != 8).sum()) == 4 * h.shape[1]
