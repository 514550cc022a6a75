"""spec_rope_kv_write's rotated queries and its inputs in one buffer: rows that share a byte with an input that other blocks read
are refused, rows between the inputs' are not."""

import itertools

import numpy as np
import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding


def test_rows_meet_as_sets_of_bytes():
    rows = lambda n, a, s, l: {a + i * s + j for i in range(n) for j in range(l)}  # noqa: E731
    for n, s, la, lb, b in itertools.product((0, 1, 2, 3), (6, 7), (1, 3, 6), (1, 2, 6), range(-25, 26)):
        assert binding._rows_meet(n, 100, s, la, 100 + b, s, lb, 1) == bool(rows(n, 100, s, la) & rows(n, 100 + b, s, lb)), (n, s, la, lb, b)
    for n, sa, sb, la, lb, b in itertools.product((0, 1, 2, 3), (4, 7), (5, 9), (1, 4), (2, 5), range(-30, 31)):
        if rows(n, 100, sa, la) & rows(n, 100 + b, sb, lb):
            assert binding._rows_meet(n, 100, sa, la, 100 + b, sb, lb, 1)
        if n == 1:
            assert binding._rows_meet(n, 100, sa, la, 100 + b, sb, lb, 1) == bool(rows(n, 100, sa, la) & rows(n, 100 + b, sb, lb))


@pytest.mark.gpu
def test_one_buffer():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    B, T, H, D, S = 2, 5, 3, 32, 12
    rng = np.random.default_rng(1)
    data = torch.from_numpy(rng.standard_normal((B, T, 4 * H, D))).to(torch.bfloat16).cuda()
    slots = torch.arange(B * T, dtype=torch.int32, device="cuda").view(B, T)
    w, _ = binding.rope_inv_freq(D, device="cuda")
    ctx = torch.tensor([3, 700], dtype=torch.int32, device="cuda")

    def call(buf, q, k, v, out):
        part = lambda i: buf[:, :, i : i + H]  # noqa: E731
        kc, vc = (torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda") for _ in range(2))
        r = binding.spec_rope_kv_write(part(k), part(v), kc, vc, slots, w, q=part(q), context_len=ctx, out=None if out is None else dict(q=part(out)))
        return r["q"].clone(), kc, vc

    want = call(data.clone(), 0, H, 2 * H, None)
    for out in (0, 3 * H):  # in place, and between an input's rows
        assert all(torch.equal(a, b) for a, b in zip(call(data.clone(), 0, H, 2 * H, out), want))
    for q, k, v, out in ((0, 0, H, 0), (0, H, 0, 0), (0, 1, 2 * H, 0), (0, H, 2 * H, H), (0, H, 2 * H, 2 * H), (0, H, 2 * H, 2 * H + 1), (0, H, 2 * H, 1)):
        with pytest.raises(ValueError, match="overlap"):
            call(data.clone(), q, k, v, out)
