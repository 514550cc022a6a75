"""spec_rope_kv_write's cosines and sines themselves, by rotating (1, 0): right relative to their own size, however close to a
whole or a quarter turn the angle is.

Tolerance.  The turns a position are cut to units of 2^-64, and 2^96 / 2 pi is cut too: the angle is off by less than
2 2^-64 p turns.  What is left of the nearest quarter turn is rounded to 32 bits, 2^-24 of itself, and so is its sine or tangent, as it is
within an eighth of a turn (x / tan x and x / sin x are at most 1 and 1.12 there).  sincospif is off by 2 ulp, 4 2^-24 of the result at
most, the factor's product and the fused product and sum (1 c - 0 s, 0 c + 1 s) by 2^-24 each: (1.12 + 4 + 2) 2^-24 <= 8 2^-24
relative, and 2 pi 2 2^-64 p absolute."""

import math

import numpy as np
import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def check(w, pos, interleaved, factor):
    h, T = len(w), len(pos)
    D = (2 * h + 7) // 8 * 8
    first = torch.arange(h, device="cuda") * (2 if interleaved else 1)
    second = first + (1 if interleaved else h)
    k = torch.zeros((1, T, 1, D), device="cuda")
    k[..., first] = 1.0
    kc, vc = torch.zeros((T, 1, D), device="cuda"), torch.zeros((T, 1, D), device="cuda")
    slots = torch.arange(T, dtype=torch.int32, device="cuda")[None]
    r = binding.spec_rope_kv_write(k, k, kc, vc, slots, torch.from_numpy(w).cuda(), positions=torch.from_numpy(pos).cuda()[None], interleaved=interleaved,
                                   factor=factor)
    assert (r["err_flags"] == 0).all()
    angle = pos[:, None].astype(np.longdouble) * w.astype(np.longdouble)  # (31 and 24 bits: exact in 64)
    for got, f in ((kc[:, 0, first], np.cos), (kc[:, 0, second], np.sin)):
        want = factor * f(angle).astype(np.float64)
        err = abs(got.double().cpu().numpy() - want)
        tol = 8 * 2.0**-24 * abs(want) + abs(factor) * 4 * math.pi * 2.0**-64 * pos[:, None]
        bad = ~(err <= tol)
        assert not bad.any(), (bad.sum(), w[np.nonzero(bad)[1][0]], pos[np.nonzero(bad)[0][0]], (err / np.maximum(tol, 1e-300)).max())


@pytest.mark.parametrize("interleaved", [False, True])
@pytest.mark.parametrize("factor", [1.0, 1.25])
def test_small_angles(interleaved, factor):
    w = np.concatenate([np.exp(np.linspace(0.0, np.log(1e-9), 124)), [2.0**-20, 2.0**-32, 1.0, 0.5]]).astype(np.float32)
    pos = np.array([0, 1, 2, 3, 4, 7, 10, 31, 100, 1000, 4097, 100000, 2**20, 10**9, 2**31 - 1], np.int32)
    check(w, pos, interleaved, factor)


@pytest.mark.parametrize("n", [4, 5, 64])
def test_close_to_quarter_turns(n):
    """Angles whose p-th multiple lies within rounding of a number of quarter turns (at small positions, where they are right to far less)."""
    rng = np.random.default_rng(n)
    pos = np.arange(1, 257, dtype=np.int32)
    quarters = rng.integers(1, 9, n)
    at = rng.integers(1, 257, n)
    check((quarters * (math.pi / 2) / at).astype(np.float32), pos, False, 1.0)
