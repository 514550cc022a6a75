"""spec_sample and spec_logits_filter on rows whose mask leaves nothing above the type's lowest value: those tokens weigh the
same, and tokens at -inf, places around the row and lanes without a token weigh nothing beside them."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding
from test_gpu_sample import DTYPES, check, cuda

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


# temperature, top-k as a part of V, top-p, min-p
RULES = [(1.0, 0, 1.0, 0.0), (0.5, 0, 0.9, 0.0), (8.0, 0, 0.37, 0.5), (1.0, 0.6, 1.0, 0.0), (1.0, 0.6, 0.7, 0.0), (2.0**-64, 0, 0.5, 0.0), (2.0**64, 0, 0.999, 0.0),
         (0.0, 0, 0.5, 0.0), (1.0, 0.01, 0.8, 1.0), (1.0, 0, 1.0, 1.0)]


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("V", [1, 7, 1000, 4097, 50001])
@pytest.mark.parametrize("shift", [0, 1])
@pytest.mark.parametrize("many", [1, 5])
def test_rows_at_the_lowest_value(dtype, V, shift, many):
    """Rows of it alone, of it and -inf (few and many), of it and the next value above; few rows stay in shared memory."""
    rng = np.random.default_rng(V)
    low = torch.finfo(dtype).min
    above = torch.tensor(low, dtype=dtype).view(torch.int32 if dtype == torch.float32 else torch.int16).sub(1).view(dtype).float().item()
    n = len(RULES)
    x = np.full((n, 4 * many, V), low)
    x[:, 1::4][rng.random((n, many, V)) < 0.5] = -np.inf
    x[:, 2::4][rng.random((n, many, V)) < 0.99] = -np.inf
    x[:, 3::4][rng.random((n, many, V)) < 0.5] = above
    x[:, :, V // 3] = low  # (one at least)
    T, k, p, m = (np.array([r[i] for r in RULES]) for i in range(4))
    k = np.where(k > 0, np.maximum(1, (k * V).astype(int)), 0)
    for part in (x[:, :2], x[:, 2:]) if many == 1 else (x,):  # (a few rows are at most 38)
        check(cuda(part, dtype), T, k, p, m, rng, shift=shift, in_place=shift == 1)


@pytest.mark.parametrize("dtype", DTYPES)
@pytest.mark.parametrize("rows", [1, 48])
def test_draws_next_to_one_stay_in_the_row(dtype, rows):
    """Every token weighs the same, so that a draw takes token floor(u V): V (1 - 2^-24) is above V - 1."""
    for V in (1, 26, 1000, 4097, 70001):
        x = torch.full((rows, 1, V), torch.finfo(dtype).min, dtype=dtype, device="cuda")
        for u in (0.0, 0.5, 0.99, 1 - 2.0**-24):
            us = torch.full((rows, 1), u, device="cuda")
            want = int(us[0, 0].double().item() * V)
            s = binding.spec_sample(x, us)
            assert (s["tokens"] == want).all() and (s["kept"] == V).all() and (s["err_flags"] == 0).all(), (V, u)
            assert ((s["probs"].double() * V - 1).abs() <= 2.0**-23).all()
