"""spec_kv_read from e4m3 caches whose scales are no powers of two (caches that something else wrote): each value is
code * s rounded to 32 bits, then to the type."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding
from test_gpu_kv_cache import E4M3, e4m3_values

pytestmark = pytest.mark.gpu


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


@pytest.mark.parametrize("D", [8, 128, 200])
def test_scales_of_any_value(D):
    rng = np.random.default_rng(D)
    S, H = 300, 3
    code = rng.integers(0, 256, (2, S, H, D)).astype(np.uint8)
    code[(code & 0x7F) == 0x7F] = 0
    scale = np.exp2(rng.uniform(-20, 4, (2, S, H))).astype(np.float32)
    # a product whose 32-bit rounding lies half-way between two bf16 values, and whose exact value does not
    scale[:, 0] = np.float32(2**23 + 2**15 + 1) / np.float32(2**23)
    kc, vc = (torch.from_numpy(x).cuda().view(E4M3) for x in code)
    ks, vs = (torch.from_numpy(x).cuda() for x in scale)
    slots = torch.from_numpy(rng.integers(0, S, (4, 90)).astype(np.int32)).cuda()
    slots[0, 0] = 0
    at = slots.cpu().numpy()
    for dtype in (torch.float32, torch.bfloat16, torch.float16):
        r = binding.spec_kv_read(kc, vc, slots, dtype, k_scale=ks, v_scale=vs)
        for c, s, o in ((code[0], scale[0], r["k"]), (code[1], scale[1], r["v"])):
            value = (np.where(c & 0x80, -1.0, 1.0) * e4m3_values()[np.minimum(c & 0x7F, 126)]).astype(np.float32) * s[..., None]
            assert value.dtype == np.float32
            assert torch.equal(o.cpu(), torch.from_numpy(value[at]).to(dtype))
