"""spec_logits_process to the bits of its definition: every step in 32 bits, rounded to nearest, in the order the header
gives (numpy's float32 operations on the host), and one rounding to the type at the end."""

import numpy as np
import pytest
import torch

import test_gpu_logits as base
from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu
F = np.float32


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def path_tokens(c, b, r):
    if c.get("draft_tokens") is not None:
        return [int(t) for t in c["draft_tokens"][b, :r]]
    out, m = [], r if c.get("parents") is not None else 0
    while m > 0:
        out.append(int(c["node_tokens"][b, m]))
        m = int(c["parents"][b, m])
    return out


def stepwise(c):
    """The processed logits, and where a rule applied."""
    x = c["logits"].float().numpy().copy()
    touched = np.zeros(x.shape, bool)
    B, R, V = x.shape
    for b in range(B):
        n, p = (int(c["history_len"][b]), int(c["prompt_len"][b])) if c.get("history") is not None else (0, 0)
        h = [int(t) for t in c["history"][b, :n]] if n else []
        h = [(j, t) for j, t in enumerate(h) if 0 <= t < V]
        prompt = {t for j, t in h if j < p}
        bias = {}
        for i in range(c["bias_tokens"].shape[1] if c.get("bias_tokens") is not None else 0):
            t = int(c["bias_tokens"][b, i])
            if 0 <= t < V:
                bias[t] = F(bias.get(t, F(0)) + F(c["bias_values"][b, i]))
        rep, pres, freq = (F(c[k][b]) for k in ("repetition", "presence", "frequency"))
        for r in range(R):
            count = {}
            for t in [t for j, t in h if j >= p] + path_tokens(c, b, r):
                count[t] = count.get(t, 0) + 1
            for t in set(count) | prompt | set(bias):
                v, k = x[b, r, t], count.get(t, 0)
                if k or t in prompt:
                    v = F(v / rep) if v > 0 else F(v * rep)
                if k:
                    v = F(v - F(F(freq * F(k)) + pres))
                if t in bias:
                    v = F(v + bias[t])
                x[b, r, t], touched[b, r, t] = v, True
            if c.get("allowed") is not None:
                w = c["allowed"][b, r].view(np.uint32)
                x[b, r, ((w[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1) == 0] = -np.inf
    return torch.from_numpy(x).to(c["logits"].dtype), touched


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,R,V,kind,Lmax,nb,mask", [
    (1, 1, 7, None, 9, 5, False),
    (3, 6, 4099, "chain", 500, 40, False),
    (2, 6, 8192, "chain", 900, 200, True),
    (2, 33, 5000, "tree", 400, 60, False),
    (5, 9, 1024, "tree", 60, 10, True),
])
def test_bits_of_the_definition(B, R, V, kind, Lmax, nb, mask, dtype):
    c = base.case(900 + B + R, B, R, V, kind, dtype, Lmax, nb, mask, hot=60)
    want, touched = stepwise(c)
    got = base.run(c)["logits"].cpu()
    assert touched.any() and bool(torch.isfinite(want.float()).any())
    words = torch.int32 if dtype == "f32" else torch.int16
    assert torch.equal(got.view(words), want.view(words))
