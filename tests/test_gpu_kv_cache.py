"""spec_kv_write and spec_kv_read against their definition in 64 bits: codes and power-of-two scales bit for
bit, rows of every head size and type, padding and bad slots, strided inputs, streams and graphs."""

import numpy as np
import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def e4m3_values():
    """The 127 finite non-negative values of e4m3 by code: subnormals m 2^-9, then (8 + m) 2^(e - 10)."""
    return np.array([(c & 7) * 2.0**-9 if c < 8 else (8 + (c & 7)) * 2.0 ** ((c >> 3) - 10) for c in range(127)])


def ref_quantise(x: np.ndarray):
    """Codes (uint8) and scales (float64) of rows x [..., D] in 64 bits: the nearest e4m3 value, ties to the
    even code."""
    x = x.astype(np.float64)
    fin = np.where(np.isfinite(x), np.abs(x), 0.0)
    a = fin.max(-1)
    scale = np.full(a.shape, 2.0**-126)
    for _ in range(260):  # doubles until the row fits
        scale = np.where(a > 448 * scale, 2 * scale, scale)
    table = e4m3_values()
    y = np.where(np.isfinite(x), np.abs(x) / scale[..., None], 0.0)
    hi = np.clip(np.searchsorted(table, y), 1, 126)
    lo = hi - 1
    dl, dh = y - table[lo], table[hi] - y
    code = np.where((dl < dh) | ((dl == dh) & (lo % 2 == 0)), lo, hi).astype(np.uint8)
    code = np.where(np.isfinite(x), code, 0x7F).astype(np.uint8)
    return code | (np.signbit(x).astype(np.uint8) << 7), scale


def same_codes(got: np.ndarray, want: np.ndarray):
    """Codes equal; of NaN only that it is NaN."""
    nan = (want & 0x7F) == 0x7F
    return np.array_equal(got[~nan], want[~nan]) and bool(((got[nan] & 0x7F) == 0x7F).all())


def rows(rng, shape, dtype):
    x = rng.standard_normal(shape) * np.exp2(rng.integers(-14, 8, shape[:-1] + (1,)))
    return torch.from_numpy(x).to(dtype).cuda()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
@pytest.mark.parametrize("B,T,H,D", [(1, 1, 1, 8), (3, 1, 8, 128), (2, 61, 2, 64), (5, 7, 3, 80), (1, 300, 1, 256),
                                     (4, 33, 4, 96), (2, 3, 5, 24), (70, 1, 1, 136)])
def test_quantised_write_and_read(dtype, B, T, H, D):
    rng = np.random.default_rng(B * 1000 + T + D)
    k, v = rows(rng, (B, T, H, D), dtype), rows(rng, (B, T, H, D), dtype)
    S = B * T + 9
    slots = rng.permutation(S)[: B * T].reshape(B, T).astype(np.int32)
    skip = rng.random((B, T)) < 0.1
    slots = np.where(skip, -1, slots).astype(np.int32)
    fill = 0x5A  # every place that no token goes to keeps it
    kc = torch.full((S, H, D), fill, dtype=torch.uint8, device="cuda").view(E4M3)
    vc = torch.full((S, H, D), fill, dtype=torch.uint8, device="cuda").view(E4M3)
    ks, vs = torch.full((S, H), -3.0, device="cuda"), torch.full((S, H), -3.0, device="cuda")
    ds = torch.from_numpy(slots).cuda()
    err = binding.spec_kv_write(k, v, kc, vc, ds, k_scale=ks, v_scale=vs)
    outs = {t: binding.spec_kv_read(kc, vc, ds, t, k_scale=ks, v_scale=vs) for t in (torch.float32, torch.bfloat16, torch.float16)}
    assert (err.cpu().numpy() == 0).all()
    for x, cache, sc, name in ((k, kc, ks, "k"), (v, vc, vs, "v")):
        code, scale = ref_quantise(x.double().cpu().numpy())
        want = np.full((S, H, D), fill, np.uint8)
        wants = np.full((S, H), -3.0)
        want[slots[~skip]] = code[~skip]
        wants[slots[~skip]] = scale[~skip]
        assert same_codes(cache.view(torch.uint8).cpu().numpy(), want)
        assert np.array_equal(sc.double().cpu().numpy(), wants)
        val = np.where(code & 0x80, -1.0, 1.0) * e4m3_values()[np.minimum(code & 0x7F, 126)] * scale[..., None]
        val[skip] = 0.0
        for t, o in outs.items():  # one rounding, to nearest even
            assert torch.equal(o[name].cpu(), torch.from_numpy(val).to(torch.float32).to(t)), (name, t)
            assert (o["err_flags"].cpu() == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_16_and_32_bit_caches_take_the_bits(dtype):
    rng = np.random.default_rng(4)
    B, T, H, D, S = 3, 5, 2, 72, 40
    words = torch.int32 if dtype == torch.float32 else torch.int16
    lim = 2**31 - 1 if dtype == torch.float32 else 2**15 - 1
    k, v = (torch.from_numpy(rng.integers(-lim, lim, (B, T, H, D))).to(words).cuda().view(dtype) for _ in range(2))
    slots = torch.from_numpy(rng.permutation(S)[: B * T].reshape(B, T).astype(np.int32)).cuda()
    slots[1, 2] = -1
    kc, vc = torch.zeros((S, H, D), dtype=dtype, device="cuda"), torch.zeros((S // 8, 8, H, D), dtype=dtype, device="cuda")
    vc3 = vc.view(S, H, D)
    assert (binding.spec_kv_write(k, v, kc, vc3, slots) == 0).all()
    r = binding.spec_kv_read(kc, vc3, slots, dtype)
    for x, o in ((k, r["k"]), (v, r["v"])):
        want = x.clone()
        want[1, 2] = 0
        assert torch.equal(o.view(words), want.view(words))
    used = set(slots.cpu().numpy().ravel().tolist()) - {-1}
    for s in set(range(S)) - used:
        assert (kc[s] == 0).all() and (vc3[s] == 0).all()


@pytest.mark.parametrize("dtype", [torch.float32, torch.bfloat16, torch.float16])
def test_values_at_the_borders(dtype):
    """All-zero rows, the largest and smallest magnitudes, maxima at 448 times a power of two and next to
    it, ties between codes, signed zeros, NaN and infinities among finite elements and alone."""
    big = float(torch.finfo(dtype).max)
    tiny = float(torch.finfo(dtype).smallest_normal)
    r = [[0.0] * 8, [-0.0] * 8, [big] + [1.0] * 7, [tiny] * 8, [tiny / 4, tiny, 0, 0, 0, 0, 0, -tiny / 2],
         [448.0, 17, 18, 19, 20, 21, 0.001, -448], [450.0, 1, 2, 3, 4, 5, 6, 7], [7.0, 0.4375, 0.46875, -0.40625, 0, 1, 2, 3],
         [float("inf"), 1, -2, 3, float("nan"), 5, -6, float("-inf")], [float("nan")] * 8, [float("inf")] * 8,
         [448.0, 2**-9, 2**-10, 3 * 2**-10, 2**-11, -(2**-10), 5 * 2**-10, 0]]
    x = torch.tensor(r, dtype=torch.float64).to(dtype).cuda().view(len(r), 1, 1, 8)
    n = len(r)
    kc, vc = torch.zeros((n, 1, 8), dtype=torch.uint8, device="cuda").view(E4M3), torch.zeros((n, 1, 8), dtype=torch.uint8, device="cuda").view(E4M3)
    ks, vs = torch.zeros((n, 1), device="cuda"), torch.zeros((n, 1), device="cuda")
    slots = torch.arange(n, dtype=torch.int32, device="cuda").view(n, 1)
    binding.spec_kv_write(x, -x, kc, vc, slots, k_scale=ks, v_scale=vs)
    for y, c, s in ((x, kc, ks), (-x, vc, vs)):
        code, scale = ref_quantise(y.double().cpu().numpy())
        assert same_codes(c.view(torch.uint8).cpu().numpy(), code.reshape(n, 1, 8))
        assert np.array_equal(s.double().cpu().numpy(), scale.reshape(n, 1))


def test_bad_slots_are_skipped_and_flagged():
    B, T, H, D, S = 4, 300, 2, 64, 1300
    rng = np.random.default_rng(8)
    k, v = rows(rng, (B, T, H, D), torch.bfloat16), rows(rng, (B, T, H, D), torch.bfloat16)
    slots = torch.from_numpy(rng.permutation(S)[: B * T].reshape(B, T).astype(np.int32)).cuda()
    slots[1, 299], slots[2, 0], slots[2, 5] = S, -2, 2**31 - 1
    kc, vc = torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda"), torch.zeros((S, H, D), dtype=torch.bfloat16, device="cuda")
    err = binding.spec_kv_write(k, v, kc, vc, slots)
    assert err.tolist() == [0, 64, 64, 0]
    r = binding.spec_kv_read(kc, vc, slots, torch.bfloat16)
    assert r["err_flags"].tolist() == [0, 64, 64, 0]
    for x, o in ((k, r["k"]), (v, r["v"])):
        want = x.clone()
        for b, t in ((1, 299), (2, 0), (2, 5)):
            want[b, t] = 0
        assert torch.equal(o, want)


def test_fused_projection_slices_streams_and_graphs():
    """K and V as slices of one projection [B][T][(Hq + 2 H) D], on a side stream, then captured and
    replayed with new inputs."""
    rng = np.random.default_rng(5)
    B, T, H, D, S = 2, 9, 2, 128, 64
    qkv = rows(rng, (B, T, 4 * H, D), torch.float16)
    k, v = qkv[:, :, 2 * H : 3 * H], qkv[:, :, 3 * H :]
    slots = torch.from_numpy(rng.permutation(S)[: B * T].reshape(B, T).astype(np.int32)).cuda()
    kc, vc = (torch.zeros((S, H, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = torch.zeros((S, H), device="cuda"), torch.zeros((S, H), device="cuda")
    out = {n: torch.zeros((B, T, H, D), dtype=torch.float16, device="cuda") for n in ("k", "v")}
    out["err_flags"] = torch.zeros(B, dtype=torch.int32, device="cuda")
    err = torch.zeros(B, dtype=torch.int32, device="cuda")

    def step():
        binding.spec_kv_write(k, v, kc, vc, slots, k_scale=ks, v_scale=vs, err_flags=err)
        binding.spec_kv_read(kc, vc, slots, torch.float16, k_scale=ks, v_scale=vs, out=out)

    def check():
        torch.cuda.synchronize()
        for x, c, s, o in ((k, kc, ks, out["k"]), (v, vc, vs, out["v"])):
            code, scale = ref_quantise(x.double().cpu().numpy())
            at = slots.long().cpu().numpy()
            assert same_codes(c.view(torch.uint8).cpu().numpy()[at], code)
            assert np.array_equal(s.double().cpu().numpy()[at], scale)
            val = np.where(code & 0x80, -1.0, 1.0) * e4m3_values()[np.minimum(code & 0x7F, 126)] * scale[..., None]
            assert torch.equal(o.cpu(), torch.from_numpy(val).to(torch.float16))

    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        step()
    side.synchronize()
    check()
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        step()
    for _ in range(3):
        qkv.copy_(rows(rng, (B, T, 4 * H, D), torch.float16))
        graph.replay()
        check()


def test_slots_beyond_32_bit_offsets():
    """The last slots of caches whose element offsets pass 2^32."""
    H, D = 8, 256
    S = 2**32 // (H * D) + 40
    kc = torch.empty((S, H, D), dtype=torch.uint8, device="cuda").view(E4M3)
    vc = torch.empty((S, H, D), dtype=torch.uint8, device="cuda").view(E4M3)
    ks, vs = torch.empty((S, H), device="cuda"), torch.empty((S, H), device="cuda")
    rng = np.random.default_rng(6)
    k, v = rows(rng, (1, 6, H, D), torch.bfloat16), rows(rng, (1, 6, H, D), torch.bfloat16)
    slots = torch.tensor([[S - 1, 0, S - 2, 2**31 // (H * D), S - 17, 2**31 // (H * D) - 1]], dtype=torch.int32, device="cuda")
    assert binding.spec_kv_write(k, v, kc, vc, slots, k_scale=ks, v_scale=vs).tolist() == [0]
    r = binding.spec_kv_read(kc, vc, slots, torch.float32, k_scale=ks, v_scale=vs)
    for x, o in ((k, r["k"]), (v, r["v"])):
        code, scale = ref_quantise(x.double().cpu().numpy())
        val = np.where(code & 0x80, -1.0, 1.0) * e4m3_values()[np.minimum(code & 0x7F, 126)] * scale[..., None]
        assert np.array_equal(o.double().cpu().numpy(), val)


def test_empty_calls():
    kc = torch.zeros((4, 2, 64), dtype=torch.bfloat16, device="cuda")
    for B, T in ((0, 3), (2, 0)):
        k = torch.zeros((B, T, 2, 64), dtype=torch.bfloat16, device="cuda")
        slots = torch.zeros((B, T), dtype=torch.int32, device="cuda")
        assert binding.spec_kv_write(k, k, kc, kc.clone(), slots).tolist() == [0] * B
        assert binding.spec_kv_read(kc, kc, slots, torch.bfloat16)["k"].shape == (B, T, 2, 64)
