"""spec_logits_process against its definition in 64 bits, token by token on the host: chains and trees,
every rule alone and together, odd vocabularies and misaligned rows, in place, bad requests, and the
sequence of verifying processed rows."""

import math

import numpy as np
import pytest
import torch

import oracle
import oracle_pins as pins
import parity
from speculative_decoding_verification_82_gb300 import binding

pytestmark = pytest.mark.gpu
DT = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16}


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def case(seed, B, R, V, kind, dtype, Lmax, nb, mask, hot=40):
    """Random inputs on the host; tokens from a small set, so that they meet."""
    rng = np.random.default_rng(seed)
    few = rng.integers(0, V, hot)
    tok = lambda *s: np.where(rng.random(s) < 0.7, few[rng.integers(0, hot, s)], rng.integers(0, V, s)).astype(np.int32)  # noqa: E731
    c = dict(logits=torch.from_numpy(rng.standard_normal((B, R, V)) * 4).to(DT[dtype]), dtype=dtype)
    c["history"] = tok(B, Lmax) if Lmax else None
    if Lmax:
        c["history_len"] = rng.integers(0, Lmax + 1, B).astype(np.int32)
        c["prompt_len"] = (c["history_len"] * rng.random(B)).astype(np.int32)
        c["history"][rng.random((B, Lmax)) < 0.05] = -1
        c["history"][rng.random((B, Lmax)) < 0.02] = V + 3
    if kind == "chain":
        c["draft_tokens"] = tok(B, R - 1)
    if kind == "tree":
        c["node_tokens"] = tok(B, R)
        c["node_tokens"][:, 0] = -7  # ignored
        c["parents"] = np.stack([pins.random_tree(rng, R, 50)[0] for _ in range(B)]).astype(np.int32)
    c["repetition"] = (0.5 + rng.random(B) * 1.5).astype(np.float32)
    c["presence"] = (rng.standard_normal(B)).astype(np.float32)
    c["frequency"] = (rng.standard_normal(B)).astype(np.float32)
    if nb:
        c["bias_tokens"] = tok(B, nb)
        c["bias_tokens"][rng.random((B, nb)) < 0.1] = -1
        c["bias_values"] = (rng.standard_normal((B, nb)) * 5).astype(np.float32)
    if mask:
        w = rng.integers(0, 2**32, (B, R, (V + 31) // 32), dtype=np.uint64)
        w[rng.random((B, R)) < 0.3] = 2**32 - 1
        w[0, 0] = 0
        c["allowed"] = w.astype(np.uint32).view(np.int32)
    return c


def run(c, logits=None, out=None):
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    x = c["logits"].cuda() if logits is None else logits
    return binding.spec_logits_process(x, out=out, **dev)


def reference(c):
    """[B, R, V] float64: the rules of the definition; and how far a result may be off (steps in 32 bits)."""
    x = c["logits"].double().numpy().copy()
    off = np.zeros_like(x)
    B, R, V = x.shape
    for b in range(B):
        n = int(c["history_len"][b]) if c.get("history") is not None else 0
        p = int(c["prompt_len"][b]) if c.get("prompt_len") is not None and n else 0
        prompt, count = set(), {}
        for j in range(n):
            t = int(c["history"][b, j])
            if 0 <= t < V:
                if j < p:
                    prompt.add(t)
                else:
                    count[t] = count.get(t, 0) + 1
        bias = {}
        for i in range(c["bias_tokens"].shape[1] if c.get("bias_tokens") is not None else 0):
            t = int(c["bias_tokens"][b, i])
            if 0 <= t < V:
                bias.setdefault(t, []).append(float(c["bias_values"][b, i]))
        rep, pres, freq = (float(c[k][b]) if c.get(k) is not None else d for k, d in (("repetition", 1), ("presence", 0), ("frequency", 0)))
        for r in range(R):
            path = []
            if c.get("draft_tokens") is not None:
                path = [int(t) for t in c["draft_tokens"][b, :r]]
            elif c.get("parents") is not None:
                m = r
                while m > 0:
                    path.append(int(c["node_tokens"][b, m]))
                    m = int(c["parents"][b, m])
            cc = dict(count)
            for t in path:
                cc[t] = cc.get(t, 0) + 1
            for t in set(cc) | prompt | set(bias):
                v, k = x[b, r, t], cc.get(t, 0)
                big = abs(v)
                if k or t in prompt:
                    v = v / rep if v > 0 else v * rep
                    big = max(big, abs(v))
                if k:
                    big += abs(freq * k) + abs(pres)
                    v = v - (freq * k + pres)
                for q in bias.get(t, ()):
                    v, big = v + q, big + abs(q)
                x[b, r, t] = v
                # at most 5 + biases roundings of quantities up to `big`, each half a step
                off[b, r, t] = (5 + len(bias.get(t, ()))) * big * 2.0**-24
            if c.get("allowed") is not None:
                w = c["allowed"][b, r].view(np.uint32)
                ok = (w[np.arange(V) // 32] >> (np.arange(V) % 32).astype(np.uint32)) & 1
                x[b, r, ok == 0] = -np.inf
    return x, off


def check(c, got):
    want, off = reference(c)
    g = got.double().cpu().numpy()
    assert np.array_equal(np.isneginf(g), np.isneginf(want))
    fin = np.isfinite(want)
    half = torch.finfo(got.dtype).eps / 2
    tiny = float(torch.finfo(got.dtype).smallest_normal)
    tol = off + half * np.maximum(np.abs(want) + off, tiny)
    assert (np.abs(g - want)[fin] <= tol[fin]).all()
    same = fin & (off == 0)  # no rule touched them
    assert np.array_equal(g[same], c["logits"].double().numpy()[same])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("B,R,V,kind,Lmax,nb,mask", [
    (1, 1, 1, None, 3, 0, False),
    (1, 1, 5, None, 4, 2, True),
    (2, 6, 1000, "chain", 64, 5, True),
    (3, 6, 4099, "chain", 300, 0, False),
    (2, 13, 8191, "tree", 100, 7, True),
    (2, 61, 2050, "tree", 0, 0, False),
    (4, 3, 12345, "chain", 1, 300, False),
    (2, 4, 33000, "chain", 700, 16, True),
    (9, 2, 4096, None, 50, 0, True),
])
def test_against_the_definition(dtype, B, R, V, kind, Lmax, nb, mask):
    c = case(B * 100 + R + V, B, R, V, kind, dtype, Lmax, nb, mask)
    r = run(c)
    assert (r["err_flags"].cpu().numpy() == 0).all()
    check(c, r["logits"])


@pytest.mark.parametrize("rule", ["repetition", "presence", "frequency", "bias_tokens", "allowed"])
def test_each_rule_alone(rule):
    c = case(77, 2, 5, 3001, "tree", "f32", 90, 9, True)
    for k in ("repetition", "presence", "frequency", "bias_tokens", "allowed"):
        if k != rule:
            c[k] = None
    if rule != "bias_tokens":
        c["bias_values"] = None
    check(c, run(c)["logits"])


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
@pytest.mark.parametrize("shift_in,shift_out", [(0, 0), (1, 1), (1, 0), (3, 2)])
def test_misaligned_rows_and_in_place(dtype, shift_in, shift_out):
    """Buffers that start off a 16-byte boundary; the elements around the output stay; the in-place call
    gives the same bits."""
    c = case(shift_in * 7 + shift_out, 2, 5, 4111, "chain", dtype, 120, 6, True)
    n = c["logits"].numel()
    buf = torch.zeros(n + 16, dtype=DT[dtype], device="cuda")
    x = buf[shift_in : shift_in + n].view(c["logits"].shape)
    x.copy_(c["logits"])
    obuf = torch.full((n + 16,), 9.5, dtype=DT[dtype], device="cuda")
    o = obuf[shift_out : shift_out + n].view(x.shape)
    got = run(c, logits=x, out=dict(logits=o))["logits"]
    check(c, got)
    assert (obuf[:shift_out] == 9.5).all() and (obuf[shift_out + n :] == 9.5).all()
    run(c, logits=x, out=dict(logits=x))
    assert torch.equal(x, o)
    assert (buf[:shift_in] == 0).all() and (buf[shift_in + n :] == 0).all()


@pytest.mark.parametrize("dtype", ["f32", "bf16", "f16"])
def test_masked_and_nonfinite_logits(dtype):
    """NaN and infinities: -inf where the mask bans them, untouched where no rule applies, through the
    arithmetic where one does; a row whose mask allows nothing is all -inf."""
    V = 100
    x = torch.zeros((1, 2, V), dtype=DT[dtype])
    x[0, :, 0], x[0, :, 1], x[0, :, 2], x[0, :, 3] = math.nan, math.inf, -math.inf, torch.finfo(DT[dtype]).min
    x[0, :, 10], x[0, :, 11], x[0, :, 12] = math.nan, math.inf, -math.inf
    allowed = np.zeros((1, 2, 4), np.uint32)
    allowed[0, 0] = 2**32 - 1
    allowed[0, 0, 0] ^= 0b1111
    c = dict(logits=x, history=np.array([[10, 11, 12]], np.int32), history_len=np.array([3], np.int32),
             repetition=np.array([2.0], np.float32), frequency=np.array([0.5], np.float32), allowed=allowed.view(np.int32))
    g = run(c)["logits"].cpu()[0]
    assert torch.isneginf(g[1]).all()
    assert torch.isneginf(g[0, :4]).all()
    assert torch.isnan(g[0, 10]) and g[0, 11] == math.inf and g[0, 12] == -math.inf
    assert (g[0, 4:10] == 0).all() and (g[0, 13:] == 0).all()
    c["allowed"] = None
    g = run(c)["logits"].cpu()[0]
    assert torch.isnan(g[:, 0]).all() and (g[:, 1] == math.inf).all() and (g[:, 2] == -math.inf).all()
    assert (g[:, 3] == torch.finfo(DT[dtype]).min).all()


def test_bad_requests_come_out_unprocessed():
    c = case(5, 12, 6, 5000, "tree", "bf16", 30, 4, True)
    c["history_len"][0] = 31
    c["history_len"][1] = -1
    c["prompt_len"][2] = c["history_len"][2] + 1
    c["parents"][3, 4] = 4
    c["parents"][4, 0] = 0
    c["node_tokens"][5, 3] = 5000
    c["node_tokens"][6, 1] = -1
    c["repetition"][7] = 0.0
    c["repetition"][8] = math.inf
    c["presence"][9] = math.nan
    c["frequency"][10] = -math.inf
    want = [32, 32, 32, 8, 8, 1, 1, 128, 128, 128, 128, 0]
    x = c["logits"].cuda()
    for out in (None, dict(logits=x.clone())):
        r = run(c, logits=x if out is None else out["logits"], out=out)
        assert r["err_flags"].tolist() == want
        assert torch.equal(r["logits"][:11], x[:11])
        assert not torch.equal(r["logits"][11], x[11])


def test_largest_shapes():
    """SPEC_MAX_LOGITS_ROWS nodes in one deep path whose tokens all lie in one chunk, SPEC_MAX_BIASES entries
    of one token, and a history longer than a block's threads many times over."""
    R, V, nb, Lmax = binding.MAX_LOGITS_ROWS, 300, binding.MAX_BIASES, 20000
    rng = np.random.default_rng(9)
    c = dict(logits=torch.from_numpy(rng.standard_normal((1, R, V))).float(),
             history=rng.integers(0, V, (1, Lmax)).astype(np.int32), history_len=np.array([Lmax], np.int32),
             prompt_len=np.array([1000], np.int32), node_tokens=rng.integers(0, V, (1, R)).astype(np.int32),
             parents=np.arange(-1, R - 1, dtype=np.int32)[None], frequency=np.array([0.01], np.float32),
             repetition=np.array([1.2], np.float32), bias_tokens=np.full((1, nb), 7, np.int32),
             bias_values=rng.standard_normal((1, nb)).astype(np.float32))
    r = run(c)
    assert r["err_flags"].tolist() == [0]
    check(c, r["logits"])


def test_chain_equals_the_tree_that_is_a_chain_and_repeats():
    c = case(21, 3, 9, 128256, "chain", "f32", 2000, 20, True)
    a = run(c)["logits"]
    assert torch.equal(a, run(c)["logits"])
    t = dict(c, draft_tokens=None, node_tokens=np.concatenate([np.zeros((3, 1), np.int32), c["draft_tokens"]], 1),
             parents=np.tile(np.arange(-1, 8, dtype=np.int32), (3, 1)))
    assert torch.equal(a, run(t)["logits"])


def test_streams_and_graph():
    c = case(31, 2, 4, 9001, "chain", "bf16", 50, 3, True)
    dev = {k: torch.from_numpy(np.ascontiguousarray(v)).cuda() for k, v in c.items() if isinstance(v, np.ndarray)}
    x = c["logits"].cuda()
    out = dict(logits=torch.zeros_like(x), err_flags=torch.zeros(2, dtype=torch.int32, device="cuda"))
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        binding.spec_logits_process(x, out=out, **dev)
    side.synchronize()
    check(c, out["logits"])
    graph = torch.cuda.CUDAGraph()
    with torch.cuda.graph(graph):
        binding.spec_logits_process(x, out=out, **dev)
    for seed in (1, 2):
        d = case(31 + seed, 2, 4, 9001, "chain", "bf16", 50, 3, True)
        x.copy_(d["logits"])
        for k in dev:
            dev[k].copy_(torch.from_numpy(np.ascontiguousarray(d[k])))
        graph.replay()
        torch.cuda.synchronize()
        check(d, out["logits"])


def test_rows_beyond_32_bit_offsets():
    """Rows that start past 2^32 bytes and 2^31 elements."""
    B, R, V = 5, 7, 64 << 20
    x = torch.zeros((B, R, V), dtype=torch.bfloat16, device="cuda")
    h = torch.tensor([[b, V - 1 - b] for b in range(B)], dtype=torch.int32, device="cuda")
    n = torch.full((B,), 2, dtype=torch.int32, device="cuda")
    f = torch.full((B,), 1.5, device="cuda")
    binding.spec_logits_process(x, history=h, history_len=n, frequency=f, out=dict(logits=x))
    for b in range(B):
        assert (x[b, :, b] == -1.5).all() and (x[b, :, V - 1 - b] == -1.5).all()
    assert int((x != 0).sum()) == 2 * B * R


def test_verifying_processed_rows():
    """A greedy chain on processed rows accepts exactly the tokens that decoding one at a time under the same
    rules would produce."""
    B, K, V = 6, 5, 2003
    c = case(41, B, K + 1, V, "chain", "f32", 60, 8, True)
    dev_rows = run(c)["logits"]
    want, _ = reference(c)
    drafts = c["draft_tokens"].copy()
    for b in range(B):  # drafts that follow the processed argmax for b tokens; rows depend on the drafts before
        for k in range(min(b, K)):
            w, _ = reference(dict(c, draft_tokens=drafts))
            drafts[b, k] = int(w[b, k].argmax()) if np.isfinite(w[b, k].max()) else drafts[b, k]
    c["draft_tokens"] = drafts
    dev_rows = run(c)["logits"]
    want, _ = reference(c)
    g = binding.spec_verify_chain(dev_rows, None, parity.i32(drafts), None, None, 0.0)
    o = oracle.verify_chain("f32", dev_rows.cpu().numpy(), None, B, K, V, 0.0, drafts, None, None)
    assert np.array_equal(g["out_tokens"].cpu().numpy(), o["out_tokens"])
    na = g["num_accepted"].cpu().numpy()
    for b in range(1, B):
        assert na[b] >= min(b, K)
        tok = g["out_tokens"].cpu().numpy()[b]
        for k in range(na[b] + 1):
            assert tok[k] == int(want[b, k].argmax())
