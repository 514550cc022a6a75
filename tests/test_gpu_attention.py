"""spec_attention against its definition in 64 bits: chains, trees and single tokens over paged caches of
16 and 8 bits, every grouping of heads, lengths around the tiles' borders, non-finite values in masked and
unwritten places, bad requests, streams and graphs, and the sequence around it (write, attend, process,
verify, compact, read)."""

import math

import numpy as np
import pytest
import torch

import oracle_pins as pins
from speculative_decoding_verification_82_gb300 import binding, synth

pytestmark = pytest.mark.gpu
E4M3 = torch.float8_e4m3fn


@pytest.fixture(scope="module", autouse=True)
def _cuda():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()


def gen(seed):
    g = torch.Generator(device="cuda")
    g.manual_seed(seed)
    return g


def make(seed, B, T, H, G, D, lens, page, dtype=torch.bfloat16, e4m3=False, tree=False, spare=3, sharp=1.5):
    """Inputs on the device; the places of the caches that no position uses hold NaN."""
    g = gen(seed)
    lens = (list(lens) * B)[:B]
    P = (max(lens) + T + page - 1) // page + 1
    pages = B * P + spare
    c = dict(q=torch.randn((B, T, H * G, D), generator=g, device="cuda").mul(sharp).to(dtype))
    table = torch.randperm(pages, generator=g, device="cuda")[: B * P].reshape(B, P).to(torch.int32)
    for name in ("k", "v"):
        x = torch.randn((pages, page, H, D), generator=g, device="cuda")
        if e4m3:
            s = torch.exp2(torch.randint(-7, 4, (pages, page, H), generator=g, device="cuda").float())
            x = (x * 100).clamp(-448, 448).to(E4M3)
            c[name + "_scale"] = s if name == "v" else s * 2.0**-8
        else:
            x = x.to(dtype)
        c[name + "_cache"] = x
    used = torch.zeros(pages * page, dtype=torch.bool, device="cuda")
    for b in range(B):
        at = torch.arange(lens[b] + T, device="cuda")
        used[(table[b].long()[at // page] * page + at % page)] = True
    for name in ("k", "v"):
        flat = c[name + "_cache"].view(-1, H, D)
        if e4m3:
            flat.view(torch.uint8)[~used] = 0x7F
        else:
            flat[~used] = math.nan
    c["page_table"], c["context_len"] = table, torch.tensor(lens, dtype=torch.int32, device="cuda")
    if tree:
        rng = np.random.default_rng(seed)
        par = np.stack([pins.random_tree(rng, T, 50)[0] for _ in range(B)]).astype(np.int32)
        c["parents"] = torch.from_numpy(par).cuda()
    return c


def call(c, **kw):
    return binding.spec_attention(c["q"], c["k_cache"], c["v_cache"], c["page_table"], c["context_len"],
                                  **{k: c[k] for k in ("parents", "chunk_len", "k_scale", "v_scale") if c.get(k) is not None}, **kw)


def sees(T, L, parents=None):
    """[T, L + T] truth values of one request."""
    s = torch.zeros((T, L + T), dtype=torch.bool)
    s[:, :L] = True
    for t in range(T):
        if parents is None:
            s[t, L : L + t + 1] = True
        else:
            m = t
            while m >= 0:
                s[t, L + m] = True
                m = int(parents[m])
    return s.cuda()


def reference(c, b, scale=None):
    """One request in 64 bits: out [T, Hq, D], the sum of weights times |v|, lse [T, Hq], and the plain sum over
    all positions of |v| (e4m3: of |code|, times the request's largest V scale) [Hq, D].  Masked values are taken out before the products, so that only attended
    ones count."""
    B, T, Hq, D = c["q"].shape
    page, H = c["k_cache"].shape[1:3]
    G = Hq // H
    L = int(c["context_len"][b])
    n = int(c["chunk_len"][b]) if c.get("chunk_len") is not None else T
    scale = D**-0.5 if scale is None else scale
    at = torch.arange(L + n, device="cuda")
    slot = c["page_table"][b].long()[at // page] * page + at % page
    kv = []
    for name in ("k", "v"):
        x = c[name + "_cache"].view(-1, H, D)
        if x.dtype == E4M3:
            x = x.view(torch.uint8)[slot].view(E4M3).double() * c[name + "_scale"].view(-1, H)[slot].double()[..., None]
        else:
            x = x[slot].double()
        kv.append(x)
    see = sees(n, L, c["parents"][b].tolist() if c.get("parents") is not None else None)
    q = c["q"][b, :n].double()
    out, mag = (torch.zeros((n, Hq, D), dtype=torch.float64, device="cuda") for _ in range(2))
    lse = torch.zeros((n, Hq), dtype=torch.float64, device="cuda")
    flat = torch.zeros((Hq, D), dtype=torch.float64, device="cuda")
    for h in range(H):
        hs = slice(h * G, (h + 1) * G)
        s = torch.einsum("tgd,nd->gtn", q[:, hs], kv[0][:, h]).mul(scale)
        s = torch.where(see, s, torch.full_like(s, -math.inf))
        lse[:, hs] = torch.logsumexp(s, -1).T
        p = torch.softmax(s, -1)
        v = kv[1][:, h]
        fin = torch.isfinite(v)
        w = torch.where(fin, v, torch.zeros_like(v)).abs()
        if c.get("v_scale") is not None:
            vs = c["v_scale"].view(-1, H)[slot][:, h].double()[:, None]
            w = w / vs * vs.max()
        flat[hs] = w.sum(0)
        out[:, hs] = torch.einsum("gtn,nd->tgd", p, torch.where(fin, v, torch.zeros_like(v)))
        mag[:, hs] = torch.einsum("gtn,nd->tgd", p, torch.where(fin, v, torch.zeros_like(v)).abs())
    return out, mag, lse, flat


def check(c, r, rows=None, scale=None):
    """Every output against the reference.  A weight and the result are each rounded to the type (half a step:
    u); everything else is in 32 bits, where the sums' and scores' errors stay below 2^-13 of the summed
    magnitudes at these sizes (at most 2^13 tokens in 16-token steps, scores below 2^7)."""
    dtype = c["q"].dtype
    u = torch.finfo(dtype).eps / 2
    B, T = c["q"].shape[:2]
    for b in range(B):
        n = int(c["chunk_len"][b]) if c.get("chunk_len") is not None else T
        if n == 0:
            continue
        out, mag, lse, flat = reference(c, b, scale)
        got = r["out"][b, :n].double()
        tol = u * (1 + u) * out.abs() + (u + 2.0**-13) * mag + float(torch.finfo(dtype).smallest_normal) * (u + 2.0**-13)
        if dtype == torch.float16 or c.get("v_scale") is not None:
            # Weights are f16 here (times the V scale of an e4m3 cache: w s), below its normals off by up to half
            # its smallest step, 2^-25, whatever their size.  They are in units of 2^(M - 7) S, M the row's
            # largest score and S at most twice the largest V scale (1 without scales), so the largest weight is
            # at least 2^7 / S and their sum too: dividing by it leaves at most 2^-25 S / 2^7 of the plain sum
            # of |v| (|code|): 2^-31 of `flat` (half of that without scales).
            tol = tol + 2.0**-31 * flat
        bad = (got - out).abs() > tol
        if rows is not None:
            keep = torch.zeros(n, dtype=torch.bool, device="cuda")
            keep[[t for t in rows[b] if t < n]] = True
            bad &= keep[:, None, None]
        assert not bad.any(), (b, bad.nonzero()[:3].tolist(), float(((got - out).abs() - tol).max()))
        if r.get("lse") is not None and rows is None:
            assert ((r["lse"][b, :n].double() - lse).abs() <= 2.0**-13 * (1 + lse.abs())).all()


SHAPES = [
    # B, T, H, G, D, lens, page, tree
    (1, 1, 1, 1, 64, [0], 8, False),
    (3, 1, 2, 1, 64, [1, 17, 0], 8, False),
    (8, 1, 8, 8, 128, [2052, 127, 128, 129, 1, 500, 1000, 255], 16, False),
    (5, 6, 2, 8, 128, [127, 122, 123, 250, 5], 16, False),
    (4, 6, 1, 7, 128, [1000, 0, 383, 384], 32, False),
    (3, 61, 2, 8, 128, [300, 66, 67], 64, True),
    (2, 61, 4, 4, 64, [1500, 0], 16, True),
    (2, 130, 1, 3, 128, [0, 200], 8, False),
    (2, 300, 2, 8, 128, [1000, 0], 128, False),
    (1, 1, 1, 16, 128, [8000], 256, False),
    (2, 5, 1, 64, 64, [700, 90], 32, False),
    (1, 3, 2, 130, 128, [513], 16, False),
    (2, 500, 1, 1, 64, [100, 37], 16, True),
    (40, 2, 3, 5, 64, [64, 63, 65, 0, 900], 16, False),
    (1, 257, 1, 2, 128, [4000], 1024, False),
]


@pytest.mark.parametrize("kind", ["bf16", "f16", "bf16-e4m3", "f16-e4m3"])
@pytest.mark.parametrize("shape", SHAPES, ids=lambda s: "-".join(map(str, s[:5])))
def test_against_the_definition(shape, kind):
    B, T, H, G, D, lens, page, tree = shape
    c = make(sum(map(ord, kind)) + B + T + G, B, T, H, G, D, lens, page, torch.bfloat16 if kind.startswith("bf16") else torch.float16,
             kind.endswith("e4m3"), tree)
    lse = torch.full((B, T, H * G), 7.0, device="cuda")
    r = call(c, lse=lse)
    assert r["err_flags"].tolist() == [0] * B
    check(c, r)
    assert torch.equal(r["out"], call(c)["out"])  # the same bits again


@pytest.mark.parametrize("T", [3, 40])
@pytest.mark.parametrize("log2", [127, 126, -126])
def test_scales_at_the_ends_of_their_range(T, log2):
    """K scales next to float's largest and smallest powers of two, against queries that bring the scores back to
    a few units.  (A score's factor, scale log2(e) 2^-126, may be subnormal: its 2^-21 of scores below 2^3 is
    within what check allows.)"""
    c = make(40, 2, T, 2, 8, 128, [300, 77], 16, e4m3=True)
    g = gen(41)
    codes = (torch.randn(c["k_cache"].shape, generator=g, device="cuda") * 2.0**-3).to(E4M3)
    unused = c["k_cache"].view(torch.uint8) == 0x7F
    c["k_cache"] = torch.where(unused, c["k_cache"].view(torch.uint8), codes.view(torch.uint8)).view(E4M3)
    first = log2 - 2 if log2 > 0 else log2
    c["k_scale"] = torch.exp2(torch.randint(first, first + 3, c["k_scale"].shape, generator=g, device="cuda").double()).float()
    c["q"] = (torch.randn(c["q"].shape, generator=g, device="cuda").double() * 2.0 ** min(3 - log2, 124)).to(torch.bfloat16)
    check(c, call(c))


@pytest.mark.parametrize("T,G", [(2, 4), (40, 8)])
def test_values_near_the_ends_of_their_range(T, G):
    """bf16 V of 2^80 and of 2^-100, with scores that rise along the prefix's tiles in either direction by less and
    by more than what is let pass without rescaling."""
    for power in (80, -100):
        for slope in (0.02, -0.02, 0.3, -0.3):
            c = make(44, 2, T, 1, G, 64, [900, 100], 16)
            c["v_cache"] = (c["v_cache"].double() * 2.0**power).to(torch.bfloat16)
            at = torch.arange(1000, device="cuda")
            for b in range(2):  # every query's first element is 1, the keys' grow along the positions
                n = int(c["context_len"][b])
                slot = c["page_table"][b].long()[at[:n] // 16] * 16 + at[:n] % 16
                c["k_cache"].view(-1, 1, 64)[slot, 0, 0] = (slope * at[:n]).to(torch.bfloat16)
            c["q"][..., 0] = 1.0
            check(c, call(c))


@pytest.mark.parametrize("D", [64, 128])
@pytest.mark.parametrize("T", [2, 40])
def test_scales_that_are_no_powers_of_two(T, D):
    """Such a scale, relative to the largest of its 32 positions, is rounded to f16, and so is its product with a
    code: a K or V element is off by d = (1 + 2^-11)^2 - 1 of itself.  Scores are then off by d sum |q k| scale at
    most, weights by the exponential of twice that."""
    c = make(42, 3, T, 2, 4, D, [500, 130, 3], 16, torch.float16, e4m3=True, sharp=0.02)
    for name in ("k_scale", "v_scale"):
        c[name] = c[name].clamp(2.0**-3, 1) * (1 + torch.rand(c[name].shape, generator=gen(43), device="cuda"))
    r = call(c, lse=torch.zeros((3, T, 8), device="cuda"))
    d = (1 + 2.0**-11) ** 2 - 1
    u = torch.finfo(torch.float16).eps / 2
    for b in range(3):
        out, mag, lse, flat = reference(c, b)
        k = (c["k_cache"].view(-1, 2, D).view(torch.uint8) & 0x7F).view(E4M3).double().nan_to_num(0) * c["k_scale"].view(-1, 2).double()[..., None]
        at = torch.arange(int(c["context_len"][b]) + T, device="cuda")
        k = k[c["page_table"][b].long()[at // 16] * 16 + at % 16]
        q = c["q"][b].double().abs().view(T, 2, 4, D)
        worst = torch.einsum("thgd,nhd->thgn", q, k).amax(-1).reshape(T, 8, 1) * D**-0.5 * d
        tol = u * (1 + u) * out.abs() + (u + 2.0**-13 + torch.expm1(2 * worst) + d * torch.exp(2 * worst)) * mag + 2.0**-31 * flat + 2.0**-25
        assert ((r["out"][b].double() - out).abs() <= tol).all()
        assert ((r["lse"][b].double() - lse).abs() <= worst[..., 0] + 2.0**-13 * (1 + lse.abs())).all()


@pytest.mark.parametrize("T,G,tree", [(6, 8, False), (61, 4, True), (300, 2, False)])
def test_ragged_chunks_leave_the_rows_behind_them(T, G, tree):
    B = 5
    c = make(3, B, T, 2, G, 128, [100, 0, 511, 30, 256], 16, tree=tree)
    c["chunk_len"] = torch.tensor([T, 1, 0, T // 2, T - 1], dtype=torch.int32, device="cuda")
    out = torch.full(c["q"].shape, 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full(c["q"].shape[:3], 6.0, device="cuda")
    r = call(c, out=dict(out=out), lse=lse)
    assert r["err_flags"].tolist() == [0] * B
    check(c, r)
    for b in range(B):
        n = int(c["chunk_len"][b])
        assert (out[b, n:] == 5.0).all() and (lse[b, n:] == 6.0).all()


@pytest.mark.parametrize("e4m3", [False, True])
def test_nonfinite_values_reach_only_who_attends_to_them(e4m3):
    """A NaN or infinity in the K or V row of one tree node: its descendants' outputs become non-finite,
    the other rows keep their bits; likewise a later token of a chain."""
    for tree in (True, False):
        T = 61
        clean = make(9, 2, T, 2, 4, 128, [70, 250], 16, e4m3=e4m3, tree=tree)
        r0 = call(clean)
        assert torch.isfinite(r0["out"]).all()
        for name, value in (("k", math.nan), ("v", math.nan), ("v", math.inf)):
            c = {k: v.clone() if isinstance(v, torch.Tensor) else v for k, v in clean.items()}
            node = 7
            for b in range(2):
                j = int(c["context_len"][b]) + node
                page = int(c["page_table"][b, j // 16])
                if e4m3:
                    c[name + "_cache"].view(torch.uint8)[page, j % 16, :, 5] = 0x7F
                else:
                    c[name + "_cache"][page, j % 16, :, 5] = value
            r = call(c)
            for b in range(2):
                see = sees(T, 0, c["parents"][b].tolist() if tree else None)[:, node]
                assert torch.equal(r["out"][b][~see], r0["out"][b][~see])
                assert (~torch.isfinite(r["out"][b][see])).any(-1).all()


def test_a_nonfinite_prefix_row_reaches_everyone_of_its_head():
    c = make(10, 2, 6, 2, 4, 64, [300, 40], 16)
    page = int(c["page_table"][0, 3])
    c["v_cache"][page, 2, 1, 9] = math.nan
    r = call(c)["out"]
    assert torch.isnan(r[0, :, 4:, 9]).all()
    assert torch.isfinite(r[0, :, :4]).all() and torch.isfinite(r[1]).all()


def test_nan_queries_stay_in_their_rows():
    c = make(11, 1, 40, 1, 8, 128, [200], 16)
    r0 = call(c)["out"]
    c["q"][0, 3, 2, 7] = math.nan
    r = call(c)["out"]
    assert torch.isnan(r[0, 3, 2]).all()
    r[0, 3, 2] = r0[0, 3, 2]
    assert torch.equal(r, r0)


def test_large_and_flat_scores():
    """Scores in the thousands (one weight takes all), equal scores (the mean of V), and a scale of one's own."""
    c = make(12, 2, 6, 2, 4, 128, [400, 31], 16)
    c["q"].mul_(64)
    check(c, call(c))
    c["q"].zero_()
    check(c, call(c))
    c = make(13, 2, 6, 2, 4, 64, [400, 31], 16)
    check(c, call(c, scale=0.3), scale=0.3)


def test_bad_requests():
    B, T = 9, 6
    c = make(14, B, T, 2, 4, 128, [100], 16, tree=True)
    P = c["page_table"].shape[1]
    c["chunk_len"] = torch.full((B,), T, dtype=torch.int32, device="cuda")
    c["context_len"][0] = -1
    c["context_len"][1] = P * 16 - T + 1
    c["chunk_len"][2] = T + 1
    c["chunk_len"][3] = -1
    c["parents"][4, 0] = 0
    c["parents"][5, 3] = 3
    c["page_table"][6, 2] = c["k_cache"].shape[0]
    c["page_table"][7, 0] = -5
    c["context_len"][8] = 2**31 - 1
    lse = torch.full((B, T, 8), 3.0, device="cuda")
    out = torch.full(c["q"].shape, 3.0, dtype=torch.bfloat16, device="cuda")
    r = call(c, lse=lse, out=dict(out=out))
    assert r["err_flags"].tolist() == [32, 32, 32, 32, 8, 8, 64, 64, 32]
    for b in (0, 1, 2, 3, 4, 5, 8):
        assert (out[b] == 0).all() and torch.isneginf(lse[b]).all()
    for b, page in ((6, 2), (7, 0)):  # the bad page's rows read as zeros
        d = dict(c)
        zero = c["k_cache"].shape[0] - 1
        d["k_cache"], d["v_cache"], d["page_table"] = c["k_cache"].clone(), c["v_cache"].clone(), c["page_table"].clone()
        d["k_cache"] = torch.cat([d["k_cache"], torch.zeros_like(d["k_cache"][:1])])
        d["v_cache"] = torch.cat([d["v_cache"], torch.zeros_like(d["v_cache"][:1])])
        d["page_table"][b, page] = zero + 1
        want, mag = reference(d, b)[:2]
        u = 2.0**-8
        assert ((out[b].double() - want).abs() <= u * (1 + u) * want.abs() + (u + 2.0**-13) * mag).all()


def test_page_table_entries_behind_the_chunk_are_not_read():
    c = make(15, 2, 3, 1, 8, 64, [29, 10], 8)
    used = [(29 + 3 + 7) // 8, (10 + 3 + 7) // 8]
    r0 = call(c)
    for b in range(2):
        c["page_table"][b, used[b] :] = -1
    r = call(c)
    assert r["err_flags"].tolist() == [0, 0]
    assert torch.equal(r["out"], r0["out"])


def test_strided_queries_and_shared_pages():
    """Queries as a slice of a fused projection; two requests over the same prefix pages."""
    c = make(16, 2, 5, 2, 4, 128, [64, 64], 16)
    c["page_table"][1, :4] = c["page_table"][0, :4]
    fused = torch.randn((2, 5, 8 + 4, 128), generator=gen(1), device="cuda").to(torch.bfloat16)
    c["q"] = fused[:, :, :8]
    check(c, call(c))


def test_streams_graphs_and_two_workspaces():
    """On a side stream; captured twice with one workspace each and replayed on two streams at once, with
    lengths that change between replays."""
    cs = [make(17 + i, 4, 6, 2, 8, 128, [900, 300, 50, 0], 16) for i in range(2)]
    outs = [dict(out=torch.zeros_like(c["q"]), err_flags=torch.zeros(4, dtype=torch.int32, device="cuda")) for c in cs]
    ws = [binding.make_attention_workspace(6, 16, 2, 128, "cuda") for _ in cs]
    side = torch.cuda.Stream()
    side.wait_stream(torch.cuda.current_stream())
    with torch.cuda.stream(side):
        r = call(cs[0], workspace=ws[0], out=outs[0])
    side.synchronize()
    check(cs[0], r)
    graphs = [torch.cuda.CUDAGraph() for _ in cs]
    for g, c, w, o in zip(graphs, cs, ws, outs):
        with torch.cuda.graph(g):
            call(c, workspace=w, out=o)
    streams = [torch.cuda.Stream(), torch.cuda.Stream()]
    for lens in ([900, 300, 50, 0], [0, 1, 900, 127], [600, 600, 600, 600]):
        for c in cs:
            c["context_len"].copy_(torch.tensor([min(x, y) for x, y in zip(lens, [900, 300, 50, 0])], dtype=torch.int32))
        torch.cuda.synchronize()
        for _ in range(5):
            for g, s in zip(graphs, streams):
                with torch.cuda.stream(s):
                    g.replay()
        torch.cuda.synchronize()
        for c, o in zip(cs, outs):
            check(c, o)


@pytest.mark.parametrize("e4m3", [False, True])
def test_pages_beyond_32_bit_offsets(e4m3):
    """Pages whose element offsets pass 2^31 (16 bits) and 2^32 (8 bits)."""
    H, D, page = 8, 128, 64
    dtype = E4M3 if e4m3 else torch.bfloat16
    pages = (2**32 if e4m3 else 2**31) // (H * D * page) + 6
    c = dict(q=torch.randn((1, 3, 16, D), generator=gen(2), device="cuda").to(torch.bfloat16))
    c["k_cache"] = torch.empty((pages, page, H, D), dtype=torch.uint8 if e4m3 else dtype, device="cuda").view(dtype)
    c["v_cache"] = torch.empty((pages, page, H, D), dtype=torch.uint8 if e4m3 else dtype, device="cuda").view(dtype)
    use = [pages - 1, pages - 6, 0, pages - 2]
    for i, p in enumerate(use):
        for j, name in enumerate(("k", "v")):
            x = torch.randn((page, H, D), generator=gen(10 * i + j), device="cuda")
            c[name + "_cache"][p] = x.to(torch.bfloat16) if not e4m3 else x.to(dtype)
    if e4m3:
        c["k_scale"], c["v_scale"] = (torch.ones((pages, page, H), device="cuda") for _ in range(2))
    c["page_table"] = torch.tensor([use], dtype=torch.int32, device="cuda")
    c["context_len"] = torch.tensor([page * 4 - 3], dtype=torch.int32, device="cuda")
    check(c, call(c))


def test_the_verification_step_end_to_end():
    """One layer's step on 61-node trees over a quantised cache: K and V written, the tree's attention, logits
    from it, processed, verified, the accepted path compacted; then the next step's context reads the
    compacted rows."""
    B, H, G, D, page, V, lens = 4, 2, 4, 128, 16, 4000, [150, 33, 64, 7]
    par = synth.eagle_tree_parents()
    T = len(par)
    g = gen(23)
    P = (max(lens) + T + page - 1) // page
    table = torch.randperm(B * P, generator=g, device="cuda").reshape(B, P).to(torch.int32)
    kc, vc = (torch.zeros((B * P, page, H, D), dtype=torch.uint8, device="cuda").view(E4M3) for _ in range(2))
    ks, vs = torch.zeros((B * P, page, 4), device="cuda")[..., :H].contiguous(), torch.zeros((B * P, page, H), device="cuda")

    def slots(first, n):
        at = first[:, None].long() + torch.arange(n, device="cuda")
        return (table.long().gather(1, at // page) * page + at % page).to(torch.int32)

    ctx = torch.tensor(lens, dtype=torch.int32, device="cuda")
    for b, n in enumerate(lens):  # the prompts, one request at a time
        k, v = (torch.randn((1, n, H, D), generator=g, device="cuda").to(torch.bfloat16) for _ in range(2))
        at = torch.arange(n, device="cuda")
        s = (table[b].long()[at // page] * page + at % page).to(torch.int32)[None].contiguous()
        binding.spec_kv_write(k, v, kc, vc, s, k_scale=ks, v_scale=vs)
    qkv = torch.randn((B, T, H * G + 2 * H, D), generator=g, device="cuda").to(torch.bfloat16)
    q, k, v = qkv[:, :, : H * G], qkv[:, :, H * G : H * G + H], qkv[:, :, H * G + H :]
    chunk_slots = slots(ctx, T)
    assert (binding.spec_kv_write(k, v, kc, vc, chunk_slots, k_scale=ks, v_scale=vs) == 0).all()
    parents = torch.from_numpy(np.tile(par, (B, 1)).astype(np.int32)).cuda()
    c = dict(q=q, k_cache=kc, v_cache=vc, k_scale=ks, v_scale=vs, page_table=table, context_len=ctx, parents=parents)
    r = call(c)
    check(c, r)
    head = torch.randn((H * G * D, V), generator=g, device="cuda").to(torch.bfloat16)
    logits = (r["out"].reshape(B, T, -1) @ head).float()
    history = torch.randint(0, V, (B, 40), generator=g, device="cuda", dtype=torch.int32)
    hl = torch.full((B,), 40, dtype=torch.int32, device="cuda")
    rep = torch.full((B,), 1.3, device="cuda")
    nodes = torch.randint(0, V, (B, T), generator=g, device="cuda", dtype=torch.int32)
    # level by level, the first child of each node on the path becomes what the processed row predicts
    for _ in range(4):
        pl = binding.spec_logits_process(logits, history=history, history_len=hl, node_tokens=nodes, parents=parents, repetition=rep)["logits"]
        best = pl.argmax(-1).to(torch.int32)
        for b in range(B):
            m = 0
            for _ in range(b + 1):
                kids = np.nonzero(par == m)[0]
                if not len(kids):
                    break
                nodes[b, kids[0]] = best[b, m]
                m = int(kids[0])
    pl = binding.spec_logits_process(logits, history=history, history_len=hl, node_tokens=nodes, parents=parents, repetition=rep)["logits"]
    t = binding.spec_verify_tree_greedy(pl, nodes, parents)
    assert (t["err_flags"] == 0).all()
    L = t["accept_len"].tolist()
    assert all(L[b] >= min(b + 1, 4) for b in range(B))
    rows0 = binding.spec_kv_read(kc, vc, chunk_slots, torch.float32, k_scale=ks, v_scale=vs)
    S = B * P * page
    err = binding.spec_kv_compact([kc.view(S, H, D), vc.view(S, H, D)], chunk_slots, parents, t["accept_len"], t["path_nodes"])
    # the scales move as their rows do (8 bytes a row here, below compaction's 16: padded copies)
    pad = [torch.nn.functional.pad(x.view(S, H), (0, 2)).contiguous() for x in (ks, vs)]
    binding.spec_kv_compact(pad, chunk_slots, parents, t["accept_len"], t["path_nodes"])
    ks.view(S, H).copy_(pad[0][:, :H])
    vs.view(S, H).copy_(pad[1][:, :H])
    assert (err == 0).all()
    rows1 = binding.spec_kv_read(kc, vc, chunk_slots, torch.float32, k_scale=ks, v_scale=vs)
    for b in range(B):
        for j, n in enumerate(t["path_nodes"][b, : L[b] + 1].tolist()):
            assert torch.equal(rows1["k"][b, j], rows0["k"][b, n]) and torch.equal(rows1["v"][b, j], rows0["v"][b, n])
    # the next token over the longer context
    c2 = dict(q=torch.randn((B, 1, H * G, D), generator=g, device="cuda").to(torch.bfloat16), k_cache=kc, v_cache=vc, k_scale=ks,
              v_scale=vs, page_table=table, context_len=ctx + t["accept_len"])
    check(c2, call(c2))


def test_empty_calls():
    c = make(30, 2, 3, 1, 2, 64, [5], 8)
    e = dict(c, q=c["q"][:0], page_table=c["page_table"][:0], context_len=c["context_len"][:0])
    assert call(e)["out"].shape[0] == 0
    e = dict(c, q=c["q"][:, :0])
    assert call(e)["out"].shape[1] == 0
    empty = [torch.empty(x.shape[:-1] + (0,), dtype=x.dtype, device="cuda") for x in (c["q"], c["k_cache"], c["v_cache"])]
    with pytest.raises(binding.SpecVerifyError):
        call(dict(c, q=empty[0], k_cache=empty[1], v_cache=empty[2]))
