"""The operators around the verification step, as cases to be timed and compared.

spec_logits_process  penalties, biases and grammar masks on the logits rows of a draft chain or tree
spec_kv_write        new K/V rows into their cache slots, quantised to e4m3 with a scale per token and head
spec_kv_read         cache rows gathered back, in 16 or 32 bits
spec_attention       attention of a chunk of new tokens (a chain or a draft tree) over a paged cache

Each operator has its plain form in elementary torch operations here (32-bit arithmetic, rounded once), and the call
of the package's entry point where `own` is true.
"""

import math

import torch

own = False

DTYPES = {"f32": torch.float32, "bf16": torch.bfloat16, "f16": torch.float16, "e4m3": torch.float8_e4m3fn}
BYTES = {"f32": 4, "bf16": 2, "f16": 2, "e4m3": 1}
DEVICE = "cuda"
# the 61-node draft tree of the benchmark's tree workloads: (expanded parents, children each) level by level
TREE_LEVELS = ((1, 10), (4, 4), (4, 3), (5, 2), (3, 2), (3, 2))


# ---------------------------------------------------------------------------------------------------------- cases ----
def listed():
    return [
        # one interactive request: a short chain, a small vocabulary, every rule at once; latency counts
        dict(name="logits_single", op="logits", B=1, R=6, V=32000, dtype="bf16", tree=False, history=512, bias=16, mask=True),
        # the batched chain verification's logits: repetition, presence and frequency over 2048-token histories
        dict(name="logits_chain_f32", op="logits", B=64, R=6, V=128256, dtype="f32", tree=False, history=2048, bias=16, mask=False),
        # the greedy tree workload's 61 rows a request under a grammar
        dict(name="logits_tree_bf16", op="logits", B=16, R=61, V=128256, dtype="bf16", tree=True, history=1021, bias=0, mask=True),
        # the K and V rows of one layer for 16 draft trees
        dict(name="kv_write_tree", op="kv_write", B=16, T=61, H=8, D=128, dtype="bf16"),
        # four 2048-token prompts of one layer, K and V taken out of the fused projection
        dict(name="kv_write_prompt", op="kv_write", B=4, T=2048, H=8, D=128, dtype="f16"),
        # the accepted rows of one request read back at full precision
        dict(name="kv_read_single", op="kv_read", B=1, T=61, H=8, D=128, dtype="f32"),
        # 16 prompts' rows of one layer handed to an engine that keeps 16 bits
        dict(name="kv_read_prompts", op="kv_read", B=16, T=2052, H=8, D=128, dtype="bf16"),
        # plain decoding, one token a request, where latency counts
        dict(name="attn_decode", op="attention", B=8, T=1, Hq=64, H=8, D=128, L=2052, page=16, dtype="bf16", cache="bf16", tree=False),
        # chains of 5 draft tokens and the last accepted one: the cache's bytes bound it
        dict(name="attn_chain_bf16", op="attention", B=64, T=6, Hq=64, H=8, D=128, L=4096, page=16, dtype="bf16", cache="bf16", tree=False),
        # the same chains over a quantised cache of twice the length
        dict(name="attn_chain_e4m3", op="attention", B=64, T=6, Hq=64, H=8, D=128, L=8192, page=32, dtype="bf16", cache="e4m3", tree=False),
        # 61-node draft trees over long contexts: the products bound it
        dict(name="attn_tree_bf16", op="attention", B=16, T=61, Hq=64, H=8, D=128, L=8192, page=64, dtype="bf16", cache="bf16", tree=True),
        # the second half of two 4096-token prompts
        dict(name="attn_prompt_f16", op="attention", B=2, T=2048, Hq=64, H=8, D=128, L=2048, page=16, dtype="f16", cache="f16", tree=False),
    ]


def _log_uniform(rng, lo, hi):
    return max(lo, min(hi, int(round(math.exp(rng.uniform(math.log(lo), math.log(hi + 0.49)))))))


def draw(rng):
    op = rng.choice(["logits", "kv_write", "kv_read", "attention", "attention"])
    if op == "logits":
        tree = rng.random() < 0.4
        R = 61 if tree else rng.randint(1, 9)
        V = rng.choice([_log_uniform(rng, 1000, 160000), 32000, 128256, 151936])
        B = _log_uniform(rng, 1, max(1, min(256, 64 * 6 * 128256 // (R * V))))
        return dict(op=op, B=B, R=R, V=V, dtype=rng.choice(["f32", "bf16", "f16"]), tree=tree,
                    history=_log_uniform(rng, 1, 8192), bias=rng.choice([0, rng.randint(1, 300)]), mask=rng.random() < 0.5)
    if op in ("kv_write", "kv_read"):
        D = rng.choice([64, 80, 96, 128, 192, 256])
        H = rng.choice([1, 2, 4, 8])
        T = rng.choice([1, 6, 61, _log_uniform(rng, 1, 4096)])
        B = _log_uniform(rng, 1, max(1, min(256, 16 * 2052 * 1024 // (T * H * D))))
        return dict(op=op, B=B, T=T, H=H, D=D, dtype=rng.choice(["f32", "bf16", "f16"]))
    D, H, group = rng.choice([64, 128, 128]), rng.choice([1, 2, 4, 8]), rng.choice([1, 2, 3, 4, 6, 7, 8, 16])
    tree = rng.random() < 0.3
    T = 61 if tree else rng.choice([1, rng.randint(2, 9), _log_uniform(rng, 1, 1500)])
    L = _log_uniform(rng, 1, 16384)
    most = min(64 * 8 * 4096 * 128 // (H * (L + T) * D), 2 * 64 * 2048 * 3000 * 128 // (H * group * T * (L + T) * D))
    B = _log_uniform(rng, 1, max(1, min(128, most)))
    dtype = rng.choice(["bf16", "f16"])
    return dict(op=op, B=B, T=T, Hq=H * group, H=H, D=D, L=L, page=rng.choice([8, 16, 32, 64, 128, 256]), dtype=dtype,
                cache=rng.choice([dtype, "e4m3"]), tree=tree)


# --------------------------------------------------------------------------------------------------------- inputs ----
def _gen(seed):
    g = torch.Generator(device=DEVICE)
    g.manual_seed(1000003 * int(seed) + 17)
    return g


def _normal(g, shape, dtype, std=1.0):
    x = torch.empty(shape, dtype=torch.float32 if dtype == torch.float8_e4m3fn else dtype, device=DEVICE)
    return x.normal_(0.0, std, generator=g)


def _ints(g, lo, hi, shape):
    return torch.randint(lo, hi, shape, generator=g, device=DEVICE, dtype=torch.int32)


def _tokens(g, V, shape):
    """Token ids as text has them: a few frequent ones, many rare ones."""
    return (torch.rand(shape, generator=g, device=DEVICE).pow(4) * V).to(torch.int32).clamp_(0, V - 1)


def _tree_parents():
    parents, level = [-1], [0]
    for expanded, children in TREE_LEVELS:
        first = len(parents)
        parents += [p for p in level[:expanded] for _ in range(children)]
        level = list(range(first, len(parents)))
    return parents


def _parents(B):
    return torch.tensor([_tree_parents()], dtype=torch.int32, device=DEVICE).repeat(B, 1)


def prepare(case, seed):
    return {"logits": _prepare_logits, "kv_write": _prepare_kv_write, "kv_read": _prepare_kv_read,
            "attention": _prepare_attention}[case["op"]](case, _gen(seed))


def _prepare_logits(c, g):
    B, R, V, dt = c["B"], c["R"], c["V"], DTYPES[c["dtype"]]
    s = dict(case=c, logits=_normal(g, (B, R, V), dt, 3.0), out=torch.empty((B, R, V), dtype=dt, device=DEVICE))
    n = c["history"]
    s["history_len"] = _ints(g, (n + 3) // 4, n + 1, (B,))
    s["prompt_len"] = (s["history_len"] * torch.rand((B,), generator=g, device=DEVICE)).to(torch.int32)
    history = _tokens(g, V, (B, n))
    s["history"] = torch.where(torch.arange(n, device=DEVICE) < s["history_len"][:, None], history, torch.full_like(history, -1))
    s["draft_tokens"] = _tokens(g, V, (B, R - 1)) if not c["tree"] else None
    s["node_tokens"] = _tokens(g, V, (B, R)) if c["tree"] else None
    s["parents"] = _parents(B) if c["tree"] else None
    s["repetition"] = 1.0 + 0.3 * torch.rand((B,), generator=g, device=DEVICE)
    s["presence"] = torch.rand((B,), generator=g, device=DEVICE)
    s["frequency"] = 0.5 * torch.rand((B,), generator=g, device=DEVICE)
    s["bias_tokens"] = s["bias_values"] = s["allowed"] = None
    if c["bias"]:
        nb = min(c["bias"], V)
        s["bias_tokens"] = torch.rand((B, V), generator=g, device=DEVICE).topk(nb, dim=1).indices.to(torch.int32).contiguous()
        s["bias_values"] = _normal(g, (B, nb), torch.float32, 4.0)
    if c["mask"]:  # a third of the rows free, the others with a sixteenth of the vocabulary allowed
        W = (V + 31) // 32
        w = [_ints(g, -2**31, 2**31 - 1, (B, R, W)) for _ in range(4)]
        free = torch.rand((B, R, 1), generator=g, device=DEVICE) < 0.33
        s["allowed"] = torch.where(free, torch.full_like(w[0], -1), w[0] & w[1] & w[2] & w[3])
    return s


def _slots(g, B, T):
    """Distinct cache slots in a random order of 16-slot pages, and the number of slots."""
    pages = (T + 15) // 16
    table = torch.randperm(B * pages + 3, generator=g, device=DEVICE)[: B * pages].reshape(B, pages, 1)
    slots = table * 16 + torch.arange(16, device=DEVICE)
    return slots.reshape(B, -1)[:, :T].to(torch.int32).contiguous(), (B * pages + 3) * 16


def _prepare_kv_write(c, g):
    B, T, H, D, dt = c["B"], c["T"], c["H"], c["D"], DTYPES[c["dtype"]]
    qkv = _normal(g, (B, T, 4 * H, D), dt)  # two query heads a KV head, then K, then V
    qkv *= torch.rand((B, T, 4 * H, 1), generator=g, device=DEVICE).mul_(3).exp_().to(dt)
    slots, S = _slots(g, B, T)
    z = lambda *shape, dtype: torch.zeros(shape, dtype=dtype, device=DEVICE)  # noqa: E731
    return dict(case=c, k=qkv[:, :, 2 * H : 3 * H], v=qkv[:, :, 3 * H :], slots=slots, S=S,
                k_cache=z(S, H, D, dtype=DTYPES["e4m3"]), v_cache=z(S, H, D, dtype=DTYPES["e4m3"]),
                k_scale=z(S, H, dtype=torch.float32), v_scale=z(S, H, dtype=torch.float32),
                err_flags=torch.empty((B,), dtype=torch.int32, device=DEVICE))


def _quantised(g, shape):
    """e4m3 codes of normal values and a power-of-two scale for each of their rows."""
    scale = torch.exp2(_ints(g, -8, -5, shape[:-1]).to(torch.float32))
    return _normal(g, shape, torch.float32, 100.0).clamp_(-448, 448).to(DTYPES["e4m3"]), scale


def _prepare_kv_read(c, g):
    B, T, H, D = c["B"], c["T"], c["H"], c["D"]
    slots, S = _slots(g, B, T)
    k_cache, k_scale = _quantised(g, (S, H, D))
    v_cache, v_scale = _quantised(g, (S, H, D))
    out = dict(k=torch.empty((B, T, H, D), dtype=DTYPES[c["dtype"]], device=DEVICE),
               v=torch.empty((B, T, H, D), dtype=DTYPES[c["dtype"]], device=DEVICE),
               err_flags=torch.empty((B,), dtype=torch.int32, device=DEVICE))
    return dict(case=c, k_cache=k_cache, v_cache=v_cache, k_scale=k_scale, v_scale=v_scale, slots=slots, out=out)


def _prepare_attention(c, g):
    B, T, Hq, H, D, L, page, dt = c["B"], c["T"], c["Hq"], c["H"], c["D"], c["L"], c["page"], DTYPES[c["dtype"]]
    P = (L + T + page - 1) // page
    pages = B * P + 5
    s = dict(case=c, q=_normal(g, (B, T, Hq, D), dt, 2.0))
    if c["cache"] == "e4m3":
        s["k_cache"], s["k_scale"] = _quantised(g, (pages, page, H, D))
        s["v_cache"], s["v_scale"] = _quantised(g, (pages, page, H, D))
    else:
        s["k_cache"], s["v_cache"] = _normal(g, (pages, page, H, D), dt), _normal(g, (pages, page, H, D), dt)
        s["k_scale"] = s["v_scale"] = None
    s["page_table"] = torch.randperm(pages, generator=g, device=DEVICE)[: B * P].reshape(B, P).to(torch.int32)
    s["context_len"] = _ints(g, L // 2, L + 1, (B,))
    s["parents"] = _parents(B) if c["tree"] else None
    s["out"] = dict(out=torch.zeros((B, T, Hq, D), dtype=dt, device=DEVICE), err_flags=torch.empty((B,), dtype=torch.int32, device=DEVICE))
    s["workspace"] = None  # made once, at the first call
    return s


# --------------------------------------------------------------------------------------------------------- passes ----
def run(state):
    return (_run_own if own else _run_plain)(state)


def _run_own(s):
    import speculative_decoding_verification_82_gb300 as sv

    c = s["case"]
    if c["op"] == "logits":
        return sv.spec_logits_process(
            s["logits"], history=s["history"], history_len=s["history_len"], prompt_len=s["prompt_len"],
            draft_tokens=s["draft_tokens"], node_tokens=s["node_tokens"], parents=s["parents"], repetition=s["repetition"],
            presence=s["presence"], frequency=s["frequency"], bias_tokens=s["bias_tokens"], bias_values=s["bias_values"],
            allowed=s["allowed"], out=dict(logits=s["out"]))["logits"]
    if c["op"] == "kv_write":
        sv.spec_kv_write(s["k"], s["v"], s["k_cache"], s["v_cache"], s["slots"], k_scale=s["k_scale"], v_scale=s["v_scale"],
                         err_flags=s["err_flags"])
        return dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])
    if c["op"] == "kv_read":
        r = sv.spec_kv_read(s["k_cache"], s["v_cache"], s["slots"], DTYPES[c["dtype"]], k_scale=s["k_scale"],
                            v_scale=s["v_scale"], out=s["out"])
        return dict(k=r["k"], v=r["v"])
    if s["workspace"] is None:
        s["workspace"] = sv.make_attention_workspace(c["T"], c["Hq"], c["H"], c["D"], s["q"].device)
    return sv.spec_attention(s["q"], s["k_cache"], s["v_cache"], s["page_table"], s["context_len"], parents=s["parents"],
                             k_scale=s["k_scale"], v_scale=s["v_scale"], workspace=s["workspace"], out=s["out"])["out"]


def _run_plain(s):
    return {"logits": _plain_logits, "kv_write": _plain_kv_write, "kv_read": _plain_kv_read,
            "attention": _plain_attention}[s["case"]["op"]](s)


def _counts(tokens, keep, V):
    """[..., V] occurrences of `tokens` [..., n] where `keep`."""
    c = torch.zeros((*tokens.shape[:-1], V), dtype=torch.float32, device=DEVICE)
    return c.scatter_add_(-1, tokens.clamp(0, V - 1).long(), keep.to(torch.float32))


def _ancestors(parents):
    """[B, N, N] truth values: j is i or one of i's ancestors (the powers of the parent relation, summed)."""
    B, N = parents.shape
    link = torch.zeros((B, N, N), dtype=torch.float64, device=DEVICE)
    link.scatter_(2, parents.clamp(min=0).long()[:, :, None], (parents >= 0).double()[:, :, None])
    return torch.matrix_power(link + torch.eye(N, dtype=torch.float64, device=DEVICE), N) > 0.5


def _plain_logits(s):
    B, R, V = s["logits"].shape
    n = s["history"].shape[1]
    pos = torch.arange(n, device=DEVICE)
    valid = pos < s["history_len"][:, None]
    out_part = valid & (pos >= s["prompt_len"][:, None])
    count = _counts(s["history"], out_part, V)[:, None]
    seen = _counts(s["history"], valid, V)[:, None]
    if s["parents"] is not None:  # row n: the tokens of n and its ancestors (the root's is in the history)
        on_path = _ancestors(s["parents"]) & (torch.arange(R, device=DEVICE) > 0)
        path_tokens = s["node_tokens"][:, None, :].expand(B, R, R)
    else:  # row k: the first k draft tokens
        on_path = (torch.arange(R - 1, device=DEVICE) < torch.arange(R, device=DEVICE)[:, None]).expand(B, R, R - 1)
        path_tokens = s["draft_tokens"][:, None, :].expand(B, R, R - 1)
    path = _counts(path_tokens, on_path, V)
    count, seen = count + path, seen + path
    x = s["logits"].to(torch.float32)
    rep = s["repetition"][:, None, None]
    x = torch.where(seen > 0, torch.where(x > 0, x / rep, x * rep), x)
    x = x - (s["frequency"][:, None, None] * count + s["presence"][:, None, None] * (count > 0))
    if s["bias_tokens"] is not None:
        bias = torch.zeros((B, V), dtype=torch.float32, device=DEVICE).scatter_add_(1, s["bias_tokens"].long(), s["bias_values"])
        x = x + bias[:, None]
    if s["allowed"] is not None:
        bits = (s["allowed"][..., None] >> torch.arange(32, device=DEVICE, dtype=torch.int32)) & 1
        x = x.masked_fill(bits.reshape(B, R, -1)[..., :V] == 0, float("-inf"))
    return x.to(s["logits"].dtype)


def _plain_codes(x):
    """e4m3 codes and their scale: the smallest power of two that brings the row's largest magnitude within 448."""
    x = x.to(torch.float32)
    m, e = torch.frexp(x.abs().amax(-1))
    scale = torch.ldexp(torch.ones_like(m), (e - 9 + (m > 0.875)).clamp(min=-126))
    return (x / scale[..., None]).to(DTYPES["e4m3"]), scale


def _plain_kv_write(s):
    slots = s["slots"].long().reshape(-1)
    for name in ("k", "v"):
        codes, scale = _plain_codes(s[name])
        # bytes are scattered: an index assignment on the codes' own type is not offered everywhere
        s[name + "_cache"].view(torch.uint8)[slots] = codes.view(torch.uint8).reshape(-1, *codes.shape[2:])
        s[name + "_scale"][slots] = scale.reshape(-1, scale.shape[-1])
    return dict(k=s["k_cache"], v=s["v_cache"], k_scale=s["k_scale"], v_scale=s["v_scale"])


def _plain_kv_read(s):
    dt, slots = DTYPES[s["case"]["dtype"]], s["slots"].long()
    row = lambda n: s[n + "_cache"].view(torch.uint8)[slots].view(DTYPES["e4m3"]).to(torch.float32) * s[n + "_scale"][slots][..., None]  # noqa: E731
    return dict(k=row("k").to(dt), v=row("v").to(dt))


def _cache_rows(s, name, wide):
    """[B, H, n, D] of the request's first n cache positions, in `wide`."""
    table = s["page_table"].long()
    cache, scale = s[name + "_cache"], s[name + "_scale"]
    if scale is None:
        x = cache[table].to(wide)
    else:
        x = cache.view(torch.uint8)[table].view(DTYPES["e4m3"]).to(wide) * scale[table].to(wide)[..., None]
    return x.reshape(x.shape[0], -1, *x.shape[3:]).transpose(1, 2)


def _plain_attention(s):
    B, T, Hq, D = s["q"].shape
    H = s["k_cache"].shape[2]
    G = Hq // H
    k, v = _cache_rows(s, "k", torch.float32), _cache_rows(s, "v", torch.float32)
    n = k.shape[2]
    q = s["q"].to(torch.float32).reshape(B, T, H, G, D).permute(0, 2, 1, 3, 4).reshape(B, H, T * G, D)
    x = (q @ k.transpose(2, 3)).mul_(1 / math.sqrt(D))
    at = torch.arange(n, device=DEVICE) - s["context_len"][:, None]  # the position within the chunk
    if s["parents"] is not None:
        see = _ancestors(s["parents"]).gather(2, at.clamp(0, T - 1)[:, None].expand(B, T, n)) & (at < T)[:, None]
        see |= (at < 0)[:, None]
    else:
        see = at[:, None] <= torch.arange(T, device=DEVICE)[:, None]
    x.masked_fill_(~see.repeat_interleave(G, 1)[:, None], float("-inf"))
    x -= x.amax(-1, keepdim=True)
    x.exp_()
    total = x.sum(-1, keepdim=True)
    o = (x @ v) / total
    return o.reshape(B, H, T, G, D).permute(0, 2, 1, 3, 4).reshape(B, T, Hq, D).to(s["q"].dtype)


# ------------------------------------------------------------------------------------------------- the definitions ----
def exact(case, seed):
    s = prepare(case, seed)
    return {"logits": _exact_logits, "kv_write": _exact_kv_write, "kv_read": _exact_kv_read,
            "attention": _exact_attention}[case["op"]](s)


def _path(parents, i):
    """Node i and its ancestors but the root."""
    nodes = []
    while i > 0:
        nodes.append(i)
        i = parents[i]
    return nodes


def _exact_logits(s):
    out = s["logits"].double()
    B, R, V = out.shape
    tree = None if s["parents"] is None else s["parents"].tolist()
    drafts = (s["draft_tokens"] if tree is None else s["node_tokens"]).tolist()
    for b in range(B):
        n, p = int(s["history_len"][b]), int(s["prompt_len"][b])
        h = s["history"][b, :n].long()
        base = torch.bincount(h[p:], minlength=V)
        prompt = torch.bincount(h[:p], minlength=V) > 0
        rep, pres, freq = (float(s[k][b]) for k in ("repetition", "presence", "frequency"))
        bias = torch.zeros(V, dtype=torch.float64, device=DEVICE)
        if s["bias_tokens"] is not None:
            bias[s["bias_tokens"][b].long()] = s["bias_values"][b].double()
        for r in range(R):
            path = drafts[b][:r] if tree is None else [drafts[b][i] for i in _path(tree[b], r)]
            c = base + torch.bincount(torch.tensor(path, dtype=torch.long, device=DEVICE), minlength=V)
            x = out[b, r]
            y = torch.where(x > 0, x / rep, x * rep)
            x = torch.where(prompt | (c > 0), y, x) - torch.where(c > 0, freq * c + pres, torch.zeros_like(x)) + bias
            if s["allowed"] is not None:
                at = torch.arange(V, device=DEVICE)
                ok = (s["allowed"][b, r].long()[at // 32] >> (at % 32)) & 1
                x = torch.where(ok == 1, x, torch.full_like(x, -math.inf))
            out[b, r] = x
    return out


def _exact_kv_write(s):
    out = {}
    for name in ("k", "v"):
        x = s[name].double()
        most = x.abs().amax(-1)
        scale = torch.exp2(torch.round(torch.log2(most / 448)).clamp(min=-126))  # within a step; the comparisons settle it
        scale = torch.where(448 * scale < most, 2 * scale, scale)
        scale = torch.where(224 * scale >= most, scale / 2, scale).clamp(min=2.0**-126)
        codes = torch.zeros(s[name + "_cache"].shape, dtype=torch.float64, device=DEVICE)
        scales = torch.zeros(s[name + "_scale"].shape, dtype=torch.float64, device=DEVICE)
        codes[s["slots"].long()] = x / scale[..., None]
        scales[s["slots"].long()] = scale
        out[name], out[name + "_scale"] = codes, scales
    return out


def _exact_kv_read(s):
    at = s["slots"].long()
    return {n: (s[n + "_cache"].double() * s[n + "_scale"].double()[..., None])[at] for n in ("k", "v")}


def _exact_attention(s):
    B, T, Hq, D = s["q"].shape
    H, page = s["k_cache"].shape[2], s["k_cache"].shape[1]
    G = Hq // H
    out = torch.empty((B, T, Hq, D), dtype=torch.float64, device=DEVICE)
    for b in range(B):
        L = int(s["context_len"][b])
        at = torch.arange(L + T, device=DEVICE)
        slot = s["page_table"][b].long()[at // page] * page + at % page
        rows = []
        for name in ("k", "v"):
            x = s[name + "_cache"].reshape(-1, H, D).view(torch.uint8 if s[name + "_scale"] is not None else s["q"].dtype)[slot]
            if s[name + "_scale"] is not None:
                x = x.view(DTYPES["e4m3"]).double() * s[name + "_scale"].reshape(-1, H)[slot].double()[..., None]
            rows.append(x.double())
        see = torch.zeros((T, L + T), dtype=torch.bool, device=DEVICE)
        see[:, :L] = True
        if s["parents"] is None:
            see[:, L:] = torch.ones((T, T), dtype=torch.bool, device=DEVICE).tril()
        else:
            parents = s["parents"][b].tolist()
            for t in range(T):
                see[t, [L] + [L + i for i in _path(parents, t)]] = True
        for h in range(H):
            x = torch.einsum("tgd,nd->gtn", s["q"][b, :, h * G : (h + 1) * G].double(), rows[0][:, h]) / math.sqrt(D)
            p = torch.softmax(x.masked_fill(~see, -math.inf), -1)
            out[b, :, h * G : (h + 1) * G] = torch.einsum("gtn,nd->tgd", p, rows[1][:, h])
    return out


# ----------------------------------------------------------------------------------------------------------- work ----
def work(case):
    c = case
    if c["op"] == "logits":
        n = c["B"] * c["R"] * c["V"]
        return dict(bytes=2 * n * BYTES[c["dtype"]] + (n // 8 if c["mask"] else 0) + 4 * c["B"] * c["history"] * 5 // 8, flops=0)
    if c["op"] in ("kv_write", "kv_read"):
        rows = 2 * c["B"] * c["T"] * c["H"]
        return dict(bytes=rows * (c["D"] * (BYTES[c["dtype"]] + 1) + 4), flops=0)
    B, T, Hq, H, D = c["B"], c["T"], c["Hq"], c["H"], c["D"]
    n = 0.75 * c["L"]  # the mean length of the prefixes
    seen = n + (4 if c["tree"] else (T + 1) / 2)  # a tree's node sees itself and its few ancestors
    row = 2 * H * (D * BYTES[c["cache"]] + (4 if c["cache"] == "e4m3" else 0))
    return dict(bytes=B * (n + T) * row + 2 * B * T * Hq * D * BYTES[c["dtype"]], flops=4 * B * T * Hq * D * seen)
