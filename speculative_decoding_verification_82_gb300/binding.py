"""Thin ctypes binding of the C ABI declared in include/spec_verify.h.

Argument marshalling only: the functions take torch CUDA tensors, check their shape, dtype and
device, allocate outputs and the workspace when the caller did not supply them, and pass raw
pointers and the current CUDA stream to the library.  Every step of the verification runs in the
library's kernels; there is no other implementation to fall back on, so a missing library raises.
"""

from __future__ import annotations

import ctypes
import math
import os
from ctypes import c_float, c_int, c_size_t, c_void_p

import torch
from torch import Tensor

from .build import LIB_PATH

SPEC_OK, SPEC_ERR_INVALID_ARG, SPEC_ERR_CUDA, SPEC_ERR_WORKSPACE, SPEC_ERR_UNSUPPORTED = range(5)
ERRF_BAD_TOKEN, ERRF_NONFINITE, ERRF_TIMEOUT, ERRF_BAD_TREE, ERRF_BAD_TEMPERATURE = 1, 2, 4, 8, 16
ERRF_BAD_LENGTH, ERRF_BAD_SLOT, ERRF_BAD_PENALTY, ERRF_BAD_SAMPLING = 32, 64, 128, 256
MAX_K, MAX_TREE_NODES, MAX_WALK_NODES, MAX_WALK_VOCAB, MAX_NGRAM = 256, 4096, 1024, 262144, 32
MAX_KV_CACHES, MAX_LOGITS_ROWS, MAX_BIASES, MAX_KV_HEAD_DIM, MAX_SAMPLE_VOCAB = 1024, 1024, 4096, 256, 262144
DTYPE_CODE = {torch.float32: 0, torch.bfloat16: 1, torch.float16: 2}
E4M3 = torch.float8_e4m3fn
CACHE_CODE = {**DTYPE_CODE, E4M3: 3}

EXPORTED = ("spec_verify_workspace_bytes", "spec_verify_workspace_reset", "spec_verify_chain",
            "spec_verify_ngram", "spec_verify_tree_greedy", "spec_verify_tree_walk", "spec_ngram_draft",
            "spec_kv_compact", "spec_kv_write", "spec_kv_read", "spec_rope_kv_write", "spec_logits_process",
            "spec_sample", "spec_logits_filter",
            "spec_attention", "spec_attention_workspace_bytes",
            "spec_verify_chain_static", "spec_status_string")
STATIC_WORKSPACE_BYTES = 4 << 20

_lib = None


class SpecVerifyError(RuntimeError):
    pass


def library(path: str | None = None) -> ctypes.CDLL:
    """Load libspecverify.so (built by __graft_entry__.build()); raises if it is missing."""
    global _lib
    if _lib is not None and path is None:
        return _lib
    p = path or LIB_PATH
    if not os.path.exists(p):
        raise SpecVerifyError(f"CUDA library not built: {p} is missing (run __graft_entry__.build())")
    lib = ctypes.CDLL(p)
    P, I, F, Z = c_void_p, c_int, c_float, c_size_t
    lib.spec_verify_workspace_bytes.argtypes = [I, I, I, I]
    lib.spec_verify_workspace_bytes.restype = Z
    lib.spec_verify_workspace_reset.argtypes = [P]
    lib.spec_verify_workspace_reset.restype = None
    lib.spec_verify_chain.argtypes = [P, P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_chain.restype = I
    lib.spec_verify_ngram.argtypes = [P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_ngram.restype = I
    lib.spec_verify_tree_greedy.argtypes = [P, I, I, I, I, P, P, P, P, P, P, P, P, Z, P]
    lib.spec_verify_tree_greedy.restype = I
    lib.spec_verify_tree_walk.argtypes = [P, P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, P, P, P]
    lib.spec_verify_tree_walk.restype = I
    lib.spec_ngram_draft.argtypes = [P, P, I, I, I, I, I, P, P, P, P, P, P]
    lib.spec_ngram_draft.restype = I
    lib.spec_kv_compact.argtypes = [ctypes.POINTER(c_void_p), I, ctypes.c_longlong, I, I, I, P, P, P, P, P, P]
    lib.spec_kv_compact.restype = I
    LL = ctypes.c_longlong
    lib.spec_kv_write.argtypes = [P, P, I, LL, LL, I, I, I, I, P, P, P, I, P, P, LL, P, P]
    lib.spec_kv_write.restype = I
    lib.spec_kv_read.argtypes = [P, P, I, P, P, LL, I, I, I, I, P, P, P, I, P, P]
    lib.spec_kv_read.restype = I
    lib.spec_rope_kv_write.argtypes = [P, P, P, I, LL, LL, LL, I, I, I, I, I, P, I, I, F, P, P, P, P, P, LL, P, P, I, P, P, LL, P, P]
    lib.spec_rope_kv_write.restype = I
    lib.spec_logits_process.argtypes = [P, I, I, I, I, P, P, P, I, P, P, P, P, P, P, P, P, I, P, P, P, P]
    lib.spec_logits_process.restype = I
    lib.spec_sample.argtypes = [P, I, I, I, I, F, P, P, P, P, P, P, P, P, P, P]
    lib.spec_sample.restype = I
    lib.spec_logits_filter.argtypes = [P, I, I, I, I, F, P, P, P, P, P, P, P, P]
    lib.spec_logits_filter.restype = I
    lib.spec_attention_workspace_bytes.argtypes = [I, I, I, I]
    lib.spec_attention_workspace_bytes.restype = Z
    lib.spec_attention.argtypes = [P, I, LL, I, I, I, I, I, P, P, I, P, P, LL, I, P, I, P, P, P, F, P, P, P, P, Z, P]
    lib.spec_attention.restype = I
    lib.spec_verify_chain_static.argtypes = [P, P, I, I, I, I, F, P, P, P, P, P, P, P, P]
    lib.spec_verify_chain_static.restype = I
    lib.spec_status_string.argtypes = [I]
    lib.spec_status_string.restype = ctypes.c_char_p
    if path is None:
        _lib = lib
    return lib


def _check(status: int) -> None:
    if status != SPEC_OK:
        name = library().spec_status_string(status).decode()
        raise SpecVerifyError(f"{name} ({status})")


def _ptr(t: torch.Tensor | None):
    return None if t is None else c_void_p(t.data_ptr())


def _stream(device) -> c_void_p:
    return c_void_p(torch.cuda.current_stream(device).cuda_stream)


def _need(t, name: str, dtype, shape, device) -> torch.Tensor:
    if type(t) is Tensor and t.dtype is dtype and t.shape == shape and t.device == device and t.is_contiguous():
        return t  # (what a step calls with; the rest finds what is wrong)
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if t.device != device:
        raise ValueError(f"{name} must be on {device}, got {t.device}")
    if dtype is not None and t.dtype != dtype:
        raise TypeError(f"{name} must be {dtype}, got {t.dtype}")
    if tuple(t.shape) != tuple(shape):
        raise ValueError(f"{name} must have shape {tuple(shape)}, got {tuple(t.shape)}")
    if not t.is_contiguous():
        raise ValueError(f"{name} must be contiguous")
    return t


def workspace_bytes(B: int, rows_per_request: int, V: int, dtype: torch.dtype) -> int:
    """Workspace bytes for B requests reading `rows_per_request` logits rows of V elements each
    (draft-model chain: 2K+1, greedy chain / n-gram: K+1, tree: N+1)."""
    return int(library().spec_verify_workspace_bytes(B, rows_per_request, V, DTYPE_CODE[dtype]))


def make_workspace(B: int, rows_per_request: int, V: int, dtype: torch.dtype, device) -> torch.Tensor:
    """A workspace for such calls (new memory: its first call clears it)."""
    n = max(256, workspace_bytes(B, rows_per_request, V, dtype))
    ws = torch.empty(n, dtype=torch.uint8, device=device)
    workspace_reset(ws)  # the caching allocator may hand out the block of an earlier workspace
    return ws


def workspace_reset(workspace: torch.Tensor) -> None:
    """Tells the library that something other than its calls wrote to `workspace` (see
    spec_verify_workspace_reset): the next call clears it first."""
    library().spec_verify_workspace_reset(ctypes.c_void_p(workspace.data_ptr()))


def _out(given, name, dtype, shape, device):
    if given is None:
        return torch.empty(shape, dtype=dtype, device=device)
    return _need(given, name, dtype, shape, device)


def _opt(given, name, dtype, shape, device):
    return None if given is None else _need(given, name, dtype, shape, device)


def _chain_like(ngram: bool, target_logits, draft_logits, draft_tokens, r, u, temperature,
                workspace, out, accept_prob, cand_tokens, pos_mass, target_probs, draft_probs,
                temperatures=None):
    lib = library()
    dev = target_logits.device
    if target_logits.dtype not in DTYPE_CODE or target_logits.dim() != 3:
        raise TypeError("target_logits must be a [B][K+1][V] float32/bfloat16/float16 tensor")
    B, K1, V = target_logits.shape
    K = K1 - 1
    T = float(temperature)
    _need(target_logits, "target_logits", None, (B, K1, V), dev)
    if draft_tokens is None:
        draft_tokens = torch.empty((B, K), dtype=torch.int32, device=dev)
    _need(draft_tokens, "draft_tokens", torch.int32, (B, K), dev)
    sampled = T > 0 or temperatures is not None  # per-request temperatures: any request may sample
    if temperatures is not None:
        _need(temperatures, "temperatures", torch.float32, (B,), dev)
    if not ngram and sampled and K > 0:
        _need(draft_logits, "draft_logits", target_logits.dtype, (B, K, V), dev)
    if sampled:
        _need(r, "r", torch.float32, (B, K), dev)
        _need(u, "u", torch.float32, (B,), dev)
    if workspace is None:
        rows = 2 * K + 1 if (not ngram and sampled and K > 0) else K1
        workspace = make_workspace(B, rows, V, target_logits.dtype, dev)
    out = dict(out or {})
    na = _out(out.get("num_accepted"), "num_accepted", torch.int32, (B,), dev)
    ot = _out(out.get("out_tokens"), "out_tokens", torch.int32, (B, K1), dev)
    rm = _out(out.get("residual_mass"), "residual_mass", torch.float32, (B,), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    ap = _opt(accept_prob, "accept_prob", torch.float32, (B, K), dev)
    ct = _opt(cand_tokens, "cand_tokens", torch.int32, (B, K1), dev)
    pm = _opt(pos_mass, "pos_mass", torch.float32, (B, K1), dev)
    tp = _opt(target_probs, "target_probs", torch.float32, (B, K1, V), dev)
    tail = (_ptr(na), _ptr(ot), _ptr(rm), _ptr(ef), _ptr(ap), _ptr(ct), _ptr(pm), _ptr(tp))
    if ngram:
        st = lib.spec_verify_ngram(_ptr(target_logits), DTYPE_CODE[target_logits.dtype], B, K, V, T,
                                   _ptr(temperatures), _ptr(draft_tokens), _ptr(r), _ptr(u), *tail, _ptr(workspace),
                                   workspace.numel(), _stream(dev))
    else:
        dp = _opt(draft_probs, "draft_probs", torch.float32, (B, K, V), dev)
        st = lib.spec_verify_chain(_ptr(target_logits), _ptr(draft_logits),
                                   DTYPE_CODE[target_logits.dtype], B, K, V, T, _ptr(temperatures),
                                   _ptr(draft_tokens),
                                   _ptr(r), _ptr(u), *tail, _ptr(dp), _ptr(workspace),
                                   workspace.numel(), _stream(dev))
    _check(st)
    return dict(num_accepted=na, out_tokens=ot, residual_mass=rm, err_flags=ef)


def spec_verify_chain(target_logits, draft_logits, draft_tokens, r, u, temperature, *,
                      workspace=None, out=None, accept_prob=None, cand_tokens=None, pos_mass=None,
                      target_probs=None, draft_probs=None, temperatures=None) -> dict:
    """Chain verification with draft logits (draft model / EAGLE head); `temperatures` [B] gives
    each request its own T.  See spec_verify.h."""
    return _chain_like(False, target_logits, draft_logits, draft_tokens, r, u, temperature,
                       workspace, out, accept_prob, cand_tokens, pos_mass, target_probs,
                       draft_probs, temperatures)


def spec_verify_ngram(target_logits, draft_tokens, r, u, temperature, *, workspace=None, out=None,
                      accept_prob=None, cand_tokens=None, pos_mass=None,
                      target_probs=None, temperatures=None) -> dict:
    """Chain verification with a one-hot (prompt n-gram lookup) draft; `temperatures` [B] gives
    each request its own T.  See spec_verify.h."""
    return _chain_like(True, target_logits, None, draft_tokens, r, u, temperature, workspace, out,
                       accept_prob, cand_tokens, pos_mass, target_probs, None, temperatures)


def spec_verify_tree_greedy(target_logits, node_tokens, parents, *, workspace=None, out=None,
                            node_argmax=None) -> dict:
    """Greedy verification of a draft tree.  See spec_verify.h."""
    lib = library()
    dev = target_logits.device
    if target_logits.dtype not in DTYPE_CODE or target_logits.dim() != 3:
        raise TypeError("target_logits must be a [B][N+1][V] float32/bfloat16/float16 tensor")
    B, N1, V = target_logits.shape
    _need(target_logits, "target_logits", None, (B, N1, V), dev)
    _need(node_tokens, "node_tokens", torch.int32, (B, N1), dev)
    _need(parents, "parents", torch.int32, (B, N1), dev)
    if workspace is None:
        workspace = make_workspace(B, N1, V, target_logits.dtype, dev)
    out = dict(out or {})
    al = _out(out.get("accept_len"), "accept_len", torch.int32, (B,), dev)
    pn = _out(out.get("path_nodes"), "path_nodes", torch.int32, (B, N1), dev)
    ot = _out(out.get("out_tokens"), "out_tokens", torch.int32, (B, N1), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    am = _opt(node_argmax, "node_argmax", torch.int32, (B, N1), dev)
    st = lib.spec_verify_tree_greedy(_ptr(target_logits), DTYPE_CODE[target_logits.dtype], B, N1 - 1,
                                     V, _ptr(node_tokens), _ptr(parents), _ptr(al), _ptr(pn),
                                     _ptr(ot), _ptr(ef), _ptr(am), _ptr(workspace),
                                     workspace.numel(), _stream(dev))
    _check(st)
    return dict(accept_len=al, path_nodes=pn, out_tokens=ot, err_flags=ef)


def spec_verify_tree_walk(target_logits, draft_logits, node_tokens, parents, r, u, temperature, *,
                          out=None, accept_prob=None, temperatures=None) -> dict:
    """Verification of a draft tree by walking it (stochastic for T > 0, greedy for T == 0),
    reading only the visited rows; `temperatures` [B] gives each request its own T.  See
    spec_verify.h."""
    lib = library()
    dev = target_logits.device
    if target_logits.dtype not in DTYPE_CODE or target_logits.dim() != 3:
        raise TypeError("target_logits must be a [B][N+1][V] float32/bfloat16/float16 tensor")
    B, N1, V = target_logits.shape
    T = float(temperature)
    _need(target_logits, "target_logits", None, (B, N1, V), dev)
    _need(node_tokens, "node_tokens", torch.int32, (B, N1), dev)
    _need(parents, "parents", torch.int32, (B, N1), dev)
    if temperatures is not None:
        _need(temperatures, "temperatures", torch.float32, (B,), dev)
    sampled = T > 0 or temperatures is not None
    if sampled:
        _need(draft_logits, "draft_logits", target_logits.dtype, (B, N1, V), dev)
        _need(r, "r", torch.float32, (B, N1), dev)
        _need(u, "u", torch.float32, (B,), dev)
    out = dict(out or {})
    al = _out(out.get("accept_len"), "accept_len", torch.int32, (B,), dev)
    pn = _out(out.get("path_nodes"), "path_nodes", torch.int32, (B, N1), dev)
    ot = _out(out.get("out_tokens"), "out_tokens", torch.int32, (B, N1), dev)
    rm = _out(out.get("residual_mass"), "residual_mass", torch.float32, (B,), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    ap = _opt(accept_prob, "accept_prob", torch.float32, (B, N1), dev)
    st = lib.spec_verify_tree_walk(_ptr(target_logits), _ptr(draft_logits) if sampled else None,
                                   DTYPE_CODE[target_logits.dtype], B, N1 - 1, V, T, _ptr(temperatures),
                                   _ptr(node_tokens), _ptr(parents), _ptr(r) if sampled else None,
                                   _ptr(u) if sampled else None, _ptr(al), _ptr(pn), _ptr(ot),
                                   _ptr(rm), _ptr(ef), _ptr(ap), _stream(dev))
    _check(st)
    return dict(accept_len=al, path_nodes=pn, out_tokens=ot, residual_mass=rm, err_flags=ef)


def spec_ngram_draft(context, context_len, K: int, *, n_max: int = 4, n_min: int = 1, out=None) -> dict:
    """Prompt n-gram lookup drafts of B contexts [B][Lmax] (int32) with lengths [B].  See
    spec_verify.h."""
    lib = library()
    dev = context.device
    if context.dim() != 2:
        raise ValueError("context must be [B][Lmax]")
    B, Lmax = context.shape
    _need(context, "context", torch.int32, (B, Lmax), dev)
    _need(context_len, "context_len", torch.int32, (B,), dev)
    out = dict(out or {})
    d = _out(out.get("draft_tokens"), "draft_tokens", torch.int32, (B, K), dev)
    dl = _out(out.get("draft_len"), "draft_len", torch.int32, (B,), dev)
    mn = _out(out.get("match_n"), "match_n", torch.int32, (B,), dev)
    me = _out(out.get("match_end"), "match_end", torch.int32, (B,), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    st = lib.spec_ngram_draft(_ptr(context), _ptr(context_len), B, Lmax, n_max, n_min, K, _ptr(d),
                              _ptr(dl), _ptr(mn), _ptr(me), _ptr(ef), _stream(dev))
    _check(st)
    return dict(draft_tokens=d, draft_len=dl, match_n=mn, match_end=me, err_flags=ef)


def spec_kv_compact(caches, slots, parents, accept_len, path_nodes, *, err_flags=None) -> torch.Tensor:
    """Moves the accepted path's KV rows into the request's first slots, in place, in every cache
    of `caches` (CUDA tensors whose first dimension is the slot).  See spec_verify.h."""
    lib = library()
    caches = list(caches)
    if not caches:
        raise ValueError("no caches")
    dev = caches[0].device
    S = caches[0].shape[0]
    row = caches[0].numel() // max(S, 1) * caches[0].element_size()
    for i, c in enumerate(caches):
        if c.device != dev or c.shape[0] != S or not c.is_contiguous():
            raise ValueError(f"cache {i}: every cache must be contiguous on {dev} with {S} slots")
        if c.numel() // max(S, 1) * c.element_size() != row:
            raise ValueError(f"cache {i}: rows of {row} bytes expected")
    B, N1 = slots.shape
    for name, t, shp in (("slots", slots, (B, N1)), ("parents", parents, (B, N1)), ("accept_len", accept_len, (B,)),
                         ("path_nodes", path_nodes, (B, N1))):
        _need(t, name, torch.int32, shp, dev)
    ef = _out(err_flags, "err_flags", torch.int32, (B,), dev)
    arr = (c_void_p * len(caches))(*[c.data_ptr() for c in caches])
    st = lib.spec_kv_compact(arr, len(caches), S, row, B, N1 - 1, _ptr(slots), _ptr(parents), _ptr(accept_len),
                             _ptr(path_nodes), _ptr(ef), _stream(dev))
    _check(st)
    return ef


# The current device, and a device's current stream as an address: what torch.cuda's functions of these names wrap
# in objects, which would be a tenth of a small call's time on the host.
_current_device = torch._C._cuda_getDevice if hasattr(torch._C, "_cuda_getDevice") else torch.cuda.current_device
_current_stream = getattr(torch._C, "_cuda_getCurrentRawStream", None) or (lambda i: torch.cuda.current_stream(i).cuda_stream)


_PLAIN = frozenset((int, float, type(None)))  # (an isinstance of Tensor that fails takes 0.1 us)


def _call(fn, device, *args) -> None:
    """fn(*args, the current stream of `device`) with `device` current, its status checked.  Tensors among
    the arguments become their addresses."""
    args = [a if type(a) in _PLAIN else a.data_ptr() if isinstance(a, Tensor) else a for a in args]
    index = device.index
    if index == _current_device():
        status = fn(*args, _current_stream(index))
    else:
        with torch.cuda.device(device):
            status = fn(*args, _current_stream(index))
    if status != SPEC_OK:
        _check(status)


def _cuda(t, name: str):
    if not isinstance(t, torch.Tensor):
        raise TypeError(f"{name} must be a torch tensor")
    if not t.is_cuda:
        raise ValueError(f"{name} must be on a CUDA device, got {t.device}")
    return t.device


def spec_logits_process(logits, *, history=None, history_len=None, prompt_len=None, draft_tokens=None,
                        node_tokens=None, parents=None, repetition=None, presence=None, frequency=None,
                        bias_tokens=None, bias_values=None, allowed=None, out=None) -> dict:
    """Penalties, biases and grammar masks on the logits rows [B][R][V] of a draft chain
    (`draft_tokens` [B][R-1]) or tree (`node_tokens`, `parents` [B][R]).  out["logits"] may be
    `logits` itself (in place).  See spec_verify.h."""
    lib = library()
    dev = _cuda(logits, "logits")
    if logits.dtype not in DTYPE_CODE or logits.dim() != 3:
        raise TypeError("logits must be a [B][R][V] float32/bfloat16/float16 tensor")
    B, R, V = logits.shape
    _need(logits, "logits", logits.dtype, (B, R, V), dev)
    i32, f32 = torch.int32, torch.float32
    Lmax = 0
    if history is not None:
        if not isinstance(history, torch.Tensor) or history.dim() != 2:
            raise ValueError("history must be a [B][Lmax] tensor")
        Lmax = history.shape[1]
        _need(history, "history", i32, (B, Lmax), dev)
        _need(history_len, "history_len", i32, (B,), dev)
    elif history_len is not None or prompt_len is not None:
        raise ValueError("history_len and prompt_len need a history")
    if prompt_len is not None:
        _need(prompt_len, "prompt_len", i32, (B,), dev)
    if draft_tokens is not None and node_tokens is not None:
        raise ValueError("give draft_tokens (a chain) or node_tokens and parents (a tree), not both")
    if (node_tokens is None) != (parents is None):
        raise ValueError("node_tokens and parents go together")
    if draft_tokens is not None:
        _need(draft_tokens, "draft_tokens", i32, (B, R - 1), dev)
    if node_tokens is not None:
        _need(node_tokens, "node_tokens", i32, (B, R), dev)
    if parents is not None:
        _need(parents, "parents", i32, (B, R), dev)
    if repetition is not None:
        _need(repetition, "repetition", f32, (B,), dev)
    if presence is not None:
        _need(presence, "presence", f32, (B,), dev)
    if frequency is not None:
        _need(frequency, "frequency", f32, (B,), dev)
    nb = 0
    if (bias_tokens is None) != (bias_values is None):
        raise ValueError("bias_tokens and bias_values go together")
    if bias_tokens is not None:
        if not isinstance(bias_tokens, torch.Tensor) or bias_tokens.dim() != 2:
            raise ValueError("bias_tokens must be a [B][num_biases] tensor")
        nb = bias_tokens.shape[1]
        _need(bias_tokens, "bias_tokens", i32, (B, nb), dev)
        _need(bias_values, "bias_values", f32, (B, nb), dev)
    if allowed is not None:
        _need(allowed, "allowed", i32, (B, R, (V + 31) // 32), dev)
    out = out or {}
    o = _out(out.get("logits"), "out logits", logits.dtype, (B, R, V), dev)
    ef = _out(out.get("err_flags"), "err_flags", i32, (B,), dev)
    a, z, n = logits.data_ptr(), o.data_ptr(), logits.numel() * logits.element_size()
    if a != z and a < z + n and z < a + n:
        raise ValueError("out logits must be logits itself or not overlap it")
    _call(lib.spec_logits_process, dev, logits, DTYPE_CODE[logits.dtype], B, R, V, history,
          history_len, prompt_len, Lmax, draft_tokens, node_tokens, parents,
          repetition, presence, frequency, bias_tokens, bias_values, nb,
          allowed, o, ef)
    return dict(logits=o, err_flags=ef)


def _sampling(logits, temperatures, top_k, top_p, min_p):
    """Checks what spec_sample and spec_logits_filter share; returns the device and B, R, V."""
    dev = _cuda(logits, "logits")
    if logits.dtype not in DTYPE_CODE or logits.dim() != 3:
        raise TypeError("logits must be a [B][R][V] float32/bfloat16/float16 tensor")
    if not logits.is_contiguous():
        raise ValueError("logits must be contiguous")
    B, R, V = logits.shape
    if temperatures is not None:
        _need(temperatures, "temperatures", torch.float32, (B,), dev)
    if top_k is not None:
        _need(top_k, "top_k", torch.int32, (B,), dev)
    if top_p is not None:
        _need(top_p, "top_p", torch.float32, (B,), dev)
    if min_p is not None:
        _need(min_p, "min_p", torch.float32, (B,), dev)
    return dev, B, R, V


def spec_sample(logits, u, temperature: float = 1.0, *, temperatures=None, top_k=None, top_p=None, min_p=None, out=None) -> dict:
    """Draws a token from each row of logits [B][R][V] with the uniforms u [B][R], under a temperature (each
    request's own with `temperatures` [B]) and the rules top_k, top_p, min_p [B].  Returns tokens, probs (each
    token's probability among those kept), kept (their number) and err_flags, all [B][R].  See spec_verify.h."""
    lib = library()
    dev, B, R, V = _sampling(logits, temperatures, top_k, top_p, min_p)
    _need(u, "u", torch.float32, (B, R), dev)
    out = out or {}
    tokens = _out(out.get("tokens"), "tokens", torch.int32, (B, R), dev)
    probs = _out(out.get("probs"), "probs", torch.float32, (B, R), dev)
    kept = _out(out.get("kept"), "kept", torch.int32, (B, R), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B, R), dev)
    _call(lib.spec_sample, dev, logits, DTYPE_CODE[logits.dtype], B, R, V, float(temperature), temperatures, top_k, top_p, min_p, u,
          tokens, probs, kept, ef)
    return dict(tokens=tokens, probs=probs, kept=kept, err_flags=ef)


def spec_logits_filter(logits, temperature: float = 1.0, *, temperatures=None, top_k=None, top_p=None, min_p=None, out=None) -> dict:
    """The rows of logits [B][R][V] with -inf for the tokens that spec_sample would never draw under the same
    temperature and rules; verifying rows filtered so, target and draft alike, is lossless against sampling under
    them.  The rows go to out["logits"], which may be logits itself.  Returns logits, kept and err_flags [B][R].
    See spec_verify.h."""
    lib = library()
    dev, B, R, V = _sampling(logits, temperatures, top_k, top_p, min_p)
    out = out or {}
    o = _out(out.get("logits"), "out logits", logits.dtype, (B, R, V), dev)
    a, b, n = o.data_ptr(), logits.data_ptr(), logits.numel() * logits.element_size()
    if a != b and a < b + n and b < a + n:
        raise ValueError("out logits must be logits itself or not overlap it")
    kept = _out(out.get("kept"), "kept", torch.int32, (B, R), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B, R), dev)
    _call(lib.spec_logits_filter, dev, logits, DTYPE_CODE[logits.dtype], B, R, V, float(temperature), temperatures, top_k, top_p, min_p,
          o, kept, ef)
    return dict(logits=o, kept=kept, err_flags=ef)


def _kv_caches(k_cache, v_cache, k_scale, v_scale, dtype, dev):
    """Checks a pair of caches [..., H, D] (slots, or pages and rows, in front); returns slots, H, D."""
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() not in (3, 4):
        raise ValueError("k_cache must be [num_slots][H][D] or [num_pages][page_size][H][D]")
    if k_cache.dtype not in (dtype, E4M3):
        raise TypeError(f"the caches must be {dtype} or {E4M3}, got {k_cache.dtype}")
    shape, code = k_cache.shape, k_cache.dtype
    _need(k_cache, "k_cache", code, shape, dev)
    _need(v_cache, "v_cache", code, shape, dev)
    if code is E4M3:
        rows = shape[:-1]
        _need(k_scale, "k_scale", torch.float32, rows, dev)
        _need(v_scale, "v_scale", torch.float32, rows, dev)
    elif k_scale is not None or v_scale is not None:
        raise ValueError("scales belong to e4m3 caches")
    return shape[0] * shape[1] if len(shape) == 4 else shape[0], shape[-2], shape[-1]


def _token_stride(t, name: str, B: int, T: int, H: int, D: int, dev) -> int:
    """Elements between consecutive tokens of a [B][T][H][D] tensor whose rows H D are contiguous
    (a slice of a fused projection, say)."""
    if t.device != dev:
        raise ValueError(f"{name} must be on {dev}, got {t.device}")
    if t.numel() == 0:
        return H * D
    s = t.stride()
    stride = s[1] if T > 1 else s[0] if B > 1 else H * D
    if (D > 1 and s[3] != 1) or (H > 1 and s[2] != D) or (B > 1 and s[0] != T * stride) or stride < H * D:
        raise ValueError(f"{name} must hold its tokens at one stride and each token's heads contiguously")
    return stride


def spec_kv_write(k, v, k_cache, v_cache, slots, *, k_scale=None, v_scale=None, err_flags=None) -> torch.Tensor:
    """Writes K and V rows [B][T][H][D] into the cache slots `slots` [B][T], quantised when the caches
    are float8_e4m3fn (then with scales).  Returns err_flags [B].  See spec_verify.h."""
    lib = library()
    dev = _cuda(k, "k")
    if k.dtype not in DTYPE_CODE or k.dim() != 4:
        raise TypeError("k must be a [B][T][H][D] float32/bfloat16/float16 tensor")
    B, T, H, D = k.shape
    if not isinstance(v, torch.Tensor) or v.dtype != k.dtype or v.shape != k.shape:
        raise ValueError("v must have k's shape and dtype")
    ks, vs = _token_stride(k, "k", B, T, H, D, dev), _token_stride(v, "v", B, T, H, D, dev)
    S, Hc, Dc = _kv_caches(k_cache, v_cache, k_scale, v_scale, k.dtype, dev)
    if (Hc, Dc) != (H, D):
        raise ValueError(f"the caches hold {Hc} heads of {Dc}, k and v {H} of {D}")
    _need(slots, "slots", torch.int32, (B, T), dev)
    ef = _out(err_flags, "err_flags", torch.int32, (B,), dev)
    _call(lib.spec_kv_write, dev, k, v, DTYPE_CODE[k.dtype], ks, vs, B, T, H, D, slots,
          k_cache, v_cache, CACHE_CODE[k_cache.dtype], k_scale, v_scale, S, ef)
    return ef


def spec_kv_read(k_cache, v_cache, slots, dtype, *, k_scale=None, v_scale=None, out=None) -> dict:
    """The rows of the cache slots `slots` [B][T] as `dtype` [B][T][H][D].  See spec_verify.h."""
    lib = library()
    dev = _cuda(k_cache, "k_cache")
    if dtype not in DTYPE_CODE:
        raise TypeError("dtype must be float32, bfloat16 or float16")
    S, H, D = _kv_caches(k_cache, v_cache, k_scale, v_scale, dtype, dev)
    if not isinstance(slots, torch.Tensor) or slots.dim() != 2:
        raise ValueError("slots must be a [B][T] tensor")
    B, T = slots.shape
    _need(slots, "slots", torch.int32, (B, T), dev)
    out = out or {}
    ko = _out(out.get("k"), "out k", dtype, (B, T, H, D), dev)
    vo = _out(out.get("v"), "out v", dtype, (B, T, H, D), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    _call(lib.spec_kv_read, dev, k_cache, v_cache, CACHE_CODE[k_cache.dtype], k_scale, v_scale,
          S, B, T, H, D, slots, ko, vo, DTYPE_CODE[dtype], ef)
    return dict(k=ko, v=vo, err_flags=ef)


def rope_inv_freq(rotary_dim: int, base: float = 10000.0, *, scaling: str | None = None, factor: float = 1.0,
                  original_len: int = 8192, fast: float = 32.0, slow: float = 1.0, device=None):
    """Angles a position of the rotary_dim / 2 pairs, base^(-2 i / rotary_dim), as float32, and the factor on
    cosines and sines, for spec_rope_kv_write.  `scaling` stretches them to contexts `factor` times as long:
    "linear" divides every angle by it (Chen et al., arXiv:2306.15595); "base" raises the base so that the
    slowest angle alone is divided by all of it; "parts" divides the angles that turn at most `slow` times in
    original_len positions, keeps those that turn `fast` times or more, ramps in between, and has the
    factor 0.1 ln(factor) + 1 (Peng et al., arXiv:2309.00071).  It ramps over the turns, as that paper writes it; a
    checkpoint served with a ramp over the pairs' numbers between two rounded bounds has other angles in between, and those are
    to be passed to spec_rope_kv_write as they are."""
    if rotary_dim < 2 or rotary_dim % 2:
        raise ValueError("rotary_dim must be even and at least 2")
    if not (base > 0 and factor >= 1):
        raise ValueError("base must be positive and factor at least 1")
    i = torch.arange(0, rotary_dim, 2, dtype=torch.float64)
    if scaling == "base" and rotary_dim > 2:
        base = base * factor ** (rotary_dim / (rotary_dim - 2))
    f = base ** (-i / rotary_dim)
    mult = 1.0
    if scaling == "linear":
        f = f / factor
    elif scaling == "parts":
        if not fast > slow:
            raise ValueError("fast must be above slow")
        keep = ((original_len * f / (2 * math.pi) - slow) / (fast - slow)).clamp(0, 1)
        f = f * keep + f / factor * (1 - keep)
        mult = 0.1 * math.log(factor) + 1.0
    elif scaling not in (None, "base"):
        raise ValueError("scaling must be None, 'linear', 'base' or 'parts'")
    return f.to(device=device, dtype=torch.float32), mult


def _rows_meet(n: int, a: int, sa: int, la: int, b: int, sb: int, lb: int, size: int) -> bool:
    """Whether n rows of la elements from address a, sa elements apart, share a byte with n of lb from b, sb apart: exact for
    equal strides (slices of one buffer), else whether the whole ranges meet."""
    if n == 0 or b >= a + ((n - 1) * sa + la) * size or a >= b + ((n - 1) * sb + lb) * size:
        return False
    d = (b - a) % (sa * size)
    return sa != sb or d < la * size or d + lb * size > sa * size


def spec_rope_kv_write(k, v, k_cache, v_cache, slots, inv_freq, *, q=None, positions=None, context_len=None, parents=None,
                       interleaved=False, factor=1.0, k_scale=None, v_scale=None, out=None) -> dict:
    """Rotates q [B][T][Hq][D] (when given) and k [B][T][H][D] to their positions and writes k and v into the
    cache slots `slots` [B][T], as spec_kv_write.  inv_freq [R / 2] float32: the angles of the first R
    elements' pairs (see rope_inv_freq).  Positions: `positions` [B][T], or context_len [B] + the token's
    place in the chunk, or its depth in the tree `parents` [B][T].  The rotated q goes to out["q"], which
    may be q itself if k and v lie apart from it.  See spec_verify.h."""
    lib = library()
    dev = _cuda(k, "k")
    dtype, shape = k.dtype, k.shape
    if dtype not in DTYPE_CODE or len(shape) != 4:
        raise TypeError("k must be a [B][T][H][D] float32/bfloat16/float16 tensor")
    B, T, H, D = shape
    if not isinstance(v, Tensor) or v.dtype is not dtype or v.shape != shape:
        raise ValueError("v must have k's shape and dtype")
    ks, vs = _token_stride(k, "k", B, T, H, D, dev), _token_stride(v, "v", B, T, H, D, dev)
    S, Hc, Dc = _kv_caches(k_cache, v_cache, k_scale, v_scale, dtype, dev)
    if Hc != H or Dc != D:
        raise ValueError(f"the caches hold {Hc} heads of {Dc}, k and v {H} of {D}")
    _need(slots, "slots", torch.int32, (B, T), dev)
    if not isinstance(inv_freq, Tensor) or inv_freq.dim() != 1:
        raise ValueError("inv_freq must hold between 1 and D / 2 angles")
    angles = inv_freq.numel()
    if not 1 <= angles <= D // 2:
        raise ValueError("inv_freq must hold between 1 and D / 2 angles")
    _need(inv_freq, "inv_freq", torch.float32, (angles,), dev)
    if (positions is None) == (context_len is None):
        raise ValueError("give positions or context_len, one of them")
    if positions is not None:
        _need(positions, "positions", torch.int32, (B, T), dev)
        if parents is not None:
            raise ValueError("parents go with context_len")
    else:
        _need(context_len, "context_len", torch.int32, (B,), dev)
    if parents is not None:
        _need(parents, "parents", torch.int32, (B, T), dev)
    out = out or {}
    Hq, qs, qo, os_ = 0, 0, out.get("q"), 0
    if q is not None:
        if not isinstance(q, Tensor) or q.dtype is not dtype or q.dim() != 4:
            raise ValueError("q must be [B][T][Hq][D] of k's dtype")
        Bq, Tq, Hq, Dq = shape = q.shape
        if Bq != B or Tq != T or Dq != D or Hq < 1:
            raise ValueError("q must be [B][T][Hq][D] of k's dtype")
        qs = _token_stride(q, "q", B, T, Hq, D, dev)
        if qo is None:
            qo = torch.empty((B, T, Hq, D), dtype=dtype, device=dev)
            os_ = Hq * D
        else:
            if not isinstance(qo, Tensor) or qo.dtype is not dtype or qo.shape != shape:
                raise ValueError("out q must have q's shape and dtype")
            os_ = _token_stride(qo, "out q", B, T, Hq, D, dev)
            # from the first byte to behind the last: a of the output, c of q, e of k, f of v
            size, last, a, c, e, f = 4 if dtype is torch.float32 else 2, B * T - 1, qo.data_ptr(), q.data_ptr(), k.data_ptr(), v.data_ptr()
            b, row, kv = a + (last * os_ + Hq * D) * size, Hq * D, H * D
            if (c < b and a < c + (last * qs + row) * size and (a != c or os_ != qs) and _rows_meet(last + 1, a, os_, row, c, qs, row, size)
                    or e < b and a < e + (last * ks + kv) * size and _rows_meet(last + 1, a, os_, row, e, ks, kv, size)
                    or f < b and a < f + (last * vs + kv) * size and _rows_meet(last + 1, a, os_, row, f, vs, kv, size)):
                raise ValueError("out q must be q itself, with k and v apart, or overlap no input")
    elif qo is not None:
        raise ValueError("out q needs q")
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    _call(lib.spec_rope_kv_write, dev, q, k, v, DTYPE_CODE[dtype], qs, ks, vs, B, T, Hq, H, D, inv_freq, 2 * angles,
          int(bool(interleaved)), float(factor), positions, context_len, parents, slots, qo, os_, k_cache, v_cache,
          CACHE_CODE[k_cache.dtype], k_scale, v_scale, S, ef)
    return dict(q=qo, err_flags=ef)


def attention_workspace_bytes(T: int, num_heads: int, num_kv_heads: int, head_dim: int) -> int:
    """Workspace bytes of a spec_attention call with chunks of T tokens (any number of requests)."""
    return int(library().spec_attention_workspace_bytes(T, num_heads, num_kv_heads, head_dim))


def make_attention_workspace(T: int, num_heads: int, num_kv_heads: int, head_dim: int, device) -> torch.Tensor:
    """A workspace for such calls; concurrent calls need one each."""
    n = max(256, attention_workspace_bytes(T, num_heads, num_kv_heads, head_dim))
    return torch.empty(n, dtype=torch.uint8, device=device)


def spec_attention(q, k_cache, v_cache, page_table, context_len, *, chunk_len=None, parents=None, scale=None,
                   k_scale=None, v_scale=None, workspace=None, out=None, lse=None) -> dict:
    """Attention of the chunk q [B][T][Hq][D] over the paged caches [num_pages][page_size][H][D]:
    the prefix of context_len[b] tokens, then the chunk (causal, or by the tree `parents` [B][T]).
    `scale` is 1 / sqrt(D) unless given; `lse` [B][T][Hq] float32 receives the log-sum-exp.  See
    spec_verify.h."""
    lib = library()
    dev = _cuda(q, "q")
    if q.dtype not in (torch.bfloat16, torch.float16) or q.dim() != 4:
        raise TypeError("q must be a [B][T][Hq][D] bfloat16/float16 tensor")
    B, T, Hq, D = q.shape
    qs = _token_stride(q, "q", B, T, Hq, D, dev)
    if not isinstance(k_cache, torch.Tensor) or k_cache.dim() != 4:
        raise ValueError("k_cache must be [num_pages][page_size][H][D]")
    _, H, Dc = _kv_caches(k_cache, v_cache, k_scale, v_scale, q.dtype, dev)
    if Dc != D or H < 1 or Hq % H != 0:
        raise ValueError(f"{Hq} query heads of {D} do not fit {H} KV heads of {Dc}")
    if not isinstance(page_table, torch.Tensor) or page_table.dim() != 2:
        raise ValueError("page_table must be a [B][pages_per_request] tensor")
    P = page_table.shape[1]
    _need(page_table, "page_table", torch.int32, (B, P), dev)
    _need(context_len, "context_len", torch.int32, (B,), dev)
    if chunk_len is not None:
        _need(chunk_len, "chunk_len", torch.int32, (B,), dev)
    if parents is not None:
        _need(parents, "parents", torch.int32, (B, T), dev)
    if lse is not None:
        _need(lse, "lse", torch.float32, (B, T, Hq), dev)
    if workspace is None:
        workspace = make_attention_workspace(T, Hq, H, D, dev)
    elif not isinstance(workspace, torch.Tensor) or workspace.device != dev or not workspace.is_contiguous():
        raise ValueError(f"workspace must be a contiguous tensor on {dev}")
    out = out or {}
    o = _out(out.get("out"), "out", q.dtype, (B, T, Hq, D), dev)
    ef = _out(out.get("err_flags"), "err_flags", torch.int32, (B,), dev)
    _call(lib.spec_attention, dev, q, DTYPE_CODE[q.dtype], qs, B, T, Hq, H, D, k_cache, v_cache,
          CACHE_CODE[k_cache.dtype], k_scale, v_scale, k_cache.shape[0], k_cache.shape[1], page_table,
          P, context_len, chunk_len, parents, max(D, 1) ** -0.5 if scale is None else float(scale), o,
          lse, ef, workspace, workspace.numel() * workspace.element_size())
    return dict(out=o, lse=lse, err_flags=ef)
