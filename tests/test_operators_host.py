"""Argument checks of the operators around verification: the C ABI on the host before any launch
(placeholder device addresses, so only where no GPU is visible), and the binding's own."""

import ctypes

import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding
from speculative_decoding_verification_82_gb300.build import build

host_only = pytest.mark.skipif(torch.cuda.is_available(), reason="placeholder device addresses: run without a GPU")
P = ctypes.c_void_p
OK, BAD, WORKSPACE, UNSUPPORTED = binding.SPEC_OK, binding.SPEC_ERR_INVALID_ARG, binding.SPEC_ERR_WORKSPACE, binding.SPEC_ERR_UNSUPPORTED


@pytest.fixture(scope="module")
def lib():
    build()
    return binding.library()


@host_only
def test_logits_process(lib):
    ok = dict(x=1 << 20, dt=1, B=2, R=4, V=100, h=2 << 20, hl=3 << 20, pl=0, Lmax=9, d=4 << 20, n=0, p=0, rep=0, pre=0, fr=0, bt=5 << 20,
              bv=6 << 20, nb=3, al=0, o=7 << 20)

    def f(**kw):
        a = dict(ok, **kw)
        return lib.spec_logits_process(P(a["x"]), a["dt"], a["B"], a["R"], a["V"], P(a["h"]), P(a["hl"]), P(a["pl"]), a["Lmax"], P(a["d"]),
                                       P(a["n"]), P(a["p"]), P(a["rep"]), P(a["pre"]), P(a["fr"]), P(a["bt"]), P(a["bv"]), a["nb"],
                                       P(a["al"]), P(a["o"]), None, None)

    assert f(B=0) == OK
    for kw in (dict(dt=3), dict(dt=9), dict(B=-1), dict(R=0), dict(V=0), dict(Lmax=-1), dict(nb=-1), dict(x=0), dict(o=0), dict(h=0), dict(hl=0),
               dict(n=8 << 20, p=9 << 20), dict(d=0, n=8 << 20), dict(d=0, p=8 << 20), dict(bt=0), dict(bv=0), dict(x=(1 << 20) + 1),
               dict(o=(7 << 20) + 1), dict(dt=0, x=(1 << 20) + 2)):
        assert f(**kw) == BAD, kw
    for kw in (dict(R=binding.MAX_LOGITS_ROWS + 1), dict(nb=binding.MAX_BIASES + 1), dict(B=65536), dict(V=2**31 - 1)):
        assert f(**kw) == UNSUPPORTED, kw


@host_only
def test_kv_write_and_read(lib):
    ok = dict(k=1 << 20, v=2 << 20, dt=1, sk=1024, sv=1024, B=2, T=3, H=8, D=128, sl=3 << 20, kc=4 << 20, vc=5 << 20, cdt=3, ks=6 << 20,
              vs=7 << 20, S=100)

    def w(**kw):
        a = dict(ok, **kw)
        return lib.spec_kv_write(P(a["k"]), P(a["v"]), a["dt"], a["sk"], a["sv"], a["B"], a["T"], a["H"], a["D"], P(a["sl"]), P(a["kc"]),
                                 P(a["vc"]), a["cdt"], P(a["ks"]), P(a["vs"]), a["S"], None, None)

    def r(**kw):
        a = dict(ok, **kw)
        return lib.spec_kv_read(P(a["kc"]), P(a["vc"]), a["cdt"], P(a["ks"]), P(a["vs"]), a["S"], a["B"], a["T"], a["H"], a["D"], P(a["sl"]),
                                P(a["k"]), P(a["v"]), a["dt"], None, None)

    for f in (w, r):
        assert f(B=0) == OK and f(T=0) == OK
        for kw in (dict(dt=3), dict(dt=7), dict(cdt=0), dict(cdt=2), dict(B=-1), dict(T=-1), dict(H=0), dict(D=0), dict(S=-1), dict(sl=0),
                   dict(k=0), dict(v=0), dict(kc=0), dict(vc=0), dict(ks=0), dict(vs=0), dict(k=(1 << 20) + 8), dict(kc=(4 << 20) + 8),
                   dict(ks=(6 << 20) + 2)):
            assert f(**kw) == BAD, kw
        for kw in (dict(D=12), dict(D=264), dict(S=2**31), dict(B=2**20, T=2**20), dict(B=2**20, T=2**8)):
            assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(sk=1000), dict(sk=1028), dict(sv=1023), dict(sk=2**62)):
        assert w(**kw) == BAD, kw


@host_only
def test_attention(lib):
    ok = dict(q=1 << 20, dt=1, sq=1024, B=2, T=6, Hq=8, H=2, D=128, kc=2 << 20, vc=3 << 20, cdt=3, ks=4 << 20, vs=5 << 20, np=10, ps=16,
              pt=6 << 20, P=4, cl=7 << 20, ch=0, par=0, sc=0.1, o=8 << 20, ws=1 << 30, wsb=1 << 40)

    def f(**kw):
        a = dict(ok, **kw)
        return lib.spec_attention(P(a["q"]), a["dt"], a["sq"], a["B"], a["T"], a["Hq"], a["H"], a["D"], P(a["kc"]), P(a["vc"]), a["cdt"],
                                  P(a["ks"]), P(a["vs"]), a["np"], a["ps"], P(a["pt"]), a["P"], P(a["cl"]), P(a["ch"]), P(a["par"]),
                                  a["sc"], P(a["o"]), None, None, P(a["ws"]), a["wsb"], None)

    assert f(B=0) == OK and f(T=0) == OK
    for kw in (dict(dt=3), dict(dt=-1), dict(cdt=2), dict(cdt=0), dict(B=-1), dict(T=-1), dict(Hq=0), dict(H=0), dict(Hq=7), dict(np=-1),
               dict(ps=0), dict(P=-1), dict(sc=0.0), dict(sc=-1.0), dict(sc=float("nan")), dict(sc=float("inf")), dict(q=0), dict(kc=0),
               dict(vc=0), dict(pt=0), dict(cl=0), dict(o=0), dict(ks=0), dict(vs=0), dict(q=(1 << 20) + 8), dict(kc=(2 << 20) + 8),
               dict(vc=(3 << 20) + 8), dict(o=(8 << 20) + 8), dict(sq=1000), dict(sq=1028)):
        assert f(**kw) == BAD, kw
    for kw in (dict(dt=0), dict(D=96), dict(D=256), dict(ps=4), dict(ps=24), dict(np=2**31), dict(B=65536), dict(par=9 << 20, T=1025)):
        assert f(**kw) == UNSUPPORTED, kw
    for kw in (dict(ws=0), dict(ws=(1 << 30) + 16), dict(wsb=100)):
        assert f(**kw) == WORKSPACE, kw


def test_attention_workspace_size(lib):
    f = lib.spec_attention_workspace_bytes
    assert f(6, 64, 8, 128) >= 256
    for bad in ((0, 64, 8, 128), (6, 0, 8, 128), (6, 64, 0, 128), (6, 60, 8, 128), (6, 64, 8, 96)):
        assert f(*bad) == 0, bad


def test_the_binding_refuses_before_the_library():
    """What the binding itself checks: kinds, devices, shapes and pairs of arguments."""
    x = torch.zeros((2, 3, 50))
    with pytest.raises(ValueError, match="CUDA device"):
        binding.spec_logits_process(x)
    with pytest.raises(TypeError):
        binding.spec_logits_process(None)
    kv = torch.zeros((2, 3, 1, 64), dtype=torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.spec_kv_write(kv, kv, kv[0], kv[0], torch.zeros((2, 3), dtype=torch.int32))
    with pytest.raises(ValueError, match="CUDA device"):
        binding.spec_kv_read(kv[0], kv[0], torch.zeros((2, 3), dtype=torch.int32), torch.bfloat16)
    with pytest.raises(ValueError, match="CUDA device"):
        binding.spec_attention(kv, kv, kv, torch.zeros((2, 3), dtype=torch.int32), torch.zeros(2, dtype=torch.int32))


@pytest.mark.gpu
def test_the_binding_refuses_what_does_not_fit():
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    i32 = lambda *s: torch.zeros(s, dtype=torch.int32, device="cuda")  # noqa: E731
    x = torch.zeros((2, 3, 50), device="cuda")
    for kw in (dict(history=i32(2, 4)), dict(history_len=i32(2)), dict(draft_tokens=i32(2, 3)), dict(node_tokens=i32(2, 3)),
               dict(parents=i32(2, 3)), dict(draft_tokens=i32(2, 2), node_tokens=i32(2, 3), parents=i32(2, 3)), dict(allowed=i32(2, 3, 1)),
               dict(repetition=torch.ones(3, device="cuda")), dict(repetition=torch.ones(2)), dict(bias_tokens=i32(2, 2)),
               dict(allowed=i32(2, 3, 4)[..., ::2])):
        with pytest.raises((TypeError, ValueError)):
            binding.spec_logits_process(x, **kw)
    buf = torch.zeros(2 * 3 * 50 + 8, device="cuda")
    with pytest.raises(ValueError, match="overlap"):
        binding.spec_logits_process(buf[:300].view(2, 3, 50), out=dict(logits=buf[8:308].view(2, 3, 50)))
    k = torch.zeros((2, 3, 2, 64), dtype=torch.bfloat16, device="cuda")
    c = torch.zeros((9, 2, 64), dtype=torch.bfloat16, device="cuda")
    c8 = torch.zeros((9, 2, 64), dtype=torch.uint8, device="cuda").view(binding.E4M3)
    s = torch.zeros((9, 2), device="cuda")
    for args, kw in (((k, k[:, :2], c, c, i32(2, 3)), {}), ((k, k, c, c8, i32(2, 3)), {}), ((k, k, c8, c8, i32(2, 3)), {}),
                     ((k, k, c, c, i32(2, 3)), dict(k_scale=s, v_scale=s)), ((k, k, c, c, i32(3, 2)), {}),
                     ((k, k, c[:, :1], c[:, :1], i32(2, 3)), {}), ((k.transpose(1, 2).contiguous().transpose(1, 2), k, c, c, i32(2, 3)), {}),
                     ((k, k, c8, c8, i32(2, 3)), dict(k_scale=s, v_scale=s[:8])), ((k.float(), k.float(), c, c, i32(2, 3)), {})):
        with pytest.raises((TypeError, ValueError)):
            binding.spec_kv_write(*args, **kw)
    q = torch.zeros((2, 3, 4, 64), dtype=torch.bfloat16, device="cuda")
    p = torch.zeros((5, 8, 2, 64), dtype=torch.bfloat16, device="cuda")
    for args, kw in (((q.float(), p, p, i32(2, 3), i32(2)), {}), ((q, c, c, i32(2, 3), i32(2)), {}), ((q[:, :, :3], p, p, i32(2, 3), i32(2)), {}),
                     ((q, p, p, i32(3, 3), i32(2)), {}), ((q, p, p, i32(2, 3), i32(3)), {}), ((q, p, p, i32(2, 3), i32(2)), dict(parents=i32(2, 4))),
                     ((q.half(), p, p, i32(2, 3), i32(2)), {}), ((q, p, p, i32(2, 3), i32(2)), dict(workspace=torch.zeros(4)))):
        with pytest.raises((TypeError, ValueError)):
            binding.spec_attention(*args, **kw)
    with pytest.raises(binding.SpecVerifyError):
        binding.spec_attention(q, p, p, i32(2, 3), i32(2), workspace=torch.zeros(16, device="cuda"))
