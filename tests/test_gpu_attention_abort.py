"""The kernel that joins spec_attention's parts, alone, over records and parts made by hand: it passes on that a CTA gave
up waiting, to every request and over the flags that the requests have, and joins what there is as ever.  (That a
wait runs out cannot be brought about from outside.)"""

import ctypes
import os
import subprocess

import pytest
import torch

from speculative_decoding_verification_82_gb300 import binding, build

pytestmark = pytest.mark.gpu

DRIVER = r"""
#include "attention_kernel.cuh"
using namespace specv::attn;
extern "C" int record_bytes() { return sizeof(Record); }
extern "C" int gave_up() { return kGaveUp; }
// Three CTAs; request 0's one item starts in CTA 0 and ends in CTA 1.
extern "C" int join(float* part_o, float2* part_ml, Record* rec, unsigned char* out, float* lse, int* err_flags, int B, int T, int G,
                    cudaStream_t stream) {
  Params P = {};
  P.part_o = part_o, P.part_ml = part_ml, P.rec = rec, P.out = out, P.lse = lse, P.err_flags = err_flags;
  P.B = B, P.T = T, P.G = G, P.H = 1, P.Hq = G, P.nqp = 1, P.lanes = 1;
  attention_combine_kernel<__nv_bfloat16, 64><<<dim3(3, (T * G + 15) / 16), 256, 0, stream>>>(P, kTile);
  return cudaGetLastError();
}
"""


@pytest.fixture(scope="module")
def lib(tmp_path_factory):
    if not torch.cuda.is_available():
        pytest.skip("needs a CUDA GPU")
    binding.library()
    d = tmp_path_factory.mktemp("join")
    (d / "join.cu").write_text(DRIVER)
    so = d / "join.so"
    subprocess.run([build._nvcc(), *build.ARCH, *build.NVCC_FLAGS, "-I", build.INCLUDE, "-I", build.CSRC, "-shared", "-cudart", "static",
                    os.fspath(d / "join.cu"), "-o", os.fspath(so)], check=True)
    return ctypes.CDLL(os.fspath(so))


@pytest.mark.parametrize("gave_up", [(), (0,), (1,), (2,), (0, 1, 2)])
def test_who_gave_up_is_passed_on(lib, gave_up):
    B, T, G, D, tile = 700, 3, 8, 64, 128
    assert lib.record_bytes() == 16
    g = torch.Generator(device="cuda").manual_seed(5)
    o = torch.randn((6, D // 4, tile, 4), generator=g, device="cuda")  # part 2 c + 1: the item that starts in c; 2 c: that ends there
    ml = torch.rand((6, tile, 2), generator=g, device="cuda") + 1
    rec = torch.tensor([[0, 0, 0, 1], [-1, 0, 0, 0], [-1, 0, 0, 0]], dtype=torch.int32)
    rec[list(gave_up), 3] |= lib.gave_up()
    rec = rec.cuda()
    out = torch.full((B, T, G, D), 5.0, dtype=torch.bfloat16, device="cuda")
    lse = torch.full((B, T, G), 6.0, device="cuda")
    flags = torch.randint(0, 2, (B,), generator=g, device="cuda", dtype=torch.int32) * binding.ERRF_BAD_SLOT
    want = flags | (binding.ERRF_TIMEOUT if gave_up else 0)
    p = [ctypes.c_void_p(t.data_ptr()) for t in (o, ml, rec, out, lse, flags)]
    assert lib.join(*p, B, T, G, ctypes.c_void_p(torch.cuda.current_stream().cuda_stream)) == 0
    torch.cuda.synchronize()
    assert torch.equal(flags, want)
    m, l = ml[..., 0].double(), ml[..., 1].double()
    w = torch.exp2(m[[1, 2]] - m[[1, 2]].amax(0))
    total = (l[[1, 2]] * w).sum(0)
    joined = (o[[1, 2]].double() * w[:, None, :, None]).sum(0).permute(1, 0, 2).reshape(tile, D) / total[:, None]
    got = out[0].view(T * G, D).double()
    # one rounding to bf16; in 32 bits a few steps of the summed magnitudes
    size = (o[[1, 2]].double().abs() * w[:, None, :, None]).sum(0).permute(1, 0, 2).reshape(tile, D) / total[:, None]
    assert ((got - joined[: T * G]).abs() <= 2.0**-8 * joined[: T * G].abs() + 2.0**-20 * size[: T * G]).all()
    z = (m[[1, 2]].amax(0) + torch.log2(total)) * 0.6931471805599453
    assert ((lse[0].view(-1).double() - z[: T * G]).abs() <= 2.0**-20 * (1 + z[: T * G].abs())).all()
    assert (out[1:] == 5).all() and (lse[1:] == 6).all()
