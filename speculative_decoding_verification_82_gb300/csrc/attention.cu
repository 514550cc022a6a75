// attention.cu -- spec_attention's C entry: argument checks, tensor maps, workspace layout, launch.
//
// Host side only; the kernels live in attention_kernel.cuh (instantiated per element type in
// attention_{bf16,f16}.cu).  No call allocates memory or synchronises the host.
#include <cuda.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include <atomic>

#include "attention_kernel.cuh"
#include "device_info.h"
#include "spec_verify.h"

namespace specv {
namespace attn {
extern template cudaError_t launch_attention<__nv_bfloat16>(const Params&, int, bool, bool, int, cudaStream_t);
extern template cudaError_t launch_attention<__half>(const Params&, int, bool, bool, int, cudaStream_t);
}  // namespace attn
}  // namespace specv

namespace {

using specv::attn::kMaxCtas;
using specv::attn::kTile;
using specv::attn::Params;
using specv::attn::Record;

// Rows of a unit of work: one row tile while a request's rows fit it, else two.
int unit_rows(long long rows) { return rows > kTile ? 2 * kTile : kTile; }

// Workspace: the partial results' O, their m and l, and the records, in 256-byte aligned regions.
struct Layout {
  size_t o, ml, rec, total;
};
Layout layout(long long rows, int D) {
  const size_t UR = (size_t)unit_rows(rows), parts = 2 * (size_t)kMaxCtas;
  Layout L;
  L.o = 0;
  L.ml = L.o + parts * UR * (size_t)D * 4;
  L.rec = L.ml + parts * UR * 8;
  L.total = (L.rec + kMaxCtas * sizeof(Record) + 255) / 256 * 256;
  return L;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*, const cuuint64_t*,
                                 const cuuint32_t*, const cuuint32_t*, CUtensorMapInterleave, CUtensorMapSwizzle,
                                 CUtensorMapL2promotion, CUtensorMapFloatOOBfill);
EncodeTiled encode_tiled() {
  static std::atomic<void*> f{nullptr};
  void* p = f.load();
  if (!p) {
    cudaDriverEntryPointQueryResult q;
    if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &p, 12000, cudaEnableDefault, &q) != cudaSuccess ||
        q != cudaDriverEntryPointSuccess)
      return nullptr;
    f.store(p);
  }
  return reinterpret_cast<EncodeTiled>(p);
}

// A cache [pages][page_size][H][D] as a 4-dimensional map; a box is one page's rows (at most a tile's) of one
// head: all of its bytes for codes, 64 elements at a time for 16 bits.
bool cache_map(CUtensorMap* m, const void* cache, bool e4m3, bool bf16, int D, int H, int page_size, long long pages) {
  const EncodeTiled f = encode_tiled();
  if (!f) return false;
  const cuuint64_t S = e4m3 ? 1 : 2;
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)H, (cuuint64_t)page_size, (cuuint64_t)(pages > 0 ? pages : 1)};
  const cuuint64_t strides[3] = {D * S, (cuuint64_t)H * D * S, (cuuint64_t)page_size * H * D * S};
  const cuuint32_t box[4] = {(cuuint32_t)(e4m3 ? D : 64), 1, (cuuint32_t)(page_size < kTile ? page_size : kTile), 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return f(m, e4m3 ? CU_TENSOR_MAP_DATA_TYPE_UINT8 : bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4,
           const_cast<void*>(cache), dims, strides, box, step, CU_TENSOR_MAP_INTERLEAVE_NONE,
           e4m3 && D == 64 ? CU_TENSOR_MAP_SWIZZLE_64B : CU_TENSOR_MAP_SWIZZLE_128B, e4m3 ? CU_TENSOR_MAP_L2_PROMOTION_L2_128B : CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// The queries [B][T][Hq][D] (tokens q_stride elements apart) as a 4-dimensional map; a box is 64 elements of one
// KV head's G query heads, for `tokens` tokens.
bool query_map(CUtensorMap* m, const void* q, bool bf16, int D, int Hq, int G, int T, int B, long long q_stride, int tokens) {
  const EncodeTiled f = encode_tiled();
  if (!f || q_stride >= (1LL << 38) / T) return false;  // (strides below 2^40 bytes)
  const cuuint64_t dims[4] = {(cuuint64_t)D, (cuuint64_t)Hq, (cuuint64_t)T, (cuuint64_t)B};
  const cuuint64_t strides[3] = {(cuuint64_t)D * 2, (cuuint64_t)q_stride * 2, (cuuint64_t)T * (cuuint64_t)q_stride * 2};
  const cuuint32_t box[4] = {64, (cuuint32_t)G, (cuuint32_t)tokens, 1};
  const cuuint32_t step[4] = {1, 1, 1, 1};
  return f(m, bf16 ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16, 4, const_cast<void*>(q), dims, strides, box,
           step, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

}  // namespace

extern "C" size_t spec_attention_workspace_bytes(int T, int num_heads, int num_kv_heads, int head_dim) {
  if (T < 1 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128)) return 0;
  return layout((long long)T * (num_heads / num_kv_heads), head_dim).total;
}

extern "C" spec_status_t spec_attention(const void* q, spec_dtype_t dtype, long long q_stride, int B, int T,
                                        int num_heads, int num_kv_heads, int head_dim, const void* k_cache,
                                        const void* v_cache, spec_dtype_t cache_dtype, const float* k_scale,
                                        const float* v_scale, long long num_pages, int page_size,
                                        const int32_t* page_table, int pages_per_request, const int32_t* context_len,
                                        const int32_t* chunk_len, const int32_t* parents, float scale, void* out,
                                        float* lse, int32_t* err_flags, void* workspace, size_t workspace_bytes,
                                        spec_stream_t stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_INVALID_ARG;
  if (dtype == SPEC_DTYPE_F32) return SPEC_ERR_UNSUPPORTED;
  if (cache_dtype != dtype && cache_dtype != SPEC_DTYPE_E4M3) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0) return SPEC_ERR_INVALID_ARG;
  if (num_pages < 0 || page_size < 1 || pages_per_request < 0) return SPEC_ERR_INVALID_ARG;
  if (!(scale > 0.f) || isinf(scale * specv::attn::kLog2e)) return SPEC_ERR_INVALID_ARG;  // (0 times infinity is a NaN)
  if (head_dim != 64 && head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (page_size < 8 || (page_size & (page_size - 1)) != 0 || num_pages > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  if (parents && T > SPEC_MAX_WALK_NODES) return SPEC_ERR_UNSUPPORTED;
  // a request's rows and positions are counted in 32 bits
  if ((long long)T * (num_heads / num_kv_heads) > INT_MAX / 2 || (long long)pages_per_request * page_size > INT_MAX / 2)
    return SPEC_ERR_UNSUPPORTED;
  if (B > 65535) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (T == 0) {  // no tokens: nothing to check, nothing wrong
    if (err_flags && cudaMemsetAsync(err_flags, 0, (size_t)B * 4, reinterpret_cast<cudaStream_t>(stream)) != cudaSuccess)
      return SPEC_ERR_CUDA;
    return SPEC_OK;
  }
  if (!q || !k_cache || !v_cache || !page_table || !context_len || !out) return SPEC_ERR_INVALID_ARG;
  const bool e4m3 = cache_dtype == SPEC_DTYPE_E4M3;
  if (e4m3 && (!k_scale || !v_scale)) return SPEC_ERR_INVALID_ARG;
  if (((uintptr_t)q | (uintptr_t)k_cache | (uintptr_t)v_cache | (uintptr_t)out) & 15u) return SPEC_ERR_INVALID_ARG;
  if (q_stride < (long long)num_heads * head_dim || q_stride % 8 != 0) return SPEC_ERR_INVALID_ARG;
  if (!workspace || ((uintptr_t)workspace & 255u) || workspace_bytes < spec_attention_workspace_bytes(T, num_heads, num_kv_heads, head_dim))
    return SPEC_ERR_WORKSPACE;
  const int sms = specv::sm_count();
  if (sms <= 0) return SPEC_ERR_CUDA;
  const int G = num_heads / num_kv_heads;
  const long long rows = (long long)T * G;
  const int UR = unit_rows(rows);
  Params A = {};
  const bool bf16 = dtype == SPEC_DTYPE_BF16;
  if (!cache_map(&A.kmap, k_cache, e4m3, bf16, head_dim, num_kv_heads, page_size, num_pages) ||
      !cache_map(&A.vmap, v_cache, e4m3, bf16, head_dim, num_kv_heads, page_size, num_pages))
    return SPEC_ERR_CUDA;
  const Layout L = layout(rows, head_dim);
  unsigned char* w = static_cast<unsigned char*>(workspace);
  A.part_o = reinterpret_cast<float*>(w + L.o);
  A.part_ml = reinterpret_cast<float2*>(w + L.ml);
  A.rec = reinterpret_cast<Record*>(w + L.rec);
  A.q = static_cast<const unsigned char*>(q);
  A.ks = k_scale;
  A.vs = v_scale;
  A.q_stride = q_stride;
  A.num_pages = num_pages;
  A.B = B;
  A.T = T;
  A.Hq = num_heads;
  A.H = num_kv_heads;
  A.G = G;
  A.P = pages_per_request;
  while ((1 << A.page_log2) < page_size) ++A.page_log2;
  A.nqp = (int)((rows + UR - 1) / UR);
  if ((long long)B * A.nqp > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  A.fd_g = specv::make_fastdiv((uint32_t)G);
  A.fd_nqp = specv::make_fastdiv((uint32_t)A.nqp);
  // a tile of query rows (64 rows where they all fit) is whole tokens: one box
  const int qrows = rows <= 64 ? 64 : kTile;
  if (qrows % G == 0) {
    const int tokens = qrows / G < T ? qrows / G : T;
    if (query_map(&A.qmap, q, bf16, head_dim, num_heads, G, T, B, q_stride, tokens)) A.q_box = tokens;
  }
  A.table = page_table;
  A.context_len = context_len;
  A.chunk_len = chunk_len;
  A.parents = parents;
  A.c = scale * specv::attn::kLog2e;
  A.out = static_cast<unsigned char*>(out);
  A.lse = lse;
  A.err_flags = err_flags;
  // Units of a request side by side where there are two or four.  (bf16 chunks of 8 heads a KV head over 8192 positions, one
  // after the other / side by side: 2 units 170 / 172 us, 4 units 309 / 294, 16 units 301 / 313.  Three and five to eight
  // would gain 3 to 4% as well: 243 / 233, 298 / 287.)
  int ctas = sms < kMaxCtas ? sms : kMaxCtas;
  A.lanes = (A.nqp == 2 || A.nqp == 4) && ctas >= A.nqp ? A.nqp : 1;
  ctas -= ctas % A.lanes;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const bool pair = UR > kTile;
  const cudaError_t e = bf16 ? specv::attn::launch_attention<__nv_bfloat16>(A, head_dim, e4m3, pair, ctas, s)
                             : specv::attn::launch_attention<__half>(A, head_dim, e4m3, pair, ctas, s);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
