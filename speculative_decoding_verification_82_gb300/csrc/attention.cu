// attention.cu -- spec_attention: attention of a chunk of new tokens over a paged KV cache (sm_103a).
//
// One warp per (token, head): the online softmax over the prefix, then over the token's own path in
// the chunk, one position at a time.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "spec_verify.h"

namespace {

constexpr int kWarps = 8;

struct AttnParams {
  const unsigned char *q, *kc, *vc;
  const float *ks, *vs;
  long long q_stride, num_pages;
  int B, T, Hq, H, page_size, P;
  const int32_t *table, *context_len, *chunk_len, *parents;
  float scale;
  unsigned char* out;
  float* lse;
  int32_t* err_flags;
};

template <typename T>
__device__ float to_f(T v);
template <>
__device__ float to_f(__nv_bfloat16 v) { return __bfloat162float(v); }
template <>
__device__ float to_f(__half v) { return __half2float(v); }
template <typename T>
__device__ T from_f(float v);
template <>
__device__ __nv_bfloat16 from_f(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __half from_f(float v) { return __float2half_rn(v); }
__device__ __forceinline__ float e4m3(uint8_t c) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)c));
  return __low2float(*reinterpret_cast<const __half2*>(&h));
}

template <typename T, int D, bool E4M3>
__global__ void __launch_bounds__(kWarps * 32) attention_kernel(const AttnParams A) {
  constexpr int N = D / 32;
  const int b = blockIdx.y, lane = threadIdx.x & 31;
  const long long L = __ldg(A.context_len + b);
  const int n = A.chunk_len ? __ldg(A.chunk_len + b) : A.T;
  int flags = 0;
  if (L < 0 || n < 0 || n > A.T || L + n > (long long)A.P * A.page_size) flags |= SPEC_ERRF_BAD_LENGTH;
  const int32_t* par = A.parents ? A.parents + (size_t)b * A.T : nullptr;
  bool bad = false;
  if (par && !flags)
    for (int i = threadIdx.x; i < n; i += blockDim.x) {
      const int p = __ldg(par + i);
      bad = bad || (i == 0 ? p != -1 : (p < 0 || p >= i));
    }
  if (__syncthreads_or(bad)) flags |= SPEC_ERRF_BAD_TREE;
  const bool failed = flags != 0;
  if (blockIdx.x == 0 && A.err_flags) {
    bool slot = false;
    if (!failed)
      for (long long j = threadIdx.x; j < (L + n + A.page_size - 1) / A.page_size; j += blockDim.x) {
        const int p = __ldg(A.table + (size_t)b * A.P + j);
        slot = slot || p < 0 || p >= A.num_pages;
      }
    if (__syncthreads_or(slot)) flags |= SPEC_ERRF_BAD_SLOT;
    if (threadIdx.x == 0) A.err_flags[b] = flags;
  }
  const int G = A.Hq / A.H;
  for (long long i = (long long)blockIdx.x * kWarps + threadIdx.x / 32; i < (long long)A.T * A.Hq; i += (long long)gridDim.x * kWarps) {
    const int t = (int)(i / A.Hq), h = (int)(i % A.Hq);
    if (!failed && t >= n) continue;
    const int kh = h / G;
    const size_t o = (((size_t)b * A.T + t) * A.Hq + h) * D;
    float q[N], acc[N], m = -INFINITY, l = 0.f;
    const T* qp = reinterpret_cast<const T*>(A.q) + ((long long)b * A.T + t) * A.q_stride + (size_t)h * D;
    for (int d = 0; d < N; ++d) {
      q[d] = failed ? 0.f : to_f(qp[d * 32 + lane]) * A.scale;
      acc[d] = 0.f;
    }
    auto attend = [&](long long j) {
      const int page = __ldg(A.table + (size_t)b * A.P + j / A.page_size);
      const bool ok = page >= 0 && page < A.num_pages;
      const size_t r = ok ? ((size_t)page * A.page_size + j % A.page_size) * A.H + kh : 0;
      float k[N], v[N], s = 0.f;
      for (int d = 0; d < N; ++d) {
        const size_t at = r * D + d * 32 + lane;
        if (!ok) {
          k[d] = v[d] = 0.f;
        } else if constexpr (E4M3) {
          k[d] = e4m3(A.kc[at]) * A.ks[r];
          v[d] = e4m3(A.vc[at]) * A.vs[r];
        } else {
          k[d] = to_f(reinterpret_cast<const T*>(A.kc)[at]);
          v[d] = to_f(reinterpret_cast<const T*>(A.vc)[at]);
        }
        s = fmaf(q[d], k[d], s);
      }
      for (int x = 16; x; x >>= 1) s += __shfl_xor_sync(0xffffffffu, s, x);
      const float mn = fmaxf(m, s);
      const float a = m == -INFINITY ? 0.f : __expf(m - mn), p = s == -INFINITY ? 0.f : __expf(s - mn);
      l = l * a + p;
      for (int d = 0; d < N; ++d) acc[d] = acc[d] * a + p * v[d];
      m = mn;
    };
    if (!failed) {
      for (long long j = 0; j < L; ++j) attend(j);
      if (par)
        for (int x = t; x >= 0; x = __ldg(par + x)) attend(L + x);
      else
        for (int x = 0; x <= t; ++x) attend(L + x);
    }
    for (int d = 0; d < N; ++d)
      reinterpret_cast<T*>(A.out)[o + d * 32 + lane] = from_f<T>(l == 0.f ? 0.f : acc[d] / l);
    if (A.lse && lane == 0) A.lse[o / D] = l == 0.f ? -INFINITY : m + logf(l);
  }
}

template <typename T, int D>
spec_status_t launch(const AttnParams& A, bool e4m3, cudaStream_t s) {
  const long long rows = (long long)A.T * A.Hq;
  const long long blocks = (rows + kWarps - 1) / kWarps;
  const dim3 grid((unsigned)(blocks < 65536 ? blocks : 65536), A.B);
  if (e4m3)
    attention_kernel<T, D, true><<<grid, kWarps * 32, 0, s>>>(A);
  else
    attention_kernel<T, D, false><<<grid, kWarps * 32, 0, s>>>(A);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" size_t spec_attention_workspace_bytes(int T, int num_heads, int num_kv_heads, int head_dim) {
  if (T < 1 || num_heads < 1 || num_kv_heads < 1 || num_heads % num_kv_heads != 0 || (head_dim != 64 && head_dim != 128)) return 0;
  return 256;
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
  if (!(scale > 0.f) || isinf(scale)) return SPEC_ERR_INVALID_ARG;
  if (head_dim != 64 && head_dim != 128) return SPEC_ERR_UNSUPPORTED;
  if (page_size < 8 || (page_size & (page_size - 1)) != 0 || num_pages > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  if (parents && T > SPEC_MAX_WALK_NODES) return SPEC_ERR_UNSUPPORTED;
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
  AttnParams A = {};
  A.q = static_cast<const unsigned char*>(q);
  A.kc = static_cast<const unsigned char*>(k_cache);
  A.vc = static_cast<const unsigned char*>(v_cache);
  A.ks = k_scale;
  A.vs = v_scale;
  A.q_stride = q_stride;
  A.num_pages = num_pages;
  A.B = B;
  A.T = T;
  A.Hq = num_heads;
  A.H = num_kv_heads;
  A.page_size = page_size;
  A.P = pages_per_request;
  A.table = page_table;
  A.context_len = context_len;
  A.chunk_len = chunk_len;
  A.parents = parents;
  A.scale = scale;
  A.out = static_cast<unsigned char*>(out);
  A.lse = lse;
  A.err_flags = err_flags;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SPEC_DTYPE_BF16)
    return head_dim == 64 ? launch<__nv_bfloat16, 64>(A, e4m3, s) : launch<__nv_bfloat16, 128>(A, e4m3, s);
  return head_dim == 64 ? launch<__half, 64>(A, e4m3, s) : launch<__half, 128>(A, e4m3, s);
}
