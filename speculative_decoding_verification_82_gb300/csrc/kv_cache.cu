// kv_cache.cu -- spec_kv_write and spec_kv_read: K and V rows into their cache slots, quantised to
// e4m3 where the cache is, and back (sm_103a).
//
// Quantisation of one row x (a token's D elements of one KV head): with a = max |x| over the finite
// elements, the scale is s = 2^e, e = ceil(log2(a / 448)), and the codes are e4m3(x / s).  With
// a = f 2^n, f in [1/2, 1), and 448 = 0.875 * 2^9, e is n - 9 if f <= 0.875 and n - 8 otherwise:
// integer arithmetic on a's bits.  Multiplying by 2^-e is exact, so each code has one rounding, and
// code * s is exact in 32 and in bf16 bits.  A power of two costs up to one of e4m3's 17 binades
// against a / 448 and no precision above the subnormal codes.
//
// Both kernels stream every byte once and are bound by HBM bandwidth, or by launch latency for a
// draft tree's few rows.  A row belongs to the smallest power of two of lanes that covers it with 16 (8 where
// head_dim asks for it) elements each, 8 lanes for 128, so its maximum is a few shuffles and every lane moves
// whole 16-byte vectors of codes; a thread has two rows in flight.  (One row and 8 elements a thread:
// 46 us where this takes 36 on 16 x 2052 tokens of 8 heads of 128 read to bf16, 15.5 where this takes 12.2
// on 4 x 2048 f16 tokens written.)
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>
#include <stdint.h>

#include "fastdiv.h"
#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;
constexpr int kRowsPerThread = 2;

struct KvRows {
  const unsigned char* src[2];  // write: k, v rows; read: the caches
  unsigned char* dst[2];        // write: the caches; read: k, v rows
  const float* scale_in[2];     // read: the scales
  float* scale_out[2];          // write: the scales
  long long stride[2];          // write: bytes between tokens of k, v
  const int32_t* slots;         // [B][T]
  int32_t* err_flags;           // [B] or null
  long long num_slots;
  unsigned rows;                // tokens * 2 * heads
  int B, T, H, D;
  int lanes_log2;               // lanes per row
  specv::FastDiv fd_2h;         // rows of one token (K heads, then V heads)
};

// 8 elements of a row (their words) as floats, and back.
template <typename T>
struct Vec8;
template <>
struct Vec8<float> {
  static constexpr int kBytes = 32;
  __device__ static void unpack(const uint32_t* w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __uint_as_float(w[i]);
  }
  __device__ static void store(unsigned char* p, const float (&f)[8]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(f[0], f[1], f[2], f[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(f[4], f[5], f[6], f[7]);
  }
};
template <>
struct Vec8<__nv_bfloat16> {
  static constexpr int kBytes = 16;
  __device__ static void unpack(const uint32_t* w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      f[2 * i] = __uint_as_float(w[i] << 16);
      f[2 * i + 1] = __uint_as_float(w[i] & 0xffff0000u);
    }
  }
  __device__ static void store(unsigned char* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __nv_bfloat162 h = __floats2bfloat162_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};
template <>
struct Vec8<__half> {
  static constexpr int kBytes = 16;
  __device__ static void unpack(const uint32_t* w, float (&f)[8]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = __half22float2(*reinterpret_cast<const __half2*>(&w[i]));
      f[2 * i] = t.x;
      f[2 * i + 1] = t.y;
    }
  }
  __device__ static void store(unsigned char* p, const float (&f)[8]) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const __half2 h = __floats2half2_rn(f[2 * i], f[2 * i + 1]);
      w[i] = *reinterpret_cast<const uint32_t*>(&h);
    }
    *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
  }
};

// e in [-126, 120]: the smallest with a <= 448 * 2^e (a finite, >= 0).
__device__ __forceinline__ int scale_exponent(float a) {
  const uint32_t u = __float_as_uint(a);
  const int e = (int)(u >> 23) - 135 + ((u & 0x7fffffu) > 0x600000u ? 1 : 0);
  return e < -126 ? -126 : e;
}
__device__ __forceinline__ float pow2f_int(int e) { return __uint_as_float((uint32_t)(e + 127) << 23); }

__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
  return r;
}
__device__ __forceinline__ float2 from_e4m3x2(uint32_t two) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"((uint16_t)two));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}

// The u-th row of this thread: a block's rows are consecutive, kThreads / lanes of them for each u.
template <int E>
__device__ __forceinline__ unsigned row_of(const KvRows& P, int u) {
  const unsigned per = (unsigned)kThreads >> P.lanes_log2;
  return (unsigned)min((uint64_t)P.rows, ((uint64_t)blockIdx.x * kRowsPerThread + u) * per + (threadIdx.x >> P.lanes_log2));
}

// Sets err_flags of the requests this block looks after: whether a slot is outside [-1, num_slots).
__device__ void check_slots(const KvRows& P) {
  if (!P.err_flags) return;
  for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
    bool bad = false;
    for (int t = threadIdx.x; t < P.T; t += kThreads) {
      const int s = __ldg(P.slots + (size_t)b * P.T + t);
      bad = bad || s < -1 || s >= P.num_slots;
    }
    bad = __syncthreads_or(bad);
    if (threadIdx.x == 0) P.err_flags[b] = bad ? SPEC_ERRF_BAD_SLOT : 0;
  }
}

// E: elements of a row per lane.  QUANT: the cache is e4m3; otherwise rows are copied bit for bit.
template <typename T, int E, bool QUANT>
__global__ void __launch_bounds__(kThreads) kv_write_kernel(const KvRows P) {
  constexpr int S = Vec8<T>::kBytes / 8;  // bytes of an element
  const unsigned lanes = 1u << P.lanes_log2;
  const int e0 = (int)(threadIdx.x & (lanes - 1)) * E;
  const bool in = e0 < P.D;
  constexpr int W = E * S / 4;  // words of a lane's elements
  size_t at[kRowsPerThread];    // the row in the cache
  int kv[kRowsPerThread];       // 0 K, 1 V, -1 nothing to write
  uint32_t raw[kRowsPerThread][W];
#pragma unroll
  for (int u = 0; u < kRowsPerThread; ++u) {
    const unsigned row = row_of<E>(P, u);
    kv[u] = -1;
    if (row >= P.rows) continue;  // rows never straddle warps: a row's lanes stay together
    const unsigned n = specv::fdiv(row, P.fd_2h);
    int h = (int)(row - n * P.fd_2h.d);
    const long long slot = __ldg(P.slots + n);
    if (slot < 0 || slot >= P.num_slots) continue;
    kv[u] = h >= P.H ? 1 : 0;
    h -= kv[u] ? P.H : 0;
    const unsigned char* src = P.src[kv[u]] + (long long)n * P.stride[kv[u]] + ((size_t)h * P.D + e0) * S;
    at[u] = (size_t)slot * P.H + h;
#pragma unroll
    for (int i = 0; i < W; i += 4) {
      const uint4 v = in ? __ldcs(reinterpret_cast<const uint4*>(src + i * 4)) : make_uint4(0, 0, 0, 0);
      raw[u][i] = v.x, raw[u][i + 1] = v.y, raw[u][i + 2] = v.z, raw[u][i + 3] = v.w;
    }
  }
#pragma unroll
  for (int u = 0; u < kRowsPerThread; ++u) {
    if (kv[u] < 0) continue;
    if constexpr (QUANT) {
      float x[E];
#pragma unroll
      for (int i = 0; i < E; i += 8) Vec8<T>::unpack(raw[u] + i * S / 4, reinterpret_cast<float(&)[8]>(x[i]));
      float a = 0.f;
#pragma unroll
      for (int i = 0; i < E; ++i) {
        const float m = fabsf(x[i]);
        a = fmaxf(a, m < INFINITY ? m : 0.f);
      }
      const unsigned group = (lanes == 32 ? 0xffffffffu : ((1u << lanes) - 1u)) << ((threadIdx.x & 31) & ~(lanes - 1));
      for (unsigned o = lanes >> 1; o; o >>= 1) a = fmaxf(a, __shfl_xor_sync(group, a, o));
      const int e = scale_exponent(a);
      const float inv = pow2f_int(-e);
      uint32_t c[E / 4];
#pragma unroll
      for (int i = 0; i < E / 4; ++i) {
        float y[4];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          y[z] = x[4 * i + z] * inv;
          y[z] = fabsf(y[z]) <= 448.f ? y[z] : NAN;  // infinities (finite elements are within 448)
        }
        c[i] = e4m3x2(y[0], y[1]) | (e4m3x2(y[2], y[3]) << 16);
      }
      if (in) {
        unsigned char* dst = P.dst[kv[u]] + at[u] * P.D + e0;
        if constexpr (E == 16)
          *reinterpret_cast<uint4*>(dst) = make_uint4(c[0], c[1], c[2], c[3]);
        else
          *reinterpret_cast<uint2*>(dst) = make_uint2(c[0], c[1]);
      }
      if (e0 == 0) P.scale_out[kv[u]][at[u]] = pow2f_int(e);
    } else if (in) {
      uint4* d = reinterpret_cast<uint4*>(P.dst[kv[u]] + (at[u] * P.D + e0) * S);
#pragma unroll
      for (int i = 0; i < W / 4; ++i) d[i] = make_uint4(raw[u][4 * i], raw[u][4 * i + 1], raw[u][4 * i + 2], raw[u][4 * i + 3]);
    }
  }
  check_slots(P);
}

template <typename T, int E, bool QUANT>
__global__ void __launch_bounds__(kThreads) kv_read_kernel(const KvRows P) {
  constexpr int S = Vec8<T>::kBytes / 8;
  constexpr int W = QUANT ? E / 4 : E * S / 4;  // words a lane reads
  const unsigned lanes = 1u << P.lanes_log2;
  const int e0 = (int)(threadIdx.x & (lanes - 1)) * E;
  unsigned char* dst[kRowsPerThread];
  bool does[kRowsPerThread];
  uint32_t w[kRowsPerThread][W];
  float scale[kRowsPerThread];
#pragma unroll
  for (int u = 0; u < kRowsPerThread; ++u) {
    const unsigned row = row_of<E>(P, u);
    does[u] = row < P.rows && e0 < P.D;
    scale[u] = 0.f;
#pragma unroll
    for (int i = 0; i < W; ++i) w[u][i] = 0;
    if (!does[u]) continue;
    const unsigned n = specv::fdiv(row, P.fd_2h);
    int h = (int)(row - n * P.fd_2h.d);
    const int kv = h >= P.H ? 1 : 0;
    h -= kv ? P.H : 0;
    dst[u] = P.dst[kv] + (((size_t)n * P.H + h) * P.D + e0) * S;
    const long long slot = __ldg(P.slots + n);
    if (slot < 0 || slot >= P.num_slots) continue;
    const size_t r = (size_t)slot * P.H + h;
    const unsigned char* src = P.src[kv] + (r * P.D + e0) * (QUANT ? 1 : S);
    if constexpr (W == 2) {
      const uint2 v = __ldcs(reinterpret_cast<const uint2*>(src));
      w[u][0] = v.x, w[u][1] = v.y;
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i) {
        const uint4 v = __ldcs(reinterpret_cast<const uint4*>(src) + i);
        w[u][4 * i] = v.x, w[u][4 * i + 1] = v.y, w[u][4 * i + 2] = v.z, w[u][4 * i + 3] = v.w;
      }
    }
    if (QUANT) scale[u] = __ldg(P.scale_in[kv] + r);
  }
#pragma unroll
  for (int u = 0; u < kRowsPerThread; ++u) {
    if (!does[u]) continue;
    if constexpr (QUANT) {
#pragma unroll
      for (int i = 0; i < E; i += 8) {
        float x[8];
#pragma unroll
        for (int z = 0; z < 4; ++z) {
          const float2 f = from_e4m3x2(w[u][i / 4 + z / 2] >> (16 * (z & 1)));
          x[2 * z] = f.x * scale[u];
          x[2 * z + 1] = f.y * scale[u];
        }
        Vec8<T>::store(dst[u] + i * S, x);
      }
    } else {
#pragma unroll
      for (int i = 0; i < W / 4; ++i)
        reinterpret_cast<uint4*>(dst[u])[i] = make_uint4(w[u][4 * i], w[u][4 * i + 1], w[u][4 * i + 2], w[u][4 * i + 3]);
    }
  }
  check_slots(P);
}

int elem_bytes(spec_dtype_t t) { return t == SPEC_DTYPE_F32 ? 4 : t == SPEC_DTYPE_E4M3 ? 1 : 2; }
int lane_elems(int D) { return D % 16 == 0 ? 16 : 8; }
bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }

// Checks shared by both calls; `done`: nothing to do.
spec_status_t plan(KvRows& P, spec_dtype_t dtype, spec_dtype_t cache, int B, int T, int H, int D, const int32_t* slots,
                   long long num_slots, int32_t* err_flags, const void* a, const void* b, const void* c, const void* d,
                   const float* ks, const float* vs, bool* done) {
  *done = false;
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_INVALID_ARG;
  if (cache != dtype && cache != SPEC_DTYPE_E4M3) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || H < 1 || D < 1 || num_slots < 0) return SPEC_ERR_INVALID_ARG;
  if (D % 8 != 0 || D > SPEC_MAX_KV_HEAD_DIM) return SPEC_ERR_UNSUPPORTED;
  if (num_slots > INT_MAX) return SPEC_ERR_UNSUPPORTED;  // a slot is an int32
  const long long tokens = (long long)B * T;
  if (H > (INT_MAX / 2) || tokens > INT_MAX || tokens * 2 * H > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) {
    *done = true;
    return SPEC_OK;
  }
  if (T > 0 && (!slots || !a || !b || !c || !d)) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(a) || !aligned16(b) || !aligned16(c) || !aligned16(d)) return SPEC_ERR_INVALID_ARG;
  if (T > 0 && cache == SPEC_DTYPE_E4M3) {
    if (!ks || !vs || ((uintptr_t)ks & 3u) || ((uintptr_t)vs & 3u)) return SPEC_ERR_INVALID_ARG;
  }
  if (T == 0 && !err_flags) {
    *done = true;
    return SPEC_OK;
  }
  P.slots = slots;
  P.err_flags = err_flags;
  P.num_slots = num_slots;
  P.rows = (unsigned)(tokens * 2 * H);
  P.B = B;
  P.T = T;
  P.H = H;
  P.D = D;
  P.lanes_log2 = 0;
  while ((lane_elems(D) << P.lanes_log2) < D) ++P.lanes_log2;
  P.fd_2h = specv::make_fastdiv((unsigned)(2 * H));
  return SPEC_OK;
}

unsigned grid_of(const KvRows& P) {
  const uint64_t per = ((uint64_t)kThreads >> P.lanes_log2) * kRowsPerThread;
  const uint64_t blocks = (P.rows + per - 1) / per;
  return blocks ? (unsigned)blocks : 1u;
}

// One of the two kernels, for elements of type T.
template <typename T, bool WRITE, bool QUANT>
void launch(const KvRows& P, cudaStream_t s) {
  const unsigned grid = grid_of(P);
  if (lane_elems(P.D) == 16) {
    if (WRITE)
      kv_write_kernel<T, 16, QUANT><<<grid, kThreads, 0, s>>>(P);
    else
      kv_read_kernel<T, 16, QUANT><<<grid, kThreads, 0, s>>>(P);
  } else {
    if (WRITE)
      kv_write_kernel<T, 8, QUANT><<<grid, kThreads, 0, s>>>(P);
    else
      kv_read_kernel<T, 8, QUANT><<<grid, kThreads, 0, s>>>(P);
  }
}
template <bool WRITE>
spec_status_t launch_any(const KvRows& P, spec_dtype_t dtype, bool quant, cudaStream_t s) {
  if (dtype == SPEC_DTYPE_F32)
    quant ? launch<float, WRITE, true>(P, s) : launch<float, WRITE, false>(P, s);
  else if (dtype == SPEC_DTYPE_BF16 && quant)
    launch<__nv_bfloat16, WRITE, true>(P, s);
  else if (quant)
    launch<__half, WRITE, true>(P, s);
  else  // 16-bit rows are copied whatever they hold
    launch<__half, WRITE, false>(P, s);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" spec_status_t spec_kv_write(const void* k, const void* v, spec_dtype_t dtype, long long k_stride,
                                       long long v_stride, int B, int T, int num_kv_heads, int head_dim,
                                       const int32_t* slots, void* k_cache, void* v_cache, spec_dtype_t cache_dtype,
                                       float* k_scale, float* v_scale, long long num_slots, int32_t* err_flags,
                                       spec_stream_t stream) {
  KvRows P = {};
  bool done;
  const spec_status_t st = plan(P, dtype, cache_dtype, B, T, num_kv_heads, head_dim, slots, num_slots, err_flags, k, v,
                                k_cache, v_cache, k_scale, v_scale, &done);
  if (st != SPEC_OK || done) return st;
  const int S = elem_bytes(dtype);
  const long long row = (long long)num_kv_heads * head_dim;
  if (T > 0 && (k_stride < row || v_stride < row || k_stride > LLONG_MAX / 4 || v_stride > LLONG_MAX / 4 ||
                (k_stride * S) % 16 != 0 || (v_stride * S) % 16 != 0))
    return SPEC_ERR_INVALID_ARG;
  P.src[0] = static_cast<const unsigned char*>(k);
  P.src[1] = static_cast<const unsigned char*>(v);
  P.dst[0] = static_cast<unsigned char*>(k_cache);
  P.dst[1] = static_cast<unsigned char*>(v_cache);
  P.scale_out[0] = k_scale;
  P.scale_out[1] = v_scale;
  P.stride[0] = k_stride * S;
  P.stride[1] = v_stride * S;
  return launch_any<true>(P, dtype, cache_dtype == SPEC_DTYPE_E4M3, reinterpret_cast<cudaStream_t>(stream));
}

extern "C" spec_status_t spec_kv_read(const void* k_cache, const void* v_cache, spec_dtype_t cache_dtype,
                                      const float* k_scale, const float* v_scale, long long num_slots, int B, int T,
                                      int num_kv_heads, int head_dim, const int32_t* slots, void* k_out, void* v_out,
                                      spec_dtype_t dtype, int32_t* err_flags, spec_stream_t stream) {
  KvRows P = {};
  bool done;
  const spec_status_t st = plan(P, dtype, cache_dtype, B, T, num_kv_heads, head_dim, slots, num_slots, err_flags, k_out,
                                v_out, k_cache, v_cache, k_scale, v_scale, &done);
  if (st != SPEC_OK || done) return st;
  P.src[0] = static_cast<const unsigned char*>(k_cache);
  P.src[1] = static_cast<const unsigned char*>(v_cache);
  P.dst[0] = static_cast<unsigned char*>(k_out);
  P.dst[1] = static_cast<unsigned char*>(v_out);
  P.scale_in[0] = k_scale;
  P.scale_in[1] = v_scale;
  return launch_any<false>(P, dtype, cache_dtype == SPEC_DTYPE_E4M3, reinterpret_cast<cudaStream_t>(stream));
}
