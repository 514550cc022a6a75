// rope_kv.cu -- spec_rope_kv_write: queries and keys rotated to their positions, keys and values written
// into their cache slots on the way, quantised to e4m3 where the cache is (sm_103a).
//
// Mathematics.  A pair (a, b) of a head's elements at position p becomes (a c - b s, b c + a s) with
// c = f cos(p w), s = f sin(p w) for the pair's angle a position w.  p w is taken modulo a turn in 64-bit
// integers: w / 2 pi, less its whole turns, in units of 2^-64, times p, wraps where turns are whole, so that no
// position is far.  What is left of the nearest quarter turn is within an eighth of a turn and goes to
// sincospif in 32 bits; the quarters are exact.
// (32-bit products p w are off by 2^-24 p w: 0.06 rad at a million positions of angle 1.)
//
// The rows of a token are its query heads, then its K heads, then its V heads.  A row belongs to the smallest
// power of two of lanes that covers it with two 8-element vectors each.  Where elements i and i + R/2 are
// paired and R/2 is whole vectors, a lane holds vector j of either half, so both elements of its pairs;
// otherwise it holds two neighbours, which have neighbouring pairs inside, and lanes exchange partners at odd
// distances through shared memory.  A block's rows are consecutive; it computes the sines and cosines of its few tokens
// once, into shared memory, while its rows are on their way.
//
// The kernel streams every byte once and is bound by HBM bandwidth (4 x 2048 f16 tokens of 64 query and 8 KV heads of
// 128, 335 MB, in 57 us: 88% of a copy's rate; with 256 threads a block 59, four rows a thread 67, one row 65), or by
// launch latency and the dependent loads (slot, length or parents, then rows' stores) for a decode's or a tree's few
// rows (8 tokens 3.9 us, 16 trees of 61 nodes into e4m3 11.2).  Halves that are not whole vectors (100 of 128 elements) take 80 us,
// where shared memory is the bound; with partners fetched from the row one element at a time 115.
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "fastdiv.h"
#include "kv_rows.cuh"
#include "spec_verify.h"

namespace {

using specv::FastDiv;
using specv::Vec8;

constexpr int kThreads = 128;
constexpr int kRowsPerThread = 2;
constexpr int kExchange = 17;  // places of a lane's 16 elements, so that lanes' start in different banks

enum Pairs { kNext = 0, kHalf = 1, kHalfOdd = 2 };  // neighbours; halves of whole vectors; halves of any size

struct Rope {
  const unsigned char* src[3];  // q, k, v rows
  unsigned char* dst[3];        // rotated q, the caches
  float* scale[2];              // of K and V, e4m3 caches
  long long stride[3];          // bytes between tokens of q, k, v
  long long out_stride;         // bytes between tokens of the rotated q
  const int32_t *slots, *positions, *context_len, *parents;
  const float* inv_freq;
  int32_t* err_flags;
  long long num_slots;
  unsigned rows;                // tokens * (Hq + 2 H)
  float factor;
  int B, T, Hq, H, D, R;
  int lanes_log2;
  int tokens_max;               // tokens that a block's rows may belong to
  int angles;                   // places of a token's cosines (R / 2, rounded up to 4)
  FastDiv fd_t, fd_rows, fd_angles;  // T; rows of a token; angles
};

// f cos(p w), f sin(p w); p >= 0.
__device__ __forceinline__ float2 turned(long long p, float w, float f) {
  const uint32_t bits = __float_as_uint(w), exponent = bits >> 23 & 255u;
  if (exponent == 255u) return make_float2(NAN, NAN);
  // turns a position: w's 24 bits times 2^96 / 2 pi, shifted to its fraction's 64 (whole numbers: products in 64-bit floats
  // take sixteen times as long as in 32 bits, 27 us of an SM's time for a prompt of 4 x 2048 tokens)
  const uint32_t m = exponent ? (bits & 0x7fffffu) | 0x800000u : bits & 0x7fffffu, e = exponent ? exponent : 1u;
  const unsigned __int128 turns = (unsigned __int128)m * ((unsigned __int128)0x28be60dbu << 64 | 0x9391054a7f09d5f4ull);
  const uint32_t shift = 182u - e;  // (w = m 2^(e - 150); it is at most 2^24)
  const uint64_t unit = shift < 128u ? (uint64_t)(turns >> shift) : 0;
  const uint64_t turn = unit * (uint64_t)p;
  const uint32_t quarter = (uint32_t)((turn + (1ull << 61)) >> 62);
  const long long rest = (long long)(turn - ((uint64_t)quarter << 62));  // within 2^61 of zero
  float s, c;
  sincospif(__ll2float_rn(rest) * 0x1p-63f, &s, &c);  // (all of it: small angles keep their 24 bits)
  float cs = quarter & 1 ? -s : c, sn = quarter & 1 ? c : s;
  if (quarter & 2) cs = -cs, sn = -sn;
  if (w < 0.f) sn = -sn;
  return make_float2(cs * f, sn * f);
}

// Whether node i's parent is one that a tree may have.
__device__ __forceinline__ bool good_link(int i, int p) { return i == 0 ? p == -1 : p >= 0 && p < i; }

// Sets err_flags of the requests this block looks after.
__device__ void check_requests(const Rope& P) {
  if (!P.err_flags) return;
  __shared__ int end;  // behind the request's last token that has a slot
  for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
    if (threadIdx.x == 0) end = 0;
    __syncthreads();
    int flags = 0, mine = 0;
    const bool short_ctx = !P.positions && __ldg(P.context_len + b) < 0;
    for (int t = threadIdx.x; t < P.T; t += kThreads) {
      const size_t n = (size_t)b * P.T + t;
      const int s = __ldg(P.slots + n);
      if (s == -1) continue;
      mine = t + 1;
      if (s < 0 || s >= P.num_slots) flags |= SPEC_ERRF_BAD_SLOT;
      if (short_ctx || (P.positions && __ldg(P.positions + n) < 0)) flags |= SPEC_ERRF_BAD_LENGTH;
    }
    if (P.parents) {
      if (mine) atomicMax(&end, mine);
      __syncthreads();
      for (int t = threadIdx.x; t < end; t += kThreads)
        if (!good_link(t, __ldg(P.parents + (size_t)b * P.T + t))) flags |= SPEC_ERRF_BAD_TREE;
    }
    int all = 0;
#pragma unroll
    for (int f : {SPEC_ERRF_BAD_SLOT, SPEC_ERRF_BAD_LENGTH, SPEC_ERRF_BAD_TREE}) all |= __syncthreads_or(flags & f) ? f : 0;
    if (threadIdx.x == 0) P.err_flags[b] = all;
  }
}

// QUANT: the caches are e4m3; otherwise of T.
template <typename T, int PAIRS, bool QUANT>
__global__ void __launch_bounds__(kThreads) rope_kernel(const __grid_constant__ Rope P) {
  constexpr int U = kRowsPerThread, S = Vec8<T>::kBytes / 8, W = Vec8<T>::kBytes / 4;  // W: words of 8 elements
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ float exchange[PAIRS == kHalfOdd ? kThreads * kExchange : 1];
  float* cosines = reinterpret_cast<float*>(smem);             // [tokens][angles]
  float* sines = cosines + (size_t)P.tokens_max * P.angles;    // [tokens][angles]
  long long* pos = reinterpret_cast<long long*>(sines + (size_t)P.tokens_max * P.angles);  // [tokens]
  int* slot_of = reinterpret_cast<int*>(pos + P.tokens_max);   // [tokens], -1: skipped
  int16_t* par = reinterpret_cast<int16_t*>(slot_of + P.tokens_max);  // [T + tokens], -2: bad
  const int tid = threadIdx.x;
  const unsigned lanes = 1u << P.lanes_log2, j = tid & (lanes - 1), per = (unsigned)kThreads >> P.lanes_log2;
  const unsigned per_token = P.fd_rows.d;
  const unsigned row0 = blockIdx.x * (U * per);                  // (rows fit an int, and each block has some)
  const unsigned first = specv::fdiv(row0, P.fd_rows);           // the block's first token
  const unsigned tokens = specv::fdiv(min(P.rows, row0 + U * per) - 1u, P.fd_rows) - first + 1;

  // this lane's two vectors of a row
  const int half = P.R / 16;
  const bool both = PAIRS == kHalf && (int)j < half;
  const int v0 = both ? (int)j : 2 * (int)j, v1 = both ? (int)j + half : 2 * (int)j + 1;
  unsigned token[U];   // from the block's first one
  int kind[U], head[U];
  const unsigned char* src[U];
  uint32_t raw[U][2][W];
#pragma unroll
  for (int u = 0; u < U; ++u) {
    const unsigned row = row0 + u * per + (tid >> P.lanes_log2);
    kind[u] = -1;
    if (row >= P.rows) continue;
    const unsigned n = specv::fdiv(row, P.fd_rows);
    int h = (int)(row - n * per_token);
    kind[u] = h < P.Hq ? 0 : h < P.Hq + P.H ? 1 : 2;
    h -= kind[u] == 0 ? 0 : kind[u] == 1 ? P.Hq : P.Hq + P.H;
    head[u] = h;
    token[u] = n - first;
    src[u] = P.src[kind[u]] + (long long)n * P.stride[kind[u]] + (size_t)h * P.D * S;
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const int v = x ? v1 : v0;
#pragma unroll
      for (int i = 0; i < W; i += 4) {
        const uint4 w = 8 * v < P.D ? __ldcs(reinterpret_cast<const uint4*>(src[u] + (size_t)v * 8 * S + i * 4)) : make_uint4(0, 0, 0, 0);
        raw[u][x][i] = w.x, raw[u][x][i + 1] = w.y, raw[u][x][i + 2] = w.z, raw[u][x][i + 3] = w.w;
      }
    }
  }

  // the tokens' places, then their cosines and sines
  const unsigned base = specv::fdiv(first, P.fd_t) * P.T;  // the first token's request's first
  if (P.parents) {
    for (unsigned i = tid; i < first + tokens - base; i += kThreads) {
      const unsigned n = base + i;
      const int t = (int)(n - specv::fdiv(n, P.fd_t) * P.T), p = __ldg(P.parents + n);
      par[i] = good_link(t, p) ? (int16_t)p : (int16_t)-2;
    }
    __syncthreads();
  }
  for (unsigned i = tid; i < tokens; i += kThreads) {
    const unsigned n = first + i, b = specv::fdiv(n, P.fd_t);
    const int s = __ldg(P.slots + n), t = (int)(n - b * P.T);
    bool fine = s >= 0 && s < P.num_slots;
    long long p;
    if (P.positions) {
      p = __ldg(P.positions + n);
      fine = fine && p >= 0;
    } else {
      p = __ldg(P.context_len + b);
      fine = fine && p >= 0;
      if (P.parents) {
        const int16_t* pr = par + (b * P.T - base);
        for (int x = t;; ++p) {  // (a good link leads to a lower node)
          const int up = pr[x];
          if (up < 0) {
            fine = fine && up == -1;
            break;
          }
          x = up;
        }
      } else {
        p += t;
      }
    }
    pos[i] = p;
    slot_of[i] = fine ? s : -1;
  }
  __syncthreads();
  for (unsigned i = tid; i < tokens * P.angles; i += kThreads) {
    const unsigned k = specv::fdiv(i, P.fd_angles), a = i - k * P.angles;
    if (2 * (int)a >= P.R || slot_of[k] < 0) continue;
    const float2 cs = turned(pos[k], __ldg(P.inv_freq + a), P.factor);
    cosines[i] = cs.x;
    sines[i] = cs.y;
  }
  __syncthreads();

#pragma unroll
  for (int u = 0; u < U; ++u) {
    const int slot = kind[u] < 0 ? -1 : slot_of[token[u]];
    const bool does = slot >= 0;
    float x[16];
    if (does && (QUANT ? true : kind[u] < 2)) {
      Vec8<T>::unpack(raw[u][0], reinterpret_cast<float(&)[8]>(x[0]));
      Vec8<T>::unpack(raw[u][1], reinterpret_cast<float(&)[8]>(x[8]));
    }
    if (does && kind[u] < 2) {
      const float *c = cosines + (size_t)token[u] * P.angles, *s = sines + (size_t)token[u] * P.angles;
      if constexpr (PAIRS == kHalf) {
        if (both) {
#pragma unroll
          for (int z = 0; z < 8; z += 4) {
            const float4 cc = *reinterpret_cast<const float4*>(c + 8 * j + z), ss = *reinterpret_cast<const float4*>(s + 8 * j + z);
            const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
            for (int i = 0; i < 4; ++i) {
              const float a = x[z + i], b = x[8 + z + i];
              x[z + i] = fmaf(a, cv[i], -b * sv[i]);
              x[8 + z + i] = fmaf(b, cv[i], a * sv[i]);
            }
          }
        }
      } else if constexpr (PAIRS == kNext) {
#pragma unroll
        for (int y = 0; y < 2; ++y) {
          const int v = 2 * (int)j + y;
          if (8 * v >= P.R) continue;
          const float4 cc = *reinterpret_cast<const float4*>(c + 4 * v), ss = *reinterpret_cast<const float4*>(s + 4 * v);
          const float cv[4] = {cc.x, cc.y, cc.z, cc.w}, sv[4] = {ss.x, ss.y, ss.z, ss.w};
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (8 * v + 2 * i >= P.R) continue;
            const float a = x[8 * y + 2 * i], b = x[8 * y + 2 * i + 1];
            x[8 * y + 2 * i] = fmaf(a, cv[i], -b * sv[i]);
            x[8 * y + 2 * i + 1] = fmaf(b, cv[i], a * sv[i]);
          }
        }
      }
    }
    if constexpr (PAIRS == kHalfOdd) {  // through shared memory, neighbouring pairs by neighbouring lanes
      float* mine = exchange + tid * kExchange;
      const bool turns = does && kind[u] < 2;
      if (turns) {
#pragma unroll
        for (int z = 0; z < 16; ++z) mine[z] = x[z];
      }
      __syncwarp();
      if (turns) {
        const float *c = cosines + (size_t)token[u] * P.angles, *s = sines + (size_t)token[u] * P.angles;
        float* row = mine - j * kExchange;
        const int h = P.R / 2;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
          const int i = (int)j + (y << P.lanes_log2), k = i + h;
          if (i >= h) continue;
          float *p = row + i + i / 16 * (kExchange - 16), *q = row + k + k / 16 * (kExchange - 16);
          const float a = *p, b = *q;
          *p = fmaf(a, c[i], -b * s[i]);
          *q = fmaf(b, c[i], a * s[i]);
        }
      }
      __syncwarp();
      if (turns) {
#pragma unroll
        for (int z = 0; z < 16; ++z) x[z] = mine[z];
      }
    }
    if (!does) continue;
    const int at[2] = {8 * v0, 8 * v1};
    if (kind[u] == 0) {
      unsigned char* dst = P.dst[0] + (long long)(first + token[u]) * P.out_stride + (size_t)head[u] * P.D * S;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (at[y] < P.D) Vec8<T>::store(dst + (size_t)at[y] * S, reinterpret_cast<const float(&)[8]>(x[8 * y]));
      continue;
    }
    const int kv = kind[u] - 1;
    const size_t row = (size_t)slot * P.H + head[u];
    if constexpr (QUANT) {
      uint32_t code[4];
      const int e = specv::quantise_row<16>(x, lanes, code);
      unsigned char* dst = P.dst[kind[u]] + row * P.D;
#pragma unroll
      for (int y = 0; y < 2; ++y)
        if (at[y] < P.D) *reinterpret_cast<uint2*>(dst + at[y]) = make_uint2(code[2 * y], code[2 * y + 1]);
      if (j == 0) P.scale[kv][row] = specv::pow2f_int(e);
    } else {
      unsigned char* dst = P.dst[kind[u]] + row * P.D * S;
#pragma unroll
      for (int y = 0; y < 2; ++y) {
        if (at[y] >= P.D) continue;
        if (kv == 0) {
          Vec8<T>::store(dst + (size_t)at[y] * S, reinterpret_cast<const float(&)[8]>(x[8 * y]));
        } else {  // values keep their bits
#pragma unroll
          for (int i = 0; i < W; i += 4)
            *reinterpret_cast<uint4*>(dst + (size_t)at[y] * S + i * 4) = make_uint4(raw[u][y][i], raw[u][y][i + 1], raw[u][y][i + 2], raw[u][y][i + 3]);
        }
      }
    }
  }
  check_requests(P);
}

template <typename T, int PAIRS>
cudaError_t launch(const Rope& P, bool quant, size_t smem, unsigned grid, cudaStream_t s) {
  if (quant)
    rope_kernel<T, PAIRS, true><<<grid, kThreads, smem, s>>>(P);
  else
    rope_kernel<T, PAIRS, false><<<grid, kThreads, smem, s>>>(P);
  return cudaGetLastError();
}
template <typename T>
cudaError_t launch_pairs(const Rope& P, int pairs, bool quant, size_t smem, unsigned grid, cudaStream_t s) {
  return pairs == kNext   ? launch<T, kNext>(P, quant, smem, grid, s)
         : pairs == kHalf ? launch<T, kHalf>(P, quant, smem, grid, s)
                          : launch<T, kHalfOdd>(P, quant, smem, grid, s);
}

bool aligned16(const void* p) { return ((uintptr_t)p & 15u) == 0; }
bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

}  // namespace

extern "C" spec_status_t spec_rope_kv_write(const void* q, const void* k, const void* v, spec_dtype_t dtype, long long q_stride,
                                            long long k_stride, long long v_stride, int B, int T, int num_heads, int num_kv_heads,
                                            int head_dim, const float* inv_freq, int rotary_dim, int interleaved, float factor,
                                            const int32_t* positions, const int32_t* context_len, const int32_t* parents,
                                            const int32_t* slots, void* q_out, long long q_out_stride, void* k_cache, void* v_cache,
                                            spec_dtype_t cache_dtype, float* k_scale, float* v_scale, long long num_slots,
                                            int32_t* err_flags, spec_stream_t stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_INVALID_ARG;
  if (cache_dtype != dtype && cache_dtype != SPEC_DTYPE_E4M3) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || T < 0 || num_heads < 0 || num_kv_heads < 1 || head_dim < 1 || num_slots < 0) return SPEC_ERR_INVALID_ARG;
  if (rotary_dim < 2 || rotary_dim % 2 != 0 || rotary_dim > head_dim || !isfinite(factor)) return SPEC_ERR_INVALID_ARG;
  if (positions && (context_len || parents)) return SPEC_ERR_INVALID_ARG;
  if (head_dim % 8 != 0 || head_dim > SPEC_MAX_KV_HEAD_DIM) return SPEC_ERR_UNSUPPORTED;
  if (num_slots > INT_MAX) return SPEC_ERR_UNSUPPORTED;  // a slot is an int32
  if (parents && T > SPEC_MAX_WALK_NODES) return SPEC_ERR_UNSUPPORTED;
  const long long tokens = (long long)B * T, per_token = (long long)num_heads + 2LL * num_kv_heads;
  if (tokens > INT_MAX || per_token > INT_MAX || tokens * per_token > INT_MAX) return SPEC_ERR_UNSUPPORTED;
  if (B == 0 || (T == 0 && !err_flags)) return SPEC_OK;
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  if (T == 0) return cudaMemsetAsync(err_flags, 0, (size_t)B * 4, s) == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
  if (num_heads == 0 ? q || q_out : !q || !q_out) return SPEC_ERR_INVALID_ARG;
  if (!k || !v || !inv_freq || !slots || !k_cache || !v_cache || (!positions && !context_len)) return SPEC_ERR_INVALID_ARG;
  if (!aligned16(q) || !aligned16(k) || !aligned16(v) || !aligned16(q_out) || !aligned16(k_cache) || !aligned16(v_cache))
    return SPEC_ERR_INVALID_ARG;
  const bool quant = cache_dtype == SPEC_DTYPE_E4M3;
  if (quant && (!k_scale || !v_scale || !aligned4(k_scale) || !aligned4(v_scale))) return SPEC_ERR_INVALID_ARG;
  if (!aligned4(inv_freq) || !aligned4(slots) || !aligned4(positions) || !aligned4(context_len) || !aligned4(parents) || !aligned4(err_flags))
    return SPEC_ERR_INVALID_ARG;
  const int S = dtype == SPEC_DTYPE_F32 ? 4 : 2;
  const long long qrow = (long long)num_heads * head_dim, row = (long long)num_kv_heads * head_dim;
  const struct {
    long long stride, least;
  } strides[4] = {{num_heads ? q_stride : 0, qrow}, {k_stride, row}, {v_stride, row}, {num_heads ? q_out_stride : 0, qrow}};
  for (const auto& x : strides)
    if (x.stride < x.least || x.stride > LLONG_MAX / 4 / tokens || (x.stride * S) % 16 != 0) return SPEC_ERR_INVALID_ARG;
  if (num_heads && q == q_out && q_stride != q_out_stride) return SPEC_ERR_INVALID_ARG;
  Rope P = {};
  P.src[0] = static_cast<const unsigned char*>(q);
  P.src[1] = static_cast<const unsigned char*>(k);
  P.src[2] = static_cast<const unsigned char*>(v);
  P.dst[0] = static_cast<unsigned char*>(q_out);
  P.dst[1] = static_cast<unsigned char*>(k_cache);
  P.dst[2] = static_cast<unsigned char*>(v_cache);
  P.scale[0] = k_scale;
  P.scale[1] = v_scale;
  P.stride[0] = q_stride * S;
  P.stride[1] = k_stride * S;
  P.stride[2] = v_stride * S;
  P.out_stride = q_out_stride * S;
  P.slots = slots;
  P.positions = positions;
  P.context_len = context_len;
  P.parents = parents;
  P.inv_freq = inv_freq;
  P.err_flags = err_flags;
  P.num_slots = num_slots;
  P.rows = (unsigned)(tokens * per_token);
  P.factor = factor;
  P.B = B;
  P.T = T;
  P.Hq = num_heads;
  P.H = num_kv_heads;
  P.D = head_dim;
  P.R = rotary_dim;
  while ((16 << P.lanes_log2) < head_dim) ++P.lanes_log2;
  const long long block_rows = (long long)(kThreads >> P.lanes_log2) * kRowsPerThread;
  const long long spanned = (block_rows - 1) / per_token + 2;
  P.tokens_max = (int)(spanned < tokens ? spanned : tokens);
  P.angles = (rotary_dim / 2 + 3) / 4 * 4;
  P.fd_t = specv::make_fastdiv((uint32_t)T);
  P.fd_rows = specv::make_fastdiv((uint32_t)per_token);
  P.fd_angles = specv::make_fastdiv((uint32_t)P.angles);
  // at most 129 tokens of 16 elements, or 9 of 256, and the lanes' exchange, so within the 48 KB that need no asking
  const size_t smem = (size_t)P.tokens_max * (P.angles * 8 + 12) + (parents ? ((size_t)T + P.tokens_max) * 2 : 0);
  const unsigned grid = (unsigned)((P.rows + block_rows - 1) / block_rows);
  const int pairs = interleaved ? kNext : rotary_dim % 16 == 0 ? kHalf : kHalfOdd;
  const cudaError_t e = dtype == SPEC_DTYPE_F32    ? launch_pairs<float>(P, pairs, quant, smem, grid, s)
                        : dtype == SPEC_DTYPE_BF16 ? launch_pairs<__nv_bfloat16>(P, pairs, quant, smem, grid, s)
                                                   : launch_pairs<__half>(P, pairs, quant, smem, grid, s);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}
