// sample_kernel.cuh -- the kernel of spec_sample and spec_logits_filter: temperature, top-k, top-p and min-p of a
// logits row, and a token drawn from what they keep (sm_103a).
//
// Mathematics.  With M the row's maximum, token i weighs w_i = exp((x_i - M) / T).  In the order of falling
// logits (equal ones by rising index) each rule keeps a first part of the row: top-k its first k tokens; top-p, of
// those, the shortest part with at least p of their weight; min-p the tokens with w_i >= m.  The shortest of the
// three parts is kept; it ends at a cut (value, index).  The draw is the first token in index order whose running
// weight exceeds u times the kept weight.
//
// A token that is kept or drawn by mistake is a wrong result however small the rounding error that caused it, so sums
// of weights are whole numbers of 2^-44 (fixed_weight.h): exact and in any order the same.
//
// One cluster of 1 to 8 CTAs takes a row, each a slice of it.  A few rows' slices stay in shared memory; otherwise each
// pass reads them again, from L2 mostly, and four CTAs share an SM, so that one's barriers and dependent steps are hidden by the
// others' passes.  The first pass takes maxima, four a thread.  CTA 0 leads: the others send it counts and sums, it decides and
// tells.
//   top-k   A bound first: the k-th largest of the threads' maxima, to 1/16 of a power of two of weight.  What
//           reaches it, hardly more than k tokens, is gathered by the leader (few of the maxima's groups have any, and only
//           those are read again), sorted, and everything else happens there: rows are filled with -inf and the kept
//           tokens put in their places.  Where that does not fit (k above 512 with one CTA, 819 with more, many equal logits), tokens are counted by 1/32
//           powers of two of weight and then, if one such bin holds too many, digit by digit of the ordered bits.
//   top-p alone  Weights are summed by 1/32 powers of two of weight, to 2^-15 of each or finer; the sums tell the bins between
//           which the cut lies.  One pass sums the weights above them and in all, exactly, and gathers what is in them, which the
//           leader sorts.  The exact sums tell whether the bins were right; if not, or if too many tokens are in them, the
//           same is done once more with what is left of the range in equal steps, and then the cut is found by halving the
//           range of the ordered bits.  Filtered bf16 rows have their values counted instead (see by_value).
//   draw    Weights are summed by warps (each holds a stretch of the row); the CTA whose stretch holds the
//           crossing goes through it once more.
// Every CTA of a cluster takes the same path; the cluster barrier is the only wait.
//
// What bounds it (us; a copy of the rows at HBM's rate in brackets).  One row of 32,000 by top-k and top-p: latency of some ten
// dependent steps, 9.8.  384 f32 rows of 128,256 filtered by top-k: 82 (59): one wave of CTAs in step, in which nothing moves while
// lists are gathered and sorted (drawn, without the writing, 49).  976 bf16 rows: filtered by top-p 232 (75): of a
// row's 100 us or so the first reading takes a tenth, the counting two tenths, the leader's sums two, the writing three to four;
// drawn without rules 213 (37, reading), weighing bound by instruction issue (about 30 a logit); drawn by top-p 374, the bins'
// additions and the weighing in turn.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <limits.h>

#include <type_traits>

#include "cluster.cuh"
#include "fastdiv.h"
#include "fixed_weight.h"
#include "spec_verify.h"
#include "verify_common.cuh"

namespace specv {
namespace sample {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kKeptCtas = 3, kMinCtas = 4;  // an SM has registers for, with slices in shared memory and without
constexpr int kMaxCluster = 8;
constexpr int kBins = 2048;
constexpr int kPerOctave = 32;     // bins a power of two of weight
constexpr int kValues = 2048;       // bf16 magnitudes counted, of either sign
constexpr int kBoundBins = 1024;   // of the threads' maxima, twice as wide
constexpr int kMaxima = 4;         // maxima a thread
constexpr int kMostTokens = 1000 * kThreads;  // a CTA: a thread's sums stay within 32 bits
constexpr int kCap = 1024;         // tokens that the leader can sort
constexpr int kRanked = 128;       // up to so many it sorts by counting
constexpr int kSegs = kMaxCluster * kWarps;
constexpr int kMsg = 8;
constexpr uint32_t kLowest = 0x00800000u;  // the ordered bits of the lowest finite float
constexpr float kLowestFloat = -3.402823466e38f;
static_assert(kBins == 8 * kThreads && kCap == 4 * kThreads && kBoundBins == 4 * kThreads && kSegs == 64, "a thread's share");

struct Params {
  const unsigned char* logits;
  unsigned char* out;          // filtered rows, or null
  const float *temps, *top_p, *min_p, *u;
  const int32_t* top_k;
  int32_t *tokens, *kept, *err_flags;
  float* probs;
  float temperature;
  int V;
  int cl;            // CTAs a row
  int vecs;          // 16-byte vectors a CTA
  float unit;        // parts of a weight in the bins' sums: as many as keep a CTA's tokens within 32 bits
  FastDiv fd_r;      // rows of a request
};

struct Shared {
  union {
    uint32_t hist[kBins];
    uint32_t values[2 * kValues];
    uint64_t cand[kCap];       // (ordered bits flipped, index, sign of a zero): sorts by falling value, rising index
  };
  Pair table[32];
  uint64_t seg[kSegs], seg2[kSegs];  // leader: sums of the warps' stretches
  uint32_t segc[kSegs];
  uint64_t w64[kWarps];
  uint64_t xsum[2][kMaxCluster];
  float xmax[kMaxCluster];
  uint32_t xfirst[kMaxCluster];
  float wf[kWarps];
  uint32_t w32[kWarps];
  uint32_t msg[kMsg];          // from the leader
  uint32_t found[4];           // bin, count before it, its own, all
  uint32_t answer;
  uint32_t count;              // leader: gathered
  uint32_t kept;               // leader: counted
  uint32_t pick;
  float sum;
  uint32_t minkey;
  uint32_t count2;
  uint64_t total[2];
  double reach;                // T ln(min_p)
};

// Bits that order as the floats do; -0 as 0.
__device__ __forceinline__ uint32_t ordered(float x) {
  const uint32_t u = __float_as_uint(x + 0.f);
  return u ^ ((uint32_t)((int32_t)u >> 31) | 0x80000000u);
}
__device__ __forceinline__ float from_ordered(uint32_t k) {
  return __uint_as_float(k & 0x80000000u ? k ^ 0x80000000u : ~k);
}

struct Cut {  // kept: above x, or x itself up to index `last`
  float x;
  int last;
  __device__ __forceinline__ bool keeps(float y, int i) const { return y > x || (y == x && i <= last); }
  // f(masked): masked(y, i) is y where it is kept, else -inf; nothing to do, or one comparison, where that is enough.
  template <typename F>
  __device__ __forceinline__ void with(F&& f) const {
    const Cut c = *this;
    if (last == INT_MAX && x == kLowestFloat)
      f([](float y, int) { return y; });
    else if (last == INT_MAX)
      f([c](float y, int) { return y >= c.x ? y : -INFINITY; });
    else
      f([c](float y, int i) { return c.keeps(y, i) ? y : -INFINITY; });
  }
};

__device__ __forceinline__ uint64_t warp_sum64(uint64_t v) {
#pragma unroll
  for (int o = 16; o; o >>= 1) v += __shfl_xor_sync(kFull, v, o);
  return v;
}
template <typename N>
__device__ __forceinline__ N warp_scan(N v, int width = 32) {
  const int lane = threadIdx.x & 31;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    if (o >= width) break;
    const N t = __shfl_up_sync(kFull, v, o);
    if (lane >= o) v += t;
  }
  return v;
}
// Sum over the block's threads up to and with this one, and over all; `part` [kWarps].  Between two calls with the same
// `part` lies another barrier.
template <typename N>
__device__ __forceinline__ N block_scan(N v, N* part, N& all) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  v = warp_scan(v);
  if (lane == 31) part[warp] = v;
  __syncthreads();
  const N p = warp_scan(lane < kWarps ? part[lane] : N(0), kWarps);
  all = __shfl_sync(kFull, p, kWarps - 1);
  const N before = __shfl_sync(kFull, p, warp ? warp - 1 : 0);
  return warp ? v + before : v;
}

__device__ __forceinline__ void red_shared(uint32_t at) { asm volatile("red.shared::cta.add.u32 [%0], 1;" ::"r"(at) : "memory"); }
// Adds v to the shared word `at` if a < b; no branch.
__device__ __forceinline__ void add_if_less(uint32_t* at, uint32_t v, float a, float b) {
  asm volatile("{\n\t.reg .pred p;\n\tsetp.lt.f32 p, %2, %3;\n\t@p red.shared::cta.add.u32 [%0], %1;\n\t}" ::"r"(smem_addr(at)), "r"(v),
               "f"(a), "f"(b)
               : "memory");
}

// Logits of T two (or one) to a word: ones where they are at least the threshold's; the least T that is at least x, and the
// next above it, as such words.
__device__ __forceinline__ uint32_t at_least_mask(uint32_t w, uint32_t t, float) {
  return __uint_as_float(w) >= __uint_as_float(t) ? ~0u : 0u;
}
__device__ __forceinline__ uint32_t at_least_mask(uint32_t w, uint32_t t, __nv_bfloat16) {
  return __hge2_mask(*reinterpret_cast<const __nv_bfloat162*>(&w), *reinterpret_cast<const __nv_bfloat162*>(&t));
}
__device__ __forceinline__ uint32_t at_least_mask(uint32_t w, uint32_t t, __half) {
  return __hge2_mask(*reinterpret_cast<const __half2*>(&w), *reinterpret_cast<const __half2*>(&t));
}
__device__ __forceinline__ uint32_t threshold(float x, float) { return __float_as_uint(x); }
__device__ __forceinline__ uint32_t threshold(float x, __nv_bfloat16) {
  return __bfloat16_as_ushort(__float2bfloat16_ru(x)) * 0x10001u;
}
__device__ __forceinline__ uint32_t threshold(float x, __half) { return __half_as_ushort(__float2half_ru(x)) * 0x10001u; }
template <typename T>
__device__ __forceinline__ uint32_t next_threshold(uint32_t t) {
  constexpr uint32_t sign = sizeof(T) == 4 ? 0x80000000u : 0x8000u, ones = sizeof(T) == 4 ? ~0u : 0xffffu;
  uint32_t b = t & ones;
  b = (b & ~sign) == 0 ? 1u : b & sign ? b - 1 : b + 1;  // (of both zeros: the smallest above)
  return sizeof(T) == 4 ? b : b * 0x10001u;
}

template <typename T>
constexpr uint32_t kSign = sizeof(T) == 4 ? 0x80000000u : 0x8000u;  // -0

template <typename T, bool KEPT, bool TOP_K, bool DRAW>
struct Row {  // one CTA's slice of a row
  static constexpr int E = Elem<T>::kPerVec, S = Elem<T>::kSize;
  static constexpr bool kCounts = !KEPT && !TOP_K && !DRAW && std::is_same<T, __nv_bfloat16>::value;  // see by_value
  const Params& P;
  Shared& sm;
  uint4* data;                // the slice, where it is kept in shared memory
  const unsigned char* base;  // its first place in global memory
  int rank, off, all, first;  // off: places before the row in its first vector; all: vectors of the row; first: row index of the slice's first place
  int slice, each_warp;       // vectors of the slice, of a warp
  int begin, end;             // this warp's
  int lane, warp;
  float most[kMaxima];        // maxima of this thread's, by turns
  WeightRow weights;
  float per_bin;              // bins a unit of logit
  int equals;                 // of the tokens equal to a cut with last = -1, as many are kept (see by_value)

  // Every thread of the cluster.
  __device__ __forceinline__ void sync() const {
    if (P.cl == 1)
      __syncthreads();
    else
      cluster_barrier();
  }

  // A logit's bits, not as constant data: rows may be filtered in place.
  __device__ __forceinline__ static uint32_t bits_at(const unsigned char* p) {
    if constexpr (S == 4)
      return __ldcg(reinterpret_cast<const unsigned int*>(p));
    else
      return __ldcg(reinterpret_cast<const unsigned short*>(p));
  }
  // Vector v of the slice; places outside the row are -inf.
  __device__ __forceinline__ uint4 fetch(int v) const {
    const int i0 = first + v * E;
    if (i0 >= 0 && i0 + E <= P.V) return __ldcg(reinterpret_cast<const uint4*>(base + (size_t)v * 16));
    uint32_t words[4];
#pragma unroll
    for (int e = 0; e < E; ++e) {
      const bool in = i0 + e >= 0 && i0 + e < P.V;
      const uint32_t x = in ? bits_at(base + ((long long)v * E + e) * S) : Elem<T>::kNegInf;
      if constexpr (S == 4)
        words[e] = x;
      else
        words[e / 2] = e & 1 ? words[e / 2] | x << 16 : x;
    }
    return make_uint4(words[0], words[1], words[2], words[3]);
  }
  __device__ __forceinline__ uint4 vector(int v, int stop) const {
    constexpr uint32_t N = Elem<T>::kNegInfWord;
    if (v >= stop) return make_uint4(N, N, N, N);
    if constexpr (KEPT)
      return data[v];
    else
      return fetch(v);
  }
  // f(values, index of the first) for this warp's vectors, 32 at a time, one or two steps fetched ahead.
  template <int AHEAD = 2, typename F>
  __device__ __forceinline__ void each(F&& f) const {
    uint4 now = vector(begin + lane, end), next = AHEAD == 2 ? vector(begin + 32 + lane, end) : now;
#pragma unroll 1
    for (int v0 = begin; v0 < end; v0 += 32) {
      float x[E];
      Elem<T>::unpack(now, x);
      if constexpr (AHEAD == 2) now = next;
      next = vector(v0 + 32 * AHEAD + lane, end);
      if constexpr (AHEAD == 1) now = next;
      f(x, first + (v0 + lane) * E);
    }
  }
  __device__ __forceinline__ uint64_t weight(float x) const { return fixed_weight(x, weights, sm.table); }
  // Distance below the maximum in bins; rises as x falls.
  __device__ __forceinline__ float depth(float x) const { return (weights.top - x) * per_bin; }
  // The two parts of two weights (see weight_cut).  What is not wanted comes as -inf and weighs nothing.
  __device__ __forceinline__ void weigh(float x0, float x1, Pair& upper, Pair& lower) const {
    Pair at, z, tail, hi, lo;
    weight_power(Pair{x0, x1}, weights, at, z, tail);
    const Pair t0 = sm.table[weight_index(at.x)], t1 = sm.table[weight_index(at.y)];
    const float s0 = weight_size(at.x), s1 = weight_size(at.y);
    weight_product(Pair{t0.x * s0, t1.x * s1}, Pair{t0.y * s0, t1.y * s1}, z, tail, hi, lo);
    weight_cut(hi, lo, upper, lower);
  }
  __device__ __forceinline__ static uint64_t weight_of(float upper, float lower) {
    return (uint64_t)(((int64_t)(float_bits(upper) - float_bits(kUpper)) << kWeightHalf) + (float_bits(lower) - float_bits(kLower)));
  }
  // A thread's sum: the parts' bits, and how many there are (1000 of at most 2^22 and of 2^21 fit 32 bits).
  struct Sum {
    uint32_t upper = 0, lower = 0, n = 0;
    __device__ __forceinline__ void add(float u, float l) {
      upper += __float_as_uint(u);
      lower += __float_as_uint(l);
    }
    __device__ __forceinline__ void add(Pair u, Pair l) {
      upper += __float_as_uint(u.x) + __float_as_uint(u.y);
      lower += __float_as_uint(l.x) + __float_as_uint(l.y);
    }
    __device__ __forceinline__ uint64_t value() const {
      return ((uint64_t)(upper - n * __float_as_uint(kUpper)) << kWeightHalf) + (uint64_t)(int64_t)(int32_t)(lower - n * __float_as_uint(kLower));
    }
  };

  // Tokens for which want(value, index) goes to the leader's list (those beyond its room are counted only).
  template <typename F>
  __device__ __forceinline__ void gather_vector(const float (&x)[E], int i0, F&& want) const {
    uint32_t hits = 0;
#pragma unroll
    for (int e = 0; e < E; ++e) hits |= want(x[e], i0 + e) ? 1u << e : 0u;
    if (!hits) return;
    uint32_t at = add_cluster_u32(peer_addr(&sm.count, 0), __popc(hits));
    const uint32_t list = peer_addr(sm.cand, 0);
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (hits >> e & 1) {
        if (at < kCap) st_cluster_u64(list + at * 8, entry(x[e], i0 + e));
        ++at;
      }
  }
  template <typename F>
  __device__ __forceinline__ void gather(F&& want) const {
    each([&](const float(&x)[E], int i0) { gather_vector(x, i0, want); });
  }

  // The same where few groups of a thread's vectors have such a token: by their maxima, a group at a time, each by the whole
  // warp (a thread that went through its own vectors would wait for each: 30,000 cycles for 50 of 128,256 tokens, not 5,000).
  template <typename F>
  __device__ __forceinline__ void gather_few(F&& want) const {
    uint32_t hits[kMaxima];
    int n = 0;
#pragma unroll
    for (int i = 0; i < kMaxima; ++i) {
      hits[i] = __ballot_sync(kFull, want(most[i], 0));
      n += __popc(hits[i]);
    }
    if (n * 4 > (end - begin) / 32) {  // not so few
      each([&](const float(&x)[E], int i0) {
        float top = x[0];
#pragma unroll
        for (int e = 1; e < E; ++e) top = fmaxf(top, x[e]);
        if (want(top, 0)) gather_vector(x, i0, want);
      });
      return;
    }
#pragma unroll
    for (int i = 0; i < kMaxima; ++i)
      while (hits[i]) {
        const int owner = __ffs(hits[i]) - 1;
        hits[i] &= hits[i] - 1;
#pragma unroll 1
        for (int v = begin + 32 * i + owner + 32 * kMaxima * lane; v < end; v += 32 * kMaxima * 32) {
          float x[E];
          Elem<T>::unpack(vector(v, end), x);
          gather_vector(x, first + v * E, want);
        }
      }
  }

  // The leader's words to every CTA; the next barrier shows them.
  __device__ __forceinline__ void tell(const uint32_t (&w)[kMsg]) const {
    if (rank == 0 && (int)threadIdx.x < P.cl) {
      const uint32_t at = peer_addr(sm.msg, threadIdx.x);
#pragma unroll
      for (int i = 0; i < kMsg; ++i) st_cluster_u32(at + 4 * i, w[i]);
    }
  }

  // The leader's list sorted; n of its places are taken.
  __device__ void sort_list(int n) const {
    const int t = threadIdx.x;
    if (n <= kRanked) {
      // by counting what comes before: a power of two of threads for each
      int N = 8;
      while (N < n) N <<= 1;
      const int G = kThreads / N, i = t / G;
      const uint64_t mine = i < n ? sm.cand[i] : 0;
      int before = 0;
      for (int j = t % G; j < n; j += G) before += sm.cand[j] < mine;
#pragma unroll
      for (int o = 16; o; o >>= 1) before += o < G ? __shfl_xor_sync(kFull, before, o) : 0;
      __syncthreads();
      if (t % G == 0 && i < n) sm.cand[before] = mine;
      __syncthreads();
      return;
    }
    if (n <= kThreads)
      sort_in_registers<1>(n);
    else if (n <= 2 * kThreads)
      sort_in_registers<2>(n);
    else
      sort_in_registers<4>(n);
  }
  // By exchanging, Q neighbours a thread, in registers within a warp (150: 6,500 cycles while others weigh, in shared memory 11,000).
  template <int Q>
  __device__ __forceinline__ void sort_in_registers(int n) const {
    const int t = threadIdx.x;
    uint64_t m[Q];
#pragma unroll
    for (int q = 0; q < Q; ++q) m[q] = Q * t + q < n ? sm.cand[Q * t + q] : ~0ull;
    auto keep = [&](int q, int k, int j, uint64_t other) {
      const int i = Q * t + q;
      m[q] = (m[q] < other) == (((i & k) == 0) == ((i & j) == 0)) ? m[q] : other;
    };
#pragma unroll 1
    for (int k = 2; k < 2 * n; k <<= 1)
#pragma unroll 1
      for (int j = k >> 1; j; j >>= 1) {
        uint64_t other[Q];
        if (j < Q) {
#pragma unroll
          for (int q = 0; q < Q; ++q) other[q] = j == 1 ? m[q ^ (Q > 1 ? 1 : 0)] : m[q ^ (Q > 2 ? 2 : 0)];
        } else if (j < 32 * Q) {
#pragma unroll
          for (int q = 0; q < Q; ++q) other[q] = __shfl_xor_sync(kFull, m[q], j / Q);
        } else {
          __syncthreads();
#pragma unroll
          for (int q = 0; q < Q; ++q) sm.cand[Q * t + q] = m[q];
          __syncthreads();
#pragma unroll
          for (int q = 0; q < Q; ++q) other[q] = sm.cand[(Q * t + q) ^ j];
        }
#pragma unroll
        for (int q = 0; q < Q; ++q) keep(q, k, j, other[q]);
      }
    __syncthreads();
#pragma unroll
    for (int q = 0; q < Q; ++q) sm.cand[Q * t + q] = m[q];
    __syncthreads();
  }
  __device__ __forceinline__ static uint64_t entry(float x, int i) {
    return (uint64_t)~ordered(x) << 32 | (uint32_t)i << 1 | (__float_as_uint(x) == 0x80000000u);
  }
  __device__ __forceinline__ static uint32_t key_of(uint64_t c) { return ~(uint32_t)(c >> 32); }
  __device__ __forceinline__ static int index_of(uint64_t c) { return (int)((uint32_t)c >> 1); }

  // The m-th (from 1) kept token equal to x: its index, in every CTA.
  __device__ int tie(float x, uint32_t m, const Cut& cut) const {
    uint32_t n = 0;
    each([&](const float(&y)[E], int i0) {
#pragma unroll
      for (int e = 0; e < E; ++e) n += y[e] == x && cut.keeps(x, i0 + e);
    });
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) st_cluster_u32(peer_addr(&sm.segc[rank * kWarps + warp], 0), n);
    sync();
    uint32_t w[kMsg] = {};
    if (rank == 0) {
      if (warp == 0) {
        uint32_t c[2];
#pragma unroll
        for (int i = 0; i < 2; ++i) c[i] = 2 * lane + i < P.cl * kWarps ? sm.segc[2 * lane + i] : 0;
        uint32_t before = warp_scan(c[0] + c[1]) - c[0] - c[1];
#pragma unroll
        for (int i = 0; i < 2; ++i) {
          if (before < m && m <= before + c[i]) sm.found[0] = 2 * lane + i, sm.found[1] = m - before;
          before += c[i];
        }
      }
      __syncthreads();
      w[0] = sm.found[0];
      w[1] = sm.found[1];
    }
    tell(w);
    sync();
    if (sm.msg[0] == (uint32_t)(rank * kWarps + warp)) {
      uint32_t left = sm.msg[1];
      bool found = false;
      each([&](const float(&y)[E], int i0) {
        uint32_t hits = 0;
#pragma unroll
        for (int e = 0; e < E; ++e) hits |= y[e] == x && cut.keeps(x, i0 + e) ? 1u << e : 0u;
        const uint32_t c = __popc(hits), incl = warp_scan(c), all = __shfl_sync(kFull, incl, 31);
        uint32_t before = incl - c;
        if (!found && before < left && left <= incl)
          for (int e = 0; e < E; ++e)
            if ((hits >> e & 1) && ++before == left)
              for (int r = 0; r < P.cl; ++r) st_cluster_u32(peer_addr(&sm.answer, r), (uint32_t)(i0 + e));
        found = found || left <= all;
        left -= all;
      });
    }
    sync();
    return (int)sm.answer;
  }

  // The first bin at which the leader's running counts reach k; all of the leader's threads, each with its share of
  // the bins.  sm.found: the bin, the count before it and its own; returns the count of all.
  template <int B>
  __device__ uint32_t find_bin(const uint32_t (&n)[B], uint32_t k) const {
    uint32_t sum = 0, total;
#pragma unroll
    for (int i = 0; i < B; ++i) sum += n[i];
    const uint32_t incl = block_scan(sum, sm.w32, total);
    k = min(k, total);
    uint32_t before = incl - sum;
#pragma unroll
    for (int i = 0; i < B; ++i) {
      if (before < k && k <= before + n[i]) sm.found[0] = B * threadIdx.x + i, sm.found[1] = before, sm.found[2] = n[i];
      before += n[i];
    }
    __syncthreads();
    return total;
  }
  // The leader's thread's eight bins, f(number, value of bin 0 .. 7 of CTA r).
  __device__ __forceinline__ void read_bins(uint32_t (&n)[8]) const {
#pragma unroll
    for (int i = 0; i < 8; ++i) n[i] = 0;
#pragma unroll 4
    for (int r = 0; r < P.cl; ++r) {
      const uint32_t at = peer_addr(&sm.hist[8 * threadIdx.x], r);
      const uint4 v = ld_cluster_v4(at), w = ld_cluster_v4(at + 16);
      n[0] += v.x, n[1] += v.y, n[2] += v.z, n[3] += v.w;
      n[4] += w.x, n[5] += w.y, n[6] += w.z, n[7] += w.w;
    }
  }
  __device__ __forceinline__ void clear_hist() const {
    uint4* h = reinterpret_cast<uint4*>(&sm.hist[8 * threadIdx.x]);
    h[0] = h[1] = make_uint4(0, 0, 0, 0);
    if (threadIdx.x == 0) sm.count = 0;
  }

  // The first k tokens.  Returns their number where the leader's list, sorted, holds (at least) all of them; else 0, and the
  // cut in every CTA.
  __device__ int top_k(uint32_t k, Cut& cut) const {
    uint32_t w[kMsg] = {};
    // (the k-th largest of as many threads' maxima as there are tokens to find says little: fewer than half)
    if (2 * k <= (uint32_t)(P.cl * kThreads * kMaxima) && 5 * k <= 4 * kCap) {
      // (the counts are zero: cleared before the first barrier)
#pragma unroll
      for (int i = 0; i < kMaxima; ++i) {
        const float mine = depth(most[i]) * 0.5f;
        if (mine < kBoundBins) atomicAdd(&sm.hist[(int)mine], 1);
      }
      sync();
      if (rank == 0) {
        uint32_t n[4] = {0, 0, 0, 0};
#pragma unroll 4
        for (int r = 0; r < P.cl; ++r) {
          const uint4 v = ld_cluster_v4(peer_addr(&sm.hist[4 * threadIdx.x], r));
          n[0] += v.x, n[1] += v.y, n[2] += v.z, n[3] += v.w;
        }
        w[0] = find_bin(n, k) >= k;
        w[1] = __float_as_uint((float)(sm.found[0] + 1));
      }
      tell(w);
      sync();
      if (sm.msg[0]) {
        const float limit = __uint_as_float(sm.msg[1]);
        auto want = [&](float x, int) { return depth(x) * 0.5f < limit; };
        gather_few(want);
        sync();
        const uint32_t n = ld_cluster_u32(peer_addr(&sm.count, 0));
        if (n <= kCap) {
          if (rank == 0) sort_list((int)n);
          return (int)k;
        }
        sync();  // (the list's place becomes counts again)
      }
    }
    // Counts by depth; where the bin of the k-th holds too many or has no end, by digits of the ordered bits: 11, 11 and 10.
    clear_hist();
    __syncthreads();
    auto place = [&](float x) { return fminf(depth(x), (float)(kBins - 1)) + 0x1p23f; };  // (its bits end in the bin)
    each([&](const float(&x)[E], int) {
#pragma unroll
      for (int e = 0; e < E; ++e) add_if_less(&sm.hist[__float_as_uint(place(x[e])) & (kBins - 1)], 1, -INFINITY, x[e]);
    });
    uint32_t prefix = 0, above = 0;  // the digits known; tokens above what has them
#pragma unroll 1
    for (int level = 0;; ++level) {
      const int shift = level < 2 ? 21 : level == 2 ? 10 : 0;
      const uint32_t last = level == 3 ? 1023 : 2047;  // digits count down
      if (level > 0) {
        clear_hist();
        __syncthreads();
        each([&](const float(&x)[E], int) {
#pragma unroll
          for (int e = 0; e < E; ++e) {
            const uint32_t key = ordered(x[e]);
            if (key >= kLowest && (level == 1 || key >> (level == 2 ? 21 : 10) == prefix)) atomicAdd(&sm.hist[last - (key >> shift & last)], 1);
          }
        });
      }
      sync();
      if (rank == 0) {
        uint32_t n[8];
        read_bins(n);
        const uint32_t total = find_bin(n, k - above);
        if (level == 0) k = min(k, total);  // (fewer finite tokens: all of them)
        w[0] = sm.found[0];
        w[1] = sm.found[1];
        w[2] = sm.found[2];
        w[3] = k;
      }
      tell(w);
      sync();
      const uint32_t bin = sm.msg[0], before = above + sm.msg[1], in = sm.msg[2];
      k = sm.msg[3];
      const bool whole = before + in <= kCap;
      const uint32_t digits = level < 2 ? last - bin : prefix << (level == 2 ? 11 : 10) | (last - bin);
      if ((whole || in <= kCap) && (level > 0 || whole || bin < kBins - 1)) {
        // (the leader's counts have been read; the list takes their place)
        if (level == 0) {
          const float most_at = 0x1p23f + (float)bin, least_at = whole ? 0.f : most_at;
          each([&](const float(&x)[E], int i0) {
            auto want = [&](float y, int) { return place(y) <= most_at && place(y) >= least_at && y > -INFINITY; };
            float best = x[0];
#pragma unroll
            for (int e = 1; e < E; ++e) best = fmaxf(best, x[e]);
            if (place(best) <= most_at) gather_vector(x, i0, want);
          });
        } else {
          gather([&](float x, int) {
            const uint32_t mine = ordered(x) >> shift;
            return x >= kLowestFloat && (mine == digits || (whole && mine > digits));
          });
        }
        sync();
        if (rank == 0) {
          sort_list((int)(whole ? before + in : in));
          if (!whole) {
            const uint64_t c = sm.cand[k - before - 1];
            w[0] = __float_as_uint(from_ordered(key_of(c)));
            w[1] = (uint32_t)index_of(c);
          }
        }
        if (whole) return (int)k;
        tell(w);
        sync();
        cut.x = __uint_as_float(sm.msg[0]);
        cut.last = (int)sm.msg[1];
        return 0;
      }
      if (level == 0) continue;
      prefix = digits;
      above = before;
      if (level == 3) {  // many equal ones
        const float x = from_ordered(prefix);
        const int i = tie(x, k - above, cut);
        cut.x = x;
        cut.last = i;
        return 0;
      }
    }
  }

  // Weight of the kept tokens of at least x, in every CTA; `it` counts the calls.
  __device__ uint64_t mass_from(float least, const Cut& cut, int it) const {
    Sum s;
    each<1>([&](const float(&x)[E], int i0) {
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        Pair u, l;
        weigh(x[e] >= least && cut.keeps(x[e], i0 + e) ? x[e] : -INFINITY, x[e + 1] >= least && cut.keeps(x[e + 1], i0 + e + 1) ? x[e + 1] : -INFINITY, u, l);
        s.add(u, l);
      }
      s.n += E;
    });
    uint64_t sum = warp_sum64(s.value());
    if (lane == 0) sm.w64[warp] = sum;
    __syncthreads();
    if (warp == 0) {
      sum = warp_sum64(lane < kWarps ? sm.w64[lane] : 0);
      if (lane < P.cl) st_cluster_u64(peer_addr(&sm.xsum[it & 1][rank], lane), sum);
    }
    sync();
    uint64_t total = 0;
    for (int r = 0; r < P.cl; ++r) total += sm.xsum[it & 1][r];
    return total;
  }

  // p of the weight `total`, rounded up; at least 1.
  __device__ __forceinline__ static uint64_t part_of(float p, uint64_t total) {
    const uint64_t f = (uint64_t)(p * 0x1p64f);
    const uint64_t hi = __umul64hi(f, total);
    return max((unsigned long long)(hi + (f * total != 0)), 1ull);
  }

  // The cut of top-p among all tokens of a bf16 row by counting values: there are 128 a power of two, and those of the 15.7
  // powers of two below the largest magnitude that weighs anything are counted each; exact sums follow from the counts.  Tokens
  // closer to zero are weighed one by one.  Returns whether that gave the cut: the value, how many such tokens there are and are
  // kept, and how many are above.  (976 rows of 128,256 filtered by 0.9: 234 us, by bins and weighing 415.  Drawn from, all are
  // weighed afterwards, and little is gained.)
  struct Found {
    float x;
    uint32_t need, equal, above;
  };
  __device__ bool by_value(float p, Found& f) const {
    constexpr int kFar = kValues - 32;  // from here on: below all weights; a bin a lane, as there may be many
    {
      uint4* h = reinterpret_cast<uint4*>(sm.values) + threadIdx.x;
#pragma unroll
      for (int i = 0; i < 2 * kValues / 4 / kThreads; ++i) h[i * kThreads] = make_uint4(0, 0, 0, 0);
      if (threadIdx.x == 0) sm.count = 0;
    }
    const uint32_t largest = max(__bfloat16_as_ushort(__float2bfloat16_rd(weights.top)) & 0x7fffu,
                                 __bfloat16_as_ushort(__float2bfloat16_rd(weights.least)) & 0x7fffu);
    const int base = max(0, (int)largest - (kFar - 1));
    __syncthreads();
    const uint32_t less = (uint32_t)(-base & 0xffff) * 0x10001u, limit = (uint32_t)(kValues - 1 - lane) * 0x10001u;
    const uint32_t counts = smem_addr(sm.values);
    Sum s;
    {
      uint4 now = vector(begin + lane, end), next = vector(begin + 32 + lane, end);
#pragma unroll 1
      for (int v0 = begin; v0 < end; v0 += 32) {
        const uint32_t words[4] = {now.x, now.y, now.z, now.w};
        const uint4 was = now;
        now = next;
        next = vector(v0 + 64 + lane, end);
        uint32_t low = ~0u;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t m = __viaddmin_s16x2_relu(words[i] & 0x7fff7fffu, less, limit), at = m | (words[i] >> 4 & 0x08000800u);
          static_assert(kValues == 0x800, "the sign's place");
          red_shared(counts + (at & 0xffffu) * 4);
          red_shared(counts + (at >> 16) * 4);
          low = __vminu2(low, m);
        }
        if (!(low & 0xffffu) || !(low >> 16)) {
          const float tiny = __uint_as_float((uint32_t)base << 16);
          float x[E];
          Elem<T>::unpack(was, x);
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            Pair a, b;
            weigh(fabsf(x[e]) <= tiny ? x[e] : -INFINITY, fabsf(x[e + 1]) <= tiny ? x[e + 1] : -INFINITY, a, b);
            s.add(a, b);
          }
          s.n += E;
        }
      }
    }
    const uint64_t near = warp_sum64(s.value());
    if (lane == 0) st_cluster_u64(peer_addr(&sm.seg[rank * kWarps + warp], 0), near);
    sync();
    uint32_t w[kMsg] = {};
    if (rank == 0) {
      // a thread's 16 values, falling: the first half of the threads the positive ones
      const int t = threadIdx.x;
      auto lowest = [](int t) { return t < kThreads / 2 ? kValues - 16 - 16 * t : 16 * t - kValues; };  // magnitude of the first in memory
      auto value = [&](int t, int m) { return __uint_as_float((uint32_t)(m + base) << 16 | (t < kThreads / 2 ? 0u : 0x80000000u)); };
      uint64_t tiny = 0, mine = 0, total;  // (tiny: those closest to zero, after the last positive value)
      uint32_t many = 0, all_n;
      if (t == kThreads / 2 - 1)
        for (int i = 0; i < P.cl * kWarps; ++i) tiny += sm.seg[i];
#pragma unroll 2
      for (int i = 0; i < 16; i += 4) {
        const int m = lowest(t) + i;
        uint4 n = make_uint4(0, 0, 0, 0);
        for (int r = 0; r < P.cl; ++r) {
          const uint4 v = ld_cluster_v4(peer_addr(&sm.values[(t < kThreads / 2 ? 0 : kValues) + m], r));
          n.x += v.x, n.y += v.y, n.z += v.z, n.w += v.w;
        }
        many += n.x + n.y + n.z + n.w;
        if (m == 0) n.x = 0;
        Pair a0, b0, a1, b1;
        weigh(value(t, m), value(t, m + 1), a0, b0);
        weigh(value(t, m + 2), value(t, m + 3), a1, b1);
        if (m < kFar) mine += n.x * weight_of(a0.x, b0.x) + n.y * weight_of(a0.y, b0.y) + n.z * weight_of(a1.x, b1.x) + n.w * weight_of(a1.y, b1.y);
      }
      mine += tiny;
      if (t == 0) sm.found[0] = 0;
      uint64_t run = block_scan(mine, sm.w64, total) - mine;
      const uint32_t above = block_scan(many, sm.w32, all_n) - many;
      const uint64_t want = part_of(p, total);
      if (run < want && want <= run + mine) sm.total[0] = want - run, sm.total[1] = tiny, sm.found[1] = t, sm.count2 = above;
      __syncthreads();
      if (warp == 0) {  // that thread's values, one a lane
        const int from = (int)sm.found[1], at = lane & 15, m = lowest(from) + (from < kThreads / 2 ? 15 - at : at);
        const uint64_t left = sm.total[0];
        uint32_t n = 0;
        for (int r = 0; r < P.cl; ++r) n += ld_cluster_u32(peer_addr(&sm.values[(from < kThreads / 2 ? 0 : kValues) + m], r));
        const float x = value(from, m);
        const uint64_t one = m > 0 ? weight(x) : 0, g = m == 0 ? sm.total[1] : m < kFar ? n * one : 0;
        const uint64_t upto = warp_scan(g, 16);
        const uint32_t n_upto = warp_scan(n, 16);
        if (lane < 16 && m > 0 && upto - g < left && left <= upto) {
          sm.found[0] = 1;
          sm.found[1] = __float_as_uint(x);
          sm.found[2] = (uint32_t)((left - (upto - g) + one - 1) / one);
          sm.found[3] = n;
          sm.count2 += n_upto - n;
        }
      }
      __syncthreads();
#pragma unroll
      for (int i = 0; i < 4; ++i) w[i] = sm.found[i];
      w[4] = sm.count2;
    }
    tell(w);
    sync();
    f = Found{__uint_as_float(sm.msg[1]), sm.msg[2], sm.msg[3], sm.msg[4]};
    return sm.msg[0] != 0;
  }

  // What top-p (p < 1) leaves of the tokens that `cut` keeps.  Returns whether that is all that is kept: then
  // their number has been written, and the draw prepared (see locate).
  __device__ bool top_p(float p, float u, uint32_t minkey, size_t row, Cut& cut) {
    float from = INFINITY, to = -INFINITY;  // the cut lies among the tokens that are at most `from` and above `to`
    uint64_t want = 0, over = 0;            // the weight that the kept ones reach; of those above `from`
    if constexpr (kCounts) {
      Found f;
      if (by_value(p, f)) {
        const bool ruled = minkey <= ordered(f.x);  // (otherwise min-p ends above)
        int last = INT_MAX;
        if (ruled && f.need < f.equal) {
          if (f.equal <= kCap)
            last = -1, equals = (int)f.need;
          else
            last = tie(f.x, f.need, cut);
        }
        cut = Cut{f.x, last};
        if (ruled && rank == 0 && threadIdx.x == 0 && P.kept) P.kept[row] = (int)(f.above + f.need);
        return ruled;
      }
    }
#pragma unroll 1
    for (int level = 0; level < 2; ++level) {
      clear_hist();
      __syncthreads();
      // Weights by bins.  First 1/32 powers of two: each weight in parts of its bin's middle's, 2^(-t / 32) by two terms;
      // bin b is the depths within 1/2 of b.  Then, where too many tokens were in them, the range left in equal steps.  Sums with
      // large constants give the bins and the whole numbers, as conversions take four times as long.
      const float head = fminf(from, weights.top), step = (float)(kBins - 2) / (head - fmaxf(to, weights.least));
      const float unit1 = P.unit * -0.021660849f, unit2 = P.unit * 2.345947e-4f;
      cut.with([&](auto&& masked) {
        if (level == 0)
          each([&](const float(&x)[E], int i0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float d = depth(masked(x[e], i0 + e)), at = d + 0x1p23f, t = d - (at - 0x1p23f);
              const float part = fmaf(t, fmaf(t, unit2, unit1), P.unit + 0x1p23f);
              add_if_less(&sm.hist[__float_as_uint(at) & (kBins - 1)], __float_as_uint(part) & 0x7fffffu, d, kWeightEnd * kPerOctave);
            }
          });
        else
          each([&](const float(&x)[E], int i0) {
#pragma unroll
            for (int e = 0; e < E; ++e) {
              const float y = masked(x[e], i0 + e);
              if (y <= from && y > fmaxf(to, weights.least))
                atomicAdd(&sm.hist[min((int)((head - y) * step), kBins - 1)],
                          __float_as_uint(fmaf(ex2((y - head) * weights.hi), P.unit, 0x1p23f)) & 0x7fffffu);
            }
          });
      });
      sync();
      uint32_t w[kMsg] = {};
      if (rank == 0) {
        float m[8], sum = 0.f, total;
#pragma unroll
        for (int i = 0; i < 8; ++i) m[i] = 0.f;
#pragma unroll 4
        for (int r = 0; r < P.cl; ++r) {
          const uint32_t at = peer_addr(&sm.hist[8 * threadIdx.x], r);
          const uint4 v = ld_cluster_v4(at), y = ld_cluster_v4(at + 16);
          m[0] += (float)v.x, m[1] += (float)v.y, m[2] += (float)v.z, m[3] += (float)v.w;
          m[4] += (float)y.x, m[5] += (float)y.y, m[6] += (float)y.z, m[7] += (float)y.w;
        }
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          m[i] *= level == 0 ? ex2((float)(8 * (int)threadIdx.x + i) * (-1.f / kPerOctave)) : 1.f;
          sum += m[i];
        }
        float before = block_scan(sum, sm.wf, total) - sum;
        if (threadIdx.x == 0) sm.found[0] = 0, sm.found[1] = kBins;
        __syncthreads();
        // the bins between which the cut lies, as far as these sums tell: each part is off by half a unit at most
        const float target = level == 0 ? p * total : (float)(want - over) * 0x1p-44f * P.unit * ex2((weights.top - head) * weights.hi);
        const float slack = total / P.unit + target * 0x1p-18f;
        uint32_t low = 0, high = kBins;
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          const float after = before + m[i];
          if (m[i] > 0.f && before <= target - slack) low = 8 * threadIdx.x + i;
          if (m[i] > 0.f && after >= target + slack) high = min(high, 8 * threadIdx.x + i);
          before = after;
        }
        low = __reduce_max_sync(kFull, low);
        high = __reduce_min_sync(kFull, high);
        if (lane == 0) atomicMax(&sm.found[0], low), atomicMin(&sm.found[1], high);
        __syncthreads();
        // as logits; none found: to the end
        const float edge = level == 0 ? 0.5f : 0.f, each_bin = level == 0 ? per_bin : step;
        w[0] = __float_as_uint(fminf(from, head - ((float)sm.found[0] - edge) / each_bin));
        w[1] = __float_as_uint(sm.found[1] < kBins ? fmaxf(to, head - ((float)sm.found[1] + (1.f - edge)) / each_bin) : to);
      }
      tell(w);
      sync();
      from = __uint_as_float(sm.msg[0]), to = __uint_as_float(sm.msg[1]);
      Sum s, above;
      cut.with([&](auto&& masked) {
        each<1>([&](const float(&x)[E], int i0) {
          uint32_t in = 0;  // (those above `to`)
          const uint32_t were = above.n;
#pragma unroll
          for (int e = 0; e < E; e += 2) {
            const float x0 = masked(x[e], i0 + e), x1 = masked(x[e + 1], i0 + e + 1);
            Pair a, b;
            weigh(x0, x1, a, b);
            s.add(a, b);
            if (x0 > from) above.add(a.x, b.x), ++above.n;
            if (x1 > from) above.add(a.y, b.y), ++above.n;
            in += x0 > to;
            in += x1 > to;
          }
          s.n += E;
          if (in != above.n - were)
            gather_vector(x, i0, [&](float y, int i) {
              const float m = masked(y, i);
              return m <= from && m > to;
            });
        });
      });
      uint64_t sum = warp_sum64(s.value());
      over = warp_sum64(above.value());
      uint32_t n = above.n;
      n = __reduce_add_sync(kFull, n);
      if (lane == 0) {
        st_cluster_u64(peer_addr(&sm.seg[rank * kWarps + warp], 0), sum);
        st_cluster_u64(peer_addr(&sm.seg2[rank * kWarps + warp], 0), over);
        st_cluster_u32(peer_addr(&sm.segc[rank * kWarps + warp], 0), n);
      }
      sync();
      if (rank == 0) {
        const int t = threadIdx.x;
        uint64_t c[2] = {0, 0}, o[2] = {0, 0};
        uint32_t m = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i)
          if (2 * lane + i < P.cl * kWarps) c[i] = sm.seg[2 * lane + i], o[i] = sm.seg2[2 * lane + i], m += sm.segc[2 * lane + i];
        sum = warp_sum64(c[0] + c[1]);
        over = warp_sum64(o[0] + o[1]);
        n = __reduce_add_sync(kFull, m);
        want = part_of(p, sum);
        const int listed = (int)sm.count;
        bool fine = listed > 0 && listed <= kCap && over < want;
        uint64_t listed_mass = 0;
        if (t == 0) sm.pick = kCap;
        __syncthreads();
        if (fine) {
          sort_list(listed);
          const int ipt = listed <= kThreads ? 1 : 4;
          uint64_t g[4], mine = 0, total;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            g[i] = i < ipt && ipt * t + i < listed ? weight(from_ordered(key_of(sm.cand[ipt * t + i]))) : 0;
            mine += g[i];
          }
          uint64_t run = block_scan(mine, sm.w64, total) - mine + over;
          listed_mass = total;
#pragma unroll
          for (int i = 0; i < 4; ++i) {
            if (run < want && want <= run + g[i]) sm.pick = ipt * t + i;
            run += g[i];
          }
          __syncthreads();
          if (DRAW && sm.pick < kCap) {
            // the draw's sums: those above the list, and what is kept of it
#pragma unroll
            for (int i = 0; i < 4; ++i)
              if (i < ipt && ipt * t + i <= (int)sm.pick)
                atomicAdd(reinterpret_cast<unsigned long long*>(&sm.seg2[seg_of(index_of(sm.cand[ipt * t + i]))]), g[i]);
            __syncthreads();
          }
        }
        fine = fine && sm.pick < kCap;
        w[0] = fine;
        w[1] = (uint32_t)want;
        w[2] = (uint32_t)(want >> 32);
        // Where the cut is, if not found: above, among them (too many) or below.
        w[3] = over >= want ? 1 : listed > kCap ? 2 : 3;
        if (w[3] == 1) over = 0;
        if (w[3] == 3) over += listed_mass;
        w[4] = (uint32_t)over;
        w[5] = (uint32_t)(over >> 32);
        if (fine) {
          const uint64_t last = sm.cand[sm.pick];
          w[1] = __float_as_uint(from_ordered(key_of(last)));
          w[2] = (uint32_t)index_of(last);
          if (minkey <= key_of(last)) {
            w[0] = 2;
            if (DRAW) find_segment(sm.seg2, u, w);
            if (t == 0 && P.kept) P.kept[row] = (int)(n + sm.pick + 1);
          }
        }
      }
      tell(w);
      sync();
      if (sm.msg[0]) {
        cut.x = __uint_as_float(sm.msg[1]);
        cut.last = (int)sm.msg[2];
        return sm.msg[0] == 2;
      }
      if (sm.msg[3] == 1) to = from, from = INFINITY;
      if (sm.msg[3] == 3) from = to, to = -INFINITY;
    }
    want = (uint64_t)sm.msg[2] << 32 | sm.msg[1];
    over = (uint64_t)sm.msg[5] << 32 | sm.msg[4];
    // The largest value whose tokens and those above it weigh enough, by halving the range of the ordered bits: the range left
    // if it holds the cut.
    uint32_t at = kLowest, beyond = ordered(weights.top) + 1;
    uint64_t over_it = 0;  // weight from `beyond` on
    int it = 0;
    {
      if (from < weights.top) beyond = ordered(from) + 1, over_it = over;
      const uint32_t low = max(ordered(to) + 1, kLowest);
      const uint64_t m = mass_from(from_ordered(low), cut, it++);
      if (m >= want)
        at = low;
      else
        beyond = low, over_it = m;
    }
    while (beyond - at > 1) {
      const uint32_t mid = at + (beyond - at) / 2;
      const uint64_t m = mass_from(from_ordered(mid), cut, it++);
      if (m >= want)
        at = mid;
      else
        beyond = mid, over_it = m;
    }
    const float x = from_ordered(at);
    const uint64_t one = weight(x);
    const uint32_t need = one ? (uint32_t)((want - over_it + one - 1) / one) : 1;
    const int i = tie(x, need, cut);
    cut.x = x;
    cut.last = i;
    return false;
  }

  // Which warp's stretch holds token i.
  __device__ __forceinline__ int seg_of(int i) const {
    const int v = (i + off) / E, r = v / P.vecs, size = min(P.vecs, all - r * P.vecs), part = (size + kWarps - 1) / kWarps;
    return r * kWarps + (v - r * P.vecs) / part;
  }
  // The leader's words 3 .. 7: the stretch in whose running weight the draw's place lies, the place in it, the weight of all.
  __device__ __forceinline__ void find_segment(const uint64_t* seg, float u, uint32_t (&w)[kMsg]) const {
    if (warp == 0) {
      uint64_t c[2];
#pragma unroll
      for (int i = 0; i < 2; ++i) c[i] = 2 * lane + i < P.cl * kWarps ? seg[2 * lane + i] : 0;
      const uint64_t incl = warp_scan(c[0] + c[1]), total = __shfl_sync(kFull, incl, 31);
      const uint64_t t = __umul64hi((uint64_t)(u * 0x1p64f), total);  // the crossing: running weight > t
      uint64_t before = incl - c[0] - c[1];
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        if (before <= t && t < before + c[i]) sm.found[2] = 2 * lane + i, sm.total[0] = t - before, sm.total[1] = total;
        before += c[i];
      }
    }
    __syncthreads();
    w[3] = sm.found[2];
    w[4] = (uint32_t)sm.total[0], w[5] = (uint32_t)(sm.total[0] >> 32);
    w[6] = (uint32_t)sm.total[1], w[7] = (uint32_t)(sm.total[1] >> 32);
  }

  // x is drawn: its part of the weight kept; the quotient of two floats each, rounded once.
  __device__ __forceinline__ float probability(float x, uint64_t total) const {
    Pair w;
    fixed_weight(x, weights, sm.table, &w);
    const float t = (float)total, low = (float)(int64_t)(total - (uint64_t)t), q = __fdiv_rn(w.x, t);
    const float rest = fmaf(-q, low, fmaf(-q, t, w.x) + w.y);
    return (q + __fdiv_rn(rest, t)) * 0x1p44f;
  }

  // Sums of what `cut` keeps, by stretches, and the leader's word on them to every CTA; the number kept is written.
  __device__ void prepare_draw(float u, const Cut& cut, size_t row) const {
    Sum s;
    uint32_t n = 0;
    cut.with([&](auto&& masked) {
      each<1>([&](const float(&x)[E], int i0) {
        float low = INFINITY;
#pragma unroll
        for (int e = 0; e < E; e += 2) {
          const float x0 = masked(x[e], i0 + e), x1 = masked(x[e + 1], i0 + e + 1);
          Pair a, b;
          weigh(x0, x1, a, b);
          s.add(a, b);
          low = fminf(low, fminf(x0, x1));
        }
        s.n += E;
        n += E;
        if (low == -INFINITY)
#pragma unroll
          for (int e = 0; e < E; ++e) n -= masked(x[e], i0 + e) == -INFINITY;
      });
    });
    const uint64_t sum = warp_sum64(s.value());
    n = __reduce_add_sync(kFull, n);
    if (lane == 0) {
      st_cluster_u64(peer_addr(&sm.seg[rank * kWarps + warp], 0), sum);
      st_cluster_u32(peer_addr(&sm.segc[rank * kWarps + warp], 0), n);
    }
    sync();
    uint32_t w[kMsg] = {};
    if (rank == 0) {
      find_segment(sm.seg, u, w);
      if (warp == 0 && P.kept) {
        n = 0;
#pragma unroll
        for (int i = 0; i < 2; ++i) n += 2 * lane + i < P.cl * kWarps ? sm.segc[2 * lane + i] : 0;
        n = __reduce_add_sync(kFull, n);
        if (lane == 0) P.kept[row] = (int)n;
      }
    }
    tell(w);
    sync();
  }
  // The token at the place the leader told, written by the CTA whose slice has it.
  __device__ void locate(const Cut& cut, size_t row) const {
    const int seg = (int)sm.msg[3] - rank * kWarps;
    if (seg < 0 || seg >= kWarps) return;
    uint64_t t = (uint64_t)sm.msg[5] << 32 | sm.msg[4];
    const uint64_t total = (uint64_t)sm.msg[7] << 32 | sm.msg[6];
    const int stop = min(slice, (seg + 1) * each_warp);
#pragma unroll 1
    for (int v0 = min(slice, seg * each_warp); v0 < stop; v0 += kThreads) {
      const int v = v0 + (int)threadIdx.x, i0 = first + v * E;
      float x[E];
      Elem<T>::unpack(vector(v, stop), x);
      uint64_t g[E], mine = 0, step;
#pragma unroll
      for (int e = 0; e < E; e += 2) {
        Pair a, b;
        weigh(cut.keeps(x[e], i0 + e) ? x[e] : -INFINITY, cut.keeps(x[e + 1], i0 + e + 1) ? x[e + 1] : -INFINITY, a, b);
        g[e] = weight_of(a.x, b.x);
        g[e + 1] = weight_of(a.y, b.y);
        mine += g[e] + g[e + 1];
      }
      const uint64_t incl = block_scan(mine, sm.w64, step);
      uint64_t before = incl - mine;
      if (before <= t && t < incl) {
#pragma unroll
        for (int e = 0; e < E; ++e) {
          if (before <= t && t < before + g[e]) {
            P.tokens[row] = i0 + e;
            if (P.probs) P.probs[row] = probability(x[e], total);
          }
          before += g[e];
        }
      }
      if (t < step) break;
      t -= step;
      __syncthreads();
    }
  }

  // The leader's list has the first k tokens: top-p and min-p among them, and the draw.  Returns how many are kept.
  __device__ int finish_list(int k, float p, float u, uint32_t minkey, size_t row) const {
    const int t = threadIdx.x, ipt = k <= kThreads ? 1 : 4;
    uint64_t g[4], mine = 0, total;
    int high = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      g[i] = 0;
      if (i < ipt && ipt * t + i < k) {
        const uint32_t key = key_of(sm.cand[ipt * t + i]);
        g[i] = weight(from_ordered(key));
        high += key >= minkey;
      }
      mine += g[i];
    }
    if (t == 0) sm.pick = k - 1, sm.kept = 0;
    uint64_t run = block_scan(mine, sm.w64, total) - mine;
    const uint64_t want = part_of(p, total), start = run;
    high = __reduce_add_sync(kFull, high);
    if (lane == 0 && high) atomicAdd(&sm.kept, high);  // (the list falls: those of at least minkey come first)
    if (p < 1.f) {
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (run < want && want <= run + g[i]) sm.pick = ipt * t + i;
        run += g[i];
      }
    }
    __syncthreads();
    const int n = min((int)sm.pick + 1, (int)sm.kept);
    if (t == 0 && P.kept) P.kept[row] = n;
    if (!DRAW) return n;
    run = start;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      run += g[i];
      if (i < ipt && ipt * t + i == n - 1) sm.total[0] = run;
    }
    // by index: (index, ordered bits)
    uint64_t own[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) own[i] = i < ipt && ipt * t + i < n ? sm.cand[ipt * t + i] : 0;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < 4; ++i)
      if (i < ipt && ipt * t + i < n) sm.cand[ipt * t + i] = (uint64_t)index_of(own[i]) << 32 | key_of(own[i]);
    __syncthreads();
    sort_list(n);
    const uint64_t kept = sm.total[0], x = __umul64hi((uint64_t)(u * 0x1p64f), kept);
    mine = 0;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      own[i] = i < ipt && ipt * t + i < n ? sm.cand[ipt * t + i] : 0;
      g[i] = i < ipt && ipt * t + i < n ? weight(from_ordered((uint32_t)own[i])) : 0;
      mine += g[i];
    }
    run = block_scan(mine, sm.w64, total) - mine;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      if (run <= x && x < run + g[i]) {
        P.tokens[row] = (int)(own[i] >> 32);
        if (P.probs) P.probs[row] = probability(from_ordered((uint32_t)own[i]), kept);
      }
      run += g[i];
    }
    return n;
  }

  __device__ __forceinline__ void put(unsigned char* to, bool vec, int v, const uint4& w) const {
    const int i0 = first + v * E;
    if (vec && i0 >= 0 && i0 + E <= P.V) {
      __stcs(reinterpret_cast<uint4*>(to + (size_t)v * 16), w);
      return;
    }
    const uint32_t words[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
    for (int e = 0; e < E; ++e)
      if (i0 + e >= 0 && i0 + e < P.V)
        Elem<T>::store_raw(to + ((long long)v * E + e) * S, S == 4 ? words[e] : words[e / 2] >> (e & 1 ? 16 : 0));
  }
  // The slice at -inf.
  __device__ void fill(unsigned char* out) const {
    constexpr uint32_t N = Elem<T>::kNegInfWord;
    unsigned char* to = out + (long long)first * S;
    const bool vec = ((uintptr_t)to & 15u) == 0;
#pragma unroll 4
    for (int v = begin + lane; v < end; v += 32) put(to, vec, v, make_uint4(N, N, N, N));
  }
  // The first n of the leader's list in their places.
  __device__ void scatter(unsigned char* out, int n) const {
    for (int i = threadIdx.x; i < n; i += kThreads) {
      const uint64_t c = sm.cand[i];
      Elem<T>::store_raw(out + (size_t)index_of(c) * S, (uint32_t)c & 1 ? kSign<T> : raw_of(from_ordered(key_of(c))));
    }
  }
  // The bits of a logit of T.
  __device__ __forceinline__ static uint32_t raw_of(float x) {
    if constexpr (S == 4) {
      return __float_as_uint(x);
    } else {
      const T t = T(x);
      return *reinterpret_cast<const uint16_t*>(&t);
    }
  }
  // The slice with what `cut` does not keep at -inf; returns how many this thread's tokens are kept, if asked (whole: as it is).
  __device__ uint32_t write(unsigned char* out, const Cut& cut, bool whole, bool count) const {
    constexpr uint32_t N = Elem<T>::kNegInfWord;
    uint32_t bits = 0, n = 0;
    unsigned char* to = out + (long long)first * S;
    const bool vec = ((uintptr_t)to & 15u) == 0;
    // equal ones are kept up to index `last`: there the cut itself is the least that is kept, behind it the next value
    const uint32_t here = threshold(cut.x, T()), behind = next_threshold<T>(here);
    constexpr int U = kMaxima;
#pragma unroll 1
    for (int v0 = begin + lane; v0 < end; v0 += 32 * U) {
      uint4 w[U];
#pragma unroll
      for (int i = 0; i < U; ++i)  // (what has no kept token is not read again)
        w[i] = !whole && most[i] < cut.x ? make_uint4(N, N, N, N) : vector(v0 + 32 * i, end);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = v0 + 32 * i, i0 = first + v * E;
        if (v >= end) continue;
        if (!whole) {
          uint32_t words[4] = {w[i].x, w[i].y, w[i].z, w[i].w}, tied = 0;
          const uint32_t least = i0 + E - 1 <= cut.last ? here : behind;
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            uint32_t m = at_least_mask(words[j], least, T());
            if (i0 <= cut.last && i0 + E - 1 > cut.last) {  // (one vector of the row)
              const uint32_t equal = at_least_mask(words[j], here, T()) & ~m;
#pragma unroll
              for (int e = 0; e < E / 4; ++e)
                if (i0 + j * (E / 4) + e <= cut.last) m |= equal & (S == 4 ? ~0u : 0xffffu << 16 * e);
            }
            if (kCounts && equals) tied |= at_least_mask(words[j], here, T()) & ~m;
            words[j] = (words[j] & m) | (N & ~m);
            if (count) bits += __popc(m);
          }
          if (tied) {
            float x[E];
            Elem<T>::unpack(w[i], x);
            gather_vector(x, i0, [&](float y, int) { return y == cut.x; });
          }
          w[i] = make_uint4(words[0], words[1], words[2], words[3]);
        }
        put(to, vec, v, w[i]);
      }
    }
    n = bits / (8 * S);
    return n;
  }
};

// KEPT: slices stay in shared memory; otherwise each pass reads them again (from L2 mostly).
// DRAW: spec_sample, otherwise spec_logits_filter.  TOP_K: some row may have one.
template <typename T, bool KEPT, bool TOP_K, bool DRAW>
__global__ void __launch_bounds__(kThreads, KEPT ? kKeptCtas : kMinCtas) sample_kernel(const __grid_constant__ Params P) {
  constexpr int E = Elem<T>::kPerVec, S = Elem<T>::kSize;
  extern __shared__ __align__(16) unsigned char smem[];
  Shared& sm = *reinterpret_cast<Shared*>(smem);
  uint4* data = reinterpret_cast<uint4*>(smem + (sizeof(Shared) + 15) / 16 * 16);
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, rank = (int)cta_rank();
  const size_t row = blockIdx.x / P.cl;
  if (P.cl > 1) asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");  // (waited for below: the others have started)
  const unsigned char* src = P.logits + row * P.V * S;
  const int off = (int)(((uintptr_t)src & 15u) / S);
  const int all = (int)(((long long)off + P.V + E - 1) / E);  // vectors that the row touches
  const int slice = max(0, min(P.vecs, all - rank * P.vecs)), each = (slice + kWarps - 1) / kWarps;
  Row<T, KEPT, TOP_K, DRAW> r{P, sm, data, src + ((long long)rank * P.vecs * E - off) * S, rank, off, all, rank * P.vecs * E - off, slice, each, min(slice, warp * each), min(slice, (warp + 1) * each), lane, warp, {}, {}, 0.f, 0};
#pragma unroll
  for (int i = 0; i < kMaxima; ++i) r.most[i] = -INFINITY;

  // -- the threads' maxima
  {
    constexpr int U = 8;
#pragma unroll 1
    for (int v0 = r.begin; v0 < r.end; v0 += 32 * U) {
      uint4 w[U];
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = v0 + 32 * i + lane;
        if (v < r.end) w[i] = r.fetch(v);
      }
#pragma unroll
      for (int i = 0; i < U; ++i) {
        const int v = v0 + 32 * i + lane;
        if (v >= r.end) continue;
        if constexpr (KEPT) data[v] = w[i];
        const uint32_t top = Elem<T>::max_word(Elem<T>::max_word(w[i].x, w[i].y), Elem<T>::max_word(w[i].z, w[i].w));
        r.most[i % kMaxima] = fmax_nan(r.most[i % kMaxima], Elem<T>::word_max(top));
      }
    }
  }
  r.clear_hist();
  if (tid == 0) sm.kept = 0;
  // -- this row's rules
  const int b = (int)fdiv((uint32_t)row, P.fd_r);
  const float temperature = P.temps ? __ldg(P.temps + b) : P.temperature;
  const int k = TOP_K ? __ldg(P.top_k + b) : 0;
  const float p = P.top_p ? __ldg(P.top_p + b) : 1.f, m = P.min_p ? __ldg(P.min_p + b) : 0.f;
  const float u = DRAW ? __ldg(P.u + row) : 0.f;
  int flags = 0;
  if (!(temperature == 0.f || (temperature >= 0x1p-64f && temperature <= 0x1p64f))) flags |= SPEC_ERRF_BAD_TEMPERATURE;
  if (k < 0 || !(p >= 0.f && p <= 1.f) || !(m >= 0.f && m <= 1.f) || (temperature != 0.f && !(u >= 0.f && u < 1.f)))
    flags |= SPEC_ERRF_BAD_SAMPLING;
  float c_hi, c_lo;
  weight_factor(flags || temperature == 0.f ? 1.f : temperature, c_hi, c_lo);
  if (tid == kThreads - 32 && m > 0.f) sm.reach = (double)temperature * log((double)m);
  float mine = r.most[0];
#pragma unroll
  for (int i = 1; i < kMaxima; ++i) mine = fmax_nan(mine, r.most[i]);
  const float wm = warp_max_nan(mine);
  if (lane == 0) sm.wf[warp] = wm;
  __syncthreads();
  if (P.cl > 1) asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
  if (warp == 0) {
    const float x = warp_max_nan(lane < kWarps ? sm.wf[lane] : -INFINITY);
    if (lane < P.cl) st_cluster_u32(peer_addr(&sm.xmax[rank], lane), __float_as_uint(x));
  }
  r.sync();
  float top = -INFINITY;
  for (int i = 0; i < P.cl; ++i) top = fmax_nan(top, sm.xmax[i]);
  if (!(top > -INFINITY && top < INFINITY)) flags |= SPEC_ERRF_NONFINITE;
  const bool lead = rank == 0 && tid == 0;
  if (lead && P.err_flags) P.err_flags[row] = flags;
  if (flags) {
    if (lead) {
      if (DRAW) P.tokens[row] = -1;
      if (P.probs) P.probs[row] = 0.f;
      if (P.kept) P.kept[row] = 0;
    }
    if (!DRAW) r.write(P.out + row * P.V * S, Cut{0.f, 0}, true, false);
    return;  // (no CTA reaches into another from here on)
  }
  r.weights = weight_row(top, c_hi, c_lo);
  r.per_bin = kPerOctave * c_hi;
  Cut cut{kLowestFloat, INT_MAX};
  bool counted = false;  // kept has been written
  if (temperature == 0.f) {
    // greedy: the first of the largest
    uint32_t at = INT_MAX;
    r.each([&](const float(&x)[E], int i0) {
#pragma unroll
      for (int e = 0; e < E; ++e)
        if (x[e] == top) at = min(at, (uint32_t)(i0 + e));
    });
    at = __reduce_min_sync(kFull, at);
    if (lane == 0) sm.w32[warp] = at;
    __syncthreads();
    if (warp == 0) {
      at = __reduce_min_sync(kFull, lane < kWarps ? sm.w32[lane] : (uint32_t)INT_MAX);
      if (lane < P.cl) st_cluster_u32(peer_addr(&sm.xfirst[rank], lane), at);
    }
    r.sync();
    at = INT_MAX;
    for (int i = 0; i < P.cl; ++i) at = min(at, sm.xfirst[i]);
    cut = Cut{top, (int)at};
    counted = true;
    if (lead) {
      if (DRAW) P.tokens[row] = (int)at;
      if (P.probs) P.probs[row] = 1.f;
      if (P.kept) P.kept[row] = 1;
    }
  } else {
    constexpr Pair table[32] = SPECV_WEIGHT_TABLE;
    if (tid < 32) {
      Pair t = table[0];
#pragma unroll
      for (int i = 1; i < 32; ++i)
        if (tid == i) t = table[i];
      sm.table[tid] = weight_entry(t, r.weights);
    }
    if (tid == 32) {
      uint32_t key = kLowest;
      if (m > 0.f) key = ordered(__double2float_ru((double)top + sm.reach));
      sm.minkey = max(key, kLowest);
    }
    __syncthreads();
    const uint32_t minkey = sm.minkey;
    const int list = TOP_K && k > 0 && k < P.V ? r.top_k((uint32_t)k, cut) : 0;
    if (TOP_K && list) {
      // (nothing of the row is looked at any more, and none reaches into another after the barrier)
      if (!DRAW) r.fill(P.out + row * P.V * S);
      r.sync();
      if (rank != 0) return;
      const int n = r.finish_list(list, p, u, minkey, row);
      if (!DRAW) r.scatter(P.out + row * P.V * S, n);
      return;
    } else {
      const bool ready = p < 1.f ? r.top_p(p, u, minkey, row, cut) : false;
      const float least = from_ordered(minkey);
      if (least > cut.x) cut = Cut{least, INT_MAX};
      if (DRAW) {
        if (!ready) r.prepare_draw(u, cut, row);
        r.locate(cut, row);
      }
      counted = counted || DRAW || ready;
    }
  }
  if (!DRAW) {
    const bool count = !counted && P.kept;
    const uint32_t n = __reduce_add_sync(kFull, r.write(P.out + row * P.V * S, cut, false, count));
    if (count) {
      if (lane == 0 && n) red_cluster_u32(peer_addr(&sm.kept, 0), n);
      r.sync();
      if (lead) P.kept[row] = (int)sm.kept;
    }
  }
  r.sync();  // none leaves while another may still reach into it
  if (decltype(r)::kCounts && r.equals && rank == 0) {
    r.sort_list((int)sm.count);
    r.scatter(P.out + row * P.V * S, r.equals);
  }
}

// Shared memory but for a slice.
constexpr size_t kSharedBytes = (sizeof(Shared) + 15) / 16 * 16;
constexpr int kMostShared = (int)kSharedBytes + (SPEC_MAX_SAMPLE_VOCAB / kMaxCluster + 8) * 4;  // slices of whole vectors

template <typename T, bool KEPT, bool TOP_K, bool DRAW>
cudaError_t launch_one(const Params& P, long long rows, cudaStream_t stream) {
  auto* kern = sample_kernel<T, KEPT, TOP_K, DRAW>;
  const size_t smem = kSharedBytes + (KEPT ? (size_t)P.vecs * 16 : 0);
  if (smem > 48 * 1024) {  // always the same limit: other threads' calls may lie between this and the launch
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kMostShared);
    if (e != cudaSuccess) return e;
  }
  cudaLaunchConfig_t cfg = {};
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeClusterDimension;
  attr[0].val.clusterDim.x = (unsigned)P.cl;
  attr[0].val.clusterDim.y = 1;
  attr[0].val.clusterDim.z = 1;
  cfg.gridDim = dim3((unsigned)(rows * P.cl));
  cfg.blockDim = dim3(kThreads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = stream;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, kern, P);
}
template <typename T, bool KEPT>
cudaError_t launch_kept(const Params& P, long long rows, cudaStream_t s) {
  if (P.top_k) return P.tokens ? launch_one<T, KEPT, true, true>(P, rows, s) : launch_one<T, KEPT, true, false>(P, rows, s);
  return P.tokens ? launch_one<T, KEPT, false, true>(P, rows, s) : launch_one<T, KEPT, false, false>(P, rows, s);
}
template <typename T>
cudaError_t launch_sample(const Params& P, bool kept, long long rows, cudaStream_t s) {
  return kept ? launch_kept<T, true>(P, rows, s) : launch_kept<T, false>(P, rows, s);
}

}  // namespace sample
}  // namespace specv
