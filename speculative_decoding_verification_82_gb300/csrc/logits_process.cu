// logits_process.cu -- spec_logits_process: penalties for repeated tokens, biases and grammar masks
// on the logits rows of a draft chain or tree (sm_103a).
//
// Row n's rules depend on the request (history counts, biases), the row (its mask) and the path from
// the root to n (the draft tokens accepted if n is).  One block takes a chunk of the vocabulary of
// one request and a group of its rows:
//   1. it scans the request's history, biases and drafted tokens once and keeps what falls into its chunk in
//      shared memory: a 32-bit entry per token (occurrences in the output; whether it is in the prompt;
//      whether it has a bias) and a list of the tokens that have an entry or are drafted;
//   2. it links every node to the nearest ancestor whose token lies in the chunk, so that a row's
//      path tokens in the chunk are a short chain (most often empty);
//   3. it streams the rows' 16-byte vectors from input to output, with -inf where the mask has a zero;
//   4. it goes over the listed tokens of every row, spread evenly over its threads, and applies their rules
//      to the input's logits (a few hundred elements of a block's 65,536, most of them in the chunks of the
//      frequent, small ids: handled where their vectors stream, they held up whole warps and blocks:
//      134 -> 121 us on 16 61-node trees of 128,256 bf16 logits; several rows in flight and groups of 8: 107).
// The rows are prefetched to L2 ahead of step 1 (107 -> 105) and stored without staying in L1 or long in L2 (80.1 -> 78.7
// on 64 chains of 6 f32 rows).
// Mask bits are read at any offset, so rows whose start is not 16-byte aligned (an odd vocabulary) take the
// same steps, with partial vectors at their ends.  Each logit is read and written once: the kernel is bound by
// HBM bandwidth.  In place (out == logits), a vector that no rule touches is neither read nor written.
//
// The arithmetic is in 32 bits with one rounding per step of the definition (no contraction), and
// sums of integer counts and of biases in list order, so results do not depend on the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "device_info.h"
#include "fastdiv.h"
#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = SPEC_MAX_LOGITS_ROWS;
constexpr int kMaxChunk = 4096;  // tokens per block
constexpr int kMaxGroup = 8;     // rows per block (16 and 61 rows: 115 and 121 us where 8 take 108)
constexpr int kScan = 8;         // history tokens a thread has in flight
constexpr uint32_t kPromptBit = 0x80000000u, kBiasBit = 0x40000000u, kCountMask = 0x3fffffffu;
constexpr uint16_t kOutside = 0xffff;

struct LogitsParams {
  const unsigned char* in;
  unsigned char* out;
  int B, R, V, W, Lmax, nb;
  int chunk, rows_per_block, groups;
  specv::FastDiv fd_b, fd_groups;
  const int32_t *history, *history_len, *prompt_len;
  const int32_t *draft_tokens, *node_tokens, *parents;
  const float *repetition, *presence, *frequency;
  const int32_t* bias_tokens;
  const float* bias_values;
  const uint32_t* allowed;
  int32_t* err_flags;
};

template <typename T>
struct Fmt;
template <>
struct Fmt<float> {
  static constexpr int VE = 4;
  using Raw = uint32_t;
  __device__ static float get(uint32_t w, int) { return __uint_as_float(w); }
  __device__ static Raw raw(float f) { return __float_as_uint(f); }
};
template <>
struct Fmt<__nv_bfloat16> {
  static constexpr int VE = 8;
  using Raw = uint16_t;
  __device__ static float get(uint32_t w, int hi) { return __uint_as_float(hi ? (w & 0xffff0000u) : (w << 16)); }
  __device__ static Raw raw(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
};
template <>
struct Fmt<__half> {
  static constexpr int VE = 8;
  using Raw = uint16_t;
  __device__ static float get(uint32_t w, int hi) {
    return __half2float(__ushort_as_half((unsigned short)(hi ? (w >> 16) : (w & 0xffffu))));
  }
  __device__ static Raw raw(float f) { return __half_as_ushort(__float2half_rn(f)); }
};

// One request's penalties.
struct Rules {
  float rep, pres, freq;
};
__device__ __forceinline__ float apply_rules(float x, uint32_t entry, uint32_t path, const Rules& q, float bias) {
  const uint32_t c = (entry & kCountMask) + path;
  if (c || (entry & kPromptBit)) x = x > 0.f ? __fdiv_rn(x, q.rep) : __fmul_rn(x, q.rep);
  if (c) x = __fsub_rn(x, __fadd_rn(__fmul_rn(q.freq, __uint2float_rn(c)), q.pres));
  if (entry & kBiasBit) x = __fadd_rn(x, bias);
  return x;
}

// Rows whose vectors a thread has in flight together, and blocks an SM: few rows and many blocks where mask words come
// before the vectors, more rows otherwise.  (16 trees of 61 rows of 128,256 bf16: with masks 100.7 us as here, 105 with 4 rows
// and 6 blocks; without 80.5, and 93 with 2 rows and 8 blocks.  64 chains of 6 f32 rows without masks: 70.7, 80 with 4 rows
// and 4 blocks.)
template <typename T, bool MASKED>
constexpr int kRowsAtOnce = sizeof(typename Fmt<T>::Raw) == 4 ? (MASKED ? 4 : 8) : (MASKED ? 2 : 4);
template <typename T, bool MASKED>
constexpr int kBlocks = sizeof(typename Fmt<T>::Raw) == 4 ? (MASKED ? 4 : 3) : (MASKED ? 8 : 6);

// ALIGNED: every row starts on a 16-byte boundary, in both buffers.  MASKED: there are masks.
template <typename T, bool ALIGNED, bool MASKED>
__global__ void __launch_bounds__(kThreads, (kBlocks<T, MASKED>)) logits_process_kernel(const LogitsParams P) {
  constexpr int kRows = kRowsAtOnce<T, MASKED>;
  constexpr int VE = Fmt<T>::VE, S = 16 / VE;
  using Raw = typename Fmt<T>::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint16_t par[kMaxRows], ltok[kMaxRows], up[kMaxRows];
  __shared__ uint32_t bitmap[kMaxChunk / 32 + 3];
  __shared__ int listed;
  const int span = P.chunk + VE;  // places for tokens with an entry: a misaligned row's last vector reaches past the chunk
  uint32_t* table = reinterpret_cast<uint32_t*>(smem);
  uint16_t* list = reinterpret_cast<uint16_t*>(table + span);  // tokens with an entry or drafted, in any order
  float* bias_sum = reinterpret_cast<float*>(list + span);      // only with biases (span is even)
  // blocks run chunk by chunk: the first chunks, which have most rules, are not left to the end
  const unsigned cg = specv::fdiv(blockIdx.x, P.fd_b);
  const int b = (int)(blockIdx.x - cg * P.fd_b.d), t = threadIdx.x;
  const int chunk = (int)specv::fdiv(cg, P.fd_groups), group = (int)cg - chunk * P.groups;
  const int t0 = chunk * P.chunk;
  const int stop = min(P.V, t0 + P.chunk);
  // A token has one block: in place, a second one would apply its rules to what the first has written.  Aligned rows'
  // vectors end with the chunk; of misaligned rows' tokens, step 4 takes those in this block's vectors.
  const int t_end = ALIGNED ? stop : min(P.V, t0 + span);
  const int words = span / 32 + 2;

  const int r0 = group * P.rows_per_block, r1 = min(P.R, r0 + P.rows_per_block);
  const bool in_place = P.in == P.out;
  if (!in_place) {  // the rows are on their way to L2 meanwhile (in place, only what a mask forbids is read)
    const unsigned char* in = P.in + (((size_t)b * P.R + r0) * (size_t)P.V + t0) * S;
    for (int r = r0; r < r1; ++r, in += (size_t)P.V * S)
      for (int o = 128 * t; o < (stop - t0) * S; o += 128 * kThreads) asm volatile("prefetch.global.L2 [%0];" ::"l"(in + o));
  }

  // -- 1. the request's lengths, penalties and tree
  for (int i = t; i < span; i += kThreads) table[i] = 0;
  for (int i = t; i < words; i += kThreads) bitmap[i] = 0;
  if (t == 0) listed = 0;
  int len = 0, plen = 0, flags = 0;
  if (P.history) {
    len = __ldg(P.history_len + b);
    plen = P.prompt_len ? __ldg(P.prompt_len + b) : 0;
    if (len < 0 || len > P.Lmax || plen < 0 || plen > len) flags |= SPEC_ERRF_BAD_LENGTH;
  }
  Rules q;
  q.rep = P.repetition ? __ldg(P.repetition + b) : 1.f;
  q.pres = P.presence ? __ldg(P.presence + b) : 0.f;
  q.freq = P.frequency ? __ldg(P.frequency + b) : 0.f;
  if (!(q.rep > 0.f) || isinf(q.rep) || !isfinite(q.pres) || !isfinite(q.freq)) flags |= SPEC_ERRF_BAD_PENALTY;
  const bool path = P.draft_tokens || P.node_tokens;
  bool bad_tree = false, bad_token = false;
  for (int n = t; n < P.R; n += kThreads) {
    int p = n - 1, tok = -1;
    if (P.parents) {
      p = __ldg(P.parents + (size_t)b * P.R + n);
      bad_tree = bad_tree || (n == 0 ? p != -1 : (p < 0 || p >= n));
    }
    if (path && n > 0) {
      tok = P.draft_tokens ? __ldg(P.draft_tokens + (size_t)b * (P.R - 1) + n - 1) : __ldg(P.node_tokens + (size_t)b * P.R + n);
      bad_token = bad_token || tok < 0 || tok >= P.V;
    }
    par[n] = (uint16_t)(n > 0 && p >= 0 && p < n ? p : 0);
    ltok[n] = n > 0 && tok >= t0 && tok < t_end ? (uint16_t)(tok - t0) : kOutside;
  }
  if (__syncthreads_or(bad_tree)) flags |= SPEC_ERRF_BAD_TREE;
  if (__syncthreads_or(bad_token)) flags |= SPEC_ERRF_BAD_TOKEN;
  if (P.err_flags && chunk == 0 && group == 0 && t == 0) P.err_flags[b] = flags;
  const bool plain = flags != 0;  // the rows come out unprocessed

  // -- 2. the chunk's entries
  if (!plain) {
    const int32_t* h = P.history + (size_t)b * P.Lmax;
    for (int j0 = t; j0 < len; j0 += kThreads * kScan) {
      int tok[kScan];
#pragma unroll
      for (int u = 0; u < kScan; ++u) {
        const int j = j0 + u * kThreads;
        tok[u] = j < len ? __ldg(h + j) : -1;
      }
#pragma unroll
      for (int u = 0; u < kScan; ++u) {
        const int j = j0 + u * kThreads;
        if (tok[u] < t0 || tok[u] >= t_end) continue;
        const int l = tok[u] - t0;
        if (j < plen)
          atomicOr(&table[l], kPromptBit);
        else
          atomicAdd(&table[l], 1u);
        atomicOr(&bitmap[l >> 5], 1u << (l & 31));
      }
    }
    const int32_t* bt = P.bias_tokens + (size_t)b * P.nb;
    const float* bv = P.bias_values + (size_t)b * P.nb;
    for (int i = t; i < P.nb; i += kThreads) {
      const int tok = __ldg(bt + i);
      if (tok < t0 || tok >= t_end) continue;
      float sum = 0.f;
      bool first = true;  // the first entry of a token adds them all up, in list order
      for (int j = 0; j < P.nb && first; ++j)
        if (__ldg(bt + j) == tok) {
          first = j >= i;
          sum = __fadd_rn(sum, __ldg(bv + j));
        }
      if (!first) continue;
      const int l = tok - t0;
      bias_sum[l] = sum;
      atomicOr(&table[l], kBiasBit);
      atomicOr(&bitmap[l >> 5], 1u << (l & 31));
    }
    for (int n = t; n < P.R; n += kThreads) {
      int m = path ? n : 0;
      while (m > 0 && ltok[m] == kOutside) m = par[m];
      up[n] = (uint16_t)m;
      if (path && ltok[n] != kOutside) atomicOr(&bitmap[ltok[n] >> 5], 1u << (ltok[n] & 31));
    }
    __syncthreads();
    for (int i = t; i < words; i += kThreads) {
      uint32_t bits = bitmap[i];
      if (!bits) continue;
      for (int at = atomicAdd(&listed, __popc(bits)); bits; bits &= bits - 1) list[at++] = (uint16_t)(32 * i + __ffs(bits) - 1);
    }
  }
  __syncthreads();

  // -- 3. the rows' vectors
  constexpr uint32_t kAll = (1u << VE) - 1u;
  constexpr int per = VE / 4;  // elements of a word
  const uint32_t inf = (uint32_t)Fmt<T>::raw(-INFINITY);

  auto forbid = [&](uint4& x, uint32_t ban) {  // -inf where ban has a bit
    uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int y = 0; y < 4; ++y) {
      if (per == 1) {
        w[y] = ban >> y & 1u ? inf : w[y];
      } else {
        const uint32_t two = ban >> (2 * y);
        w[y] = two & 1u ? (w[y] & 0xffff0000u) | inf : w[y];
        w[y] = two & 2u ? (w[y] & 0xffffu) | (inf << 16) : w[y];
      }
    }
    x = make_uint4(w[0], w[1], w[2], w[3]);
  };

  if constexpr (ALIGNED) {
    // kRows rows at a time: their vectors are in flight together
    for (int ra = r0; ra < r1; ra += kRows) {
      const size_t row = ((size_t)b * P.R + ra) * (size_t)P.V;
      const unsigned char* in = P.in + row * S;
      unsigned char* out = P.out + row * S;
      const uint32_t* mask = MASKED && !plain ? P.allowed + ((size_t)b * P.R + ra) * (size_t)P.W : nullptr;
      if (in_place && !mask) break;
      const size_t pitch = (size_t)P.V * S;
      bool has[kRows];
#pragma unroll
      for (int u = 0; u < kRows; ++u) has[u] = ra + u < r1;
      for (int tk = t0 + t * VE; tk < stop; tk += kThreads * VE) {
        uint4 x[kRows];
        uint32_t ban[kRows];
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          ban[u] = mask && has[u] ? ~__ldg(mask + (size_t)u * P.W + (tk >> 5)) >> (tk & 31) & kAll : 0u;
#pragma unroll
        for (int u = 0; u < kRows; ++u)
          if (has[u] && (!in_place || ban[u])) {
            const uint4* at = reinterpret_cast<const uint4*>(in + u * pitch + (size_t)tk * S);
            x[u] = MASKED && per == 2 ? __ldcs(at) : *at;
          }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (ban[u]) forbid(x[u], ban[u]);
          if (has[u] && (!in_place || ban[u])) __stcs(reinterpret_cast<uint4*>(out + u * pitch + (size_t)tk * S), x[u]);
        }
      }
    }
  } else {
    // likewise, a row's vectors starting `a` elements before it: this block's are those whose first token lies
    // in [t0, stop), in block 0 also the one that starts before the row
    for (int ra = r0; ra < r1; ra += kRows) {
      const size_t row = ((size_t)b * P.R + ra) * (size_t)P.V;
      const uint32_t* mask = MASKED && !plain ? P.allowed + ((size_t)b * P.R + ra) * (size_t)P.W : nullptr;
      if (in_place && !mask) break;
      const size_t pitch = (size_t)P.V * S;
      for (int v = t0 / VE + t; v <= (stop + VE - 1) / VE; v += kThreads) {
        uint4 x[kRows];
        uint32_t ban[kRows];
        int tk[kRows];  // the vector's first token; P.V: not this block's
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          const unsigned char* in = P.in + row * S + u * pitch;
          tk[u] = v * VE - (int)(((uintptr_t)in & 15u) / S);
          ban[u] = 0;
          if (ra + u >= r1 || tk[u] >= stop || (tk[u] < t0 && t0 > 0)) tk[u] = P.V;
          if (tk[u] >= P.V) continue;
          if (mask) {  // bit i is token tk + i
            const uint32_t* m = mask + (size_t)u * P.W;
            const int ts = max(tk[u], 0), w = ts >> 5;
            ban[u] = __funnelshift_r(~__ldg(m + w), w + 1 < P.W ? ~__ldg(m + w + 1) : 0u, ts & 31);
            if (tk[u] < 0) ban[u] <<= -tk[u];
            ban[u] &= kAll;
          }
          if (tk[u] >= 0 && tk[u] + VE <= P.V && (!in_place || ban[u]))
            x[u] = *reinterpret_cast<const uint4*>(in + (size_t)tk[u] * S);
        }
#pragma unroll
        for (int u = 0; u < kRows; ++u) {
          if (tk[u] >= P.V || (in_place && !ban[u])) continue;
          const unsigned char* in = P.in + row * S + u * pitch + (long long)tk[u] * S;
          unsigned char* out = P.out + row * S + u * pitch + (long long)tk[u] * S;
          if (tk[u] >= 0 && tk[u] + VE <= P.V) {
            if (ban[u]) forbid(x[u], ban[u]);
            if ((((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0) {
              *reinterpret_cast<uint4*>(out) = x[u];
            } else {
              const uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
              for (int i = 0; i < VE; ++i)
                *reinterpret_cast<Raw*>(out + i * S) = (Raw)(per == 2 && (i & 1) ? w[i / per] >> 16 : w[i / per]);
            }
          } else {  // the row's ends, element by element
            for (int i = 0; i < VE; ++i)
              if (tk[u] + i >= 0 && tk[u] + i < P.V)
                *reinterpret_cast<Raw*>(out + i * S) = ban[u] >> i & 1u ? (Raw)inf : *reinterpret_cast<const Raw*>(in + i * S);
          }
        }
      }
    }
  }
  if (plain || listed == 0) return;
  __syncthreads();  // the rules' elements are written over the vectors'

  // -- 4. the listed tokens, row by row, spread over the threads
  const int n = listed;
  int r = r0, k = t;
  for (;;) {
    while (k >= n && r < r1) k -= n, ++r;
    if (r >= r1) break;
    const int l = list[k], tok = t0 + l;
    k += kThreads;
    const size_t row = ((size_t)b * P.R + r) * (size_t)P.V;
    if (!ALIGNED) {  // whose is the vector it lies in?
      const int a = (int)(((uintptr_t)(P.in + row * S) & 15u) / S), first = (tok + a) / VE * VE - a;
      if ((first < t0 && t0 > 0) || first >= stop) continue;
    }
    uint32_t c = 0;
    for (int m = up[r]; m > 0; m = up[par[m]]) c += ltok[m] == l;
    const uint32_t entry = table[l];
    if (!entry && !c) continue;  // drafted, but not on this row's path
    if (MASKED && !(__ldg(P.allowed + ((size_t)b * P.R + r) * (size_t)P.W + (tok >> 5)) >> (tok & 31) & 1u)) continue;
    const float f = Fmt<T>::get(*reinterpret_cast<const Raw*>(P.in + (row + tok) * S), 0);
    *reinterpret_cast<Raw*>(P.out + (row + tok) * S) = Fmt<T>::raw(apply_rules(f, entry, c, q, (entry & kBiasBit) ? bias_sum[l] : 0.f));
  }
}

template <typename T>
spec_status_t launch(const LogitsParams& P, unsigned grid, size_t smem, cudaStream_t stream) {
  const bool aligned = (((uintptr_t)P.in | (uintptr_t)P.out | ((uintptr_t)P.V * (16 / Fmt<T>::VE))) & 15u) == 0;
  auto* k = aligned ? (P.allowed ? logits_process_kernel<T, true, true> : logits_process_kernel<T, true, false>)
                    : (P.allowed ? logits_process_kernel<T, false, true> : logits_process_kernel<T, false, false>);
  k<<<grid, kThreads, smem, stream>>>(P);
  return cudaGetLastError() == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" spec_status_t spec_logits_process(const void* logits, spec_dtype_t dtype, int B, int R, int V,
                                             const int32_t* history, const int32_t* history_len,
                                             const int32_t* prompt_len, int Lmax, const int32_t* draft_tokens,
                                             const int32_t* node_tokens, const int32_t* parents,
                                             const float* repetition, const float* presence, const float* frequency,
                                             const int32_t* bias_tokens, const float* bias_values, int num_biases,
                                             const uint32_t* allowed, void* out, int32_t* err_flags,
                                             spec_stream_t stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || R < 1 || V < 1 || Lmax < 0 || num_biases < 0) return SPEC_ERR_INVALID_ARG;
  if (R > SPEC_MAX_LOGITS_ROWS || num_biases > SPEC_MAX_BIASES || B > 65535) return SPEC_ERR_UNSUPPORTED;
  if (V > INT_MAX - 2 * kMaxChunk || Lmax > (int)kCountMask) return SPEC_ERR_UNSUPPORTED;
  if (B == 0) return SPEC_OK;
  if (!logits || !out) return SPEC_ERR_INVALID_ARG;
  if (Lmax > 0 && (!history || !history_len)) return SPEC_ERR_INVALID_ARG;
  if (draft_tokens && node_tokens) return SPEC_ERR_INVALID_ARG;
  if ((node_tokens != nullptr) != (parents != nullptr)) return SPEC_ERR_INVALID_ARG;
  if (num_biases > 0 && (!bias_tokens || !bias_values)) return SPEC_ERR_INVALID_ARG;
  const int S = dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (((uintptr_t)logits % S) || ((uintptr_t)out % S)) return SPEC_ERR_INVALID_ARG;
  const int sms = specv::sm_count();
  if (sms <= 0) return SPEC_ERR_CUDA;
  LogitsParams P = {};
  P.in = static_cast<const unsigned char*>(logits);
  P.out = static_cast<unsigned char*>(out);
  P.B = B;
  P.R = R;
  P.V = V;
  P.W = (int)(((long long)V + 31) / 32);
  P.Lmax = Lmax;
  P.nb = num_biases;
  P.history = Lmax > 0 ? history : nullptr;
  P.history_len = history_len;
  P.prompt_len = prompt_len;
  P.draft_tokens = R > 1 ? draft_tokens : nullptr;
  P.node_tokens = node_tokens;
  P.parents = parents;
  P.repetition = repetition;
  P.presence = presence;
  P.frequency = frequency;
  P.bias_tokens = bias_tokens;
  P.bias_values = bias_values;
  P.allowed = allowed;
  P.err_flags = err_flags;
  // Blocks: at least four per SM.  First smaller chunks (more scans of the history, which come from
  // L2), then groups of rows.
  const long long want = 4LL * sms;
  P.chunk = kMaxChunk;
  auto chunks = [&] { return ((long long)V + P.chunk - 1) / P.chunk; };
  while (P.chunk > 1024 && chunks() * B < want) P.chunk /= 2;
  long long groups = (want + chunks() * B - 1) / (chunks() * B);
  if (groups < (R + kMaxGroup - 1) / kMaxGroup) groups = (R + kMaxGroup - 1) / kMaxGroup;
  if (groups > R) groups = R;
  P.rows_per_block = (int)((R + groups - 1) / groups);
  P.groups = (int)((R + P.rows_per_block - 1) / P.rows_per_block);
  if (chunks() * P.groups > INT_MAX / B) return SPEC_ERR_UNSUPPORTED;
  P.fd_b = specv::make_fastdiv((uint32_t)B);
  P.fd_groups = specv::make_fastdiv((uint32_t)P.groups);
  const unsigned grid = (unsigned)(chunks() * P.groups * B);
  const size_t smem = (size_t)(P.chunk + 8) * (num_biases > 0 ? 10 : 6);  // at most 41,040 bytes beside 6.7 KB static
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SPEC_DTYPE_F32) return launch<float>(P, grid, smem, st);
  if (dtype == SPEC_DTYPE_BF16) return launch<__nv_bfloat16>(P, grid, smem, st);
  return launch<__half>(P, grid, smem, st);
}
