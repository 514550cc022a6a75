// logits_process.cu -- spec_logits_process: penalties for repeated tokens, biases and grammar masks
// on the logits rows of a draft chain or tree (sm_103a).
//
// Row n's rules depend on the request (history counts, biases), the row (its mask) and the path from
// the root to n (the draft tokens accepted if n is).  One block takes a chunk of the vocabulary of
// one request and a group of its rows:
//   1. it scans the request's history and biases once and keeps what falls into its chunk in shared
//      memory: a 32-bit entry per token (occurrences in the output; whether it is in the prompt;
//      whether it has a bias) and a bitmap of the tokens with an entry;
//   2. it links every node to the nearest ancestor whose token lies in the chunk, so that a row's
//      path tokens in the chunk are a short list (most often empty);
//   3. it streams the rows' 16-byte vectors.  A vector whose bits in the bitmap and in the row's
//      mask are all trivial, as nearly all are, passes through untouched; only tokens with a bit
//      set look up their entry.
// The bitmaps are read at any bit offset, so rows whose start is not 16-byte aligned (an odd
// vocabulary) take the same path.  Each logit is read and written once: the kernel is bound by HBM
// bandwidth.  In place (out == logits), a vector that no rule touches is neither read nor written.
//
// The arithmetic is in 32 bits with one rounding per step of the definition (no contraction), and
// sums of integer counts and of biases in list order, so results do not depend on the launch.
#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_runtime.h>
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "spec_verify.h"

namespace {

constexpr int kThreads = 256;
constexpr int kMaxRows = SPEC_MAX_LOGITS_ROWS;
constexpr int kMaxChunk = 4096;  // tokens per block
constexpr int kUnroll = 4;       // vectors a thread has in flight
constexpr uint32_t kPromptBit = 0x80000000u, kBiasBit = 0x40000000u, kCountMask = 0x3fffffffu;
constexpr uint16_t kOutside = 0xffff;

struct LogitsParams {
  const unsigned char* in;
  unsigned char* out;
  int B, R, V, W, Lmax, nb;
  int chunk, rows_per_block;
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
  __device__ static uint32_t put(uint32_t, int, float f) { return __float_as_uint(f); }
};
template <>
struct Fmt<__nv_bfloat16> {
  static constexpr int VE = 8;
  using Raw = uint16_t;
  __device__ static float get(uint32_t w, int hi) { return __uint_as_float(hi ? (w & 0xffff0000u) : (w << 16)); }
  __device__ static Raw raw(float f) { return __bfloat16_as_ushort(__float2bfloat16_rn(f)); }
  __device__ static uint32_t put(uint32_t w, int hi, float f) {
    const uint32_t r = raw(f);
    return hi ? ((w & 0xffffu) | (r << 16)) : ((w & 0xffff0000u) | r);
  }
};
template <>
struct Fmt<__half> {
  static constexpr int VE = 8;
  using Raw = uint16_t;
  __device__ static float get(uint32_t w, int hi) {
    return __half2float(__ushort_as_half((unsigned short)(hi ? (w >> 16) : (w & 0xffffu))));
  }
  __device__ static Raw raw(float f) { return __half_as_ushort(__float2half_rn(f)); }
  __device__ static uint32_t put(uint32_t w, int hi, float f) {
    const uint32_t r = raw(f);
    return hi ? ((w & 0xffffu) | (r << 16)) : ((w & 0xffff0000u) | r);
  }
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

template <typename T>
__global__ void __launch_bounds__(kThreads) logits_process_kernel(const LogitsParams P) {
  constexpr int VE = Fmt<T>::VE, S = 16 / VE;
  using Raw = typename Fmt<T>::Raw;
  extern __shared__ __align__(16) unsigned char smem[];
  __shared__ uint16_t par[kMaxRows], ltok[kMaxRows], up[kMaxRows];
  __shared__ uint32_t bitmap[kMaxChunk / 32 + 3];
  const int span = P.chunk + VE;  // tokens with an entry: a chunk's last vector may reach past its end
  uint32_t* table = reinterpret_cast<uint32_t*>(smem);
  float* bias_sum = reinterpret_cast<float*>(smem) + span;  // only with biases
  const int b = blockIdx.y, t = threadIdx.x;
  const int t0 = blockIdx.x * P.chunk;
  const int t_end = min(P.V, t0 + span);
  const int words = span / 32 + 2;

  // -- 1. the request's lengths, penalties and tree
  for (int i = t; i < span; i += kThreads) table[i] = 0;
  for (int i = t; i < words; i += kThreads) bitmap[i] = 0;
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
  if (P.err_flags && blockIdx.x == 0 && blockIdx.z == 0 && t == 0) P.err_flags[b] = flags;
  const bool plain = flags != 0;  // the rows come out unprocessed

  // -- 2. the chunk's entries
  if (!plain) {
    const int32_t* h = P.history + (size_t)b * P.Lmax;
    for (int j = t; j < len; j += kThreads) {
      const int tok = __ldg(h + j);
      if (tok < t0 || tok >= t_end) continue;
      const int l = tok - t0;
      if (j < plen)
        atomicOr(&table[l], kPromptBit);
      else
        atomicAdd(&table[l], 1u);
      atomicOr(&bitmap[l >> 5], 1u << (l & 31));
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
    }
  }
  __syncthreads();

  // -- 3. the rows
  const bool in_place = P.in == P.out;
  const int r0 = blockIdx.z * P.rows_per_block, r1 = min(P.R, r0 + P.rows_per_block);
  for (int r = r0; r < r1; ++r) {
    const size_t row = ((size_t)b * P.R + r) * (size_t)P.V;
    const unsigned char* in = P.in + row * S;
    unsigned char* out = P.out + row * S;
    const int a = (int)(((uintptr_t)in & 15u) / S);  // elements before the row in its first vector
    const bool same = (((uintptr_t)in ^ (uintptr_t)out) & 15u) == 0;
    const uint32_t* mask = P.allowed ? P.allowed + ((size_t)b * P.R + r) * (size_t)P.W : nullptr;
    const int head = plain ? 0 : up[r];
    // this block's vectors: those whose first token (v VE - a) lies in [t0, t0 + chunk); block 0 also
    // takes the one that starts before the row
    const int v0 = t0 == 0 ? 0 : (t0 + a + VE - 1) / VE;
    const int v1 = (min(P.V, t0 + P.chunk) + a + VE - 1) / VE;
    for (int vb = v0; vb < v1; vb += kThreads * kUnroll) {
      uint4 x[kUnroll];
      uint32_t nz[kUnroll], ban[kUnroll];  // bits: tokens with an entry or on the path; not allowed
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = vb + u * kThreads + t;
        nz[u] = ban[u] = 0;
        if (v >= v1) continue;
        const int tok = v * VE - a;
        const bool whole = tok >= 0 && tok + VE <= P.V;
        if (!plain) {
          // bit i is token tok + i; tok may be negative in block 0's first vector only
          const int l = tok - t0;
          const int ls = l < 0 ? 0 : l;
          nz[u] = __funnelshift_r(bitmap[ls >> 5], bitmap[(ls >> 5) + 1], ls & 31);
          if (l < 0) nz[u] <<= -l;
          for (int m = head; m > 0; m = up[par[m]]) {
            const int d = (int)ltok[m] - l;
            if (d >= 0 && d < VE) nz[u] |= 1u << d;
          }
          if (mask) {
            const int ts = tok < 0 ? 0 : tok, w = ts >> 5;
            const uint32_t lo = ~__ldg(mask + w), hi = w + 1 < P.W ? ~__ldg(mask + w + 1) : 0u;
            ban[u] = __funnelshift_r(lo, hi, ts & 31);
            if (tok < 0) ban[u] <<= -tok;
          }
          const uint32_t all = (1u << VE) - 1u;
          nz[u] &= all;
          ban[u] &= all;
        }
        if (whole && (!in_place || (nz[u] | ban[u]))) x[u] = __ldcs(reinterpret_cast<const uint4*>(in + (long long)tok * S));
      }
#pragma unroll
      for (int u = 0; u < kUnroll; ++u) {
        const int v = vb + u * kThreads + t;
        if (v >= v1) continue;
        const int tok = v * VE - a;
        const bool whole = tok >= 0 && tok + VE <= P.V;
        const uint32_t touched = nz[u] | ban[u];
        if (in_place && !touched) continue;
        const int l = tok - t0;
        auto value = [&](float f, int i) {  // token tok + i with value f, under its rules
          if (ban[u] >> i & 1u) return -INFINITY;
          uint32_t n = 0;
          for (int m = head; m > 0; m = up[par[m]]) n += (int)ltok[m] == l + i;
          const uint32_t entry = table[l + i];
          return apply_rules(f, entry, n, q, (entry & kBiasBit) ? bias_sum[l + i] : 0.f);
        };
        if (whole) {
          uint32_t w[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
          if (touched) {
#pragma unroll
            for (int i = 0; i < VE; ++i)
              if (touched >> i & 1u) {
                constexpr int per = VE / 4;
                w[i / per] = Fmt<T>::put(w[i / per], i % per, value(Fmt<T>::get(w[i / per], i % per), i));
              }
          }
          if (same) {
            *reinterpret_cast<uint4*>(out + (long long)tok * S) = make_uint4(w[0], w[1], w[2], w[3]);
          } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) {
              const uint32_t word = w[i / (VE / 4)];
              *reinterpret_cast<Raw*>(out + (long long)(tok + i) * S) =
                  (Raw)(VE == 8 && (i & 1) ? word >> 16 : word);
            }
          }
        } else {  // the row's ends, element by element
          for (int i = 0; i < VE; ++i) {
            if (tok + i < 0 || tok + i >= P.V) continue;
            Raw e = *reinterpret_cast<const Raw*>(in + (long long)(tok + i) * S);
            if (touched >> i & 1u) e = Fmt<T>::raw(value(Fmt<T>::get(e, 0), i));
            *reinterpret_cast<Raw*>(out + (long long)(tok + i) * S) = e;
          }
        }
      }
    }
  }
}

int sm_count_cached() {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0) return -1;
  static int cache[64] = {0};
  if (dev < 64 && cache[dev] > 0) return cache[dev];
  int n = 0;
  if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess) return -1;
  if (dev < 64) cache[dev] = n;
  return n;
}

template <typename T>
spec_status_t launch(const LogitsParams& P, dim3 grid, size_t smem, cudaStream_t stream) {
  logits_process_kernel<T><<<grid, kThreads, smem, stream>>>(P);
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
  const int sms = sm_count_cached();
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
  if (groups > R) groups = R;
  if (groups < 1) groups = 1;
  P.rows_per_block = (int)((R + groups - 1) / groups);
  const dim3 grid((unsigned)chunks(), (unsigned)B, (unsigned)((R + P.rows_per_block - 1) / P.rows_per_block));
  const size_t smem = (size_t)(P.chunk + 8) * 4 * (num_biases > 0 ? 2 : 1);  // at most 32,832 bytes beside 6.7 KB static
  const cudaStream_t st = reinterpret_cast<cudaStream_t>(stream);
  if (dtype == SPEC_DTYPE_F32) return launch<float>(P, grid, smem, st);
  if (dtype == SPEC_DTYPE_BF16) return launch<__nv_bfloat16>(P, grid, smem, st);
  return launch<__half>(P, grid, smem, st);
}
