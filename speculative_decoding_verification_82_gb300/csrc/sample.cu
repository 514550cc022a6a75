// sample.cu -- spec_sample's and spec_logits_filter's C entries: argument checks, cluster geometry, launch.
//
// Host side only; the kernel lives in sample_kernel.cuh (instantiated per element type in sample_{f32,bf16,f16}.cu).
#include <limits.h>
#include <math.h>
#include <stdint.h>

#include "device_info.h"
#include "sample_kernel.cuh"
#include "spec_verify.h"

namespace specv {
namespace sample {
extern template cudaError_t launch_sample<float>(const Params&, bool, long long, cudaStream_t);
extern template cudaError_t launch_sample<__nv_bfloat16>(const Params&, bool, long long, cudaStream_t);
extern template cudaError_t launch_sample<__half>(const Params&, bool, long long, cudaStream_t);
}  // namespace sample
}  // namespace specv

namespace {

using specv::sample::kMaxCluster;
using specv::sample::Params;

bool aligned4(const void* p) { return ((uintptr_t)p & 3u) == 0; }

// Both calls; `out`: filtered rows, or `tokens`: draws.
spec_status_t run(const void* logits, spec_dtype_t dtype, int B, int R, int V, float temperature, const float* temperatures,
                  const int32_t* top_k, const float* top_p, const float* min_p, const float* u, void* out, int32_t* tokens,
                  float* probs, int32_t* kept, int32_t* err_flags, spec_stream_t stream) {
  if (dtype != SPEC_DTYPE_F32 && dtype != SPEC_DTYPE_BF16 && dtype != SPEC_DTYPE_F16) return SPEC_ERR_INVALID_ARG;
  if (B < 0 || R < 0 || V < 1) return SPEC_ERR_INVALID_ARG;
  if (!temperatures && !(temperature == 0.f || (temperature >= 0x1p-64f && temperature <= 0x1p64f))) return SPEC_ERR_INVALID_ARG;
  if (V > SPEC_MAX_SAMPLE_VOCAB) return SPEC_ERR_UNSUPPORTED;
  const long long rows = (long long)B * R;
  if (rows > INT_MAX / kMaxCluster) return SPEC_ERR_UNSUPPORTED;
  if (rows == 0) return SPEC_OK;
  const uintptr_t S = dtype == SPEC_DTYPE_F32 ? 4 : 2;
  if (!logits || (uintptr_t)logits % S || (uintptr_t)out % S) return SPEC_ERR_INVALID_ARG;
  for (const void* p : {(const void*)temperatures, (const void*)top_k, (const void*)top_p, (const void*)min_p, (const void*)u,
                        (const void*)tokens, (const void*)probs, (const void*)kept, (const void*)err_flags})
    if (!aligned4(p)) return SPEC_ERR_INVALID_ARG;
  const int sms = specv::sm_count();
  if (sms <= 0) return SPEC_ERR_CUDA;
  Params P = {};
  P.logits = static_cast<const unsigned char*>(logits);
  P.out = static_cast<unsigned char*>(out);
  P.temps = temperatures;
  P.top_k = top_k;
  P.top_p = top_p;
  P.min_p = min_p;
  P.u = u;
  P.tokens = tokens;
  P.probs = probs;
  P.kept = kept;
  P.err_flags = err_flags;
  P.temperature = temperature;
  P.V = V;
  P.fd_r = specv::make_fastdiv((uint32_t)R);
  const long long E = 16 / (long long)S, vecs = (V + 2 * E - 2) / E;  // (a row may start and end inside a vector)
  // A few rows: as many CTAs a row as there are (while slices are above 8 KB), and slices in shared memory.  More: CTAs enough to
  // fill the SMs, one and a half or two and a half each, of slices above 16 KB; without top-k, which does little but read, also until
  // slices are 128 KB, as then what four CTAs an SM read again stays in L2 (80 MB of 129); and while there are fewer than six CTAs an
  // SM until they are 40,000 tokens where all are weighed (not where bf16 values are counted).
  // us with 1 / 2 / 4 / 8 CTAs a row.  By top-k: 96 f32 rows of 128,256 filtered 36 / 31 / 25 / 37, 256 bf16 rows of 151,936
  // 44 / 53 / 53 / 74, 384 f32 rows 84 / 101 / 101 / 122.  Drawn by top-p alone: 96 f32 rows 113 / 83 / 62 / 70, 384 244 / 221 / 198 /
  // 225; 48 bf16 rows of 32,000 33 / 25 / 23 / 26, 192 41 / 35 / 46 / 65, 384 56 / 61 / 75 / 117.  768 bf16 rows of 128,256 filtered so
  // 201 / 184 / 205 / 310; 256 drawn from without rules 80 / 74 / 65 / 71, filtered by top-p 72 / 68 / 79 / 118; 200 of 50,257 drawn from without
  // rules 36 / 31 / 33 / 42.  One f32 row by top-p, slices in shared memory or not, 23.8 / 27.5.
  P.cl = 1;
  const bool in_smem = rows * kMaxCluster <= 2 * sms;
  const bool weighed = !top_k && !(out && dtype == SPEC_DTYPE_BF16);
  const auto above = [&](long long kilobytes) { return vecs * 16 > P.cl * kilobytes * 1024; };
  while (P.cl < kMaxCluster && (in_smem ? above(8)
                                        : (2 * rows * P.cl < (top_k ? 3 : 5) * sms && above(16)) || (!top_k && above(128)) ||
                                              (weighed && rows * P.cl < 6 * sms && vecs * E > P.cl * 40000LL) ||
                                              vecs * E > P.cl * (long long)specv::sample::kMostTokens))
    P.cl *= 2;
  P.vecs = (int)((vecs + P.cl - 1) / P.cl);
  P.unit = 1 << 20;
  while (P.unit * (float)(P.vecs * E) > 0x1.8p31f) P.unit *= 0.5f;  // (a part may be 1.02 units)
  const cudaStream_t s = reinterpret_cast<cudaStream_t>(stream);
  const cudaError_t e = dtype == SPEC_DTYPE_F32    ? specv::sample::launch_sample<float>(P, in_smem, rows, s)
                        : dtype == SPEC_DTYPE_BF16 ? specv::sample::launch_sample<__nv_bfloat16>(P, in_smem, rows, s)
                                                   : specv::sample::launch_sample<__half>(P, in_smem, rows, s);
  return e == cudaSuccess ? SPEC_OK : SPEC_ERR_CUDA;
}

}  // namespace

extern "C" spec_status_t spec_sample(const void* logits, spec_dtype_t dtype, int B, int R, int V, float temperature,
                                     const float* temperatures, const int32_t* top_k, const float* top_p, const float* min_p,
                                     const float* u, int32_t* tokens, float* probs, int32_t* kept, int32_t* err_flags,
                                     spec_stream_t stream) {
  if (B > 0 && R > 0 && V > 0 && V <= SPEC_MAX_SAMPLE_VOCAB && (!u || !tokens)) return SPEC_ERR_INVALID_ARG;
  return run(logits, dtype, B, R, V, temperature, temperatures, top_k, top_p, min_p, u, nullptr, tokens, probs, kept, err_flags, stream);
}

extern "C" spec_status_t spec_logits_filter(const void* logits, spec_dtype_t dtype, int B, int R, int V, float temperature,
                                            const float* temperatures, const int32_t* top_k, const float* top_p,
                                            const float* min_p, void* out, int32_t* kept, int32_t* err_flags, spec_stream_t stream) {
  if (B > 0 && R > 0 && V > 0 && V <= SPEC_MAX_SAMPLE_VOCAB && !out) return SPEC_ERR_INVALID_ARG;
  return run(logits, dtype, B, R, V, temperature, temperatures, top_k, top_p, min_p, nullptr, out, nullptr, nullptr, kept, err_flags, stream);
}
