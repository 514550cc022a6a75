// attention_kernel.cuh -- the attention kernel of spec_attention (sm_103a): tcgen05 products over TMA-loaded
// pages, one CTA per SM, work split evenly over the SMs along the KV axis.
//
// Mathematics.  For a row (token t, query head) with scores s_j = scale q . k_j over the positions j it
// attends to, the output is sum_j 2^(c s_j - m) v_j / sum_j 2^(c s_j - m), c = log2(e), for any m.  One
// pass over the tiles keeps a running m, the sum l of the weights in 32 bits and the weighted sum O in
// 32-bit accumulators; when m has to grow, l and O are multiplied by 2^(m_old - m_new).  m follows the
// maximum only when that outgrows it by more than 2^16 (bf16) or 2^8 (f16, whose range ends there): weights up
// to that are as exact, in their type and in 32-bit sums, as below 1, and O is seldom touched.  (One row of a warp
// is enough to have its O rescaled: 61-node trees over 8192 positions, scores of 2 standard deviations, took
// 174 us with 2^8 and 161 with 2^16.)  Two partial results of a row join by the same factor.
//
// Rows.  The query heads of one KV head read the same K and V, so the rows of a (request, KV head) are
// its tokens times its group of heads: row r is token r / G, head r % G.  A tile is 128 rows by 128
// positions.  Two streams run on each SM, each with its own S and O accumulators in tensor memory and
// its own softmax warpgroup, so that one stream's softmax overlaps the other's products:
//   pair  (more than 128 rows): the streams hold two row tiles and share every K and V tile;
//   split (up to 128 rows): the streams share one row tile and take alternate K and V tiles; their
//         results join at the end.  Padded rows cost tensor time, which the loads hide: a 128-position
//         tile of 16-bit K and V takes about 2,800 cycles of an SM's share of HBM, its products 1,024.
//
// Work.  The tiles of all (request, row tile, KV head) items in sequence are cut into equal ranges, one
// per CTA, so ragged lengths and few requests still fill every SM.  Ends of ranges that fall inside an
// item leave partial results (O, m, l) in the workspace, which attention_combine_kernel joins.  Where a request
// has two or four row units, as many CTAs side by side take the same range of tiles for one unit each (a lane
// each), so that all but one read K and V from L2.
//
// Roles.  Warps 0-3 and 4-7: softmax of stream 0 and 1, a thread per row.  Warp 8: one lane issues the
// products of both streams in turn (the tensor cores run them in that order, which the places that scores
// and weights share rely on).  Warps 9 and 11: TMA loads of K and V pages into a ring of tiles, each every
// second box (a lane takes about 54 cycles to issue one: with 16-position pages, one warp's 860 a tile held
// up the products: 64 chains over 4096 positions: 164 -> 151 us).  Warp 10: query rows and tree parents.  Warps
// 12-15 and 16-19 (e4m3): K and V codes to 16 bits.  Every wait is bounded: one that gives up sets the CTA's
// abort flag, every role leaves, copies and products in flight are waited for, and the requests get
// SPEC_ERRF_TIMEOUT; the joining kernel repeats it, since CTAs that start later write their requests' flags over it.
//
// Measured, 64 query heads over 8 KV heads of 128: 64 chains of 6 tokens over 4096 bf16 positions 149 us (5.5 TB/s of K and V:
// bound by HBM), over 8192 e4m3 positions 230 us (3.7 TB/s: bound by the codes' way to f16 beside the softmax); 16 trees of 61
// nodes over 8192 157 us (1.25 PFLOP/s) and 2 x 2048 f16 tokens after 2048 295 us (1.17), both with pauses between the calls; after
// seconds of calls the power cap lowers the clock, and they take 174 and 301.  A tile's products take 1,024 cycles
// alone and 1,200-1,270 here, where the scores' operands come out of shared memory at all the 128 bytes a clock it has, and
// two streams do not quite cover a softmax of 1,215 cycles and the products it waits for.
#pragma once

#include <cuda.h>
#include <math.h>

#include <type_traits>

#include "fastdiv.h"
#include "verify_common.cuh"

namespace specv {
namespace attn {

constexpr int kTile = 128;       // rows of a row tile, positions of a KV tile
constexpr int kMaxCtas = 160;    // at most this many CTAs (the workspace's partial results)
constexpr int kMaxTree = SPEC_MAX_WALK_NODES;
constexpr float kLog2e = 1.4426950408889634f;

constexpr int kGaveUp = 1 << 30;
struct Record {  // an item whose tiles several CTAs share: it starts in the CTA that writes the record
  int b, qp, h;  // b < 0: none
  int last;      // the last CTA with a part of it (every P.lanes-th from this one on); kGaveUp: a wait of this CTA ran out
};

struct Params {
  CUtensorMap kmap, vmap, qmap;
  const unsigned char* q;
  const float *ks, *vs;
  const int32_t *table, *context_len, *chunk_len, *parents;
  unsigned char* out;
  float* lse;
  int32_t* err_flags;
  float* part_o;   // [2 kMaxCtas][D / 4][unit rows] float4
  float2* part_ml; // [2 kMaxCtas][unit rows]: m (log2), l
  Record* rec;     // [kMaxCtas]
  long long q_stride, num_pages;
  int B, T, Hq, H, G, P, page_log2;
  int nqp;         // row units (pair: 256 rows, split: 128) of a request with T tokens
  int lanes;       // 1, or nqp: CTA c works on units c % lanes alone
  int q_box;       // tokens of qmap's box, 0: query rows are gathered by loads
  FastDiv fd_g, fd_nqp;
  float c;         // scale * log2(e)
};

template <int D, bool E4M3, bool PAIR>
struct Cfg {
  static constexpr int kHalves = D / 64;               // 64-element (128-byte) column halves of a tile
  static constexpr int kHalfBytes = kTile * 128;
  static constexpr int kTileBytes = kHalves * kHalfBytes;
  static constexpr int kRawBytes = kTile * D;          // a tile of codes
  static constexpr int kQTiles = PAIR ? 2 : 1;         // (split: two buffers while 64 rows do, else one)
  static constexpr int kRaw = E4M3 ? (D == 64 ? 6 : PAIR ? 3 : 4) : 0;
  static constexpr int kSlots = E4M3 ? (D == 64 ? 6 : PAIR ? 3 : 4) : (D == 64 ? 10 : PAIR ? 5 : 6);
  // The ring's order is K(0), K(1), V(0), K(2), V(1), ...: a tile's V is wanted a softmax later than its K.
  // What the softmax takes of a tile's scales is written with its K and kept as long as its softmax is due.  The streams
  // may drift apart, but by no more than the raw ring is long: its copies are in sequence, and one whose slot is
  // taken stops it.  So no tile 8 or more ahead is converted meanwhile.
  static constexpr int kScales = E4M3 ? 8 : 0;
  static constexpr int kQ = 0;
  static constexpr int kKv = kQTiles * kTileBytes;
  static constexpr int kRawAt = kKv + kSlots * kTileBytes;
  static constexpr int kParAt = kRawAt + kRaw * kRawBytes;  // parents: 16 bits each (pair), 2 x 128 bytes (split)
  static constexpr int kScaleAt = kParAt + (PAIR ? 2 * kMaxTree : 2 * kTile);
  static constexpr int kQexpAt = kScaleAt + kScales * 48;  // exponents of the query rows' scales
  static constexpr int kMlAt = kQexpAt + (E4M3 ? 2 * kTile : 0);          // split: a float2 a row
  static constexpr int kBars = kMlAt + (PAIR ? 0 : kTile * 8);
  static constexpr int kBytes = kBars + 560;
  static constexpr int kConvert = 12;                      // the first of the warps that convert codes (8 of them)
  static constexpr int kThreads = (kConvert + (E4M3 ? 8 : 0)) * 32;
  static constexpr int kLaunchRegs = 65536 / kThreads / 8 * 8;  // registers a thread at launch
  static constexpr int kMoreRegs = E4M3 ? 120 : 192, kLessRegs = E4M3 ? 80 : 120;
  static_assert(8 * kMoreRegs + (kThreads / 32 - 8) * kLessRegs <= kThreads / 32 * kLaunchRegs, "registers");
  static_assert(kBytes <= 232448 && kBars % 16 == 0, "shared memory");
  static_assert(kRaw <= kSlots, "see the converters");
};

// ------------------------------------------------------------------------- PTX wrappers ----
__device__ __forceinline__ void tc_alloc(uint32_t* at) {
  asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], 512;" ::"r"(smem_addr(at)) : "memory");
  asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tc_free(uint32_t t) {
  asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, 512;" ::"r"(t) : "memory");
}
__device__ __forceinline__ void tc_fence_before() { asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_fence_after() { asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_ld() { asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_wait_st() { asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory"); }
__device__ __forceinline__ void tc_commit(uint64_t* bar) {
  asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];" ::"r"(smem_addr(bar)) : "memory");
}
__device__ __forceinline__ void tc_mma_ss(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
__device__ __forceinline__ void tc_mma_ts(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
  asm volatile(
      "{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
      "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n\t}" ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc)
      : "memory");
}
// 32 columns of this warp's 32 lanes.
__device__ __forceinline__ void tc_ld32(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
        "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
        "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
      : "r"(t));
}
__device__ __forceinline__ void tc_st32(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x32.b32 [%32], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, "
      "%16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]),
      "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]), "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]),
      "r"(r[29]), "r"(r[30]), "r"(r[31]), "r"(t)
      : "memory");
}
__device__ __forceinline__ void tc_ld16(uint32_t t, uint32_t* r) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15}, [%16];"
      : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
        "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
      : "r"(t));
}
__device__ __forceinline__ void tc_st8(uint32_t t, const uint32_t* r) {
  asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%8], {%0, %1, %2, %3, %4, %5, %6, %7};" ::"r"(r[0]), "r"(r[1]),
               "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(t)
               : "memory");
}
__device__ __forceinline__ void tc_st16(uint32_t t, const uint32_t* r) {
  asm volatile(
      "tcgen05.st.sync.aligned.32x32b.x16.b32 [%16], "
      "{%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15};" ::"r"(r[0]),
      "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]), "r"(r[8]), "r"(r[9]), "r"(r[10]),
      "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]), "r"(t)
      : "memory");
}
template <int W>
__device__ __forceinline__ void tc_ld_cols(uint32_t t, uint32_t* r) {
  if constexpr (W == 32)
    tc_ld32(t, r);
  else
    tc_ld16(t, r);
}
template <int W>
__device__ __forceinline__ void tc_st_cols(uint32_t t, const uint32_t* r) {
  if constexpr (W == 32)
    tc_st32(t, r);
  else
    tc_st16(t, r);
}
// Two 32-bit operations in one instruction.
__device__ __forceinline__ float2 fma2(float2 a, float2 b, float2 c) {
  float2 r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
__device__ __forceinline__ float2 add2(float2 a, float2 b) {
  float2 r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
// A box of the 4-dimensional map at (x, y, z, w); x is a multiple of 16 bytes.
__device__ __forceinline__ void tma_load_4d(uint32_t dst, const CUtensorMap* map, int x, int y, int z, int w, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], [%6];" ::"r"(
          dst),
      "l"(map), "r"(x), "r"(y), "r"(z), "r"(w), "r"(smem_addr(bar))
      : "memory");
}
__device__ __forceinline__ void mbar_arrive_expect(uint64_t* bar, uint32_t bytes) {
  asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_addr(bar)), "r"(bytes) : "memory");
}
// True for one lane of the (whole) warp.
__device__ __forceinline__ bool elect_one() {
  uint32_t p;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
  return p != 0;
}
// One arrival for a warp, after what each of its lanes did (and fenced) before.
__device__ __forceinline__ void mbar_arrive_warp(uint64_t* bar) {
  __syncwarp();
  if ((threadIdx.x & 31) == 0) mbar_arrive(bar);
}
__device__ __forceinline__ void sts128(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
  asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};" ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}
__device__ __forceinline__ uint4 lds128_at(uint32_t at) {
  uint4 v;
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
  return v;
}

// Matrix descriptor: a 128-byte-swizzled tile at `at`.  K-major operands (Q, K): rows of 128 bytes, 8-row
// groups 1024 bytes apart.  V (positions are its K axis, its D elements contiguous): 64-element columns
// `lbo` bytes apart, 8-position groups 1024 bytes apart.
__device__ __forceinline__ uint64_t tile_desc(uint32_t at, uint32_t lbo) {
  return (uint64_t)((at & 0x3ffffu) >> 4) | ((uint64_t)(lbo >> 4) << 16) | ((uint64_t)(1024 >> 4) << 32) | (1ull << 46) | (2ull << 61);
}

template <typename T>
struct Half;
template <>
struct Half<__nv_bfloat16> {
  static constexpr uint32_t kFmt = 1;       // tcgen05 operand format
  static constexpr uint32_t kExp = 0x7f80u; // exponent bits
  static constexpr float kGrow = 16.f;      // how far (log2) the maximum may outgrow m before O is rescaled
  __device__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
template <>
struct Half<__half> {
  static constexpr uint32_t kFmt = 0;
  static constexpr uint32_t kExp = 0x7c00u;
  static constexpr float kGrow = 8.f;
  __device__ static uint32_t pack(float lo, float hi) {
    uint32_t r;
    asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
  }
};
// -------------------------------------------------------------------------- work items ----
// One request's lengths; bad: they do not fit, and the request has no tiles.
struct Lens {
  int L, n;
  bool bad;
};
__device__ __forceinline__ Lens request_lens(const Params& P, int b) {
  Lens r;
  r.L = __ldg(P.context_len + b);
  r.n = P.chunk_len ? __ldg(P.chunk_len + b) : P.T;
  r.bad = r.L < 0 || r.n < 0 || r.n > P.T || (long long)r.L + r.n > ((long long)P.P << P.page_log2);
  return r;
}
// KV tiles of row unit qp (UR rows): up to its last token in a chain, the whole chunk in a tree.
template <int UR>
__device__ __forceinline__ int unit_tiles(const Params& P, const Lens& s, int qp) {
  const int rows = s.n * P.G, r0 = qp * UR;  // (T G and the positions are at most INT_MAX / 2)
  if (s.bad || r0 >= rows) return 0;
  const int last = P.parents ? s.n - 1 : (int)fdiv((unsigned)min(r0 + UR, rows) - 1u, P.fd_g);
  return (s.L + last + kTile) / kTile;
}

struct Plan {  // a CTA's range of the tile sequence
  long long take;     // its tiles
  int b, qp, h, off;  // where it starts: item and tile
};

// A stretch of one item's tiles: offsets [off, off + take) of its tiles counted from the last one.
struct Seg {
  int b, qp, h, L, n;
  int nt, off, take;
};

template <int UR>
struct SegIter {
  long long left;
  int b, qp, h, off;
  __device__ explicit SegIter(const Plan& pl) : left(pl.take), b(pl.b), qp(pl.qp), h(pl.h), off(pl.off) {}
  __device__ bool next(const Params& P, Seg& s) {
    if (left <= 0) return false;
    while (b < P.B) {
      const Lens r = request_lens(P, b);
      const int nt = unit_tiles<UR>(P, r, qp);
      if (nt > 0) {
        s.b = b, s.qp = qp, s.h = h, s.L = r.L, s.n = r.n, s.nt = nt, s.off = off;
        s.take = (int)(left < nt - off ? left : nt - off);
        left -= s.take;
        off = 0;
        if (++h == P.H) h = 0;
      }
      if (nt == 0 || h == 0) {
        if (P.lanes > 1)
          ++b;
        else if (++qp == P.nqp)
          qp = 0, ++b;
      }
      if (nt > 0) return true;
    }
    return false;
  }
};

// ------------------------------------------------------------------------------- kernel ----
template <typename T, int D, bool E4M3, bool PAIR>
__global__ void __launch_bounds__(Cfg<D, E4M3, PAIR>::kThreads, 1) attention_kernel(const __grid_constant__ Params P) {
  using C = Cfg<D, E4M3, PAIR>;
  constexpr int UR = PAIR ? 2 * kTile : kTile;
  constexpr int NS = C::kSlots, NR = C::kRaw > 0 ? C::kRaw : 1;
  extern __shared__ __align__(1024) unsigned char smem[];  // (no static shared memory: swizzled tiles start on 1 KB)
  const uint32_t sbase = smem_addr(smem);
  uint64_t* bars = reinterpret_cast<uint64_t*>(smem + C::kBars);
  uint64_t* full = bars;               // [NS] a KV tile is in place
  uint64_t* empty = full + NS;         // [NS] its products are done
  uint64_t* raw_full = empty + NS;     // [NR] a tile of codes is in place
  uint64_t* raw_empty = raw_full + NR; // [NR] it has been converted
  uint64_t* s_full = raw_empty + NR;   // [2] a stream's scores
  uint64_t* p_ready = s_full + 2;      // [2] its weights (and O rescaled)
  uint64_t* o_full = p_ready + 2;      // [2] its O is complete
  uint64_t* q_full = o_full + 2;       // [2] query rows of a segment
  uint64_t* q_empty = q_full + 2;      // [2]
  uint64_t* mark = q_empty + 2;        // [8] a masked tile's V has been looked over
  uint64_t* join = mark + 8;           // [3] split: m and l of stream 1; the factors; both O have been read
  uint64_t* q_raw = join + 3;          // [1] bf16 queries before they become f16
  uint64_t* drain = q_raw + 1;         // [1] after an abort
  static_assert((2 * NS + 2 * NR + 23) * 8 <= 384, "barriers");
  uint32_t* words = reinterpret_cast<uint32_t*>(smem + C::kBars + 384);
  uint32_t* tmem_at = words;                                 // [1]
  volatile int* abort = reinterpret_cast<int*>(words + 1);   // [1]
  volatile int* tree_bad = reinterpret_cast<int*>(words + 2);// [2] the request's tree is malformed
  uint32_t* poison = words + 4;                              // [8][4] positions of a tile with a non-finite V
  Plan& plan = *reinterpret_cast<Plan*>(smem + C::kBars + 528);
  static_assert(sizeof(Plan) <= 32, "plan");
  long long* scan = reinterpret_cast<long long*>(smem + C::kParAt);  // [warps], set-up only
  using Parent = typename std::conditional<PAIR, uint16_t, uint8_t>::type;   // (split: at most 128 tokens)
  constexpr Parent kNoParent = (Parent)~(Parent)0;
  Parent* par = reinterpret_cast<Parent*>(smem + C::kParAt);                // pair [kMaxTree], split [2][128]
  float* exps = reinterpret_cast<float*>(smem + C::kScaleAt);               // [kScales][2^k, v, 2^-v][4]: see the converters
  uint8_t* qexp = smem + C::kQexpAt;                                        // pair [256], split [2][128]
  constexpr int ES = C::kScales > 0 ? C::kScales : 1;
  using OT = typename std::conditional<E4M3, __half, T>::type;              // the products' operands
  const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;

  // -- set-up, and this CTA's range of the tile sequence
  if (tid == 0) {
    for (int i = 0; i < NS; ++i) {
      mbar_init(full + i, E4M3 ? 4 : 2);
      mbar_init(empty + i, 1);
    }
    for (int i = 0; i < NR; ++i) {
      mbar_init(raw_full + i, 2);
      mbar_init(raw_empty + i, 4);
    }
    for (int i = 0; i < 2; ++i) {
      mbar_init(s_full + i, 1);
      mbar_init(p_ready + i, 4);
      mbar_init(o_full + i, 1);
      mbar_init(q_full + i, 32);
      mbar_init(q_empty + i, 1 + 8);
    }
    for (int i = 0; i < 8; ++i) mbar_init(mark + i, 4);
    for (int i = 0; i < 3; ++i) mbar_init(join + i, i == 1 ? 4 : 8);
    mbar_init(q_raw, 1);
    mbar_init(drain, 1);
    fence_mbar_init();
    *abort = 0;
    plan.take = 0;
  }
  if (warp == 8) tc_alloc(tmem_at);
  {
    // units of this CTA's lane: all (b, qp) in sequence, or (b, lane)
    const int step = P.lanes > 1 ? 1 : P.nqp, lane_qp = P.lanes > 1 ? (int)(blockIdx.x % P.lanes) : 0;
    const int U = P.B * step;  // (at most INT_MAX)
    const int ctas = gridDim.x / P.lanes, cta = blockIdx.x / P.lanes;
    const int each = (int)(((unsigned)U + C::kThreads - 1) / C::kThreads);
    const int ua = (int)min((long long)U, (long long)each * tid), ub = (int)min((long long)U, (long long)ua + each);
    const int b0 = P.lanes > 1 ? ua : (int)fdiv((unsigned)ua, P.fd_nqp), qp0 = P.lanes > 1 ? 0 : ua - b0 * P.nqp;
    long long sum = 0;
    for (int u = ua, b = b0, qp = qp0; u < ub; ++u) {
      sum += (long long)unit_tiles<UR>(P, request_lens(P, b), lane_qp + qp) * P.H;
      if (++qp == step) qp = 0, ++b;
    }
    long long incl = sum;
    for (int o = 1; o < 32; o <<= 1) {
      const long long v = __shfl_up_sync(kFull, incl, o);
      if (lane >= o) incl += v;
    }
    if (lane == 31) scan[warp] = incl;
    if (tid == 0) P.rec[blockIdx.x].b = -1, P.rec[blockIdx.x].last = 0;
    __syncthreads();  // (and before the one thread that may write the record)
    long long before = 0, total = 0;
    for (int w = 0; w < C::kThreads / 32; ++w) {
      before += w < warp ? scan[w] : 0;
      total += scan[w];
    }
    const long long per = max(1LL, (total + ctas - 1) / ctas);
    const long long start = min(total, per * cta), end = min(total, start + per);
    long long at = before + incl - sum;
    const bool has_start = start < end && start >= at && start < at + sum;
    const bool has_end = start < end && end < total && end >= at && end < at + sum;
    if (has_start || has_end)
      for (int u = ua, b = b0, qp = qp0; u < ub; ++u) {
        const int nt = unit_tiles<UR>(P, request_lens(P, b), lane_qp + qp);
        const long long next = at + (long long)nt * P.H;
        if (has_start && start >= at && start < next) {
          plan.take = end - start;
          plan.b = b;
          plan.qp = lane_qp + qp;
          plan.h = (int)((start - at) / nt);
          plan.off = (int)((start - at) % nt);
        }
        if (has_end && end >= at && end < next) {
          const int h = (int)((end - at) / nt);
          const long long item = at + (long long)h * nt;
          if (item >= start && item < end) {  // it starts here and goes on
            Record r;
            r.b = b, r.qp = lane_qp + qp, r.h = h;
            r.last = (int)((item + nt - 1) / per) * P.lanes + lane_qp;
            P.rec[blockIdx.x] = r;
          }
        }
        at = next;
        if (++qp == step) qp = 0, ++b;
      }
  }
  tc_fence_before();
  __syncthreads();
  tc_fence_after();
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
  const uint32_t tmem = *tmem_at;
  // tensor memory columns: S of both streams (their weights take its first half), then their O
  auto col_s = [&](int s) { return tmem + s * kTile; };
  auto col_o = [&](int s) { return tmem + (2 + s) * kTile; };

  // tiles of stream s in a segment
  auto stream_tiles = [&](const Seg& g, int s) {
    if (PAIR) return s == 0 || g.qp * UR + kTile < g.n * P.G ? g.take : 0;
    return (g.take + 1 - s) / 2;
  };
  // places in the ring, from the segment's first, of the K and V of its tile i
  auto k_at = [](int i) { return i == 0 ? 0 : 2 * i - 1; };
  auto v_at = [](const Seg& g, int i) { return i + 1 < g.take ? 2 * i + 2 : 2 * i + 1; };
  // Query buffers: pair one of two tiles; split two of 64 rows or one of 128 (products read 128 rows of
  // whatever is there: a row's scores concern that row alone).
  const int qbufs = !PAIR && P.T * P.G <= 64 ? 2 : 1;
  const int qhalf = !PAIR && P.T * P.G <= 64 ? C::kHalfBytes / 2 : C::kHalfBytes;  // bytes of a column half
  const int qbytes = qhalf * C::kHalves;                                           // and of a row tile
  bool ok = true;  // no wait gave up

  // The softmax warps take registers over from the others, each group of four warps alike; the launch's total stays.
  if (warp < 8)
    asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(C::kMoreRegs));
  else
    asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(C::kLessRegs));
  if (warp < 8) {
    // ======================================================================= softmax ====
    const int s = warp >> 2, row = tid & 127;
    const uint32_t lanes = (uint32_t)(warp & 3) << 21;  // this warp's 32 lanes of tensor memory
    const uint32_t S = col_s(s) + lanes, O = col_o(s) + lanes;
    if (s == 1) {
      // requests' flags, and zeros for those whose lengths do not fit
      for (int b = blockIdx.x; b < P.B; b += gridDim.x) {
        const Lens r = request_lens(P, b);
        int flags = r.bad ? SPEC_ERRF_BAD_LENGTH : 0;
        bool bad = false;
        if (!r.bad && P.parents)
          for (int i = row; i < r.n; i += kTile) {
            const int p = __ldg(P.parents + (size_t)b * P.T + i);
            bad = bad || (i == 0 ? p != -1 : (p < 0 || p >= i));
          }
        int any;
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(any) : "r"((int)bad) : "memory");
        if (any) flags |= SPEC_ERRF_BAD_TREE;
        bad = false;
        if (!flags) {
          const int pages = (int)(((long long)r.L + r.n + (1LL << P.page_log2) - 1) >> P.page_log2);
          for (int i = row; i < pages && r.n > 0; i += kTile) {
            const int p = __ldg(P.table + (size_t)b * P.P + i);
            bad = bad || p < 0 || p >= P.num_pages;
          }
        }
        asm volatile("{\n\t.reg .pred p, q;\n\tsetp.ne.b32 p, %1, 0;\n\tbar.red.or.pred q, 1, 128, p;\n\tselp.b32 %0, 1, 0, q;\n\t}" : "=r"(any) : "r"((int)bad) : "memory");
        if (any) flags |= SPEC_ERRF_BAD_SLOT;
        if (row == 0 && P.err_flags) P.err_flags[b] = flags;
        if (r.bad) {
          const size_t rows = (size_t)P.T * P.Hq;
          uint4* o = reinterpret_cast<uint4*>(P.out + (size_t)b * rows * D * 2);
          for (size_t i = row; i < rows * D / 8; i += kTile) o[i] = make_uint4(0, 0, 0, 0);
          if (P.lse)
            for (size_t i = row; i < rows; i += kTile) P.lse[(size_t)b * rows + i] = -INFINITY;
        }
      }
    }
    // Registers: what spills goes to an L1 that shared memory leaves little of, at L2's latency (e4m3 with 50 words of it:
    // every role ran at half its pace).  With 120 a thread columns come 16 at a time and loops are unrolled in part.
    constexpr int kSteps = E4M3 ? 2 : 4, W = E4M3 ? 16 : 32;
    uint32_t ph_s = 0, ph_o = 0, ph_join = 0;  // parities of s_full, o_full, join
    uint32_t ph_mark = 0;  // bit i: parity of mark[i]
    uint32_t kv = 0;              // KV tiles before this segment
    SegIter<UR> it(plan);
    Seg g, coming;
    bool more = it.next(P, g);
    for (int seg = 0; ok && more; ++seg, g = coming) {
      const int cnt = stream_tiles(g, s), cnt1 = s == 1 ? cnt : stream_tiles(g, 1);
      const int r0 = g.qp * UR + (PAIR ? s * kTile : 0);  // (a unit's rows fit an int: T G <= INT_MAX)
      const int rows = g.n * P.G;
      const int r = r0 + row;
      const bool live = r < rows;
      const bool warp_live = r0 + (warp & 3) * 32 < rows;
      const int t = live ? (int)fdiv((unsigned)r, P.fd_g) : 0;
      const int qb = seg % qbufs;
      const Parent* pr = par + (PAIR ? 0 : qb * kTile);
      // positions below `all` are seen by every row of the unit
      const int all = P.parents ? g.L : g.L + (int)fdiv((unsigned)(g.qp * UR), P.fd_g) + 1;
      const int stop = g.L + g.n;
      // the segment's first tiles (from the end) are masked
      if (PAIR && cnt == 0) {  // stream 0 marks them alone
        const int marked = max(0, min(g.take, g.nt - g.off - all / kTile));
        for (int k = 0; k < marked; ++k) ph_mark ^= 1u << (k & 7);
      }
      int node = t;  // tree: the next ancestor to mark
      float m = -INFINITY, l = 0.f;
      ok = mbar_wait_warp(q_full + qb, (uint32_t)((seg / qbufs) & 1), abort);  // parents are in place
      const bool bad_tree = ok && P.parents && tree_bad[qb];
      // e4m3: scores come in units of the row's query scale (a power of two; see the query warp)
      float cq = P.c;
      if constexpr (E4M3 && !std::is_same<T, __half>::value)
        cq *= __uint_as_float((uint32_t)qexp[PAIR ? s * kTile + row : qb * kTile + row] << 23);
      for (int k = 0; ok && k < cnt; ++k) {
        const int i = PAIR ? k : 2 * k + s;  // the segment's tile
        const int j0 = (g.nt - 1 - (g.off + i)) * kTile;
        const bool masked = j0 + kTile > all;
        const uint32_t vseq = 2 * kv + v_at(g, i), vslot = vseq % NS, vpar = (vseq / NS) & 1;
        ok = mbar_wait_warp(s_full + s, ph_s, abort);
        ph_s ^= 1;
        if (!ok) break;
        tc_fence_after();
        uint32_t seen[4] = {0, 0, 0, 0};  // a masked tile's positions that the row sees
        if (masked) {
          // the prefix, then the row's path
          const int lim = P.parents ? g.L - j0 : g.L + t + 1 - j0;
#pragma unroll
          for (int w = 0; w < 4; ++w) {
            const int x = lim - 32 * w;
            seen[w] = x >= 32 ? ~0u : x <= 0 ? 0u : (1u << x) - 1u;
          }
          if (P.parents) {
            while (node >= 0 && g.L + node >= j0) {
              const int x = g.L + node - j0;
              if (x < kTile) {
                const uint32_t bit = 1u << (x & 31);
                seen[0] |= x < 32 ? bit : 0u;
                seen[1] |= (x >> 5) == 1 ? bit : 0u;
                seen[2] |= (x >> 5) == 2 ? bit : 0u;
                seen[3] |= (x >> 5) == 3 ? bit : 0u;
              }
              const Parent p = pr[node];
              node = p == kNoParent ? -1 : (int)p;
            }
          }
          // what it does not see becomes -inf in place
          if (warp_live) {
#pragma unroll 1
            for (int w = 0; w < kTile; w += W) {
              uint32_t bits = w < 32 ? seen[0] : w < 64 ? seen[1] : w < 96 ? seen[2] : seen[3];
              if constexpr (W == 16) bits = bits >> (w & 16) & 0xffffu;
              __syncwarp();
              if (__all_sync(kFull, bits == (W == 16 ? 0xffffu : ~0u))) continue;
              uint32_t x[W];
              tc_ld_cols<W>(S + w, x);
              tc_wait_ld();
#pragma unroll
              for (int j = 0; j < W; ++j) x[j] = bits & (1u << j) ? x[j] : 0xff800000u;
              tc_st_cols<W>(S + w, x);
            }
            tc_wait_st();
          }
        }
        if (warp_live) {
          // Scores to log2 units (c > 0).  e4m3: positions 32 w on are in units of 2^k[w], their V rows in units of
          // 2^v[w].  The factor is kept above zero and finite: hidden scores are -inf, and -inf times 0 would be a NaN, as
          // would 0 times infinity.  (Scores are below 2^33 here, and above 2^-48 or 0: where the product is below
          // 2^-126 they are nothing against 1 either way, where it overflows they are above 2^80 or 0.)
          const float* sc = exps + (E4M3 ? (kv + i) % ES * 12 : 0);
          auto factor = [&](int w) { return E4M3 ? fminf(fmaxf(cq * sc[w], 0x1p-126f), 0x1.fffffep127f) : P.c; };
          // Two passes over the scores, 32 at a time, the next ones on their way: the maximum, then the
          // weights, which take the place of scores already read.
          uint32_t x[2][16];
          float top = -INFINITY;
          tc_ld16(S, x[0]);
#pragma unroll kSteps
          for (int w = 0; w < 4; ++w) {
            float most = -INFINITY;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              tc_wait_ld();
              tc_ld16(S + (w < 3 || z == 0 ? 32 * w + 16 * z + 16 : 0), x[1 - z]);
              const uint32_t* y = x[z];
              float m0 = __uint_as_float(y[0]), m1 = __uint_as_float(y[1]);
#pragma unroll
              for (int j = 2; j < 16; j += 2) {
                m0 = fmaxf(m0, __uint_as_float(y[j]));
                m1 = fmaxf(m1, __uint_as_float(y[j + 1]));
              }
              most = fmaxf(most, fmaxf(m0, m1));
            }
            if constexpr (E4M3)
              top = fmaxf(top, fmaf(most, factor(w), sc[4 + w]));
            else
              top = fmaxf(top, most * P.c);
          }
          // f16 weights: 2^7 up, so that they stay below 2^15 after the growth allowed, and only those
          // below 2^-21 of the largest get subnormal
          if constexpr (std::is_same<OT, __half>::value) top -= 7.f;
          if (k == 0) {
            m = top;
          } else {
            const bool grow = top > m + Half<OT>::kGrow;
            if (__any_sync(kFull, grow)) {
              float a = 1.f;
              if (grow) {
                a = m == -INFINITY ? 0.f : ex2(m - top);
                m = top;
                l *= a;
              }
              tc_wait_ld();
#pragma unroll 1
              for (int w = 0; w < D; w += W) {
                uint32_t o[W];
                tc_ld_cols<W>(O + w, o);
                tc_wait_ld();
#pragma unroll
                for (int j = 0; j < W; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * a);
                tc_st_cols<W>(O + w, o);
              }
            }
          }
          const float mm = m == -INFINITY ? 0.f : -m;
#pragma unroll kSteps
          for (int w = 0; w < 4; ++w) {
            const float c = factor(w), up = E4M3 ? mm + sc[4 + w] : mm;
            const float2 c2 = make_float2(c, c), m2 = make_float2(up, up);
            float2 s0 = make_float2(0.f, 0.f), s1 = s0;
#pragma unroll
            for (int z = 0; z < 2; ++z) {
              tc_wait_ld();
              if (w < 3 || z == 0) tc_ld16(S + 32 * w + 16 * z + 16, x[1 - z]);
              const uint32_t* y = x[z];
              uint32_t p[8];
#pragma unroll
              for (int j = 0; j < 16; j += 4) {
                float2 a = fma2(make_float2(__uint_as_float(y[j]), __uint_as_float(y[j + 1])), c2, m2);
                float2 b = fma2(make_float2(__uint_as_float(y[j + 2]), __uint_as_float(y[j + 3])), c2, m2);
                a.x = ex2(a.x), a.y = ex2(a.y), b.x = ex2(b.x), b.y = ex2(b.y);
                s0 = add2(s0, a);
                s1 = add2(s1, b);
                p[j / 2] = Half<OT>::pack(a.x, a.y);  // rounded to the type the product takes
                p[j / 2 + 1] = Half<OT>::pack(b.x, b.y);
              }
              tc_st8(S + 16 * w + 8 * z, p);
            }
            const float sum = (s0.x + s0.y) + (s1.x + s1.y);
            l = E4M3 ? fmaf(sum, sc[8 + w], l) : l + sum;
          }
          tc_wait_st();
        }
        if (masked) {
          // V rows that no one may see become zeros (0 times a NaN is a NaN): those behind the chunk, and
          // those with a non-finite element, whose readers are marked instead
          // The streams may be several tiles apart (pair: by fewer than 8, since the ring's tiles are freed by
          // both), so marks take turns.
          const int mi = PAIR ? k & 7 : 4 * s + (k & 3);
          uint64_t* mb = mark + mi;
          if (!PAIR || s == 0) {
            ok = mbar_wait_warp(full + vslot, vpar, abort);
            if (!ok) break;
            const uint32_t at = sbase + C::kKv + vslot * C::kTileBytes + row * 128 + ((row & 7) << 4);  // (its piece 0; piece y: at ^ (y << 4))
            const bool hide = j0 + row >= stop;
            uint32_t bad = 0;  // the top bit of a half is set when its exponent is all ones
#pragma unroll
            for (int x = 0; x < C::kHalves; ++x)
#pragma unroll
              for (int y = 0; y < 8; ++y) {
                const uint4 v = lds128_at((at ^ (y << 4)) + x * C::kHalfBytes);  // (any order: no bank twice)
                constexpr uint32_t E = Half<OT>::kExp * 0x10001u, one = (0x8000u - Half<OT>::kExp) * 0x10001u;
                bad |= ((v.x & E) + one) | ((v.y & E) + one) | ((v.z & E) + one) | ((v.w & E) + one);
              }
            const bool nan = !hide && (bad & 0x80008000u);
            if (hide || nan) {
#pragma unroll
              for (int x = 0; x < C::kHalves; ++x)
#pragma unroll
                for (int y = 0; y < 8; ++y) sts128((at ^ (y << 4)) + x * C::kHalfBytes, 0, 0, 0, 0);
            }
            const uint32_t w = __ballot_sync(kFull, nan);
            if (lane == 0) poison[mi * 4 + (warp & 3)] = w;
            fence_proxy_async_shared();
            mbar_arrive_warp(mb);
          }
          ok = mbar_wait_warp(mb, (ph_mark >> mi) & 1, abort);
          ph_mark ^= 1u << mi;
          if (!ok) break;
          const uint32_t* bad = poison + mi * 4;
          if ((bad[0] & seen[0]) | (bad[1] & seen[1]) | (bad[2] & seen[2]) | (bad[3] & seen[3])) l = NAN;
        }
        // V is in place when the weights are said to be, so that issuing has one wait for both.  (Stream 1's
        // products follow stream 0's: in pair, stream 0 waits for both.)
        if ((warp & 3) == 0 && (!PAIR || s == 0)) {
          ok = mbar_wait_warp(full + vslot, vpar, abort);
          if (!ok) break;
        }
        tc_fence_before();
        mbar_arrive_warp(p_ready + s);
      }
      // the segment's parents (and, with the products', its queries) may be replaced
      mbar_arrive_warp(q_empty + qb);
      more = it.next(P, coming);  // (its lengths are read while the last products run)
      if (ok && cnt > 0) {
        ok = mbar_wait_warp(o_full + s, ph_o, abort);
        ph_o ^= 1;
        tc_fence_after();
      }
      kv += g.take;
      if (bad_tree) m = -INFINITY, l = 0.f;
      const bool whole = g.take == g.nt;
      const int slot = 2 * blockIdx.x + (g.off > 0 ? 0 : 1);
      const int urow = PAIR ? s * kTile + row : row;  // row of the unit
      float f0 = 1.f, f1 = 0.f;                       // factors of the streams' O (pair: of its own)
      int c0 = 0;
      bool two = false;
      if constexpr (!PAIR) {
        // Join the streams: the first warpgroup makes the factors of both, each takes half of the columns.  (Not
        // through tensor memory: the next item's scores are on their way to S.)
        float2* ml = reinterpret_cast<float2*>(smem + C::kMlAt) + row;
        if (s == 1) *ml = make_float2(m, l);
        tc_fence_before();
        mbar_arrive_warp(join);
        if (ok) ok = mbar_wait_warp(join, ph_join, abort);
        if (s == 0) {
          const float2 o = *ml;
          const float M = fmaxf(m, o.x);
          f0 = m == -INFINITY ? 0.f : ex2(m - M);
          f1 = o.x == -INFINITY ? 0.f : ex2(o.x - M);
          l = l * f0 + o.y * f1;  // (a NaN of either stays)
          m = M;
          const float norm = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
          f0 *= norm;
          f1 *= norm;
          *ml = make_float2(f0, f1);
          mbar_arrive_warp(join + 1);
        } else {
          if (ok) ok = mbar_wait_warp(join + 1, ph_join, abort);
          const float2 o = *ml;
          f0 = o.x;
          f1 = o.y;
        }
        tc_fence_after();
        two = cnt1 > 0;
        c0 = s * (D / 2);
      } else {
        f0 = whole ? (l == 0.f ? 0.f : 1.f / l) : 1.f;
      }
      const bool work = ok && warp_live && (!PAIR || cnt > 0);
      if (work) {
        const size_t orow = live ? ((size_t)g.b * P.T + t) * P.Hq + g.h * P.G + (r - t * P.G) : 0;
        uint4* dst = reinterpret_cast<uint4*>(P.out + (orow * D + c0) * 2);
        float4* part = reinterpret_cast<float4*>(P.part_o) + ((size_t)slot * (D / 4) + c0 / 4) * UR + urow;
#pragma unroll 1
        for (int x = 0; x < (PAIR ? D : D / 2); x += W, dst += W / 8, part += W / 4 * UR) {
          __syncwarp();
          uint32_t o[W];
          tc_ld_cols<W>(col_o(PAIR ? s : 0) + lanes + c0 + x, o);
          tc_wait_ld();
#pragma unroll
          for (int j = 0; j < W; ++j) o[j] = __float_as_uint(__uint_as_float(o[j]) * f0);
          if (!PAIR && two) {
            uint32_t o1[W];
            tc_ld_cols<W>(col_o(1) + lanes + c0 + x, o1);
            tc_wait_ld();
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = __float_as_uint(fmaf(__uint_as_float(o1[j]), f1, __uint_as_float(o[j])));
          }
          if (bad_tree) {
#pragma unroll
            for (int j = 0; j < W; ++j) o[j] = 0;
          }
          if (live && whole) {
#pragma unroll
            for (int j = 0; j < W / 8; ++j) {
              uint32_t w[4];
#pragma unroll
              for (int z = 0; z < 4; ++z)
                w[z] = Half<T>::pack(__uint_as_float(o[8 * j + 2 * z]), __uint_as_float(o[8 * j + 2 * z + 1]));
              dst[j] = make_uint4(w[0], w[1], w[2], w[3]);
            }
          } else if (live) {
#pragma unroll
            for (int j = 0; j < W / 4; ++j)
              part[j * UR] = make_float4(__uint_as_float(o[4 * j]), __uint_as_float(o[4 * j + 1]),
                                         __uint_as_float(o[4 * j + 2]), __uint_as_float(o[4 * j + 3]));
          }
        }
        if (live && (PAIR || s == 0)) {
          if (!whole)
            P.part_ml[(size_t)slot * UR + urow] = make_float2(m, l);
          else if (P.lse)
            P.lse[orow] = l == 0.f ? -INFINITY : (m + log2f(l)) * 0.69314718055994531f;
        }
      }
      if constexpr (!PAIR) {
        tc_fence_before();
        mbar_arrive_warp(join + 2);  // both accumulators have been read before either is written again
        if (ok) ok = mbar_wait_warp(join + 2, ph_join, abort);
        ph_join ^= 1;
      }
    }
  } else if (warp == 8) {
    // ====================================================================== products ====
    // (the warp stays together, so that addresses and descriptors are uniform; one lane issues)
    constexpr uint32_t fmt = Half<OT>::kFmt;
    constexpr uint32_t base = (1u << 4) | (fmt << 7) | (fmt << 10) | ((uint32_t)(kTile >> 4) << 24);
    constexpr uint32_t id_qk = base | ((uint32_t)(kTile >> 3) << 17);
    constexpr uint32_t id_pv = base | (1u << 16) | ((uint32_t)(D >> 3) << 17);  // V: its D axis contiguous
    const bool lead = elect_one();
    uint32_t ph_p = 0;  // bit s: p_ready of stream s
    uint32_t kv = 0;
    SegIter<UR> it(plan);
    Seg g;
    for (int seg = 0; ok && it.next(P, g); ++seg) {
      const int qb = seg % qbufs;
      const int cnt0 = stream_tiles(g, 0), cnt1 = stream_tiles(g, 1);
      ok = mbar_wait_warp(q_full + qb, (uint32_t)((seg / qbufs) & 1), abort);
      const int last_s = PAIR ? (cnt1 > 0 ? 1 : 0) : (g.take - 1) & 1, last_k = (last_s ? cnt1 : cnt0) - 1;
      // S of stream s from its k-th tile; the last reader of the K tile frees it, and the segment's last one the queries,
      // so that the next ones arrive while the last weights and sums are still at work
      auto mma_qk = [&](int s, int k, uint32_t slot) {
        const uint64_t q = tile_desc(sbase + C::kQ + (PAIR ? s : qb) * qbytes, 16);
        const uint64_t b = tile_desc(sbase + C::kKv + slot * C::kTileBytes, 16);
#pragma unroll
        for (int x = 0; x < D / 16; ++x)
          tc_mma_ss(col_s(s), q + (((x / 4) * qhalf + (x % 4) * 32) >> 4), b + (((x / 4) * C::kHalfBytes + (x % 4) * 32) >> 4),
                    id_qk, x > 0);
        tc_commit(s_full + s);
        if (!PAIR || s == 1 || cnt1 == 0) tc_commit(empty + slot);
        if (s == last_s && k == last_k) tc_commit(q_empty + qb);
      };
      auto qk = [&](int s, int k) {  // from the stream's k-th tile
        const uint32_t seq = 2 * kv + k_at(PAIR ? k : 2 * k + s), slot = seq % NS;
        ok = ok && mbar_wait_warp(full + slot, (seq / NS) & 1, abort);
        if (!ok) return;
        tc_fence_after();
        if (lead) mma_qk(s, k, slot);
        __syncwarp();
      };
      // O of stream s from its k-th tile, then S of its next, with nothing in between where that K is in place
      // (V is; see the softmax warps).  Issuing ends as the products run out, so what lies between two
      // steps leaves the tensor cores idle: one wait, and slots that are counted on, not divided for.
      auto step = [&](int s, int k, uint32_t vslot, uint32_t kslot, uint32_t kpar) {
        const bool more = k + 1 < (s ? cnt1 : cnt0);
        const uint64_t v = tile_desc(sbase + C::kKv + vslot * C::kTileBytes, C::kHalfBytes);
        ok = ok && mbar_wait_warp(p_ready + s, (ph_p >> s) & 1, abort);
        ph_p ^= 1u << s;
        if (!ok) return;
        tc_fence_after();
        const bool next = more && __all_sync(kFull, mbar_test_wait(full + kslot, kpar));
        if (lead) {
#pragma unroll
          for (int x = 0; x < kTile / 16; ++x) tc_mma_ts(col_o(s), col_s(s) + 8 * x, v + ((x * 2048) >> 4), id_pv, k > 0 || x > 0);
          if (next) mma_qk(s, k + 1, kslot);
          if (!PAIR || s == 1 || cnt1 == 0) tc_commit(empty + vslot);
          if (!more) tc_commit(o_full + s);
        }
        __syncwarp();
        if (more && !next) qk(s, k + 1);
      };
      qk(0, 0);
      if (cnt1 > 0) qk(1, 0);
      // the slots of V(i) and of the K taken after it (pair: K(i + 1), split: K(i + 2)), and that K's parity
      uint32_t vs = (2 * kv + 2) % NS, ks = (2 * kv + (PAIR ? 1 : 3)) % NS, kp = ((2 * kv + (PAIR ? 1 : 3)) / NS) & 1;
      auto last_v = [&](int i, uint32_t slot) { return i + 1 < g.take ? slot : slot == 0 ? NS - 1u : slot - 1u; };
      auto advance = [&] {
        vs += 2;
        vs -= vs >= NS ? NS : 0;
        ks += 2;
        if (ks >= NS) ks -= NS, kp ^= 1;
      };
      for (int k = 0; ok && k < cnt0; ++k) {
        step(0, k, last_v(PAIR ? k : 2 * k, vs), ks, kp);
        if (!PAIR) advance();
        if (k < cnt1) step(1, k, last_v(PAIR ? k : 2 * k + 1, vs), ks, kp);
        advance();
      }
      kv += g.take;
    }
    if (!ok) {  // products in flight end before tensor memory is given back
      *abort = 1;
      if (lead) {
        tc_commit(drain);
        const long long t0 = clock64();
        while (!mbar_try_wait(drain, 0) && clock64() - t0 < kWaitLimitCycles) {
        }
      }
      __syncwarp();
    }
  } else if (warp == 9 || warp == 11) {
    // ========================================================================= loads ====
    constexpr int N = E4M3 ? NR : NS;              // the ring that copies land in
    constexpr int kBoxes = E4M3 ? 1 : C::kHalves;  // column boxes of a row
    constexpr uint32_t kStage = E4M3 ? C::kRawBytes : C::kTileBytes;
    uint64_t* fb = E4M3 ? raw_full : full;
    uint64_t* eb = E4M3 ? raw_empty : empty;
    const uint32_t ring = sbase + (E4M3 ? C::kRawAt : C::kKv);
    const int box_log2 = P.page_log2 < 7 ? P.page_log2 : 7;  // rows of a box
    const int pieces = kTile >> box_log2;
    // this lane's box of a tile (at most 16 pieces of 2 boxes, every second one this warp's), and the warp's bytes
    const int which = warp == 9 ? 0 : 1, box = 2 * lane + which, piece = box / kBoxes, col = box % kBoxes;
    const bool mine = piece < pieces;
    const uint32_t bytes = (uint32_t)(pieces * kBoxes + 1 - which) / 2 * (kStage / (uint32_t)(pieces * kBoxes));
    uint32_t seq = 0;  // (2^31 tiles a CTA are out of reach)
    SegIter<UR> it(plan);
    Seg g;
    while (ok && it.next(P, g)) {
      const int32_t* table = P.table + (size_t)g.b * P.P;
      const int stop = g.L + g.n;
      auto page_of = [&](int i) {  // this lane's page in the segment's tile i; -1 reads zeros
        const int j = (g.nt - 1 - (g.off + i)) * kTile + (piece << box_log2);
        if (!mine || i >= g.take || j >= stop) return -1;
        const int p = __ldg(table + (j >> P.page_log2));
        return p >= 0 && p < P.num_pages ? p : -1;
      };
      auto load = [&](bool v, int i, int page) {
        const int j = (g.nt - 1 - (g.off + i)) * kTile + (piece << box_log2);
        const uint32_t slot = seq % N;
        if (seq >= N) ok = mbar_wait_warp(eb + slot, (seq / N - 1) & 1, abort);
        if (!ok) return;
        if (lane == 0) mbar_arrive_expect(fb + slot, bytes);
        __syncwarp();
        if (mine)
          tma_load_4d(ring + slot * kStage + col * C::kHalfBytes + ((uint32_t)piece << box_log2) * (E4M3 ? D : 128),
                      v ? &P.vmap : &P.kmap, col * 64, g.h, j & ((1 << P.page_log2) - 1), page, fb + slot);
        ++seq;
      };
      int was = -1, now = page_of(0), next = page_of(1);
      for (int i = 0; ok && i <= g.take; ++i) {  // K(i), V(i - 1)
        if (i < g.take) load(false, i, now);
        if (ok && i > 0) load(true, i - 1, was);
        was = now;
        now = next;
        next = page_of(i + 2);
      }
    }
    if (!ok) *abort = 1;
    // copies in flight land before the CTA ends, whoever gave up on them (else they have landed already)
    for (uint32_t x = seq > N ? seq - N : 0; x < seq; ++x) {
      const long long t0 = clock64();
      while (!mbar_try_wait(fb + x % N, (x / N) & 1) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else if (warp == 10) {
    // ======================================================================= queries ====
    const int ql = lane;
    int last = -1;               // the last segment whose queries were asked for
    int tree_of[2] = {-1, -1};   // the requests whose parents the buffers hold
    SegIter<UR> it(plan);
    Seg g;
    for (int seg = 0; ok && it.next(P, g); ++seg) {
      const int qb = seg % qbufs, use = seg / qbufs;
      if (use > 0) ok = mbar_wait_warp(q_empty + qb, (uint32_t)((use - 1) & 1), abort);
      if (!ok) break;
      const int r0 = g.qp * UR, rows = min(UR, g.n * P.G - r0);
      constexpr int V = D / 8;  // 16-byte vectors of a row
      constexpr bool kConvert = E4M3 && !std::is_same<T, __half>::value;  // bf16 to f16
      const uint32_t qat = sbase + C::kQ + (PAIR ? 0 : qb) * qbytes;
      uint32_t landing = 0;  // bytes on their way to q_full
      if (P.q_box > 0) {
        // whole tokens of G rows fit the tile: boxes of (64 elements, G heads, tokens)
        const int tiles = PAIR && rows > kTile ? 2 : 1;
        const uint32_t bytes = (uint32_t)(tiles * C::kHalves * 128 * P.G * P.q_box);
        if (ql == 0) {
          uint64_t* bar = kConvert ? q_raw : q_full + qb;
          mbar_arrive_expect(bar, bytes);
          const int t0 = (int)fdiv((unsigned)r0, P.fd_g);
          for (int x = 0; x < tiles; ++x)
            for (int y = 0; y < C::kHalves; ++y)
              tma_load_4d(qat + x * qbytes + y * qhalf, &P.qmap, y * 64, g.h * P.G, t0 + x * P.q_box, g.b, bar);
        }
        last = seg;
        if (kConvert) ok = mbar_wait_warp(q_raw, (uint32_t)(seg & 1), abort);
        landing = bytes;
      } else {
        const unsigned char* q = P.q + ((long long)g.b * P.T * P.q_stride + (long long)g.h * P.G * D + ql % V * 8) * 2;
        constexpr int R = 32 / V;  // rows a pass
        int r = ql / V;
        int t = (int)fdiv((unsigned)(r0 + r), P.fd_g), gg = r0 + r - t * P.G;
        while (r < rows) {
          uint4 x[4];
          int n = 0;
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (r + u * R < rows) {
              x[u] = __ldg(reinterpret_cast<const uint4*>(q + (t * P.q_stride + (long long)gg * D) * 2));
              for (gg += R; gg >= P.G; gg -= P.G) ++t;
              n = u + 1;
            }
#pragma unroll
          for (int u = 0; u < 4; ++u)
            if (u < n) {
              const int rr = r + u * R, c = ql % V;
              sts128(qat + (rr / kTile) * qbytes + (c / 8) * qhalf + (rr % kTile) * 128 + (((c % 8) ^ (rr & 7)) << 4), x[u].x,
                     x[u].y, x[u].z, x[u].w);
            }
          r += 4 * R;
        }
        __syncwarp();
      }
      if constexpr (kConvert) {
        if (!ok) break;
        // bf16 to f16 in place: a power of two brings the row's largest finite magnitude to 2^14 .. 2^15, so
        // that only elements below 2^-38 of it lose bits
        constexpr int N = V / 4;  // 16-byte vectors of one of a row's four lanes
        for (int r = ql / 4; r < (rows + 7) / 8 * 8; r += 8) {  // (all lanes stay: their maxima are exchanged)
          const uint32_t at = qat + (r / kTile) * qbytes + (r % kTile) * 128;
          uint4 v[N];
          uint32_t top = 0;
#pragma unroll
          for (int y = 0; y < N; ++y) {
            const int c = N * (ql & 3) + y;
            v[y] = lds128_at(at + (c / 8) * qhalf + (c % 8) * 16);
            const uint32_t w[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
#pragma unroll
            for (int z = 0; z < 4; ++z) {
              const uint32_t lo = (w[z] >> 7) & 0xffu, hi = (w[z] >> 23) & 0xffu;  // exponents
              top = max(top, max(lo == 255u ? 0u : lo, hi == 255u ? 0u : hi));
            }
          }
          top = max(top, __shfl_xor_sync(kFull, top, 1));
          top = max(top, __shfl_xor_sync(kFull, top, 2));
          const uint32_t e = max(top, 15u);  // the row in units of 2^(e - 141)
          const float f = __uint_as_float((268u - e) << 23);
          if (r >= rows) continue;
#pragma unroll
          for (int y = 0; y < N; ++y) {
            const int c = N * (ql & 3) + y;
            const uint32_t w[4] = {v[y].x, v[y].y, v[y].z, v[y].w};
            uint32_t o[4];
#pragma unroll
            for (int z = 0; z < 4; ++z)
              o[z] = Half<__half>::pack(__uint_as_float(w[z] << 16) * f, __uint_as_float(w[z] & 0xffff0000u) * f);
            sts128(at + (c / 8) * qhalf + (c % 8) * 16, o[0], o[1], o[2], o[3]);
          }
          // the factor back is 2^(e - 141); its float exponent e - 14 is at least 1
          if ((ql & 3) == 0) qexp[PAIR ? r : qb * kTile + r] = (uint8_t)(e - 14);
        }
        landing = 0;
      }
      if (P.parents && g.b != tree_of[qb]) {  // (the heads and row units of a request follow one another)
        tree_of[qb] = g.b;
        Parent* pr = par + (PAIR ? 0 : qb * kTile);
        bool bad = false;
        for (int i = lane; i < g.n; i += 32) {
          const int p = __ldg(P.parents + (size_t)g.b * P.T + i);
          const bool fine = i == 0 ? p == -1 : (p >= 0 && p < i);
          bad = bad || !fine;
          pr[i] = i > 0 && fine ? (Parent)p : kNoParent;
        }
        bad = __any_sync(kFull, bad);
        if (lane == 0) tree_bad[qb] = bad;
        __syncwarp();
      }
      fence_proxy_async_shared();
      if (landing == 0 || ql > 0) mbar_arrive(q_full + qb);  // (thread 0 arrived with its copies)
    }
    // these copies land, too
    constexpr bool raw = E4M3 && !std::is_same<T, __half>::value;
    for (int x = last; x >= 0 && x > last - (raw ? 1 : qbufs); --x) {
      uint64_t* bar = raw ? q_raw : q_full + x % qbufs;
      const long long t0 = clock64();
      while (!mbar_try_wait(bar, (uint32_t)((raw ? x : x / qbufs) & 1)) && clock64() - t0 < kWaitLimitCycles) {
      }
    }
  } else {
    // ================================================================= codes to 16 bits ====
    if constexpr (E4M3) {
      // Four warps take the K tiles, four the V tiles, 32 positions each.  Where no row behind the 64th lives, the live
      // softmax warps are all in the first two quarters of the SM: then the two K warps of the other quarters take
      // positions n and n + 64 each (64 chains of 6 tokens by 8 heads over 8192 positions: 252 -> 229 us; with 64
      // columns, whose conversion is half as long, 206 -> 229, so not there).
      const int cw = warp - C::kConvert, v = cw >= 4;
      const bool half = D == 128 && !PAIR && !v && P.T * P.G <= kTile / 2;
      const int unit = half ? (cw & 3) - 2 : cw & 3, row = unit * 32 + lane;
      const int page_mask = (1 << P.page_log2) - 1;
      const unsigned page_rows = (unsigned)P.H << P.page_log2;  // scales of a page
      uint32_t kv = 0;
      SegIter<UR> it(plan);
      Seg g;
      while (unit >= 0 && ok && it.next(P, g)) {
        const int stop = g.L + g.n;
        const int32_t* table = P.table + (size_t)g.b * P.P;
        // the page of a row (-1: none), and its scales
        auto page_of = [&](int j) { return j >= 0 && j < stop ? __ldg(table + (j >> P.page_log2)) : -1; };
        auto scales_of = [&](int j, int p) {
          if (p < 0 || p >= P.num_pages) return make_float2(0.f, 0.f);
          const unsigned long long at = (unsigned long long)(unsigned)p * page_rows + (unsigned)((j & page_mask) * P.H + g.h);
          return make_float2(v ? 0.f : __ldg(P.ks + at), __ldg(P.vs + at));
        };
        // A scale goes with its codes in units of 2^e, e the exponent of the largest finite scale of its
        // 32 rows (V: within the range that the weights' reference exponent covers).
        auto exponent = [](float x) {
          const uint32_t mag = __float_as_uint(fabsf(x));
          return (int)(__reduce_max_sync(kFull, mag < 0x7f800000u ? mag : 0u) >> 23) - 127;
        };
        // pages are fetched two tiles ahead, scales one (behind the segment: unused)
        int j = (g.nt - 1 - g.off) * kTile + row;
        float2 now[2] = {scales_of(j, page_of(j)), make_float2(0.f, 0.f)};
        int page[2] = {page_of(j - kTile), -1};
        if (half) {
          now[1] = scales_of(j + 64, page_of(j + 64));
          page[1] = page_of(j + 64 - kTile);
        }
#pragma unroll 1
        for (int i = 0; ok && i < g.take; ++i, j -= kTile) {
          float2 next[2] = {scales_of(j - kTile, page[0]), make_float2(0.f, 0.f)};
          page[0] = page_of(j - 2 * kTile);
          if (half) {
            next[1] = scales_of(j + 64 - kTile, page[1]);
            page[1] = page_of(j + 64 - 2 * kTile);
          }
          const uint32_t seq = 2 * kv + (v ? v_at(g, i) : k_at(i)), rs = seq % NR, slot = seq % NS;
          ok = mbar_wait_warp(raw_full + rs, (seq / NR) & 1, abort);
          // (Place seq - NS may be the other warpgroup's.  It has its slot: the raw ring is no longer than this
          // one, and a raw tile is given back only once its slot is had.  So at most one phase is to come.)
          if (ok && seq >= NS) ok = mbar_wait_warp(empty + slot, (seq / NS - 1) & 1, abort);
          if (!ok) break;
          // Places of the row's 16-byte piece 0; piece y is at ^ (y << 4): pieces of a 128-byte row are exchanged by its
          // row of 8, those of a 64-byte row by its pair of rows of 4 (the copy's and the products' swizzles)
          uint32_t src = sbase + C::kRawAt + rs * C::kRawBytes + row * D + (D == 128 ? (row & 7) << 4 : ((row >> 1) & 3) << 4);
          uint32_t dst = sbase + C::kKv + slot * C::kTileBytes + row * 128 + ((row & 7) << 4);
#pragma unroll 1
          for (int n = 0; n < (half ? 2 : 1); ++n, src += 64 * D, dst += 64 * 128) {
            uint4 code[D / 16];
#pragma unroll
            for (int y = 0; y < D / 16; ++y) code[y] = lds128_at(src ^ (y << 4));
            const int ve = max(-60, min(100, exponent(now[0].y)));
            const int e = v ? ve : max(-126, min(126, exponent(now[0].x)));
            if (!v && lane == 0) {
              float* at = exps + (kv + i) % ES * 12 + unit + 2 * n;
              at[0] = __uint_as_float((uint32_t)(e + 127) << 23);
              at[4] = (float)ve;
              at[8] = __uint_as_float((uint32_t)(127 - ve) << 23);
            }
            const __half2 rel = __float2half2_rn((v ? now[0].y : now[0].x) * __uint_as_float((uint32_t)(127 - e) << 23));
            mbar_arrive_warp(raw_empty + rs);  // (its codes are in registers)
#pragma unroll
            for (int y = 0; y < D / 16; ++y) {
              const uint32_t w[4] = {code[y].x, code[y].y, code[y].z, code[y].w};
              uint32_t o[8];
#pragma unroll
              for (int z = 0; z < 8; ++z) {
                uint32_t c;
                asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(c) : "h"((uint16_t)(w[z >> 1] >> (16 * (z & 1)))));
                const __half2 f = __hmul2(*reinterpret_cast<const __half2*>(&c), rel);
                o[z] = *reinterpret_cast<const uint32_t*>(&f);
              }
              const uint32_t at = (dst ^ ((y & 3) << 5)) + (y >> 2) * C::kHalfBytes;
              sts128(at, o[0], o[1], o[2], o[3]);
              sts128(at ^ 16, o[4], o[5], o[6], o[7]);
            }
            fence_proxy_async_shared();
            mbar_arrive_warp(full + slot);
            now[0] = now[1];
          }
          now[0] = next[0], now[1] = next[1];
        }
        kv += g.take;
      }
    }
  }
  if (!ok) *abort = 1;
  tc_fence_before();
  __syncthreads();
  if (warp == 8) {
    tc_fence_after();
    tc_free(tmem);
  }
  if (*abort && P.err_flags)
    for (int b = tid; b < P.B; b += C::kThreads) atomicOr(P.err_flags + b, SPEC_ERRF_TIMEOUT);
  if (*abort && tid == 0) P.rec[blockIdx.x].last |= kGaveUp;
}

// Joins the parts of the items that several CTAs share.  Block (c, y): the item that starts in CTA c, 8 of its
// rows (16 where a row has 64 columns); a thread takes four columns of a row.  The first two parts' factors and values
// are loaded side by side: the call's tail is 3 us of a decode's 20 and 8 of 155 for 61-node trees (40 MB of parts); with
// the factors first, and then part by part, 6 and 14.
template <typename T, int D>
__global__ void __launch_bounds__(256) attention_combine_kernel(const __grid_constant__ Params P, int UR) {
  constexpr int R = 1024 / D;  // rows of a block
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const int c = blockIdx.x;
  const Record rec = P.rec[c];
  auto pass_on = [&] {
    if (!(rec.last & kGaveUp) || blockIdx.y != 0 || !P.err_flags) return;
    for (int b = threadIdx.x; b < P.B; b += 256) atomicOr(P.err_flags + b, SPEC_ERRF_TIMEOUT);
  };
  if (rec.b < 0) return pass_on();
  const int n = P.chunk_len ? __ldg(P.chunk_len + rec.b) : P.T;
  const int rows = min((long long)UR, (long long)n * P.G - (long long)rec.qp * UR);
  const int row = blockIdx.y * R + threadIdx.x % R, q4 = threadIdx.x / R;
  if (row >= rows) return pass_on();
  const float2* ml = P.part_ml + row;
  const float4* po = reinterpret_cast<const float4*>(P.part_o) + (size_t)q4 * UR + row;
  auto slot = [&](int x) { return (size_t)(2 * x + (x == c)); };
  // the first two parts (most items have no more), then one at a time
  const int second = c + P.lanes;
  const float2 v0 = ml[slot(c) * UR], v1 = ml[slot(second) * UR];
  const float4 p0 = po[slot(c) * (D / 4) * UR], p1 = po[slot(second) * (D / 4) * UR];
  float M = fmaxf(v0.x, v1.x), l;
  auto factor = [](float m, float M) { return m == -INFINITY ? 0.f : ex2(m - M); };
  float w0 = factor(v0.x, M), w1 = factor(v1.x, M);
  l = v0.y * w0 + v1.y * w1;
  if (v0.y != v0.y || v1.y != v1.y) l = NAN;
  float4 o = make_float4(fmaf(p1.x, w1, p0.x * w0), fmaf(p1.y, w1, p0.y * w0), fmaf(p1.z, w1, p0.z * w0), fmaf(p1.w, w1, p0.w * w0));
  const int last = rec.last & ~kGaveUp;
  for (int x = second + P.lanes; x <= last; x += P.lanes) {
    const float2 v = ml[slot(x) * UR];
    const float4 p = po[slot(x) * (D / 4) * UR];
    const float N = fmaxf(M, v.x), a = factor(M, N), w = factor(v.x, N);
    l = v.y == v.y ? fmaf(v.y, w, l * a) : NAN;
    o = make_float4(fmaf(p.x, w, o.x * a), fmaf(p.y, w, o.y * a), fmaf(p.z, w, o.z * a), fmaf(p.w, w, o.w * a));
    M = N;
  }
  const int r = rec.qp * UR + row, t = r / P.G;
  const size_t orow = ((size_t)rec.b * P.T + t) * P.Hq + rec.h * P.G + (r - t * P.G);
  const float inv = l == 0.f ? 0.f : 1.f / l;
  uint2 w2;
  w2.x = Half<T>::pack(o.x * inv, o.y * inv);
  w2.y = Half<T>::pack(o.z * inv, o.w * inv);
  *reinterpret_cast<uint2*>(P.out + (orow * D + 4 * q4) * 2) = w2;
  if (q4 == 0 && P.lse) P.lse[orow] = l == 0.f ? -INFINITY : (M + log2f(l)) * 0.69314718055994531f;
  pass_on();
}

// Launches both kernels on `stream`.
template <typename T, int D, bool E4M3, bool PAIR>
cudaError_t launch_one(const Params& P, int ctas, cudaStream_t stream) {
  using C = Cfg<D, E4M3, PAIR>;
  auto* k = attention_kernel<T, D, E4M3, PAIR>;
  cudaError_t e = cudaFuncSetAttribute(k, cudaFuncAttributeMaxDynamicSharedMemorySize, C::kBytes);
  if (e != cudaSuccess) return e;
  k<<<ctas, C::kThreads, C::kBytes, stream>>>(P);
  if ((e = cudaGetLastError()) != cudaSuccess) return e;
  constexpr int UR = PAIR ? 2 * kTile : kTile;
  const long long rows = (long long)P.T * P.G < UR ? (long long)P.T * P.G : UR;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3((unsigned)ctas, (unsigned)((rows + 1024 / D - 1) / (1024 / D)));
  cfg.blockDim = dim3(256);
  cfg.stream = stream;
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, attention_combine_kernel<T, D>, P, UR);
}

template <typename T>
cudaError_t launch_attention(const Params& P, int D, bool e4m3, bool pair, int ctas, cudaStream_t stream) {
  if (D == 64) {
    if (e4m3) return pair ? launch_one<T, 64, true, true>(P, ctas, stream) : launch_one<T, 64, true, false>(P, ctas, stream);
    return pair ? launch_one<T, 64, false, true>(P, ctas, stream) : launch_one<T, 64, false, false>(P, ctas, stream);
  }
  if (e4m3) return pair ? launch_one<T, 128, true, true>(P, ctas, stream) : launch_one<T, 128, true, false>(P, ctas, stream);
  return pair ? launch_one<T, 128, false, true>(P, ctas, stream) : launch_one<T, 128, false, false>(P, ctas, stream);
}

}  // namespace attn
}  // namespace specv
