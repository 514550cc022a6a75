// fixed_weight.h -- exp((x - M) / T) as a whole number of 2^-44, for sums whose borders decide which token is
// kept or drawn: whole numbers add up exactly, in any order.
//
// With c = log2(e) / T in two floats, x c = P + r: P the nearest whole number of 1/32 (the rounding of a sum with a large
// constant gives it) and r, |r| <= 1/64, in two floats.  Then the weight is 2^(P - M c) 2^r: the first factor is a power of
// two times one of 32 values that hold 2^(-j / 32) and what M c lacks to a whole number of 1/32, two floats each, set
// up once a row; the second is 1 + z + z^2/2 + z^3/6 + z^4/24, z = r ln 2, |z| < 0.011 (what is left out is below
// 2^-39).  The product, two floats, is cut by rounded sums again: whole numbers of 2^-22 and what remains, whole numbers of
// 2^-44; the sums' bit patterns, less the constants', are those numbers, and threads add them up in 32 bits.  Rows whose
// maximum is too large for the constant's 128 are moved to a maximum of 0 first, the rounding errors kept.  -inf weighs
// nothing, next to the lowest float as the maximum, too.
//
// A weight is off by 2^-37 of itself on average (root mean square), and never by more than 2^-33 of it and
// 2^-44 (tests/test_fixed_weight.py, tests/test_fixed_weight_lowest.py).  Two elements at a time share most instructions, and a pass that sums weights
// executes about 30 an element, reading and unpacking included (64-bit products and shifts of whole numbers instead: 89).
#pragma once

#include <math.h>
#include <stdint.h>

#include "fastdiv.h"

namespace specv {

constexpr int kWeightBits = 44, kWeightHalf = 22;
constexpr float kWeightEnd = 46.5f;      // such a weight, 2^-46.5, is nothing
constexpr float kGrid = 393216.f;        // 1.5 2^18: floats next to it are whole numbers of 1/32
constexpr float kUpper = 3.f;            // 1.5 2^1: of 2^-22
constexpr float kLower = 0x1.8p-21f;     // of 2^-44

// 2^(-j / 32) in two floats.
#define SPECV_WEIGHT_TABLE                                                    \
  {                                                                           \
      {0x1p+0f, 0x0p+0f}, {0x1.f50766p-1f, -0x1.246ebp-27f},                  \
      {0x1.ea4afap-1f, 0x1.52486cp-28f}, {0x1.dfc974p-1f, -0x1.908c94p-26f},  \
      {0x1.d5818ep-1f, -0x1.822dbcp-28f}, {0x1.cb720ep-1f, -0x1.8837ccp-28f}, \
      {0x1.c199bep-1f, -0x1.3d56b2p-28f}, {0x1.b7f77p-1f, -0x1.a09438p-26f},  \
      {0x1.ae89fap-1f, -0x1.a94b14p-27f}, {0x1.a5503cp-1f, -0x1.b83b54p-26f}, \
      {0x1.9c4918p-1f, 0x1.51f848p-28f}, {0x1.93737cp-1f, -0x1.e64744p-26f},  \
      {0x1.8ace54p-1f, 0x1.15506ep-28f}, {0x1.82589ap-1f, -0x1.accc7cp-27f},  \
      {0x1.7a1148p-1f, -0x1.829fdp-26f}, {0x1.71f75ep-1f, 0x1.1d8beep-26f},   \
      {0x1.6a09e6p-1f, 0x1.9fcef4p-27f}, {0x1.6247ecp-1f, -0x1.f8b55p-26f},   \
      {0x1.5ab07ep-1f, -0x1.5bd5ecp-28f}, {0x1.5342b6p-1f, -0x1.2c561p-26f},  \
      {0x1.4bfdaep-1f, -0x1.593abcp-26f}, {0x1.44e086p-1f, 0x1.8624b4p-31f},  \
      {0x1.3dea64p-1f, 0x1.824684p-26f}, {0x1.371a74p-1f, -0x1.18aac6p-26f},  \
      {0x1.306fep-1f, 0x1.4636e2p-26f}, {0x1.29e9ep-1f, -0x1.5c0424p-26f},    \
      {0x1.2387a6p-1f, 0x1.ceac48p-26f}, {0x1.1d4874p-1f, -0x1.d2e8cap-26f},  \
      {0x1.172b84p-1f, -0x1.c15742p-28f}, {0x1.11301ep-1f, -0x1.fdb496p-26f}, \
      {0x1.0b5586p-1f, 0x1.9f3122p-26f}, {0x1.059b0ep-1f, -0x1.9d4f52p-26f}   \
  }

SPECV_HD int32_t float_bits(float x) {
#if defined(__CUDA_ARCH__)
  return __float_as_int(x);
#else
  union {
    float f;
    int32_t i;
  } u;
  u.f = x;
  return u.i;
#endif
}
SPECV_HD float bits_float(int32_t x) {
#if defined(__CUDA_ARCH__)
  return __int_as_float(x);
#else
  union {
    int32_t i;
    float f;
  } u;
  u.i = x;
  return u.f;
#endif
}

// One float, or two that share their instructions.
struct Pair {
  float x, y;
};
SPECV_HD float mul(float a, float b) {
#if defined(__CUDA_ARCH__)
  return __fmul_rn(a, b);
#else
  return a * b;
#endif
}
SPECV_HD float add(float a, float b) {
#if defined(__CUDA_ARCH__)
  return __fadd_rn(a, b);
#else
  return a + b;
#endif
}
SPECV_HD float mad(float a, float b, float c) { return fmaf(a, b, c); }
SPECV_HD float at_least(float a, float b) { return fmaxf(a, b); }
SPECV_HD Pair at_least(Pair a, float b) { return Pair{fmaxf(a.x, b), fmaxf(a.y, b)}; }
SPECV_HD void all_of(float& d, float v) { d = v; }
SPECV_HD void all_of(Pair& d, float v) { d.x = d.y = v; }
#if defined(__CUDA_ARCH__)
__device__ __forceinline__ Pair mul(Pair a, Pair b) {
  Pair r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "mul.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Pair add(Pair a, Pair b) {
  Pair r;
  asm("{\n\t.reg .b64 a, b;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\t"
      "add.rn.f32x2 a, a, b;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y));
  return r;
}
__device__ __forceinline__ Pair mad(Pair a, Pair b, Pair c) {
  Pair r;
  asm("{\n\t.reg .b64 a, b, c;\n\tmov.b64 a, {%2, %3};\n\tmov.b64 b, {%4, %5};\n\tmov.b64 c, {%6, %7};\n\t"
      "fma.rn.f32x2 a, a, b, c;\n\tmov.b64 {%0, %1}, a;\n\t}"
      : "=f"(r.x), "=f"(r.y)
      : "f"(a.x), "f"(a.y), "f"(b.x), "f"(b.y), "f"(c.x), "f"(c.y));
  return r;
}
#else
SPECV_HD Pair mul(Pair a, Pair b) { return Pair{a.x * b.x, a.y * b.y}; }
SPECV_HD Pair add(Pair a, Pair b) { return Pair{a.x + b.x, a.y + b.y}; }
SPECV_HD Pair mad(Pair a, Pair b, Pair c) { return Pair{fmaf(a.x, b.x, c.x), fmaf(a.y, b.y, c.y)}; }
#endif
template <typename V>
SPECV_HD V of(float v) {
  V d;
  all_of(d, v);
  return d;
}
// a - b; two elements' instructions have no minus signs of their own.
template <typename V>
SPECV_HD V sub(V a, V b) {
  return mad(b, of<V>(-1.f), a);
}

struct WeightRow {  // a row's constants
  float top;        // M
  float hi, lo;     // c
  float grid;       // kGrid and the maximum's P
  float least;      // logits below it weigh as little as it
  float reach;      // how far down weights reach
  bool far;         // logits are taken less M
};

// c of a temperature in [2^-64, 2^64]: the quotient, and the quotient of what remains.
SPECV_HD void weight_factor(float temperature, float& hi, float& lo) {
  constexpr float kLog2e = 0x1.715476p+0f, kLog2eLow = 0x1.4ae0cp-26f;
#if defined(__CUDA_ARCH__)
  hi = __fdiv_rn(kLog2e, temperature);
  lo = __fdiv_rn(fmaf(-hi, temperature, kLog2e) + kLog2eLow, temperature);
#else
  hi = kLog2e / temperature;
  lo = (fmaf(-hi, temperature, kLog2e) + kLog2eLow) / temperature;
#endif
}
SPECV_HD WeightRow weight_row(float top, float hi, float lo) {
  WeightRow r;
  r.top = top;
  r.hi = hi;
  r.lo = lo;
  const float p = mul(top, hi);
  r.far = !(fabsf(p) <= 128.f);
  r.grid = r.far ? kGrid : add(kGrid, sub(add(p, kGrid), kGrid));
#if defined(__CUDA_ARCH__)
  r.reach = __fdiv_rd(kWeightEnd, hi);
  r.least = __fsub_rd(top, r.reach);
#else
  r.reach = kWeightEnd / hi;
  r.least = nextafterf(top - r.reach, -INFINITY);  // (or the float below: it makes no difference)
#endif
  r.least = fmaxf(r.least, -3.402823466e38f);
  return r;
}

constexpr float kLn2 = 0x1.62e430p-1f, kLn2Low = -0x1.05c610p-29f;

// 2^(r + rl) - 1 as z + tail.
template <typename V>
SPECV_HD void weight_series(V r, V rl, V& z, V& tail) {
  z = mul(r, of<V>(kLn2));
  const V rest = mad(r, of<V>(kLn2), mul(r, of<V>(-kLn2)));  // what z's rounding left
  const V zl = mad(rl, of<V>(kLn2), mad(r, of<V>(kLn2Low), rest)), y = add(z, zl);
  tail = mad(mul(y, y), mad(mad(y, of<V>(1.f / 24.f), of<V>(1.f / 6.f)), y, of<V>(0.5f)), zl);
}
// First half of a weight: the sum whose bits hold P, and 2^r - 1 as z + tail.
template <typename V>
SPECV_HD void weight_power(V x, const WeightRow& R, V& at, V& z, V& tail) {
  V low = of<V>(0.f);
  const V given = x;
  x = at_least(x, R.least);
  if (R.far) {  // x - M and its rounding error
    const V m = of<V>(R.top), d = sub(x, m), back = sub(d, x);
    low = sub(sub(x, sub(d, back)), add(m, back));
    // (`least` may be a long way off, next to a large M, or be M itself, the lowest float: what it raised is lowered again)
    x = at_least(add(d, sub(given, x)), -R.reach);
  }
  const V np = mul(x, of<V>(-R.hi));  // -x c, as far as it goes
  at = add(np, of<V>(R.grid));
  const V r = sub(add(at, of<V>(-R.grid)), np);
  V rl = mad(x, of<V>(R.lo), mad(x, of<V>(R.hi), np));
  if (R.far) rl = mad(low, of<V>(R.hi), rl);
  weight_series(r, rl, z, tail);
}
// (th + tl) (1 + z + tail) as the sum of hi and lo.
template <typename V>
SPECV_HD void weight_product(V th, V tl, V z, V tail, V& hi, V& lo) {
  hi = mad(th, z, th);
  lo = mad(tl, z, mad(th, tail, mad(th, z, sub(th, hi))));
  lo = add(lo, tl);
}
// Whole numbers of 2^-22 and of 2^-44 as the bits of two floats, above those of kUpper and kLower.
template <typename V>
SPECV_HD void weight_cut(V hi, V lo, V& upper, V& lower) {
  upper = add(add(hi, lo), of<V>(kUpper));
  lower = add(add(sub(hi, add(upper, of<V>(-kUpper))), lo), of<V>(kLower));
}
// The table's entry j for a row: {2^(-j / 32) in two floats} less what the maximum's P lacks.
SPECV_HD Pair weight_entry(Pair t, const WeightRow& R) {
  if (R.far) return t;
  float z, tail, hi, lo;
  const float p = mul(R.top, R.hi);
  const float r = sub(p, sub(add(p, kGrid), kGrid)), rl = mad(R.top, R.lo, mad(R.top, R.hi, -p));
  weight_series(-r, -rl, z, tail);
  weight_product(t.x, t.y, z, tail, hi, lo);
  const float sum = add(hi, lo);
  return Pair{sum, sub(lo, sub(sum, hi))};
}
// The table's entry for a sum `at`: its places below the maximum's P in 1/32 are its low bits (kGrid's are 0), j the last five.
SPECV_HD int weight_index(float at) { return float_bits(at) & 31; }
// 2^-(the whole powers of two below): `at` is at most kGrid + 47.
SPECV_HD float weight_size(float at) { return bits_float((int32_t)(0x3f800000u - (((uint32_t)float_bits(at) & ~31u) << 18))); }

// One weight; x is at most R.top.  `both`: in two floats.
SPECV_HD uint64_t fixed_weight(float x, const WeightRow& R, const Pair* table, Pair* both = nullptr) {
  float at, z, tail, hi, lo, upper, lower;
  weight_power(x, R, at, z, tail);
  const Pair t = table[weight_index(at)];
  const float s = weight_size(at);
  weight_product(mul(t.x, s), mul(t.y, s), z, tail, hi, lo);
  if (both) both->x = add(hi, lo), both->y = sub(lo, sub(both->x, hi));
  weight_cut(hi, lo, upper, lower);
  return (uint64_t)(((int64_t)(float_bits(upper) - float_bits(kUpper)) << kWeightHalf) + (float_bits(lower) - float_bits(kLower)));
}

}  // namespace specv
