"""Host check of csrc/fixed_weight.h at both ends of the floats: a masked logit (-inf) weighs nothing whatever the row's
maximum is, the lowest finite float too, alone and beside another; finite ones keep fixed_weight.h's bound."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_82_gb300", "csrc")

DRIVER = r"""
#include <cfloat>
#include <cmath>
#include <cstdio>
#include <initializer_list>
#include "fixed_weight.h"
using namespace specv;
static const Pair base[32] = SPECV_WEIGHT_TABLE;
int main() {
  int bad = 0;
  const float lowest = -FLT_MAX, next = std::nextafterf(lowest, 0.f), bf16_lowest = -0x1.fep127f;
  for (float t : {0x1p-64f, 0x1p-20f, 0.5f, 1.f, 8.f, 0x1p20f, 0x1p64f})
    for (float top : {lowest, next, bf16_lowest, -65504.f, -0x1p100f, 0.f, 65504.f, 0x1p100f, FLT_MAX}) {
      float hi, lo;
      weight_factor(t, hi, lo);
      const WeightRow row = weight_row(top, hi, lo);
      Pair table[32];
      for (int j = 0; j < 32; ++j) table[j] = weight_entry(base[j], row);
      const float xs[] = {-INFINITY, lowest, next, bf16_lowest, -65504.f, std::nextafterf(top, -INFINITY), top};
      for (float x : xs)
        for (float y : xs) {
          if (!(x <= top && y <= top)) continue;
          Pair at, z, tail, h, l, up, low;
          weight_power(Pair{x, y}, row, at, z, tail);
          const Pair p = table[weight_index(at.x)], q = table[weight_index(at.y)], size{weight_size(at.x), weight_size(at.y)};
          weight_product(mul(Pair{p.x, q.x}, size), mul(Pair{p.y, q.y}, size), z, tail, h, l);
          weight_cut(h, l, up, low);
          const float us[2] = {up.x, up.y}, ls[2] = {low.x, low.y}, in[2] = {x, y};
          for (int e = 0; e < 2; ++e) {
            const uint64_t one = fixed_weight(in[e], row, table);
            const uint64_t two = (uint64_t)(((int64_t)(float_bits(us[e]) - float_bits(kUpper)) << kWeightHalf) + (float_bits(ls[e]) - float_bits(kLower)));
            const double w = std::exp2(-((double)top - (double)in[e]) / (double)t * 1.4426950408889634);
            const bool fine = in[e] == -INFINITY ? one == 0 : std::fabs(std::ldexp((double)one, -kWeightBits) - w) <= std::ldexp(w, -33) + std::ldexp(1.0, -44);
            if (!fine || one != two)
              if (bad++ < 5) std::printf("x %a top %a T %a: %llu alone, %llu beside another\n", in[e], top, t, (unsigned long long)one, (unsigned long long)two);
          }
        }
    }
  std::printf("%d bad\n", bad);
  return bad != 0;
}
"""


def test_lowest_floats(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    src, exe = tmp_path / "t.cpp", tmp_path / "t"
    src.write_text(DRIVER)
    subprocess.run([cxx, "-O2", "-std=c++17", "-ffp-contract=off", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True)
    assert r.returncode == 0, r.stdout
