"""Host check of csrc/device_info.h: the count of the current device, errors passed on, and no data race between
threads that ask for the first time at once (the thread sanitizer's verdict).

The header is plain C++ over two calls of the CUDA runtime, which the driver program stands in for."""

import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CSRC = os.path.join(ROOT, "speculative_decoding_verification_82_gb300", "csrc")

RUNTIME = r"""
#pragma once
enum cudaError_t { cudaSuccess = 0, cudaErrorUnknown = 1 };
enum cudaDeviceAttr { cudaDevAttrMultiProcessorCount = 16 };
cudaError_t cudaGetDevice(int*);
cudaError_t cudaDeviceGetAttribute(int*, cudaDeviceAttr, int);
"""

DRIVER = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "device_info.h"
static thread_local int current = 0;
static std::atomic<int> lookups{0};
cudaError_t cudaGetDevice(int* d) { *d = current; return current == -2 ? cudaErrorUnknown : cudaSuccess; }
cudaError_t cudaDeviceGetAttribute(int* v, cudaDeviceAttr a, int d) {
  lookups.fetch_add(1, std::memory_order_relaxed);  // (orders nothing between the threads)
  if (d == 7) return cudaErrorUnknown;
  *v = a == cudaDevAttrMultiProcessorCount ? 100 + d : 0;
  return cudaSuccess;
}
int main() {
  int wrong[8] = {}, bad = 0;
  std::atomic<int> ready{0};
  std::vector<std::thread> t;
  for (int i = 0; i < 8; ++i)
    t.emplace_back([&, i] {
      ++ready;
      while (ready < 8) std::this_thread::yield();  // all start at once
      for (int k = 0; k < 2000; ++k) {
        current = (k + i) % 6 + (k % 5 == 0 ? 64 : 0);  // devices beyond the kept ones, too
        int dev = -1;
        wrong[i] += specv::sm_count(&dev) != 100 + current || dev != current;
      }
    });
  for (auto& x : t) x.join();
  for (int w : wrong) bad += w;
  current = 7;
  bad += specv::sm_count() != -1;
  current = -2;
  bad += specv::sm_count() != -1;
  current = 3;
  const int before = lookups;
  bad += specv::sm_count() != 103 || lookups != before;
  std::printf("bad %d\n", bad);
  return bad != 0;
}
"""


def compile_and_run(cxx, folder, flags):
    exe = os.path.join(folder, "t")
    r = subprocess.run([cxx, "-O1", "-std=c++17", "-pthread", *flags, "-I", folder, "-I", CSRC, os.path.join(folder, "t.cpp"), "-o", exe],
                       capture_output=True, text=True)
    assert r.returncode == 0, r.stderr
    return subprocess.run([exe], capture_output=True, text=True)


@pytest.mark.parametrize("flags", [[], ["-fsanitize=thread"]], ids=["plain", "thread sanitizer"])
def test_device_count_from_many_threads(tmp_path, flags):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    if flags:  # does it run here at all?
        (tmp_path / "t.cpp").write_text("int main() { return 0; }\n")
        try:
            if compile_and_run(cxx, str(tmp_path), flags).returncode != 0:
                pytest.skip("the thread sanitizer does not run here")
        except AssertionError:
            pytest.skip("no thread sanitizer")
    (tmp_path / "cuda_runtime_api.h").write_text(RUNTIME)
    (tmp_path / "t.cpp").write_text(DRIVER)
    r = compile_and_run(cxx, str(tmp_path), flags)
    assert r.returncode == 0, r.stdout + r.stderr
    assert "bad 0" in r.stdout


def test_every_caller_shares_it():
    """No other translation unit keeps a count of its own."""
    for name in os.listdir(CSRC):
        with open(os.path.join(CSRC, name)) as f:
            assert name == "device_info.h" or "cudaDevAttrMultiProcessorCount" not in f.read(), name
