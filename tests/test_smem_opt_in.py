"""The opt-in to dynamic shared memory when two host threads ask for one kernel
with different sizes at once, on the CPU: the library's header compiled with a
stand-in for the CUDA calls that lets the smaller request overtake the larger
one's record."""
import os
import shutil
import subprocess

import pytest

from paged_kv_cache_67_gb300 import build as libbuild

SOURCE = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "pkv_internal.h"

static std::atomic<int> limit{0}, small_recorded{0}, large_inside{0};
static int configured[64] = {0};

static void wait_for(std::atomic<int> &flag) {   // half a second at most
  for (int i = 0; i < 500 && !flag; ++i) std::this_thread::sleep_for(std::chrono::milliseconds(1));
}

extern "C" cudaError_t cudaGetDevice(int *dev) { *dev = 0; return cudaSuccess; }
extern "C" cudaError_t cudaFuncSetAttribute(const void *, cudaFuncAttribute, int bytes) {
  limit = bytes;
  if (bytes == 2000) {        // set, but not recorded before the smaller one is
    large_inside = 1;
    wait_for(small_recorded);
  }
  return cudaSuccess;
}

int main() {
  const void *kern = &limit;   // any address
  std::thread large([&] { pkv::allow_smem(kern, 2000, configured); });
  wait_for(large_inside);
  std::thread small([&] { pkv::allow_smem(kern, 1000, configured); small_recorded = 1; });
  large.join();
  small.join();
  std::printf("%d %d\n", (int)limit, configured[0]);
  return 0;
}
"""


def test_the_limit_never_falls_below_the_record(tmp_path):
    include = os.path.join(os.path.dirname(os.path.dirname(libbuild.nvcc())), "include")
    if not os.path.exists(os.path.join(include, "cuda_runtime.h")) or not shutil.which("g++"):
        pytest.skip("needs g++ and the CUDA headers")
    src, exe = tmp_path / "race.cpp", tmp_path / "race"
    src.write_text(SOURCE)
    subprocess.run(["g++", "-std=c++17", "-I", include, "-I", libbuild.INCLUDE, "-I", libbuild.CSRC, str(src), "-o",
                    str(exe), "-pthread"], check=True)
    limit, record = map(int, subprocess.run([str(exe)], capture_output=True, text=True, check=True).stdout.split())
    assert record == 2000 and limit >= record
