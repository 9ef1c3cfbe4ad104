"""The kernels' shared-memory limits under several host threads: csa2_smem_limit.cuh compiled for the host,
with a stand-in for the call that sets a limit."""
import os
import shutil
import subprocess

import pytest

CSRC = os.path.join(os.path.dirname(os.path.dirname(os.path.abspath(__file__))), "fp4_compressed_sparse_gb300", "csrc")

PROGRAM = r"""
#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>
#include "csa2_smem_limit.cuh"

int main() {
  using namespace std::chrono;
  csa2::SmemLimits limits;
  int a = 0, b = 0;
  // a kernel's limit, as the driver would hold it: the last one set.  The thread with the small size
  // misses first, and its call takes effect after the other one's, if that may overtake it.
  std::atomic<int> limit{0}, calls{0};
  std::atomic<bool> in_small{false}, large_set{false};
  std::thread small([&] {
    limits.raise(0, &a, 60, [&] {
      in_small = true;
      for (auto t = steady_clock::now(); !large_set && steady_clock::now() - t < milliseconds(500);) std::this_thread::yield();
      limit = 60, ++calls;
      return 0;
    });
  });
  std::thread large([&] {
    while (!in_small) std::this_thread::yield();
    limits.raise(0, &a, 200, [&] { limit = 200, ++calls; large_set = true; return 0; });
  });
  small.join();
  large.join();
  limits.raise(0, &a, 200, [&] { limit = 200, ++calls; return 0; });
  std::printf("%d %d\n", limit.load(), calls.load());
  // what is high enough is not set again; another kernel or device is; a failure is tried again
  int n = 0;
  auto set = [&] { ++n; return 0; };
  limits.raise(0, &a, 200, set), limits.raise(0, &a, 100, set);
  std::printf("%d ", n);
  limits.raise(0, &b, 100, set), limits.raise(1, &a, 100, set);
  std::printf("%d ", n);
  std::printf("%d ", limits.raise(0, &b, 300, [&] { return 7; }));
  limits.raise(0, &b, 300, set);
  std::printf("%d\n", n);
}
"""


def test_the_larger_limit_stays(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None:
        pytest.skip("no host compiler")
    src, exe = tmp_path / "limits.cc", tmp_path / "limits"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-O1", "-pthread", "-I", CSRC, str(src), "-o", str(exe)], check=True)
    out = subprocess.run([str(exe)], check=True, capture_output=True, text=True, timeout=60).stdout.split("\n")
    assert out[0] == "200 2"
    assert out[1] == "0 2 7 3"
