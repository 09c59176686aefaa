"""The record of the shared memory that a kernel may use, which host threads
share, against a stand-in for the CUDA runtime that plays the order of events in
which two first launches of different sizes meet."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))
CUDA = os.environ.get("CUDA_HOME", "/usr/local/cuda")

PROGRAM = r"""
#include "smem_once.cuh"

#include <atomic>
#include <chrono>
#include <cstdio>
#include <thread>

using namespace std::chrono_literals;
constexpr int kLarge = 196608, kSmall = 49152;
int device = 0, limit[128], calls = 0;
bool fail = false;
std::atomic<bool> large_set{false}, small_set{false};

// up to 300 ms for `flag`
void until(std::atomic<bool>& flag) {
  for (int i = 0; i < 300 && !flag; ++i) std::this_thread::sleep_for(1ms);
}

extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) { return *d = device, cudaSuccess; }
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, cudaFuncAttribute, int v) {
  ++calls;
  if (fail) return cudaErrorInvalidValue;
  if (v == kSmall) until(large_set);   // the smaller size is set last ...
  limit[device] = v;
  if (v == kLarge) {
    large_set = true;
    until(small_set);                  // ... and the larger one recorded last
    std::this_thread::sleep_for(50ms);
  } else {
    small_set = true;
  }
  return cudaSuccess;
}

#define CHECK(x) if (!(x)) return std::printf("line %d: %s\n", __LINE__, #x), 1
int main() {
  pararnn::SmemOnce once;
  std::thread a([&] { once.allow(nullptr, kLarge); }), b([&] { once.allow(nullptr, kSmall); });
  a.join(), b.join();
  CHECK(once.allow(nullptr, kLarge) == 0 && limit[0] >= kLarge);
  const int before = calls;
  CHECK(once.allow(nullptr, kSmall) == 0 && calls == before && limit[0] >= kLarge);
  device = 100;                        // each device has its own
  CHECK(once.allow(nullptr, kSmall) == 0 && limit[100] == kSmall && once.allow(nullptr, kSmall) == 0);
  CHECK(calls == before + 1);
  fail = true;                         // a refusal is returned and not recorded
  CHECK(once.allow(nullptr, kLarge) == (int)cudaErrorInvalidValue);
  fail = false;
  CHECK(once.allow(nullptr, kLarge) == 0 && limit[100] == kLarge);
  device = 128;                        // none of this number
  CHECK(once.allow(nullptr, kSmall) == (int)cudaErrorInvalidDevice);
  return 0;
}
"""


def test_two_threads_with_different_sizes(tmp_path):
    gxx = shutil.which("g++")
    if gxx is None or not os.path.exists(f"{CUDA}/include/cuda_runtime.h"):
        pytest.skip("no host compiler or CUDA headers")
    src, exe = tmp_path / "once.cc", tmp_path / "once"
    src.write_text(PROGRAM)
    subprocess.run([gxx, "-std=c++17", "-pthread", "-I", f"{CUDA}/include", "-I",
                    f"{ROOT}/nonlinear_rnn_paragru_b200/csrc", str(src), "-o", str(exe)], check=True)
    r = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert r.returncode == 0, r.stdout
