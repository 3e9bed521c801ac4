"""The step kernels' raised limit of dynamic LDS (CPU): set once for each kernel on each device, compiled against a stand-in
for the runtime that keeps what was set."""
import os
import subprocess

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

RUNTIME = """
#pragma once
#include <map>
#include <utility>
enum hipError_t { hipSuccess, hipErrorUnknown };
enum { hipDeviceAttributeMaxSharedMemoryPerBlock, hipFuncAttributeMaxDynamicSharedMemorySize };
inline int device, calls;
inline bool fails;
inline std::map<std::pair<int, const void*>, int> limit;
inline hipError_t hipGetDevice(int* d) { *d = device; return hipSuccess; }
inline hipError_t hipDeviceGetAttribute(int* v, int, int) { *v = 163840; return hipSuccess; }
inline hipError_t hipFuncSetAttribute(const void* f, int, int n) {
  ++calls;
  if (fails) return hipErrorUnknown;
  limit[{device, f}] = n;
  return hipSuccess;
}
"""

MAIN = """
#include <cassert>
#include <cstdio>
#include "lds_limit.h"
int main() {
  int a, b;
  for (int again = 0; again < 2; ++again)
    for (device = 0; device < 3; ++device) {
      assert(qmoe::raise_dyn_lds(&a, 16384) == hipSuccess && qmoe::raise_dyn_lds(&b, 0) == hipSuccess);
      assert(limit.at({device, &a}) == 163840 - 16384 && limit.at({device, &b}) == 163840);
    }
  assert(calls == 6);
  fails = true;
  int c;
  assert(qmoe::raise_dyn_lds(&c, 0) == hipErrorUnknown);
  fails = false;
  assert(qmoe::raise_dyn_lds(&c, 0) == hipSuccess && limit.at({device, &c}) == 163840);
  puts("fine");
}
"""


def test_limit_of_each_device(tmp_path):
    (tmp_path / "hip").mkdir()
    (tmp_path / "hip" / "hip_runtime.h").write_text(RUNTIME)
    (tmp_path / "main.cpp").write_text(MAIN)
    exe = str(tmp_path / "main")
    csrc = os.path.join(ROOT, "bit_quantized_moe_02_amd", "csrc")
    subprocess.run(["g++", "-std=c++17", "-O1", "-I", str(tmp_path), "-I", csrc, str(tmp_path / "main.cpp"), "-o", exe, "-lpthread"],
                   check=True, timeout=120)
    r = subprocess.run([exe], stdout=subprocess.PIPE, stderr=subprocess.STDOUT, text=True, timeout=60)
    assert r.returncode == 0 and r.stdout == "fine\n", r.stdout
