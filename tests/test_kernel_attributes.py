"""The table of kernel attributes without a GPU: every kernel asked for once on every
device, any number of them.  The CUDA calls are counted stand-ins."""
import os
import shutil
import subprocess

import pytest

ROOT = os.path.dirname(os.path.dirname(os.path.abspath(__file__)))

STAND_INS = r"""
#include <cuda_runtime_api.h>
thread_local int device = 0;
int asked = 0, raised = 0;
extern "C" {
cudaError_t cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
cudaError_t cudaFuncSetAttribute(const void*, cudaFuncAttribute, int) { ++raised; return cudaSuccess; }
cudaError_t cudaFuncGetAttributes(cudaFuncAttributes* a, const void* k) {
  if (!k) return cudaErrorInvalidDeviceFunction;
  ++asked;
  a->numRegs = (int)((size_t)k % 251) + device;
  return cudaSuccess;
}
}
"""

PROGRAM = r"""
#include <cstdio>
#include <thread>
#include <vector>
#include "kvc_launch.cuh"
extern thread_local int device;
extern int asked, raised;
static char kernels[3000];
int main() {
  int regs = 0;
  auto all = [&](int smem) {
    for (device = 0; device < 8; ++device)
      for (auto& k : kernels)
        if (kvc::prepare_kernel(&k, smem, &regs) != cudaSuccess || regs != (int)((size_t)&k % 251) + device) return false;
    device = 0;
    return true;
  };
  if (!all(100) || asked != 24000 || raised != 24000) return std::printf("first: %d %d\n", asked, raised), 1;
  if (!all(100) || !all(50) || asked != 24000 || raised != 24000) return std::printf("again: %d %d\n", asked, raised), 1;
  if (!all(200) || asked != 24000 || raised != 48000) return std::printf("raised: %d %d\n", asked, raised), 1;
  if (kvc::prepare_kernel(nullptr, 1) != cudaErrorInvalidDeviceFunction) return std::printf("no kernel\n"), 1;
  std::vector<std::thread> threads;
  for (int i = 0; i < 8; ++i)
    threads.emplace_back([] {
      for (auto& k : kernels) kvc::prepare_kernel(&k, 300);
    });
  for (auto& t : threads) t.join();
  if (asked != 24000 || raised != 51000) return std::printf("threads: %d %d\n", asked, raised), 1;
  return 0;
}
"""


def test_any_number_of_kernels_and_devices(tmp_path):
    nvcc = shutil.which("nvcc") or "/usr/local/cuda/bin/nvcc"
    if not os.path.exists(nvcc):
        pytest.skip("no nvcc")
    lib = os.path.join(os.path.dirname(os.path.dirname(os.path.realpath(nvcc))), "lib64")
    src, fakes, exe = tmp_path / "table.cu", tmp_path / "fakes.cpp", tmp_path / "table"
    src.write_text(PROGRAM)
    fakes.write_text(STAND_INS)
    subprocess.run([nvcc, "-std=c++17", "-gencode", "arch=compute_103a,code=sm_103a", "-cudart", "shared",
                    "-I", os.path.join(ROOT, "rank_quantized_kv_gb300", "csrc"), "-o", str(exe), str(src), str(fakes),
                    "-Xlinker", "-rpath," + lib, "-lpthread"],
                   check=True)
    out = subprocess.run([str(exe)], capture_output=True, text=True, timeout=60)
    assert out.returncode == 0, out.stdout
