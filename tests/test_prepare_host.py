"""The kernels' shared-memory opt-in (pa_prepare.cpp) against a stand-in for the two CUDA calls it makes (no GPU needed)."""
import os
import shutil
import subprocess

import pytest

from paged_attention_decode_gb300 import build as pa_build

PROGRAM = r"""
#include <cuda_runtime.h>
#include <cstdio>
#include <cstdlib>

namespace pa { bool prepare_kernel(const void* fn, size_t smem); }

static int device = 0, calls = 0, last_bytes = 0;
static cudaError_t answer = cudaSuccess;
extern "C" cudaError_t CUDARTAPI cudaGetDevice(int* d) { *d = device; return cudaSuccess; }
extern "C" cudaError_t CUDARTAPI cudaFuncSetAttribute(const void*, enum cudaFuncAttribute, int bytes) {
  ++calls;
  last_bytes = bytes;
  return answer;
}

#define CHECK(x) do { if (!(x)) { std::printf("line %d: %s\n", __LINE__, #x); return 1; } } while (0)

int main() {
  static char kernels[5000];
  answer = cudaErrorInvalidValue;  // a refusal is passed on, and not remembered
  CHECK(!pa::prepare_kernel(&kernels[0], 100));
  answer = cudaSuccess;
  calls = 0;
  for (int round = 0; round < 3; ++round)
    for (int d = 0; d < 3; ++d) {
      device = d;
      for (int k = 0; k < 5000; ++k) CHECK(pa::prepare_kernel(&kernels[k], 1000 + k));
    }
  CHECK(calls == 3 * 5000);  // once per kernel and device
  device = 200;              // a device of any number
  CHECK(pa::prepare_kernel(&kernels[7], 4321) && last_bytes == 4321);
  return 0;
}
"""


def test_every_kernel_is_prepared_once_however_many_there_are(tmp_path):
    cxx = shutil.which("g++") or shutil.which("c++")
    if cxx is None:
        pytest.skip("no C++ compiler")
    (tmp_path / "main.cpp").write_text(PROGRAM)
    cuda = os.path.join(os.path.dirname(os.path.dirname(pa_build._nvcc())), "include")
    exe = str(tmp_path / "prepare")
    subprocess.run([cxx, "-std=c++17", "-O1", f"-I{cuda}", str(tmp_path / "main.cpp"),
                    os.path.join(pa_build.CSRC, "pa_prepare.cpp"), "-o", exe, "-pthread"], check=True)
    run = subprocess.run([exe], capture_output=True, text=True, timeout=60)
    assert run.returncode == 0, run.stdout
