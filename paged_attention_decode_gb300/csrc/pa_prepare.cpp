// pa_prepare.cpp -- the shared-memory opt-in of the kernels, once per kernel and device
// (declared beside the launch helpers in pa_internal.cuh).
#include <cuda_runtime.h>

#include <cstddef>
#include <mutex>
#include <set>
#include <utility>

namespace pa {

bool prepare_kernel(const void* fn, size_t smem) {
  static std::mutex mu;
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess) return false;
  try {
    std::lock_guard<std::mutex> lock(mu);
    static auto& done = *new std::set<std::pair<int, const void*>>();  // (never destroyed: calls may outlive statics)
    if (done.count({dev, fn})) return true;
    if (cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) != cudaSuccess) return false;
    done.insert({dev, fn});
    return true;
  } catch (...) {  // no memory to remember it by (the entries are C): opted in, once more the next time
    return cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem) == cudaSuccess;
  }
}

}  // namespace pa
