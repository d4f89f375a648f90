// Host-side helpers of the serving operators (not part of the ABI).
#pragma once
#include <atomic>
#include <cstdint>

#include "fa_paged.h"
#include "host.h"

namespace fa {

// log2 of a page size the kernels take, -1 for any other.
inline int page_log2_of(int page) {
  return page == 16 ? 4 : page == 32 ? 5 : page == 64 ? 6 : page == 128 ? 7 : -1;
}

// Whether all of these addresses are multiples of `bytes` (a power of two).
template <class... P>
bool all_aligned(size_t bytes, const P*... p) {
  return ((reinterpret_cast<uintptr_t>(p) | ... | 0) & (bytes - 1)) == 0;
}

// Launches with programmatic stream serialization like launch() (host.h), for kernels
// whose dynamic shared memory limit is raised once per device instead of every call;
// `raised` is a word of bits, one per device, kept by the caller for each kernel.
template <class Kernel, class Params>
fa_status launch_raised(int kind, Kernel kernel, dim3 grid, dim3 block, size_t smem, cudaStream_t st, const Params& p,
                        std::atomic<unsigned long long>& raised) {
  int dev = 0;
  cudaError_t e = cudaGetDevice(&dev);
  const unsigned long long bit = 1ull << (dev & 63);
  if (e == cudaSuccess && !(raised.load(std::memory_order_relaxed) & bit)) {
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
    if (e == cudaSuccess) raised.fetch_or(bit);
  }
  if (e != cudaSuccess) return record_cuda_error(e);
  cudaLaunchAttribute attr[1];
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cfg.attrs = attr;
  cfg.numAttrs = 1;
  prof_before(kind, st);
  e = cudaLaunchKernelEx(&cfg, kernel, p);
  if (e == cudaSuccess) e = cudaGetLastError();
  prof_after(kind, st);
  return e == cudaSuccess ? FA_OK : record_cuda_error(e);
}

// Shape, gains, pointers and alignment of a cache (paged.cu).
fa_status kv4_cache_checks(const fa_kv4_cache* c);

}  // namespace fa
