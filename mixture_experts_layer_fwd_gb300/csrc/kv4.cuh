// The paged NVFP4 key/value cache: layout of a record and the helpers that
// every kernel on it shares.
//
// A layer's pool is [num_pages][Hkv] records.  One record holds `P` tokens of
// one kv head: key codes [P][D/2], key scales [P][D/16], value codes, value
// scales, one after the other (P * D * 9/8 bytes).  Records are contiguous so
// that one bulk copy brings everything an attention step needs of a page and
// head into shared memory, and a page of a layer is one contiguous block.
// P % 16 == 0 and D in {64, 128} make every section start on a 16-byte
// boundary and the record a multiple of 16 bytes.
#pragma once

#include <atomic>

#include "nvfp4.cuh"

namespace moe {
namespace kv4 {

__host__ __device__ constexpr int codes_bytes(int P, int D) { return P * D / 2; }
__host__ __device__ constexpr int scale_bytes(int P, int D) { return P * D / 16; }
__host__ __device__ constexpr int record_bytes(int P, int D) { return 2 * (codes_bytes(P, D) + scale_bytes(P, D)); }

inline bool page_size_ok(int P) { return P == 32 || P == 64 || P == 128; }
inline bool head_dim_ok(int D) { return D == 64 || D == 128; }

// Programmatic dependent launch: the next kernel of the call may start its
// prologue now; and: wait for the results of the one before.
DEVINL void launch_dependents() { asm volatile("griddepcontrol.launch_dependents;" ::: "memory"); }
DEVINL void wait_for_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
template <class... Params, class... Args>
inline int launch_after(void (*kernel)(Params...), dim3 grid, int threads, int smem, cudaStream_t s, Args... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid, cfg.blockDim = dim3(threads), cfg.dynamicSmemBytes = smem, cfg.stream = s;
  cudaLaunchAttribute a{};
  a.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  a.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &a, cfg.numAttrs = 1;
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, args...);
  if (e != cudaSuccess) {
    set_cuda_error(e);
    return MOE_ERR_CUDA;
  }
  return MOE_OK;
}

// Pairs of fp32 in one register pair; each half is one IEEE operation.
DEVINL uint64_t pair(float a, float b) {
  uint64_t r;
  asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(a), "f"(b));
  return r;
}
DEVINL void unpair(uint64_t v, float& a, float& b) { asm("mov.b64 {%0, %1}, %2;" : "=f"(a), "=f"(b) : "l"(v)); }
DEVINL uint64_t fma2(uint64_t a, uint64_t b, uint64_t c) {
  uint64_t r;
  asm("fma.rn.f32x2 %0, %1, %2, %3;" : "=l"(r) : "l"(a), "l"(b), "l"(c));
  return r;
}
DEVINL uint64_t add2(uint64_t a, uint64_t b) {
  uint64_t r;
  asm("add.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
  return r;
}

// Lets a kernel use `bytes` of shared memory on the current device; `set` is the
// kernel's own, by device.  Calls of several threads may come here at once: each
// sets the same value.
template <class... Params>
inline int allow_smem(void (*kernel)(Params...), int bytes, std::atomic<bool> (&set)[64]) {
  int dev = 0;
  if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return MOE_ERR_CUDA;
  if (!set[dev].load(std::memory_order_relaxed)) {
    const cudaError_t e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (e != cudaSuccess) {
      set_cuda_error(e);
      return MOE_ERR_CUDA;
    }
    set[dev].store(true, std::memory_order_relaxed);
  }
  return MOE_OK;
}

}  // namespace kv4
}  // namespace moe
