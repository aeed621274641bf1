// Global-to-LDS copies shared by the matrix-core kernels (device side).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {
namespace dma {
// LDS byte address of a __shared__ object (wave-uniform).
__device__ __forceinline__ uint32_t lds_addr(const void *p) {
  return static_cast<uint32_t>(
      reinterpret_cast<uintptr_t>((__attribute__((address_space(3))) const void *)p));
}

// One wave-wide LDS DMA (64 lanes x 16 B into the 1 KB block at LDS byte
// address m0), written as inline assembly so the compiler does not drain
// every load in flight before later LDS reads; the explicit waits cover it.
// The s_nop separates the compiler's write of M0 from the copy that reads it.
__device__ __forceinline__ void dma16(const void *src, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off" : : "v"(src), "{m0}"(m0) : "memory");
}
// The same copy with the non-temporal policy, for data read exactly once (a
// weight block used by a single row block): streaming it past the caches
// raises the sustained read rate from about 6.1 to 7.2 TB/s on MI355X.
__device__ __forceinline__ void dma16_nt(const void *src, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, off nt" : : "v"(src), "{m0}"(m0) : "memory");
}

// The same copy addressed as a wave-uniform 64-bit base in SGPRs plus a 32-bit
// per-lane byte offset (the instruction's SGPR-base form): advancing along K
// then costs one scalar add per base instead of a 64-bit vector add per copy.
__device__ __forceinline__ void dma16s(uint32_t voff, const void *sbase, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1" : : "v"(voff), "s"(sbase), "{m0}"(m0) : "memory");
}

__device__ __forceinline__ void dma16s_nt(uint32_t voff, const void *sbase, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %0, %1 nt" : : "v"(voff), "s"(sbase), "{m0}"(m0) : "memory");
}

// 4 bytes per lane (256 B per wave), for scale bytes.
__device__ __forceinline__ void dma4s(uint32_t voff, const void *sbase, uint32_t m0) {
  asm volatile("s_nop 0\n\tglobal_load_lds_dword %0, %1" : : "v"(voff), "s"(sbase), "{m0}"(m0) : "memory");
}

// Wait until at most N of this wave's copies are in flight and its LDS reads
// are done, then meet the other waves.
template <int N>
__device__ __forceinline__ void wait_and_barrier() {
  asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(N) : "memory");
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
}
}  // namespace dma
}  // namespace moe
