// Dropout of rows: y = x / (1 - p) where an element stays, 0 where it is dropped.
// The same call on the gradient is its backward: the mask is made again from
// seed, stream and the element's index (philox.h).
//
// One pass: a thread makes the eight numbers of one block for eight elements, about
// 100 operations for 32 bytes of bf16, which the loads and stores still cover (without
// the generator: 36 us where this takes 37).  32011 x 1408 bf16 elements take 31 us,
// 5.8 TB/s in and out, with stores past the caches (37 us without); what the caches of 256 MB do
// not hold a part of moves at 4.4 to 4.6 (8.6 GB).
#include "moe_common.h"
#include "philox.h"

namespace moe {
namespace {

template <typename T>
__global__ __launch_bounds__(256) void dropout_kernel(const T *x, T *y, int64_t rows, int64_t d,
                                                      const int32_t *n_rows, Dropout drop) {
  constexpr int kVec = 16 / sizeof(T);   // elements of 16 bytes
  int64_t kept = rows;
  if (n_rows) {
    const int64_t n = *n_rows;
    kept = n < 0 ? 0 : n < rows ? n : rows;
  }
  const int64_t total = kept * d, blocks = (total + 7) / 8;
  const DropKey key = drop_key(drop);
  for (int64_t b = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x; b < blocks;
       b += static_cast<int64_t>(gridDim.x) * 256) {
    const int64_t at = b * 8;
    const uint4 r = drop.cut ? philox_block(key, static_cast<uint64_t>(b)) : make_uint4(0, 0, 0, 0);
    if (at + 8 <= total) {
#pragma unroll
      for (int h = 0; h < 8 / kVec; ++h) {
        union { uint4 q; T e[kVec]; } v;
        v.q = *reinterpret_cast<const uint4 *>(x + at + h * kVec);
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
          const float f = Act<T>::to_f32(v.e[j]) * drop.keep;
          v.e[j] = Act<T>::from_f32(half_of(r, h * kVec + j) >= drop.cut ? f : 0.0f);
        }
        __builtin_nontemporal_store(__builtin_bit_cast(u32x4_nt_t, v.q), reinterpret_cast<u32x4_nt_t *>(y + at + h * kVec));
      }
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j)
        if (at + j < total) {
          const float f = Act<T>::to_f32(x[at + j]) * drop.keep;
          y[at + j] = Act<T>::from_f32(half_of(r, j) >= drop.cut ? f : 0.0f);
        }
    }
  }
}

}  // namespace

hipError_t launch_dropout(bool bf16, const void *x, void *y, int64_t rows, int64_t d,
                          const int32_t *n_rows, const Dropout &drop, hipStream_t s) {
  const int64_t blocks = (rows * d + 7) / 8, want = (blocks + 255) / 256;
  const dim3 grid(static_cast<unsigned>(want < 2048 ? want : 2048));
  if (bf16)
    hipLaunchKernelGGL((dropout_kernel<uint16_t>), grid, dim3(256), 0, s,
                       static_cast<const uint16_t *>(x), static_cast<uint16_t *>(y), rows, d, n_rows, drop);
  else
    hipLaunchKernelGGL((dropout_kernel<float>), grid, dim3(256), 0, s, static_cast<const float *>(x),
                       static_cast<float *>(y), rows, d, n_rows, drop);
  return hipGetLastError();
}

}  // namespace moe
