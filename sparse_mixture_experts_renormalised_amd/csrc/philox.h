// Counter-based random numbers (device side): Philox4x32 with ten rounds, from
// J. K. Salmon, M. A. Moraes, R. O. Dror, D. E. Shaw, "Parallel random numbers:
// as easy as 1, 2, 3" (SC 2011).  A block of four 32-bit words depends on its
// counter and key alone, so a mask is made again wherever it is needed and is
// never stored.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace moe {

// Which of eight consecutive elements stay: element i of a tensor uses the
// 16-bit number i % 8 of block i / 8 (words in order, low half first), and is
// dropped where that number is below `cut` (the probability in steps of 2^-16).
struct Dropout {
  const uint64_t *rng;   // device: {seed, stream}; null: nothing is dropped
  uint32_t cut;          // 0 .. 65535
  float keep;            // 65536 / (65536 - cut)
};

struct DropKey {
  uint32_t k0, k1, s0, s1;
};

__device__ __forceinline__ DropKey drop_key(const Dropout &d) {
  DropKey k{0, 0, 0, 0};
  if (d.rng) {
    const uint64_t seed = d.rng[0], stream = d.rng[1];
    k.k0 = static_cast<uint32_t>(seed);
    k.k1 = static_cast<uint32_t>(seed >> 32);
    k.s0 = static_cast<uint32_t>(stream);
    k.s1 = static_cast<uint32_t>(stream >> 32);
  }
  return k;
}

// Block `block` of the stream: eight 16-bit numbers in four words.
__device__ __forceinline__ uint4 philox_block(const DropKey &key, uint64_t block) {
  uint32_t c0 = static_cast<uint32_t>(block), c1 = static_cast<uint32_t>(block >> 32);
  uint32_t c2 = key.s0, c3 = key.s1, k0 = key.k0, k1 = key.k1;
#pragma unroll
  for (int r = 0; r < 10; ++r) {
    const uint64_t p0 = static_cast<uint64_t>(0xD2511F53u) * c0;
    const uint64_t p1 = static_cast<uint64_t>(0xCD9E8D57u) * c2;
    c0 = static_cast<uint32_t>(p1 >> 32) ^ c1 ^ k0;
    c2 = static_cast<uint32_t>(p0 >> 32) ^ c3 ^ k1;
    c1 = static_cast<uint32_t>(p1);
    c3 = static_cast<uint32_t>(p0);
    k0 += 0x9E3779B9u;
    k1 += 0xBB67AE85u;
  }
  return make_uint4(c0, c1, c2, c3);
}

// Number j (0 .. 7) of a block.
__device__ __forceinline__ uint32_t half_of(const uint4 &b, int j) {
  const uint32_t w = j < 2 ? b.x : j < 4 ? b.y : j < 6 ? b.z : b.w;
  return j & 1 ? w >> 16 : w & 0xFFFFu;
}

}  // namespace moe
