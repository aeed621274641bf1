// The whole layer for 1 to 16 tokens in two kernels ([DSMoE] output equation
// with the routing of [TopK] and the capacity limit of [TopK] 解決策2).
//
// With so few tokens the layer is one pass over the weights of the experts
// the tokens meet, and the rest is latency.  The general path starts seven or
// more kernels and keeps per-expert row lists in memory; here
//
//   kernel 1 (few_logits_kernel) computes the router's logits, one workgroup
//     per expert, and clears the states, counts and row of zeros of kernel 2;
//   kernel 2 (few_layer_kernel) does the rest.  Every workgroup repeats the
//     top-K selection, gates and capacity from the logits (T * N numbers)
//     into LDS.  Then come the hidden rows of every met or shared expert (up
//     items), and after them the output rows (down items).
//
// The 16 tokens are the 16 columns of one matrix instruction, and the rows of
// a weight matrix are its rows: a wave multiplies 16 R weight rows by a share
// of the reduction axis, every lane loading its weights straight from memory
// in the instruction's own layout (each lane of a row takes 16 or 32
// neighbouring bytes, so a row is read in whole 64- or 128-byte pieces).  A token that
// is not routed to the expert is a column of zeros that is never loaded.
//
// Hidden values carry the gate (g * SiLU(.)), so a down item sums over all
// (expert, hidden) pairs in one accumulator and no per-expert output exists.
// They are kept in two bf16 parts (value, and what its rounding left: 16
// significant bits, for the price of a second matrix instruction on a
// bandwidth-bound path); float32 layers keep float32.
//
// Waiting.  A down item needs every hidden row.  The up items are dealt to as
// many shares as there are workgroups, and a share has a state: free, taken,
// done.  A workgroup takes its own share first, and where it then waits for all
// shares to be done, it takes any that is still free (its workgroup has not
// started yet).  So a share that is waited for is either taken, by a workgroup
// that runs and does not wait before it is done, or will be taken by one that
// waits: every wait ends, whatever the number of resident workgroups and
// whatever else runs on the device.  One counter that deals the items out would
// be simpler, but atomics on one address cost about 80 ns each here.
//
// Results do not depend on timing: sums are split in a way fixed by the sizes
// and joined in a fixed order.
#include <type_traits>

#include "moe_common.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

enum : uint32_t { kFree = 0, kTaken = 1, kDone = 2 };   // states of an up share
constexpr int kTok = 16;            // columns of the matrix instruction
constexpr int kWaves = 4;
constexpr int kThreads = kWaves * 64;
constexpr int kGrid = 512;          // most workgroups: two per CU

// ---------------------------------------------------------------------------
// Kernel 1: logits
// ---------------------------------------------------------------------------
template <typename T>
__device__ __forceinline__ float4 load4(const T *p);
template <>
__device__ __forceinline__ float4 load4<float>(const float *p) {
  return *reinterpret_cast<const float4 *>(p);
}
template <>
__device__ __forceinline__ float4 load4<uint16_t>(const uint16_t *p) {
  const uint2 v = *reinterpret_cast<const uint2 *>(p);
  return make_float4(__uint_as_float(v.x << 16), __uint_as_float(v.x & 0xFFFF0000u),
                     __uint_as_float(v.y << 16), __uint_as_float(v.y & 0xFFFF0000u));
}

// Words to clear for kernel 2: the states and counts, and the row of zeros.
struct FewZero {
  uint32_t *p[5];
  int n[5];
};

// Activations of MXFP4 layers enter the scaled matrix instructions as sums of
// E4M3 numbers: per block of 32 a scale 2^E, E the smallest integer with
// max|v| <= 448 * 2^E, and parts v / 2^E = p0 + p1 / 16 + p2 / 256 + ..., each
// part the nearest E4M3 number to what the ones before it left, times 16.  A
// part holds four significant bits, and what it leaves is at most 1/16 of it.
// So two parts hold a bf16 number (eight bits) exactly, down to 2^-14 of the
// block's largest; below, they are off by at most 2^-22 of the largest.  The
// parts' scales are 2^E, 2^(E-4), 2^(E-8).  E is at least -119, so that these
// are scale bytes; a block that holds an infinity or a NaN gets byte 255.
constexpr int kMinPartE = -119;
__device__ __forceinline__ int part_exponent(uint32_t amax_bits) {
  if (amax_bits == 0) return 0;
  const int e = static_cast<int>(amax_bits >> 23) - 126;         // a = m 2^e, 448 = 0.875 * 2^9
  const int E = (amax_bits & 0x7FFFFFu) <= 0x600000u ? e - 9 : e - 8;
  return max(E, kMinPartE);
}
// Next part of four numbers (as four E4M3 bytes), and what it leaves, times 16.
__device__ __forceinline__ uint32_t take_part(float (&v)[4]) {
  int w = __builtin_amdgcn_cvt_pk_fp8_f32(v[0], v[1], 0, false);
  w = __builtin_amdgcn_cvt_pk_fp8_f32(v[2], v[3], w, true);
  const f32x2_t lo = __builtin_amdgcn_cvt_pk_f32_fp8(w, false);
  const f32x2_t hi = __builtin_amdgcn_cvt_pk_f32_fp8(w, true);
  v[0] = (v[0] - lo.x) * 16.0f;
  v[1] = (v[1] - lo.y) * 16.0f;
  v[2] = (v[2] - hi.x) * 16.0f;
  v[3] = (v[3] - hi.y) * 16.0f;
  return static_cast<uint32_t>(w);
}

// Token rows as two parts: eight lanes a block, four elements each.
__device__ __forceinline__ void split_tokens(const uint16_t *x, int64_t unit, int64_t units,
                                             uint32_t *xq, uint8_t *xs) {
  if (unit >= units) return;                // units is a multiple of 8: whole blocks leave
  const float4 q = load4<uint16_t>(x + unit * 4);
  float v[4] = {q.x, q.y, q.z, q.w};
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(v[j]) & 0x7FFFFFFFu);
#pragma unroll
  for (int off = 1; off < 8; off <<= 1)
    amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), off)));
  const int E = part_exponent(amax);
#pragma unroll
  for (int j = 0; j < 4; ++j) v[j] = __builtin_ldexpf(v[j], -E);
  xq[unit] = take_part(v);
  xq[units + unit] = take_part(v);
  if ((unit & 7) == 0) xs[unit >> 3] = static_cast<uint8_t>(amax >= 0x7F800000u ? 255 : E + 127);
}

// One workgroup per expert: thread i sums elements 4i, 4i + 4096, ... of
// W_e . x_t for each token, then the wave and the sixteen waves are added in a
// fixed tree.  TT is T rounded up to a power of two (the loads of a step are
// issued together); columns past T repeat the last token and are not stored.
// Workgroups past the experts split the token rows into parts (xq not null).
constexpr int kLogitThreads = 1024;
template <typename T, int TT>
__global__ __launch_bounds__(kLogitThreads) void few_logits_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    float *__restrict__ logits, int tokens, int d, int N, FewZero zero, uint32_t *xq, uint8_t *xs) {
  constexpr int NW = kLogitThreads / 64;
  __shared__ float s_part[NW][TT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x;
  if constexpr (sizeof(T) == 2)
    if (e >= N) {
      split_tokens(x, static_cast<int64_t>(e - N) * kLogitThreads + tid,
                   static_cast<int64_t>(tokens) * d / 4, xq, xs);
      return;
    }
  const float *wr = w + static_cast<int64_t>(e) * d;
  float acc[TT];
#pragma unroll
  for (int t = 0; t < TT; ++t) acc[t] = 0.0f;
  for (int k = tid * 4; k < d; k += kLogitThreads * 4) {
    const float4 wv = load4<float>(wr + k);
    float4 xv[TT];
#pragma unroll
    for (int t = 0; t < TT; ++t)
      xv[t] = load4<T>(x + static_cast<int64_t>(min(t, tokens - 1)) * d + k);
#pragma unroll
    for (int t = 0; t < TT; ++t) {
      acc[t] = __builtin_fmaf(wv.x, xv[t].x, acc[t]);
      acc[t] = __builtin_fmaf(wv.y, xv[t].y, acc[t]);
      acc[t] = __builtin_fmaf(wv.z, xv[t].z, acc[t]);
      acc[t] = __builtin_fmaf(wv.w, xv[t].w, acc[t]);
    }
  }
#pragma unroll
  for (int r = 0; r < 5; ++r)
    for (int i = e * kLogitThreads + tid; i < zero.n[r]; i += N * kLogitThreads) zero.p[r][i] = 0;
#pragma unroll
  for (int off = 32; off >= 1; off >>= 1)
#pragma unroll
    for (int t = 0; t < TT; ++t) acc[t] += __shfl_xor(acc[t], off);
  if (lane == 0)
#pragma unroll
    for (int t = 0; t < TT; ++t) s_part[wave][t] = acc[t];
  __syncthreads();
  if (tid < tokens) {
    float v[NW];
#pragma unroll
    for (int i = 0; i < NW; ++i) v[i] = s_part[i][tid];
#pragma unroll
    for (int n = NW / 2; n >= 1; n /= 2)
#pragma unroll
      for (int i = 0; i < n; ++i) v[i] += v[i + n];
    logits[static_cast<int64_t>(tid) * N + e] = bias ? v[0] + bias[e] : v[0];
  }
}

// ---------------------------------------------------------------------------
// Kernel 2
// ---------------------------------------------------------------------------
struct FewArgs {
  const void *x;                         // token rows (MXFP4 layers: their parts [2][T][d])
  const uint8_t *xs;                     // scale bytes of the parts
  const float *logits, *sel_bias;
  const void *w1, *b1, *w2, *b2, *ws1, *bs1, *ws2, *bs2;
  const uint8_t *c1, *c2, *cs1, *cs2;   // scale bytes of MXFP4 weights
  // hidden rows and one of zeros: float [rows + 1][f], bf16 parts [2][rows + 1][f]
  // or E4M3 parts [3][rows + 1][f] with scale bytes hs
  void *h;
  uint8_t *hs;
  float *part;                           // [S][T][d] parts of split outputs
  uint32_t *state;                       // [grid] of the up shares
  uint32_t *arrived;                     // [row blocks] finished parts of split outputs
  void *y;
  int32_t *idx;
  float *gate;
  int32_t *counts;
  int T, d, N, K, Ks, f, S;
  int cap;                               // rows an expert keeps (T or more: no limit)
};

// The three kinds of weights.
//   CH      elements of the reduction axis in a chunk, what the four lanes of a
//           row load together
//   ABYTES  bytes of a row's chunk, in pieces of 64 neighbouring bytes, 16 a lane
//   BBYTES  bytes of a chunk of one part of the activations, in such pieces too
//   PUP, PDN  parts of the activations of the first and of the second Linear
//   UNIT    16-row tiles that hidden rows are dealt out in (a block of hidden
//           values has 32 rows)
enum { kWF32, kWBf16, kWMx };
template <int W> struct Kind;
template <> struct Kind<kWF32> {
  using Act = float;
  static constexpr int CH = 16, ABYTES = 64, BBYTES = 64, PUP = 1, PDN = 1, UNIT = 1;
};
template <> struct Kind<kWBf16> {
  using Act = uint16_t;
  static constexpr int CH = 64, ABYTES = 128, BBYTES = 128, PUP = 1, PDN = 2, UNIT = 1;
};
template <> struct Kind<kWMx> {
  using Act = uint16_t;
  static constexpr int CH = 128, ABYTES = 64, BBYTES = 128, PUP = 2, PDN = 3, UNIT = 2;
};
constexpr int kMaxTiles = 4;        // 16-row tiles of a wave
constexpr int kDepth = 2;           // chunks in flight per wave

template <int W> struct AFrag {
  u32x4_t v[Kind<W>::ABYTES / 64];
  int s;
};
template <int W, int P> struct BFrag {
  u32x4_t v[P][Kind<W>::BBYTES / 64];
  int s;
};

// Chunk c of the row whose first byte for this lane is base + row (base is
// wave-uniform), and of a row of activations.
template <int W>
__device__ __forceinline__ void load_a(AFrag<W> &a, const uint8_t *base, uint32_t row, int c) {
#pragma unroll
  for (int j = 0; j < Kind<W>::ABYTES / 64; ++j)
    a.v[j] = *reinterpret_cast<const u32x4_t *>(
        base + (row + static_cast<uint32_t>(c) * Kind<W>::ABYTES + j * 64));
}
template <int W, int P>
__device__ __forceinline__ void load_b(BFrag<W, P> &b, const uint8_t *base, int64_t part, uint32_t row,
                                       int c) {
#pragma unroll
  for (int p = 0; p < P; ++p)
#pragma unroll
    for (int j = 0; j < Kind<W>::BBYTES / 64; ++j)
      b.v[p][j] = *reinterpret_cast<const u32x4_t *>(
          base + p * part + (row + static_cast<uint32_t>(c) * Kind<W>::BBYTES + j * 64));
}

// acc += A (B_0 + B_1 + ...), 16 weight rows x 16 columns.  For MXFP4 weights
// a lane's 16 bytes of codes are one block; its E4M3 operand holds elements
// 16 q .. +15 and 64 + 16 q .. +15 of the chunk's 128.
template <int W, int P>
__device__ __forceinline__ void mma(f32x4_t &acc, const AFrag<W> &a, const BFrag<W, P> &b) {
  if constexpr (W == kWF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[0][j]),
                                                 __uint_as_float(b.v[0][0][j]), acc, 0, 0, 0);
  } else if constexpr (W == kWBf16) {
#pragma unroll
    for (int j = 0; j < 2; ++j)
#pragma unroll
      for (int p = 0; p < P; ++p)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v[j]),
                                                      __builtin_bit_cast(bf16x8_t, b.v[p][j]), acc, 0,
                                                      0, 0);
  } else {
    const i32x8_t av = {(int)a.v[0][0], (int)a.v[0][1], (int)a.v[0][2], (int)a.v[0][3], 0, 0, 0, 0};
#pragma unroll
    for (int p = 0; p < P; ++p) {
      const i32x8_t bv = {(int)b.v[p][0][0], (int)b.v[p][0][1], (int)b.v[p][0][2], (int)b.v[p][0][3],
                          (int)b.v[p][1][0], (int)b.v[p][1][1], (int)b.v[p][1][2], (int)b.v[p][1][3]};
      acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc, 4, 0, 0, a.s, 0,
                                                             b.s - 4 * p);
    }
  }
}

// Larger float, larger key; NaN sorts somewhere, so that a selection always
// names distinct experts in range.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v);
  return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}

// Largest value of the wave: within each row of 16 lanes by lane permutations,
// then the four rows.
__device__ __forceinline__ uint32_t wave_max(uint32_t v) {
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0xB1, 0xF, 0xF, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x4E, 0xF, 0xF, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x141, 0xF, 0xF, true)));
  v = max(v, static_cast<uint32_t>(__builtin_amdgcn_mov_dpp(static_cast<int>(v), 0x140, 0xF, 0xF, true)));
  const uint32_t a = __builtin_amdgcn_readlane(v, 0), b = __builtin_amdgcn_readlane(v, 16);
  const uint32_t c = __builtin_amdgcn_readlane(v, 32), d = __builtin_amdgcn_readlane(v, 48);
  return max(max(a, b), max(c, d));
}

// Stores and loads of data that other workgroups of the same launch read or
// wrote: at device scope, so they pass the L2 caches of the eight XCDs, which
// are not coherent with each other.  A fence in their place would write back a
// whole L2 for every item (measured: 121 us for the layer that takes 116 MB of
// weights, against REPLACED us this way).
template <typename T>
__device__ __forceinline__ void put_shared(T *p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T get_shared(const T *p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
// This wave's device-scope stores have arrived.
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float act_f32(const void *p, int64_t i, float) {
  return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ float act_f32(const void *p, int64_t i, uint16_t) {
  return bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}

template <int W>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  using KD = Kind<W>;
  using Act = typename KD::Act;
  __shared__ int16_t s_pair[kMaxRouted * kTok];    // hidden row of (entry, token), or -1
  __shared__ int16_t s_list[kMaxRouted];           // expert of each entry
  __shared__ alignas(4) uint16_t s_mask[kMaxRouted];   // tokens of each expert
  __shared__ float s_gate[kTok * 64];
  __shared__ int16_t s_idx[kTok * 64];
  __shared__ float s_red[kWaves][kMaxTiles][256];
  __shared__ uint32_t s_last;
  __shared__ int s_free, s_claim;
  __shared__ int s_ne;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int T = a.T, K = a.K, N = a.N, Ks = a.Ks, d = a.d, f = a.f;

  // ---- routing ----
  auto claim = [&](int w) {
    uint32_t was = kFree;
    __hip_atomic_compare_exchange_strong(a.state + w, &was, kTaken, __ATOMIC_RELAXED, __ATOMIC_RELAXED,
                                         __HIP_MEMORY_SCOPE_AGENT);
    return was == kFree;
  };
  int mine_claim = 0;                      // the last wave has the fewest tokens
  if (tid == kThreads - 64) mine_claim = claim(blockIdx.x);
  if (tid == 0) s_free = kGrid;
  for (int e = tid; e < N; e += kThreads) s_mask[e] = 0;
  for (int t = wave; t < T; t += kWaves) {
    constexpr int NJ = kMaxRouted / 64;
    uint32_t key[NJ];
    float val[NJ];
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j * 64 >= N) break;
      const int e = j * 64 + lane;
      val[j] = e < N ? a.logits[static_cast<int64_t>(t) * N + e] : 0.0f;
    }
#pragma unroll
    for (int j = 0; j < NJ; ++j) {
      if (j * 64 >= N) break;
      const int e = j * 64 + lane;
      const float v = a.sel_bias && e < N ? val[j] + a.sel_bias[e] : val[j];
      key[j] = e < N ? max(order_key(v), 1u) : 0;
    }
    float mine = -__builtin_inff();
    int mine_e = 0;
    for (int k = 0; k < K; ++k) {
      // this lane's best, the wave's, and the lowest id among equals
      uint32_t best = 0;
      int at = lane;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (j * 64 >= N) break;
        if (key[j] > best) {
          best = key[j];
          at = j * 64 + lane;
        }
      }
      const uint32_t top = wave_max(best);
      uint64_t who = __ballot(best == top);
      int e = __builtin_amdgcn_readlane(at, __builtin_ctzll(who));
      while (who &= who - 1) e = min(e, __builtin_amdgcn_readlane(at, __builtin_ctzll(who)));
      float logit = 0.0f;
#pragma unroll
      for (int j = 0; j < NJ; ++j) {
        if (j * 64 >= N) break;
        if (e == j * 64 + lane) {
          key[j] = 0;
          logit = val[j];
        }
      }
      logit = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(logit), e & 63));
      if (lane == k) {
        mine_e = e;
        mine = logit;
      }
    }
    float top = mine;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) top = fmaxf(top, __shfl_xor(top, off));
    float g = lane < K ? expf(mine - top) : 0.0f, sum = g;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) sum += __shfl_xor(sum, off);
    if (lane < K) {
      s_idx[t * 64 + lane] = static_cast<int16_t>(mine_e);
      s_gate[t * 64 + lane] = g / sum;
      if (blockIdx.x == 0) {
        if (a.idx) a.idx[t * K + lane] = mine_e;
        if (a.gate) a.gate[t * K + lane] = g / sum;
      }
    }
  }
  if (tid == kThreads - 64) s_claim = mine_claim;
  __syncthreads();
  // token masks
  for (int i = tid; i < T * 64; i += kThreads)
    if ((i & 63) < K) {
      const int e = s_idx[i];
      atomicOr(reinterpret_cast<uint32_t *>(s_mask) + (e >> 1), (1u << (i >> 6)) << ((e & 1) * 16));
    }
  __syncthreads();
  // an expert keeps its first cap tokens; the met experts, in order
  if (a.cap < T) {
    for (int e = tid; e < N; e += kThreads) {
      uint32_t m = s_mask[e], kept = 0;
      for (int c = 0; c < a.cap && m; ++c) {
        kept |= m & (0u - m);
        m &= m - 1;
      }
      s_mask[e] = static_cast<uint16_t>(kept);
    }
    __syncthreads();
  }
  if (blockIdx.x == 0 && a.counts)
    for (int e = tid; e < N; e += kThreads) a.counts[e] = __popc(s_mask[e]);
  if (wave == 0) {
    int base = 0;
    for (int e0 = 0; e0 < N; e0 += 64) {
      const int e = e0 + lane;
      const bool met = e < N && s_mask[e] != 0;
      const uint64_t b = __ballot(met);
      if (met) s_list[base + __popcll(b & ((1ull << lane) - 1))] = static_cast<int16_t>(e);
      base += __popcll(b);
    }
    if (lane == 0) s_ne = base;
  }
  __syncthreads();
  const int ne = uniform(s_ne), entries = ne + Ks;
  for (int i = tid; i < ne * kTok; i += kThreads) {
    const int e = s_list[i >> 4], t = i & 15;
    int row = -1;
    if ((s_mask[e] >> t) & 1)
      for (int k = 0; k < K; ++k)
        if (s_idx[t * 64 + k] == e) row = t * K + k;
    s_pair[i] = static_cast<int16_t>(row);
  }
  __syncthreads();

  // ---- the sums ----
  const int col = lane & 15, q = lane >> 4;
  const int pairs = T * (K + Ks);
  // hidden row of (entry, token): routed pairs first, then the shared experts
  auto hidden_row = [&](int i, int t) -> int {
    if (i < ne) return s_pair[i * kTok + t];
    return t < T ? T * K + (i - ne) * T + t : -1;
  };

  // Sums of R tiles of 16 weight rows over every `step`-th chunk from chunk cc
  // of entry i on, n of them.  row[r] is the byte offset of the lane's row, at
  // the first chunk, from the matrix at wb[r] (scale bytes: row / 16 from
  // cb[r]); `next` moves those and the activations' row br to entry i.
  auto walk = [&](auto parts, auto &acc, const uint8_t *bb, const uint8_t *bs, int64_t part, int nch,
                  const uint8_t *(&wb)[kMaxTiles], const uint8_t *(&cb)[kMaxTiles],
                  const uint32_t (&row)[kMaxTiles], uint32_t &br, int i, int cc, int n, int step,
                  auto next) {
    constexpr int R = std::extent_v<std::remove_reference_t<decltype(acc)>>;
    constexpr int P = decltype(parts)::value, D = kDepth;
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    struct Stage {
      AFrag<W> a[R];
      BFrag<W, P> b;
    } st[D];
    auto fetch = [&](Stage &s) {
      load_b<W, P>(s.b, bb, part, br * KD::BBYTES + q * 16, cc);
      if constexpr (W == kWMx) s.b.s = bs[br * 4 + cc * 4 + q];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        load_a<W>(s.a[r], wb[r], row[r] * KD::ABYTES + q * 16, cc);
        if constexpr (W == kWMx) s.a[r].s = cb[r][row[r] * 4 + cc * 4 + q];
      }
      cc += step;
      if (cc >= nch) {
        do {
          cc -= nch;
          ++i;
        } while (cc >= nch);
        next(i);
      }
    };
    auto use = [&](Stage &s) {
#pragma unroll
      for (int r = 0; r < R; ++r) mma<W, P>(acc[r], s.a[r], s.b);
    };
    if (n < D) {
      for (int c = 0; c < n; ++c) {
        fetch(st[0]);
        use(st[0]);
      }
      return;
    }
#pragma unroll
    for (int k = 0; k < D; ++k) fetch(st[k]);
    int left = n - D;
    for (; left >= D; left -= D) {
#pragma unroll
      for (int k = 0; k < D; ++k) {
        use(st[k]);
        fetch(st[k]);
      }
    }
#pragma unroll
    for (int k = 0; k < D; ++k) {
      use(st[k]);
      if (k < left) fetch(st[k]);
    }
#pragma unroll
    for (int k = 0; k < D; ++k)
      if (k < left) use(st[k]);
  };

  // ---- hidden rows ----
  // All tiles of all entries form one row; share w is a range of it.  A wave
  // sums up to kMaxTiles tiles, over the whole reduction axis when the range
  // is long enough to keep the four waves busy that way, else over half or a
  // quarter of it (`ks` waves a tile), joined through LDS.
  const int grid = gridDim.x;
  constexpr int U = KD::UNIT;
  const int per_entry = (f / 16 + U - 1) / U;              // units of an entry (f is a multiple of 16)
  const int units = entries * per_entry;
  const int ks = units * U > 8 * grid ? 1 : units * U > 4 * grid ? 2 : 4;
  const int64_t hsize = static_cast<int64_t>(pairs + 1) * f;
  // Hidden values of the sums z[0 .. U-1][4]: tiles u*U .., rows 4q .. 4q+3,
  // for token `col`.
  auto hidden_out = [&](int u, f32x4_t (&z)[U]) {
    const int i = u / per_entry, r0 = (u - i * per_entry) * U * 16 + q * 4;
    const bool routed = i < ne;
    const int64_t e = routed ? s_list[i] : i - ne;
    const void *bias = routed ? a.b1 : a.bs1;
    const int hr = hidden_row(i, col);
    const float g = routed && hr >= 0 ? s_gate[col * 64 + (hr - col * K)] : 1.0f;
#pragma unroll
    for (int x = 0; x < U; ++x)
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (bias) z[x][j] += act_f32(bias, e * f + r0 + x * 16 + j, Act{});
        z[x][j] = g * silu(z[x][j]);
      }
    const int64_t at = static_cast<int64_t>(hr) * f + r0;
    if constexpr (W == kWF32) {
      uint64_t *hp = static_cast<uint64_t *>(a.h);
      if (hr < 0) return;
#pragma unroll
      for (int j = 0; j < 2; ++j)
        put_shared(hp + at / 2 + j, __float_as_uint(z[0][2 * j]) |
                                        static_cast<uint64_t>(__float_as_uint(z[0][2 * j + 1])) << 32);
    } else if constexpr (W == kWBf16) {
      uint64_t *hp = static_cast<uint64_t *>(a.h);
      if (hr < 0) return;
      uint32_t hi[2], lo[2];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        hi[j] = pack_bf16x2(z[0][2 * j], z[0][2 * j + 1]);
        lo[j] = pack_bf16x2(z[0][2 * j] - __uint_as_float(hi[j] << 16),
                            z[0][2 * j + 1] - __uint_as_float(hi[j] & 0xFFFF0000u));
      }
      put_shared(hp + at / 4, hi[0] | static_cast<uint64_t>(hi[1]) << 32);
      put_shared(hp + (hsize + at) / 4, lo[0] | static_cast<uint64_t>(lo[1]) << 32);
    } else {
      // the four lanes of a token hold its block of 32
      uint32_t amax = 0;
#pragma unroll
      for (int x = 0; x < U; ++x)
#pragma unroll
        for (int j = 0; j < 4; ++j) amax = max(amax, __float_as_uint(z[x][j]) & 0x7FFFFFFFu);
      amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 16)));
      amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 32)));
      const int E = part_exponent(amax);
      if (hr < 0) return;
      uint32_t *hp = static_cast<uint32_t *>(a.h);
#pragma unroll
      for (int x = 0; x < U; ++x) {
        float v[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) v[j] = __builtin_ldexpf(z[x][j], -E);
#pragma unroll
        for (int p = 0; p < KD::PDN; ++p) put_shared(hp + (p * hsize + at + x * 16) / 4, take_part(v));
      }
      if (q == 0)
        put_shared(a.hs + at / 32, static_cast<uint8_t>(amax >= 0x7F800000u ? 255 : E + 127));
    }
  };
  // Units u0 .. u0+m-1; a wave group takes RU = ceil(m / groups) of them.
  auto up_pass = [&](auto units_each, int u0, int m) {
    constexpr int RU = decltype(units_each)::value, R = RU * U;
    const int group = wave / ks, kw = wave - group * ks, nch = d / KD::CH;
    const uint8_t *wb[kMaxTiles], *cb[kMaxTiles];
    uint32_t row[kMaxTiles];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      // past the range: its last unit again, not stored
      const int u = u0 + min(group * RU + r / U, m - 1), i = u / per_entry;
      const bool routed = i < ne;
      const int64_t e = routed ? uniform(s_list[i]) : i - ne;
      const int r0 = (u - i * per_entry) * U * 16 + r % U * 16 + col;
      wb[r] = static_cast<const uint8_t *>(routed ? a.w1 : a.ws1) + e * f * nch * KD::ABYTES;
      cb[r] = W == kWMx ? (routed ? a.c1 : a.cs1) + e * f * nch * 4 : nullptr;
      row[r] = static_cast<uint32_t>(r0) * nch;
    }
    // A column without a token repeats one: columns do not mix, and it is not
    // stored.  Loads under a condition could not be counted, and each wait
    // would be for all of them.
    uint32_t br = static_cast<uint32_t>(min(col, T - 1)) * nch;
    f32x4_t acc[R];
    walk(std::integral_constant<int, KD::PUP>{}, acc, static_cast<const uint8_t *>(a.x), a.xs,
         static_cast<int64_t>(T) * nch * KD::BBYTES, nch, wb, cb, row, br, 0, kw,
         max(0, (nch - kw + ks - 1) / ks), ks, [](int) {});
    if (ks == 1) {
#pragma unroll
      for (int x = 0; x < RU; ++x)
        if (group * RU + x < m) {
          f32x4_t z[U];
#pragma unroll
          for (int y = 0; y < U; ++y) z[y] = acc[x * U + y];
          hidden_out(u0 + group * RU + x, z);
        }
      return;
    }
#pragma unroll
    for (int r = 0; r < R; ++r) *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
    __syncthreads();
    for (int x = wave; x < m; x += kWaves) {
      const int gr = x / RU, rr = (x - gr * RU) * U;
      f32x4_t z[U];
#pragma unroll
      for (int y = 0; y < U; ++y) {
        z[y] = *reinterpret_cast<const f32x4_t *>(&s_red[gr * ks][rr + y][lane * 4]);
        for (int w = 1; w < ks; ++w)
          z[y] += *reinterpret_cast<const f32x4_t *>(&s_red[gr * ks + w][rr + y][lane * 4]);
      }
      hidden_out(u0 + x, z);
    }
    __syncthreads();
  };
  auto up_share = [&](int w) {
    int u = static_cast<int>(static_cast<int64_t>(units) * w / grid);
    const int end = static_cast<int>(static_cast<int64_t>(units) * (w + 1) / grid);
    const int groups = kWaves / ks, most = groups * (kMaxTiles / U);
    while (u < end) {
      // passes of equal length
      const int passes = (end - u + most - 1) / most, m = (end - u + passes - 1) / passes;
      const int each = (m + groups - 1) / groups;
      if (each == 1) up_pass(std::integral_constant<int, 1>{}, u, m);
      else if (each == 2) up_pass(std::integral_constant<int, 2>{}, u, m);
      if constexpr (U == 1) {
        if (each == 3) up_pass(std::integral_constant<int, 3>{}, u, m);
        else if (each == 4) up_pass(std::integral_constant<int, 4>{}, u, m);
      }
      u += m;
    }
    wait_stores();
    __syncthreads();
    if (tid == 0) put_shared(a.state + w, static_cast<uint32_t>(kDone));
  };
  if (s_claim) up_share(blockIdx.x);
  for (;;) {
    int free = kGrid;
    bool done = true;
    for (int w = tid; w < grid; w += kThreads) {
      const uint32_t v = get_shared(a.state + w);
      done = done && v == kDone;
      if (v == kFree) free = min(free, w);
    }
    if (free < kGrid) atomicMin(&s_free, free);
    if (__syncthreads_and(done)) break;
    const int w = s_free;
    __syncthreads();
    if (w < kGrid) {
      if (tid == 0) {
        s_claim = claim(w);
        s_free = kGrid;
      }
      __syncthreads();
      if (s_claim) up_share(w);
    } else {
      __builtin_amdgcn_s_sleep(4);
    }
  }
  if (tid == 0) __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
  __syncthreads();

  // ---- output rows ----
  constexpr int RB = 16 * kMaxTiles;
  const int n_down = (d + RB - 1) / RB * a.S;
  for (int item = blockIdx.x; item < n_down; item += grid) {
    // rows r0 .. r0+RB-1: part s of the (entry, hidden) chunks
    const int blk = item / a.S, s = item - blk * a.S, r0 = blk * RB;
    const int nch = f / KD::CH, total = entries * nch;
    const int c0 = static_cast<int>(static_cast<int64_t>(total) * s / a.S) + wave;
    const int c1 = static_cast<int>(static_cast<int64_t>(total) * (s + 1) / a.S);
    const int i0 = uniform(c0 / nch), n = max(0, (c1 - c0 + kWaves - 1) / kWaves);
    const uint8_t *wb[kMaxTiles], *cb[kMaxTiles];
    uint32_t row[kMaxTiles], br = 0;
#pragma unroll
    for (int r = 0; r < kMaxTiles; ++r) row[r] = static_cast<uint32_t>(min(r0 + r * 16 + col, d - 1)) * nch;
    // the entry's matrix, and the hidden row of each column: the row of zeros
    // for one without a token there
    auto enter = [&](int i) {
      if (i >= entries) return;
      const bool routed = i < ne;
      const int64_t e = routed ? uniform(s_list[i]) : i - ne;
      const uint8_t *w = static_cast<const uint8_t *>(routed ? a.w2 : a.ws2) + e * d * nch * KD::ABYTES;
      const uint8_t *c = W == kWMx ? (routed ? a.c2 : a.cs2) + e * d * nch * 4 : nullptr;
#pragma unroll
      for (int r = 0; r < kMaxTiles; ++r) {
        wb[r] = w;
        cb[r] = c;
      }
      const int hr = hidden_row(i, col);
      br = static_cast<uint32_t>(hr < 0 ? pairs : hr) * nch;
    };
    enter(i0);
    f32x4_t acc[kMaxTiles];
    walk(std::integral_constant<int, KD::PDN>{}, acc, static_cast<const uint8_t *>(a.h), a.hs,
         static_cast<int64_t>(pairs + 1) * nch * KD::BBYTES, nch, wb, cb, row, br, i0, c0 - i0 * nch, n,
         kWaves, enter);
#pragma unroll
    for (int r = 0; r < kMaxTiles; ++r)
      *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
    __syncthreads();
    // wave: tile r, as many as there are waves; lane: token col, rows 4q .. 4q+3
    static_assert(kMaxTiles == kWaves, "one tile per wave");
    const int orow = r0 + wave * 16 + q * 4;
    const bool out = col < T && orow < d;
    f32x4_t z = *reinterpret_cast<const f32x4_t *>(&s_red[0][wave][lane * 4]);
#pragma unroll
    for (int w = 1; w < kWaves; ++w) z += *reinterpret_cast<const f32x4_t *>(&s_red[w][wave][lane * 4]);
    bool finish = true;
    if (a.S > 1) {
      const int64_t at = static_cast<int64_t>(col) * d + orow, size = static_cast<int64_t>(T) * d;
      uint64_t *pp = reinterpret_cast<uint64_t *>(a.part);
      if (out)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          put_shared(pp + (s * size + at) / 2 + j,
                     __float_as_uint(z[2 * j]) | static_cast<uint64_t>(__float_as_uint(z[2 * j + 1])) << 32);
      wait_stores();
      __syncthreads();
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(a.arrived + blk, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      finish = s_last == static_cast<uint32_t>(a.S - 1);
      if (finish && out) {
        z = f32x4_t{0, 0, 0, 0};
        for (int k = 0; k < a.S; ++k)
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            const uint64_t v = get_shared(pp + (k * size + at) / 2 + j);
            z[2 * j] += __uint_as_float(static_cast<uint32_t>(v));
            z[2 * j + 1] += __uint_as_float(static_cast<uint32_t>(v >> 32));
          }
      }
    }
    if (finish && out) {
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        if (a.bs2)
          for (int i = 0; i < Ks; ++i)
            z[j] += act_f32(a.bs2, static_cast<int64_t>(i) * d + orow + j, Act{});
        if (a.b2)
          for (int k = 0; k < K; ++k) {
            const int e = s_idx[col * 64 + k];
            if ((s_mask[e] >> col) & 1)
              z[j] += s_gate[col * 64 + k] * act_f32(a.b2, static_cast<int64_t>(e) * d + orow + j, Act{});
          }
      }
      const int64_t at = static_cast<int64_t>(col) * d + orow;
      if constexpr (W == kWF32) {
        *reinterpret_cast<f32x4_t *>(static_cast<float *>(a.y) + at) = z;
      } else {
        uint2 o;
        o.x = pack_bf16x2(z[0], z[1]);
        o.y = pack_bf16x2(z[2], z[3]);
        *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.y) + at) = o;
      }
    }
    __syncthreads();
  }
}

// Parts that a row block of the second Linear is cut into along its reduction
// axis: as many as leave the least of the last round of items empty, a few
// percent of which a smaller number is worth.
int down_parts(int blocks) {
  int best = 1;
  double least = 1e30;
  for (int s = 1; s <= 16; ++s) {
    const int n = blocks * s, rounds = (n + kGrid - 1) / kGrid;
    const double cost = static_cast<double>(rounds) * kGrid / n * (1.0 + 0.005 * s);
    if (cost < least) {
      least = cost;
      best = s;
    }
  }
  return best;
}

constexpr int kDownRows = 16 * kMaxTiles;

struct FewWs {
  size_t logits, ctr, h, hs, x, xs, part, bytes;
  int parts, n_ctr;
};

FewWs few_ws(FewKind kind, int T, int d, int N, int K, int Ks, int f) {
  FewWs w;
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t o = at;
    at += (b + 255) & ~size_t(255);
    return o;
  };
  const int blocks = (d + kDownRows - 1) / kDownRows;
  const size_t rows = static_cast<size_t>(T) * (K + Ks) + 1;
  w.parts = down_parts(blocks);
  w.n_ctr = kGrid + blocks;
  w.logits = take(sizeof(float) * T * N);
  w.ctr = take(sizeof(uint32_t) * w.n_ctr);
  w.h = take((kind == kFewMxfp4 ? 3 : 4) * rows * f);
  w.hs = take(kind == kFewMxfp4 ? rows * (f / 32) : 0);
  w.x = take(kind == kFewMxfp4 ? static_cast<size_t>(2) * T * d : 0);
  w.xs = take(kind == kFewMxfp4 ? static_cast<size_t>(T) * (d / 32) : 0);
  w.part = take(w.parts > 1 ? sizeof(float) * w.parts * T * d : 0);
  w.bytes = at;
  return w;
}

}  // namespace

// One size for both calls of a shape (plain and MXFP4 weights).
size_t few_workspace_bytes(bool bf16, int T, int d, int N, int K, int Ks, int f) {
  if (!bf16) return few_ws(kFewF32, T, d, N, K, Ks, f).bytes;
  const size_t p = few_ws(kFewBf16, T, d, N, K, Ks, f).bytes;
  const size_t q = few_ws(kFewMxfp4, T, d, N, K, Ks, f).bytes;
  return p > q ? p : q;
}

hipError_t launch_few_layer(const FewLayer &p, void *ws, hipStream_t s) {
  const FewWs L = few_ws(p.kind, p.T, p.d, p.N, p.K, p.Ks, p.f);
  const bool mx = p.kind == kFewMxfp4;
  char *base = static_cast<char *>(ws);
  float *logits = reinterpret_cast<float *>(base + L.logits);
  uint32_t *ctr = reinterpret_cast<uint32_t *>(base + L.ctr);
  uint32_t *xq = mx ? reinterpret_cast<uint32_t *>(base + L.x) : nullptr;
  uint8_t *xs = reinterpret_cast<uint8_t *>(base + L.xs), *hs = reinterpret_cast<uint8_t *>(base + L.hs);
  // the row of zeros behind the hidden rows, in each part
  const size_t rows = static_cast<size_t>(p.T) * (p.K + p.Ks);
  FewZero zero{{ctr}, {L.n_ctr}};
  const int n_parts = mx ? 3 : p.kind == kFewBf16 ? 2 : 1, bytes = mx ? 1 : p.kind == kFewBf16 ? 2 : 4;
  for (int i = 0; i < n_parts; ++i) {
    zero.p[1 + i] = reinterpret_cast<uint32_t *>(base + L.h + ((i * (rows + 1) + rows) * p.f) * bytes);
    zero.n[1 + i] = p.f * bytes / 4;
  }
  if (mx) {
    zero.p[4] = reinterpret_cast<uint32_t *>(hs + rows * (p.f / 32));
    zero.n[4] = p.f / 128;
  }
  const float *in_logit = p.select_only ? nullptr : p.router_bias;
  const int split = mx ? (p.T * (p.d / 4) + kLogitThreads - 1) / kLogitThreads : 0;
  auto route = [&](auto x0, auto kernel) {
    using X = decltype(x0);
    hipLaunchKernelGGL(kernel, dim3(p.N + split), dim3(kLogitThreads), 0, s,
                       static_cast<const X *>(p.x), p.w_router, in_logit, logits, p.T, p.d, p.N, zero,
                       xq, xs);
  };
  auto route_t = [&](auto x0) {
    using X = decltype(x0);
    if (p.T <= 1) route(x0, few_logits_kernel<X, 1>);
    else if (p.T <= 2) route(x0, few_logits_kernel<X, 2>);
    else if (p.T <= 4) route(x0, few_logits_kernel<X, 4>);
    else if (p.T <= 8) route(x0, few_logits_kernel<X, 8>);
    else route(x0, few_logits_kernel<X, 16>);
  };
  if (p.kind == kFewF32) route_t(0.0f);
  else route_t(uint16_t{0});
  hipError_t e = hipGetLastError();
  if (e != hipSuccess) return e;
  FewArgs a;
  a.x = mx ? static_cast<const void *>(xq) : p.x;
  a.xs = xs;
  a.logits = logits;
  a.sel_bias = p.select_only ? p.router_bias : nullptr;
  a.w1 = p.w1; a.b1 = p.b1; a.w2 = p.w2; a.b2 = p.b2;
  a.ws1 = p.ws1; a.bs1 = p.bs1; a.ws2 = p.ws2; a.bs2 = p.bs2;
  a.c1 = p.c1; a.c2 = p.c2; a.cs1 = p.cs1; a.cs2 = p.cs2;
  a.h = base + L.h;
  a.hs = hs;
  a.part = reinterpret_cast<float *>(base + L.part);
  a.state = ctr;
  a.arrived = ctr + kGrid;
  a.y = p.y; a.idx = p.idx; a.gate = p.gate; a.counts = p.counts;
  a.T = p.T; a.d = p.d; a.N = p.N; a.K = p.K; a.Ks = p.Ks; a.f = p.f;
  a.S = L.parts;
  a.cap = p.cap;
  const int urows = mx ? 16 * Kind<kWMx>::UNIT : 16;
  const int64_t met = (p.T * p.K < p.N ? p.T * p.K : p.N) + p.Ks;
  const int64_t up = met * ((p.f + urows - 1) / urows), down = static_cast<int64_t>((p.d + kDownRows - 1) / kDownRows) * L.parts;
  const int64_t items = up > down ? up : down;
  const dim3 grid(static_cast<unsigned>(items < kGrid ? items : kGrid));
  if (p.kind == kFewF32) hipLaunchKernelGGL(few_layer_kernel<kWF32>, grid, dim3(kThreads), 0, s, a);
  else if (p.kind == kFewBf16) hipLaunchKernelGGL(few_layer_kernel<kWBf16>, grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL(few_layer_kernel<kWMx>, grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
