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
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

enum : uint32_t { kFree = 0, kTaken = 1, kDone = 2 };   // states of an up share
constexpr int kTok = 16;            // columns of the matrix instruction
constexpr int kWaves = 8;
constexpr int kThreads = kWaves * 64;

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

// One workgroup per expert: thread i sums elements 4i, 4i + 4096, ... of
// W_e . x_t for each token, then the wave and the sixteen waves are added in a
// fixed tree.  TT is T rounded up to a power of two (the loads of a step are
// issued together); columns past T repeat the last token and are not stored.
constexpr int kLogitThreads = 1024;
struct FewZero {   // words to clear for kernel 2
  uint32_t *p[3];
  int n[3];
};
template <typename T, int TT>
__global__ __launch_bounds__(kLogitThreads) void few_logits_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    float *__restrict__ logits, int tokens, int d, int N, FewZero zero) {
  constexpr int NW = kLogitThreads / 64;
  __shared__ float s_part[NW][TT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x;
#pragma unroll
  for (int r = 0; r < 3; ++r)
    for (int i = e * kLogitThreads + tid; i < zero.n[r]; i += N * kLogitThreads) zero.p[r][i] = 0;
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
  const void *x;
  const float *logits, *sel_bias;
  const void *w1, *b1, *w2, *b2, *ws1, *bs1, *ws2, *bs2;
  const uint8_t *c1, *c2, *cs1, *cs2;   // scale bytes of MXFP4 weights
  void *h;                               // hidden rows and one of zeros: float, or bf16 parts [2][rows + 1][f]
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

// The three kinds of weights.  CH elements of the reduction axis make a chunk:
// what the four lanes of a row load together.  A row's chunk is read in NA
// pieces of 64 neighbouring bytes, 16 to a lane; lane q finds the activations
// that belong to its piece j at byte q * BLANE + j * BSTEP of theirs.
enum { kWF32, kWBf16, kWMx };
template <int W> struct Kind;
template <> struct Kind<kWF32> {
  using Act = float;
  static constexpr int CH = 16, NA = 1, NB = 1, ABYTES = 64, BBYTES = 64, BLANE = 16, BSTEP = 64;
};
template <> struct Kind<kWBf16> {
  using Act = uint16_t;
  static constexpr int CH = 64, NA = 2, NB = 2, ABYTES = 128, BBYTES = 128, BLANE = 16, BSTEP = 64;
};
template <> struct Kind<kWMx> {
  using Act = uint16_t;
  static constexpr int CH = 128, NA = 1, NB = 4, ABYTES = 64, BBYTES = 256, BLANE = 64, BSTEP = 16;
};

template <int W> struct AFrag {
  u32x4_t v[Kind<W>::NA];
  uint32_t s;
};
template <int W> struct BFrag {
  u32x4_t v[Kind<W>::NB];
};

// Part of chunk c of this lane's row: row is the row's (and the lane's) byte
// offset from the matrix, which lies at a wave-uniform address.
template <int W>
__device__ __forceinline__ void load_a(AFrag<W> &a, const uint8_t *base, uint32_t row, int c) {
#pragma unroll
  for (int j = 0; j < Kind<W>::NA; ++j)
    a.v[j] = *reinterpret_cast<const u32x4_t *>(
        base + (row + static_cast<uint32_t>(c) * Kind<W>::ABYTES + j * 64));
}
template <int W>
__device__ __forceinline__ void load_b(BFrag<W> &b, const uint8_t *base, uint32_t row, int c) {
#pragma unroll
  for (int j = 0; j < Kind<W>::NB; ++j)
    b.v[j] = *reinterpret_cast<const u32x4_t *>(
        base + (row + static_cast<uint32_t>(c) * Kind<W>::BBYTES + j * Kind<W>::BSTEP));
}

// Eight E2M1 codes times the block's power of two, as bf16 (exact).
__device__ __forceinline__ bf16x8_t widen_mx(uint32_t c, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

// Chunks in flight per wave.
template <int W> constexpr int kDepth = 2;

// acc += A (B0 + B1), 16 weight rows x 16 columns.
template <int W, bool TWO>
__device__ __forceinline__ void mma(f32x4_t &acc, const AFrag<W> &a, const BFrag<W> &b0,
                                    const BFrag<W> &b1) {
  if constexpr (W == kWF32) {
#pragma unroll
    for (int j = 0; j < 4; ++j)
      acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[0][j]),
                                                 __uint_as_float(b0.v[0][j]), acc, 0, 0, 0);
  } else if constexpr (W == kWBf16) {
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      const bf16x8_t av = __builtin_bit_cast(bf16x8_t, a.v[j]);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, b0.v[j]), acc,
                                                    0, 0, 0);
      if constexpr (TWO)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, b1.v[j]),
                                                      acc, 0, 0, 0);
    }
  } else {
    const float sc = __uint_as_float(a.s << 23);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const bf16x8_t av = widen_mx(a.v[0][j], sc);
      acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, b0.v[j]), acc,
                                                    0, 0, 0);
      if constexpr (TWO)
        acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(av, __builtin_bit_cast(bf16x8_t, b1.v[j]),
                                                      acc, 0, 0, 0);
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
__device__ __forceinline__ void put_shared(uint32_t *p, uint32_t v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ __forceinline__ float get_shared(const float *p) {
  return __uint_as_float(__hip_atomic_load(reinterpret_cast<const uint32_t *>(p), __ATOMIC_RELAXED,
                                           __HIP_MEMORY_SCOPE_AGENT));
}
// This wave's device-scope stores have arrived.
__device__ __forceinline__ void wait_stores() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

__device__ __forceinline__ float act_f32(const void *p, int64_t i, float) {
  return static_cast<const float *>(p)[i];
}
__device__ __forceinline__ float act_f32(const void *p, int64_t i, uint16_t) {
  return bf16_to_f32(static_cast<const uint16_t *>(p)[i]);
}

template <int W, int R>
__global__ __launch_bounds__(kThreads, 4) void few_layer_kernel(FewArgs a) {
  using KD = Kind<W>;
  using Act = typename KD::Act;
  constexpr bool TWO = W != kWF32;
  constexpr int RB = 16 * R;
  __shared__ int16_t s_pair[kMaxRouted * kTok];    // hidden row of (entry, token), or -1
  __shared__ int16_t s_list[kMaxRouted];           // expert of each entry
  __shared__ alignas(4) uint16_t s_mask[kMaxRouted];   // tokens of each expert
  __shared__ float s_gate[kTok * 64];
  __shared__ int16_t s_idx[kTok * 64];
  __shared__ float s_red[kWaves][R][256];
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
  if (tid == 0) {
    s_claim = claim(blockIdx.x);
    s_free = kThreads;
  }
  for (int e = tid; e < N; e += kThreads) s_mask[e] = 0;
  for (int t = wave; t < T; t += kWaves) {
    uint32_t key[kMaxRouted / 64];
#pragma unroll
    for (int j = 0; j < kMaxRouted / 64; ++j) {
      if (j * 64 >= N) break;
      const int e = j * 64 + lane;
      key[j] = 0;
      if (e < N) {
        float v = a.logits[static_cast<int64_t>(t) * N + e];
        if (a.sel_bias) v += a.sel_bias[e];
        key[j] = max(order_key(v), 1u);
      }
    }
    float mine = 0.0f;
    int mine_e = 0;
    for (int k = 0; k < K; ++k) {
      // this lane's best, the wave's, and the lowest id among equals
      uint32_t best = 0;
      int at = lane;
#pragma unroll
      for (int j = 0; j < kMaxRouted / 64; ++j) {
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
#pragma unroll
      for (int j = 0; j < kMaxRouted / 64; ++j) {
        if (j * 64 >= N) break;
        if (e == j * 64 + lane) key[j] = 0;
      }
      if (lane == k) mine_e = e;
    }
    if (lane < K) mine = a.logits[static_cast<int64_t>(t) * N + mine_e];
    float top = lane < K ? mine : -__builtin_inff();
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
  __syncthreads();
  // token masks: thread (t, k) pairs, one token at a time per 64 threads
  for (int i = tid; i < T * 64; i += kThreads)
    if ((i & 63) < K) {
      const int e = s_idx[i];
      atomicOr(reinterpret_cast<uint32_t *>(s_mask) + (e >> 1), (1u << (i >> 6)) << ((e & 1) * 16));
    }
  __syncthreads();
  // an expert keeps its first cap tokens
  for (int e = tid; e < N; e += kThreads) {
    uint32_t m = s_mask[e], kept = 0;
    for (int c = 0; c < a.cap && m; ++c) {
      kept |= m & (0u - m);
      m &= m - 1;
    }
    s_mask[e] = static_cast<uint16_t>(kept);
    if (blockIdx.x == 0 && a.counts) a.counts[e] = __popc(kept);
  }
  __syncthreads();
  // met experts, in order
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

  // ---- items ----
  const int fblk = (f + RB - 1) / RB, dblk = (d + RB - 1) / RB;
  const int n_up = entries * fblk, n_down = dblk * a.S;
  const int col = lane & 15, q = lane >> 4;
  const int64_t pairs = static_cast<int64_t>(T) * K + static_cast<int64_t>(Ks) * T;
  // hidden row of (entry, token): routed pairs first, then the shared experts
  auto hidden_row = [&](int i, int t) -> int {
    if (i < ne) return s_pair[i * kTok + t];
    return t < T ? T * K + (i - ne) * T + t : -1;
  };

  // Sum over every kWaves-th of the chunks from chunk cc of entry i on, n of
  // them, running on into the next entries: 16 R rows from r0 of the Linear `up`, against x or the hidden rows.
  auto walk = [&](auto is_up, int i, int cc, int n, int r0, f32x4_t (&acc)[R]) {
    constexpr bool UP = decltype(is_up)::value;
    constexpr bool B2 = TWO && !UP;
    constexpr int D = kDepth<W>;
    const int rows = UP ? f : d, nch = (UP ? d : f) / KD::CH;
    const uint8_t *rw = static_cast<const uint8_t *>(UP ? a.w1 : a.w2);
    const uint8_t *sw = static_cast<const uint8_t *>(UP ? a.ws1 : a.ws2);
    const uint8_t *rc = UP ? a.c1 : a.c2, *sc = UP ? a.cs1 : a.cs2;
    const uint8_t *bb = static_cast<const uint8_t *>(UP ? a.x : a.h);
    const int64_t msize = static_cast<int64_t>(rows) * nch;       // chunks of a matrix
    uint32_t row[R];
#pragma unroll
    for (int r = 0; r < R; ++r) row[r] = static_cast<uint32_t>(min(r0 + r * 16 + col, rows - 1)) * nch;
    const uint8_t *wb = nullptr, *cb = nullptr;
    uint32_t bo = 0;
    auto enter = [&]() {
      const bool routed = i < ne;
      const int64_t e = routed ? uniform(s_list[i]) : i - ne;
      wb = (routed ? rw : sw) + e * msize * KD::ABYTES;
      if constexpr (W == kWMx) cb = (routed ? rc : sc) + e * msize * 4;
      // Every lane loads (loads under a condition cannot be counted, and each
      // wait would be for all of them).  An up item's column without a token
      // repeats some token: columns do not mix, and it is not stored.  In a
      // down item it takes the row of zeros, since the sum runs over entries.
      int br = UP ? min(col, T - 1) : hidden_row(i, col);
      if (br < 0) br = static_cast<int>(pairs);
      bo = static_cast<uint32_t>(br) * nch * KD::BBYTES + q * KD::BLANE;
    };
    enter();
    struct Stage {
      AFrag<W> a[R];
      BFrag<W> b0, b1;
    } st[D];
    auto fetch = [&](Stage &s) {
      load_b<W>(s.b0, bb, bo, cc);
      if constexpr (B2) load_b<W>(s.b1, bb + (pairs + 1) * f * 2, bo, cc);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        load_a<W>(s.a[r], wb, row[r] * KD::ABYTES + q * 16, cc);
        if constexpr (W == kWMx) s.a[r].s = cb[row[r] * 4 + q + cc * 4];
      }
      cc += kWaves;
      if (cc >= nch) {
        do {
          cc -= nch;
          ++i;
        } while (cc >= nch);
        if (i < entries) enter();
      }
    };
    auto use = [&](Stage &s) {
#pragma unroll
      for (int r = 0; r < R; ++r) mma<W, B2>(acc[r], s.a[r], s.b0, s.b1);
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
  // sum of the eight waves' parts of (row rl, token t)
  auto sum_waves = [&](int rl, int t) {
    const int r16 = rl & 15, at = ((r16 >> 2) * 16 + t) * 4 + (r16 & 3);
    float z = 0.0f;
#pragma unroll
    for (int w = 0; w < kWaves; ++w) z += s_red[w][rl >> 4][at];
    return z;
  };

  // ---- hidden rows: the share of workgroup w ----
  const int grid = gridDim.x;
  auto up_share = [&](int w) {
    for (int item = w; item < n_up; item += grid) {
      f32x4_t acc[R];
#pragma unroll
      for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
      // hidden rows r0 .. r0+RB-1 of entry i, for its tokens
      const int i = item / fblk, r0 = (item - i * fblk) * RB, nch = d / KD::CH;
      // the waves take neighbouring chunks, so that a row is read in long pieces
      if (wave < nch) walk(std::true_type{}, i, wave, (nch - wave + kWaves - 1) / kWaves, r0, acc);
#pragma unroll
      for (int r = 0; r < R; ++r)
        *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
      __syncthreads();
      const bool routed = i < ne;
      const int64_t e = routed ? s_list[i] : i - ne;
      const void *bias = routed ? a.b1 : a.bs1;
      // thread: token t, two neighbouring rows
      for (int o = tid; o < kTok * RB / 2; o += kThreads) {
        const int t = o / (RB / 2), rl = o % (RB / 2) * 2, row = r0 + rl;
        const int hr = hidden_row(i, t);
        if (hr < 0 || row >= f) continue;
        const float g = routed ? s_gate[t * 64 + (hr - t * K)] : 1.0f;
        float v[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          float z = sum_waves(rl + j, t);
          if (bias) z += act_f32(bias, e * f + row + j, Act{});
          v[j] = g * silu(z);
        }
        const int64_t at_h = static_cast<int64_t>(hr) * f + row;
        if constexpr (TWO) {
          uint32_t *hp = static_cast<uint32_t *>(a.h);
          const uint32_t hi = pack_bf16x2(v[0], v[1]);
          put_shared(hp + at_h / 2, hi);
          put_shared(hp + ((pairs + 1) * f + at_h) / 2,
                     pack_bf16x2(v[0] - __uint_as_float(hi << 16),
                                 v[1] - __uint_as_float(hi & 0xFFFF0000u)));
        } else {
          put_shared(static_cast<uint32_t *>(a.h) + at_h, __float_as_uint(v[0]));
          put_shared(static_cast<uint32_t *>(a.h) + at_h + 1, __float_as_uint(v[1]));
        }
      }
      __syncthreads();
    }
    wait_stores();
    __syncthreads();
    if (tid == 0) put_shared(a.state + w, kDone);
  };
  if (s_claim) up_share(blockIdx.x);
  for (;;) {
    uint32_t v = kDone;
    if (tid < grid) v = __hip_atomic_load(a.state + tid, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
    if (v == kFree) atomicMin(&s_free, tid);
    if (__syncthreads_and(v == kDone)) break;
    const int w = s_free;
    __syncthreads();
    if (w < kThreads) {
      if (tid == 0) {
        s_claim = claim(w);
        s_free = kThreads;
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
  for (int item = blockIdx.x; item < n_down; item += grid) {
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    // output rows r0 .. r0+RB-1: part s of the (entry, hidden) chunks
    const int blk = item / a.S, s = item - blk * a.S, r0 = blk * RB;
    const int nch = f / KD::CH, total = entries * nch;
    const int c0 = static_cast<int>(static_cast<int64_t>(total) * s / a.S) + wave;
    const int c1 = static_cast<int>(static_cast<int64_t>(total) * (s + 1) / a.S);
    if (c0 < c1) {
      const int i = uniform(c0 / nch);
      walk(std::false_type{}, i, c0 - i * nch, (c1 - c0 + kWaves - 1) / kWaves, r0, acc);
    }
#pragma unroll
    for (int r = 0; r < R; ++r)
      *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
    __syncthreads();
    bool finish = a.S == 1;
    if (a.S > 1) {
      for (int o = tid; o < T * RB; o += kThreads) {
        const int t = o / RB, rl = o % RB;
        if (r0 + rl < d)
          put_shared(reinterpret_cast<uint32_t *>(a.part) + (static_cast<int64_t>(s) * T + t) * d + r0 + rl,
                     __float_as_uint(sum_waves(rl, t)));
      }
      wait_stores();
      __syncthreads();
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(a.arrived + blk, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      finish = s_last == static_cast<uint32_t>(a.S - 1);
    }
    if (finish) {
      for (int o = tid; o < T * RB; o += kThreads) {
        const int t = o / RB, rl = o % RB, row = r0 + rl;
        if (row >= d) continue;
        float z = 0.0f;
        if (a.S == 1) z = sum_waves(rl, t);
        else
          for (int k = 0; k < a.S; ++k) z += get_shared(a.part + (static_cast<int64_t>(k) * T + t) * d + row);
        if (a.bs2)
          for (int i = 0; i < Ks; ++i) z += act_f32(a.bs2, static_cast<int64_t>(i) * d + row, Act{});
        if (a.b2)
          for (int k = 0; k < K; ++k) {
            const int e = s_idx[t * 64 + k];
            if ((s_mask[e] >> t) & 1)
              z += s_gate[t * 64 + k] * act_f32(a.b2, static_cast<int64_t>(e) * d + row, Act{});
          }
        const int64_t at_y = static_cast<int64_t>(t) * d + row;
        if constexpr (TWO) static_cast<uint16_t *>(a.y)[at_y] = f32_to_bf16(z);
        else static_cast<float *>(a.y)[at_y] = z;
      }
    }
    __syncthreads();
  }
}

// Parts that a row block of the second Linear is cut into along its reduction
// axis, so that there are enough items for the chip.
int down_parts(int d, int rb) {
  const int blocks = (d + rb - 1) / rb;
  int s = 1;
  while (blocks * s < 512 && s < 16) s *= 2;
  return s;
}

constexpr int kRows = 2;   // 16-row tiles of an item
constexpr int kGrid = 512;   // most workgroups: two per CU
static_assert(kGrid <= kThreads, "one state per thread where they are looked through");

struct FewWs {
  size_t logits, ctr, h, part, bytes;
  int parts, n_ctr;
};

FewWs few_ws(int T, int d, int N, int K, int Ks, int f) {
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  FewWs w;
  w.parts = down_parts(d, 16 * kRows);
  w.n_ctr = kGrid + (d + 16 * kRows - 1) / (16 * kRows);
  size_t at = 0;
  w.logits = at;
  at += up(sizeof(float) * T * N);
  w.ctr = at;
  at += up(sizeof(uint32_t) * w.n_ctr);
  w.h = at;
  at += up(sizeof(float) * (static_cast<size_t>(T) * K + static_cast<size_t>(Ks) * T + 1) * f);
  w.part = at;
  at += w.parts > 1 ? up(sizeof(float) * w.parts * T * d) : 0;
  w.bytes = at;
  return w;
}

}  // namespace

size_t few_workspace_bytes(int T, int d, int N, int K, int Ks, int f) {
  return few_ws(T, d, N, K, Ks, f).bytes;
}

hipError_t launch_few_layer(const FewLayer &p, void *ws, hipStream_t s) {
  const FewWs L = few_ws(p.T, p.d, p.N, p.K, p.Ks, p.f);
  char *base = static_cast<char *>(ws);
  float *logits = reinterpret_cast<float *>(base + L.logits);
  uint32_t *ctr = reinterpret_cast<uint32_t *>(base + L.ctr);
  // the row of zeros behind the hidden rows, of both parts where there are two
  const int64_t pairs = static_cast<int64_t>(p.T) * (p.K + p.Ks);
  uint32_t *h = reinterpret_cast<uint32_t *>(base + L.h);
  FewZero zero{{ctr, nullptr, nullptr}, {L.n_ctr, 0, 0}};
  if (p.kind == kFewF32) {
    zero.p[1] = h + pairs * p.f;
    zero.n[1] = p.f;
  } else {
    zero.p[1] = h + pairs * p.f / 2;
    zero.p[2] = h + (2 * pairs + 1) * p.f / 2;
    zero.n[1] = zero.n[2] = p.f / 2;
  }
  const float *in_logit = p.select_only ? nullptr : p.router_bias;
  auto route = [&](auto x0, auto kernel) {
    using X = decltype(x0);
    hipLaunchKernelGGL(kernel, dim3(p.N), dim3(kLogitThreads), 0, s, static_cast<const X *>(p.x),
                       p.w_router, in_logit, logits, p.T, p.d, p.N, zero);
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
  a.x = p.x;
  a.logits = logits;
  a.sel_bias = p.select_only ? p.router_bias : nullptr;
  a.w1 = p.w1; a.b1 = p.b1; a.w2 = p.w2; a.b2 = p.b2;
  a.ws1 = p.ws1; a.bs1 = p.bs1; a.ws2 = p.ws2; a.bs2 = p.bs2;
  a.c1 = p.c1; a.c2 = p.c2; a.cs1 = p.cs1; a.cs2 = p.cs2;
  a.h = base + L.h;
  a.part = reinterpret_cast<float *>(base + L.part);
  a.state = ctr;
  a.arrived = ctr + kGrid;
  a.y = p.y; a.idx = p.idx; a.gate = p.gate; a.counts = p.counts;
  a.T = p.T; a.d = p.d; a.N = p.N; a.K = p.K; a.Ks = p.Ks; a.f = p.f;
  a.S = L.parts;
  a.cap = p.cap;
  const int rb = 16 * kRows;
  const int64_t met = (p.T * p.K < p.N ? p.T * p.K : p.N) + p.Ks;
  const int64_t up = met * ((p.f + rb - 1) / rb), down = static_cast<int64_t>((p.d + rb - 1) / rb) * L.parts;
  const int64_t items = up > down ? up : down;
  const dim3 grid(static_cast<unsigned>(items < kGrid ? items : kGrid));
  if (p.kind == kFewF32)
    hipLaunchKernelGGL((few_layer_kernel<kWF32, kRows>), grid, dim3(kThreads), 0, s, a);
  else if (p.kind == kFewBf16)
    hipLaunchKernelGGL((few_layer_kernel<kWBf16, kRows>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((few_layer_kernel<kWMx, kRows>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
