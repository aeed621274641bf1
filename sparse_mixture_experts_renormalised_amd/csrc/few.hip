// The whole layer for 1 to 16 tokens in two kernels ([DSMoE] output equation
// with the routing of [TopK] and the capacity limit of [TopK] 解決策2).
//
// With so few tokens the layer is one pass over the weights of the experts
// the tokens meet, and the rest is latency.  The general path starts seven or
// more kernels and keeps per-expert row lists in memory; here
//
//   kernel 1 (few_logits_kernel) computes the router's logits, one workgroup
//     per expert, and clears the counters that kernel 2 uses;
//   kernel 2 (few_layer_kernel) does the rest.  Every workgroup repeats the
//     top-K selection, gates and capacity from the logits (T * N numbers)
//     into LDS, and then takes work items in order from one counter: first
//     the hidden rows of every met or shared expert (up items), then the
//     output rows (down items).
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
// Waiting.  A down item needs every hidden row, so it waits until the count of
// finished up items is complete.  Items are taken in counter order, so an up
// item belongs to a workgroup that is already running, and no workgroup waits
// while it holds an unfinished up item (the item fetched ahead has a higher
// number than the one in work): every wait ends, whatever the number of
// resident workgroups and whatever else runs on the device.
//
// Results do not depend on timing: sums are split in a way fixed by the sizes
// and joined in a fixed order.
#include "moe_common.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef __bf16 bf16x2_t __attribute__((ext_vector_type(2)));

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

// One workgroup per expert: thread i sums elements 4i, 4i + 1024, ... of
// W_e . x_t for each token, then the wave and the four waves are added in a
// fixed tree.
template <typename T>
__global__ __launch_bounds__(256) void few_logits_kernel(const T *__restrict__ x,
                                                         const float *__restrict__ w,
                                                         const float *__restrict__ bias,
                                                         float *__restrict__ logits, int tokens,
                                                         int d, int N, uint32_t *ctr, int n_ctr) {
  __shared__ float s_part[4][kTok];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x;
  if (e == 0)
    for (int i = tid; i < n_ctr; i += 256) ctr[i] = 0;
  const float *wr = w + static_cast<int64_t>(e) * d;
  float acc[kTok];
#pragma unroll
  for (int t = 0; t < kTok; ++t) acc[t] = 0.0f;
  for (int k = tid * 4; k < d; k += 1024) {
    const float4 wv = load4<float>(wr + k);
#pragma unroll
    for (int t = 0; t < kTok; ++t) {
      if (t >= tokens) break;
      const float4 xv = load4<T>(x + static_cast<int64_t>(t) * d + k);
      acc[t] = __builtin_fmaf(wv.x, xv.x, acc[t]);
      acc[t] = __builtin_fmaf(wv.y, xv.y, acc[t]);
      acc[t] = __builtin_fmaf(wv.z, xv.z, acc[t]);
      acc[t] = __builtin_fmaf(wv.w, xv.w, acc[t]);
    }
  }
#pragma unroll
  for (int t = 0; t < kTok; ++t) {
    if (t >= tokens) break;
#pragma unroll
    for (int off = 32; off >= 1; off >>= 1) acc[t] += __shfl_xor(acc[t], off);
    if (lane == 0) s_part[wave][t] = acc[t];
  }
  __syncthreads();
  if (tid < tokens) {
    float v = (s_part[0][tid] + s_part[1][tid]) + (s_part[2][tid] + s_part[3][tid]);
    if (bias) v += bias[e];
    logits[static_cast<int64_t>(tid) * N + e] = v;
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
  void *h;                               // hidden rows: float, or bf16 parts [2][rows][f]
  float *part;                           // [S][T][d] parts of split outputs
  uint32_t *ctr;                         // ticket, finished up items, arrivals per row block
  void *y;
  int32_t *idx;
  float *gate;
  int32_t *counts;
  int T, d, N, K, Ks, f, S;
  int cap;                               // rows an expert keeps (T or more: no limit)
};

// The three kinds of weights.  CH elements of the reduction axis make a chunk:
// what the four lanes of a row load together.  A lane's A part lies at byte
// lane_a() of the row's chunk, and the activations that belong to it
// at byte lane_b() of theirs.
enum { kWF32, kWBf16, kWMx };
template <int W> struct Kind;
template <> struct Kind<kWF32> {
  using Act = float;
  static constexpr int CH = 16, NA = 1, NB = 1, ABYTES = 64, BBYTES = 64;
};
template <> struct Kind<kWBf16> {
  using Act = uint16_t;
  static constexpr int CH = 64, NA = 2, NB = 2, ABYTES = 128, BBYTES = 128;
};
template <> struct Kind<kWMx> {
  using Act = uint16_t;
  static constexpr int CH = 128, NA = 1, NB = 4, ABYTES = 64, BBYTES = 256;
};

template <int W> struct AFrag {
  u32x4_t v[Kind<W>::NA];
  uint32_t s;
};
template <int W> struct BFrag {
  u32x4_t v[Kind<W>::NB];
};

template <int W>
__device__ __forceinline__ void load_a(AFrag<W> &a, const uint8_t *p, const uint8_t *sp, int c) {
#pragma unroll
  for (int j = 0; j < Kind<W>::NA; ++j)
    a.v[j] = __builtin_nontemporal_load(
        reinterpret_cast<const u32x4_t *>(p + static_cast<int64_t>(c) * Kind<W>::ABYTES) + j);
  if constexpr (W == kWMx) a.s = sp[c * 4];
}
template <int W>
__device__ __forceinline__ void load_b(BFrag<W> &b, const uint8_t *p, bool live, int c) {
#pragma unroll
  for (int j = 0; j < Kind<W>::NB; ++j) {
    b.v[j] = u32x4_t{0, 0, 0, 0};
    if (live)
      b.v[j] = *(reinterpret_cast<const u32x4_t *>(p + static_cast<int64_t>(c) * Kind<W>::BBYTES) + j);
  }
}

// Eight E2M1 codes times the block's power of two, as bf16 (exact).
__device__ __forceinline__ bf16x8_t widen_mx(uint32_t c, float scale) {
  const bf16x2_t a = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 0);
  const bf16x2_t b = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 1);
  const bf16x2_t d = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 2);
  const bf16x2_t e = __builtin_amdgcn_cvt_scalef32_pk_bf16_fp4(c, scale, 3);
  return bf16x8_t{a[0], a[1], b[0], b[1], d[0], d[1], e[0], e[1]};
}

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
  __shared__ uint32_t s_ticket, s_last;
  __shared__ int s_ne;
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int T = a.T, K = a.K, N = a.N, Ks = a.Ks, d = a.d, f = a.f;

  // ---- routing ----
  if (tid == 0) s_ticket = atomicAdd(a.ctr, 1u);
  for (int e = tid; e < N; e += kThreads) s_mask[e] = 0;
  for (int t = wave; t < T; t += kWaves) {
    uint32_t key[kMaxRouted / 64];
#pragma unroll
    for (int j = 0; j < kMaxRouted / 64; ++j) {
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
      uint64_t best = 0;
#pragma unroll
      for (int j = 0; j < kMaxRouted / 64; ++j) {
        const uint64_t c = (static_cast<uint64_t>(key[j]) << 32) | (0xFFFFFFFFu - (j * 64 + lane));
        if (key[j] != 0 && c > best) best = c;
      }
#pragma unroll
      for (int off = 32; off >= 1; off >>= 1) {
        const uint64_t o = __shfl_xor(static_cast<unsigned long long>(best), off);
        if (o > best) best = o;
      }
      const int e = static_cast<int>(0xFFFFFFFFu - static_cast<uint32_t>(best));
#pragma unroll
      for (int j = 0; j < kMaxRouted / 64; ++j)
        if (e == j * 64 + lane) key[j] = 0;
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
  const uint32_t n_up = static_cast<uint32_t>(entries) * fblk;
  const uint32_t n_all = n_up + static_cast<uint32_t>(dblk) * a.S;
  const int col = lane & 15, q = lane >> 4;
  const int64_t pairs = static_cast<int64_t>(T) * K + static_cast<int64_t>(Ks) * T;
  // hidden row of (entry, token): routed pairs first, then the shared experts
  auto hidden_row = [&](int i, int t) -> int {
    if (i < ne) return s_pair[i * kTok + t];
    return t < T ? T * K + (i - ne) * T + t : -1;
  };
  bool waited = false;
  uint32_t item = s_ticket;
  while (item < n_all) {
    uint32_t next = 0;
    if (tid == 0) next = atomicAdd(a.ctr, 1u);
    f32x4_t acc[R];
#pragma unroll
    for (int r = 0; r < R; ++r) acc[r] = f32x4_t{0, 0, 0, 0};
    if (item < n_up) {
      // hidden rows r0 .. r0+RB-1 of entry i, for its tokens
      const int i = item / fblk, r0 = (item - i * fblk) * RB;
      const bool routed = i < ne;
      const int64_t e = routed ? s_list[i] : i - ne;
      const uint8_t *wb = static_cast<const uint8_t *>(routed ? a.w1 : a.ws1);
      const uint8_t *sb = routed ? a.c1 : a.cs1;
      const int nch = d / KD::CH;
      const uint8_t *wp[R], *sp[R];
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const int64_t row = e * f + min(r0 + r * 16 + col, f - 1);
        wp[r] = wb + row * nch * KD::ABYTES + q * (KD::NA * 16);
        sp[r] = W == kWMx ? sb + row * nch * 4 + q : nullptr;
      }
      const bool live = hidden_row(i, col) >= 0;
      const uint8_t *xp = static_cast<const uint8_t *>(a.x) +
                          static_cast<int64_t>(live ? col : 0) * nch * KD::BBYTES + q * (KD::NB * 16);
      for (int c = wave; c < nch; c += kWaves) {
        AFrag<W> fa[R];
        BFrag<W> fb;
        load_b<W>(fb, xp, live, c);
#pragma unroll
        for (int r = 0; r < R; ++r) load_a<W>(fa[r], wp[r], sp[r], c);
#pragma unroll
        for (int r = 0; r < R; ++r) mma<W, false>(acc[r], fa[r], fb, fb);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
      __syncthreads();
      // thread: token t, row rl of the item
      for (int o = tid; o < kTok * RB; o += kThreads) {
        const int t = o / RB, rl = o % RB, r16 = rl & 15;
        const int at = ((r16 >> 2) * 16 + t) * 4 + (r16 & 3);
        float z = 0.0f;
#pragma unroll
        for (int w = 0; w < kWaves; ++w) z += s_red[w][rl >> 4][at];
        const int hr = hidden_row(i, t), row = r0 + rl;
        if (hr >= 0 && row < f) {
          const void *b = routed ? a.b1 : a.bs1;
          if (b) z += act_f32(b, e * f + row, Act{});
          float g = 1.0f;
          if (routed) g = s_gate[t * 64 + (hr - t * K)];
          const float v = g * silu(z);
          const int64_t at_h = static_cast<int64_t>(hr) * f + row;
          if constexpr (TWO) {
            uint16_t *hp = static_cast<uint16_t *>(a.h);
            const uint16_t hi = f32_to_bf16(v);
            hp[at_h] = hi;
            hp[pairs * f + at_h] = f32_to_bf16(v - bf16_to_f32(hi));
          } else {
            static_cast<float *>(a.h)[at_h] = v;
          }
        }
      }
      __syncthreads();
      if (tid == 0)
        __hip_atomic_fetch_add(a.ctr + 1, 1u, __ATOMIC_RELEASE, __HIP_MEMORY_SCOPE_AGENT);
    } else {
      // output rows r0 .. r0+RB-1: part s of the (entry, hidden) chunks
      const int j = item - n_up, blk = j / a.S, s = j - blk * a.S, r0 = blk * RB;
      const int nch = f / KD::CH;
      const int total = entries * nch;
      const int c_end = static_cast<int>(static_cast<int64_t>(total) * (s + 1) / a.S);
      int c = static_cast<int>(static_cast<int64_t>(total) * s / a.S) + wave;
      if (!waited) {
        if (tid == 0) {
          while (__hip_atomic_load(a.ctr + 1, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) < n_up)
            __builtin_amdgcn_s_sleep(2);
          __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "agent");
        }
        __syncthreads();
        waited = true;
      }
      for (; c < c_end; c += kWaves) {
        const int i = c / nch, cc = c - i * nch;
        const bool routed = i < ne;
        const int64_t e = routed ? s_list[i] : i - ne;
        const uint8_t *wb = static_cast<const uint8_t *>(routed ? a.w2 : a.ws2);
        const uint8_t *sb = routed ? a.c2 : a.cs2;
        const int hr = hidden_row(i, col);
        const uint8_t *hp = static_cast<const uint8_t *>(a.h) +
                            static_cast<int64_t>(max(hr, 0)) * nch * KD::BBYTES + q * (KD::NB * 16);
        AFrag<W> fa[R];
        BFrag<W> b0, b1;
        load_b<W>(b0, hp, hr >= 0, cc);
        if constexpr (TWO) load_b<W>(b1, hp + pairs * f * 2, hr >= 0, cc);
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const int64_t row = e * d + min(r0 + r * 16 + col, d - 1);
          load_a<W>(fa[r], wb + row * nch * KD::ABYTES + q * (KD::NA * 16),
                    W == kWMx ? sb + row * nch * 4 + q : nullptr, cc);
        }
#pragma unroll
        for (int r = 0; r < R; ++r) mma<W, TWO>(acc[r], fa[r], b0, b1);
      }
#pragma unroll
      for (int r = 0; r < R; ++r)
        *reinterpret_cast<f32x4_t *>(&s_red[wave][r][lane * 4]) = acc[r];
      __syncthreads();
      bool finish = a.S == 1;
      if (a.S > 1) {
        for (int o = tid; o < T * RB; o += kThreads) {
          const int t = o / RB, rl = o % RB, r16 = rl & 15;
          const int at = ((r16 >> 2) * 16 + t) * 4 + (r16 & 3);
          float z = 0.0f;
#pragma unroll
          for (int w = 0; w < kWaves; ++w) z += s_red[w][rl >> 4][at];
          if (r0 + rl < d) a.part[(static_cast<int64_t>(s) * T + t) * d + r0 + rl] = z;
        }
        __syncthreads();
        if (tid == 0)
          s_last = __hip_atomic_fetch_add(a.ctr + 2 + blk, 1u, __ATOMIC_ACQ_REL,
                                          __HIP_MEMORY_SCOPE_AGENT);
        __syncthreads();
        finish = s_last == static_cast<uint32_t>(a.S - 1);
      }
      if (finish) {
        for (int o = tid; o < T * RB; o += kThreads) {
          const int t = o / RB, rl = o % RB, r16 = rl & 15, row = r0 + rl;
          if (row >= d) continue;
          float z = 0.0f;
          if (a.S == 1) {
            const int at = ((r16 >> 2) * 16 + t) * 4 + (r16 & 3);
#pragma unroll
            for (int w = 0; w < kWaves; ++w) z += s_red[w][rl >> 4][at];
          } else {
            for (int p = 0; p < a.S; ++p) z += a.part[(static_cast<int64_t>(p) * T + t) * d + row];
          }
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
    }
    if (tid == 0) s_ticket = next;
    __syncthreads();
    item = s_ticket;
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

struct FewWs {
  size_t logits, ctr, h, part, bytes;
  int parts, n_ctr;
};

FewWs few_ws(int T, int d, int N, int K, int Ks, int f) {
  auto up = [](size_t b) { return (b + 255) & ~size_t(255); };
  FewWs w;
  w.parts = down_parts(d, 16 * kRows);
  w.n_ctr = 2 + (d + 16 * kRows - 1) / (16 * kRows);
  size_t at = 0;
  w.logits = at;
  at += up(sizeof(float) * T * N);
  w.ctr = at;
  at += up(sizeof(uint32_t) * w.n_ctr);
  w.h = at;
  at += up(sizeof(float) * (static_cast<size_t>(T) * K + static_cast<size_t>(Ks) * T) * f);
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
  const float *in_logit = p.select_only ? nullptr : p.router_bias;
  if (p.kind == kFewF32)
    hipLaunchKernelGGL(few_logits_kernel<float>, dim3(p.N), dim3(256), 0, s,
                       static_cast<const float *>(p.x), p.w_router, in_logit, logits, p.T, p.d, p.N,
                       ctr, L.n_ctr);
  else
    hipLaunchKernelGGL(few_logits_kernel<uint16_t>, dim3(p.N), dim3(256), 0, s,
                       static_cast<const uint16_t *>(p.x), p.w_router, in_logit, logits, p.T, p.d,
                       p.N, ctr, L.n_ctr);
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
  a.ctr = ctr;
  a.y = p.y; a.idx = p.idx; a.gate = p.gate; a.counts = p.counts;
  a.T = p.T; a.d = p.d; a.N = p.N; a.K = p.K; a.Ks = p.Ks; a.f = p.f;
  a.S = L.parts;
  a.cap = p.cap;
  const int met = p.T * p.K < p.N ? p.T * p.K : p.N;
  const int64_t items = static_cast<int64_t>(met + p.Ks) * ((p.f + 16 * kRows - 1) / (16 * kRows)) +
                        static_cast<int64_t>((p.d + 16 * kRows - 1) / (16 * kRows)) * L.parts;
  const dim3 grid(static_cast<unsigned>(items < 512 ? items : 512));
  if (p.kind == kFewF32)
    hipLaunchKernelGGL((few_layer_kernel<kWF32, kRows>), grid, dim3(kThreads), 0, s, a);
  else if (p.kind == kFewBf16)
    hipLaunchKernelGGL((few_layer_kernel<kWBf16, kRows>), grid, dim3(kThreads), 0, s, a);
  else
    hipLaunchKernelGGL((few_layer_kernel<kWMx, kRows>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
