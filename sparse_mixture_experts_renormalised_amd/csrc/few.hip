// The whole layer for 1 to 16 tokens in two kernels ([DSMoE] output equation
// with the routing of [TopK] and the capacity limit of [TopK] 解決策2).
//
// With so few tokens the layer is one pass over the weights of the experts
// the tokens meet, and the rest is latency.  The general path starts seven or
// more kernels and keeps per-expert row lists in memory; here
//
//   kernel 1 (few_logits_kernel) computes the router's logits, one workgroup
//     per expert, lays the tokens out for kernel 2 and clears its counters;
//   kernel 2 (few_layer_kernel) does the rest.  Every workgroup repeats the
//     top-K selection, gates and capacity from the logits (T * N numbers)
//     into LDS.  Then come the hidden rows of every met or shared expert, and
//     after them the output rows.
//
// Layout of the products.  A wave reads weights straight from memory into
// the operand registers of 16 x 16 matrix instructions, 16 bytes a lane.  In
// the instruction's own order neighbouring lanes belong to different rows,
// and the 64 lanes' addresses are then looked up one by one (measured: 64
// clocks a load instead of 16, which bound the kernel at a third of the
// memory's rate).  So its 16 rows are taken as 4 weight rows x 4 pieces b of a
// chunk of the reduction axis, and its 16 columns as 4 tokens x 4 pieces b':
//
//   A[(row, b)][q] = W[row][piece 4q + b],  B[q][(token, b')] = x[token][piece 4q + b']
//
// (q: the four lanes that share a row), so four neighbouring lanes read 64
// neighbouring bytes, on both sides.  Entry ((row, b), (token, b')) of the
// result is of use where b = b', and the four of them add up to the product
// of the row with the token.  Each instruction still takes 1 KB of new weights;
// five to sixteen tokens take two or four of them.
//
// Hidden values carry the gate (g * SiLU(.)), so an output row is one sum over
// all (expert, hidden) pairs and no per-expert output exists.  bf16 layers keep
// them in two bf16 parts (value, and what its rounding left: 16 significant
// bits), MXFP4 layers in three E4M3 parts (below), float32 layers in float32.
//
// Waiting.  Output rows need every hidden row.  The hidden rows are dealt to as
// many shares as there are workgroups, and a share has a state: free, taken,
// done.  A workgroup takes its own share first, and where it then waits for all
// shares to be done, it takes any that is still free (its workgroup has not
// started yet).  So a share that is waited for is either taken, by a workgroup
// that runs and does not wait before it is done, or will be taken by one that
// waits: every wait ends, whatever the number of resident workgroups and
// whatever else runs on the device.  One counter that deals the items out would
// be simpler, but atomics on one address cost about 80 ns each here.
//
// Results do not depend on timing: sums are split in a way fixed by the sizes and
// the experts that are met, and joined in a fixed order.
#include <math.h>

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

// Activations of MXFP4 layers enter the scaled matrix instructions as sums of
// E4M3 numbers: per block of 32 a scale 2^E, E the smallest integer with
// max|v| <= 448 * 2^E, and parts v / 2^E = p0 + p1 / 16 + p2 / 256 + ..., each
// part the nearest E4M3 number to what the ones before it left, times 16.  A
// part holds four significant bits, and what it leaves is at most 1/16 of it.
// So two parts hold a bf16 number (eight bits) exactly, down to 2^-13 of the
// block's largest; below, they are off by at most half the smallest step, 2^-14
// of 2^E and with it 2^-21 of the largest.  The parts' scales are 2^E, 2^(E-4), 2^(E-8).  E is at least -119, so that these
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

// The three kinds of layers.  A chunk is what the 16 lanes of a weight row load
// together: 16 pieces of 16 bytes.
//   CH        elements of a chunk;  EB: element bytes times 8
//   CB        bytes of a chunk of one part of the activations, in NB loads
//   PUP, PDN  parts of the activations of the first and of the second Linear
// The activations are kept in the workspace, padded with zeros to whole chunks.
// A chunk of E4M3 parts is stored in the order in which its 16-byte pieces are
// loaded: the instruction's 8-bit operand holds elements 16 q .. +15 (first
// load) and 64 + 16 q .. +15 (second) of the 128 it multiplies, while the lane
// with 4-bit codes holds 32 q .. +31.
enum { kWF32, kWBf16, kWMx };
template <int W> struct Kind;
template <> struct Kind<kWF32> {
  using Act = float;
  static constexpr int CH = 64, CB = 256, NB = 1, PUP = 1, PDN = 1;
};
template <> struct Kind<kWBf16> {
  using Act = uint16_t;
  static constexpr int CH = 128, CB = 256, NB = 1, PUP = 1, PDN = 2;
};
template <> struct Kind<kWMx> {
  using Act = uint16_t;
  static constexpr int CH = 512, CB = 512, NB = 2, PUP = 2, PDN = 3;
};
// Byte of element k (of a chunk of E4M3 parts) within the chunk.
__device__ __forceinline__ int part_byte(int k) {
  const int blk = k >> 5, q = blk >> 2, b = blk & 3, e = k & 31;
  return (q >> 1) * 256 + ((q & 1) * 2 + (e >> 4)) * 64 + b * 16 + (e & 15);
}

// What kernel 1 does beside the logits.
struct FewPrep {
  int kind;
  void *x;                    // tokens [parts][T][chunks of d]
  uint8_t *xs;                // scale bytes of their blocks [T][16 a chunk]
  uint32_t *ctr, *h, *hs;     // to clear: counters, hidden rows' padding and zeros
  int n_ctr, h_rows, h_parts, h_chunks, h_words, hs_words;   // h_words: of a chunk
  bool h_pad;                 // the last chunk of a hidden row has padding
};

// Four elements of a token row: copied, or split into parts (eight lanes a block).
template <typename T>
__device__ __forceinline__ void prepare_tokens(const FewPrep &p, const T *x, int64_t i, int tokens, int d) {
  const int ch = p.kind == kWMx ? Kind<kWMx>::CH : sizeof(T) == 4 ? Kind<kWF32>::CH : Kind<kWBf16>::CH;
  const int nch = (d + ch - 1) / ch, row4 = nch * ch / 4;
  const int t = static_cast<int>(i / row4), k = static_cast<int>(i - static_cast<int64_t>(t) * row4) * 4;
  if (t >= tokens) return;                  // rows are whole blocks: eight lanes leave together
  float4 q = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (k < d) q = load4<T>(x + static_cast<int64_t>(t) * d + k);
  if constexpr (sizeof(T) == 4) {
    reinterpret_cast<float4 *>(p.x)[i] = q;
  } else if (p.kind == kWBf16) {
    reinterpret_cast<uint2 *>(p.x)[i] = make_uint2(pack_bf16x2(q.x, q.y), pack_bf16x2(q.z, q.w));
  } else {
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
    uint8_t *to = static_cast<uint8_t *>(p.x) + (static_cast<int64_t>(t) * nch + k / ch) * ch + part_byte(k % ch);
    *reinterpret_cast<uint32_t *>(to) = take_part(v);
    *reinterpret_cast<uint32_t *>(to + static_cast<int64_t>(tokens) * nch * ch) = take_part(v);
    if (k % 32 == 0)
      p.xs[static_cast<int64_t>(t) * nch * 16 + k / 32] =
          static_cast<uint8_t>(amax >= 0x7F800000u ? 255 : E + 127);
  }
}

// One workgroup per expert: thread i sums elements 4i, 4i + 4096, ... of
// W_e . x_t for each token, then the wave and the sixteen waves are added in a
// fixed tree.  TT is T rounded up to a power of two (the loads of a step are
// issued together); columns past T repeat the last token and are not stored.
// The workgroups past the experts lay out the tokens.
constexpr int kLogitThreads = 1024;
template <typename T, int TT>
__global__ __launch_bounds__(kLogitThreads) void few_logits_kernel(
    const T *__restrict__ x, const float *__restrict__ w, const float *__restrict__ bias,
    float *__restrict__ logits, int tokens, int d, int N, FewPrep prep) {
  constexpr int NW = kLogitThreads / 64;
  __shared__ float s_part[NW][TT];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int e = blockIdx.x;
  if (e >= N) {
    prepare_tokens<T>(prep, x, static_cast<int64_t>(e - N) * kLogitThreads + tid, tokens, d);
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
  // counters, scale bytes, the row of zeros of each part, and the last chunk
  // of every hidden row where that has padding
  {
    const int at = e * kLogitThreads + tid, step = N * kLogitThreads;
    const int row = prep.h_chunks * prep.h_words, rows = prep.h_rows * prep.h_parts;
    for (int i = at; i < prep.n_ctr; i += step) prep.ctr[i] = 0;
    for (int i = at; i < prep.hs_words; i += step) prep.hs[i] = 0;
    for (int i = at; i < prep.h_parts * row; i += step) {
      const int p = i / row;
      prep.h[(static_cast<int64_t>(p + 1) * prep.h_rows - 1) * row + (i - p * row)] = 0;
    }
    if (prep.h_pad)
      for (int64_t i = at; i < static_cast<int64_t>(rows) * prep.h_words; i += step) {
        const int64_t r = i / prep.h_words;
        prep.h[(r + 1) * row - prep.h_words + (i - r * prep.h_words)] = 0;
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
  const void *x;                         // tokens as kernel 1 laid them out
  const uint8_t *xs;                     // scale bytes of their parts
  const float *logits, *sel_bias;
  const void *w1, *b1, *w2, *b2, *ws1, *bs1, *ws2, *bs2;
  const uint8_t *c1, *c2, *cs1, *cs2;   // scale bytes of MXFP4 weights
  void *h;                               // hidden rows and one of zeros [parts][rows + 1][chunks of f]
  uint8_t *hs;                           // scale bytes of their parts [rows + 1][16 a chunk]
  float *part;                           // [S][T][d] parts of split outputs
  uint32_t *state;                       // [grid] of the shares of hidden rows
  uint32_t *arrived;                     // [row blocks] finished parts of split outputs
  uint32_t *over;                        // [kTok] tokens with a hidden value that is not finite
  void *y;
  int32_t *idx;
  float *gate;
  int32_t *counts;
  int T, d, N, K, Ks, f, S;
  int cap;                               // rows an expert keeps (T or more: no limit)
};

constexpr int kMaxTiles = 4;             // 4-row tiles of a wave
constexpr int kDownRows = 4 * kMaxTiles;   // output rows of an item
// Chunks in flight per wave, by what the activations leave of 256 registers.
template <int W, int TB> constexpr int kDepth = W == kWMx ? (TB == 1 ? 3 : 2) : TB == 4 ? 2 : 3;
// The parts of sixteen tokens' chunk would fill the registers, and four times
// the matrix instructions would take longer than the weights: there the four
// waves walk the same chunks of rows of their own, share the tokens through
// LDS, and turn the weights in registers into 16 whole rows.
template <int W, int TB> constexpr bool kShare = W == kWMx && TB == 4;
constexpr int kShareDepth = 4;

// Weights are read once: past the caches (measured: 4% of the whole layer).
__device__ __forceinline__ u32x4_t load_once(const uint8_t *p) {
  return __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p));
}

struct AFrag {
  u32x4_t v;
  int s;
};
template <int W, int TB, int P> struct BFrag {
  u32x4_t v[TB][P][Kind<W>::NB];
  int s[TB];
};

// acc += A (B_0 + B_1 + ...), one 16-byte piece a lane.
template <int W, int TB, int P>
__device__ __forceinline__ void mma(f32x4_t (&acc)[TB], const AFrag &a, const BFrag<W, TB, P> &b) {
#pragma unroll
  for (int t = 0; t < TB; ++t)
#pragma unroll
    for (int p = 0; p < P; ++p) {
      if constexpr (W == kWF32) {
#pragma unroll
        for (int j = 0; j < 4; ++j)
          acc[t] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(a.v[j]),
                                                        __uint_as_float(b.v[t][p][0][j]), acc[t], 0, 0, 0);
      } else if constexpr (W == kWBf16) {
        acc[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(__builtin_bit_cast(bf16x8_t, a.v),
                                                         __builtin_bit_cast(bf16x8_t, b.v[t][p][0]),
                                                         acc[t], 0, 0, 0);
      } else {
        const i32x8_t av = {(int)a.v[0], (int)a.v[1], (int)a.v[2], (int)a.v[3], 0, 0, 0, 0};
        const u32x4_t l = b.v[t][p][0], h = b.v[t][p][Kind<W>::NB - 1];
        const i32x8_t bv = {(int)l[0], (int)l[1], (int)l[2], (int)l[3],
                            (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
        acc[t] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(av, bv, acc[t], 4, 0, 0, a.s, 0,
                                                                  b.s[t] - 4 * p);
      }
    }
}

// 4 x 4 transpose between the four registers and four neighbouring lanes:
// v[j] of lane b becomes what v[b] of lane j was.
__device__ __forceinline__ void transpose4(uint32_t (&v)[4], bool odd, bool high) {
#pragma unroll
  for (int k = 0; k < 4; k += 2) {
    const uint32_t other = __builtin_amdgcn_mov_dpp(odd ? v[k] : v[k + 1], 0xB1, 0xF, 0xF, true);
    v[k] = odd ? other : v[k];
    v[k + 1] = odd ? v[k + 1] : other;
  }
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const uint32_t other = __builtin_amdgcn_mov_dpp(high ? v[k] : v[k + 2], 0x4E, 0xF, 0xF, true);
    v[k] = high ? other : v[k];
    v[k + 2] = high ? v[k + 2] : other;
  }
}

// Larger float, larger key, and zeros of either sign the same one (-0 + 0 = +0);
// NaN sorts somewhere, so that a selection always names distinct experts in range.
__device__ __forceinline__ uint32_t order_key(float v) {
  const uint32_t u = __float_as_uint(v + 0.0f);
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
// are not coherent with each other.  The flag that announces them is stored once the
// count of stores in flight has come down to none: a device-scope store counts until
// it has reached the memory that all XCDs share, so that no other order of memory is
// asked for than the instructions' own on gfx950.  A release would also write back a
// whole L2, which holds nothing that is shared: one for every share and part takes
// the one-token layer of 116 MB of weights from 33 to 63 us, and sixteen MXFP4 tokens
// from 148 to 180.
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

// TB: tokens in fours (1, 2 or 4).
template <int W, int TB>
__global__ __launch_bounds__(kThreads, 2) void few_layer_kernel(FewArgs a) {
  using KD = Kind<W>;
  using Act = typename KD::Act;
  __shared__ uint8_t s_slot[kTok][kMaxRouted];     // slot k of (token, expert), where the mask has it
  __shared__ int16_t s_list[kMaxRouted];           // expert of each entry
  __shared__ alignas(4) uint16_t s_mask[kMaxRouted];   // tokens of each expert
  __shared__ float s_gate[kTok * 64];
  __shared__ int16_t s_idx[kTok * 64];
  __shared__ float s_red[kWaves][TB][64];
  constexpr bool SHARE = kShare<W, TB>;
  // two chunks of the sixteen tokens' parts, and their scale bytes
  __shared__ __attribute__((aligned(16))) uint8_t s_b[SHARE ? 2 : 1][SHARE ? KD::PDN * kTok * 512 : 16];
  __shared__ __attribute__((aligned(16))) uint8_t s_bs[SHARE ? 2 : 1][SHARE ? kTok * 16 : 16];
  __shared__ uint32_t s_amax[kWaves][kTok];
  __shared__ uint32_t s_last, s_over;
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
  if (tid == 0) s_free = kGrid, s_over = 0;
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
      s_slot[i >> 6][e] = static_cast<uint8_t>(i & 63);
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

  // ---- the sums ----
  // lane: column (token tl of four, piece b), q; as a row of A: (row ar of a tile, b)
  const int b = lane & 3, tl = (lane >> 2) & 3, ar = tl, q = lane >> 4, piece = q * 4 + b;
  const int pairs = T * (K + Ks);
  // hidden row of (entry, token): routed pairs first, then the shared experts
  auto hidden_row = [&](int i, int t) -> int {
    if (i >= ne) return t < T ? T * K + (i - ne) * T + t : -1;
    const int e = s_list[i];
    return (s_mask[e] >> t) & 1 ? t * K + s_slot[t][e] : -1;
  };
  // z of walk() from its sums: register i of a lane is entry ((row q, piece i),
  // (token tl, piece b)) of tile r: take i = b, add the four lanes b, and let
  // lane b keep tile b.
  auto gather = [&](auto &acc, f32x4_t &z) {
    constexpr int R = std::extent_v<std::remove_reference_t<decltype(acc)>>;
#pragma unroll
    for (int t = 0; t < TB; ++t) {
      float keep = 0.0f;
#pragma unroll
      for (int r = 0; r < R; ++r) {
        const f32x4_t v = acc[r][t];
        float x = b == 0 ? v[0] : b == 1 ? v[1] : b == 2 ? v[2] : v[3];
        x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0xB1, 0xF, 0xF, true));
        x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x4E, 0xF, 0xF, true));
        keep = b == r ? x : keep;
      }
      z[t] = keep;
    }
  };
  // Sums of R tiles of four weight rows with the tokens over every `step`-th
  // chunk from chunk cc of entry i on, n of them.  row[r]: pieces before the
  // lane's row in the matrix wb[r] (its scale bytes cb[r]) of `pieces` a row;
  // `next` moves those and the activations' rows br to entry i.  On return
  // each lane holds z[t]: row 4 b + q of the 4 R, token 4 t + tl (b < R).
  auto walk = [&](auto tiles, auto parts, f32x4_t &z, const uint8_t *bb, const uint8_t *bs,
                  int64_t part, int pieces, const uint8_t *(&wb)[kMaxTiles],
                  const uint8_t *(&cb)[kMaxTiles], const uint32_t (&row)[kMaxTiles],
                  uint32_t (&br)[TB], int i, int cc, int n, int step, auto next) {
    constexpr int R = decltype(tiles)::value, P = decltype(parts)::value, D = kDepth<W, TB>;
    const int nch = (pieces + 15) >> 4;
    f32x4_t acc[R][TB];
#pragma unroll
    for (int r = 0; r < R; ++r)
#pragma unroll
      for (int t = 0; t < TB; ++t) acc[r][t] = f32x4_t{0, 0, 0, 0};
    struct Stage {
      AFrag a[R];
      BFrag<W, TB, P> b;
    } st[D];
    auto fetch = [&](Stage &s) {
#pragma unroll
      for (int t = 0; t < TB; ++t) {
        const uint32_t at = (br[t] * nch + cc) * KD::CB + piece * 16;
#pragma unroll
        for (int p = 0; p < P; ++p)
#pragma unroll
          for (int j = 0; j < KD::NB; ++j)
            s.b.v[t][p][j] = *reinterpret_cast<const u32x4_t *>(bb + p * part + (at + j * 256));
        if constexpr (W == kWMx) s.b.s[t] = bs[(br[t] * nch + cc) * 16 + piece];
      }
      // past the end of a row: its last piece again, times the padding's zeros
      const uint32_t at = min(cc * 16 + piece, pieces - 1);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        s.a[r].v = load_once(wb[r] + (row[r] + at) * 16);
        if constexpr (W == kWMx) s.a[r].s = cb[r][row[r] + at];
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
      for (int r = 0; r < R; ++r) mma<W, TB, P>(acc[r], s.a[r], s.b);
      // done here, not later, or the operands outlive the next loads
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < TB; ++t) asm volatile("" : "+v"(acc[r][t]));
    };
    if (n < D) {
      for (int c = 0; c < n; ++c) {
        fetch(st[0]);
        use(st[0]);
      }
    } else {
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
    }
    gather(acc, z);
  };

  // The same for waves that share the activations (kShare): n chunks from chunk
  // cc of entry i on, the same for all four waves, each for four tiles of its
  // own.  The four lanes b and the registers of the four tiles are transposed:
  // operand j then holds piece 4 q + j of row q' of tile b, sixteen rows in all,
  // and is multiplied by piece 4 q + j of sixteen tokens (column lane % 16).
  // srow: pieces before the row of tile b of this lane, for the scale bytes.
  // A chunk of the sixteen rows br goes from memory through registers into LDS one
  // step ahead, 2 P pieces of 16 bytes a thread (rows tid / 32 and 8 more); piece
  // u of row t lies at u ^ t, so that the rows read together use all banks.
  // On return z[r] is row r of tile q, token lane % 16.
  auto walk_shared = [&](auto parts, f32x4_t &z, const uint8_t *bb, const uint8_t *bs, int64_t part,
                         int pieces, const uint8_t *(&wb)[kMaxTiles], const uint8_t *(&cb)[kMaxTiles],
                         const uint32_t (&row)[kMaxTiles], uint32_t srow, uint32_t (&br)[2],
                         uint32_t &bsr, int i, int cc, int n,
                         auto next) __attribute__((always_inline)) {
    constexpr int P = decltype(parts)::value, R = kMaxTiles, D = kShareDepth;
    const int nch = (pieces + 15) >> 4;
    f32x4_t acc[2] = {{0, 0, 0, 0}, {0, 0, 0, 0}};
    z = acc[0];
    if (n <= 0) return;
    struct Stage {
      u32x4_t a[R];
      int s;
    } st[D];
    u32x4_t bv[P][2];
    uint32_t bsv;
    int bi = i, bc = cc;                   // entry and chunk of the next activations
    auto fetch_b = [&]() {
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          bv[p][j] = *reinterpret_cast<const u32x4_t *>(
              bb + p * part + ((br[j] * nch + bc) * 512 + (tid & 31) * 16));
      bsv = *reinterpret_cast<const uint32_t *>(bs + ((bsr * nch + bc) * 16 + (lane & 3) * 4));
      if (++bc == nch) {
        bc = 0;
        next(++bi, true);
      }
    };
    auto store_b = [&](int buf) {
      const int tok = tid >> 5, u = tid & 31;
#pragma unroll
      for (int p = 0; p < P; ++p)
#pragma unroll
        for (int j = 0; j < 2; ++j)
          *reinterpret_cast<u32x4_t *>(
              &s_b[SHARE ? buf : 0][p * 8192 + (tok + 8 * j) * 512 + (u ^ (tok + 8 * j)) * 16]) = bv[p][j];
      if (wave == 0) *reinterpret_cast<uint32_t *>(&s_bs[SHARE ? buf : 0][lane * 4]) = bsv;
    };
    auto fetch_a = [&](Stage &s) {
      const uint32_t at = min(cc * 16 + piece, pieces - 1);
#pragma unroll
      for (int r = 0; r < R; ++r)
        s.a[r] = load_once(wb[r] + (row[r] + at) * 16);
      s.s = *reinterpret_cast<const int *>(cb[0] + (srow + min(cc * 16 + q * 4, pieces - 4)));
      if (++cc == nch) {
        cc = 0;
        next(++i, false);
      }
    };
    auto use = [&](Stage &s, int buf) {
#pragma unroll
      for (int w = 0; w < 4; ++w) {
        uint32_t v[4] = {s.a[0][w], s.a[1][w], s.a[2][w], s.a[3][w]};
        transpose4(v, b & 1, b & 2);
#pragma unroll
        for (int r = 0; r < R; ++r) s.a[r][w] = v[r];
      }
      const int col = lane & 15;
      const uint32_t sc = *reinterpret_cast<const uint32_t *>(&s_bs[SHARE ? buf : 0][col * 16 + q * 4]);
      auto product = [&](auto jj) {
        constexpr int j = decltype(jj)::value;
        const i32x8_t a8 = {(int)s.a[j][0], (int)s.a[j][1], (int)s.a[j][2], (int)s.a[j][3], 0, 0, 0, 0};
#pragma unroll
        for (int p = 0; p < P; ++p) {
          const uint8_t *at = &s_b[SHARE ? buf : 0][p * 8192 + col * 512 + ((q * 4 + j) ^ col) * 16];
          const u32x4_t l = *reinterpret_cast<const u32x4_t *>(at);
          const u32x4_t h = *reinterpret_cast<const u32x4_t *>(at + 256);
          const i32x8_t b8 = {(int)l[0], (int)l[1], (int)l[2], (int)l[3],
                              (int)h[0], (int)h[1], (int)h[2], (int)h[3]};
          // the scale bytes of piece j, those of the activations 4 p lower (the
          // zeros of padding may borrow from each other: they multiply zeros)
          acc[p & 1] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(
              a8, b8, acc[p & 1], 4, 0, j, s.s, j, static_cast<int>(sc - 0x04040404u * p));
        }
      };
      product(std::integral_constant<int, 0>{});
      product(std::integral_constant<int, 1>{});
      product(std::integral_constant<int, 2>{});
      product(std::integral_constant<int, 3>{});
      // holds the products in their place
      asm volatile("" : "+v"(acc[0]), "+v"(acc[1])::"memory");
    };
    // LDS operations are done, and every wave is here
    auto meet = [&]() { asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory"); };
    // step k of n: stage k % D, buffer k % 2; weights D - 1 chunks ahead
    fetch_b();
#pragma unroll
    for (int k = 0; k < D - 1; ++k)
      if (k < n) fetch_a(st[k]);
    store_b(0);
    meet();
    int k = 0;
    constexpr int STEP = D;
    static_assert(D % 2 == 0, "stage and buffer of a step");
    for (; k + STEP + D - 1 <= n; k += STEP) {
#pragma unroll
      for (int x = 0; x < STEP; ++x) {
        fetch_b();
        fetch_a(st[(x + D - 1) % D]);
        use(st[x % D], x & 1);
        store_b(1 - (x & 1));
        meet();
      }
    }
#pragma unroll
    for (int x = 0; x < STEP + D - 1; ++x) {
      if (k + x < n) {
        const bool more = k + x + 1 < n;
        if (more) fetch_b();
        if (k + x + D - 1 < n) fetch_a(st[(x + D - 1) % D]);
        use(st[x % D], x & 1);
        if (more) store_b(1 - (x & 1));
        meet();
      }
    }
    // registers: tiles, lanes q: rows of a tile; the other way round
    const f32x4_t sum = acc[0] + acc[1];
    uint32_t v[4] = {__float_as_uint(sum[0]), __float_as_uint(sum[1]), __float_as_uint(sum[2]),
                     __float_as_uint(sum[3])};
#pragma unroll
    for (int x = 0; x < 4; x += 2) {
      const uint32_t other = __shfl_xor(q & 1 ? v[x] : v[x + 1], 16);
      v[x] = q & 1 ? other : v[x];
      v[x + 1] = q & 1 ? v[x + 1] : other;
    }
#pragma unroll
    for (int x = 0; x < 2; ++x) {
      const uint32_t other = __shfl_xor(q & 2 ? v[x] : v[x + 2], 32);
      v[x] = q & 2 ? other : v[x];
      v[x + 2] = q & 2 ? v[x + 2] : other;
    }
#pragma unroll
    for (int x = 0; x < 4; ++x) z[x] = __uint_as_float(v[x]);
  };

  // ---- hidden rows ----
  // All 4-row tiles of all entries form one row.  A share is a range of it,
  // dealt to the waves, each over the whole reduction axis.  MXFP4 layers deal
  // in blocks of 32 rows (the hidden values' scale blocks), which the
  // workgroup's waves share.
  const int grid = gridDim.x;
  const int h_chunks = (f + KD::CH - 1) / KD::CH;
  const int64_t h_part = static_cast<int64_t>(pairs + 1) * h_chunks * KD::CB;
  // Tiles u0 .. u0+m-1 of the row of tiles (m <= R; past them the last again, not stored).
  auto up_pass = [&](auto tiles, int u0, int m) __attribute__((always_inline)) {
    constexpr int R = decltype(tiles)::value;
    const int per_entry = f / 4, pieces = W == kWMx ? d / 32 : d * static_cast<int>(sizeof(Act)) / 16;
    const uint8_t *wb[kMaxTiles], *cb[kMaxTiles];
    uint32_t row[kMaxTiles], br[TB];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const int u = u0 + min(r, m - 1), i = u / per_entry;
      const bool routed = i < ne;
      const int64_t e = routed ? uniform(s_list[i]) : i - ne;
      wb[r] = static_cast<const uint8_t *>(routed ? a.w1 : a.ws1) + e * f * pieces * 16;
      cb[r] = W == kWMx ? (routed ? a.c1 : a.cs1) + e * f * pieces : nullptr;
      row[r] = static_cast<uint32_t>((u - i * per_entry) * 4 + ar) * pieces;
    }
    // A column without a token repeats one: columns do not mix, and it is not
    // stored.  Loads under a condition could not be counted, and each wait
    // would be for all of them.
#pragma unroll
    for (int t = 0; t < TB; ++t) br[t] = min(t * 4 + tl, T - 1);
    const int nch = (pieces + 15) >> 4;
    f32x4_t z = {0, 0, 0, 0};
    const uint8_t *xb = static_cast<const uint8_t *>(a.x);
    const int64_t part = static_cast<int64_t>(T) * nch * KD::CB;
    if constexpr (SHARE) {
      uint32_t rows[2] = {static_cast<uint32_t>(min(tid >> 5, T - 1)),
                          static_cast<uint32_t>(min((tid >> 5) + 8, T - 1))};
      uint32_t brow = min(lane >> 2, T - 1);
      // the tiles of a pass are of one entry
      const int us = u0 + min(b, m - 1);
      const uint32_t srow = static_cast<uint32_t>((us - us / per_entry * per_entry) * 4 + ar) * pieces;
      walk_shared(std::integral_constant<int, KD::PUP>{}, z, xb, a.xs, part, pieces, wb, cb, row, srow,
                  rows, brow, 0, 0, nch, [](int, bool) {});
    } else {
      walk(tiles, std::integral_constant<int, KD::PUP>{}, z, xb, a.xs, part, pieces, wb, cb, row, br, 0,
           0, nch, 1, [](int) {});
    }
    // The lane's values: row q of tile b for up to 4 TB tokens, or the four rows of
    // tile q for one.
    constexpr int NV = SHARE ? 4 : TB;
    const int tile = SHARE ? q : b, u = u0 + min(tile, m - 1), i = u / per_entry;
    const bool routed = i < ne;
    const int64_t e = routed ? s_list[i] : i - ne;
    const void *bias = routed ? a.b1 : a.bs1;
    auto hidden_of = [&](int v) { return (u - i * per_entry) * 4 + (SHARE ? v : q); };
    auto token_of = [&](int v) { return SHARE ? lane & 15 : v * 4 + tl; };
    uint32_t amax[TB] = {};
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      const int hidden = hidden_of(v), token = token_of(v), hr = tile < m ? hidden_row(i, token) : -1;
      if (bias) z[v] += act_f32(bias, e * f + hidden, Act{});
      const float g = routed && hr >= 0 ? s_gate[token * 64 + (hr - token * K)] : 1.0f;
      z[v] = g * silu(z[v]);
      bool over = (__float_as_uint(z[v]) & 0x7F800000u) == 0x7F800000u;
      uint8_t *hp = static_cast<uint8_t *>(a.h) + (static_cast<int64_t>(hr) * h_chunks + hidden / KD::CH) * KD::CB;
      if constexpr (W == kWF32) {
        if (hr >= 0) put_shared(reinterpret_cast<uint32_t *>(hp) + hidden % KD::CH, __float_as_uint(z[v]));
      } else if constexpr (W == kWBf16) {
        const uint16_t hi = f32_to_bf16(z[v]);
        over = (hi & 0x7F80u) == 0x7F80u;
        if (hr >= 0) {
          put_shared(reinterpret_cast<uint16_t *>(hp) + hidden % KD::CH, hi);
          put_shared(reinterpret_cast<uint16_t *>(hp + h_part) + hidden % KD::CH,
                     f32_to_bf16(z[v] - bf16_to_f32(hi)));
        }
      }
      if (over && hr >= 0) atomicOr(&s_over, 1u << token);
      // lanes without a tile hold another one's values, and not this row's gate
      uint32_t &most = amax[SHARE ? 0 : v];
      if (tile < m) most = max(most, __float_as_uint(z[v]) & 0x7FFFFFFFu);
    }
    if constexpr (W == kWMx) {
      // largest of each token's values in the wave (lanes q, and b where those are
      // tiles), then in the waves that share the block: all four, or two and two
      constexpr int NT = SHARE ? 1 : TB;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        if constexpr (!SHARE) {
          amax[t] = max(amax[t], static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax[t]), 1)));
          amax[t] = max(amax[t], static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax[t]), 2)));
        }
        amax[t] = max(amax[t], static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax[t]), 16)));
        amax[t] = max(amax[t], static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax[t]), 32)));
        if (q == 0 && (SHARE || b == 0)) s_amax[wave][token_of(t)] = amax[t];
      }
      __syncthreads();
      const int w0 = m == 2 ? 0 : wave & 2, w1 = m == 2 ? kWaves : w0 + 2;
#pragma unroll
      for (int t = 0; t < NT; ++t) {
        const int hidden = hidden_of(0), token = token_of(t), hr = tile < m ? hidden_row(i, token) : -1;
        uint32_t most = 0;
        for (int w = w0; w < w1; ++w) most = max(most, s_amax[w][token]);
        const int E = part_exponent(most), chunk = hidden / KD::CH, in_chunk = hidden % KD::CH;
        float x[4];
#pragma unroll
        for (int v = 0; v < 4; ++v) x[v] = SHARE ? __builtin_ldexpf(z[v], -E) : 0.0f;
        if (!SHARE) x[0] = __builtin_ldexpf(z[t], -E);
        uint8_t *hp = static_cast<uint8_t *>(a.h) + (static_cast<int64_t>(hr) * h_chunks + chunk) * KD::CB +
                      part_byte(in_chunk);
#pragma unroll
        for (int p = 0; p < KD::PDN; ++p) {
          const uint32_t c = take_part(x);
          if (hr >= 0) {
            if constexpr (SHARE) put_shared(reinterpret_cast<uint32_t *>(hp + p * h_part), c);
            else put_shared(hp + p * h_part, static_cast<uint8_t>(c));
          }
        }
        if (hr >= 0 && hidden % 32 == 0)
          put_shared(a.hs + (static_cast<int64_t>(hr) * h_chunks + chunk) * 16 + in_chunk / 32,
                     static_cast<uint8_t>(most >= 0x7F800000u ? 255 : E + 127));
      }
      __syncthreads();
    }
  };
  auto up_share = [&](int w) {
    if constexpr (W == kWMx) {
      const int units = entries * (f / 32), end = static_cast<int>(static_cast<int64_t>(units) * (w + 1) / grid);
      for (int u = static_cast<int>(static_cast<int64_t>(units) * w / grid); u < end;) {
        const int m = u + 1 < end ? 4 : 2;       // two units, or the last one
        if (SHARE || m == 4) up_pass(std::integral_constant<int, 4>{}, u * 8 + wave * m, m);
        else up_pass(std::integral_constant<int, 2>{}, u * 8 + wave * m, m);
        u += m / 2;
      }
    } else {
      const int units = entries * (f / 4), waves = grid * kWaves, v = w * kWaves + wave;
      int u = static_cast<int>(static_cast<int64_t>(units) * v / waves);
      const int end = static_cast<int>(static_cast<int64_t>(units) * (v + 1) / waves);
      while (u < end) {
        // passes of equal length
        const int passes = (end - u + kMaxTiles - 1) / kMaxTiles, m = (end - u + passes - 1) / passes;
        if (m == 1) up_pass(std::integral_constant<int, 1>{}, u, m);
        else if (m == 2) up_pass(std::integral_constant<int, 2>{}, u, m);
        else up_pass(std::integral_constant<int, 4>{}, u, m);
        u += m;
      }
    }
    wait_stores();
    __syncthreads();
    if (wave == 0) {
      // one store a token in all, nearly: hundreds on one address take their time
      if (lane < kTok && (s_over >> lane) & 1 && get_shared(a.over + lane) == 0) put_shared(a.over + lane, 1u);
      wait_stores();
      if (lane == 0) put_shared(a.state + w, static_cast<uint32_t>(kDone));
    }
  };
  if (s_claim) up_share(blockIdx.x);

  // ---- output rows: an item's chunks are split over S items and, where the
  // waves do not have rows of their own, over the waves ----
  constexpr int DROWS = SHARE ? kDownRows * kWaves : kDownRows, DSTEP = SHARE ? 1 : kWaves;
  const int n_down = d / DROWS * a.S, total = entries * h_chunks;
  const int down_pieces = W == kWMx ? f / 32 : f * static_cast<int>(sizeof(Act)) / 16;
  // While the last hidden rows are computed, what each wave takes first of the
  // weights comes into the caches (one token, bf16 and MXFP4: 35.5 -> 33.4 us and
  // 50.9 -> 48.9; two chunks 33.3 and 49.3, eight 35.7 and 50.7).
  if (static_cast<int>(blockIdx.x) < n_down && total > 0) {
    constexpr int AHEAD = 4;
    const int blk = blockIdx.x / a.S, s = blockIdx.x - blk * a.S;
    const int r0 = blk * DROWS + (SHARE ? wave * kDownRows : 0);
    const int c0 = static_cast<int>(static_cast<int64_t>(total) * s / a.S) + (SHARE ? 0 : wave);
    u32x4_t v[AHEAD][kMaxTiles];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = min(c0 + k * DSTEP, total - 1), i = uniform(c / h_chunks);
      const int64_t e = i < ne ? uniform(s_list[i]) : i - ne;
      const uint8_t *w = static_cast<const uint8_t *>(i < ne ? a.w2 : a.ws2) + e * d * down_pieces * 16;
      const uint32_t at = min((c - i * h_chunks) * 16 + piece, down_pieces - 1);
#pragma unroll
      for (int r = 0; r < kMaxTiles; ++r)
        v[k][r] = *reinterpret_cast<const u32x4_t *>(
            w + (static_cast<uint32_t>(r0 + r * 4 + ar) * down_pieces + at) * 16);
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
#pragma unroll
      for (int r = 0; r < kMaxTiles; ++r) asm volatile("" ::"v"(v[k][r]));
  }
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

  for (int item = blockIdx.x; item < n_down; item += grid) {
    const int blk = item / a.S, s = item - blk * a.S, r0 = blk * DROWS + (SHARE ? wave * kDownRows : 0);
    const int pieces = down_pieces;
    const int c0 = static_cast<int>(static_cast<int64_t>(total) * s / a.S) + (SHARE ? 0 : wave);
    const int c1 = static_cast<int>(static_cast<int64_t>(total) * (s + 1) / a.S);
    const int i0 = uniform(c0 / h_chunks);
    const uint8_t *wb[kMaxTiles], *cb[kMaxTiles];
    uint32_t row[kMaxTiles];
#pragma unroll
    for (int r = 0; r < kMaxTiles; ++r) row[r] = static_cast<uint32_t>(r0 + r * 4 + ar) * pieces;
    auto enter_w = [&](int i) {              // the entry's matrix
      const bool routed = i < ne;
      const int64_t e = routed ? uniform(s_list[i]) : i - ne;
      const uint8_t *w = static_cast<const uint8_t *>(routed ? a.w2 : a.ws2) + e * d * pieces * 16;
      const uint8_t *c = W == kWMx ? (routed ? a.c2 : a.cs2) + e * d * pieces : nullptr;
#pragma unroll
      for (int r = 0; r < kMaxTiles; ++r) {
        wb[r] = w;
        cb[r] = c;
      }
    };
    // the hidden row of a token: the row of zeros where it has none in the entry
    auto hidden_or_zeros = [&](int i, int t) -> uint32_t {
      const int hr = hidden_row(i, t);
      return hr < 0 ? pairs : hr;
    };
    f32x4_t z = {0, 0, 0, 0};
    const uint8_t *hb = static_cast<const uint8_t *>(a.h);
    // The zeros of tokens without a hidden row do not hide an infinity or a NaN
    // among the weights.  A sum that is not finite is therefore added up again, by
    // its lane, from the token's own entries, until it is NaN.  A token with a hidden
    // value that is not finite has no finite output and keeps its sums: a padded
    // batch may hold such tokens, and one lane takes milliseconds for a sum.
    auto own_entries = [&](int orow, int token) {
      float sum = 0.0f;
      int c = static_cast<int>(static_cast<int64_t>(total) * s / a.S);
#pragma nounroll
      while (c < c1) {
        const int i = c / h_chunks, hr = hidden_row(i, token), end = min(c1, (i + 1) * h_chunks);
        if (hr < 0) {
          c = end;
          continue;
        }
        const int64_t wrow = (i < ne ? static_cast<int64_t>(s_list[i]) : i - ne) * d + orow;
        const uint8_t *w = static_cast<const uint8_t *>(i < ne ? a.w2 : a.ws2) + wrow * pieces * 16;
        const uint8_t *cw = W == kWMx ? (i < ne ? a.c2 : a.cs2) + wrow * pieces : nullptr;
#pragma nounroll
        for (; c < end; ++c) {
          const int hc = c - i * h_chunks;
          const int64_t hat = static_cast<int64_t>(hr) * h_chunks + hc;
          const uint8_t *hv = hb + hat * KD::CB;
          const int k0 = hc * KD::CH, n = min(KD::CH, f - k0);
#pragma nounroll
          for (int k = 0; k < n; ++k) {
            float x, y;
            if constexpr (W == kWF32) {
              x = reinterpret_cast<const float *>(hv)[k];
              y = reinterpret_cast<const float *>(w)[k0 + k];
            } else if constexpr (W == kWBf16) {
              x = bf16_to_f32(reinterpret_cast<const uint16_t *>(hv)[k]) +
                  bf16_to_f32(reinterpret_cast<const uint16_t *>(hv + h_part)[k]);
              y = bf16_to_f32(reinterpret_cast<const uint16_t *>(w)[k0 + k]);
            } else {
              const int hs = a.hs[hat * 16 + k / 32], ws = cw[(k0 + k) / 32];
              x = 0.0f;
              for (int p = 0; p < KD::PDN; ++p)
                x += __builtin_ldexpf(__builtin_amdgcn_cvt_f32_fp8(hv[p * h_part + part_byte(k)], 0),
                                      hs - 127 - 4 * p);
              const uint32_t code = w[(k0 + k) / 2] >> (k & 1 ? 4 : 0);
              y = __builtin_ldexpf(__builtin_amdgcn_cvt_scalef32_pk_f32_fp4(code & 15, 1.0f, 0)[0], ws - 127);
              if (hs == 255 || ws == 255) y = __uint_as_float(0x7FC00000u);
            }
            sum = fmaf(x, y, sum);
            if (__builtin_isnan(sum)) return sum;
          }
        }
      }
      return sum;
    };
    if constexpr (SHARE) {
      uint32_t rows[2], brow = 0;
      auto enter_b = [&](int i) {
        rows[0] = hidden_or_zeros(i, tid >> 5);
        rows[1] = hidden_or_zeros(i, (tid >> 5) + 8);
        brow = hidden_or_zeros(i, lane >> 2);
      };
      const int n = max(0, c1 - c0);
      if (n > 0) {
        enter_w(i0);
        enter_b(i0);
      }
      walk_shared(std::integral_constant<int, KD::PDN>{}, z, hb, a.hs, h_part, pieces, wb, cb, row,
                  static_cast<uint32_t>(r0 + b * 4 + ar) * pieces, rows, brow, i0, c0 - i0 * h_chunks, n,
                  [&](int i, bool of_b) {
                    if (i >= entries) return;
                    if (of_b) enter_b(i);
                    else enter_w(i);
                  });
    } else {
      uint32_t br[TB];
      auto enter = [&](int i) {
        if (i >= entries) return;
        enter_w(i);
#pragma unroll
        for (int t = 0; t < TB; ++t) br[t] = hidden_or_zeros(i, t * 4 + tl);
      };
      enter(i0);
      walk(std::integral_constant<int, kMaxTiles>{}, std::integral_constant<int, KD::PDN>{}, z, hb, a.hs,
           h_part, pieces, wb, cb, row, br, i0, c0 - i0 * h_chunks,
           max(0, (c1 - c0 + kWaves - 1) / kWaves), kWaves, enter);
#pragma unroll
      for (int t = 0; t < TB; ++t) s_red[wave][t][lane] = z[t];
      __syncthreads();
    }
    // Outputs of this lane: where the wave has rows of its own, the four rows of
    // tile q for token lane % 16, else row q of tile b for token 4 wave + tl
    // (waves past TB: none).
    constexpr int OUT = SHARE ? 4 : 1;
    const int token = SHARE ? lane & 15 : wave * 4 + tl;
    const bool out = token < T && (SHARE || wave < TB);
    auto row_of = [&](int t) { return r0 + (SHARE ? q * 4 + t : b * 4 + q); };
    float v[OUT];
#pragma unroll
    for (int t = 0; t < OUT; ++t) {
      v[t] = SHARE ? z[t] : 0.0f;
      if (!SHARE && out)
#pragma unroll
        for (int w = 0; w < kWaves; ++w) v[t] += s_red[w][min(wave, TB - 1)][lane];
    }
#pragma unroll
    for (int t = 0; t < OUT; ++t)
      if (T > 1 && out && (__float_as_uint(v[t]) & 0x7F800000u) == 0x7F800000u &&
          get_shared(a.over + token) == 0)
        v[t] = own_entries(row_of(t), token);
    bool finish = true;
    if (a.S > 1) {
      const int64_t size = static_cast<int64_t>(T) * d;
      if (out)
#pragma unroll
        for (int t = 0; t < OUT; ++t)
          put_shared(a.part + s * size + static_cast<int64_t>(token) * d + row_of(t), v[t]);
      wait_stores();
      __syncthreads();
      if (tid == 0)
        s_last = __hip_atomic_fetch_add(a.arrived + blk, 1u, __ATOMIC_RELAXED,
                                        __HIP_MEMORY_SCOPE_AGENT);
      __syncthreads();
      finish = s_last == static_cast<uint32_t>(a.S - 1);
      if (finish && out)
#pragma unroll
        for (int t = 0; t < OUT; ++t) {
          v[t] = 0.0f;
          for (int k = 0; k < a.S; ++k)
            v[t] += get_shared(a.part + k * size + static_cast<int64_t>(token) * d + row_of(t));
        }
    }
    if (finish && out)
#pragma unroll
      for (int t = 0; t < OUT; ++t) {
        const int orow = row_of(t);
        if (a.bs2)
          for (int i = 0; i < Ks; ++i) v[t] += act_f32(a.bs2, static_cast<int64_t>(i) * d + orow, Act{});
        if (a.b2)
          for (int k = 0; k < K; ++k) {
            const int e = s_idx[token * 64 + k];
            if ((s_mask[e] >> token) & 1)
              v[t] += s_gate[token * 64 + k] * act_f32(a.b2, static_cast<int64_t>(e) * d + orow, Act{});
          }
        const int64_t at = static_cast<int64_t>(token) * d + orow;
        if constexpr (W == kWF32) static_cast<float *>(a.y)[at] = v[t];
        else static_cast<uint16_t *>(a.y)[at] = f32_to_bf16(v[t]);
      }
    __syncthreads();
  }
}

// How the output rows are dealt out: rows of an item, and the parts S its
// chunks are cut into.  More parts fill the chip and shorten the last round, but
// an item costs about as much as six chunks beside its own; the cost of a round
// is that and the chunks that a wave sums, for as many experts as tokens that
// are routed evenly would meet.
struct DownPlan {
  int rows, parts;
};
DownPlan down_plan(FewKind kind, int T, int d, int N, int K, int Ks, int f) {
  const bool share = kind == kFewMxfp4 && T > 8;
  const int ch = kind == kFewF32 ? Kind<kWF32>::CH : kind == kFewBf16 ? Kind<kWBf16>::CH : Kind<kWMx>::CH;
  DownPlan p{share ? kDownRows * kWaves : kDownRows, 1};
  const double met = N * (1.0 - pow(1.0 - static_cast<double>(K) / N, T)) + Ks;
  const double chunks = met * ((f + ch - 1) / ch) / (share ? 1 : kWaves);
  const int blocks = d / p.rows;
  double least = 1e300;
  for (int s = 1; s <= 16; ++s) {
    const int rounds = (blocks * s + kGrid - 1) / kGrid;
    const double cost = rounds * (6.0 + chunks / s);
    if (cost < least) {
      least = cost;
      p.parts = s;
    }
  }
  return p;
}

struct FewWs {
  size_t logits, ctr, h, hs, x, xs, part, bytes;
  int parts, blocks, n_ctr;
};

// Bytes of a row of n activations in one part.
size_t few_row_bytes(FewKind k, int n) {
  const int ch = k == kFewF32 ? Kind<kWF32>::CH : k == kFewBf16 ? Kind<kWBf16>::CH : Kind<kWMx>::CH;
  const int cb = k == kFewMxfp4 ? Kind<kWMx>::CB : 256;
  return static_cast<size_t>((n + ch - 1) / ch) * cb;
}

FewWs few_ws(FewKind kind, int T, int d, int N, int K, int Ks, int f) {
  FewWs w;
  size_t at = 0;
  auto take = [&](size_t b) {
    const size_t o = at;
    at += (b + 255) & ~size_t(255);
    return o;
  };
  const bool mx = kind == kFewMxfp4;
  const size_t rows = static_cast<size_t>(T) * (K + Ks) + 1;
  const int x_parts = mx ? Kind<kWMx>::PUP : 1, h_parts = mx ? Kind<kWMx>::PDN : kind == kFewBf16 ? 2 : 1;
  const DownPlan plan = down_plan(kind, T, d, N, K, Ks, f);
  w.parts = plan.parts;
  w.blocks = d / plan.rows;
  w.n_ctr = kGrid + w.blocks + kTok;
  w.logits = take(sizeof(float) * T * N);
  w.ctr = take(sizeof(uint32_t) * w.n_ctr);
  w.h = take(h_parts * rows * few_row_bytes(kind, f));
  w.hs = take(mx ? rows * (few_row_bytes(kind, f) / 32) : 0);
  w.x = take(x_parts * T * few_row_bytes(kind, d));
  w.xs = take(mx ? T * (few_row_bytes(kind, d) / 32) : 0);
  w.part = take(w.parts > 1 ? sizeof(float) * w.parts * T * d : 0);
  w.bytes = at;
  return w;
}

template <int TB>
hipError_t launch_layer(FewKind kind, dim3 grid, const FewArgs &a, hipStream_t s) {
  if (kind == kFewF32) hipLaunchKernelGGL((few_layer_kernel<kWF32, TB>), grid, dim3(kThreads), 0, s, a);
  else if (kind == kFewBf16) hipLaunchKernelGGL((few_layer_kernel<kWBf16, TB>), grid, dim3(kThreads), 0, s, a);
  else hipLaunchKernelGGL((few_layer_kernel<kWMx, TB>), grid, dim3(kThreads), 0, s, a);
  return hipGetLastError();
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
  FewPrep prep;
  prep.kind = mx ? kWMx : p.kind == kFewBf16 ? kWBf16 : kWF32;
  prep.x = base + L.x;
  prep.xs = reinterpret_cast<uint8_t *>(base + L.xs);
  prep.ctr = ctr;
  prep.h = reinterpret_cast<uint32_t *>(base + L.h);
  prep.hs = reinterpret_cast<uint32_t *>(base + L.hs);
  prep.n_ctr = L.n_ctr;
  prep.h_rows = p.T * (p.K + p.Ks) + 1;
  prep.h_parts = mx ? Kind<kWMx>::PDN : p.kind == kFewBf16 ? 2 : 1;
  const int ch = mx ? Kind<kWMx>::CH : p.kind == kFewBf16 ? Kind<kWBf16>::CH : Kind<kWF32>::CH;
  prep.h_words = (mx ? Kind<kWMx>::CB : 256) / 4;
  prep.h_chunks = (p.f + ch - 1) / ch;
  prep.hs_words = mx ? prep.h_rows * prep.h_chunks * 4 : 0;
  prep.h_pad = p.f % ch != 0;
  const float *in_logit = p.select_only ? nullptr : p.router_bias;
  const int64_t quads = static_cast<int64_t>(p.T) * ((p.d + ch - 1) / ch) * (ch / 4);
  const int blocks = static_cast<int>((quads + kLogitThreads - 1) / kLogitThreads);
  auto route = [&](auto x0, auto kernel) {
    using X = decltype(x0);
    hipLaunchKernelGGL(kernel, dim3(p.N + blocks), dim3(kLogitThreads), 0, s,
                       static_cast<const X *>(p.x), p.w_router, in_logit, logits, p.T, p.d, p.N, prep);
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
  a.x = base + L.x;
  a.xs = prep.xs;
  a.logits = logits;
  a.sel_bias = p.select_only ? p.router_bias : nullptr;
  a.w1 = p.w1; a.b1 = p.b1; a.w2 = p.w2; a.b2 = p.b2;
  a.ws1 = p.ws1; a.bs1 = p.bs1; a.ws2 = p.ws2; a.bs2 = p.bs2;
  a.c1 = p.c1; a.c2 = p.c2; a.cs1 = p.cs1; a.cs2 = p.cs2;
  a.h = base + L.h;
  a.hs = reinterpret_cast<uint8_t *>(base + L.hs);
  a.part = reinterpret_cast<float *>(base + L.part);
  a.state = ctr;
  a.arrived = ctr + kGrid;
  a.over = a.arrived + L.blocks;
  a.y = p.y; a.idx = p.idx; a.gate = p.gate; a.counts = p.counts;
  a.T = p.T; a.d = p.d; a.N = p.N; a.K = p.K; a.Ks = p.Ks; a.f = p.f;
  a.S = L.parts;
  a.cap = p.cap;
  // a workgroup for every share that can have rows, and for every output item
  const int64_t met = (p.T * p.K < p.N ? p.T * p.K : p.N) + p.Ks;
  const int64_t up = met * (mx ? p.f / 32 : (p.f / 4 + kWaves - 1) / kWaves);
  const int64_t down = static_cast<int64_t>(L.blocks) * L.parts;
  const int64_t items = up > down ? up : down;
  const dim3 grid(static_cast<unsigned>(items < kGrid ? items : kGrid));
  return p.T <= 4 ? launch_layer<1>(p.kind, grid, a, s)
                  : p.T <= 8 ? launch_layer<2>(p.kind, grid, a, s) : launch_layer<4>(p.kind, grid, a, s);
}

}  // namespace moe
