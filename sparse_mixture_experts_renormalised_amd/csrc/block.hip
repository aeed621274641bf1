// The layer as a residual block: the routed and shared expert rows combined,
// normalised, dropped out, gated and added to the residual stream, and the
// next block's normalised input, in one pass over the token's row; and the
// gradients of all of it.
//
//   b = sum_i S_i[t] + sum_{k kept} g[t,k] Y[slot_row[t,k]]      (or a given row)
//   n = Norm_out(b),  h = residual + scale gate[t] Drop(n),  next = Norm_in(h)
//
// with Norm(v) = v^ w + bias, v^ = v (none), v r (rms, r = (mean v^2 + eps)^-1/2)
// or (v - m) r (layer).  Backward, for gradients G of h and N of next:
//
//   dh = G + r (N w - m2 - h^ m1),  m1 = mean(N w h^), m2 = mean(N w) (layer; rms: 0)
//   u = scale gate Drop'(dh),  d_gate = scale sum Drop'(dh) n
//   db = r (u w - m2' - b^ m1'),  dw = sum over tokens of u b^ and N h^
//   dY[slot] = g db,  dg = <db, Y[slot]>
//
// A workgroup takes a token's whole row into registers (8 elements a thread and
// chunk), so every tensor is read once and statistics cost a reduction instead
// of a second read; sums and statistics are float32, variances are taken around
// the mean.  Tokens are dealt to workgroups in a fixed way and the weights'
// gradients are added in a fixed order: equal calls give equal bits.
//
// Bound by memory, with loads in batches (a token's own rows, then two or four to eight
// expert rows) so that many are on their way.  4096 tokens of 7168 in bf16, eight experts
// and a shared one: forward 188 us (0.76 GB, 4.1 TB/s), gradient 288 us (1.29 GB, 4.5
// TB/s), where a copy of two 4 GiB halves reaches 4.8; over a float32 stream 212 and 338, all
// in float32 388 and 592 (1.53 and 2.58 GB, 3.9 and 4.4 TB/s).  1001 tokens of 1408 in float32 with
// LayerNorms and biases: gradient 20 us, 34 MB in the caches and two launches.  16 tokens of
// 2048: forward 5.6 us, a launch and three dependent reads.
#include "block.h"

namespace moe {
namespace {

constexpr int kMaxPart = 4;   // weights whose gradients are summed: w_in, b_in, w_out, b_out

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

// Eight elements as they lie in memory, so that many can be on their way at once.
template <typename T>
struct Raw {
  static constexpr int N = sizeof(T) / 2;   // 16-byte pieces
  u32x4_t q[N];
  __device__ __forceinline__ void load(const T *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = reinterpret_cast<const u32x4_t *>(p)[i];
  }
  // past the caches, for rows that are read once
  __device__ __forceinline__ void load_once(const T *p) {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = __builtin_nontemporal_load(reinterpret_cast<const u32x4_t *>(p) + i);
  }
  __device__ __forceinline__ void zero() {
#pragma unroll
    for (int i = 0; i < N; ++i) q[i] = (u32x4_t){0, 0, 0, 0};
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (N == 2) return __uint_as_float(q[i / 4][i % 4]);
    const uint32_t w = q[0][i / 2];
    return __uint_as_float(i & 1 ? w & 0xFFFF0000u : w << 16);
  }
};

template <typename T>
__device__ __forceinline__ void load8(const T *p, float (&v)[8]) {
  Raw<T> r;
  r.load(p);
#pragma unroll
  for (int i = 0; i < 8; ++i) v[i] = r.get(i);
}

template <typename T>
__device__ __forceinline__ void pack8(const float (&v)[8], Raw<T> &r) {
  if constexpr (Raw<T>::N == 2) {
#pragma unroll
    for (int i = 0; i < 8; ++i) r.q[i / 4][i % 4] = __float_as_uint(v[i]);
  } else {
#pragma unroll
    for (int i = 0; i < 4; ++i) r.q[0][i] = pack_bf16x2(v[2 * i], v[2 * i + 1]);
  }
}
template <typename T>
__device__ __forceinline__ void store8(T *p, const float (&v)[8]) {
  Raw<T> r;
  pack8(v, r);
#pragma unroll
  for (int i = 0; i < Raw<T>::N; ++i) reinterpret_cast<u32x4_t *>(p)[i] = r.q[i];
}
// past the caches: rows that are not read again soon (with these, wide rows take 187 us
// instead of 194, their gradient 288 instead of 294)
template <typename T>
__device__ __forceinline__ void store8_once(T *p, const float (&v)[8]) {
  Raw<T> r;
  pack8(v, r);
#pragma unroll
  for (int i = 0; i < Raw<T>::N; ++i) __builtin_nontemporal_store(r.q[i], reinterpret_cast<u32x4_t *>(p) + i);
}

// Sum of a wave's 64 values, in every lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ float dpp_add(float v) {
  const int o = __builtin_amdgcn_update_dpp(0, __float_as_int(v), CTRL, ROWS, 0xF, false);
  return v + __int_as_float(o);
}
__device__ __forceinline__ float wave_sum(float v) {
  v = dpp_add<0xB1, 0xF>(v);     // quad_perm [1,0,3,2]
  v = dpp_add<0x4E, 0xF>(v);     // quad_perm [2,3,0,1]
  v = dpp_add<0x141, 0xF>(v);    // row_half_mirror: the other four of eight
  v = dpp_add<0x140, 0xF>(v);    // row_mirror: the other eight of sixteen
  v = dpp_add<0x142, 0xA>(v);    // row_bcast15 into rows 1 and 3
  v = dpp_add<0x143, 0xC>(v);    // row_bcast31 into rows 2 and 3
  return __int_as_float(__builtin_amdgcn_readlane(__float_as_int(v), 63));
}

// Sums of N values over the NW waves of a workgroup.  Two buffers in turn: a
// wave that writes one again has passed the other's barrier, which every wave
// reaches after it read the first.
template <int NW, int N>
struct Sums {
  float buf[2][N][NW];
};
template <int NW, int N, int M>
__device__ __forceinline__ void block_sum(Sums<NW, N> &s, int &turn, float (&v)[M]) {
  static_assert(M <= N, "buffer too small");
#pragma unroll
  for (int i = 0; i < M; ++i) v[i] = wave_sum(v[i]);
  if constexpr (NW > 1) {
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int i = 0; i < M; ++i) s.buf[turn][i][threadIdx.x >> 6] = v[i];
    __syncthreads();
#pragma unroll
    for (int i = 0; i < M; ++i) {
      v[i] = 0.0f;
#pragma unroll
      for (int w = 0; w < NW; ++w) v[i] += s.buf[turn][i][w];
    }
    turn ^= 1;
  }
}

// Normalises v in place; returns r.  Chunks behind the row's end hold zeros.
template <int NW, int CH, int N>
__device__ __forceinline__ float normalise(float (&v)[CH][8], int kind, float eps, float inv_d, int nvec,
                                           Sums<NW, N> &s, int &turn) {
  if (kind == kNormNone) return 1.0f;
  if (kind == kNormLayer) {
    float m[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) m[0] += v[c][j];
    block_sum(s, turn, m);
#pragma unroll
    for (int c = 0; c < CH; ++c)
      if (static_cast<int>(NW == 1 ? threadIdx.x & 63 : threadIdx.x) + c * NW * 64 < nvec)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[c][j] -= m[0] * inv_d;
  }
  float q[1] = {0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) q[0] += v[c][j] * v[c][j];
  block_sum(s, turn, q);
  const float r = 1.0f / sqrtf(q[0] * inv_d + eps);
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) v[c][j] *= r;
  return r;
}

// Eight weights (ones or zeros where there are none).
__device__ __forceinline__ void load_w(const float *w, int at, float none, float (&v)[8]) {
  if (w) {
    load8(w + at, v);
  } else {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] = none;
  }
}

template <typename A, typename R, int NW, int CH>
__global__ __launch_bounds__(NW * 64) void block_join_kernel(BlockJoin a) {
  __shared__ Sums<NW, 1> s_sum;
  int turn = 0;
  const int tid = threadIdx.x, nvec = a.d / 8;
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const DropKey key = drop_key(a.drop);
  const A *y_rows = static_cast<const A *>(a.y_rows), *shared = static_cast<const A *>(a.shared_out);
  const bool has_branch = a.branch || a.y_rows;
  for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
    const int64_t row = t * a.d;
    // expert rows in batches: a batch is on its way before its first row is added
    constexpr int BATCH = CH * static_cast<int>(sizeof(A)) >= 8 ? 4 : 8;
    Raw<R> res[CH];
    float h[CH][8], b[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int vec = tid + c * NW * 64;
#pragma unroll
      for (int j = 0; j < 8; ++j) b[c][j] = 0.0f;
      res[c].zero();
      if (vec < nvec) {
        res[c].load(static_cast<const R *>(a.residual) + row + vec * 8);
        if (a.branch) load8(static_cast<const A *>(a.branch) + row + vec * 8, b[c]);
      }
    }
    if (a.y_rows) {
      // shared experts first, then slots in order, as moe_combine adds them
      for (int i = 0; i < a.n_shared; ++i)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int vec = tid + c * NW * 64;
          if (vec < nvec) {
            Raw<A> v;
            v.load_once(shared + (i * a.T + t) * a.d + vec * 8);
#pragma unroll
            for (int j = 0; j < 8; ++j) b[c][j] += v.get(j);
          }
        }
      for (int k0 = 0; k0 < a.K; k0 += BATCH) {
        Raw<A> v[BATCH][CH];
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          const int64_t r = k0 + i < a.K ? a.slot_row[t * a.K + k0 + i] : -1;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int vec = tid + c * NW * 64;
            if (r >= 0 && vec < nvec) v[i][c].load_once(y_rows + r * a.d + vec * 8);
          }
        }
#pragma unroll
        for (int i = 0; i < BATCH; ++i) {
          if (k0 + i >= a.K || a.slot_row[t * a.K + k0 + i] < 0) continue;
          const float g = a.topk_gate[t * a.K + k0 + i];
#pragma unroll
          for (int c = 0; c < CH; ++c)
            if (tid + c * NW * 64 < nvec)
#pragma unroll
              for (int j = 0; j < 8; ++j) b[c][j] += g * v[i][c].get(j);
        }
      }
    }
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) h[c][j] = res[c].get(j);
    if (has_branch) {
      if (a.branch_out)
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int vec = tid + c * NW * 64;
          if (vec < nvec) store8_once(static_cast<A *>(a.branch_out) + row + vec * 8, b[c]);
        }
      normalise<NW, CH>(b, a.norm_out, a.eps, inv_d, nvec, s_sum, turn);
      const float f = a.gate ? a.scale * a.gate[t] : a.scale;
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int vec = tid + c * NW * 64;
        if (vec >= nvec) continue;
        float w[8], o[8];
        load_w(a.w_out, vec * 8, 1.0f, w);
        load_w(a.b_out, vec * 8, 0.0f, o);
        const uint4 q = a.drop.cut ? philox_block(key, static_cast<uint64_t>(t) * nvec + vec)
                                   : make_uint4(0, 0, 0, 0);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          const float n = b[c][j] * w[j] + o[j];
          h[c][j] += half_of(q, j) >= a.drop.cut ? f * a.drop.keep * n : 0.0f;
        }
      }
    }
    if (a.out)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int vec = tid + c * NW * 64;
        if (vec < nvec) store8_once(static_cast<R *>(a.out) + row + vec * 8, h[c]);
      }
    if (!a.next) continue;
    normalise<NW, CH>(h, a.norm_in, a.eps, inv_d, nvec, s_sum, turn);
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int vec = tid + c * NW * 64;
      if (vec >= nvec) continue;
      float w[8], o[8];
      load_w(a.w_in, vec * 8, 1.0f, w);
      load_w(a.b_in, vec * 8, 0.0f, o);
#pragma unroll
      for (int j = 0; j < 8; ++j) o[j] += h[c][j] * w[j];
      store8(static_cast<A *>(a.next) + row + vec * 8, o);
    }
  }
}

// Gradient of the rows before a norm, in place of that of the normalised ones
// (already times the weights); hat and r as the norm left them.
template <int NW, int CH, int N>
__device__ __forceinline__ void norm_grad(float (&g)[CH][8], const float (&hat)[CH][8], float r, int kind,
                                          float inv_d, Sums<NW, N> &s, int &turn) {
  if (kind == kNormNone) return;
  float m[2] = {0.0f, 0.0f};
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      m[0] += g[c][j] * hat[c][j];
      m[1] += g[c][j];
    }
  block_sum(s, turn, m);
  const float m1 = m[0] * inv_d, m2 = kind == kNormLayer ? m[1] * inv_d : 0.0f;
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) g[c][j] = r * (g[c][j] - m2 - hat[c][j] * m1);
}

constexpr int kSlots = 2;   // slots whose rows are read, and whose products are summed, together

// TOKENS: tokens that a workgroup has in hand (rows of one wave), so that they leave one
// part of each sum over tokens.
template <typename A, typename R, int NW, int CH, int TOKENS, bool BIAS>
__global__ __launch_bounds__(NW * 64 * TOKENS, NW == 8 && CH <= 2 ? 4 : 1) void block_join_grad_kernel(BlockJoinGrad a) {
  __shared__ Sums<NW, kSlots> s_sum;
  int turn = 0;
  static_assert(TOKENS == 1 || (NW == 1 && CH == 1), "several tokens: rows of one wave");
  // (the token's number stays in scalar registers: its slots and gates are scalar loads)
  const int tid = TOKENS == 1 ? threadIdx.x : threadIdx.x & 63, nvec = a.d / 8;
  const int mine = TOKENS == 1 ? 0 : __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const float inv_d = 1.0f / static_cast<float>(a.d);
  const DropKey key = drop_key(a.drop);
  const bool slots = a.branch && (a.d_y_rows || a.d_topk_gate);
  float swi[CH][8], swo[CH][8], sbi[BIAS ? CH : 1][8], sbo[BIAS ? CH : 1][8];
#pragma unroll
  for (int c = 0; c < CH; ++c)
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      swi[c][j] = swo[c][j] = 0.0f;
      if (BIAS) sbi[c][j] = sbo[c][j] = 0.0f;
    }
  for (int64_t t = static_cast<int64_t>(blockIdx.x) * TOKENS + mine; t < a.T; t += static_cast<int64_t>(gridDim.x) * TOKENS) {
    const int64_t row = t * a.d;
    // everything of the token's own rows is on its way before the first sum
    Raw<A> rn[CH], rb[CH];
    Raw<R> rh[CH], ro[CH];
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int vec = tid + c * NW * 64;
      rn[c].zero(), rb[c].zero(), rh[c].zero(), ro[c].zero();
      if (vec >= nvec) continue;
      if (a.d_next) {
        rh[c].load(static_cast<const R *>(a.h) + row + vec * 8);
        rn[c].load(static_cast<const A *>(a.d_next) + row + vec * 8);
      }
      if (a.branch) rb[c].load(static_cast<const A *>(a.branch) + row + vec * 8);
      if (a.d_out) ro[c].load(static_cast<const R *>(a.d_out) + row + vec * 8);
    }
    float dh[CH][8], hat[CH][8];
#pragma unroll
    for (int c = 0; c < CH; ++c)
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        hat[c][j] = rh[c].get(j);
        dh[c][j] = rn[c].get(j);
      }
    if (a.d_next) {
      const float r = normalise<NW, CH>(hat, a.norm_in, a.eps, inv_d, nvec, s_sum, turn);
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int vec = tid + c * NW * 64;
        if (vec >= nvec) continue;
        float w[8];
        load_w(a.w_in, vec * 8, 1.0f, w);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
          swi[c][j] += dh[c][j] * hat[c][j];
          if (BIAS) sbi[c][j] += dh[c][j];
          dh[c][j] *= w[j];
        }
      }
      norm_grad<NW, CH>(dh, hat, r, a.norm_in, inv_d, s_sum, turn);
    }
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int vec = tid + c * NW * 64;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // behind the row's end LayerNorm's mean left something
        dh[c][j] = vec < nvec ? dh[c][j] + ro[c].get(j) : 0.0f;
        hat[c][j] = rb[c].get(j);
      }
      if (a.d_residual && vec < nvec) store8_once(static_cast<R *>(a.d_residual) + row + vec * 8, dh[c]);
    }
    if (!a.branch) continue;
    const float r = normalise<NW, CH>(hat, a.norm_out, a.eps, inv_d, nvec, s_sum, turn);
    const float f = a.gate ? a.scale * a.gate[t] : a.scale;
    float dg[1] = {0.0f};
#pragma unroll
    for (int c = 0; c < CH; ++c) {
      const int vec = tid + c * NW * 64;
      if (vec >= nvec) continue;
      float w[8], o[8];
      load_w(a.w_out, vec * 8, 1.0f, w);
      load_w(a.d_gate ? a.b_out : nullptr, vec * 8, 0.0f, o);
      const uint4 q = a.drop.cut ? philox_block(key, static_cast<uint64_t>(t) * nvec + vec)
                                 : make_uint4(0, 0, 0, 0);
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        // a dropped element takes no part, whatever its value is
        const bool stays = half_of(q, j) >= a.drop.cut;
        const float u = stays ? dh[c][j] * a.drop.keep : 0.0f, v = stays ? hat[c][j] : 0.0f;
        dg[0] += u * (v * w[j] + o[j]);
        const float g = f * u;
        swo[c][j] += g * v;
        if (BIAS) sbo[c][j] += g;
        dh[c][j] = g * w[j];
      }
    }
    if (a.d_gate) {
      block_sum(s_sum, turn, dg);
      if (tid == 0) a.d_gate[t] = a.scale * dg[0];
    }
    if (!a.d_branch && !slots) continue;
    norm_grad<NW, CH>(dh, hat, r, a.norm_out, inv_d, s_sum, turn);
    if (a.d_branch)
#pragma unroll
      for (int c = 0; c < CH; ++c) {
        const int vec = tid + c * NW * 64;
        if (vec < nvec) store8_once(static_cast<A *>(a.d_branch) + row + vec * 8, dh[c]);
      }
    if (!slots) continue;
    for (int k0 = 0; k0 < a.K; k0 += kSlots) {
      Raw<A> y[kSlots][CH];
      if (a.d_topk_gate)
#pragma unroll
        for (int i = 0; i < kSlots; ++i) {
          const int64_t sr = k0 + i < a.K ? a.slot_row[t * a.K + k0 + i] : -1;
#pragma unroll
          for (int c = 0; c < CH; ++c) {
            const int vec = tid + c * NW * 64;
            y[i][c].zero();
            if (sr >= 0 && vec < nvec) y[i][c].load_once(static_cast<const A *>(a.y_rows) + sr * a.d + vec * 8);
          }
        }
      float dot[kSlots];
#pragma unroll
      for (int i = 0; i < kSlots; ++i) {
        dot[i] = 0.0f;
        const int64_t sr = k0 + i < a.K ? a.slot_row[t * a.K + k0 + i] : -1;
        if (sr < 0) continue;
        const float g = a.topk_gate[t * a.K + k0 + i];
#pragma unroll
        for (int c = 0; c < CH; ++c) {
          const int vec = tid + c * NW * 64;
          if (a.d_topk_gate)
#pragma unroll
            for (int j = 0; j < 8; ++j) dot[i] += dh[c][j] * y[i][c].get(j);
          if (a.d_y_rows && vec < nvec) {
            float v[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) v[j] = g * dh[c][j];
            store8_once(static_cast<A *>(a.d_y_rows) + sr * a.d + vec * 8, v);
          }
        }
      }
      if (a.d_topk_gate) {
        block_sum(s_sum, turn, dot);
        if (tid < kSlots && k0 + tid < a.K)
          a.d_topk_gate[t * a.K + k0 + tid] = tid == 0 ? dot[0] : dot[1];
      }
    }
  }
  if constexpr (TOKENS > 1) {
    // the sums of its tokens, in order, in the first one's registers
    __shared__ float s_rows[kMaxPart][TOKENS - 1][8][64];
    auto give = [&](int which, const float (&v)[8]) {
#pragma unroll
      for (int j = 0; j < 8; ++j) s_rows[which][mine - 1][j][tid] = v[j];
    };
    auto take = [&](int which, float (&v)[8]) {
#pragma unroll
      for (int i = 0; i < TOKENS - 1; ++i)
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] += s_rows[which][i][j][tid];
    };
    if (mine > 0) {
      if (a.sum[0]) give(0, swi[0]);
      if (BIAS && a.sum[1]) give(1, sbi[0]);
      if (a.sum[2]) give(2, swo[0]);
      if (BIAS && a.sum[3]) give(3, sbo[0]);
    }
    __syncthreads();
    if (mine > 0) return;
    if (a.sum[0]) take(0, swi[0]);
    if (BIAS && a.sum[1]) take(1, sbi[0]);
    if (a.sum[2]) take(2, swo[0]);
    if (BIAS && a.sum[3]) take(3, sbo[0]);
  }
  // this workgroup's part of the weights' gradients: part[which][workgroup][d]
#pragma unroll
  for (int c = 0; c < CH; ++c) {
    const int vec = tid + c * NW * 64;
    if (vec >= nvec) continue;
    const int64_t at = static_cast<int64_t>(blockIdx.x) * a.d + vec * 8, step = static_cast<int64_t>(gridDim.x) * a.d;
    if (a.sum[0]) store8(a.part + at, swi[c]);
    if (BIAS && a.sum[1]) store8(a.part + step + at, sbi[BIAS ? c : 0]);
    if (a.sum[2]) store8(a.part + 2 * step + at, swo[c]);
    if (BIAS && a.sum[3]) store8(a.part + 3 * step + at, sbo[BIAS ? c : 0]);
  }
}

// Sums of the workgroups' parts: 32 columns (a line) a workgroup, four a thread, 128
// ranges of parts whose sums are added in order.
__global__ __launch_bounds__(1024) void block_sum_parts_kernel(const float *part, int parts, int d,
                                                               float *o0, float *o1, float *o2, float *o3) {
  float *out = blockIdx.y == 0 ? o0 : blockIdx.y == 1 ? o1 : blockIdx.y == 2 ? o2 : o3;
  if (!out) return;
  __shared__ __attribute__((aligned(16))) float s[128][32];
  __shared__ float s_last[16][32];
  const int quad = threadIdx.x & 7, w = threadIdx.x >> 3, col = blockIdx.x * 32 + quad * 4;
  float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
  if (col < d) {
    const float *p = part + (static_cast<int64_t>(blockIdx.y) * parts) * d + col;
    const int per = (parts + 127) / 128, end = min(parts, (w + 1) * per);
#pragma unroll 8
    for (int i = w * per; i < end; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(p + static_cast<int64_t>(i) * d);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
  }
  *reinterpret_cast<float4 *>(&s[w][quad * 4]) = v;
  __syncthreads();
  const int c = threadIdx.x & 31, r = threadIdx.x >> 5;
  if (r < 16) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += s[r * 8 + i][c];
    s_last[r][c] = sum;
  }
  __syncthreads();
  if (r == 0 && blockIdx.x * 32 + c < d) {
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < 16; ++i) sum += s_last[i][c];
    out[blockIdx.x * 32 + c] = sum;
  }
}

// Shape of a workgroup for rows of nvec chunks of 8 elements: waves, and chunks a thread.
struct Shape {
  int nw, ch, tokens;
};
Shape join_shape(int nvec) {
  if (nvec <= 64) return {1, 1, 1};
  if (nvec <= 128) return {2, 1, 1};
  if (nvec <= 256) return {4, 1, 1};
  if (nvec <= 512) return {4, 2, 1};
  if (nvec <= 1024) return {4, 4, 1};
  return {8, 4, 1};
}
// Rows of one wave: four of 129 tokens or more to a workgroup (3861 tokens of 296: 26.0 us
// with parts of one, 15.8; 108 tokens of 8: 10.5 and 12.5).
Shape grad_shape(int64_t T, int nvec) {
  if (nvec <= 64) return {1, 1, T <= 128 ? 1 : 4};
  if (nvec <= 128) return {2, 1, 1};
  if (nvec <= 256) return {4, 1, 1};
  if (nvec <= 512) return {8, 1, 1};
  if (nvec <= 1024) return {8, 2, 1};
  return {8, 4, 1};
}

// Workgroups of the gradient: sixteen waves fill a CU.  Every one leaves a part of each
// sum over tokens, which costs as much as a token's row, so that it takes two tokens or
// more where there are many (33 tokens of 1408: 8.5 us, two each 10.9, four each 16.2;
// 1001: 24.3, 20.0 and 21.5; 187 of 248, four waves: 11.1, two a wave 16.1).
unsigned grad_grid(int64_t T, int d) {
  const Shape s = grad_shape(T, d / 8);
  const int64_t most = 4096 / (s.nw * s.tokens) < 2048 ? 4096 / (s.nw * s.tokens) : 2048;
  const int64_t each = s.tokens == 1 ? (T <= 128 ? 1 : 2) : s.tokens * (T <= 1024 ? 1 : 2);
  const int64_t want = (T + each - 1) / each;
  return static_cast<unsigned>(want < most ? want : most);
}

template <typename A, typename R, int NW, int CH>
void launch_join(const BlockJoin &a, hipStream_t s) {
  const int64_t most = 8192 / NW;
  const dim3 grid(static_cast<unsigned>(a.T < most ? a.T : most));
  hipLaunchKernelGGL((block_join_kernel<A, R, NW, CH>), grid, dim3(NW * 64), 0, s, a);
}

template <typename A, typename R, int NW, int CH, int TOKENS = 1>
void launch_grad(const BlockJoinGrad &a, hipStream_t s) {
  const dim3 grid(grad_grid(a.T, a.d)), threads(NW * 64 * TOKENS);
  if (a.sum[1] || a.sum[3])
    hipLaunchKernelGGL((block_join_grad_kernel<A, R, NW, CH, TOKENS, true>), grid, threads, 0, s, a);
  else
    hipLaunchKernelGGL((block_join_grad_kernel<A, R, NW, CH, TOKENS, false>), grid, threads, 0, s, a);
}

template <typename A, typename R>
void dispatch_shape(const BlockJoin &a, hipStream_t s) {
  const Shape sh = join_shape(a.d / 8);
  if (sh.nw == 1) launch_join<A, R, 1, 1>(a, s);
  else if (sh.nw == 2) launch_join<A, R, 2, 1>(a, s);
  else if (sh.ch == 1) launch_join<A, R, 4, 1>(a, s);
  else if (sh.ch == 2) launch_join<A, R, 4, 2>(a, s);
  else if (sh.nw == 4) launch_join<A, R, 4, 4>(a, s);
  else launch_join<A, R, 8, 4>(a, s);
}
template <typename A, typename R>
void dispatch_shape(const BlockJoinGrad &a, hipStream_t s) {
  const Shape sh = grad_shape(a.T, a.d / 8);
  if (sh.tokens == 4) launch_grad<A, R, 1, 1, 4>(a, s);
  else if (sh.nw == 1) launch_grad<A, R, 1, 1>(a, s);
  else if (sh.nw == 2) launch_grad<A, R, 2, 1>(a, s);
  else if (sh.nw == 4) launch_grad<A, R, 4, 1>(a, s);
  else if (sh.ch == 1) launch_grad<A, R, 8, 1>(a, s);
  else if (sh.ch == 2) launch_grad<A, R, 8, 2>(a, s);
  else launch_grad<A, R, 8, 4>(a, s);
}

template <typename Args>
void dispatch_types(const Args &a, hipStream_t s) {
  if (!a.act_bf16) dispatch_shape<float, float>(a, s);
  else if (a.res_bf16) dispatch_shape<uint16_t, uint16_t>(a, s);
  else dispatch_shape<uint16_t, float>(a, s);
}

}  // namespace

hipError_t launch_block_join(const BlockJoin &a, hipStream_t s) {
  dispatch_types(a, s);
  return hipGetLastError();
}

size_t block_join_grad_workspace_bytes(int64_t T, int d) {
  return sizeof(float) * kMaxPart * grad_grid(T, d) * d;
}

hipError_t launch_block_join_grad(const BlockJoinGrad &a, hipStream_t s) {
  if (a.T > 0) {
    dispatch_types(a, s);
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (a.sum[0] || a.sum[1] || a.sum[2] || a.sum[3]) {
    hipLaunchKernelGGL(block_sum_parts_kernel, dim3((a.d + 31) / 32, 4), dim3(1024), 0, s, a.part,
                       a.T > 0 ? static_cast<int>(grad_grid(a.T, a.d)) : 0, a.d, a.sum[0], a.sum[1], a.sum[2],
                       a.sum[3]);
  }
  return hipGetLastError();
}

}  // namespace moe
