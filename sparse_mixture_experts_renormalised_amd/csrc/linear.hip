// Single Linears of every expert and their gradients on the float32 matrix
// instructions (v_mfma_f32_32x32x2_f32, whose products and sums are float32's).
//
// All three products are C[q][p] = sum_j Q(j, q) P(j, p), where p is the axis
// along which C lies contiguous:
//
//   forward          q row      p output feature   j input feature
//   input gradient   q row      p input feature    j output feature
//   weight gradient  q output feature  p input feature  j row of the group
//
// A workgroup computes 64 x 64 of C, four waves of 32 x 32.  Steps of 32 along j
// go through registers into LDS as [j][64]; an operand whose memory runs along j
// is turned on the way.  P is the instruction's first operand, so that a lane
// ends up with four neighbouring elements of one row of C.
#include "linear.h"

namespace moe {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kTile = 64, kStep = 32, kPitch = kTile + 4, kMaxGroups = kMaxRouted + kMaxShared;

template <typename T>
__device__ __forceinline__ void get8(const T *p, float (&v)[8]) {
  constexpr int n = 16 / sizeof(T);
#pragma unroll
  for (int h = 0; h < 8 / n; ++h) {
    union { uint4 q; T e[n]; } u;
    u.q = reinterpret_cast<const uint4 *>(p)[h];
#pragma unroll
    for (int i = 0; i < n; ++i) v[h * n + i] = Act<T>::to_f32(u.e[i]);
  }
}

template <typename T>
__device__ __forceinline__ void put4(T *p, const float (&v)[4]) {
  if constexpr (sizeof(T) == 4)
    *reinterpret_cast<float4 *>(p) = make_float4(v[0], v[1], v[2], v[3]);
  else
    *reinterpret_cast<uint2 *>(p) = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
}

template <typename T>
__device__ __forceinline__ void get4(const T *p, float (&v)[4]) {
  if constexpr (sizeof(T) == 4) {
    const float4 q = *reinterpret_cast<const float4 *>(p);
    v[0] = q.x, v[1] = q.y, v[2] = q.z, v[3] = q.w;
  } else {
    const uint2 q = *reinterpret_cast<const uint2 *>(p);
    v[0] = __uint_as_float(q.x << 16), v[1] = __uint_as_float(q.x & 0xFFFF0000u);
    v[2] = __uint_as_float(q.y << 16), v[3] = __uint_as_float(q.y & 0xFFFF0000u);
  }
}

// First 64-row tile of every group, in LDS (forward and input gradient).
__device__ int tile_prefix(const Linear &a, int *pref, int *tmp) {
  const int per = (a.groups + 255) / 256, g0 = min(static_cast<int>(threadIdx.x) * per, a.groups);
  const int g1 = min(g0 + per, a.groups);
  auto tiles = [&](int g) { return (a.offsets[g + 1] - a.offsets[g] + kTile - 1) / kTile; };
  int local = 0;
  for (int g = g0; g < g1; ++g) local += tiles(g);
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  int incl = local;
#pragma unroll
  for (int off = 1; off < 64; off <<= 1) {
    const int o = __shfl_up(incl, off);
    if (lane >= off) incl += o;
  }
  if (lane == 63) tmp[wave] = incl;
  __syncthreads();
  int run = incl - local, total = 0;
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    if (w < wave) run += tmp[w];
    total += tmp[w];
  }
  for (int g = g0; g < g1; ++g) {
    pref[g] = run;
    run += tiles(g);
  }
  if (threadIdx.x == 0) pref[a.groups] = total;
  __syncthreads();
  return total;
}

// Eight elements of an operand: along j of one line (turned into LDS), or along
// the line axis of one j.  `line` and `j` are clamped by the caller; `zero`
// stores zeros.
template <typename T, bool ALONG_J>
struct Operand {
  float v[8];
  __device__ __forceinline__ void load(const T *p, bool zero) {
    if (zero) {
#pragma unroll
      for (int i = 0; i < 8; ++i) v[i] = 0.0f;
    } else {
      get8(p, v);
    }
  }
  __device__ __forceinline__ void store(float (*s)[kPitch], int tid) const {
    if constexpr (ALONG_J) {
      const int line = tid & 63, j = (tid >> 6) * 8;
#pragma unroll
      for (int i = 0; i < 8; ++i) s[j + i][line] = v[i];
    } else {
      float4 *p = reinterpret_cast<float4 *>(&s[tid >> 3][(tid & 7) * 8]);
      p[0] = make_float4(v[0], v[1], v[2], v[3]);
      p[1] = make_float4(v[4], v[5], v[6], v[7]);
    }
  }
};

template <typename T, typename O, int MODE>
__global__ __launch_bounds__(256) void linear_f32_kernel(Linear a) {
  constexpr bool kQAlongJ = MODE != kLinWeightGrad, kPAlongJ = MODE == kLinForward;
  __shared__ __attribute__((aligned(16))) float s_q[kStep][kPitch], s_p[kStep][kPitch];
  __shared__ int s_pref[kMaxGroups + 1], s_tmp[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wq = (wave & 1) * 32, wp = (wave >> 1) * 32;
  const int np = MODE == kLinForward ? a.n_out : a.k;                 // extent of p
  const int ptiles = (np + kTile - 1) / kTile;
  const int qtiles = MODE == kLinWeightGrad ? (a.n_out + kTile - 1) / kTile : tile_prefix(a, s_pref, s_tmp);
  const int64_t total = static_cast<int64_t>(qtiles) * ptiles * (MODE == kLinWeightGrad ? a.groups : 1);
  const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *w = static_cast<const T *>(a.w);
  for (int64_t L = blockIdx.x; L < total; L += gridDim.x) {
    const int p0 = static_cast<int>(L % ptiles) * kTile;
    int64_t rest = L / ptiles;
    int g, q0;
    if (MODE == kLinWeightGrad) {
      q0 = static_cast<int>(rest % qtiles) * kTile;
      g = static_cast<int>(rest / qtiles);
    } else {
      int lo = 0, hi = a.groups;                                     // pref[lo] <= tile < pref[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= rest) lo = mid; else hi = mid;
      }
      g = lo;
      q0 = static_cast<int>(rest - s_pref[g]) * kTile;
    }
    const int64_t row0 = a.offsets[g];
    const int rows = a.offsets[g + 1] - static_cast<int>(row0);
    const int nq = MODE == kLinWeightGrad ? a.n_out : rows;
    const int nj = MODE == kLinForward ? a.k : MODE == kLinInputGrad ? a.n_out : rows;
    const T *wg = w + static_cast<int64_t>(g) * a.n_out * a.k;
    // this thread's eight elements of either operand at step j0
    auto q_src = [&](int j0, bool *zero) -> const T * {
      if constexpr (kQAlongJ) {
        const int j = j0 + (tid >> 6) * 8, q = min(q0 + (tid & 63), nq - 1);
        *zero = j >= nj;
        if (MODE == kLinForward)
          return x + (a.index ? static_cast<int64_t>(a.index[row0 + q]) : row0 + q) * a.k + j;
        return dy + (row0 + q) * a.n_out + j;
      } else {
        const int j = j0 + (tid >> 3), q = q0 + (tid & 7) * 8;
        *zero = j >= nj || q >= nq;
        return dy + (row0 + j) * a.n_out + q;
      }
    };
    auto p_src = [&](int j0, bool *zero) -> const T * {
      if constexpr (kPAlongJ) {
        const int j = j0 + (tid >> 6) * 8, p = min(p0 + (tid & 63), np - 1);
        *zero = j >= nj;
        return wg + static_cast<int64_t>(p) * a.k + j;
      } else {
        const int j = j0 + (tid >> 3), p = p0 + (tid & 7) * 8;
        *zero = j >= nj || p >= np;
        if (MODE == kLinInputGrad) return wg + static_cast<int64_t>(j) * a.k + p;
        const int64_t r = a.index && !*zero ? static_cast<int64_t>(a.index[row0 + j]) : row0 + j;
        return x + r * a.k + p;
      }
    };
    f32x16_t acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    float db = 0.0f;
    const bool sum_dy = MODE == kLinWeightGrad && a.dbias && p0 == 0;
    Operand<T, kQAlongJ> rq;
    Operand<T, kPAlongJ> rp;
    auto fetch = [&](int j0) {
      bool zero;
      const T *s = q_src(j0, &zero);
      rq.load(s, zero);
      s = p_src(j0, &zero);
      rp.load(s, zero);
    };
    if (nj > 0) fetch(0);
    for (int j0 = 0; j0 < nj; j0 += kStep) {
      __syncthreads();
      rq.store(s_q, tid);
      rp.store(s_p, tid);
      __syncthreads();
      if (j0 + kStep < nj) fetch(j0 + kStep);
#pragma unroll
      for (int j = 0; j < kStep; j += 2)
        acc = __builtin_amdgcn_mfma_f32_32x32x2f32(s_p[j + (lane >> 5)][wp + (lane & 31)],
                                                   s_q[j + (lane >> 5)][wq + (lane & 31)], acc, 0, 0, 0);
      if (sum_dy && tid < kTile) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < kStep; ++j) part += s_q[j][tid];
        db += part;
      }
    }
    if (sum_dy && tid < kTile && q0 + tid < nq) {
      O *o = static_cast<O *>(a.dbias) + static_cast<int64_t>(g) * a.n_out + q0 + tid;
      *o = Act<O>::from_f32(a.accumulate ? Act<O>::to_f32(*o) + db : db);
    }
    const int q = q0 + wq + (lane & 31);
    if (q >= nq) continue;
    const int64_t out_row = MODE == kLinWeightGrad ? static_cast<int64_t>(g) * a.n_out + q : row0 + q;
    O *out = static_cast<O *>(a.out) + out_row * np;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int p = p0 + wp + b * 8 + (lane >> 5) * 4;
      if (p >= np) continue;
      float v[4] = {acc[4 * b], acc[4 * b + 1], acc[4 * b + 2], acc[4 * b + 3]}, o[4];
      if (MODE == kLinForward) {
        if (a.bias) {
          get4(static_cast<const T *>(a.bias) + static_cast<int64_t>(g) * a.n_out + p, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] += o[i];
        }
        if (a.pre) put4(static_cast<O *>(a.pre) + out_row * np + p, v);
        if (a.silu)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = silu(v[i]);
      } else if (MODE == kLinInputGrad) {
        if (a.act_pre) {
          get4(static_cast<const T *>(a.act_pre) + out_row * np + p, o);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] *= silu_slope(o[i]);
        }
      } else if (a.accumulate) {
        get4(out + p, o);
#pragma unroll
        for (int i = 0; i < 4; ++i) v[i] += o[i];
      }
      put4(out + p, v);
    }
  }
}

template <typename T, typename O, int MODE>
void launch(const Linear &p, hipStream_t s) {
  const int64_t pt = ((MODE == kLinForward ? p.n_out : p.k) + kTile - 1) / kTile;
  const int64_t qt = MODE == kLinWeightGrad ? static_cast<int64_t>(p.groups) * ((p.n_out + kTile - 1) / kTile)
                                            : p.max_rows / kTile + (p.max_rows < p.groups ? p.max_rows : p.groups);
  const int64_t most = 1 << 20, want = pt * qt;
  hipLaunchKernelGGL((linear_f32_kernel<T, O, MODE>), dim3(static_cast<unsigned>(want < most ? want : most)),
                     dim3(256), 0, s, p);
}

template <typename T>
void dispatch(const Linear &p, hipStream_t s) {
  if (p.mode == kLinForward) launch<float, float, kLinForward>(p, s);   // bf16: launch_grouped_gemm
  else if (p.mode == kLinInputGrad) launch<T, T, kLinInputGrad>(p, s);
  else if (p.out_bf16) launch<T, uint16_t, kLinWeightGrad>(p, s);
  else launch<T, float, kLinWeightGrad>(p, s);
}

}  // namespace

hipError_t launch_linear_f32(const Linear &p, hipStream_t s) {
  if (p.bf16) dispatch<uint16_t>(p, s);
  else dispatch<float>(p, s);
  return hipGetLastError();
}

}  // namespace moe
