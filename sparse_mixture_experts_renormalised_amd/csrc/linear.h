// Launchers of the single Linears of every expert and of their gradients
// (linear.hip, linear_mfma.hip).  Not part of the public interface.
#pragma once

#include "moe_common.h"

namespace moe {

// Three products of the rows offsets[g] .. offsets[g+1]-1 of every group:
//   kLinForward     y[r]    = act(x[index[r]] W_g^T + bias_g)
//   kLinInputGrad   dx[r]   = (dy[r] W_g) silu'(pre[r])
//   kLinWeightGrad  dW_g (+)= sum_r dy[r]^T x[index[r]],  dbias_g (+)= sum_r dy[r]
enum LinearMode { kLinForward, kLinInputGrad, kLinWeightGrad };

struct Linear {
  LinearMode mode;
  bool bf16;                    // type of rows and weights
  bool out_bf16;                // type of dw and dbias
  const int32_t *offsets;       // [groups + 1], device
  int groups, n_out, k;
  int64_t max_rows;             // host upper bound on offsets[groups]
  int64_t x_rows;               // rows of x
  const void *x;                // forward, weight gradient: [x_rows][k]
  const int32_t *index;         // row r reads x[index[r]] (null: r)
  const void *dy;               // gradients: [max_rows][n_out]
  const void *w;                // [groups][n_out][k]
  const void *bias;             // [groups][n_out] or null
  bool silu;
  void *pre;                    // forward: values before the SiLU, or null
  const void *act_pre;          // input gradient: values before the SiLU that made x, or null
  void *out;                    // y, dx or dw
  void *dbias;                  // [groups][n_out] or null
  bool accumulate;              // add to dw and dbias
};

// float32 (all three) and the bf16 gradients that linear_mfma_fits leaves to it; ws:
// linear_f32_workspace_bytes of scratch.
size_t linear_f32_workspace_bytes(int groups, int n_out, int k, int64_t max_rows);
hipError_t launch_linear_f32(const Linear &p, void *ws, hipStream_t s);

// bf16 operands, where linear_mfma_fits: 32-bit offsets, gradients with more than a little
// to do, the forward where the layer's kernels would be slower; ws: linear_mfma_workspace_bytes of scratch.
bool linear_mfma_fits(const Linear &p);
size_t linear_mfma_workspace_bytes(int groups, int n_out, int k, int64_t max_rows);
hipError_t launch_linear_mfma(const Linear &p, void *ws, hipStream_t s);

// Derivative of z sigmoid(z): s + z s (1 - s), with the hardware exp2 and reciprocal
// (about 1 ulp each), for outputs that round to bfloat16: rounding the exponent alone costs
// |z| 2^-24 of the value.
__device__ __forceinline__ float silu_slope(float z) {
  const float s = __builtin_amdgcn_rcpf(1.0f + __builtin_amdgcn_exp2f(-z * 1.4426950408889634f));
  return fmaf(s, fmaf(-z, s, z), s);
}

// The SiLU and its derivative for float32 outputs, from e = exp(-|z|) and d = 1 / (1 + e):
// sigmoid(z) is d for z >= 0 and e d below, and 1 - sigmoid(z) the other of the two.  e is
// 2^n 2^f with a remainder f that two fused products leave exact to 2^-26, and reaches below
// the normal numbers; d is the hardware's reciprocal and a Newton step (the library's expf and
// division take the small float32 Linear from 14.6 us to 15.4, the fast exponential, off by
// |z| 2^-24, to 14.3).
struct SiluParts {
  float e, d;
};
__device__ __forceinline__ SiluParts silu_parts(float z) {
  const float v = -fminf(fabsf(z), 256.0f);   // e is 0 from 104 on
  const float n = rintf(v * 1.4426950408889634f);
  const float f = fmaf(v, 1.925962991e-8f, fmaf(v, 1.4426950216293335f, -n));   // log2(e) in two parts
  SiluParts p;
  p.e = ldexpf(__builtin_amdgcn_exp2f(f), static_cast<int>(n));
  const float r = __builtin_amdgcn_rcpf(1.0f + p.e);
  p.d = fmaf(fmaf(-(1.0f + p.e), r, 1.0f), r, r);
  return p;
}
__device__ __forceinline__ float silu_f32(float z) {
  const SiluParts p = silu_parts(z);
  return (z >= 0.0f ? z : z * p.e) * p.d;
}
__device__ __forceinline__ float silu_slope_f32(float z) {
  const SiluParts p = silu_parts(z);
  const float ed = p.e * p.d;
  return z >= 0.0f ? p.d * fmaf(z, ed, 1.0f) : ed * fmaf(z, p.d, 1.0f);
}

}  // namespace moe
