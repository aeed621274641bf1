// Microscaled 4-bit floating point (MXFP4): quantisation of rows, and the
// grouped expert product of quantised rows.
//
// Format.  32 consecutive elements of a row form a block.  An element is an
// E2M1 code (sign, two exponent bits with bias 1, one mantissa bit: 0, 0.5,
// 1, 1.5, 2, 3, 4, 6 and their negatives), two codes to a byte with the
// even element in the low four bits; a block has one scale byte B that stands
// for 2^(B - 127), and 255 for NaN.  The scale is chosen as the FP8 dispatch
// chooses its own: 2^E with E the smallest integer for which no element has
// to be clipped, max|x| <= 6 * 2^E (E = 0 for a block of zeros, and E limited
// to the byte's range -127 .. 127).  Codes are x / 2^E, an exact quotient
// outside float32's subnormal range, rounded to nearest with ties to the even
// code.  A block that holds an infinity or a NaN has no such scale: its byte
// is 255 and its codes 0.
#include "moe_common.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));

// ---------------------------------------------------------------------------
// Quantisation
// ---------------------------------------------------------------------------

// Scale exponent of a block from the bits of its largest magnitude a > 0
// (float32, finite): a = m * 2^e with m in [0.5, 1) and 6 = 0.75 * 2^3, so
// E = e - 3 when m <= 0.75, else e - 2.  Subnormal a lies below 6 * 2^-127.
__device__ __forceinline__ int mx_exponent(uint32_t bits) {
  if (bits == 0) return 0;
  const int e = static_cast<int>(bits >> 23) - 126;
  const int E = (bits & 0x7FFFFFu) <= 0x400000u ? e - 3 : e - 2;
  return max(E, -127);
}

template <typename T> struct Unit;   // 8 elements of a row: one lane's share
template <> struct Unit<uint16_t> {
  uint4 v;
  __device__ __forceinline__ void load(const uint16_t *p) { v = *reinterpret_cast<const uint4 *>(p); }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      f[2 * j] = __uint_as_float(w[j] << 16);
      f[2 * j + 1] = __uint_as_float(w[j] & 0xFFFF0000u);
    }
  }
};
template <> struct Unit<float> {
  float4 a, b;
  __device__ __forceinline__ void load(const float *p) {
    a = *reinterpret_cast<const float4 *>(p);
    b = *reinterpret_cast<const float4 *>(p + 4);
  }
  __device__ __forceinline__ void get(float (&f)[8]) const {
    f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
    f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
  }
};

__device__ __forceinline__ void store_wide(uint16_t *p, const float (&f)[8]) {
  u32x4_t o;
#pragma unroll
  for (int j = 0; j < 4; ++j) o[j] = pack_bf16x2(f[2 * j], f[2 * j + 1]);
  __builtin_nontemporal_store(o, reinterpret_cast<u32x4_t *>(p));
}
__device__ __forceinline__ void store_wide(float *p, const float (&f)[8]) {
  f32x4_t a = {f[0], f[1], f[2], f[3]}, b = {f[4], f[5], f[6], f[7]};
  __builtin_nontemporal_store(a, reinterpret_cast<f32x4_t *>(p));
  __builtin_nontemporal_store(b, reinterpret_cast<f32x4_t *>(p) + 1);
}

// One lane takes 8 elements, four neighbouring lanes a block.  Outputs are
// dense, so they are addressed by the unit's number alone; only a row stride
// other than d needs the row, unit / (d / 8), as the high half of a product
// with magic = floor(2^64 / (d / 8)) + 1 (exact while units * d / 8 < 2^64).
template <typename T, bool STRIDED, bool WIDE>
__global__ __launch_bounds__(256) void quantize_mxfp4_kernel(
    const T *__restrict__ x, int64_t units, uint32_t upr, uint64_t magic, int64_t stride,
    uint32_t *__restrict__ codes, uint8_t *__restrict__ scales, T *__restrict__ wide) {
  const int64_t u = static_cast<int64_t>(blockIdx.x) * 256 + threadIdx.x;
  if (u >= units) return;              // units is a multiple of 4: whole blocks leave together
  const T *src = x + u * 8;
  if constexpr (STRIDED) {
    const uint64_t row = upr == 1 ? u : __umul64hi(u, magic);
    src = x + row * stride + (u - row * upr) * 8;
  }
  Unit<T> in;
  in.load(src);
  float f[8];
  in.get(f);
  uint32_t amax = 0;
#pragma unroll
  for (int j = 0; j < 8; ++j) amax = max(amax, __float_as_uint(f[j]) & 0x7FFFFFFFu);
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 1)));
  amax = max(amax, static_cast<uint32_t>(__shfl_xor(static_cast<int>(amax), 2)));
  const bool bad = amax >= 0x7F800000u;
  const int E = mx_exponent(amax);
  uint32_t c = 0;
  if (!bad) {
    float q[8];
#pragma unroll
    for (int j = 0; j < 8; ++j) q[j] = __builtin_ldexpf(f[j], -E);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[0], q[1], 1.0f, 0);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[2], q[3], 1.0f, 1);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[4], q[5], 1.0f, 2);
    c = __builtin_amdgcn_cvt_scalef32_pk_fp4_f32(c, q[6], q[7], 1.0f, 3);
  }
  codes[u] = c;
  if ((threadIdx.x & 3) == 0) scales[u >> 2] = static_cast<uint8_t>(bad ? 255 : E + 127);
  if constexpr (WIDE) {
    float o[8];
    const f32x2_t p0 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 0);
    const f32x2_t p1 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 1);
    const f32x2_t p2 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 2);
    const f32x2_t p3 = __builtin_amdgcn_cvt_scalef32_pk_f32_fp4(c, 1.0f, 3);
    const float v[8] = {p0.x, p0.y, p1.x, p1.y, p2.x, p2.y, p3.x, p3.y};
#pragma unroll
    for (int j = 0; j < 8; ++j) o[j] = bad ? __uint_as_float(0x7FC00000u) : __builtin_ldexpf(v[j], E);
    store_wide(wide + u * 8, o);
  }
}

template <typename T>
hipError_t quantize(const void *x, int64_t rows, int d, int64_t stride, uint8_t *codes,
                    uint8_t *scales, void *wide, hipStream_t s) {
  const int64_t units = rows * (d / 8);
  const uint32_t upr = static_cast<uint32_t>(d / 8);
  const uint64_t magic = upr > 1 ? ~uint64_t(0) / upr + 1 : 0;
  const dim3 grid(static_cast<unsigned>((units + 255) / 256));
  const bool strided = stride != d && rows > 1;
  auto go = [&](auto kernel) {
    hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s, static_cast<const T *>(x), units, upr, magic,
                       stride, reinterpret_cast<uint32_t *>(codes), scales, static_cast<T *>(wide));
    return hipGetLastError();
  };
  if (strided)
    return wide ? go(quantize_mxfp4_kernel<T, true, true>) : go(quantize_mxfp4_kernel<T, true, false>);
  return wide ? go(quantize_mxfp4_kernel<T, false, true>) : go(quantize_mxfp4_kernel<T, false, false>);
}

// ---------------------------------------------------------------------------
// Grouped product
// ---------------------------------------------------------------------------
constexpr int kMaxGroups = kMaxRouted + kMaxShared;

struct MxArgs {
  const uint8_t *x, *xs;         // rows of codes, rows of scale bytes
  const int32_t *index;          // source row of each row, or null
  const int32_t *offsets;
  const uint8_t *w, *ws;
  const uint16_t *bias;
  uint16_t *y;
  int groups, n_out, k;
};

// Group of tile mt from the tile prefix: largest g with pref[g] <= mt.
__device__ __forceinline__ int mx_find_group(const int *pref, int n, int mt) {
  int lo = 0, hi = n;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= mt) lo = mid; else hi = mid;
  }
  return lo;
}

// 16 rows x 64 features per wave, operands straight from memory: the 64 lanes
// of v_mfma_scale_f32_16x16x128_f8f6f4 hold 16 rows x four blocks of 32
// elements, each lane one block (16 bytes) and that block's scale byte.
template <bool SILU>
__global__ __launch_bounds__(256) void mx_linear_kernel(MxArgs a) {
  __shared__ int s_pref[kMaxGroups + 1];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  if (tid < 64) {
    int run = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      const int g = g0 + tid;
      const int n = g < a.groups ? (a.offsets[g + 1] - a.offsets[g] + 15) / 16 : 0;
      int incl = n;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
      }
      if (g < a.groups) s_pref[g] = run + incl - n;
      run += __shfl(incl, 63);
    }
    if (tid == 0) s_pref[a.groups] = run;
  }
  __syncthreads();
  const int tiles = s_pref[a.groups];
  const int r16 = lane & 15, q = lane >> 4;
  const int64_t kb = a.k / 2, ksb = a.k / 32;
  for (int mt = blockIdx.y; mt < tiles; mt += gridDim.y) {
    const int g = mx_find_group(s_pref, a.groups, mt);
    const int64_t first = a.offsets[g];
    const int64_t rows = a.offsets[g + 1] - first;
    const int64_t r0 = static_cast<int64_t>(mt - s_pref[g]) * 16;
    const int64_t rr = first + min(r0 + r16, rows - 1);
    const int64_t src = a.index ? static_cast<int64_t>(a.index[rr]) : rr;
    const uint8_t *xp = a.x + src * kb + q * 16, *xsp = a.xs + src * ksb + q;
    const int n0 = blockIdx.x * 256 + wave * 64;
    const uint8_t *wp[4], *wsp[4];
    f32x4_t acc[4] = {};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int64_t n = static_cast<int64_t>(g) * a.n_out + min(n0 + i * 16 + r16, a.n_out - 1);
      wp[i] = a.w + n * kb + q * 16;
      wsp[i] = a.ws + n * ksb + q;
    }
    for (int k = 0; k < a.k / 128; ++k) {
      const u32x4_t xv = *reinterpret_cast<const u32x4_t *>(xp + k * 64);
      const int sx = xsp[k * 4];
      const i32x8_t b = {(int)xv[0], (int)xv[1], (int)xv[2], (int)xv[3], 0, 0, 0, 0};
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const u32x4_t wv = *reinterpret_cast<const u32x4_t *>(wp[i] + k * 64);
        const int sw = wsp[i][k * 4];
        const i32x8_t w = {(int)wv[0], (int)wv[1], (int)wv[2], (int)wv[3], 0, 0, 0, 0};
        acc[i] = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(w, b, acc[i], 4, 4, 0, sw, 0, sx);
      }
    }
    if (r0 + r16 >= rows) continue;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int n = n0 + i * 16 + q * 4;
      if (n >= a.n_out) continue;
      float o[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        o[j] = acc[i][j];
        if (a.bias) o[j] += bf16_to_f32(a.bias[static_cast<int64_t>(g) * a.n_out + n + j]);
        if (SILU) o[j] = silu_fast(o[j]);
      }
      uint2 p;
      p.x = pack_bf16x2(o[0], o[1]);
      p.y = pack_bf16x2(o[2], o[3]);
      *reinterpret_cast<uint2 *>(a.y + (first + r0 + r16) * a.n_out + n) = p;
    }
  }
}

}  // namespace

hipError_t launch_quantize_mxfp4(bool bf16, const void *x, int64_t rows, int d, int64_t stride,
                                 uint8_t *codes, uint8_t *scales, void *wide, hipStream_t s) {
  return bf16 ? quantize<uint16_t>(x, rows, d, stride, codes, scales, wide, s)
              : quantize<float>(x, rows, d, stride, codes, scales, wide, s);
}

hipError_t launch_linear_mxfp4(const MxLinear &p, hipStream_t s) {
  MxArgs a{p.x, p.xs, p.index, p.offsets, p.w, p.ws, static_cast<const uint16_t *>(p.bias),
           static_cast<uint16_t *>(p.y), p.groups, p.n_out, p.k};
  const int64_t tiles = p.max_rows / 16 + (p.max_rows < p.groups ? p.max_rows : p.groups) + 1;
  const dim3 grid((p.n_out + 255) / 256, static_cast<unsigned>(tiles < 2048 ? tiles : 2048));
  if (p.silu)
    hipLaunchKernelGGL(mx_linear_kernel<true>, grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL(mx_linear_kernel<false>, grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

size_t linear_mxfp4_workspace_bytes(int, int, int, int64_t) { return 0; }

}  // namespace moe
