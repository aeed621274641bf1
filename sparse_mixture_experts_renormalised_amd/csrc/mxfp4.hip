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
#include "lds_dma.h"
#include "moe_common.h"

namespace moe {
namespace {

typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));
typedef float f32x4_t __attribute__((ext_vector_type(4)));
typedef int i32x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));

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

// A launch has fewer than 2^32 lanes: at most kLaunchUnits each, whole rows.
constexpr int64_t kLaunchUnits = int64_t(1) << 30;

template <typename T>
hipError_t quantize(const void *x, int64_t rows, int d, int64_t stride, uint8_t *codes,
                    uint8_t *scales, void *wide, hipStream_t s) {
  const uint32_t upr = static_cast<uint32_t>(d / 8);
  const uint64_t magic = upr > 1 ? ~uint64_t(0) / upr + 1 : 0;
  const bool strided = stride != d && rows > 1;
  const int64_t most = kLaunchUnits / upr;               // 4 or more: d < 2^31
  for (int64_t r = 0; r < rows; r += most) {
    const int64_t units = (rows - r < most ? rows - r : most) * upr;
    const dim3 grid(static_cast<unsigned>((units + 255) / 256));
    auto go = [&](auto kernel) {
      hipLaunchKernelGGL(kernel, grid, dim3(256), 0, s,
                         static_cast<const T *>(x) + r * (strided ? stride : d), units, upr, magic, stride,
                         reinterpret_cast<uint32_t *>(codes) + r * upr, scales + r * (upr / 4),
                         wide ? static_cast<T *>(wide) + r * d : nullptr);
      return hipGetLastError();
    };
    const hipError_t e =
        strided ? (wide ? go(quantize_mxfp4_kernel<T, true, true>) : go(quantize_mxfp4_kernel<T, true, false>))
                : (wide ? go(quantize_mxfp4_kernel<T, false, true>)
                        : go(quantize_mxfp4_kernel<T, false, false>));
    if (e != hipSuccess) return e;
  }
  return hipSuccess;
}

// ---------------------------------------------------------------------------
// Grouped product: y[r, n] = act(sum_k X[r, k] W_g[n, k] + bias_g[n]).
//
// Both operands enter the scaled matrix instructions as they lie in memory:
// v_mfma_scale_f32_*_f8f6f4 multiplies 4-bit codes, applies each block's two
// scale bytes and adds in float32, so nothing is widened.  Weights are the
// first operand, so a lane ends up with four consecutive features of a row.
//
// Two ways, in one kernel where only the device can choose (a kernel each would
// cost every call a launch, 3 us or more):
//   * tiles of 256 x 256 (128 x 256 and 64 x 256 for a group's last rows),
//     operands through LDS, one workgroup a CU: every group, where there are
//     tiles for most of the CUs, and else the groups of more than kStreamRows
//     rows;
//   * else the groups of up to kStreamRows rows: units of 16 features, operands
//     straight from memory to registers, which a few groups have enough of.
// Measured on MI355X: 256 groups, 207 rows in about 84 of them, 7168 -> 2048:
// 115 us, 5.7 TB/s (134 us straight from memory); 64 groups, 32768 rows, 2048 ->
// 1408 with SiLU: 93 us; 256 groups, 32768 rows, 2048 -> 7168: 581 us, 4.3 TB/s;
// 8 groups, 8192 rows, 4096 -> 14336 with bias and SiLU: 340 us, 2.8 PFLOP/s.  Cards
// differ by up to 8 %; the figures below compare two forms on one card each.
// ---------------------------------------------------------------------------
constexpr int kMaxGroups = kMaxRouted + kMaxShared;
constexpr int kXcds = 8;
constexpr int kStreamRows = 64;
namespace tile {
constexpr int BN = 256;                // features of a tile
}

struct MxArgs {
  const uint8_t *x, *xs;         // rows of codes, rows of scale bytes
  const int32_t *index;          // source row of each row, or null
  const int32_t *offsets;
  const uint8_t *w, *ws;
  const uint16_t *bias;
  uint16_t *y;
  int groups, n_out, k;
};

__device__ __forceinline__ int64_t source_row(const MxArgs &a, int64_t r) {
  return a.index ? static_cast<int64_t>(a.index[r]) : r;
}

__device__ __forceinline__ i32x8_t codes32(u32x4_t v) {
  return i32x8_t{(int)v[0], (int)v[1], (int)v[2], (int)v[3], 0, 0, 0, 0};
}

// 256-row tiles of a group and the height of the tile that takes what is left:
// 0, 64 or 128 (a remainder above 128 rows is a full tile).
__device__ __forceinline__ int mx_full_tiles(int rows, int *tail) {
  const int r = rows % 256;
  *tail = r == 0 || r > 128 ? 0 : r <= 64 ? 64 : 128;
  return rows / 256 + (r > 128 ? 1 : 0);
}

// The least number of rows that a group taken in tiles has: 1 if the tiles of all
// groups fill the chip, tiles of more than 16 rows counting twice, else
// kStreamRows + 1.  Timed with 1, 16, 17 and 64 rows a group, straight from memory
// and in tiles (us):
//   7168 -> 2048   64 tiles  15  22  24  40    33  35  35  38
//                 128        27  36  37  61    36  37  37  40
//                 192        39  52  55  94    38  39  39  43
//                 512        88 119 121 218    81  83  83  91
//   2048 -> 1408   66 tiles 9.5  11  12  19    13  13  13  15
//                 126        11  15  15  26    13  14  14  15
//                 192        15  19  20  33    14  15  15  16
//                 510        33  38  40  69    28  28  29  31
//   2048 -> 7168   56 tiles 8.8 9.0 9.6  19    13  13  13  14
//                 140        13  18  19  29    14  14  14  15
//                 196        18  21  22  36    15  15  15  16
//                 504        31  39  41  70    30  30  30  33
// So the rule takes the faster way but for groups of 16 and of 64 rows somewhat below
// the border (140 tiles of 16 rows: 18 us for 14; 66 of 64: 19 for 15).
constexpr int kFill = 192;
struct Plan {
  int least;                           // of the groups taken in tiles
  bool tiles, units;                   // is there any work of either kind
};
// Also copies the groups' row counts into LDS.  Every thread calls it.
__device__ __forceinline__ Plan mx_plan(const MxArgs &a, int tiles_wide, int threads, int *s_rows,
                                        int (&s_plan)[3]) {
  if (threadIdx.x < 3) s_plan[threadIdx.x] = 0;
  __syncthreads();
  int sum = 0;
  bool big = false, small = false;
  for (int g = threadIdx.x; g < a.groups; g += threads) {
    const int rows = a.offsets[g + 1] - a.offsets[g];
    int tail;
    const int n = mx_full_tiles(rows, &tail) + (tail ? 1 : 0);
    sum += rows <= 16 ? n : 2 * n;
    big |= rows > kStreamRows;
    small |= rows > 0 && rows <= kStreamRows;
    s_rows[g] = rows;
  }
#pragma unroll
  for (int off = 32; off; off >>= 1) sum += __shfl_xor(sum, off);
  big = __ballot(big) != 0;
  small = __ballot(small) != 0;
  if ((threadIdx.x & 63) == 0) {
    atomicAdd(&s_plan[0], sum);
    if (big) s_plan[1] = 1;
    if (small) s_plan[2] = 1;
  }
  __syncthreads();
  const bool all = uniform(s_plan[0]) >= (kFill + tiles_wide - 1) / tiles_wide;
  return Plan{all ? 1 : kStreamRows + 1, all || uniform(s_plan[1]), !all && uniform(s_plan[2])};
}

// ---- few rows ----
// A wave takes units of 16 features over the whole reduction axis, reading the
// weights straight into the operand registers of 16x16x128 instructions, 16
// bytes (one block) a lane and several chunks ahead.  A chunk is what the 16
// lanes of a row read together: 16 blocks, 512 elements.  So that neighbouring
// lanes read neighbouring bytes (in the instruction's own order they belong to
// different rows, and the addresses of a load are then looked up one by one, 64
// clocks instead of 16), load r of a lane (a, b, q) is block 4 q + b of row
// 4 r + a, four rows a load.  From there
//   * up to 16 rows of X: rows (a, b) x columns (row t of four, b') with
//       A[(a, b)][q] = W[4 r + a][block 4 q + b],  B[q][(t, b')] = X[t][block 4 q + b'],
//     of whose 16 x 16 results those with b = b' are of use and the four of
//     them add up: no data moves, and one, two or four instructions a load;
//   * up to 64: the loads r and lanes b are transposed, which gives sixteen
//     whole rows for four instructions, W's and X's alike.
namespace stream {
constexpr int R = 4, UN = 4 * R;

// Operands that MODE columns take: MODE 1, 2, 4 fours of rows (diagonal), or 8
// and 16: two and four tiles of 16 (transposed).
template <int MODE> constexpr bool kTurn = MODE >= 8;
template <int MODE> constexpr int kLoadsB = MODE;                           // 16-byte loads of X
template <int MODE> constexpr int kScalesB = kTurn<MODE> ? MODE / 4 : MODE;  // and of its scales
template <int MODE> constexpr int kDepth = MODE == 1 ? 6 : MODE == 2 ? 5 : MODE == 16 ? 2 : 3;

// 4 x 4 transpose between four registers and four neighbouring lanes.
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
__device__ __forceinline__ void transpose4(u32x4_t *v, bool odd, bool high) {
#pragma unroll
  for (int w = 0; w < 4; ++w) {
    uint32_t x[4] = {v[0][w], v[1][w], v[2][w], v[3][w]};
    transpose4(x, odd, high);
#pragma unroll
    for (int r = 0; r < 4; ++r) v[r][w] = x[r];
  }
}

// acc += A B with the scale bytes J of both.
template <int J>
__device__ __forceinline__ void product(f32x4_t &acc, u32x4_t a, u32x4_t b, int sa, int sb) {
  acc = __builtin_amdgcn_mfma_scale_f32_16x16x128_f8f6f4(codes32(a), codes32(b), acc, 4, 4, J, sa, J, sb);
}

// Units u0 .. u0 + count - 1 of a group whose rows first .. first + rows - 1 fit MODE.
template <int MODE, bool SILU>
__device__ __forceinline__ void run(const MxArgs &a, int g, int64_t first, int rows, int u0, int count) {
  constexpr int D = kDepth<MODE>, NB = kLoadsB<MODE>, NS = kScalesB<MODE>, NA = kTurn<MODE> ? MODE / 4 : R * MODE;
  const int lane = threadIdx.x & 63;
  const int b = lane & 3, ar = (lane >> 2) & 3, q = lane >> 4, piece = q * 4 + b;
  const int pieces = a.k / 32, nch = (pieces + 15) >> 4, tail = pieces & 15;
  const uint8_t *w = a.w + static_cast<int64_t>(g) * a.n_out * pieces * 16;
  const uint8_t *ws = a.ws + static_cast<int64_t>(g) * a.n_out * pieces;
  // blocks before this lane's row of X in each load, and its scale row
  uint32_t bo[NB], bso[NS];
#pragma unroll
  for (int i = 0; i < NB; ++i) {
    // columns 4 i + ar (diagonal), or row 4 r + ar of tile i / 4
    const int r = min(i * 4 + ar, rows - 1);
    bo[i] = static_cast<uint32_t>(source_row(a, first + r)) * pieces;
  }
#pragma unroll
  for (int i = 0; i < NS; ++i) {
    if (!kTurn<MODE>) {
      bso[i] = bo[i];
    } else {
      const int r = min(i * 16 + b * 4 + ar, rows - 1);     // row of the turned column
      bso[i] = static_cast<uint32_t>(source_row(a, first + r)) * pieces;
    }
  }
  f32x4_t acc[NA];
#pragma unroll
  for (int i = 0; i < NA; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
  struct Stage {
    u32x4_t a[R], b[NB];
    int sa[kTurn<MODE> ? 1 : R], sb[NS];
  } st[D];
  int fu = u0, fc = 0, uu = u0, uc = 0;         // unit and chunk of the next fetch, of the next use
  auto fetch = [&](Stage &s) {
    const uint32_t at = min(fc * 16 + piece, pieces - 1), at4 = min(fc * 16 + q * 4, pieces - 4);
#pragma unroll
    for (int i = 0; i < NB; ++i) s.b[i] = *reinterpret_cast<const u32x4_t *>(a.x + (bo[i] + at) * 16);
#pragma unroll
    for (int i = 0; i < NS; ++i)
      s.sb[i] = kTurn<MODE> ? *reinterpret_cast<const int *>(a.xs + (bso[i] + at4)) : a.xs[bso[i] + at];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      const uint32_t row = min(fu * UN + r * 4 + ar, a.n_out - 1) * pieces;
      s.a[r] = __builtin_nontemporal_load(     // read once
          reinterpret_cast<const u32x4_t *>(w + (row + at) * 16));
      if (!kTurn<MODE>) s.sa[r] = ws[row + at];
    }
    if (kTurn<MODE>)
      s.sa[0] = *reinterpret_cast<const int *>(
          ws + (static_cast<uint32_t>(min(fu * UN + b * 4 + ar, a.n_out - 1)) * pieces + at4));
    if (++fc == nch) {
      fc = 0;
      ++fu;
    }
  };
  auto finish = [&]() {
    const int64_t gn = static_cast<int64_t>(g) * a.n_out;
    if constexpr (!kTurn<MODE>) {
      // register i of a lane: entry ((row q, block i), (column ar, block b)) of load
      // r; take i = b, add the four lanes b, and let lane b keep load b
#pragma unroll
      for (int t = 0; t < MODE; ++t) {
        float z = 0.0f;
#pragma unroll
        for (int r = 0; r < R; ++r) {
          const f32x4_t v = acc[r * MODE + t];
          float x = b == 0 ? v[0] : b == 1 ? v[1] : b == 2 ? v[2] : v[3];
          x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0xB1, 0xF, 0xF, true));
          x += __uint_as_float(__builtin_amdgcn_mov_dpp(__float_as_uint(x), 0x4E, 0xF, 0xF, true));
          z = b == r ? x : z;
        }
        const int n = uu * UN + b * 4 + q, row = t * 4 + ar;
        if (row < rows && n < a.n_out) {
          if (a.bias) z += bf16_to_f32(a.bias[gn + n]);
          if (SILU) z = silu_fast(z);
          a.y[(first + row) * a.n_out + n] = f32_to_bf16(z);
        }
      }
    } else {
      // register i of a lane: feature 4 i + q, column lane % 16, which is row
      // 4 b + ar; turned so that a lane holds features 4 q .. 4 q + 3
#pragma unroll
      for (int c = 0; c < NA; ++c) {
        uint32_t v[4] = {__float_as_uint(acc[c][0]), __float_as_uint(acc[c][1]),
                         __float_as_uint(acc[c][2]), __float_as_uint(acc[c][3])};
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
        const int n = uu * UN + q * 4, row = c * 16 + b * 4 + ar;
        if (row < rows && n < a.n_out) {
          float z[4];
#pragma unroll
          for (int x = 0; x < 4; ++x) {
            z[x] = __uint_as_float(v[x]);
            if (a.bias) z[x] += bf16_to_f32(a.bias[gn + n + x]);
            if (SILU) z[x] = silu_fast(z[x]);
          }
          uint2 o;
          o.x = pack_bf16x2(z[0], z[1]);
          o.y = pack_bf16x2(z[2], z[3]);
          *reinterpret_cast<uint2 *>(a.y + (first + row) * a.n_out + n) = o;
        }
      }
    }
#pragma unroll
    for (int i = 0; i < NA; ++i) acc[i] = f32x4_t{0, 0, 0, 0};
  };
  auto use = [&](Stage &s) {
    if (tail && uc == nch - 1) {
      // past the end of a row both sides hold its last block: X's count as zeros
      const bool past = piece >= tail;
#pragma unroll
      for (int i = 0; i < NB; ++i)
#pragma unroll
        for (int x = 0; x < 4; ++x) s.b[i][x] = past ? 0u : s.b[i][x];
    }
    if constexpr (!kTurn<MODE>) {
#pragma unroll
      for (int r = 0; r < R; ++r)
#pragma unroll
        for (int t = 0; t < MODE; ++t) product<0>(acc[r * MODE + t], s.a[r], s.b[t], s.sa[r], s.sb[t]);
    } else {
      transpose4(s.a, b & 1, b & 2);
#pragma unroll
      for (int c = 0; c < NA; ++c) {
        transpose4(s.b + c * 4, b & 1, b & 2);
        product<0>(acc[c], s.a[0], s.b[c * 4 + 0], s.sa[0], s.sb[c]);
        product<1>(acc[c], s.a[1], s.b[c * 4 + 1], s.sa[0], s.sb[c]);
        product<2>(acc[c], s.a[2], s.b[c * 4 + 2], s.sa[0], s.sb[c]);
        product<3>(acc[c], s.a[3], s.b[c * 4 + 3], s.sa[0], s.sb[c]);
      }
    }
    // done here, not later, or the operands outlive the next loads
#pragma unroll
    for (int i = 0; i < NA; ++i) asm volatile("" : "+v"(acc[i]));
    if (++uc == nch) {
      finish();
      uc = 0;
      ++uu;
    }
  };
  const int n = count * nch;
  if (n < D) {
    for (int k = 0; k < n; ++k) {
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
}
}  // namespace stream

// What a unit of a group of `rows` rows takes, in quarters of one of a few rows
// (0: not this kernel's): with more rows X takes more registers and fewer chunks
// are in flight.
__device__ __forceinline__ int mx_unit_cost(int rows) {
  return rows <= 0 || rows > kStreamRows ? 0 : rows <= 8 ? 4 : rows <= 16 ? 5 : rows <= 32 ? 7 : 10;
}

// Every wave takes a range of equal cost of the units of all groups of up to
// kStreamRows rows: those whose first quarter lies in it.
template <bool SILU>
__device__ __forceinline__ void mx_units(const MxArgs &a, const int *s_rows, int64_t *s_pref) {
  using namespace stream;
  const int tid = threadIdx.x, lane = tid & 63;
  const int per = (a.n_out + UN - 1) / UN;
  if (tid < 64) {
    int64_t base = 0;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      const int g = g0 + lane;
      const int c = g < a.groups ? mx_unit_cost(s_rows[g]) : 0;
      int incl = c;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (lane >= off) incl += o;
      }
      if (g < a.groups) s_pref[g] = base + static_cast<int64_t>(incl - c) * per;
      base += static_cast<int64_t>(__shfl(incl, 63)) * per;
    }
    if (tid == 0) s_pref[a.groups] = base;
  }
  __syncthreads();
  const int64_t total = s_pref[a.groups];
  const int mine = blockDim.x / 64, v = blockIdx.x * mine + uniform(tid >> 6), waves = gridDim.x * mine;
  const int64_t lo = total * v / waves, hi = total * (v + 1) / waves;
  if (lo >= hi) return;
  int g = 0, up = a.groups;                // s_pref[g] <= lo < s_pref[up]
  while (up - g > 1) {
    const int mid = (g + up) >> 1;
    if (s_pref[mid] <= lo) g = mid; else up = mid;
  }
  for (; g < a.groups && s_pref[g] < hi; ++g) {
    const int ug = uniform(g);
    const int first = uniform(a.offsets[ug]), rows = uniform(a.offsets[ug + 1]) - first;
    const int cost = mx_unit_cost(rows);
    if (cost == 0) continue;
    const int64_t base = s_pref[ug];
    const int u0 = uniform(static_cast<int>(max(int64_t(0), (lo - base + cost - 1) / cost)));
    const int u1 = uniform(static_cast<int>(min(static_cast<int64_t>(per), (hi - base + cost - 1) / cost)));
    if (u0 >= u1) continue;
    if (rows <= 4) run<1, SILU>(a, ug, first, rows, u0, u1 - u0);
    else if (rows <= 8) run<2, SILU>(a, ug, first, rows, u0, u1 - u0);
    else if (rows <= 16) run<4, SILU>(a, ug, first, rows, u0, u1 - u0);
    else if (rows <= 32) run<8, SILU>(a, ug, first, rows, u0, u1 - u0);
    else run<16, SILU>(a, ug, first, rows, u0, u1 - u0);
  }
}

// Where the host knows that there are units alone, in smaller workgroups: a few
// units then lie on more CUs, and the loads of the chunks ahead keep all registers
// (8 groups, 7168 -> 2048, 1 and 8 rows each: 15 and 17 us, and 21 and 23 in the
// kernel below; one group of 64 rows 30 and 52).
constexpr int kUnitWaves = 4;
template <bool SILU>
__global__ __launch_bounds__(kUnitWaves * 64, 2) void mx_units_kernel(MxArgs a) {
  __shared__ int64_t s_pref[kMaxGroups + 1];
  __shared__ int s_rows[kMaxGroups];
  for (int g = threadIdx.x; g < a.groups; g += kUnitWaves * 64) s_rows[g] = a.offsets[g + 1] - a.offsets[g];
  __syncthreads();
  mx_units<SILU>(a, s_rows, s_pref);
}

// ---- many rows ----
// Tiles of BM rows x 256 features, eight waves of BM/2 x 64 (TM x 2 blocks of
// 32 x 32), two on every SIMD so that one's LDS reads and epilogue arithmetic run
// beside the other's matrix instructions (four waves of BM/2 x 128 read a third
// less LDS and took 115, 620 and 362 us where these took 101, 571 and 334).  A
// step of 256 elements is 128 bytes per row; two LDS buffers hold the steps'
// codes.  Half a step's fragments are read while the other half is multiplied,
// and once every wave holds the second half the copies of the step after next
// take the buffer, spread among that half's matrix instructions.  The scale bytes
// come in pairs of steps (16 bytes per row), in two LDS buffers of their own.
//
// What bounds it: with every tile's first copies and its stores between two tiles'
// steps, memory and matrix units wait for each other at the ends of a tile (the
// last of the cases above without the epilogue: 25 % less).  Copies of the next
// tile's first step under the epilogue took longer all the same, as the second
// step's then wait for the stores (111, 603 and 377 us), and so did two
// workgroups a CU with 128 x 256 tiles, which read half a line at a time (101, 681
// and 414 us).
//
// 16-byte chunk c of tile row r lies at position c ^ ((r / 2) % 8) of its
// 128-byte row, so that the 16 rows read together cover all banks once.
namespace tile {
constexpr int NT = 512, NS = 2, TN = 2, BUF = 2 * 512 * 128, SBUF = 512 * 16;

__device__ __forceinline__ int swz(int r, int c) { return c ^ ((r >> 1) & 7); }

// Workgroup barrier that waits for this wave's LDS reads; matrix instructions
// may move across it.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
}

// ONCE: no other tile reads these weights (a group's last rows), which then go past
// the caches; weights of full tiles and of their halves mostly serve several.
template <int BM, bool ONCE = (BM < 256)>
struct Tile {
  static constexpr int TM = BM / 64, AC = BM / 64, BC = 4, NCP = AC + BC;   // code copies per wave
  static constexpr int SC = 2, N = NCP + SC;                                // scale, all copies
  static constexpr int STEP = (BM + BN) * 128, SPAIR = 512 * 16;            // LDS bytes
  static constexpr int MF = NS * TN * TM;

  // Byte offsets of this lane's part of each copy, from wave-uniform bases (the
  // host refuses operands of 4 GiB or more), at step 0.
  struct Src {
    uint32_t a[AC], b[BC];     // 16-byte chunks of X and W rows
    uint32_t sa[SC], sb[SC];   // their scale rows
    const uint8_t *abase, *bbase, *sabase, *sbbase;
    int tadj;                  // byte correction of this lane in a half last step
    int nk, nd;                // steps, 128-element units
  };
  struct Frags {
    u32x4_t a[NS][TM], b[NS][TN];
  };
  struct Scales {
    uint32_t a[TM], b[TN];     // byte ks: scale of this lane's block of slice ks
  };
  using Acc = f32x16_t[TN][TM];

  static __device__ __forceinline__ void source(const MxArgs &a, int g, int64_t first, int64_t row0,
                                                int64_t rows, int n0, int tid, Src &s) {
    const int64_t kb = a.k / 2, ksb = a.k / 32;
    const int c = (tid & 7) ^ ((tid >> 4) & 7);       // row = tid/8 + 32i
    // scale copy j of wave w: rows 16 (w + 8 j) .. +15, four lanes of 4 bytes a
    // row (rows past the tile repeat the last one, here and for the codes)
    const int sr = (tid >> 6) * 16 + ((tid & 63) >> 2);
    int64_t ra[AC], rs[SC];
#pragma unroll
    for (int i = 0; i < AC; ++i) ra[i] = first + min(row0 + (tid >> 3) + i * 64, rows - 1);
#pragma unroll
    for (int j = 0; j < SC; ++j) rs[j] = first + min(row0 + sr + j * 128, rows - 1);
    if (a.index) {
#pragma unroll
      for (int i = 0; i < AC; ++i) ra[i] = a.index[ra[i]];
#pragma unroll
      for (int j = 0; j < SC; ++j) rs[j] = a.index[rs[j]];
    }
#pragma unroll
    for (int i = 0; i < AC; ++i) s.a[i] = static_cast<uint32_t>(ra[i] * kb) + c * 16;
    s.abase = a.x;
    s.sabase = a.xs;
    s.sbbase = a.ws + static_cast<int64_t>(g) * a.n_out * ksb;
    s.bbase = a.w + static_cast<int64_t>(g) * a.n_out * kb;
#pragma unroll
    for (int i = 0; i < BC; ++i)
      s.b[i] = static_cast<uint32_t>(min(n0 + (tid >> 3) + i * 64, a.n_out - 1)) *
                   static_cast<uint32_t>(kb) + c * 16;
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      s.sa[j] = static_cast<uint32_t>(rs[j] * ksb);
      s.sb[j] = static_cast<uint32_t>(min(n0 + sr + j * 128, a.n_out - 1)) * static_cast<uint32_t>(ksb);
    }
    s.nd = a.k / 128;
    s.nk = (s.nd + 1) / 2;
    s.tadj = (s.nd & 1) && c >= 4 ? -64 : 0;
  }

  // Byte offset of step kb for this lane; a half last step reads its first
  // half twice (the second is not multiplied).
  static __device__ __forceinline__ int step_off(const Src &s, int kb) {
    return kb * 128 + (kb == s.nk - 1 ? s.tadj : 0);
  }
  // Of the cases above, the first takes 127 us with the last rows' weights in the caches
  // (116), the third 582 (573); the second 101 with full tiles' weights past them (98),
  // and 91 with their halves' (90).
  static __device__ __forceinline__ void copy(const Src &s, int i, int off, uint32_t base, int wave) {
    if (i < AC) dma::dma16s(s.a[i] + off, s.abase, base + (8 * i + wave) * 1024);
    else if (ONCE) dma::dma16s_nt(s.b[i - AC] + off, s.bbase, base + BM * 128 + (8 * (i - AC) + wave) * 1024);
    else dma::dma16s(s.b[i - AC] + off, s.bbase, base + BM * 128 + (8 * (i - AC) + wave) * 1024);
  }
  // Scale copies: the rows of X (which 0) or W (1) for the steps 2p and 2p + 1.
  static __device__ __forceinline__ int pair_off(const Src &s, int p, int lane) {
    return min(4 * p + (lane & 3), s.nd - 1) * 4;
  }
  static __device__ __forceinline__ void scale_copy(const Src &s, int j, bool of_w, int off,
                                                    uint32_t base, int wave) {
    dma::dma4s((of_w ? s.sb[j] : s.sa[j]) + off, of_w ? s.sbbase : s.sabase,
               base + (of_w ? 256 * 16 : 0) + (8 * j + wave) * 256);
  }

  // Scales of a step: lane half h takes block 2 ks + h in slice ks, so of the
  // row's eight scale bytes it keeps the even or the odd four.
  static __device__ __forceinline__ void scales(const uint8_t *sbuf, int half, Scales &f, int wm, int wn,
                                                int lane) {
    const int h = lane >> 5, r32 = lane & 31;
    const uint32_t pick = h ? 0x07050301u : 0x06040200u;
#pragma unroll
    for (int mi = 0; mi < TM; ++mi) {
      const int row = wm * (BM / 2) + mi * 32 + r32;
      const uint2 sv = *reinterpret_cast<const uint2 *>(sbuf + row * 16 + half * 8);
      f.a[mi] = __builtin_amdgcn_perm(sv.y, sv.x, pick);
    }
#pragma unroll
    for (int ni = 0; ni < TN; ++ni) {
      const int row = 256 + wn * 64 + ni * 32 + r32;
      const uint2 sv = *reinterpret_cast<const uint2 *>(sbuf + row * 16 + half * 8);
      f.b[ni] = __builtin_amdgcn_perm(sv.y, sv.x, pick);
    }
  }
  // Fragments of the slices 2 H and 2 H + 1 of a step.
  template <int H>
  static __device__ __forceinline__ void read(const uint8_t *buf, Frags &f, int wm, int wn, int lane) {
    const int h = lane >> 5, r32 = lane & 31;
#pragma unroll
    for (int ks = 0; ks < NS; ++ks) {
      const int c = (2 * H + ks) * 2 + h;
#pragma unroll
      for (int mi = 0; mi < TM; ++mi) {
        const int row = wm * (BM / 2) + mi * 32 + r32;
        f.a[ks][mi] = *reinterpret_cast<const u32x4_t *>(buf + row * 128 + swz(row, c) * 16);
      }
#pragma unroll
      for (int ni = 0; ni < TN; ++ni) {
        const int row = wn * 64 + ni * 32 + r32;
        f.b[ks][ni] =
            *reinterpret_cast<const u32x4_t *>(buf + BM * 128 + row * 128 + swz(row, c) * 16);
      }
    }
  }

  // Matrix instructions M0 .. M1-1 of half a step, in (slice, ni, mi) order.
  template <int H, int M0, int M1>
  static __device__ __forceinline__ void mfma(const Frags &f, const Scales &c, Acc &acc) {
    if constexpr (M0 < M1) {
      constexpr int ks = M0 / (TN * TM), ni = (M0 / TM) % TN, mi = M0 % TM;
      acc[ni][mi] = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(
          codes32(f.b[ks][ni]), codes32(f.a[ks][mi]), acc[ni][mi], 4, 4, 2 * H + ks, c.b[ni], 2 * H + ks,
          c.a[mi]);
      mfma<H, M0 + 1, M1>(f, c, acc);
    }
  }

  // Copies I.. of a step spread over three quarters of its second half.
  template <int I>
  static __device__ __forceinline__ void copies_mfmas(const Src &s, int off, bool of_w, int soff,
                                                      uint32_t base, uint32_t sbase, int wave,
                                                      const Frags &f, const Scales &c, Acc &acc) {
    if constexpr (I < N) {
      constexpr int M3 = MF / 4 * 3;
      if constexpr (I < NCP) copy(s, I, off, base, wave);
      else scale_copy(s, I - NCP, of_w, soff, sbase, wave);
      mfma<1, I * M3 / N, (I + 1) * M3 / N>(f, c, acc);
      __builtin_amdgcn_sched_barrier(0);
      copies_mfmas<I + 1>(s, off, of_w, soff, base, sbase, wave, f, c, acc);
    }
  }

  static __device__ __forceinline__ void body(const Src &s, uint8_t *buf, uint8_t *sbuf, Acc &acc,
                                              int wave, int wm, int wn, int lane) {
#pragma unroll
    for (int i = 0; i < TN; ++i)
#pragma unroll
      for (int j = 0; j < TM; ++j)
#pragma unroll
        for (int r = 0; r < 16; ++r) acc[i][j][r] = 0.0f;
    const uint32_t b0 = uniform(static_cast<int>(dma::lds_addr(buf))), b1 = b0 + STEP;
    const uint32_t sb0 = uniform(static_cast<int>(dma::lds_addr(sbuf)));
    Frags f0, f1;
    Scales c;
    const int soff0 = pair_off(s, 0, lane), soff1 = pair_off(s, 1, lane);
#pragma unroll
    for (int j = 0; j < SC; ++j) {
      scale_copy(s, j, false, soff0, sb0, wave);
      scale_copy(s, j, true, soff0, sb0, wave);
      scale_copy(s, j, false, soff1, sb0 + SPAIR, wave);
    }
    const int off0 = step_off(s, 0);
#pragma unroll
    for (int i = 0; i < NCP; ++i) copy(s, i, off0, b0, wave);
    if (s.nk > 1) {
      const int off1 = step_off(s, 1);
#pragma unroll
      for (int i = 0; i < NCP; ++i) copy(s, i, off1, b1, wave);
      dma::wait_and_barrier<NCP>();
    } else {
      dma::wait_and_barrier<0>();
    }
    scales(sbuf, 0, c, wm, wn, lane);
    read<0>(buf, f0, wm, wn, lane);
    __builtin_amdgcn_sched_barrier(0);
    // Step kb, with the copies of step kb + 2 into the buffer that its
    // fragments have left.  Scales of the pair p of steps 2p, 2p + 1: those of
    // X during step 2p - 3, when the second step of pair p - 2, the buffer's
    // last user, is in registers; those of W during step 2p - 2.
    int kb = 0;
    for (; kb + 2 < s.nk; ++kb) {
      const int cur = kb & 1;
      read<1>(buf + (cur ? STEP : 0), f1, wm, wn, lane);
      mfma<0, 0, MF>(f0, c, acc);
      lds_barrier();                       // every wave holds its fragments of step kb
      __builtin_amdgcn_sched_barrier(0);
      const int p = (kb + 3) >> 1;
      copies_mfmas<0>(s, step_off(s, kb + 2), cur == 0, pair_off(s, p, lane), cur ? b1 : b0,
                      sb0 + (p & 1) * SPAIR, wave, f1, c, acc);
      dma::wait_and_barrier<N>();          // step kb + 1 has landed for every wave
      mfma<1, MF / 4 * 3, MF>(f1, c, acc);
      read<0>(buf + (cur ? 0 : STEP), f0, wm, wn, lane);
      scales(sbuf + (((kb + 1) >> 1) & 1) * SPAIR, 1 - cur, c, wm, wn, lane);
      __builtin_amdgcn_sched_barrier(0);
    }
    if (kb + 1 < s.nk) {
      read<1>(buf + (kb & 1) * STEP, f1, wm, wn, lane);
      mfma<0, 0, MF>(f0, c, acc);
      mfma<1, 0, MF>(f1, c, acc);
      dma::wait_and_barrier<0>();
      ++kb;
      scales(sbuf + ((kb >> 1) & 1) * SPAIR, kb & 1, c, wm, wn, lane);
      read<0>(buf + (kb & 1) * STEP, f0, wm, wn, lane);
    }
    mfma<0, 0, MF>(f0, c, acc);
    if (!(s.nd & 1)) {
      read<1>(buf + (kb & 1) * STEP, f1, wm, wn, lane);
      mfma<1, 0, MF>(f1, c, acc);
    }
    lds_barrier();                       // buffers are free
  }

  // Bias, SiLU and bf16 rounding into LDS rows of 256 features (16-byte chunks
  // swizzled by the row), then whole-row stores.
  template <bool SILU, bool BIAS>
  static __device__ __forceinline__ void epilogue(const Acc &acc, const MxArgs &a, int g,
                                                  int64_t first, int64_t row0, int64_t rows, int n0,
                                                  uint8_t *buf, int wm, int wn, int lane, int tid) {
    uint16_t *st = reinterpret_cast<uint16_t *>(buf);
#pragma unroll
    for (int ni = 0; ni < TN; ++ni)
#pragma unroll
      for (int q = 0; q < 4; ++q) {
        const int nl = wn * 64 + ni * 32 + q * 8 + (lane >> 5) * 4, n = n0 + nl;
        float bv[4] = {0.0f, 0.0f, 0.0f, 0.0f};
        if (BIAS && n < a.n_out) {
          const uint2 b = *reinterpret_cast<const uint2 *>(a.bias + static_cast<int64_t>(g) * a.n_out + n);
          bv[0] = __uint_as_float(b.x << 16);
          bv[1] = __uint_as_float(b.x & 0xFFFF0000u);
          bv[2] = __uint_as_float(b.y << 16);
          bv[3] = __uint_as_float(b.y & 0xFFFF0000u);
        }
#pragma unroll
        for (int mi = 0; mi < TM; ++mi) {
          const int ml = wm * (BM / 2) + mi * 32 + (lane & 31);
          float o[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            o[j] = acc[ni][mi][q * 4 + j];
            if (BIAS) o[j] += bv[j];
            if (SILU) o[j] = silu_fast(o[j]);
          }
          uint2 p;
          p.x = pack_bf16x2(o[0], o[1]);
          p.y = pack_bf16x2(o[2], o[3]);
          *reinterpret_cast<uint2 *>(st + ml * BN + ((nl >> 3) ^ (ml & 31)) * 8 + ((nl >> 2) & 1) * 4) = p;
        }
      }
    lds_barrier();
    const int c = tid & 31, r0 = tid >> 5, n = n0 + c * 8;
    if (n < a.n_out) {
      uint16_t *out = a.y + (first + row0 + r0) * a.n_out + n;
      const int64_t lim = rows - row0 - r0;
#pragma unroll 8
      for (int j = 0; j < BM / 16; ++j) {
        const int r = r0 + 16 * j;
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(st + r * BN + ((c ^ (r & 31)) << 3));
        if (16 * j < lim) store_nt(out + static_cast<int64_t>(16 * j) * a.n_out, v);
      }
    }
    lds_barrier();
  }

  template <bool SILU>
  static __device__ __forceinline__ void run(const MxArgs &a, int g, int64_t row0, int n0, uint8_t *buf,
                                             uint8_t *sbuf) {
    const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
    const int wm = wave & 1, wn = wave >> 1;
    const int64_t first = a.offsets[g], rows = a.offsets[g + 1] - first;
    Src s;
    source(a, g, first, row0, rows, n0, tid, s);
    Acc acc;
    body(s, buf, sbuf, acc, wave, wm, wn, lane);
    if (a.bias) epilogue<SILU, true>(acc, a, g, first, row0, rows, n0, buf, wm, wn, lane, tid);
    else epilogue<SILU, false>(acc, a, g, first, row0, rows, n0, buf, wm, wn, lane, tid);
  }
};
}  // namespace tile

// Persistent workgroups, one per CU, first on the units, then on the tiles.  The
// full tiles, in bands of four row tiles, then the 128- and the 64-row tiles are
// each split into eight contiguous shares, one per XCD (workgroups are dealt to
// the XCDs round-robin by number), so that tiles running together on an XCD share
// operands in its L2.
template <bool SILU>
__global__ __launch_bounds__(tile::NT, 2) void mx_linear_kernel(MxArgs a) {
  using namespace tile;
  __shared__ __attribute__((aligned(16))) uint8_t s_buf[BUF];
  __shared__ __attribute__((aligned(16))) uint8_t s_sc[2 * SBUF];
  __shared__ int s_pref[kMaxGroups + 1];
  __shared__ int16_t s_t128[kMaxGroups], s_t64[kMaxGroups];
  __shared__ int s_cnt[2], s_plan[3];
  const int tid = threadIdx.x, nt = (a.n_out + BN - 1) / BN;
  const Plan plan = mx_plan(a, nt, NT, s_pref, s_plan);
  if (plan.units) {
    static_assert(sizeof(int64_t) * (kMaxGroups + 1) <= sizeof(s_buf), "");
    mx_units<SILU>(a, s_pref, reinterpret_cast<int64_t *>(s_buf));
  }
  if (!plan.tiles) return;
  __syncthreads();                       // s_buf and the row counts have been used
  const int least = plan.least;
  if (tid < 64) {
    int full = 0, n128 = 0, n64 = 0;
    const uint64_t below = (1ull << tid) - 1;
    for (int g0 = 0; g0 < a.groups; g0 += 64) {
      const int g = g0 + tid, rows = g < a.groups ? s_pref[g] : 0;
      int t = 0;
      const int n = rows >= least ? mx_full_tiles(rows, &t) : 0;
      int incl = n;
#pragma unroll
      for (int off = 1; off < 64; off <<= 1) {
        const int o = __shfl_up(incl, off);
        if (tid >= off) incl += o;
      }
      if (g < a.groups) s_pref[g] = full + incl - n;
      full += __shfl(incl, 63);
      const uint64_t m128 = __ballot(t == 128), m64 = __ballot(t == 64);
      if (t == 128) s_t128[n128 + __popcll(m128 & below)] = static_cast<int16_t>(g);
      if (t == 64) s_t64[n64 + __popcll(m64 & below)] = static_cast<int16_t>(g);
      n128 += __popcll(m128);
      n64 += __popcll(m64);
    }
    if (tid == 0) {
      s_pref[a.groups] = full;
      s_cnt[0] = n128;
      s_cnt[1] = n64;
    }
  }
  __syncthreads();
  const int total[3] = {uniform(s_pref[a.groups]) * nt, uniform(s_cnt[0]) * nt, uniform(s_cnt[1]) * nt};
  const int xcd = blockIdx.x % kXcds, slot = blockIdx.x / kXcds, slots = gridDim.x / kXcds;
  int begin[3], cnt[3];
#pragma unroll
  for (int l = 0; l < 3; ++l) {
    const int part = (total[l] + kXcds - 1) / kXcds;
    begin[l] = min(xcd * part, total[l]);
    cnt[l] = min(begin[l] + part, total[l]) - begin[l];
  }
  // A last round of full tiles for at most half of the workgroups is dealt out as
  // halves (64 groups of 370 to 1290 rows, 100 full tiles for the 32 workgroups of
  // an XCD: 98 -> 91 us).
  const int rest = cnt[0] % slots, split = 2 * rest <= slots ? rest : 0, fulls = cnt[0] - split;
  for (int it = slot; it < cnt[0] + split + cnt[1] + cnt[2]; it += slots) {
    if (it < fulls + 2 * split) {
      constexpr int GM = 4;
      const int half = it < fulls ? -1 : (it - fulls) & 1;
      const int L = begin[0] + (half < 0 ? it : fulls + (it - fulls) / 2), tm = s_pref[a.groups];
      const int band = L / (GM * nt), m0 = band * GM, gm = min(GM, tm - m0), r = L - band * GM * nt;
      const int mt = m0 + r % gm, n = r / gm;
      int lo = 0, hi = a.groups;         // s_pref[lo] <= mt < s_pref[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_pref[mid] <= mt) lo = mid; else hi = mid;
      }
      const int g = uniform(lo);
      const int64_t row0 = static_cast<int64_t>(mt - s_pref[g]) * 256;
      if (half < 0) Tile<256>::run<SILU>(a, g, row0, n * BN, s_buf, s_sc);
      else Tile<128, false>::run<SILU>(a, g, row0 + half * 128, n * BN, s_buf, s_sc);
    } else {
      const int i = it - fulls - 2 * split;
      const bool wide = i < cnt[1];
      const int q = wide ? begin[1] + i : begin[2] + i - cnt[1];
      const int g = uniform(wide ? s_t128[q / nt] : s_t64[q / nt]), n0 = (q % nt) * BN;
      const int64_t row0 = (a.offsets[g + 1] - a.offsets[g]) / 256 * 256;
      if (wide) Tile<128>::run<SILU>(a, g, row0, n0, s_buf, s_sc);
      else Tile<64>::run<SILU>(a, g, row0, n0, s_buf, s_sc);
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
  // The groups' row counts are on the device; but there may neither be a group of
  // more than kStreamRows rows nor tiles enough.
  const int64_t met = p.max_rows < p.groups ? p.max_rows : p.groups;
  const int64_t wide = (p.n_out + tile::BN - 1) / tile::BN;
  if (p.max_rows <= kStreamRows && (met + p.max_rows / 17) * wide < kFill) {
    const int64_t units = met * ((p.n_out + stream::UN - 1) / stream::UN);
    const int64_t blocks = (units + kUnitWaves - 1) / kUnitWaves;
    const dim3 grid(static_cast<unsigned>(blocks < 512 ? blocks : 512)), block(kUnitWaves * 64);
    if (p.silu) hipLaunchKernelGGL(mx_units_kernel<true>, grid, block, 0, s, a);
    else hipLaunchKernelGGL(mx_units_kernel<false>, grid, block, 0, s, a);
    return hipGetLastError();
  }
  if (p.silu) hipLaunchKernelGGL(mx_linear_kernel<true>, dim3(256), dim3(tile::NT), 0, s, a);
  else hipLaunchKernelGGL(mx_linear_kernel<false>, dim3(256), dim3(tile::NT), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
