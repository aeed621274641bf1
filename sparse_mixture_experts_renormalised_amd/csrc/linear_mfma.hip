// Gradients of the single Linears of every expert on the bf16 matrix
// instructions (v_mfma_f32_32x32x16_bf16, float32 sums):
//
//   input gradient   dx[r][p] = sum_j dy[r][j] W_g[j][p]      (times silu'(pre))
//   weight gradient  dw_g[q][p] = sum_r dy[r][q] x[idx r][p]  (and dbias)
//
// Both are C[q][p] = sum_j Q(j, q) P(j, p) with operands whose memory does not run
// along the sum: P (weights, or x) lies [j][p], and so does dy as Q of the weight
// gradient.  Such an operand goes to LDS as it lies and is turned by the transposing
// LDS reads (ds_read_b64_tr_b16: sixteen lanes read 4 x 16 elements and get a column
// of four each); dy as Q of the input gradient lies [q][j] and is read in 16-byte
// pieces.
//
// A workgroup of four waves computes 128 x 256 of C, a wave 64 x 128 (eight 32 x 32
// blocks).  Steps of 32 along j are copied global -> LDS into a ring of three, two
// steps ahead; the fragments of the next 16 j are read while those of the last are
// multiplied; one barrier a step.  72 KB of LDS and at most 256 registers leave room
// for two workgroups on a CU, so that one's first copies and its epilogue run under
// the other's products.  P is the instruction's first operand: a lane ends up with
// four neighbouring elements of one row of C.
#include "lds_dma.h"
#include "linear.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef short s16x8_t __attribute__((ext_vector_type(8)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kQ = 128, kP = 256, kJ = 32, kRing = 3, kXcds = 8;
constexpr int kQBytes = kQ * kJ * 2, kPBytes = kP * kJ * 2, kStage = kQBytes + kPBytes;
constexpr int kQCopies = kQBytes / 4096, kPCopies = kPBytes / 4096, kCopies = kQCopies + kPCopies;
constexpr int kMaxGroups = kMaxRouted + kMaxShared;
constexpr int kTileFloats = kQ * kP;
constexpr int kSplitSlots = 512;         // workgroups that a split may fill: two a CU
constexpr int kMinSteps = 8;             // steps of a part, at least

struct Args {
  Linear l;
  float *part;                           // parts of split sums, kTileFloats each (or null)
  int most_parts;                        // parts of a tile, at most (1: never split)
};

// ---------------------------------------------------------------------------
// Global to LDS
// ---------------------------------------------------------------------------
// Buffer descriptor of n bytes from p; what lies behind reads as zero.
__device__ __forceinline__ u32x4_t descriptor(const void *p, int64_t n) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  u32x4_t d;
  d[0] = uniform(static_cast<int>(a));
  d[1] = uniform(static_cast<int>(a >> 32) & 0xFFFF);
  d[2] = uniform(static_cast<int>(n <= 0 ? 0u : n < 0xFFFFFF00ll ? static_cast<uint32_t>(n) : 0xFFFFFF00u));
  d[3] = 0x00020000;
  return d;
}
// One wave's 1 KB copy, 16 bytes a lane from the descriptor's start + off; lanes out of
// its range write zeros.
__device__ __forceinline__ void dma16b(uint32_t off, u32x4_t desc, uint32_t m0) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(off), "s"(desc), "{m0}"(m0) : "memory");
}

__device__ __forceinline__ const char *uniform_ptr(const void *p) {
  const uint64_t u = reinterpret_cast<uint64_t>(p);
  const uint32_t lo = uniform(static_cast<int>(u)), hi = uniform(static_cast<int>(u >> 32));
  return reinterpret_cast<const char *>((static_cast<uint64_t>(hi) << 32) | lo);
}

// ---------------------------------------------------------------------------
// LDS to fragments.  Operands [j][n] (n = 128 or 256 columns): rows of 2n bytes whose
// 64-byte pieces sit at piece ^ (j & 3), so that the four rows of a transposing read
// cover all banks.  Operands [q][j]: rows of 64 bytes whose 16-byte pieces sit at
// piece ^ ((q >> 2) & 3), so that sixteen rows do.
// ---------------------------------------------------------------------------
typedef __attribute__((address_space(3))) s16x4_t lds_s16x4_t;
typedef __attribute__((address_space(3))) bf16x8_t lds_bf16x8_t;

// Byte offset, within an operand's stage, of this lane's part of column block
// (32 columns) `block`, rows 0 .. 3 of its half of a slice.
template <int N>
__device__ __forceinline__ uint32_t turned_at(int block, int lane) {
  const int t = (lane & 15) >> 2;
  return ((lane >> 5) * 8 + t) * (2 * N) + ((block ^ t) << 6) + ((lane >> 4) & 1) * 32 + (lane & 3) * 8;
}
template <int N>
__device__ __forceinline__ bf16x8_t read_turned(uint32_t at) {
  const s16x4_t a = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t *>(at));
  const s16x4_t b = __builtin_amdgcn_ds_read_tr16_b64_v4i16(reinterpret_cast<lds_s16x4_t *>(at + 8 * N));
  return __builtin_bit_cast(bf16x8_t, __builtin_shufflevector(a, b, 0, 1, 2, 3, 4, 5, 6, 7));
}

struct Frags {
  bf16x8_t q[2], p[4];
};

// First element of 64-bit offsets that the tile needs.
struct Tile {
  int g, q0, p0;           // group, first row (or output feature), first column
  int64_t row0;            // first row of the group
  int rows;
  int s0, s1;              // steps of this part
};

// Tile prefix over groups (input gradient), in LDS.
__device__ int tile_prefix(const Linear &a, int *pref, int *tmp) {
  const int per = (a.groups + 255) / 256, g0 = min(static_cast<int>(threadIdx.x) * per, a.groups);
  const int g1 = min(g0 + per, a.groups);
  auto tiles = [&](int g) { return (a.offsets[g + 1] - a.offsets[g] + kQ - 1) / kQ; };
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

struct Plan {
  int64_t tiles;
  int qtiles, ptiles, parts, steps;
};

// Parts of every tile's sum, so that few tiles still fill the chip.
template <int MODE>
__device__ __forceinline__ Plan make_plan(const Args &a, int qtiles) {
  Plan p;
  p.qtiles = qtiles;
  p.ptiles = (a.l.k + kP - 1) / kP;
  p.tiles = static_cast<int64_t>(qtiles) * p.ptiles * (MODE == kLinWeightGrad ? a.l.groups : 1);
  p.parts = 1;
  if (a.most_parts > 1 && p.tiles > 0 && p.tiles * 2 <= kSplitSlots)
    p.parts = min(a.most_parts, static_cast<int>(kSplitSlots / p.tiles));
  return p;
}

// Tile `at` of the list, in the order in which neighbours share operands: the rows of a
// group (or output features) within a band of 8 tiles, then columns, then bands.
template <int MODE>
__device__ __forceinline__ Tile tile_at(const Args &a, const Plan &p, const int *pref, int64_t at, int part) {
  Tile t;
  int q;
  int64_t first = 0;                     // first q tile of the band's group
  int in_group;                          // q tiles of that group
  if (MODE == kLinWeightGrad) {
    const int64_t per = static_cast<int64_t>(p.qtiles) * p.ptiles;
    t.g = static_cast<int>(at / per);
    at -= t.g * per;
    in_group = p.qtiles;
  } else {
    // all groups' q tiles before this one's times the columns
    int lo = 0, hi = a.l.groups;
    const int64_t u = at / p.ptiles;     // pref[lo] <= u < pref[hi]
    while (hi - lo > 1) {
      const int mid = (lo + hi) >> 1;
      if (pref[mid] <= u) lo = mid; else hi = mid;
    }
    t.g = lo;
    first = pref[lo];
    in_group = pref[lo + 1] - pref[lo];
    at -= first * p.ptiles;
  }
  constexpr int kBand = 8;
  const int l = static_cast<int>(at), band = l / (kBand * p.ptiles), rest = l - band * kBand * p.ptiles;
  const int h = min(kBand, in_group - band * kBand);
  q = band * kBand + rest % h;
  t.q0 = q * kQ;
  t.p0 = (rest / h) * kP;
  t.row0 = a.l.offsets[t.g];
  t.rows = a.l.offsets[t.g + 1] - static_cast<int>(t.row0);
  const int steps = MODE == kLinWeightGrad ? (t.rows + kJ - 1) / kJ : a.l.n_out / kJ;
  const int per = (steps + p.parts - 1) / p.parts;
  t.s0 = min(steps, part * per);
  t.s1 = min(steps, t.s0 + per);
  return t;
}

// ---------------------------------------------------------------------------
// Sources of a tile's copies
// ---------------------------------------------------------------------------
template <int MODE, bool GATHER>
struct Source {
  uint32_t q[kQCopies], p[kPCopies];     // this lane's byte offsets in a step
  const char *qbase, *pbase;             // step 0 of the part
  int64_t qstep, pstep;                  // bytes of a step
  int64_t left;                          // rows of the group from the part's step 0 (weight gradient)
  const __attribute__((address_space(4))) int32_t *index;
  int rows, j0;
  uint32_t pcol;

  __device__ __forceinline__ void init(const Args &a, const Tile &t, int wave, int lane) {
    const int n = a.l.n_out, k = a.l.k;
    if constexpr (MODE == kLinInputGrad) {
      // [q][j]: 16 rows of 64 bytes a copy
      const int c = (lane & 3) ^ ((lane >> 4) & 3);
#pragma unroll
      for (int i = 0; i < kQCopies; ++i) {
        const int r = min(16 * (4 * i + wave) + (lane >> 2), t.rows - 1 - t.q0);
        q[i] = static_cast<uint32_t>(r) * n * 2 + c * 16;
      }
      qbase = uniform_ptr(static_cast<const uint16_t *>(a.l.dy) + (t.row0 + t.q0) * n + t.s0 * kJ);
      qstep = kJ * 2;
    } else {
      // [j][128 columns]: 4 rows of 256 bytes a copy
      const int c = (lane & 15) ^ ((lane >> 4) * 4);
#pragma unroll
      for (int i = 0; i < kQCopies; ++i)
        q[i] = static_cast<uint32_t>(4 * (4 * i + wave) + (lane >> 4)) * n * 2 + min(t.q0 + c * 8, n - 8) * 2;
      qbase = uniform_ptr(static_cast<const uint16_t *>(a.l.dy) + (t.row0 + static_cast<int64_t>(t.s0) * kJ) * n);
      qstep = static_cast<int64_t>(kJ) * n * 2;
    }
    // [j][256 columns]: 2 rows of 512 bytes a copy
    const int j = 2 * wave + (lane >> 5), c = (lane & 31) ^ ((j & 3) * 4);
    pcol = min(t.p0 + c * 8, k - 8) * 2;
#pragma unroll
    for (int i = 0; i < kPCopies; ++i) p[i] = static_cast<uint32_t>(8 * i + j) * k * 2 + pcol;
    pstep = static_cast<int64_t>(kJ) * k * 2;
    if constexpr (MODE == kLinInputGrad) {
      pbase = uniform_ptr(static_cast<const uint16_t *>(a.l.w) +
                          (static_cast<int64_t>(t.g) * n + static_cast<int64_t>(t.s0) * kJ) * k);
    } else if constexpr (GATHER) {
      pbase = uniform_ptr(a.l.x);
      index = (const __attribute__((address_space(4))) int32_t *)(uniform_ptr(a.l.index + t.row0));
    } else {
      pbase = uniform_ptr(static_cast<const uint16_t *>(a.l.x) + (t.row0 + static_cast<int64_t>(t.s0) * kJ) * k);
    }
    j0 = t.s0 * kJ;
    // rows of this part's steps end where the part ends
    rows = MODE == kLinWeightGrad ? min(t.rows, t.s1 * kJ) : 0;
    left = rows - j0;
  }

  // The copies of step s (counted from the part's first) into the stage at LDS byte m0.
  __device__ __forceinline__ void copy(const Args &a, int s, uint32_t m0, int wave, int lane) const {
    m0 += wave * 1024;
    if constexpr (MODE == kLinInputGrad) {
      const char *qb = qbase + s * qstep, *pb = pbase + s * pstep;
#pragma unroll
      for (int i = 0; i < kQCopies; ++i) dma::dma16s(q[i], qb, m0 + i * 4096);
#pragma unroll
      for (int i = 0; i < kPCopies; ++i) dma::dma16s(p[i], pb, m0 + kQBytes + i * 4096);
    } else {
      const int64_t have = left - static_cast<int64_t>(s) * kJ;    // rows from this step on
      const u32x4_t dq = descriptor(qbase + s * qstep, have * a.l.n_out * 2);
#pragma unroll
      for (int i = 0; i < kQCopies; ++i) dma16b(q[i], dq, m0 + i * 4096);
      if constexpr (GATHER) {
        const uint32_t bytes = static_cast<uint32_t>(a.l.x_rows * a.l.k * 2);
        const u32x4_t dp = descriptor(pbase, a.l.x_rows * a.l.k * 2);
#pragma unroll
        for (int i = 0; i < kPCopies; ++i) {
          const int j = j0 + s * kJ + 8 * i + 2 * wave;
          const int i0 = index[max(0, min(j, rows - 1))], i1 = index[max(0, min(j + 1, rows - 1))];
          const uint32_t at = static_cast<uint32_t>(lane >> 5 ? i1 : i0) * static_cast<uint32_t>(a.l.k * 2) + pcol;
          dma16b(j + (lane >> 5) < rows ? at : bytes, dp, m0 + kQBytes + i * 4096);
        }
      } else {
        const u32x4_t dp = descriptor(pbase + s * pstep, have * a.l.k * 2);
#pragma unroll
        for (int i = 0; i < kPCopies; ++i) dma16b(p[i], dp, m0 + kQBytes + i * 4096);
      }
    }
  }
};

// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
typedef f32x16_t Acc[4][2];              // [column block][row block] of 32 x 32

__device__ __forceinline__ void multiply(const Frags &f, Acc &acc) {
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 2; ++q)
      acc[p][q] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.p[p], f.q[q], acc[p][q], 0, 0, 0);
}

__device__ __forceinline__ float sum8(bf16x8_t v) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += static_cast<float>(v[i]);
  return s;
}

// The other workgroup of the CU has its own ring: 72 KB each.
template <int MODE, bool GATHER>
__global__ __launch_bounds__(256, 2) void linear_grad_kernel(Args a) {
  __shared__ __attribute__((aligned(1024))) char s_ring[kRing * kStage];
  __shared__ int s_pref[MODE == kLinInputGrad ? kMaxGroups + 1 : 1], s_tmp[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  const int wq = wave & 1, wp = wave >> 1;
  const Plan plan = make_plan<MODE>(a, MODE == kLinInputGrad ? tile_prefix(a.l, s_pref, s_tmp)
                                                             : (a.l.n_out + kQ - 1) / kQ);
  // workgroups are dealt to the XCDs in turn: each XCD takes a contiguous share
  const int64_t items = plan.tiles * plan.parts, share = (items + kXcds - 1) / kXcds;
  const int64_t slot = blockIdx.x / kXcds, item = (blockIdx.x % kXcds) * share + slot;
  if (slot >= share || item >= items) return;
  const int64_t at = item / plan.parts;
  const int part = static_cast<int>(item % plan.parts);
  const Tile t = tile_at<MODE>(a, plan, s_pref, at, part);

  Acc acc;
#pragma unroll
  for (int p = 0; p < 4; ++p)
#pragma unroll
    for (int q = 0; q < 2; ++q)
#pragma unroll
      for (int i = 0; i < 16; ++i) acc[p][q][i] = 0.0f;
  float bias[2] = {0.0f, 0.0f};
  const bool sum_dy = MODE == kLinWeightGrad && a.l.dbias && t.p0 == 0 && wp == 0;

  const uint32_t ring = uniform(static_cast<int>(dma::lds_addr(s_ring)));
  // read offsets of this lane within a stage
  uint32_t qat[2], pat[4];
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (MODE == kLinInputGrad) {
      const int row = wq * 64 + i * 32 + (lane & 31);
      qat[i] = ring + row * 64 + (((lane >> 5) ^ ((row >> 2) & 3)) << 4);
    } else {
      qat[i] = ring + turned_at<kQ>(wq * 2 + i, lane);
    }
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) pat[i] = ring + kQBytes + turned_at<kP>(wp * 4 + i, lane);
  auto read = [&](Frags &f, uint32_t stage, int slice) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      if constexpr (MODE == kLinInputGrad)   // pieces 2 slice + half: slice flips bit 1
        f.q[i] = *reinterpret_cast<lds_bf16x8_t *>((qat[i] ^ (slice << 5)) + stage);
      else
        f.q[i] = read_turned<kQ>(qat[i] + stage + slice * (16 * kQ * 2));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) f.p[i] = read_turned<kP>(pat[i] + stage + slice * (16 * kP * 2));
  };

  const int steps = t.s1 - t.s0;
  if (steps > 0) {
    Source<MODE, GATHER> src;
    src.init(a, t, wave, lane);
    const int last = steps - 1;
    // Steps behind the last are copied too, from the last one's place: what they
    // bring is not multiplied, and every wait counts the same copies.
    auto copy = [&](int s, uint32_t stage) { src.copy(a, min(s, last), ring + stage, wave, lane); };
    copy(0, 0);
    copy(1, kStage);
    copy(2, 2 * kStage);
    dma::wait_and_barrier<2 * kCopies>();
    Frags f0, f1;
    read(f0, 0, 0);
    uint32_t stage = 0;
    for (int s = 0; s < steps; ++s) {
      const uint32_t next = stage == (kRing - 1) * kStage ? 0 : stage + kStage;
      read(f1, stage, 1);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f0, acc);
      if (sum_dy) {
        bias[0] += sum8(f0.q[0]);
        bias[1] += sum8(f0.q[1]);
      }
      // this step's stage is read, the next one has landed for every wave
      dma::wait_and_barrier<kCopies>();
      copy(s + 3, stage);
      read(f0, next, 0);
      __builtin_amdgcn_sched_barrier(0);
      multiply(f1, acc);
      if (sum_dy) {
        bias[0] += sum8(f1.q[0]);
        bias[1] += sum8(f1.q[1]);
      }
      stage = next;
    }
    dma::wait_and_barrier<0>();
  }

  if (sum_dy && plan.parts == 1) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const float v = bias[i] + __shfl_xor(bias[i], 32);
      const int q = t.q0 + wq * 64 + i * 32 + (lane & 31);
      if (lane < 32 && q < a.l.n_out) {
        const int64_t o = static_cast<int64_t>(t.g) * a.l.n_out + q;
        if (a.l.out_bf16) {
          uint16_t *d = static_cast<uint16_t *>(a.l.dbias) + o;
          *d = f32_to_bf16(a.l.accumulate ? bf16_to_f32(*d) + v : v);
        } else {
          float *d = static_cast<float *>(a.l.dbias) + o;
          *d = a.l.accumulate ? *d + v : v;
        }
      }
    }
  }

  const int np = a.l.k, nq = MODE == kLinWeightGrad ? a.l.n_out : t.rows;
  const int64_t out_row = MODE == kLinWeightGrad ? static_cast<int64_t>(t.g) * a.l.n_out : t.row0;
#pragma unroll
  for (int qi = 0; qi < 2; ++qi) {
    const int q = t.q0 + wq * 64 + qi * 32 + (lane & 31);
    if (q >= nq) continue;
#pragma unroll
    for (int pi = 0; pi < 4; ++pi)
#pragma unroll
      for (int b = 0; b < 4; ++b) {
        const int p = t.p0 + wp * 128 + pi * 32 + b * 8 + (lane >> 5) * 4;
        if (p >= np) continue;
        float v[4] = {acc[pi][qi][4 * b], acc[pi][qi][4 * b + 1], acc[pi][qi][4 * b + 2], acc[pi][qi][4 * b + 3]};
        const int64_t o = (out_row + q) * np + p;
        if (MODE == kLinInputGrad || a.l.out_bf16) {
          uint2 *d = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.l.out) + o);
          if (MODE == kLinInputGrad && a.l.act_pre) {
            const uint2 z = *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.l.act_pre) + o);
            v[0] *= silu_slope(__uint_as_float(z.x << 16));
            v[1] *= silu_slope(__uint_as_float(z.x & 0xFFFF0000u));
            v[2] *= silu_slope(__uint_as_float(z.y << 16));
            v[3] *= silu_slope(__uint_as_float(z.y & 0xFFFF0000u));
          }
          if (MODE == kLinWeightGrad && a.l.accumulate) {
            const uint2 z = *d;
            v[0] += __uint_as_float(z.x << 16);
            v[1] += __uint_as_float(z.x & 0xFFFF0000u);
            v[2] += __uint_as_float(z.y << 16);
            v[3] += __uint_as_float(z.y & 0xFFFF0000u);
          }
          *d = make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
        } else {
          float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.l.out) + o);
          if (a.l.accumulate) {
            const float4 z = *d;
            v[0] += z.x, v[1] += z.y, v[2] += z.z, v[3] += z.w;
          }
          *d = make_float4(v[0], v[1], v[2], v[3]);
        }
      }
  }
}

}  // namespace

bool linear_grad_fits(const Linear &p) {
  // a gathered x is addressed by 32-bit byte offsets, lines of a step by 32-bit ones
  if (!p.bf16 || p.mode == kLinForward) return false;
  if (p.mode == kLinWeightGrad && p.index && p.x_rows > (0xFFFFFF00ll / 2) / p.k) return false;
  return p.n_out < (1 << 22) && p.k < (1 << 22);
}

hipError_t launch_linear_grad(const Linear &p, void *ws, hipStream_t s) {
  Args a{p, static_cast<float *>(ws), 1};
  const int64_t pt = (p.k + kP - 1) / kP;
  const int64_t qt = p.mode == kLinWeightGrad ? static_cast<int64_t>(p.groups) * ((p.n_out + kQ - 1) / kQ)
                                              : p.max_rows / kQ + (p.max_rows < p.groups ? p.max_rows : p.groups);
  const int64_t share = (pt * qt + kXcds - 1) / kXcds;
  if (share * kXcds >= (int64_t(1) << 31)) return hipErrorInvalidValue;
  const dim3 grid(static_cast<unsigned>(share * kXcds));
  if (p.mode == kLinInputGrad)
    hipLaunchKernelGGL((linear_grad_kernel<kLinInputGrad, false>), grid, dim3(256), 0, s, a);
  else if (p.index)
    hipLaunchKernelGGL((linear_grad_kernel<kLinWeightGrad, true>), grid, dim3(256), 0, s, a);
  else
    hipLaunchKernelGGL((linear_grad_kernel<kLinWeightGrad, false>), grid, dim3(256), 0, s, a);
  return hipGetLastError();
}

}  // namespace moe
