// Single Linears of every expert and their gradients on the bf16 matrix
// instructions (v_mfma_f32_32x32x16_bf16, float32 sums):
//
//   forward          y[r][p] = act(sum_j x[idx r][j] W_g[p][j] + bias_g[p])
//   input gradient   dx[r][p] = sum_j dy[r][j] W_g[j][p]      (times silu'(pre))
//   weight gradient  dw_g[q][p] = sum_r dy[r][q] x[idx r][p]  (and dbias)
//
// All are C[q][p] = sum_j Q(j, q) P(j, p).  The gradients have operands whose memory does
// not run along the sum: P (weights, or x) lies [j][p], and so does dy as Q of the weight
// gradient.  Such an operand goes to LDS as it lies and is turned by the transposing
// LDS reads (ds_read_b64_tr_b16: sixteen lanes read 4 x 16 elements and get a column
// of four each); those that lie along the sum (both of the forward, dy as Q of the input
// gradient) are read in 16-byte pieces.
//
// Steps of 32 along j are copied global -> LDS into a ring, RING - 1 steps ahead; the
// fragments of the next 16 j are read while those of the last are multiplied; one
// barrier a step.  Workgroups are persistent and the stream of steps runs on from one
// tile into the next: while a tile's sums go out, by way of the one ring stage that has
// just been read, the next tile's first steps are on their way.  What a descriptor does
// not cover reads as zero, so rows behind a group's end, steps behind a short tile's
// and copies behind the last tile need no case of their own, and every wait counts the
// same copies.  P is the instruction's first operand: a lane ends up with four
// neighbouring elements of one row of C.
//
// Measured (clocks of the chip move between 1.5 and 2.2 GHz under the power limit, so that
// times differ by several per cent from run to run):
//   input gradient, 8192 rows on 8 experts of 4096 x 14336 with the SiLU's slope: 895 to
//     970 us, 1000 to 1070 TFLOP/s (one library product an expert, without the slope: 845).
//     Matrix instructions are busy 59% of the clocks, workgroups 92%; a step takes 1250
//     clocks of the 1024 that its products take, a tile's slopes and stores 12 000.
//   weight gradient of one group of 32768 rows, 4096 x 4096: 854 us, 1290 TFLOP/s;
//     gathered rows 935.  64 groups of 512, 2048 x 1408, to float32: 255 to 310 us, where
//     the 850 MB alone take 178 at a copy's rate: steps and stores take turns, as all
//     workgroups come to a tile's end at about the same time.  256 groups of 128, to bf16:
//     450 us, 3.8 TB/s.
//   forward of 64 groups of 512 gathered rows, 2048 -> 1408, with the SiLU and the values
//     before it: 245 to 300 us; 3.7 rounds of tiles (CUs are busy 79% of the time), matrix
//     instructions 36%.
//   input gradient of 207 rows on 256 experts of 2048 x 7168: 425 us, 5.8 TB/s of weights.
// Tiles of 128 x 256 with two workgroups a CU took 1134 us for the first and 306 for the
// 64 groups, four waves of 128 x 128 1099 and 391.
#include "lds_dma.h"
#include "linear.h"

namespace moe {
namespace {

typedef __bf16 bf16x8_t __attribute__((ext_vector_type(8)));
typedef short s16x4_t __attribute__((ext_vector_type(4)));
typedef float f32x16_t __attribute__((ext_vector_type(16)));
typedef uint32_t u32x4_t __attribute__((ext_vector_type(4)));

constexpr int kJ = 32, kXcds = 8, kCus = 256;
constexpr int kMaxGroups = kMaxRouted + kMaxShared;
constexpr int kMinSteps = 8;             // as many parts as leave this many steps to each of the longest
                                         // sum; those of a shorter group are shorter, the last ones empty
constexpr int kTileCost = 6;             // what a tile costs beside its steps, in steps

// A wave's 32 x 32 blocks along either axis of C, and the workgroup's tile of QW x 2
// waves, 256 columns wide.
template <int QB_, int QW_, int RING_>
struct Shape {
  static constexpr int QB = QB_, PB = 4, QW = QW_, WAVES = 2 * QW, NT = 64 * WAVES, RING = RING_;
  static constexpr int Q = 32 * QB * QW, P = 64 * PB;
  static constexpr int QBYTES = Q * kJ * 2, PBYTES = P * kJ * 2, STAGE = QBYTES + PBYTES;
  static constexpr int QCOPIES = QBYTES / (1024 * WAVES), PCOPIES = PBYTES / (1024 * WAVES);
  static constexpr int COPIES = QCOPIES + PCOPIES;
  static constexpr int WGS = RING * STAGE <= 80 * 1024 ? 2 : 1;   // workgroups on a CU
  static constexpr int SLOTS = kCus * WGS;
  static constexpr int PART = Q * P + Q;   // floats of a part: a tile and its sums of dy
  static_assert(QCOPIES * 1024 * WAVES == QBYTES && PCOPIES * 1024 * WAVES == PBYTES, "whole copies");
  static_assert(STAGE >= WAVES * 4096, "4 KB of a stage for every wave's way out");
};

struct Args {
  Linear l;
  float *part;                           // parts of split sums (or null)
  int most_parts;                        // parts of a tile, at most (1: never split)
};

// ---------------------------------------------------------------------------
// Global to LDS
// ---------------------------------------------------------------------------
// Buffer descriptor of n bytes from p; what lies behind reads as zero and is not
// written.
__device__ __forceinline__ u32x4_t descriptor(const void *p, int64_t n) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  u32x4_t d;
  d[0] = uniform(static_cast<int>(a));
  d[1] = uniform(static_cast<int>(a >> 32) & 0xFFFF);
  d[2] = uniform(static_cast<int>(n <= 0 ? 0u : n < 0xFFFFFF00ll ? static_cast<uint32_t>(n) : 0xFFFFFF00u));
  d[3] = 0x00020000;
  return d;
}
__device__ __forceinline__ __amdgpu_buffer_rsrc_t resource(u32x4_t d) {
  void *p = reinterpret_cast<void *>((static_cast<uint64_t>(d[1]) << 32) | d[0]);
  return __builtin_amdgcn_make_buffer_rsrc(p, 0, d[2], d[3]);
}
// One wave's 1 KB copy, 16 bytes a lane from the descriptor's start + off; lanes out of
// its range write zeros.
__device__ __forceinline__ void dma16b(uint32_t off, u32x4_t desc, uint32_t m0) {
  asm volatile("s_nop 0\n\tbuffer_load_dwordx4 %0, %1, 0 offen lds" : : "v"(off), "s"(desc), "{m0}"(m0) : "memory");
}
// The same with 4 bytes a lane.
__device__ __forceinline__ void dma4b(uint32_t off, u32x4_t desc, uint32_t m0) {
  asm volatile("s_nop 0\n\tbuffer_load_dword %0, %1, 0 offen lds" : : "v"(off), "s"(desc), "{m0}"(m0) : "memory");
}
// 16 bytes a lane out, past the caches (whole lines that nothing here reads again).  As
// the copies' waits count these stores, every lane issues all of them: the descriptor
// drops what lies behind the tile's rows, and kNoColumn what lies behind its columns.
constexpr uint32_t kNoColumn = 0xFFFFFF00u;
template <bool ONCE = true>
__device__ __forceinline__ void store16b(uint32_t off, u32x4_t desc, u32x4_t v) {
  __builtin_amdgcn_raw_buffer_store_b128(v, resource(desc), off, 0, ONCE ? 2 : 0);
}

// 16 bytes a lane; zeros where the descriptor does not reach.
__device__ __forceinline__ u32x4_t load16b(uint32_t off, u32x4_t desc) {
  return __builtin_amdgcn_raw_buffer_load_b128(resource(desc), off, 0, 0);
}

// This wave's LDS operations are done, and every wave is here; waits for no copy.
__device__ __forceinline__ void lds_barrier() {
  asm volatile("s_waitcnt lgkmcnt(0)\n\ts_barrier" ::: "memory");
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

template <typename S>
struct Frags {
  bf16x8_t q[S::QB], p[S::PB];
};

// ---------------------------------------------------------------------------
// Tiles
// ---------------------------------------------------------------------------
struct Tile {
  int g, q0, p0;           // group, first row (or output feature), first column
  int64_t row0;            // first row of the group
  int rows;                // of the group
  int s0, s1;              // steps of this part of the sum
};

// Exclusive prefix over the groups, in LDS: 32-bit sums of count(g).
template <int NT, typename F>
__device__ int group_prefix(int groups, F count, int *pref, int *tmp) {
  const int per = (groups + NT - 1) / NT, g0 = min(static_cast<int>(threadIdx.x) * per, groups);
  const int g1 = min(g0 + per, groups);
  int local = 0;
  for (int g = g0; g < g1; ++g) local += count(g);
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
  for (int w = 0; w < NT / 64; ++w) {
    if (w < wave) run += tmp[w];
    total += tmp[w];
  }
  for (int g = g0; g < g1; ++g) {
    pref[g] = run;
    run += count(g);
  }
  if (threadIdx.x == 0) pref[groups] = total;
  __syncthreads();
  return total;
}

// Largest g with pref[g] <= v (a group that is not empty, for v below the total).
__device__ __forceinline__ int group_of(const int *pref, int groups, int v) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (uniform(pref[mid]) <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// x / y for 0 <= x < 2^31, 0 < y: the float quotient is off by at most 2^-22 of itself,
// so two rounds of it leave a remainder within y, which the last step sets right.  The
// compiler's own division takes several times as long.
__device__ __forceinline__ int quotient(int x, int y) {
  const float r = __builtin_amdgcn_rcpf(static_cast<float>(y));
  int q = static_cast<int>(static_cast<float>(x) * r);
  int rest = x - q * y;
  const int more = static_cast<int>(static_cast<float>(rest) * r);
  q += more;
  rest -= more * y;
  return uniform(q - (rest < 0 ? 1 : 0) + (rest >= y ? 1 : 0));
}

struct Plan {
  int tiles, first, end;       // tiles in all; this XCD's items (parts of tiles)
  int qtiles, ptiles, parts;
};

// Elements of a row of C, and of a sum that is not over rows.
template <int MODE>
__device__ __forceinline__ int columns_of(const Linear &a) {
  return MODE == kLinForward ? a.n_out : a.k;
}
template <int MODE>
__device__ __forceinline__ int terms_of(const Linear &a) {
  return MODE == kLinForward ? a.k : a.n_out;
}

// Steps of a tile of a group of that many rows.
template <int MODE>
__device__ __forceinline__ int steps_of(const Linear &a, int rows) {
  return MODE == kLinWeightGrad ? (rows + kJ - 1) / kJ : terms_of<MODE>(a) / kJ;
}

// The work of this XCD.  Few tiles are split along their sums, so that they fill the
// chip; many are dealt out so that every XCD gets a contiguous share (neighbours read
// the same operands) of about the same cost.  pref: first q tile of every group (input
// gradient), off: the offsets, both in LDS.
template <typename S, int MODE>
__device__ Plan make_plan(const Args &a, int *pref, int *off, int *tmp, int xcd) {
  Plan p;
  const Linear &l = a.l;
  for (int g = threadIdx.x; g <= l.groups; g += S::NT) off[g] = l.offsets[g];
  __syncthreads();
  auto rows = [&](int g) { return off[g + 1] - off[g]; };
  p.ptiles = (columns_of<MODE>(l) + S::P - 1) / S::P;
  if (MODE != kLinWeightGrad) {
    p.qtiles = uniform(group_prefix<S::NT>(l.groups, [&](int g) { return (rows(g) + S::Q - 1) / S::Q; }, pref, tmp));
    p.tiles = p.qtiles * p.ptiles;
  } else {
    p.qtiles = (l.n_out + S::Q - 1) / S::Q;
    p.tiles = p.qtiles * p.ptiles * l.groups;
  }
  p.parts = 1;
  if (a.most_parts > 1 && p.tiles > 0 && p.tiles * 2 <= S::SLOTS) p.parts = min(a.most_parts, S::SLOTS / p.tiles);
  const int items = p.tiles * p.parts;
  if (MODE != kLinWeightGrad || p.parts > 1) {
    p.first = static_cast<int>(static_cast<int64_t>(items) * xcd / kXcds);
    p.end = static_cast<int>(static_cast<int64_t>(items) * (xcd + 1) / kXcds);
  } else {
    const int per = p.qtiles * p.ptiles;
    auto cost = [&](int g) { return max(S::RING, steps_of<MODE>(l, rows(g))) + kTileCost; };
    const int total = uniform(group_prefix<S::NT>(l.groups, cost, pref, tmp));
    // item at which x eighths of the cost are done: whole groups, then tiles of one
    auto border = [&](int x) {
      if (x == kXcds) return items;
      const int64_t want = static_cast<int64_t>(total) * x;          // in eighths
      const int g = group_of(pref, l.groups, static_cast<int>(want / kXcds));
      const int64_t in = want - static_cast<int64_t>(uniform(pref[g])) * kXcds;
      return g * per + static_cast<int>(in * per / (static_cast<int64_t>(uniform(cost(g))) * kXcds));
    };
    p.first = border(xcd);
    p.end = border(xcd + 1);
  }
  p.first = uniform(p.first);
  p.end = uniform(p.end);
  p.parts = uniform(p.parts);
  return p;
}

// An item: a part of a tile, in the order in which neighbours share operands: the q tiles
// of a group within a band of 8, then columns, then bands.  g: a group that is not
// behind the item's.
template <typename S, int MODE>
__device__ __forceinline__ Tile tile_at(const Args &a, const Plan &p, const int *pref, const int *off, int item, int g) {
  Tile t;
  int at = p.parts > 1 ? quotient(item, p.parts) : item;
  const int part = item - at * p.parts;
  int in_group = p.qtiles;               // q tiles of the group
  if (MODE == kLinWeightGrad) {
    const int per = p.qtiles * p.ptiles;
    t.g = quotient(at, per);
    at -= t.g * per;
  } else {
    const int q = quotient(at, p.ptiles);
    int next = uniform(pref[g + 1]);
    while (next <= q) next = uniform(pref[++g + 1]);
    const int first = uniform(pref[g]);
    t.g = g;
    in_group = next - first;
    at -= first * p.ptiles;
  }
  t.row0 = uniform(off[t.g]);
  t.rows = uniform(off[t.g + 1]) - static_cast<int>(t.row0);
  constexpr int kBand = 8;
  const int band = quotient(at, kBand * p.ptiles), rest = at - band * kBand * p.ptiles;
  const int h = min(kBand, in_group - band * kBand), column = quotient(rest, h);
  t.q0 = (band * kBand + rest - column * h) * S::Q;
  t.p0 = column * S::P;
  t.s0 = 0;
  t.s1 = steps_of<MODE>(a.l, t.rows);
  if (p.parts > 1) {
    const int steps = t.s1, per = quotient(steps + p.parts - 1, p.parts);
    t.s0 = min(steps, part * per);
    t.s1 = min(steps, t.s0 + per);
  }
  return t;
}

// ---------------------------------------------------------------------------
// Sources of a tile's copies
// ---------------------------------------------------------------------------
// Indexes of a gathered x in the forward, for one wave: those of a tile's rows that it
// copies, a dword each, in one of two slots in turn.  They come four steps ahead of the
// tile's first copy, when waits for copies have covered them.
template <typename S>
struct RowIndex {
  static constexpr int BYTES = 2 * S::WAVES * 256;
  static_assert(S::QCOPIES * 16 <= 64, "one copy for the rows of a wave");
  u32x4_t desc;
  uint32_t base;           // this wave's part of slot 0
  int slot;                // the one that was filled last

  __device__ __forceinline__ void init(const Args &a, uint32_t lds, int wave) {
    desc = descriptor(a.l.index, a.l.max_rows * 4);
    base = lds + wave * 256;
    slot = 0;
  }
  __device__ __forceinline__ uint32_t place() const { return base + slot * S::WAVES * 256; }
  __device__ __forceinline__ void start(const Tile &t, int wave, int lane) {
    slot ^= 1;
    const int r = min(16 * (S::WAVES * (lane >> 4) + wave) + (lane & 15), t.rows - 1 - t.q0);
    dma4b(lane < 16 * S::QCOPIES ? static_cast<uint32_t>(t.row0 + t.q0 + r) * 4 : kNoColumn, desc, place());
  }
};

// GATHER: the rows of x through the index (weight gradient: P, step by step; forward: Q,
// once for the tile).
template <typename S, int MODE, bool GATHER>
struct Source {
  static constexpr bool STEPWISE = GATHER && MODE == kLinWeightGrad;
  uint32_t q[S::QCOPIES], p[S::PCOPIES]; // this lane's byte offsets in a step
  u32x4_t dq, dp;                        // where the step lies
  uint32_t qstep, pstep, pcol;           // bytes of a step; byte offset of this lane's column
  int left;                              // rows (not weight gradient: steps) of the part from this step on
  uint32_t at[STEPWISE ? S::PCOPIES : 1];  // a gathered x: indexes of this lane's rows in the step to come

  // index: where RowIndex put the tile's (forward)
  __device__ __forceinline__ void init(const Args &a, const Tile &t, uint32_t index, int wave, int lane) {
    const int n = a.l.n_out, k = a.l.k;
    const int64_t j0 = static_cast<int64_t>(t.s0) * kJ;
    if constexpr (MODE == kLinWeightGrad) {
      left = static_cast<int>(min(t.rows, t.s1 * kJ) - j0);
      lines<S::Q, S::QCOPIES>(q, n, t.q0, wave, lane);
      qstep = static_cast<uint32_t>(kJ) * n * 2;
      dq = descriptor(static_cast<const uint16_t *>(a.l.dy) + (t.row0 + j0) * n, 0);
    } else {
      const int nj = terms_of<MODE>(a.l);
      const uint16_t *from = static_cast<const uint16_t *>(MODE == kLinForward ? a.l.x : a.l.dy) + j0;
      if constexpr (GATHER) {
        typedef __attribute__((address_space(3))) const volatile uint32_t lds_u32_t;
        const lds_u32_t *r = reinterpret_cast<lds_u32_t *>(index + (lane >> 2) * 4);
#pragma unroll
        for (int i = 0; i < S::QCOPIES; ++i) q[i] = r[16 * i] * static_cast<uint32_t>(nj * 2) + piece(lane);
      } else {
        rows_along<S::QCOPIES>(q, nj, t.rows - 1 - t.q0, wave, lane);
        from += (t.row0 + t.q0) * nj;
      }
      left = t.s1 - t.s0;
      qstep = kJ * 2;
      dq = descriptor(from, 0);
    }
    if constexpr (MODE == kLinForward) {
      rows_along<S::PCOPIES>(p, k, n - 1 - t.p0, wave, lane);
      pstep = kJ * 2;
      dp = descriptor(static_cast<const uint16_t *>(a.l.w) + (static_cast<int64_t>(t.g) * n + t.p0) * k + j0, 0);
    } else {
      pcol = lines<S::P, S::PCOPIES>(p, k, t.p0, wave, lane);
      pstep = static_cast<uint32_t>(kJ) * k * 2;
      if constexpr (MODE == kLinInputGrad)
        dp = descriptor(static_cast<const uint16_t *>(a.l.w) + (static_cast<int64_t>(t.g) * n + j0) * k, 0);
      else
        dp = descriptor(static_cast<const uint16_t *>(a.l.x) + (GATHER ? 0 : (t.row0 + j0) * k), 0);
    }
    cover(a);
  }
  // Behind the last tile: steps without data.
  __device__ __forceinline__ void none(const Args &a) {
    left = 0;
    cover(a);
  }
  // To the next step.
  __device__ __forceinline__ void advance(const Args &a) {
    left -= MODE == kLinWeightGrad ? kJ : 1;
    add(dq, qstep);
    if constexpr (!STEPWISE) add(dp, pstep);
    cover(a);
  }

  // Offsets of an operand [line][j] of lines of nj elements, clamped to the last one: 1 KB
  // copies of 16 lines each.
  static __device__ __forceinline__ uint32_t piece(int lane) { return ((lane & 3) ^ ((lane >> 4) & 3)) * 16; }
  template <int COPIES>
  static __device__ __forceinline__ void rows_along(uint32_t (&at)[COPIES], int nj, int last, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < COPIES; ++i)
      at[i] = static_cast<uint32_t>(min(16 * (S::WAVES * i + wave) + (lane >> 2), last)) * nj * 2 + piece(lane);
  }
  // Offsets of an operand [j][N columns] with lines of `width` elements: 1 KB copies
  // of 512 / N lines each.  Returns the column's byte offset.
  template <int N, int COPIES>
  static __device__ __forceinline__ uint32_t lines(uint32_t (&at)[COPIES], int width, int col0, int wave, int lane) {
    constexpr int LINES = 512 / N, LANES = 64 / LINES;   // lines of a copy, lanes of a line
    const int j = LINES * wave + lane / LANES, c = (lane % LANES) ^ ((j & 3) * 4);
    const uint32_t col = min(col0 + c * 8, width - 8) * 2;
#pragma unroll
    for (int i = 0; i < COPIES; ++i) at[i] = static_cast<uint32_t>(S::WAVES * LINES * i + j) * width * 2 + col;
    return col;
  }
  static __device__ __forceinline__ void add(u32x4_t &d, uint32_t bytes) {
    const uint64_t v = ((static_cast<uint64_t>(d[1]) << 32) | d[0]) + bytes;
    d[0] = uniform(static_cast<int>(v));
    d[1] = uniform(static_cast<int>(v >> 32));
  }
  // The rows of this step that are there.
  __device__ __forceinline__ void cover(const Args &a) {
    if constexpr (MODE != kLinWeightGrad) {   // lines along j are clamped
      const uint32_t line = terms_of<MODE>(a.l) * 2;
      dq[2] = uniform(left > 0 ? GATHER ? static_cast<uint32_t>(a.l.x_rows) * line : S::Q * line : 0);
      dp[2] = uniform(left > 0 ? MODE == kLinForward ? S::P * line : pstep : 0);
    } else {
      const uint32_t have = min(max(left, 0), kJ);
      dq[2] = uniform(have * a.l.n_out * 2);
      dp[2] = uniform(GATHER ? (left > 0 ? static_cast<uint32_t>(a.l.x_rows * a.l.k * 2) : 0) : have * a.l.k * 2);
    }
  }
  // The step's indexes, which lie at LDS byte `from`; and this lane's offsets from them.
  __device__ __forceinline__ void load_index(uint32_t from, int lane) {
    static_assert(!STEPWISE || (S::P == 256 && S::PCOPIES == 2), "two copies of two lines");
    typedef __attribute__((address_space(3))) const volatile uint32_t lds_u32_t;
    const lds_u32_t *r = reinterpret_cast<lds_u32_t *>(from + (lane >> 5) * 4);
#pragma unroll
    for (int i = 0; i < S::PCOPIES; ++i) at[i] = r[2 * i];
  }
  __device__ __forceinline__ void gather(const Args &a, int wave, int lane) {
#pragma unroll
    for (int i = 0; i < S::PCOPIES; ++i) {
      const uint32_t o = at[i] * static_cast<uint32_t>(a.l.k * 2) + pcol;
      p[i] = 2 * (S::WAVES * i + wave) + (lane >> 5) < left ? o : kNoColumn;
    }
  }
  // Copy number i of the step into the stage at LDS byte m0 (this wave's first KB).
  __device__ __forceinline__ void copy(int i, uint32_t m0) const {
    const int pi = i - S::QCOPIES;
    m0 += i * 1024 * S::WAVES;
    if (pi < 0) dma16b(q[i], dq, m0);
    else dma16b(p[pi], dp, m0);
  }
};

// Indexes of a gathered x, for one wave: it needs four rows a step, so that one copy of
// 64 dwords brings sixteen steps' into a slot of its own, in a ring of four.  They come
// four steps ahead and are read one step ahead, when a wait for copies has covered them.  (As scalar loads
// they cost a sixth of the products: every wait for LDS reads then waits for them too.)
template <typename S>
struct IndexStream {
  static constexpr int STEPS = 16, SLOTS = 4, BYTES = SLOTS * S::WAVES * 256;
  u32x4_t desc;
  uint32_t base;           // this wave's part of slot 0
  int issue, use, pos;     // slot to fill, slot in use, step in it
  int row, end;            // first row of the next chunk of the tile, and the group's end

  __device__ __forceinline__ void init(const Args &a, uint32_t lds, int wave) {
    desc = descriptor(a.l.index, a.l.max_rows * 4);
    base = lds + wave * 256;
    issue = 0;
    use = pos = 0;
  }
  static __device__ __forceinline__ uint32_t slot(int i) { return i * S::WAVES * 256; }
  __device__ __forceinline__ void chunk(int wave, int lane) {
    const int r = row + (lane >> 2) * kJ + 2 * (S::WAVES * ((lane >> 1) & 1) + wave) + (lane & 1);
    dma4b(r < end ? static_cast<uint32_t>(r) * 4 : kNoColumn, desc, base + slot(issue));
    issue = (issue + 1) % SLOTS;
    row += STEPS * kJ;
  }
  // The first chunk of a tile that comes next.
  __device__ __forceinline__ void start(const Tile &t, int wave, int lane) {
    row = static_cast<int>(t.row0) + t.s0 * kJ;
    end = static_cast<int>(t.row0) + t.rows;
    chunk(wave, lane);
  }
  __device__ __forceinline__ uint32_t place() const { return base + slot(use) + pos * 16; }
  // At a step behind which `left` steps of its tile are left: to the next one.
  __device__ __forceinline__ void next(int left, int wave, int lane) {
    if (pos == STEPS - 4 && left > 3) chunk(wave, lane);
    pos = left > 0 ? (pos + 1) % STEPS : 0;
    if (pos == 0) use = (use + 1) % SLOTS;
  }
};

__device__ __forceinline__ float sum8(bf16x8_t v) {
  float s = 0.0f;
#pragma unroll
  for (int i = 0; i < 8; ++i) s += static_cast<float>(v[i]);
  return s;
}

// Reads of the fragments of one slice (16 j), number i of them: rows first.
template <typename S, int MODE>
struct Reader {
  uint32_t q[S::QB], p[S::PB];           // this lane's byte addresses in stage 0
  __device__ __forceinline__ void init(uint32_t ring, int wq, int wp, int lane) {
#pragma unroll
    for (int i = 0; i < S::QB; ++i) {
      if constexpr (MODE != kLinWeightGrad) {
        q[i] = ring + along(wq * S::QB + i, lane);
      } else {
        q[i] = ring + turned_at<S::Q>(wq * S::QB + i, lane);
      }
    }
#pragma unroll
    for (int i = 0; i < S::PB; ++i)
      p[i] = ring + S::QBYTES + (MODE == kLinForward ? along(wp * S::PB + i, lane) : turned_at<S::P>(wp * S::PB + i, lane));
  }
  static __device__ __forceinline__ uint32_t along(int block, int lane) {
    const int row = block * 32 + (lane & 31);
    return row * 64 + (((lane >> 5) ^ ((row >> 2) & 3)) << 4);
  }
  __device__ __forceinline__ void read(Frags<S> &f, uint32_t stage, int slice, int i) const {
    if (i < S::QB) {
      if constexpr (MODE != kLinWeightGrad)   // pieces 2 slice + half: slice flips bit 1
        f.q[i] = *reinterpret_cast<lds_bf16x8_t *>((q[i] ^ (slice << 5)) + stage);
      else
        f.q[i] = read_turned<S::Q>(q[i] + stage + slice * (16 * S::Q * 2));
    } else if constexpr (MODE == kLinForward) {
      f.p[i - S::QB] = *reinterpret_cast<lds_bf16x8_t *>((p[i - S::QB] ^ (slice << 5)) + stage);
    } else {
      f.p[i - S::QB] = read_turned<S::P>(p[i - S::QB] + stage + slice * (16 * S::P * 2));
    }
  }
};

// ---------------------------------------------------------------------------
// A tile's sums to memory
// ---------------------------------------------------------------------------
// Each wave takes its blocks through 4 KB of LDS of its own, so that stores are whole
// lines of 128 bytes: a lane holds four columns of each of 32 rows, and storing those
// as they are took 417 us of 741 for 1.48 GB of weight gradients.  Rows of 128 bytes
// keep their 16-byte piece c at c ^ (row % 8).
// Lanes hand elements to each other there: LDS operations of one wave run in order, and
// this keeps the compiler from moving or merging them across lanes' accesses.
__device__ __forceinline__ void wave_order() {
  __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
  __builtin_amdgcn_wave_barrier();
  asm volatile("" ::: "memory");
}

// v plus four bf16.
__device__ __forceinline__ void add4(float (&v)[4], uint2 z) {
  v[0] += __uint_as_float(z.x << 16), v[1] += __uint_as_float(z.x & 0xFFFF0000u);
  v[2] += __uint_as_float(z.y << 16), v[3] += __uint_as_float(z.y & 0xFFFF0000u);
}

template <typename S>
constexpr int kStores16 = S::QB * (S::PB / 2) * 4;   // stores of a wave's tile in bf16

// float32: 32 x 32 elements a pass.  PART: a part of a split sum, which is read again at
// once and stays in the caches.
template <typename S, bool PART>
__device__ __forceinline__ void out_f32(const f32x16_t (&acc)[S::PB][S::QB], char *lds, u32x4_t dst, int pitch, int r0,
                                        int c0, int columns, bool accumulate, int lane) {
  const int piece = lane & 7;
#pragma unroll
  for (int qi = 0; qi < S::QB; ++qi)
#pragma unroll
    for (int pi = 0; pi < S::PB; ++pi) {
      const int w = lane & 31;
#pragma unroll
      for (int b = 0; b < 4; ++b)
        *reinterpret_cast<float4 *>(lds + w * 128 + (((b * 2 + (lane >> 5)) ^ (w & 7)) << 4)) =
            make_float4(acc[pi][qi][4 * b], acc[pi][qi][4 * b + 1], acc[pi][qi][4 * b + 2], acc[pi][qi][4 * b + 3]);
      wave_order();
      const int c = c0 + pi * 32 + piece * 4;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 3);
        u32x4_t v = *reinterpret_cast<const u32x4_t *>(lds + r * 128 + ((piece ^ (r & 7)) << 4));
        const uint32_t at = c < columns ? (static_cast<uint32_t>(r0 + qi * 32 + r) * pitch + c) * 4 : kNoColumn;
        if (!PART && accumulate) {
          const u32x4_t z = load16b(at, dst);
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = __float_as_uint(__uint_as_float(v[e]) + __uint_as_float(z[e]));
        }
        store16b<!PART>(at, dst, v);
      }
      wave_order();
    }
}

// bf16: 32 x 64 elements a pass, with C's biases (or null) added and through the SiLU.
template <typename S, bool SILU>
__device__ __forceinline__ void out_bf16(const f32x16_t (&acc)[S::PB][S::QB], char *lds, u32x4_t dst, int pitch, int r0,
                                         int c0, int columns, const uint16_t *bias, int lane) {
  const int piece = lane & 7;
#pragma unroll
  for (int qi = 0; qi < S::QB; ++qi)
#pragma unroll
    for (int pp = 0; pp < S::PB / 2; ++pp) {
      const int w = lane & 31;
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const f32x16_t &x = acc[pp * 2 + h / 4][qi];
        const int b = h % 4;
        float v[4] = {x[4 * b], x[4 * b + 1], x[4 * b + 2], x[4 * b + 3]};
        const int bc = c0 + pp * 64 + h * 8 + (lane >> 5) * 4;
        if (bias && bc < columns) add4(v, *reinterpret_cast<const uint2 *>(bias + bc));
        if (SILU)
#pragma unroll
          for (int e = 0; e < 4; ++e) v[e] = silu_fast(v[e]);
        *reinterpret_cast<uint2 *>(lds + w * 128 + ((h ^ (w & 7)) << 4) + ((lane >> 5) << 3)) =
            make_uint2(pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]));
      }
      wave_order();
      const int c = c0 + pp * 64 + piece * 8;
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int r = i * 8 + (lane >> 3);
        const u32x4_t v = *reinterpret_cast<const u32x4_t *>(lds + r * 128 + ((piece ^ (r & 7)) << 4));
        store16b(c < columns ? (static_cast<uint32_t>(r0 + qi * 32 + r) * pitch + c) * 2 : kNoColumn, dst, v);
      }
      wave_order();
    }
}

// bf16 with another array of C's shape: `other` added (dw as it was), or its SiLU's
// slope as a factor.  The sums stay float32 until then: 16 x 64 elements a pass, rows of
// 256 bytes with piece c at c ^ row; the other array comes a pass ahead.
template <typename S, bool SLOPE>
__device__ __forceinline__ void out_bf16_with(const f32x16_t (&acc)[S::PB][S::QB], char *lds, u32x4_t dst, u32x4_t other,
                                              int pitch, int r0, int c0, int columns, int lane) {
  constexpr int PASSES = S::QB * (S::PB / 2) * 2;
  const int piece = lane & 7;
  auto where = [&](int pass, int i) {
    const int qi = pass / S::PB, pp = pass / 2 % (S::PB / 2), half = pass & 1;
    const int r = r0 + qi * 32 + half * 16 + i * 8 + (lane >> 3), c = c0 + pp * 64 + piece * 8;
    return c < columns ? (static_cast<uint32_t>(r) * pitch + c) * 2 : kNoColumn;
  };
  u32x4_t z[2][2];
#pragma unroll
  for (int i = 0; i < 2; ++i) z[0][i] = load16b(where(0, i), other);
#pragma unroll
  for (int pass = 0; pass < PASSES; ++pass) {
    const int qi = pass / S::PB, pp = pass / 2 % (S::PB / 2), half = pass & 1, w = lane & 15;
    if (pass + 1 < PASSES)
#pragma unroll
      for (int i = 0; i < 2; ++i) z[(pass + 1) & 1][i] = load16b(where(pass + 1, i), other);
    if (((lane >> 4) & 1) == half)
#pragma unroll
      for (int h = 0; h < 8; ++h) {
        const f32x16_t &x = acc[pp * 2 + h / 4][qi];
        const int b = h % 4;
        *reinterpret_cast<float4 *>(lds + w * 256 + (((h * 2 + (lane >> 5)) ^ w) << 4)) =
            make_float4(x[4 * b], x[4 * b + 1], x[4 * b + 2], x[4 * b + 3]);
      }
    wave_order();
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int r = i * 8 + (lane >> 3);
      float v[8];
#pragma unroll
      for (int h = 0; h < 2; ++h) {
        const float4 f = *reinterpret_cast<const float4 *>(lds + r * 256 + (((piece * 2 + h) ^ r) << 4));
        v[4 * h] = f.x, v[4 * h + 1] = f.y, v[4 * h + 2] = f.z, v[4 * h + 3] = f.w;
      }
      const u32x4_t o = z[pass & 1][i];
#pragma unroll
      for (int e = 0; e < 8; ++e) {
        const float u = __uint_as_float(e & 1 ? o[e / 2] & 0xFFFF0000u : o[e / 2] << 16);
        v[e] = SLOPE ? v[e] * silu_slope(u) : v[e] + u;
      }
      const u32x4_t packed = {pack_bf16x2(v[0], v[1]), pack_bf16x2(v[2], v[3]), pack_bf16x2(v[4], v[5]),
                              pack_bf16x2(v[6], v[7])};
      store16b(where(pass, i), dst, packed);
    }
    wave_order();
  }
}

template <typename O>
__device__ __forceinline__ void store_bias(O *d, float v, bool accumulate) {
  *d = Act<O>::from_f32(accumulate ? Act<O>::to_f32(*d) + v : v);
}

// ---------------------------------------------------------------------------
// Kernel
// ---------------------------------------------------------------------------
template <typename S, int MODE, bool GATHER>
__global__ __launch_bounds__(S::NT, S::WGS * S::WAVES / 4) void linear_mfma_kernel(Args a) {
  constexpr bool STEPWISE = Source<S, MODE, GATHER>::STEPWISE;
  constexpr int QB = S::QB, PB = S::PB, NF = QB + PB, NM = QB * PB, GROUPS = 8, PER = NM / GROUPS, RING = S::RING;
  static_assert(NM % GROUPS == 0 && NF <= GROUPS && RING >= 3, "reads among the products, two steps ahead");
  // The copies of a step are spread over the half step behind the barrier that frees its
  // stage, and the half step after: together they would wait for each other.
  constexpr int EARLY = S::COPIES / 2, LATE = S::COPIES - EARLY;
  static_assert(EARLY * 2 <= GROUPS && LATE * 2 <= GROUPS, "at most one for two products");
  __shared__ __attribute__((aligned(1024))) char s_ring[RING * S::STAGE];
  __shared__ int s_pref[kMaxGroups + 1], s_off[kMaxGroups + 1], s_tmp[S::WAVES];
  __shared__ __attribute__((aligned(256))) char s_index[STEPWISE ? IndexStream<S>::BYTES : GATHER ? RowIndex<S>::BYTES : 4];
  const int tid = threadIdx.x, lane = tid & 63, wave = uniform(tid >> 6);
  // Waves w and w + 4 share a SIMD: with blocks that lie behind a tile's rows (or columns)
  // left out, the SIMDs still have about the same to multiply.
  const int wp = wave / S::QW, wq = (wave + wp * (S::QW / 2)) % S::QW;
  // workgroups are dealt to the XCDs in turn
  const Plan plan = make_plan<S, MODE>(a, s_pref, s_off, s_tmp, blockIdx.x % kXcds);
  const int stride = gridDim.x / kXcds;
  int item = plan.first + blockIdx.x / kXcds;
  if (item >= plan.end) return;

  const uint32_t ring = uniform(static_cast<int>(dma::lds_addr(s_ring)));
  const uint32_t base = ring + wave * 1024;
  Reader<S, MODE> rd;
  rd.init(ring, wq, wp, lane);

  // The stream of steps: `fill` is the tile whose steps are being copied, RING ahead of
  // the one that is multiplied.  A tile has RING steps at least, so that `fill` is that
  // one's tile or the next.
  Source<S, MODE, GATHER> src;
  constexpr bool ROWWISE = GATHER && !STEPWISE;
  IndexStream<S> rows;
  RowIndex<S> once;
  int fill_item = item;
  Tile fill = tile_at<S, MODE>(a, plan, s_pref, s_off, item, 0), ahead = fill;
  int fill_left = max(fill.s1 - fill.s0, RING), steps = fill_left;   // the one at hand among them
  // Four steps before a tile's end, the next one is looked up.
  auto look_ahead = [&]() {
    static_assert(RING >= 4, "a tile has four steps at least");
    if (fill_left != 4 || fill_item + stride >= plan.end) return;
    ahead = tile_at<S, MODE>(a, plan, s_pref, s_off, fill_item + stride, fill.g);
    if constexpr (STEPWISE) rows.start(ahead, wave, lane);
    if constexpr (ROWWISE) once.start(ahead, wave, lane);
  };
  // The next tile, where this one's steps are all copied; then the next step.
  bool fresh = false;
  auto next_tile = [&]() {
    if (fill_left > 1) return;
    fill_item += stride;
    if (fill_item < plan.end) {
      int el = lane;
      asm volatile("" : "+v"(el));       // as for the sums below
      fill = ahead;
      src.init(a, fill, ROWWISE ? once.place() : 0, wave, el);
      fill_left = max(fill.s1 - fill.s0, RING) + 1;
      fresh = true;
    } else {
      src.none(a);
      fill_left = 0x7FFFFFFF;
    }
  };
  auto next_step = [&]() {
    if (!fresh) src.advance(a);
    --fill_left;
    fresh = false;
    if constexpr (STEPWISE) src.gather(a, wave, lane);
    look_ahead();
    if constexpr (STEPWISE) {
      rows.next(fill_left - 1, wave, lane);
      src.load_index(rows.place(), lane);
    }
  };
  if constexpr (ROWWISE) {
    once.init(a, uniform(static_cast<int>(dma::lds_addr(s_index))), wave);
    once.start(fill, wave, lane);
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
  }
  src.init(a, fill, ROWWISE ? once.place() : 0, wave, lane);
  if constexpr (STEPWISE) {
    rows.init(a, uniform(static_cast<int>(dma::lds_addr(s_index))), wave);
    rows.start(fill, wave, lane);
  }
  look_ahead();
  if constexpr (STEPWISE) {
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");   // no copies yet that would cover these
    src.load_index(rows.place(), lane);
    src.gather(a, wave, lane);
    rows.next(fill_left - 1, wave, lane);
    src.load_index(rows.place(), lane);
  }
#pragma unroll
  for (int s = 0; s < RING; ++s) {
#pragma unroll
    for (int i = 0; i < (s == RING - 1 ? EARLY : S::COPIES); ++i) src.copy(i, base + s * S::STAGE);
    if (s < RING - 1) next_step();
  }
  dma::wait_and_barrier<(RING - 2) * S::COPIES + EARLY>();
  Frags<S> f0, f1;
#pragma unroll
  for (int i = 0; i < NF; ++i) rd.read(f0, 0, 0, i);

  Tile t = fill;
  uint32_t stage = 0;
  bool stored = false;                   // this wave's last tile had stores
  f32x16_t acc[PB][QB];
  auto before = [&](uint32_t at) { return at == 0 ? (RING - 1) * S::STAGE : at - S::STAGE; };
  auto after = [&](uint32_t at) { return at == (RING - 1) * S::STAGE ? 0u : at + S::STAGE; };
  // products of fragments f; after the first product of group i, `start(i)` starts reads
  // or copies
  auto multiply = [&](const Frags<S> &f, auto start) {
#pragma unroll
    for (int i = 0; i < GROUPS; ++i) {
#pragma unroll
      for (int m = i * PER; m < (i + 1) * PER; ++m) {
        acc[m / QB][m % QB] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(f.p[m / QB], f.q[m % QB], acc[m / QB][m % QB], 0, 0, 0);
        if (m == i * PER) {
          __builtin_amdgcn_sched_barrier(0);
          start(i);
        }
      }
      __builtin_amdgcn_sched_barrier(0);
    }
  };
  // Fragments of the next slice, the last of them some products before the barrier that
  // waits for it.
  auto read_some = [&](Frags<S> &f, uint32_t at, int slice, int group) {
    constexpr int AHEAD = NF > 6 ? NF - 6 : 0;             // all read after six groups
#pragma unroll
    for (int i = 0; i < NF; ++i)
      if ((i < 2 * AHEAD ? i / 2 : i - AHEAD) == group) rd.read(f, at, slice, i);
  };

  while (true) {
#pragma unroll
    for (int p = 0; p < PB; ++p)
#pragma unroll
      for (int q = 0; q < QB; ++q)
#pragma unroll
        for (int i = 0; i < 16; ++i) acc[p][q][i] = 0.0f;
    float bias[QB];
#pragma unroll
    for (int q = 0; q < QB; ++q) bias[q] = 0.0f;
    const int nq = (MODE == kLinWeightGrad ? a.l.n_out : t.rows) - t.q0, np = columns_of<MODE>(a.l);
    const bool busy = wq * QB * 32 < nq && t.p0 + wp * PB * 32 < np;   // blocks of this wave are there
    const bool sum_dy = MODE == kLinWeightGrad && a.l.dbias && t.p0 == 0 && wp == 0;
    auto add_dy = [&](const Frags<S> &f) {
      if (sum_dy)
#pragma unroll
        for (int q = 0; q < QB; ++q) bias[q] += sum8(f.q[q]);
    };
    // First half of a step, with the rest of the last step's copies.
    auto half = [&]() {
      const uint32_t old = base + before(stage);
      if (busy) {
        multiply(f0, [&](int i) {
          read_some(f1, stage, 1, i);
          if (i % (GROUPS / LATE) == 1 && i / (GROUPS / LATE) < LATE) src.copy(EARLY + i / (GROUPS / LATE), old);
        });
        add_dy(f0);
      } else {
#pragma unroll
        for (int i = 0; i < LATE; ++i) src.copy(EARLY + i, old);
      }
    };
    // Second half, behind the barrier: this step's stage is read, the next one has landed.
    auto rest = [&]() {
      const uint32_t next = after(stage);
      if (busy) {
        multiply(f1, [&](int i) {
          if (i == 0) next_step();
          read_some(f0, next, 0, i);
          if (i % (GROUPS / EARLY) == 1 && i / (GROUPS / EARLY) < EARLY) src.copy(i / (GROUPS / EARLY), base + stage);
        });
        add_dy(f1);
      } else {
        next_step();
#pragma unroll
        for (int i = 0; i < EARLY; ++i) src.copy(i, base + stage);
      }
      stage = next;
    };
    // The last tile's stores are younger than the next stage's copies in these steps.
    for (int s = 0; s < RING - 2; ++s) {
      half();
      next_tile();
      if (stored) dma::wait_and_barrier<(RING - 2) * S::COPIES + kStores16<S>>();
      else dma::wait_and_barrier<(RING - 2) * S::COPIES>();
      __builtin_amdgcn_sched_barrier(0);
      rest();
    }
    for (int s = RING - 2; s < steps - 1; ++s) {
      half();
      next_tile();
      dma::wait_and_barrier<(RING - 2) * S::COPIES>();
      __builtin_amdgcn_sched_barrier(0);
      rest();
    }
    half();
    next_tile();
    dma::wait_and_barrier<(RING - 2) * S::COPIES>();
    __builtin_amdgcn_sched_barrier(0);
    const uint32_t next = after(stage);
    if (busy) {
      multiply(f1, [&](int i) { read_some(f0, next, 0, i); });
      add_dy(f1);
    } else {
      // the next tile may have work for this wave
#pragma unroll
      for (int i = 0; i < NF; ++i) rd.read(f0, next, 0, i);
    }
    stored = busy;

    // the sums, by way of the stage just read.  The lane is hidden from the compiler, or
    // it would keep the offsets of every pass in registers through all tiles.
    int el = lane;
    asm volatile("" : "+v"(el));
    char *lds = s_ring + stage + wave * 4096;
    const int r0 = wq * QB * 32, c0 = t.p0 + wp * PB * 32;
    if (!busy) {
    } else if (plan.parts > 1) {
      float *part = a.part + static_cast<int64_t>(item) * S::PART;
      out_f32<S, true>(acc, lds, descriptor(part, S::Q * S::P * 4), S::P, r0, wp * PB * 32, S::P, false, el);
    } else {
      const int64_t row = (MODE == kLinWeightGrad ? static_cast<int64_t>(t.g) * a.l.n_out : t.row0) + t.q0;
      const int64_t size = static_cast<int64_t>(min(S::Q, nq)) * np;
      if (MODE == kLinWeightGrad && !a.l.out_bf16) {
        out_f32<S, false>(acc, lds, descriptor(static_cast<float *>(a.l.out) + row * np, size * 4), np, r0, c0, np,
                   a.l.accumulate, el);
      } else {
        const u32x4_t dst = descriptor(static_cast<uint16_t *>(a.l.out) + row * np, size * 2);
        if (MODE == kLinForward) {
          const uint16_t *bias =
              a.l.bias ? static_cast<const uint16_t *>(a.l.bias) + static_cast<int64_t>(t.g) * np : nullptr;
          if (a.l.pre)
            out_bf16<S, false>(acc, lds, descriptor(static_cast<uint16_t *>(a.l.pre) + row * np, size * 2), np, r0, c0, np,
                               bias, el);
          if (a.l.silu) out_bf16<S, true>(acc, lds, dst, np, r0, c0, np, bias, el);
          else out_bf16<S, false>(acc, lds, dst, np, r0, c0, np, bias, el);
        } else if (MODE == kLinInputGrad && a.l.act_pre)
          out_bf16_with<S, true>(acc, lds, dst, descriptor(static_cast<const uint16_t *>(a.l.act_pre) + row * np, size * 2),
                                 np, r0, c0, np, el);
        else if (MODE == kLinWeightGrad && a.l.accumulate)
          out_bf16_with<S, false>(acc, lds, dst, dst, np, r0, c0, np, el);
        else
          out_bf16<S, false>(acc, lds, dst, np, r0, c0, np, nullptr, el);
      }
    }
    if (sum_dy && busy)
#pragma unroll
      for (int i = 0; i < QB; ++i) {
        const float v = bias[i] + __shfl_xor(bias[i], 32);
        const int q = t.q0 + r0 + i * 32 + (el & 31);
        if (el >= 32) continue;
        if (plan.parts > 1) {
          a.part[static_cast<int64_t>(item) * S::PART + S::Q * S::P + q - t.q0] = v;
        } else if (q < a.l.n_out) {
          const int64_t o = static_cast<int64_t>(t.g) * a.l.n_out + q;
          if (a.l.out_bf16) store_bias(static_cast<uint16_t *>(a.l.dbias) + o, v, a.l.accumulate);
          else store_bias(static_cast<float *>(a.l.dbias) + o, v, a.l.accumulate);
        }
      }
    item += stride;
    if (item >= plan.end) break;
    // every wave is through with the stage; its copies now make `fill` the next tile
    lds_barrier();
    next_step();
#pragma unroll
    for (int i = 0; i < EARLY; ++i) src.copy(i, base + stage);
    t = fill;
    steps = max(t.s1 - t.s0, RING);
    stage = next;
  }
  // copies in flight write to LDS, which may be another workgroup's once this one ends
  dma::wait_and_barrier<0>();
}

template <typename S>
struct Threads256 : S {
  static constexpr int NT = 256;
};

// Sums of the parts of split tiles, in order, and what the kernel would have done with
// them.  32 workgroups a tile, float4 a thread, several parts on their way together (with
// 16 workgroups and one part after another, 9 tiles of 28 parts took 51 us).
constexpr int kPartGroups = 32;
template <typename S, int MODE>
__global__ __launch_bounds__(256) void linear_mfma_parts_kernel(Args a) {
  __shared__ int s_pref[kMaxGroups + 1], s_off[kMaxGroups + 1], s_tmp[4];
  const Plan plan = make_plan<Threads256<S>, MODE>(a, s_pref, s_off, s_tmp, 0);
  const int at = blockIdx.x / kPartGroups;
  if (plan.parts <= 1 || at >= plan.tiles) return;
  const Tile t = tile_at<S, MODE>(a, plan, s_pref, s_off, at * plan.parts, 0);
  const float *part = a.part + static_cast<int64_t>(at) * plan.parts * S::PART;
  const int np = columns_of<MODE>(a.l), rows = MODE == kLinWeightGrad ? a.l.n_out : t.rows;
  const int64_t row = (MODE == kLinWeightGrad ? static_cast<int64_t>(t.g) * a.l.n_out : t.row0) + t.q0;
  constexpr int kEach = S::Q * S::P / 4 / kPartGroups;   // float4 of a workgroup
  for (int e = threadIdx.x; e < kEach; e += 256) {
    const int i = (blockIdx.x % kPartGroups) * kEach + e, r = i / (S::P / 4), c = i % (S::P / 4) * 4;
    if (t.q0 + r >= rows || t.p0 + c >= np) continue;
    float4 v = make_float4(0.0f, 0.0f, 0.0f, 0.0f);
#pragma unroll 8
    for (int k = 0; k < plan.parts; ++k) {
      const float4 x = *reinterpret_cast<const float4 *>(part + static_cast<int64_t>(k) * S::PART + i * 4);
      v.x += x.x, v.y += x.y, v.z += x.z, v.w += x.w;
    }
    const int64_t o = (row + r) * np + t.p0 + c;
    if (MODE == kLinWeightGrad && !a.l.out_bf16) {
      float4 *d = reinterpret_cast<float4 *>(static_cast<float *>(a.l.out) + o);
      if (a.l.accumulate) {
        const float4 z = *d;
        v.x += z.x, v.y += z.y, v.z += z.z, v.w += z.w;
      }
      *d = v;
    } else {
      uint2 *d = reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.l.out) + o);
      if (MODE == kLinForward) {
        float u[4] = {v.x, v.y, v.z, v.w};
        if (a.l.bias)
          add4(u, *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.l.bias) + static_cast<int64_t>(t.g) * np +
                                                   t.p0 + c));
        v = make_float4(u[0], u[1], u[2], u[3]);
        if (a.l.pre)
          *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(a.l.pre) + o) =
              make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        if (a.l.silu) v.x = silu_fast(v.x), v.y = silu_fast(v.y), v.z = silu_fast(v.z), v.w = silu_fast(v.w);
      } else if (MODE == kLinWeightGrad ? a.l.accumulate : a.l.act_pre != nullptr) {
        const uint2 z = MODE == kLinWeightGrad
                            ? *d : *reinterpret_cast<const uint2 *>(static_cast<const uint16_t *>(a.l.act_pre) + o);
        const float u[4] = {__uint_as_float(z.x << 16), __uint_as_float(z.x & 0xFFFF0000u), __uint_as_float(z.y << 16),
                            __uint_as_float(z.y & 0xFFFF0000u)};
        if (MODE == kLinWeightGrad)
          v.x += u[0], v.y += u[1], v.z += u[2], v.w += u[3];
        else
          v.x *= silu_slope(u[0]), v.y *= silu_slope(u[1]), v.z *= silu_slope(u[2]), v.w *= silu_slope(u[3]);
      }
      *d = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
    }
  }
  if (MODE == kLinWeightGrad && a.l.dbias && t.p0 == 0 && blockIdx.x % kPartGroups == 0)
    for (int r = threadIdx.x; r < S::Q && t.q0 + r < rows; r += 256) {
      float v = 0.0f;
      for (int k = 0; k < plan.parts; ++k) v += part[static_cast<int64_t>(k) * S::PART + S::Q * S::P + r];
      const int64_t o = row + r;
      if (a.l.out_bf16) store_bias(static_cast<uint16_t *>(a.l.dbias) + o, v, a.l.accumulate);
      else store_bias(static_cast<float *>(a.l.dbias) + o, v, a.l.accumulate);
    }
}

// Rows of the longest group that the choices below count on: four times the mean's.
int64_t longest_rows(int groups, int64_t max_rows) {
  return max_rows / groups < max_rows / 4 ? max_rows / groups * 4 + 4 : max_rows;
}

// Tiles at most, and parts of a tile at most (1: the sizes never need a split).
template <typename S>
int64_t tile_bound(int mode, int groups, int n_out, int k, int64_t max_rows) {
  const int64_t pt = ((mode == kLinForward ? n_out : k) + S::P - 1) / S::P;
  if (mode == kLinWeightGrad) return pt * groups * ((n_out + S::Q - 1) / S::Q);
  return pt * (max_rows / S::Q + (max_rows < groups ? max_rows : groups));
}
template <typename S>
int part_bound(int mode, int groups, int n_out, int k, int64_t max_rows) {
  if (tile_bound<S>(mode, groups, n_out, k, max_rows) > S::SLOTS) return 1;
  // groups of several times the mean's rows are split, where all are short nothing is
  const int64_t rows = longest_rows(groups, max_rows);
  const int64_t steps = mode == kLinWeightGrad ? (rows + kJ - 1) / kJ : (mode == kLinForward ? k : n_out) / kJ;
  const int64_t parts = steps / kMinSteps;
  return static_cast<int>(parts < 1 ? 1 : parts < S::SLOTS ? parts : S::SLOTS);
}

template <typename S, int MODE, bool GATHER>
void launch_mode(const Args &a, hipStream_t s) {
  const int64_t items = tile_bound<S>(MODE, a.l.groups, a.l.n_out, a.l.k, a.l.max_rows) * a.most_parts;
  const int64_t want = (items + kXcds - 1) / kXcds * kXcds;
  hipLaunchKernelGGL((linear_mfma_kernel<S, MODE, GATHER>), dim3(static_cast<unsigned>(want < S::SLOTS ? want : S::SLOTS)),
                     dim3(S::NT), 0, s, a);
  if (a.most_parts > 1) {
    const int64_t tiles = tile_bound<S>(MODE, a.l.groups, a.l.n_out, a.l.k, a.l.max_rows);
    const int64_t split = tiles < S::SLOTS / 2 ? tiles : S::SLOTS / 2;
    hipLaunchKernelGGL((linear_mfma_parts_kernel<S, MODE>), dim3(static_cast<unsigned>(split * kPartGroups)), dim3(256), 0, s, a);
  }
}

template <typename S>
hipError_t launch_shape(const Linear &p, void *ws, hipStream_t s) {
  const Args a{p, static_cast<float *>(ws), part_bound<S>(p.mode, p.groups, p.n_out, p.k, p.max_rows)};
  if (p.mode == kLinInputGrad) launch_mode<S, kLinInputGrad, false>(a, s);
  else if (p.mode == kLinForward && p.index) launch_mode<S, kLinForward, true>(a, s);
  else if (p.mode == kLinForward) launch_mode<S, kLinForward, false>(a, s);
  else if (p.index && p.max_rows > 0) launch_mode<S, kLinWeightGrad, true>(a, s);
  else launch_mode<S, kLinWeightGrad, false>(a, s);
  return hipGetLastError();
}

using Tiles = Shape<2, 4, 4>;

// The forward goes here from 64 rows a group on, up to 512 where there are more than 256
// tiles; below, the layer's kernels stream weights faster, above, their 256 x 256 tiles are.
// Layer's kernels / this one, us in a graph over two sets of operands, by rows of each group:
//   groups x n_out x k     16       32       64      128      256      512     1024
//   8 x 2048 x 2048      27/27    35/27    39/27    52/31    38/47    45/58    62/63
//   64 x 2048 x 2048    115/142  124/141  144/146  151/153  194/171  268/287  482/547
//   64 x 512 x 4096      77/97    82/95    98/97   101/105  160/144  159/155  261/272
//   64 x 4096 x 512      66/67    66/64    74/69    88/77   122/99   185/174  346/355
//   8 x 14336 x 4096    183/185  217/231  231/223  286/233  279/283  438/481  769/844
//   64 x 192 x 512       16/23    18/23    21/24    27/26    23/29    24/40    30/24
// and of unequal lengths (shares of a Zipf law of exponent 0.8), by the mean:
//   8 x 2048 x 2048      28/26    38/29    64/32    64/36    66/42    48/50    87/98
//   64 x 2048 x 2048    151/148  158/179  172/179  180/178  241/202  326/318  546/560
//   64 x 1408 x 2048    119/113  124/100  132/111  140/115  176/163  247/237  410/414
// At 384 rows of 2048 x 2048 it is 297/248, so that groups of exactly two of the layer's tiles
// are the exception there.  The device alone knows the lengths; the choice is by the mean.  It
// is the wrong one where tiles fill a quarter to a half of the CUs and are split, since writing
// and adding the parts then costs more than shorter sums save (8 x 2048 x 2048 at 256 and 512
// rows, 8 x 4096 x 512 at 256 25/40), and where a short sum's one tile of columns is partly
// filled (64 x 192 x 512, 28962 rows on 8 x 192 x 512 23/35).  With few tiles and long sums 1221
// rows on 2 x 6272 x 2304 take 74/53, 138 on 1 x 5376 x 128 19/10.
constexpr int64_t kFewTiles = 256;
bool forward_pays(const Linear &p) {
  const int64_t tiles = tile_bound<Tiles>(kLinForward, p.groups, p.n_out, p.k, p.max_rows);
  const int64_t rows = p.max_rows / p.groups;
  return rows >= 64 && (rows <= 512 || tiles <= kFewTiles);
}

// Gradients of short sums and few tiles go through the float32 kernel's 64 x 64 tiles.  Here a
// launch alone takes 7 to 9 us, with a prologue that fills the ring and a code of many lines.
//   Input gradient, in ns, against this kernel: the float32 one takes 2500 less and 40 less
// for every group, 1100 more for each 64 of the sum, and from its 257th tile on 2 and 4 for
// each 64 of the sum more a tile.
//   Weight gradient: the float32 one is the faster up to about 1024 tiles of two steps, 1280
// where they are more than a round here.
// This kernel / the float32 one, us in a graph; groups, rows of all of them (of unequal lengths);
// behind the semicolon the sizes that stay here:
//   input gradient, n_out x k
//     64 x 64      1, 1024 7.2/5.8   64, 4096 9.9/6.3   256, 16384 22/8.1
//     64 x 1024    1, 1024 8.6/6.4   16, 1024 8.7/7.6;  64, 1024 10.7/11.8  16, 16384 17/36
//     128 x 256    64, 1024 10.2/10.2  256, 1024 19.5/17.2;  64, 16384 12/20
//     192 x 64     64, 1024 10.6/9.7   256, 4096 20/13;  16, 1024 8.3/10.0
//     192 x 8192   ;  16, 16 15/37   64, 128 46/143
//   weight gradient, n_out x k
//     64 x 320     1, 64 8/6   64, 128 10/7   256, 128 16/13;  1, 512 13/12
//     320 x 448    4, 64 10/5   16, 256 12/9;  64, 64 14/20
//     2048 x 1408  1, 64 11/10;  1, 128 11/15   4, 2 16/21
bool little(const Linear &p) {
  if (p.mode == kLinForward) return false;
  const int64_t outputs = p.n_out / 64, columns = p.k / 64;
  if (p.mode == kLinWeightGrad) {
    const int64_t tiles = p.groups * outputs * columns, rows = longest_rows(p.groups, p.max_rows);
    const int64_t here = tile_bound<Tiles>(p.mode, p.groups, p.n_out, p.k, p.max_rows);
    return p.max_rows <= 512 && rows <= 128 && tiles <= (here > Tiles::SLOTS ? 1280 : 1024) &&
           tiles * ((rows + kJ - 1) / kJ) <= 2048;
  }
  if (outputs > 4) return false;         // measured up to 256 terms and 256 groups
  const int64_t tiles = columns * (p.max_rows / 64 + (p.max_rows < p.groups ? p.max_rows : p.groups));
  const int64_t behind = tiles > 256 ? tiles - 256 : 0;
  return 1100 * outputs + (2 + 4 * outputs) * behind < 2500 + 40 * p.groups;
}

}  // namespace

// Widths whose lines of a tile stay below 4 GiB, a gathered x and its indexes that do, and
// items that are counted in 31 bits.  Weight gradients of a larger gathered x go through the
// float32 kernel's tiles at a tenth to a quarter of the speed (rows, n_out x k; just below
// 4 GiB / beyond, us: 100000, 64 x 7168 264/1050; 32768, 1024 x 7168 445/4830).
bool linear_mfma_fits(const Linear &p) {
  if (!p.bf16 || p.n_out >= (1 << 20) || p.k >= (1 << 20)) return false;
  if (tile_bound<Tiles>(p.mode, p.groups, p.n_out, p.k, p.max_rows) >= (int64_t(1) << 30)) return false;
  if (little(p) || (p.mode == kLinForward && !forward_pays(p))) return false;
  return p.mode == kLinInputGrad || !p.index || (p.x_rows <= 0xFFFFFE00ll / 2 / p.k && p.max_rows <= 0xFFFFFE00ll / 4);
}

size_t linear_mfma_workspace_bytes(int groups, int n_out, int k, int64_t max_rows) {
  for (int mode : {kLinForward, kLinInputGrad, kLinWeightGrad})
    if (part_bound<Tiles>(mode, groups, n_out, k, max_rows) > 1)
      return static_cast<size_t>(Tiles::SLOTS) * Tiles::PART * sizeof(float);
  return 0;
}

hipError_t launch_linear_mfma(const Linear &p, void *ws, hipStream_t s) {
  return launch_shape<Tiles>(p, ws, s);
}

}  // namespace moe
