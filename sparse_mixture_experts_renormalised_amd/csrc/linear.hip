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
//
// Where there are few tiles, long sums are split along j: parts of a tile go to a
// workspace and a second kernel adds them in order.  A step takes about 1.2 us, however
// few workgroups there are (a load's latency and the products), so that one group of 2967
// rows took 125 us and takes 18.5 in parts of 128 rows (20.6 of 256, 28.2 of 512, 25.7 of
// 64).  So it is for the bf16 gradients that come here with long sums, those of a gathered x
// of 4 GiB and more (400000 rows, 64 x 7168: 16400 us whole, 3800 split) and of widths of 2^20
// and more (3 rows, input gradient through 2^20 outputs to 64: 33700 and 174).
//
// 16 groups of 512 rows, 1024 x 1024: forward 229-241 us, input gradient 205, weight
// gradient 203 (71 to 85 TFLOP/s of the 149 that one large library product reaches), bound
// by the steps' latency at four to five workgroups a CU.  16 to 40 rows on 8 experts of
// 512 x 256: 11 us, eight steps.
#include "linear.h"

namespace moe {
namespace {

typedef float f32x16_t __attribute__((ext_vector_type(16)));

constexpr int kTile = 64, kStep = 32, kPitch = kTile + 4,  kMaxGroups = kMaxRouted + kMaxShared;
constexpr int kPart = kTile * kTile + kTile;   // floats of a part: a tile and its sums of dy
constexpr int kMinChunk = 128;                 // terms of a part, at least
constexpr int kMinTerms = 512;                 // of a split sum (256: 11.7 us split, 11.0 whole)
constexpr int64_t kFewTiles = 512, kItems = 1024;

struct Args {
  Linear l;
  float *part;       // parts of split sums
  int chunk;         // terms of a part (0: nothing is split)
};

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

// Exclusive prefix over the groups, in LDS, of ceil(rows / unit), with `least` at least:
// first 64-row tile of every group, or first part.
__device__ int row_prefix(const Linear &a, int unit, int least, int *pref, int *tmp) {
  const int per = (a.groups + 255) / 256, g0 = min(static_cast<int>(threadIdx.x) * per, a.groups);
  const int g1 = min(g0 + per, a.groups);
  auto tiles = [&](int g) { return max(least, (a.offsets[g + 1] - a.offsets[g] + unit - 1) / unit); };
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

// A thread's share of an operand's step, in 16-byte pieces.  Along j: a lane reads
// neighbouring pieces of a line of its own, so that turning them into LDS needs no bank
// twice (neighbouring lanes on one line took as long: 245 us and 241, 17 GFLOP); else
// neighbouring lanes read those of one j.
template <typename T, bool ALONG_J>
struct Operand {
  static constexpr int E = 16 / sizeof(T);         // elements of a piece
  static constexpr int PIECES = kTile / E, LINES = 256 / PIECES;   // pieces of a j, j of a pass
  static constexpr int N = kStep * kTile / 256 / E;
  uint4 raw[N];
  bool there[N];
  // line (or j) of piece i, and its first element along j (or along the lines)
  static __device__ __forceinline__ int line(int i, int tid) { return ALONG_J ? tid & 63 : i * LINES + tid / PIECES; }
  static __device__ __forceinline__ int at(int i, int tid) {
    return ALONG_J ? ((tid >> 6) * N + i) * E : tid % PIECES * E;
  }
  __device__ __forceinline__ void load(int i, const T *p, bool is_there) {
    raw[i] = *reinterpret_cast<const uint4 *>(p);
    there[i] = is_there;
  }
  __device__ __forceinline__ void store(float (*s)[kPitch], int tid) const {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      union { uint4 q; T e[E]; } u;
      u.q = raw[i];
      float v[E];
#pragma unroll
      for (int e = 0; e < E; ++e) v[e] = there[i] ? Act<T>::to_f32(u.e[e]) : 0.0f;
      if constexpr (ALONG_J) {
#pragma unroll
        for (int e = 0; e < E; ++e) s[at(i, tid) + e][line(i, tid)] = v[e];
      } else {
#pragma unroll
        for (int e = 0; e < E; e += 4)
          *reinterpret_cast<float4 *>(&s[line(i, tid)][at(i, tid) + e]) = make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
      }
    }
  }
};

// Largest g with pref[g] <= v, for v below the total.
__device__ __forceinline__ int group_of(const int *pref, int groups, int64_t v) {
  int lo = 0, hi = groups;
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (pref[mid] <= v) lo = mid; else hi = mid;
  }
  return lo;
}

// x mod d, and x / d in x's place; in 32 bits where x has no more.
__device__ __forceinline__ int remainder(int64_t &x, int d) {
  if (x >> 32) {
    const int64_t q = x / d;
    const int r = static_cast<int>(x - q * d);
    x = q;
    return r;
  }
  const uint32_t v = static_cast<uint32_t>(x), q = v / static_cast<uint32_t>(d);
  x = q;
  return static_cast<int>(v - q * static_cast<uint32_t>(d));
}

// Work items: parts of tiles.  Forward and input gradient have equally many for every
// tile (the part runs fastest), a group of the weight gradient has as its rows ask for
// (the tile runs fastest).
template <int MODE>
struct Items {
  int ptiles, qtiles, parts;   // parts: of every tile (0: of the groups, by pref)
  int64_t total;
  __device__ __forceinline__ Items(const Args &p, int *pref, int *tmp) {
    const Linear &a = p.l;
    ptiles = ((MODE == kLinForward ? a.n_out : a.k) + kTile - 1) / kTile;
    parts = 1;
    if (MODE == kLinWeightGrad) {
      qtiles = (a.n_out + kTile - 1) / kTile;
      const int tiles = qtiles * ptiles;
      if (p.chunk) parts = 0;
      total = static_cast<int64_t>(tiles) * (p.chunk ? row_prefix(a, p.chunk, 1, pref, tmp) : a.groups);
    } else {
      const int nj = MODE == kLinForward ? a.k : a.n_out;
      if (p.chunk) parts = (nj + p.chunk - 1) / p.chunk;
      qtiles = row_prefix(a, kTile, 0, pref, tmp);
      total = static_cast<int64_t>(qtiles) * ptiles * parts;
    }
  }
};

// Four sums of a row of C to memory: bias, SiLU, its slope, or what is there.
template <typename T, typename O, int MODE>
__device__ __forceinline__ void put_sums(const Linear &a, int g, int64_t out_row, int p, float (&v)[4]) {
  const int np = MODE == kLinForward ? a.n_out : a.k;
  O *out = static_cast<O *>(a.out) + out_row * np + p;
  float o[4];
  if (MODE == kLinForward) {
    if (a.bias) {
      get4(static_cast<const T *>(a.bias) + static_cast<int64_t>(g) * a.n_out + p, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] += o[i];
    }
    if (a.pre) put4(static_cast<O *>(a.pre) + out_row * np + p, v);
    if (a.silu)
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] = silu_f32(v[i]);   // bf16's forward is not here
  } else if (MODE == kLinInputGrad) {
    if (a.act_pre) {
      get4(static_cast<const T *>(a.act_pre) + out_row * np + p, o);
#pragma unroll
      for (int i = 0; i < 4; ++i) v[i] *= sizeof(T) == 4 ? silu_slope_f32(o[i]) : silu_slope(o[i]);
    }
  } else if (a.accumulate) {
    get4(out, o);
#pragma unroll
    for (int i = 0; i < 4; ++i) v[i] += o[i];
  }
  put4(out, v);
}
template <typename O>
__device__ __forceinline__ void put_bias(const Linear &a, int g, int q, float v) {
  O *o = static_cast<O *>(a.dbias) + static_cast<int64_t>(g) * a.n_out + q;
  *o = Act<O>::from_f32(a.accumulate ? Act<O>::to_f32(*o) + v : v);
}

template <typename T, typename O, int MODE>
__global__ __launch_bounds__(256) void linear_f32_kernel(Args args) {
  const Linear &a = args.l;
  constexpr bool kQAlongJ = MODE != kLinWeightGrad, kPAlongJ = MODE == kLinForward;
  __shared__ __attribute__((aligned(16))) float s_q[kStep][kPitch], s_p[kStep][kPitch];
  __shared__ int s_pref[kMaxGroups + 1], s_tmp[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int wq = (wave & 1) * 32, wp = (wave >> 1) * 32;
  const int np = MODE == kLinForward ? a.n_out : a.k;                 // extent of p
  const Items<MODE> items(args, s_pref, s_tmp);
  const T *x = static_cast<const T *>(a.x), *dy = static_cast<const T *>(a.dy), *w = static_cast<const T *>(a.w);
  for (int64_t L = blockIdx.x; L < items.total; L += gridDim.x) {
    int part = 0, g, q0;
    int64_t rest = L;
    if (MODE != kLinWeightGrad) part = remainder(rest, items.parts);
    const int p0 = remainder(rest, items.ptiles) * kTile;
    bool split = items.parts > 1;
    if (MODE == kLinWeightGrad) {
      q0 = remainder(rest, items.qtiles) * kTile;
      g = static_cast<int>(rest);
      if (items.parts == 0) {
        g = group_of(s_pref, a.groups, rest);
        part = static_cast<int>(rest) - s_pref[g];
        split = s_pref[g + 1] - s_pref[g] > 1;
      }
    } else {
      g = group_of(s_pref, a.groups, rest);
      q0 = static_cast<int>(rest - s_pref[g]) * kTile;
    }
    const int64_t row0 = a.offsets[g];
    const int rows = a.offsets[g + 1] - static_cast<int>(row0);
    const int nq = MODE == kLinWeightGrad ? a.n_out : rows;
    const int terms = MODE == kLinForward ? a.k : MODE == kLinInputGrad ? a.n_out : rows;
    const int first = split ? part * args.chunk : 0, nj = split ? min(terms, first + args.chunk) : terms;
    const T *wg = w + static_cast<int64_t>(g) * a.n_out * a.k;
    using Q = Operand<T, kQAlongJ>;
    using P = Operand<T, kPAlongJ>;
    Q rq;
    P rp;
    // lines along j; those behind the last, and pieces behind the sum's end, read one that
    // is there
    const T *ql = nullptr, *pl = nullptr;
    if constexpr (kQAlongJ) {
      const int64_t r = row0 + min(q0 + Q::line(0, tid), nq - 1);
      ql = MODE == kLinForward ? x + (a.index ? a.index[r] : r) * a.k : dy + r * a.n_out;
    }
    if constexpr (kPAlongJ) pl = wg + static_cast<int64_t>(min(p0 + P::line(0, tid), np - 1)) * a.k;
    auto fetch = [&](int j0) {
#pragma unroll
      for (int i = 0; i < Q::N; ++i) {
        if constexpr (kQAlongJ) {
          const int j = j0 + Q::at(i, tid);
          rq.load(i, ql + min(j, nj - Q::E), j < nj);
        } else {
          const int j = j0 + Q::line(i, tid);
          rq.load(i, dy + (row0 + min(j, nj - 1)) * a.n_out + min(q0 + Q::at(i, tid), nq - Q::E), j < nj);
        }
      }
#pragma unroll
      for (int i = 0; i < P::N; ++i) {
        if constexpr (kPAlongJ) {
          const int j = j0 + P::at(i, tid);
          rp.load(i, pl + min(j, nj - P::E), j < nj);
        } else {
          const int j = j0 + P::line(i, tid), p = min(p0 + P::at(i, tid), np - P::E);
          const int64_t r = min(j, nj - 1);
          if (MODE == kLinInputGrad)
            rp.load(i, wg + r * a.k + p, j < nj);
          else
            rp.load(i, x + (a.index ? a.index[row0 + r] : row0 + r) * a.k + p, j < nj);
        }
      }
    };
    f32x16_t acc;
#pragma unroll
    for (int i = 0; i < 16; ++i) acc[i] = 0.0f;
    float db = 0.0f;
    const bool sum_dy = MODE == kLinWeightGrad && a.dbias && p0 == 0;
    if (nj > first) fetch(first);
    for (int j0 = first; j0 < nj; j0 += kStep) {
      __syncthreads();
      rq.store(s_q, tid);
      rp.store(s_p, tid);
      __syncthreads();
      if (j0 + kStep < nj) fetch(j0 + kStep);
      // four products while the next four's elements are read (left to itself the compiler
      // reads two products' and waits for them)
      constexpr int kAhead = 4;
      float fp[2][kAhead], fq[2][kAhead];
      auto read = [&](int b, int j0) {
#pragma unroll
        for (int i = 0; i < kAhead; ++i) {
          fp[b][i] = s_p[j0 + 2 * i + (lane >> 5)][wp + (lane & 31)];
          fq[b][i] = s_q[j0 + 2 * i + (lane >> 5)][wq + (lane & 31)];
        }
      };
      read(0, 0);
#pragma unroll
      for (int j = 0; j < kStep; j += 2 * kAhead) {
        const int b = j / (2 * kAhead) & 1;
        if (j + 2 * kAhead < kStep) read(b ^ 1, j + 2 * kAhead);
        __builtin_amdgcn_sched_barrier(0);
#pragma unroll
        for (int i = 0; i < kAhead; ++i)
          acc = __builtin_amdgcn_mfma_f32_32x32x2f32(fp[b][i], fq[b][i], acc, 0, 0, 0);
        __builtin_amdgcn_sched_barrier(0);
      }
      if (sum_dy && tid < kTile) {
        float part = 0.0f;
#pragma unroll
        for (int j = 0; j < kStep; ++j) part += s_q[j][tid];
        db += part;
      }
    }
    float *to = args.part + L * kPart;
    if (sum_dy && tid < kTile && q0 + tid < nq) {
      if (split) to[kTile * kTile + tid] = db;
      else put_bias<O>(a, g, q0 + tid, db);
    }
    const int q = q0 + wq + (lane & 31);
    if (q >= nq) continue;
    const int64_t out_row = MODE == kLinWeightGrad ? static_cast<int64_t>(g) * a.n_out + q : row0 + q;
#pragma unroll
    for (int b = 0; b < 4; ++b) {
      const int p = p0 + wp + b * 8 + (lane >> 5) * 4;
      if (p >= np) continue;
      float v[4] = {acc[4 * b], acc[4 * b + 1], acc[4 * b + 2], acc[4 * b + 3]};
      if (split) put4(to + (q - q0) * kTile + p - p0, v);
      else put_sums<T, O, MODE>(a, g, out_row, p, v);
    }
  }
}

// Sums of the parts of split tiles, in order; four workgroups a tile, float4 a thread.
template <typename T, typename O, int MODE>
__global__ __launch_bounds__(256) void linear_f32_parts_kernel(Args args) {
  const Linear &a = args.l;
  __shared__ int s_pref[kMaxGroups + 1], s_tmp[4];
  const Items<MODE> items(args, s_pref, s_tmp);
  const int np = MODE == kLinForward ? a.n_out : a.k;
  int64_t rest = blockIdx.x / 4;
  const int ptile = remainder(rest, items.ptiles);
  int g, q0, parts = items.parts, nq;
  int64_t first, step, row0;             // item of the first part, and from part to part
  if (MODE == kLinWeightGrad) {
    const int tiles = items.qtiles * items.ptiles, qtile = remainder(rest, items.qtiles);
    g = static_cast<int>(rest);
    if (g >= a.groups) return;
    parts = s_pref[g + 1] - s_pref[g];
    first = static_cast<int64_t>(s_pref[g]) * tiles + qtile * items.ptiles + ptile;
    step = tiles;
    q0 = qtile * kTile;
    nq = a.n_out;
    row0 = static_cast<int64_t>(g) * a.n_out;
  } else {
    if (rest >= items.qtiles) return;
    g = group_of(s_pref, a.groups, rest);
    first = static_cast<int64_t>(blockIdx.x / 4) * parts;
    step = 1;
    q0 = static_cast<int>(rest - s_pref[g]) * kTile;
    row0 = a.offsets[g];
    nq = a.offsets[g + 1] - static_cast<int>(row0);
  }
  if (parts <= 1) return;
  const float *from = args.part + first * kPart;
  const int r = (blockIdx.x % 4) * (kTile / 4) + threadIdx.x / 16, c = threadIdx.x % 16 * 4, p = ptile * kTile + c;
  if (q0 + r < nq && p < np) {
    float v[4] = {0.0f, 0.0f, 0.0f, 0.0f};
#pragma unroll 8
    for (int i = 0; i < parts; ++i) {
      const float4 x = *reinterpret_cast<const float4 *>(from + i * step * kPart + r * kTile + c);
      v[0] += x.x, v[1] += x.y, v[2] += x.z, v[3] += x.w;
    }
    put_sums<T, O, MODE>(a, g, row0 + q0 + r, p, v);
  }
  const int q = q0 + threadIdx.x;
  if (MODE == kLinWeightGrad && a.dbias && ptile == 0 && blockIdx.x % 4 == 0 && threadIdx.x < kTile && q < nq) {
    float v = 0.0f;
    for (int i = 0; i < parts; ++i) v += from[i * step * kPart + kTile * kTile + threadIdx.x];
    put_bias<O>(a, g, q, v);
  }
}

// Tiles, at most.
int64_t tile_bound(int mode, int groups, int n_out, int k, int64_t max_rows) {
  const int64_t pt = ((mode == kLinForward ? n_out : k) + kTile - 1) / kTile;
  return pt * (mode == kLinWeightGrad ? static_cast<int64_t>(groups) * ((n_out + kTile - 1) / kTile)
                                      : max_rows / kTile + (max_rows < groups ? max_rows : groups));
}

// Terms of a part, so that few tiles become about kItems items; 0 where there are enough
// tiles, or where the sums are too short for two parts (weight gradients: where groups of
// four times the mean's rows are).
int chunk_of(int mode, int groups, int n_out, int k, int64_t max_rows) {
  const int64_t tiles = tile_bound(mode, groups, n_out, k, max_rows);
  if (tiles >= kFewTiles || tiles == 0) return 0;
  int64_t terms = mode == kLinForward ? k : n_out, all = terms * tiles;
  if (mode == kLinWeightGrad) {
    all = max_rows * (tiles / groups);
    terms = max_rows / groups * 4 < max_rows ? max_rows / groups * 4 + 4 : max_rows;
  }
  int64_t chunk = (all / kItems + kStep - 1) / kStep * kStep;
  if (chunk < kMinChunk) chunk = kMinChunk;
  return terms >= 2 * chunk && terms >= kMinTerms ? static_cast<int>(chunk) : 0;
}
// Items, at most.
int64_t item_bound(int mode, int groups, int n_out, int k, int64_t max_rows, int chunk) {
  const int64_t tiles = tile_bound(mode, groups, n_out, k, max_rows);
  if (!chunk) return tiles;
  if (mode == kLinWeightGrad) return tiles / groups * (max_rows / chunk + groups);
  return tiles * (((mode == kLinForward ? k : n_out) + chunk - 1) / chunk);
}

template <typename T, typename O, int MODE>
void launch(const Linear &p, void *ws, hipStream_t s) {
  const int chunk = ws ? chunk_of(MODE, p.groups, p.n_out, p.k, p.max_rows) : 0;
  const Args a{p, static_cast<float *>(ws), chunk};
  const int64_t most = 1 << 20, want = item_bound(MODE, p.groups, p.n_out, p.k, p.max_rows, chunk);
  hipLaunchKernelGGL((linear_f32_kernel<T, O, MODE>), dim3(static_cast<unsigned>(want < most ? want : most)),
                     dim3(256), 0, s, a);
  if (chunk)
    hipLaunchKernelGGL((linear_f32_parts_kernel<T, O, MODE>),
                       dim3(static_cast<unsigned>(4 * tile_bound(MODE, p.groups, p.n_out, p.k, p.max_rows))), dim3(256),
                       0, s, a);
}

}  // namespace

size_t linear_f32_workspace_bytes(int groups, int n_out, int k, int64_t max_rows) {
  int64_t most = 0;
  for (int mode : {kLinForward, kLinInputGrad, kLinWeightGrad}) {
    const int chunk = chunk_of(mode, groups, n_out, k, max_rows);
    const int64_t items = chunk ? item_bound(mode, groups, n_out, k, max_rows, chunk) : 0;
    if (items > most) most = items;
  }
  return static_cast<size_t>(most) * kPart * sizeof(float);
}

hipError_t launch_linear_f32(const Linear &p, void *ws, hipStream_t s) {
  if (!p.bf16) {
    if (p.mode == kLinForward) launch<float, float, kLinForward>(p, ws, s);
    else if (p.mode == kLinInputGrad) launch<float, float, kLinInputGrad>(p, ws, s);
    else launch<float, float, kLinWeightGrad>(p, ws, s);
  } else if (p.mode == kLinInputGrad) {
    launch<uint16_t, uint16_t, kLinInputGrad>(p, ws, s);
  } else if (p.out_bf16) {
    launch<uint16_t, uint16_t, kLinWeightGrad>(p, ws, s);
  } else {
    launch<uint16_t, float, kLinWeightGrad>(p, ws, s);
  }
  return hipGetLastError();
}

}  // namespace moe
