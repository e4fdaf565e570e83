// Products grouped by expert on the matrix cores, on the tiles of dense_tile.h: each expert's rows by
// its own weight, in one launch whatever the row counts are.
#include <cmath>

#include "dense_tile.h"
#include "grouped_kernels.h"

namespace moe {

// Rows of each of the tiles of at most bm rows that n rows take: as many for each where blocks of 16 rows without any
// are left out (tiles of 320), else bm.  Tile i's are i * height .. min(n, (i + 1) * height), never none.
__host__ __device__ __forceinline__ int tile_height(int n, int bm) {
  if (bm <= 256 || n <= bm) return bm;
  const int t = ceil_div(n, bm);
  return ceil_div(ceil_div(n, t), 16) * 16;
}

// The m-tiles of all experts in order: t[0].x of them, t[1 + i] = {first row, rows, expert}.
// A workgroup sums the tile counts in LDS, then every thread looks up the experts of its tiles.
constexpr int kTableThreads = 1024;
static_assert(kMaxE <= kTableThreads, "an expert per thread");
__global__ __launch_bounds__(kTableThreads) void k_group_tiles(Groups g, int bm, int cap, int4* t) {
  __shared__ int32_t starts[kMaxE + 1];
  __shared__ int32_t sums[kTableThreads / kWave];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  int n = 0;
  if (tid < g.E) {
    const int2 r = group_rows(g, tid);
    n = ceil_div(r.y - r.x, bm);
  }
  const int mine = wave_inclusive_scan(n, lane);
  if (lane == 63) sums[wave] = mine;
  __syncthreads();
  int before = 0;
  for (int w = 0; w < wave; ++w) before += sums[w];
  if (tid == 0) starts[0] = 0;
  if (tid < g.E) starts[tid + 1] = before + mine;
  __syncthreads();
  const int total = min(starts[g.E], cap);
  if (blockIdx.x == 0 && tid == 0) t[0] = make_int4(total, 0, 0, 0);
  for (int i = blockIdx.x * kTableThreads + tid; i < total; i += gridDim.x * kTableThreads) {
    const int e = min(upper_index(starts, g.E, i), g.E - 1);
    const int2 r = group_rows(g, e);
    const int h = tile_height(r.y - r.x, bm), first = r.x + (i - starts[e]) * h;
    t[1 + i] = make_int4(first, min(h, r.y - first), e, 0);
  }
}

// The same without a table: how many m-tiles there are, and where one of them is.  Each wave sums the tile counts of
// its lanes' experts.  It costs a workgroup about a microsecond, where the table's launch costs a call 4.6.
struct TileFinder {
  const Groups g;
  int bm, per, before, total;   // a lane's experts, tiles before them, of all
  __device__ __forceinline__ int tiles(int e) const {
    if (e >= g.E) return 0;
    const int2 r = group_rows(g, e);
    return ceil_div(r.y - r.x, bm);
  }
  __device__ __forceinline__ TileFinder(const Groups& groups, int rows) : g(groups), bm(rows) {
    const int lane = threadIdx.x & 63;
    per = ceil_div(g.E, 64);
    int mine = 0;
    for (int i = 0; i < per; ++i) mine += tiles(lane * per + i);
    const int upto = wave_inclusive_scan(mine, lane);
    before = upto - mine;
    total = __builtin_amdgcn_readlane(upto, 63);
  }
  // {first row, rows, expert} of m-tile t < total.
  __device__ __forceinline__ int4 at(int t) const {
    const int lane = threadIdx.x & 63;
    int4 found = make_int4(0, 0, 0, 0);
    bool here = false;
    for (int i = 0, b = before; i < per; ++i) {
      const int e = lane * per + i, n = tiles(e);
      if (t >= b && t < b + n) {
        const int2 r = group_rows(g, e);
        const int h = tile_height(r.y - r.x, bm), first = r.x + (t - b) * h;
        found = make_int4(first, min(h, r.y - first), e, 0);
        here = true;
      }
      b += n;
    }
    const int who = __builtin_ctzll(__ballot(here));
    return make_int4(__builtin_amdgcn_readlane(found.x, who), __builtin_amdgcn_readlane(found.y, who),
                     __builtin_amdgcn_readlane(found.z, who), 0);
  }
};

// Products on these tiles may be cut along the contraction.
template <typename T, int BM, int BN>
constexpr bool kCuts = BM == 64 && BN == 64 && sizeof(T) != 1;

// The tile of workgroup `block`: rows of one expert by columns of its weight.  table: the m-tiles, or NULL.
template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool B_COL, bool PAIR, int KIND,
          bool STREAM, int HEIGHT>
__device__ __forceinline__ void rows_tile(const DenseJob& j, const DenseEpi& e, const Groups& g, const int4* table,
                                          int64_t w_stride, const MmSlices& cut, int block, uint16_t* s0, uint16_t* s1,
                                          uint16_t* s2, uint16_t* s3) {
  const int tn = ceil_div(j.N, PAIR ? BN / 2 : BN);
  const MmSlices sl = kCuts<T, BM, BN> ? cut : MmSlices{nullptr, 1, 1, 0, 0};
  MmWhere w;
  int4 tile;
  if (table) {
    const int total = uniform(table[0].x);
    if (total == 0) return;
    w = mm_where(block, total, tn, 1, sl.slices);
    if (!w.ok) return;
    tile = table[1 + w.mt];
  } else {
    const TileFinder f(g, HEIGHT);
    if (f.total == 0) return;
    w = mm_where(block, f.total, tn, 1, sl.slices);
    if (!w.ok) return;
    tile = f.at(w.mt);
  }
  const int64_t row = uniform(tile.x), expert = uniform(tile.z);
  w.mt = 0;
  const MmPart at{uniform(tile.y), j.K, row * j.lda, expert * w_stride, row * e.ldo, row, expert * j.N};
  mm_body<T, O, BM, BN, WM, WN, S, SB, DB, false, B_COL, PAIR, KIND, true, STREAM, HEIGHT>(j, e, sl, w, at, s0, s1, s2, s3);
}

// Zeros in the bytes lo .. hi of p (2-byte aligned), in 16-byte chunks but for the ends.
__device__ __forceinline__ void zero_bytes(char* p, int64_t lo, int64_t hi) {
  const int64_t a = reinterpret_cast<int64_t>(p) + lo, b = reinterpret_cast<int64_t>(p) + hi;
  const int64_t a16 = min((a + 15) & ~15ll, b), b16 = max(b & ~15ll, a16), step = 16 * blockDim.x;
  for (int64_t i = a16 + 16 * threadIdx.x; i < b16; i += step) __builtin_nontemporal_store(u32x4{0, 0, 0, 0}, reinterpret_cast<u32x4*>(i));
  const int64_t edge = 2 * threadIdx.x;
  if (a + edge < a16) *reinterpret_cast<uint16_t*>(a + edge) = 0;
  if (b16 + edge < b) *reinterpret_cast<uint16_t*>(b16 + edge) = 0;
}

// The same of the weight gradients: columns of one expert's gradient by columns of its rows.  An expert without rows
// has its gradient's bytes filled with zeros, a share by each workgroup.
template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB>
__device__ __forceinline__ void dw_tile(const DenseJob& j, const DenseEpi& e, const Groups& g, int block, uint16_t* s0,
                                        uint16_t* s1, uint16_t* s2, uint16_t* s3) {
  MmWhere w = mm_where(block, ceil_div(j.M, BM), ceil_div(j.N, BN), g.E * j.batch, 1);
  if (!w.ok) return;
  const int expert = uniform(w.z / j.batch);
  w.z -= expert * j.batch;
  const int2 r = group_rows(g, expert);
  const int64_t row = uniform(r.x);
  if (uniform(r.y - r.x) == 0) {
    const int tiles = ceil_div(j.M, BM) * ceil_div(j.N, BN), tile = w.mt * ceil_div(j.N, BN) + w.nt;
    const int64_t bytes = (int64_t)j.M * e.ldo * (sizeof(T) == 4 || e.out_f32 ? 4 : 2);
    // shares end at even bytes
    return zero_bytes(static_cast<char*>(e.out[w.z]) + expert * bytes, bytes / 2 * tile / tiles * 2, bytes / 2 * (tile + 1) / tiles * 2);
  }
  const MmPart at{j.M, uniform(r.y - r.x), row * j.lda, row * j.ldb, (int64_t)expert * j.M * e.ldo, 0, 0};
  mm_body<T, T, BM, BN, WM, WN, S, SB, DB, true, true, false, DENSE_STORE, true>(j, e, MmSlices{nullptr, 1, 1, 0, 0}, w, at, s0, s1,
                                                                           s2, s3);
}

template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool B_COL, bool PAIR, int KIND,
          bool STREAM, int HEIGHT>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_grouped_mm(DenseJob j, DenseEpi e, Groups g,
                                                               const int4* __restrict__ table, int64_t w_stride, MmSlices sl) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  rows_tile<T, O, BM, BN, WM, WN, S, SB, DB, B_COL, PAIR, KIND, STREAM, HEIGHT>(j, e, g, table, w_stride, sl, blockIdx.x, s0, s1, s2, s3);
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_grouped_dw(DenseJob j, DenseEpi e, Groups g) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  dw_tile<T, BM, BN, WM, WN, S, SB, DB>(j, e, g, blockIdx.x, s0, s1, s2, s3);
}

// A backward pass's two products on 64 x 64 tiles in one launch: small ones leave the device half empty on their own.
// The first `first` workgroups are dx's (dx_first) or the weight gradients', whichever's contraction is longer.
template <typename T, int S, int DB>
__global__ __launch_bounds__(256, 2) void k_grouped_two(DenseJob jx, DenseEpi ex, int64_t w_stride, MmSlices sl, DenseJob jw,
                                                        DenseEpi ew, int first, bool dx_first, Groups g, const int4* __restrict__ table) {
  constexpr int STAGE = kMmStage<64, 64, 128>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  const bool early = (int)blockIdx.x < first;
  const int block = early ? blockIdx.x : blockIdx.x - first;
  if (early == dx_first)
    rows_tile<T, T, 64, 64, 2, 2, S, 128, DB, true, false, DENSE_STORE, false, 64>(jx, ex, g, table, w_stride, sl, block, s0, s1, s2, s3);
  else
    dw_tile<T, 64, 64, 2, 2, S, 128, DB>(jw, ew, g, block, s0, s1, s2, s3);
}

// The slices' sums in ascending order, then the epilogue, for the rows of all experts; eight columns per thread.
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_grouped_join(DenseEpi e, MmSlices sl, int N, Groups g) {
  const int first = min(max(g.offsets[0], 0), g.R), rows = min(g.offsets[g.E], g.R) - first, n8 = sl.ldp / 8;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)rows * n8; i += (int64_t)gridDim.x * 256) {
    const int m = first + (int)(i / n8), n = (int)(i % n8) * 8;
    float a[8] = {}, b[8] = {};
#pragma unroll 4
    for (int s = 0; s < sl.slices; ++s) {
      const f32x4* p = sl.at(s, 0, m, n, sl.rows);
      for (int k = 0; k < 8; ++k) a[k] += p[k >> 2][k & 3];
      if (KIND == DENSE_GATED) {
        p = sl.at(s, 1, m, n, sl.rows);
        for (int k = 0; k < 8; ++k) b[k] += p[k >> 2][k & 3];
      }
    }
    with_act<KIND>(e.act, [&](auto act) __attribute__((always_inline)) {
      mm_out8<T, KIND, act()>(e, 0, 0, m, n, N, a, b, Raw8<T>{}, Raw8<T>{});
    });
  }
}

// m-tiles of bm rows that R rows of E experts can take at most.
static int64_t most_tiles(int R, int E, int bm) { return R / bm + (R < E ? R : E); }

// Tile of a grouped product by estimated time, from what a kernel takes per round of `at_once` workgroups on the
// device: us per contraction step of 128 bytes and besides (a single round of up to 256 workgroups, one to a CU: `alone`),
// measured (MI355X).  The tallest tile, 320 x 256 in turns (256 for weight gradients, whose operands' columns are powers of
// two in LDS), reads each weight panel least often: 32768 rows of 128 experts, 768 -> 2048, take 149 us, where 256 x 256
// (half of the experts have a few rows more) takes 189 and 128 x 256 180; 62580 rows of 32, 7168 -> 2048 gated, 3315, 3432 and
// 4161.  Two workgroups of 128 x 256 on a CU overlap one's first loads and stores with the other's products, which is best
// for the shortest contractions (1024 rows of each of 32 experts, 256 -> 2048: 61 us, 64 on the tallest; 512 -> 2048: 89 and
// 90); 64 x 64 leave fewest CUs idle (64 rows of each of 8, 2048 -> 768 gated: 14 us, 35 on 128 x 256; the 149 us above: 272).
struct GroupedTile {
  int bm, bn, at_once;
  double step, fixed, step_alone, fixed_alone;
  int slices = 1;   // of the contraction
};
constexpr GroupedTile kTiles[] = {{320, 256, 256, 2.0, 11.5, 2.0, 11.5},
                                  {128, 256, 512, 2.2, 7.0, 1.3, 6.0},
                                  {64, 64, 512, 0.42, 3.0, 0.19, 2.5}};
constexpr GroupedTile kTileF32 = {64, 64, 512, 0.84, 2.0, 0.57, 2.5};
// Besides, there is no activation to meet and no tile to look up.
constexpr GroupedTile kTilesDw[] = {{256, 256, 256, 1.75, 5.6, 1.75, 11.5},
                                    {128, 256, 512, 2.2, 5.0, 1.3, 6.0},
                                    {64, 64, 512, 0.42, 3.0, 0.19, 2.5}};
// Rows so few that an expert's mostly fit one tile: each weight is read once, in whole lines, and past the caches (2048
// rows of 896 experts, 1024 -> 4096: 1191 us, 1299 on 64 x 64, which kept them; in integers 640, 763 and on 128 x 256 685).
// The row counts are on the device, so the rule goes by their average: where one expert has most of the rows, its tiles read
// its weights again each (8000 rows of one of 512 experts, 1024 -> 1024: 42 us, 25 as rows of one expert; in integers 36, 26).
constexpr GroupedTile kStreamTile = {64, 128, 512};
constexpr int kStreamRows = 16;   // an expert's, on average

static double rounds_us(const GroupedTile& c, double items, double steps) {
  if (items <= 256) return steps * c.step_alone + c.fixed_alone;
  const double rounds = items / c.at_once;
  return (rounds < 1 ? 1 : rounds + 0.5) * (steps * c.step + c.fixed);
}

// Tiles of bm rows that an expert with about `rows` takes, on average over row counts spread normally around it (by
// their square root and a twentieth): 1 + the chances of more than one tile's, two tiles' .. rows.  Of many tiles the last
// is half empty.
static double mean_tiles(double rows, int bm) {
  if (rows > 8.0 * bm) return rows / bm + 0.5;
  const double spread = sqrt(rows) + 0.05 * rows;
  double tiles = 1 + floor(fmax(0.0, rows - 4 * spread) / bm);
  for (double i = tiles; i * bm < rows + 4 * spread; ++i) tiles += 0.5 * erfc((i * bm - rows) / (spread * 1.4142135623730951));
  return tiles;
}

// R rows of E experts by their N columns, spread evenly as far as the host knows (200 rows of one of 64 experts, 4096 -> 1024,
// are not cut for it: 32 us, 13 as rows of one expert).  Products whose 64 x 64 tiles are too few for the device are cut along the
// contraction, at least 4 steps a slice; the slices' sums are written and read again, and joined by a launch of their
// own, at 4 us and 5 TB/s.  Whole and cut: 238 rows of 3 experts, 6960 -> 512, 34.1 and 14.8 us; 100 of 4, 2048 -> 768,
// 11.4 and 9.4; dx and dw of 2 fp32 rows of 3, 192 -> 3328, 64.5 and 13.9.  Integer products are left whole (256 rows of one
// expert, 7168 -> 2048: 23 us, of which the codes are 5).
static GroupedTile tile_of(GroupedType t, int R, int E, int N, int K, int segs, bool pair, bool b_col) {
  if (t != GROUPED_F32 && !b_col && R <= (int64_t)kStreamRows * E && (int64_t)(R < E ? R : E) * ceil_div(N, pair ? 64 : 128) >= 512) return kStreamTile;
  const double experts = R < E ? R : E, steps = ceil_div(K, t == GROUPED_INT8 ? 128 : t == GROUPED_BF16 ? 64 : 32) * segs;
  GroupedTile best{};
  double least = 0;
  auto consider = [&](GroupedTile c) {
    const double items = experts * mean_tiles(R / experts, c.bm) * ceil_div(N, pair ? c.bn / 2 : c.bn);
    const int most = c.bm == 64 && t != GROUPED_INT8 && items < 256 ? 32 : 1;
    for (int s = 1; s == 1 || (s <= most && 4 * s <= steps); s += s < 4 ? 1 : s / 2) {
      const double us = rounds_us(c, items * s, ceil(steps / s)) + (s > 1 ? 4.0 + (double)s * (pair ? 2 : 1) * R * N * 8 / 5e6 : 0.0);
      if (best.bm && us >= least) continue;
      least = us;
      best = c;
      best.slices = s;
    }
  };
  if (t == GROUPED_F32) consider(kTileF32);
  else for (const GroupedTile& c : kTiles) consider(c);
  return best;
}

static size_t table_bytes(const GroupedTile& c, int R, int E) { return (16 * (size_t)(1 + most_tiles(R, E, c.bm)) + 255) / 256 * 256; }
static int row_of_sums(int N) { return (N + 7) / 8 * 8; }

size_t grouped_scratch_bytes(GroupedType t, int R, int E, int N, int K, int segs, bool pair, bool b_col) {
  const GroupedTile c = tile_of(t, R, E, N, K, segs, pair, b_col);
  return table_bytes(c, R, E) + (c.slices > 1 ? (size_t)c.slices * (pair ? 2 : 1) * R * row_of_sums(N) * 4 : 0);
}

// Rows of the weights of experts that have rows, padded: eight elements of a row per thread; blockIdx.y the expert.
__global__ __launch_bounds__(256) void k_pad_weights(const uint16_t* w0, const uint16_t* w1, uint16_t* p0, uint16_t* p1, Groups g,
                                                     int64_t rows, int cols, int ld) {
  const int2 r = group_rows(g, blockIdx.y);
  if (r.x == r.y) return;
  const int per = ld / 8;
  const int64_t total = rows * per, in = blockIdx.y * rows * cols, out = blockIdx.y * rows * ld;
  for (int z = 0; z < (w1 ? 2 : 1); ++z) {
    const uint16_t* src = (z ? w1 : w0) + in;
    uint16_t* dst = (z ? p1 : p0) + out;
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
      const int64_t row = i / per;
      const int c = (int)(i - row * per) * 8;
      float v[8];
      load8(src + row * cols + c, cols - c, v);
      store8(dst + i * 8, v);
    }
  }
}

hipError_t launch_pad_weights(const void* w0, const void* w1, void* p0, void* p1, const Groups& g, int N, int cols, int64_t ld,
                              hipStream_t st) {
  const int64_t want = ((int64_t)N * (ld / 8) + 255) / 256, most = 65536 / g.E + 1;
  k_pad_weights<<<dim3((unsigned)(want < most ? want : most), g.E), 256, 0, st>>>(
      static_cast<const uint16_t*>(w0), static_cast<const uint16_t*>(w1), static_cast<uint16_t*>(p0), static_cast<uint16_t*>(p1), g, N,
      cols, (int)ld);
  return hipGetLastError();
}

static unsigned whole_eights(int64_t items) { return (unsigned)((items + 7) / 8 * 8); }

// The workgroups of a product by rows, and its m-tiles: in the table, unless so few workgroups would read it (two rounds
// of the device) that each had better look for itself (*table NULL then).
struct RowsGrid {
  GroupedTile c;
  unsigned blocks;
  MmSlices sl;
};
static hipError_t rows_grid(const DenseJob& j, GroupedType t, const Groups& g, RowsGrid* r, const int4** table, void* scratch,
                            hipStream_t st) {
  r->c = tile_of(t, g.R, g.E, j.N, j.K, j.segs, j.pair, j.b_col);
  const int64_t tiles = most_tiles(g.R, g.E, r->c.bm), items = tiles * ceil_div(j.N, j.pair ? r->c.bn / 2 : r->c.bn) * r->c.slices;
  r->blocks = whole_eights(items);
  r->sl = MmSlices{nullptr, r->c.slices, j.pair ? 2 : 1, row_of_sums(j.N), g.R};
  if (r->c.slices > 1) r->sl.part = reinterpret_cast<float*>(static_cast<char*>(scratch) + table_bytes(r->c, g.R, g.E));
  *table = nullptr;
  if (items <= 2 * r->c.at_once) return hipSuccess;
  *table = static_cast<int4*>(scratch);
  const int64_t blocks = (tiles + kTableThreads - 1) / kTableThreads;
  k_group_tiles<<<(unsigned)(blocks < 64 ? blocks : 64), kTableThreads, 0, st>>>(g, r->c.bm, (int)tiles, static_cast<int4*>(scratch));
  return hipGetLastError();
}

template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB = 128, int DB = 16, bool STREAM = false, int HEIGHT = BM>
static void go(const DenseJob& j, const DenseEpi& e, const Groups& g, const int4* t, const RowsGrid& r, int64_t w_stride, hipStream_t st) {
  const unsigned grid = r.blocks;
  const int block = WM * WN * 64;
  if (j.pair) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, true, DENSE_GATED, STREAM, HEIGHT><<<grid, block, 0, st>>>(j, e, g, t, w_stride, r.sl);
  else if constexpr (sizeof(T) == 1) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, false, DENSE_STORE, STREAM, HEIGHT><<<grid, block, 0, st>>>(j, e, g, t, w_stride, r.sl);
  else if (!STREAM && j.b_col) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, !STREAM, false, DENSE_STORE, STREAM, HEIGHT><<<grid, block, 0, st>>>(j, e, g, t, w_stride, r.sl);
  else k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, false, DENSE_STORE, STREAM, HEIGHT><<<grid, block, 0, st>>>(j, e, g, t, w_stride, r.sl);
}
template <typename T, typename O>
static void go_tile(const DenseJob& j, const DenseEpi& e, const Groups& g, const int4* t, const RowsGrid& r, int64_t w_stride,
                    hipStream_t st) {
  if (r.c.bm == 320) go<T, O, 384, 256, 2, 4, 4, 64, 16, false, 320>(j, e, g, t, r, w_stride, st);
  else if (r.c.bm == 128) go<T, O, 128, 256, 2, 2, 3, 64>(j, e, g, t, r, w_stride, st);
  else if (r.c.bn == kStreamTile.bn) go<T, O, 64, 128, 1, 4, 3, 128, 16, true>(j, e, g, t, r, w_stride, st);
  else go<T, O, 64, 64, 2, 2, 4>(j, e, g, t, r, w_stride, st);
}

static bool whole_chunks(const DenseJob& j) { return j.lda % 4 == 0 && j.ldb % 4 == 0; }

// The epilogue of a product's slices, if it was cut.
template <typename T>
static void join_kind(const DenseJob& j, const DenseEpi& e, const RowsGrid& r, const Groups& g, hipStream_t st) {
  const int64_t want = ((int64_t)g.R * (r.sl.ldp / 8) + 255) / 256;
  const unsigned grid = (unsigned)(want < 4096 ? want : 4096);
  if (j.pair) k_grouped_join<T, DENSE_GATED><<<grid, 256, 0, st>>>(e, r.sl, j.N, g);
  else k_grouped_join<T, DENSE_STORE><<<grid, 256, 0, st>>>(e, r.sl, j.N, g);
}
static hipError_t join(const DenseJob& j, const DenseEpi& e, GroupedType t, const RowsGrid& r, const Groups& g, hipStream_t st) {
  hipError_t s = hipGetLastError();
  if (s != hipSuccess || !r.sl.part) return s;
  if (t == GROUPED_F32) join_kind<float>(j, e, r, g, st);
  else join_kind<uint16_t>(j, e, r, g, st);
  return hipGetLastError();
}

hipError_t launch_grouped(const DenseJob& j, const DenseEpi& e, GroupedType t, bool out_bf16, const Groups& g,
                          int64_t w_stride, void* scratch, hipStream_t st) {
  RowsGrid r;
  const int4* tab;
  if (hipError_t s = rows_grid(j, t, g, &r, &tab, scratch, st); s != hipSuccess) return s;
  if (t == GROUPED_F32) {
    if (whole_chunks(j)) go<float, float, 64, 64, 2, 2, 3>(j, e, g, tab, r, w_stride, st);
    else go<float, float, 64, 64, 2, 2, 3, 128, 4>(j, e, g, tab, r, w_stride, st);
  } else if (t == GROUPED_BF16) {
    go_tile<uint16_t, uint16_t>(j, e, g, tab, r, w_stride, st);
  } else if (out_bf16) {
    go_tile<int8_t, uint16_t>(j, e, g, tab, r, w_stride, st);
  } else {
    go_tile<int8_t, float>(j, e, g, tab, r, w_stride, st);
  }
  return join(j, e, t, r, g, st);
}

// Tile of the weight gradients: as many rows for every expert (32768 rows of 128, 2048 -> 768 gated: 331 us on 256 x 256, 365
// on 128 x 256).  Their contraction is not cut: few experts with small weights and many rows have too few tiles for the device,
// each of which walks all rows of its expert (fp32, 32768 rows of one, 64 -> 64: one tile, 629 us; 14922 of 2, 2317 -> 64: 191;
// bf16, 20000 of one, 256 -> 192: 92; 8000 of one of 64, 512 -> 512: 136).
static const GroupedTile& dw_tile_of(const DenseJob& j, GroupedType t, const Groups& g) {
  if (t == GROUPED_F32) return kTilesDw[2];
  const double steps = (g.R / (double)g.E / 64 + 0.5) * j.segs;
  const GroupedTile* best = nullptr;
  double least = 0;
  for (const GroupedTile& c : kTilesDw) {
    const double us = rounds_us(c, (double)g.E * j.batch * ceil_div(j.M, c.bm) * ceil_div(j.N, c.bn), steps);
    if (!best || us < least) best = &c, least = us;
  }
  return *best;
}
static unsigned dw_blocks(const DenseJob& j, const GroupedTile& c, const Groups& g) {
  return whole_eights((int64_t)ceil_div(j.M, c.bm) * ceil_div(j.N, c.bn) * g.E * j.batch);
}

static hipError_t launch_dw(const DenseJob& j, const DenseEpi& e, GroupedType t, const Groups& g, const GroupedTile& c, hipStream_t st) {
  const unsigned grid = dw_blocks(j, c, g);
  if (t == GROUPED_F32) {
    if (whole_chunks(j)) k_grouped_dw<float, 64, 64, 2, 2, 3, 128, 16><<<grid, 256, 0, st>>>(j, e, g);
    else k_grouped_dw<float, 64, 64, 2, 2, 3, 128, 4><<<grid, 256, 0, st>>>(j, e, g);
  } else if (c.bm == 256) {
    k_grouped_dw<uint16_t, 256, 256, 2, 4, 4, 64, 16><<<grid, 512, 0, st>>>(j, e, g);
  } else if (c.bm == 128) {
    k_grouped_dw<uint16_t, 128, 256, 2, 2, 3, 64, 16><<<grid, 256, 0, st>>>(j, e, g);
  } else {
    k_grouped_dw<uint16_t, 64, 64, 2, 2, 4, 128, 16><<<grid, 256, 0, st>>>(j, e, g);
  }
  return hipGetLastError();
}

hipError_t launch_grouped_grads(const GroupedProduct* dx, const GroupedProduct* dw, GroupedType t, const Groups& g,
                                int64_t w_stride, void* scratch, hipStream_t st) {
  if (!dw) return launch_grouped(dx->j, dx->e, t, t == GROUPED_BF16, g, w_stride, scratch, st);
  const GroupedTile& c = dw_tile_of(dw->j, t, g);
  if (!dx || c.bm != 64 || tile_of(t, g.R, g.E, dx->j.N, dx->j.K, dx->j.segs, false, true).bm != 64) {
    if (hipError_t r = launch_dw(dw->j, dw->e, t, g, c, st); r != hipSuccess || !dx) return r;
    return launch_grouped(dx->j, dx->e, t, t == GROUPED_BF16, g, w_stride, scratch, st);
  }
  RowsGrid r;
  const int4* tab;
  if (hipError_t s = rows_grid(dx->j, t, g, &r, &tab, scratch, st); s != hipSuccess) return s;
  const bool dx_first = (int64_t)dx->j.K * dx->j.segs / r.c.slices >= (int64_t)g.R / g.E * dw->j.segs;
  const unsigned blocks = dw_blocks(dw->j, c, g), first = dx_first ? r.blocks : blocks, all = r.blocks + blocks;
  auto go = [&](auto kernel) { kernel<<<all, 256, 0, st>>>(dx->j, dx->e, w_stride, r.sl, dw->j, dw->e, (int)first, dx_first, g, tab); };
  if (t == GROUPED_BF16) go(k_grouped_two<uint16_t, 4, 16>);
  else if (whole_chunks(dx->j) && whole_chunks(dw->j)) go(k_grouped_two<float, 3, 16>);
  else go(k_grouped_two<float, 3, 4>);
  return join(dx->j, dx->e, t, r, g, st);
}

}  // namespace moe
