// Products grouped by expert on the matrix cores, on the tiles of dense_tile.h: each expert's rows by
// its own weight, in one launch whatever the row counts are.
#include "dense_tile.h"
#include "grouped_kernels.h"

namespace moe {

// The m-tiles of all experts in order: t[0].x of them, t[1 + i] = {first row, rows of the expert from there on, expert}.
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
    const int first = r.x + (i - starts[e]) * bm;
    t[1 + i] = make_int4(first, r.y - first, e, 0);
  }
}

template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool B_COL, bool PAIR, int KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_grouped_mm(DenseJob j, DenseEpi e, const int4* __restrict__ table,
                                                               int64_t w_stride) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  const int total = uniform(table[0].x);
  if (total == 0) return;
  MmWhere w = mm_where(blockIdx.x, total, ceil_div(j.N, PAIR ? BN / 2 : BN), 1, 1);
  if (!w.ok) return;
  const int4 tile = table[1 + w.mt];
  const int64_t row = uniform(tile.x), expert = uniform(tile.z);
  w.mt = 0;
  const MmPart at{uniform(tile.y), j.K, row * j.lda, expert * w_stride, row * e.ldo, row, expert * j.N};
  mm_body<T, O, BM, BN, WM, WN, S, SB, DB, false, B_COL, PAIR, KIND, true>(j, e, MmSlices{nullptr, 1, 1, 0}, w, at, s0, s1,
                                                                           s2, s3);
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_grouped_dw(DenseJob j, DenseEpi e, Groups g) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  MmWhere w = mm_where(blockIdx.x, ceil_div(j.M, BM), ceil_div(j.N, BN), g.E * j.batch, 1);
  if (!w.ok) return;
  const int expert = uniform(w.z / j.batch);
  w.z -= expert * j.batch;
  const int2 r = group_rows(g, expert);
  const int64_t row = uniform(r.x);
  const MmPart at{j.M, uniform(r.y - r.x), row * j.lda, row * j.ldb, (int64_t)expert * j.M * e.ldo, 0, 0};
  mm_body<T, T, BM, BN, WM, WN, S, SB, DB, true, true, false, DENSE_STORE>(j, e, MmSlices{nullptr, 1, 1, 0}, w, at, s0, s1,
                                                                           s2, s3);
}

// m-tiles of bm rows that R rows of E experts can take at most.
static int64_t most_tiles(int R, int E, int bm) { return R / bm + (R < E ? R : E); }

// Tile of a grouped product by estimated time, from what a kernel takes per round of `at_once` workgroups on the
// device: us per contraction step of 128 bytes and besides (a single round of up to 256 workgroups, one to a CU: `alone`),
// measured (MI355X).  256 x 256 tiles in turns have the fewest bytes through a CU's L1 and are best for long
// contractions (62580 rows of 32 experts, 7168 -> 2048 gated: 3414 us, 4167 on 128 x 256); two workgroups of
// 128 x 256 on a CU overlap one's first loads and stores with the other's products, which is best for short
// ones (32768 rows of 128 experts, 768 -> 2048: 182 us, 193 on 256 x 256, 272 on 64 x 64); 64 x 64 waste least on a few rows of
// many experts (2048 rows of 896, 1024 -> 4096: 1084 us; 1130 and 1255).
struct GroupedTile {
  int bm, bn, at_once;
  double step, fixed, step_alone, fixed_alone;
};
constexpr GroupedTile kTiles[] = {{256, 256, 256, 1.75, 11.5, 1.75, 11.5},
                                  {128, 256, 512, 2.2, 7.0, 1.3, 6.0},
                                  {64, 64, 512, 0.42, 3.0, 0.19, 2.5}};

static double rounds_us(const GroupedTile& c, double items, double steps) {
  if (items <= 256) return steps * c.step_alone + c.fixed_alone;
  const double rounds = items / c.at_once;
  return (rounds < 1 ? 1 : rounds + 0.5) * (steps * c.step + c.fixed);
}

// R rows of E experts by their N columns: half a tile's rows are empty in an expert's last one, on average.
static GroupedTile tile_of(GroupedType t, int R, int E, int N, int K, int segs, bool pair) {
  if (t == GROUPED_F32) return kTiles[2];
  const double experts = R < E ? R : E, steps = ceil_div(K, t == GROUPED_INT8 ? 128 : 64) * segs;
  const GroupedTile* best = nullptr;
  double least = 0;
  for (const GroupedTile& c : kTiles) {
    double m = R / (double)c.bm + 0.5 * experts;
    if (m < experts) m = experts;
    const double us = rounds_us(c, m * ceil_div(N, pair ? c.bn / 2 : c.bn), steps);
    if (!best || us < least) best = &c, least = us;
  }
  return *best;
}

size_t grouped_table_bytes(GroupedType t, int R, int E, int N, int K, int segs, bool pair) {
  return 16 * (size_t)(1 + most_tiles(R, E, tile_of(t, R, E, N, K, segs, pair).bm));
}

template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB = 128, int DB = 16>
static void go(const DenseJob& j, const DenseEpi& e, const int4* t, int64_t tiles, int64_t w_stride, hipStream_t st) {
  const int64_t items = tiles * ceil_div(j.N, j.pair ? BN / 2 : BN);
  const dim3 grid((unsigned)((items + 7) / 8 * 8)), block(WM * WN * 64);
  if (j.pair) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, true, DENSE_GATED><<<grid, block, 0, st>>>(j, e, t, w_stride);
  else if constexpr (sizeof(T) == 1) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e, t, w_stride);
  else if (j.b_col) k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, true, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e, t, w_stride);
  else k_grouped_mm<T, O, BM, BN, WM, WN, S, SB, DB, false, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e, t, w_stride);
}

template <typename T, typename O>
static void go_tile(const GroupedTile& c, const DenseJob& j, const DenseEpi& e, const int4* t, int64_t tiles,
                    int64_t w_stride, hipStream_t st) {
  if (c.bm == 256) go<T, O, 256, 256, 2, 4, 4, 64>(j, e, t, tiles, w_stride, st);
  else if (c.bm == 128) go<T, O, 128, 256, 2, 2, 3, 64>(j, e, t, tiles, w_stride, st);
  else go<T, O, 64, 64, 2, 2, 4>(j, e, t, tiles, w_stride, st);
}

static bool whole_chunks(const DenseJob& j) { return j.lda % 4 == 0 && j.ldb % 4 == 0; }

hipError_t launch_grouped(const DenseJob& j, const DenseEpi& e, GroupedType t, bool out_bf16, const Groups& g,
                          int64_t w_stride, void* table, hipStream_t st) {
  const GroupedTile c = tile_of(t, g.R, g.E, j.N, j.K, j.segs, j.pair);
  const int bm = c.bm;
  const int64_t tiles = most_tiles(g.R, g.E, bm);
  int4* tab = static_cast<int4*>(table);
  const int64_t blocks = (tiles + kTableThreads - 1) / kTableThreads;
  k_group_tiles<<<(unsigned)(blocks < 64 ? blocks : 64), kTableThreads, 0, st>>>(g, bm, (int)tiles, tab);
  if (hipError_t r = hipGetLastError(); r != hipSuccess) return r;
  if (t == GROUPED_F32) {
    if (whole_chunks(j)) go<float, float, 64, 64, 2, 2, 3>(j, e, tab, tiles, w_stride, st);
    else go<float, float, 64, 64, 2, 2, 3, 128, 4>(j, e, tab, tiles, w_stride, st);
  } else if (t == GROUPED_BF16) {
    go_tile<uint16_t, uint16_t>(c, j, e, tab, tiles, w_stride, st);
  } else if (out_bf16) {
    go_tile<int8_t, uint16_t>(c, j, e, tab, tiles, w_stride, st);
  } else {
    go_tile<int8_t, float>(c, j, e, tab, tiles, w_stride, st);
  }
  return hipGetLastError();
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB = 128, int DB = 16>
static void go_dw(const DenseJob& j, const DenseEpi& e, const Groups& g, hipStream_t st) {
  const int64_t items = (int64_t)ceil_div(j.M, BM) * ceil_div(j.N, BN) * g.E * j.batch;
  k_grouped_dw<T, BM, BN, WM, WN, S, SB, DB><<<(unsigned)((items + 7) / 8 * 8), WM * WN * 64, 0, st>>>(j, e, g);
}

hipError_t launch_grouped_dw(const DenseJob& j, const DenseEpi& e, GroupedType t, const Groups& g, hipStream_t st) {
  if (t == GROUPED_BF16) {
    // as many rows for every expert; the epilogue only stores
    const double steps = (g.R / (double)g.E / 64 + 0.5) * j.segs;
    int best = 0;
    double least = 0;
    for (int i = 0; i < 3; ++i) {
      const GroupedTile& c = kTiles[i];
      const double us = rounds_us(c, (double)g.E * j.batch * ceil_div(j.M, c.bm) * ceil_div(j.N, c.bn), steps);
      if (i == 0 || us < least) best = i, least = us;
    }
    if (best == 0) go_dw<uint16_t, 256, 256, 2, 4, 4, 64>(j, e, g, st);
    else if (best == 1) go_dw<uint16_t, 128, 256, 2, 2, 3, 64>(j, e, g, st);
    else go_dw<uint16_t, 64, 64, 2, 2, 4>(j, e, g, st);
  }
  else if (whole_chunks(j)) go_dw<float, 64, 64, 2, 2, 3>(j, e, g, st);
  else go_dw<float, 64, 64, 2, 2, 3, 128, 4>(j, e, g, st);
  return hipGetLastError();
}

}  // namespace moe
