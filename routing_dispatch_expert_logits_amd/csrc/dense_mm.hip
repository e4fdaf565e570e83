// Dense products on the matrix cores, fp32 accumulate, on the tiles of dense_tile.h.
#include "dense_tile.h"

namespace moe {

// The tile of workgroup `block` of one product.
template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool A_COL, bool B_COL, bool PAIR, int KIND>
__device__ __forceinline__ void dense_tile(const DenseJob& j, const DenseEpi& e, const MmSlices& sl, int block, uint16_t* s0,
                                           uint16_t* s1, uint16_t* s2, uint16_t* s3) {
  const MmWhere w = mm_where(block, ceil_div(j.M, BM), ceil_div(j.N, PAIR ? BN / 2 : BN), j.batch, sl.slices);
  mm_body<T, T, BM, BN, WM, WN, S, SB, DB, A_COL, B_COL, PAIR, KIND>(j, e, sl, w, MmPart{j.M, j.K, 0, 0, 0, 0, 0}, s0, s1,
                                                                     s2, s3);
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool A_COL, bool B_COL, bool PAIR,
          int KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_dense_mm(DenseJob j, DenseEpi e, MmSlices sl) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  dense_tile<T, BM, BN, WM, WN, S, SB, DB, A_COL, B_COL, PAIR, KIND>(j, e, sl, blockIdx.x, s0, s1, s2, s3);
}

// A small backward pass's two products, dx on the first `first` workgroups and dw on the others:
// neither fills the device, and a launch of its own costs each about 5 us.
template <typename T, int BN, int WM, int WN, int S, int DB>
__global__ __launch_bounds__(256, 2) void k_dense_mm_two(DenseJob jx, DenseEpi ex, MmSlices sx, int first, DenseJob jw,
                                                         DenseEpi ew, MmSlices sw) {
  constexpr int STAGE = kMmStage<64, BN, 128>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  if ((int)blockIdx.x < first)
    dense_tile<T, 64, BN, WM, WN, S, 128, DB, false, true, false, DENSE_STORE>(jx, ex, sx, blockIdx.x, s0, s1, s2, s3);
  else
    dense_tile<T, 64, BN, WM, WN, S, 128, DB, true, true, false, DENSE_STORE>(jw, ew, sw, blockIdx.x - first, s0, s1, s2, s3);
}

// A product's slices' sums in ascending order, then the epilogue; eight columns per thread of
// workgroup `block` of `blocks`.
struct MmJoin {
  int M, N, batch, blocks;
  DenseEpi e;
  MmSlices sl;
};
template <typename T, int KIND>
__device__ __forceinline__ void join(const MmJoin& j, int block) {
  const int n8 = j.sl.ldp / 8;
  const int64_t total = (int64_t)j.batch * j.M * n8;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < total; i += (int64_t)j.blocks * 256) {
    const int64_t row = i / n8;
    const int n = (int)(i - row * n8) * 8, z = (int)(row / j.M), m = (int)(row - (int64_t)z * j.M);
    float a[8] = {}, b[8] = {};
#pragma unroll 4
    for (int s = 0; s < j.sl.slices; ++s) {
      const f32x4* p = j.sl.at(s, z, m, n, j.M);
      for (int k = 0; k < 8; ++k) a[k] += p[k >> 2][k & 3];
      if (KIND == DENSE_GATED) {
        p = j.sl.at(s, 1, m, n, j.M);
        for (int k = 0; k < 8; ++k) b[k] += p[k >> 2][k & 3];
      }
    }
    Raw8<T> res, bias;
    load_bias<T, KIND>(j.e, n, j.N, &bias);
    load_residual<T, KIND>(j.e, m, n, j.M, j.N, &res);
    with_act<KIND>(j.e.act, [&](auto act) __attribute__((always_inline)) { mm_out8<T, KIND, act()>(j.e, z, 0, m, n, j.N, a, b, bias, res); });
  }
}
template <typename T, int KIND>
__global__ __launch_bounds__(256) void k_dense_join(MmJoin j) { join<T, KIND>(j, blockIdx.x); }

// What a backward pass has left to join, in one launch: the slices of dx, of dw, and column
// sums.  A launch of its own costs each about 4 us, as much as most of them take.
template <typename T>
__global__ __launch_bounds__(256) void k_dense_tail(MmJoin x, MmJoin w, ColSum sum) {
  __shared__ float s[16][16];
  const int block = blockIdx.x;
  if (block < x.blocks) join<T, DENSE_STORE>(x, block);
  else if (block < x.blocks + w.blocks) join<T, DENSE_STORE>(w, block - x.blocks);
  else col_sum(sum, block - x.blocks - w.blocks, 0, s);
}

// Workgroups of a product: its tiles' slices, a whole number for each of the 8 XCDs.
static unsigned mm_grid(const DenseJob& j, const MmSlices& sl, int bm, int bn) {
  const int64_t items = (int64_t)ceil_div(j.M, bm) * ceil_div(j.N, j.pair ? bn / 2 : bn) * j.batch * sl.slices;
  return (unsigned)((items + 7) / 8 * 8);
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB = 128, int DB = 16>
static void mm_go(const DenseJob& j, const DenseEpi& e, const MmSlices& sl, hipStream_t st) {
  const dim3 grid(mm_grid(j, sl, BM, BN)), block(WM * WN * 64);
  if (j.pair) k_dense_mm<T, BM, BN, WM, WN, S, SB, DB, false, false, true, DENSE_GATED><<<grid, block, 0, st>>>(j, e, sl);
  else if (e.kind == DENSE_LINEAR) k_dense_mm<T, BM, BN, WM, WN, S, SB, DB, false, false, false, DENSE_LINEAR><<<grid, block, 0, st>>>(j, e, sl);
  else if (!j.a_col) k_dense_mm<T, BM, BN, WM, WN, S, SB, DB, false, true, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e, sl);
  else if constexpr ((BM & (BM - 1)) == 0) k_dense_mm<T, BM, BN, WM, WN, S, SB, DB, true, true, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e, sl);
}

// Tile and slice count of one product, by estimated time.  A tile's constants are what its
// kernel takes per contraction step and per workgroup beside the steps, on a CU that works
// through several or has just one, measured with operands that
// come from memory (MI355X).  bf16: 4096^3 takes 104 us on 256 x 256 tiles, 116 on 256 x 128,
// 133 on 128 x 128 and 193 on 64 x 64; 2048^3, an eighth of the work with a quarter of the
// tiles, 54, 27, 21 and 27; 512 x 2048 x 2048 52, 26, 16 and 10.  fp32 is bound by its matrix
// instructions on 64 x 64 tiles already (4096^3: 967 us, 142 TFLOP/s; 128 x 128 the same).
struct MmTileCost {
  int bm, bn;
  double step, fixed;              // us, several workgroups after or beside each other
  double step_alone, fixed_alone;  // us, one
};
constexpr MmTileCost kTilesBf16[] = {{256, 256, 1.50, 8.0, 1.50, 8.0},
                                     {256, 128, 0.88, 4.5, 0.80, 4.5},
                                     {192, 128, 0.68, 4.0, 0.62, 4.0},  // not for column A operands
                                     {128, 128, 0.50, 3.0, 0.47, 3.0},
                                     {64, 64, 0.165, 1.3, 0.19, 2.5}};
constexpr MmTileCost kTilesF32[] = {{64, 64, 0.42, 1.0, 0.57, 2.5}, {64, 32, 0.22, 0.8, 0.35, 2.5}};
struct MmPlan {
  MmTileCost tile;
  int slices, planes, ldp;
  double us;
  double items, each, join;  // workgroups with work, the time of one among others, and the slices' join
  int cut;   // 256 x 256 tiles for this many output columns, and a launch of its own for the rest; 0: none
};
// whole: no slices; only: tiles of 64 rows and this many columns.
static MmPlan mm_plan(bool bf16, int M, int N, int K, int segs, int batch, bool pair, bool a_col, bool whole = false,
                      int only = 0) {
  constexpr int CUS = 256;
  MmPlan best{{}, 1, pair ? 2 : batch, (N + 7) / 8 * 8, 0.0, 0.0, 0.0, 0.0, 0};
  const int steps = ceil_div(K, bf16 ? 64 : 32) * segs;  // of 128 bytes
  for (int t = 0; t < (bf16 ? 5 : 2); ++t) {
    const MmTileCost& c = bf16 ? kTilesBf16[t] : kTilesF32[t];
    if ((only && (c.bm != 64 || c.bn != only)) || (c.bm == 192 && a_col)) continue;
    const int64_t tiles = (int64_t)ceil_div(M, c.bm) * ceil_div(N, pair ? c.bn / 2 : c.bn) * batch;
    for (int s = 1; s <= (whole ? 1 : 32) && s <= ceil_div(steps, 4); s += s < 4 ? 1 : s / 2) {
      const int64_t rounds = (tiles * s + CUS - 1) / CUS;
      double us = rounds == 1 ? ceil_div(steps, s) * c.step_alone + c.fixed_alone
                              : rounds * (ceil_div(steps, s) * c.step + c.fixed);
      // the slices' sums are written and read again, and joined by a launch of their own
      const double join = s > 1 ? 4.0 + (double)s * best.planes * M * N * 8 / 5e6 : 0.0;
      us += join;
      if (!best.tile.bm || us < best.us) {
        best.us = us;
        best.tile = c;
        best.slices = s;
        best.items = (double)tiles * s;
        best.each = ceil_div(steps, s) * c.step + c.fixed;
        best.join = join;
      }
    }
  }
  // Whole rounds of 256 x 256 tiles and smaller ones for the columns that would start another:
  // 8192 x 2048 x 7168 has 896 such tiles, three and a half rounds of 256.
  const MmTileCost& c = kTilesBf16[0];
  const int on = pair ? c.bn / 2 : c.bn, tn = ceil_div(N, on);
  const int64_t column = (int64_t)ceil_div(M, c.bm) * batch;  // tiles of one tile column
  if (bf16 && !whole && !only && column * tn > CUS) {
    const int64_t rounds = column * tn / CUS, n = rounds * CUS / column;
    if (n >= 1 && n < tn) {
      const MmPlan rest = mm_plan(bf16, M, N - (int)n * on, K, segs, batch, pair, a_col, true);
      const double us = rounds * (steps * c.step + c.fixed) + 3.0 + rest.us;
      if (us < best.us) {
        best.us = us;
        best.tile = c;
        best.slices = 1;
        best.cut = (int)n * on;
      }
    }
  }
  return best;
}

static size_t part_bytes(const MmPlan& p, int M) {
  return p.slices > 1 ? (size_t)p.slices * p.planes * M * p.ldp * 4 : 0;
}
// A backward pass's product may run on its own or together with the other one, on tiles of 64
// rows and 64 columns (fp32: or 32), with slices of their own.  fp32, dx and dw, 64 columns
// against 32: 128 x 1024 x 4096 31.8 and 37.6 us, 300 x 2000 x 1000 28.7 and 38.9; 32 are better
// where few tiles of 64 would leave the CUs uneven (1000 x 1032 x 2056: 91 and 80).  Whole rounds of
// tiles are not in this estimate, and where they decide it can miss: 3000 x 1000 x 1000 takes 125 us,
// and 116 where each product keeps the width and slices that it would choose on its own.
constexpr int kTogether[] = {64, 32};
size_t dense_part_bytes(bool bf16, int M, int N, int K, int segs, int batch, bool pair, bool a_col, bool backward) {
  size_t most = part_bytes(mm_plan(bf16, M, N, K, segs, batch, pair, a_col), M);
  for (int t = 0; backward && t < (bf16 ? 1 : 2); ++t) {
    const size_t both = part_bytes(mm_plan(bf16, M, N, K, segs, batch, pair, a_col, false, kTogether[t]), M);
    most = most > both ? most : both;
  }
  return most;
}

static MmPlan plan_of(const DenseJob& j, bool bf16) { return mm_plan(bf16, j.M, j.N, j.K, j.segs, j.batch, j.pair, j.a_col); }
static MmSlices slices_of(const MmPlan& p, float* part) {
  return MmSlices{p.slices > 1 ? part : nullptr, p.slices, p.planes, p.ldp};
}

// fp32 operands whose rows are whole 16-byte chunks.
static bool whole_chunks(const DenseJob& j) { return j.lda % 4 == 0 && j.ldb % 4 == 0; }

static MmJoin join_of(const DenseJob& j, const DenseEpi& e, const MmPlan& p, float* part) {
  MmJoin w{j.M, j.N, j.batch, 0, e, slices_of(p, part)};
  const int64_t want = ((int64_t)j.batch * j.M * (p.ldp / 8) + 255) / 256;
  if (p.slices > 1) w.blocks = (int)(want < 4096 ? want : 4096);
  return w;
}

// One launch; its slices are still to be joined.
static hipError_t launch_planned(const DenseJob& j, const DenseEpi& e, const MmPlan& p, bool bf16, float* part,
                                 hipStream_t st) {
  const MmSlices sl = slices_of(p, part);
  const int bm = p.tile.bm, bn = p.tile.bn;
  if (!bf16) {
    if (bn == 64 && whole_chunks(j)) mm_go<float, 64, 64, 2, 2, 3>(j, e, sl, st);
    else if (bn == 64) mm_go<float, 64, 64, 2, 2, 3, 128, 4>(j, e, sl, st);
    else if (whole_chunks(j)) mm_go<float, 64, 32, 4, 1, 3>(j, e, sl, st);
    else mm_go<float, 64, 32, 4, 1, 3, 128, 4>(j, e, sl, st);
  } else if (bn == 256) {
    mm_go<uint16_t, 256, 256, 2, 4, 4, 64>(j, e, sl, st);
  } else if (bm == 256) {
    mm_go<uint16_t, 256, 128, 4, 2, 3>(j, e, sl, st);
  } else if (bm == 192) {
    mm_go<uint16_t, 192, 128, 4, 2, 3>(j, e, sl, st);
  } else if (bm == 128) {
    mm_go<uint16_t, 128, 128, 2, 4, 4>(j, e, sl, st);
  } else {
    mm_go<uint16_t, 64, 64, 2, 2, 4>(j, e, sl, st);
  }
  return hipGetLastError();
}

// A product cut at output column p.cut: the columns left of it in `left` (with e), the others in
// `right` with `er`.
static void cut_product(const DenseJob& j, const DenseEpi& e, const MmPlan& p, bool bf16, DenseJob& left,
                        DenseJob& right, DenseEpi& er) {
  left = right = j;
  er = e;
  const int es = bf16 ? 2 : 4, oes = e.kind == DENSE_STORE && e.out_f32 ? 4 : es;
  left.N = p.cut;
  right.N = j.N - p.cut;
  if (j.b_col) right.b_from = j.b_from + p.cut;
  for (auto& z : right.B)
    for (auto& b : z)
      if (b) b = static_cast<const char*>(b) + (j.b_col ? (int64_t)p.cut : p.cut * j.ldb) * es;
  auto on = [&](auto* v, int size) {
    return v ? static_cast<decltype(v)>(const_cast<char*>(static_cast<const char*>(v) + (int64_t)p.cut * size)) : v;
  };
  er.bias = on(e.bias, es);
  er.residual = on(e.residual, es);
  for (int i = 0; i < 2; ++i) {
    er.out[i] = on(e.out[i], oes);
    er.save[i] = on(e.save[i], es);
  }
}

static MmPlan plan_of_rest(const DenseJob& right, bool bf16) {
  return mm_plan(bf16, right.M, right.N, right.K, right.segs, right.batch, right.pair, right.a_col, true);
}

// The product by its plan, in one or two launches; its slices are still to be joined.
static hipError_t launch_sliced(const DenseJob& j, const DenseEpi& e, const MmPlan& p, bool bf16, float* part,
                                hipStream_t st) {
  if (!p.cut) return launch_planned(j, e, p, bf16, part, st);
  DenseJob left, right;
  DenseEpi er;
  cut_product(j, e, p, bf16, left, right, er);
  if (hipError_t r = launch_planned(left, e, p, bf16, nullptr, st); r != hipSuccess) return r;
  return launch_planned(right, er, plan_of_rest(right, bf16), bf16, nullptr, st);
}

// The forward products; the epilogue where the slices meet.
hipError_t launch_dense(const DenseJob& j, const DenseEpi& e, bool bf16, float* part, hipStream_t st) {
  const MmPlan p = plan_of(j, bf16);
  if (hipError_t r = launch_sliced(j, e, p, bf16, part, st); r != hipSuccess || p.slices == 1) return r;
  const MmJoin w = join_of(j, e, p, part);
  auto go = [&](auto kernel) { kernel<<<w.blocks, 256, 0, st>>>(w); };
  if (j.pair && bf16) go(k_dense_join<uint16_t, DENSE_GATED>);
  else if (j.pair) go(k_dense_join<float, DENSE_GATED>);
  else if (bf16) go(k_dense_join<uint16_t, DENSE_LINEAR>);
  else go(k_dense_join<float, DENSE_LINEAR>);
  return hipGetLastError();
}

hipError_t launch_dense_grads(const DenseProduct* dx, const DenseProduct* dw, const ColSum& sum, bool bf16,
                              hipStream_t st) {
  MmPlan px{}, pw{};
  if (dx) px = plan_of(dx->j, bf16);
  if (dw) pw = plan_of(dw->j, bf16);
  bool together = false;
  if (dx && dw) {
    // on 64-row tiles where that is less than each on its best: they overlap, and a launch is saved
    MmPlan sx{}, sw{};
    double best = 0.0;
    for (int t = 0; t < (bf16 ? 1 : 2); ++t) {
      const MmPlan x = mm_plan(bf16, dx->j.M, dx->j.N, dx->j.K, dx->j.segs, dx->j.batch, false, false, false, kTogether[t]);
      const MmPlan w = mm_plan(bf16, dw->j.M, dw->j.N, dw->j.K, dw->j.segs, dw->j.batch, false, true, false, kTogether[t]);
      // all workgroups' time over the CUs, half of the last one's, and the joins
      const double us = (x.items * x.each + w.items * w.each) / 256 + 0.5 * (x.each > w.each ? x.each : w.each) + x.join + w.join;
      if (t == 0 || us < best) best = us, sx = x, sw = w;
    }
    together = 0.8 * (sx.us + sw.us) <= px.us + pw.us + 3.0;
    if (together) px = sx, pw = sw;
  }
  // with no slices to join the sums are joined while the pass that wrote them has them in cache
  const MmJoin x = dx ? join_of(dx->j, dx->e, px, dx->part) : MmJoin{}, w = dw ? join_of(dw->j, dw->e, pw, dw->part) : MmJoin{};
  const bool tail = x.blocks + w.blocks > 0;
  if (!tail)
    if (hipError_t r = launch_col_sum(sum, st); r != hipSuccess) return r;
  if (together) {
    const MmSlices sx = slices_of(px, dx->part), sw = slices_of(pw, dw->part);
    const int bn = px.tile.bn;
    const unsigned first = mm_grid(dx->j, sx, 64, bn), all = first + mm_grid(dw->j, sw, 64, bn);
    const bool whole = whole_chunks(dx->j) && whole_chunks(dw->j);
    auto go = [&](auto kernel) { kernel<<<all, 256, 0, st>>>(dx->j, dx->e, sx, (int)first, dw->j, dw->e, sw); };
    if (bf16) go(k_dense_mm_two<uint16_t, 64, 2, 2, 4, 16>);
    else if (bn == 64 && whole) go(k_dense_mm_two<float, 64, 2, 2, 3, 16>);
    else if (bn == 64) go(k_dense_mm_two<float, 64, 2, 2, 3, 4>);
    else if (whole) go(k_dense_mm_two<float, 32, 4, 1, 3, 16>);
    else go(k_dense_mm_two<float, 32, 4, 1, 3, 4>);
    if (hipError_t r = hipGetLastError(); r != hipSuccess) return r;
  } else {
    if (dx)
      if (hipError_t r = launch_sliced(dx->j, dx->e, px, bf16, dx->part, st); r != hipSuccess) return r;
    if (dw)
      if (hipError_t r = launch_sliced(dw->j, dw->e, pw, bf16, dw->part, st); r != hipSuccess) return r;
  }
  if (!tail) return hipSuccess;
  const unsigned blocks = x.blocks + w.blocks + (sum.P ? ceil_div(sum.N, 16) : 0);
  if (bf16) k_dense_tail<uint16_t><<<blocks, 256, 0, st>>>(x, w, sum);
  else k_dense_tail<float><<<blocks, 256, 0, st>>>(x, w, sum);
  return hipGetLastError();
}

}  // namespace moe
