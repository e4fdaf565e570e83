// What the products grouped by expert may read, checked on the host without running a kernel: the tiles
// that a call's launches take are replayed with the kernels' own address functions, and each lane's load that
// the buffer range lets through has to lie inside its operand, and each load that a stored result needs has to be let
// through.
//
//   grouped_bounds bf16|f32|int8 R K N E offset[0] .. offset[E]    prints the tile heights of the forward
//   products (linear, gated), dx and dw
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "grouped_mm.hip"

using namespace moe;

static int failures = 0;
static int R, K, N, E;
static int* offsets;

// The loads of one side of a tile for one contraction step: `start` the operand's first element that the step's tile has, of
// `span` bytes; `valid` rows or columns of the product from there on; `rows` contraction elements; `bytes` what the
// buffer range lets through.
template <typename Tile, bool COL, int DB>
static void side(const char* what, int64_t start, int64_t span, int64_t ld, int valid, int rows, int bytes) {
  constexpr int ES = Tile::ES;
  for (int q = 0; q < Tile::INSTR; ++q)
    for (int lane = 0; lane < 64; ++lane) {
      uint32_t off = Tile::src(q, lane, ld, valid);
      if (!COL && Tile::element(q, lane) >= rows) off = kOutOfRange;
      const bool read = off < (uint32_t)(bytes > 0 ? bytes : 0);
      const int64_t lo = start * ES + off;
      bool need;
      if (COL) {
        const int k = (int)(off / ES / ld), c = (int)(off / ES - k * ld);
        need = k < rows && c < valid;
      } else {
        need = Tile::row(q, lane) < valid && Tile::element(q, lane) < rows;
      }
      if ((read && (lo < 0 || lo + DB > span)) || (need && !read)) {
        if (++failures < 20)
          fprintf(stderr, "%s: byte %lld of %lld %s\n", what, (long long)lo, (long long)span, read ? "read" : "left out");
        return;
      }
    }
}

static int least(int a, int b) { return a < b ? a : b; }
static int held(int v, int lo) { return v < lo ? lo : v > R ? R : v; }

// Rows by weights: the first and last contraction step of each expert's first and last m-tile, first and last n-tile.
template <typename T, int BM, int BN, int SB, int DB, bool B_COL, int HEIGHT = BM>
static void by_rows(const char* what, int contraction, int cols, int64_t lda, int64_t ldb, int64_t w_stride, int on) {
  constexpr int ES = sizeof(T), BK = SB / ES;
  using TA = MmTile<T, BM, false, SB, DB>;
  using TB = MmTile<T, BN, B_COL, SB, DB>;
  for (int e = 0; e < E; ++e) {
    const int lo = held(offsets[e], 0), hi = held(offsets[e + 1], lo);
    const int h = tile_height(hi - lo, HEIGHT);
    for (int row = lo; row < hi; row += h) {
      if (row > lo && row + 2 * h < hi) continue;
      const int valid = least(h, hi - row);
      for (int k0 : {0, (contraction - 1) / BK * BK}) {
        const int rows = least(BK, contraction - k0);
        side<TA, false, DB>(what, row * lda + k0, R * lda * ES, lda, valid, rows, mm_row_bytes(valid, lda, ES) - k0 * ES);
        for (int n0 = 0; n0 < cols; n0 += on) {
          if (n0 > 0 && n0 + 2 * on < cols) continue;
          if (B_COL)
            side<TB, true, DB>(what, e * w_stride + n0 + k0 * ldb, E * w_stride * ES, ldb, least(on, cols - n0), rows,
                               mm_col_bytes(rows, ldb, n0, ES));
          else
            side<TB, false, DB>(what, e * w_stride + n0 * ldb + k0, E * w_stride * ES, ldb, least(on, cols - n0), rows,
                                mm_row_bytes(least(on, cols - n0), ldb, ES) - k0 * ES);
        }
      }
    }
  }
}

// Weight gradients: an expert's rows are the contraction.
template <typename T, int BM, int BN, int SB, int DB>
static void by_experts(const char* what, int64_t lda, int64_t ldb) {
  constexpr int ES = sizeof(T), BK = SB / ES;
  using TA = MmTile<T, BM, true, SB, DB>;
  using TB = MmTile<T, BN, true, SB, DB>;
  for (int e = 0; e < E; ++e) {
    const int lo = held(offsets[e], 0), hi = held(offsets[e + 1], lo), n = hi - lo;
    if (n == 0) continue;   // no step, empty buffers
    for (int k0 : {0, (n - 1) / BK * BK}) {
      const int rows = least(BK, n - k0);
      for (int m0 = 0; m0 < N; m0 += BM)
        if (m0 == 0 || m0 + 2 * BM >= N)
          side<TA, true, DB>(what, (lo + k0) * lda + m0, R * lda * ES, lda, least(BM, N - m0), rows, mm_col_bytes(rows, lda, m0, ES));
      for (int n0 = 0; n0 < K; n0 += BN)
        if (n0 == 0 || n0 + 2 * BN >= K)
          side<TB, true, DB>(what, (lo + k0) * ldb + n0, R * ldb * ES, ldb, least(BN, K - n0), rows, mm_col_bytes(rows, ldb, n0, ES));
    }
  }
}

int main(int argc, char** argv) {
  const GroupedType t = !strcmp(argv[1], "bf16") ? GROUPED_BF16 : !strcmp(argv[1], "f32") ? GROUPED_F32 : GROUPED_INT8;
  R = atoi(argv[2]); K = atoi(argv[3]); N = atoi(argv[4]); E = atoi(argv[5]);
  offsets = static_cast<int*>(malloc((E + 1) * sizeof(int)));
  for (int i = 0; i <= E; ++i) offsets[i] = atoi(argv[6 + i]);
  const int64_t ldk = t == GROUPED_INT8 ? (K + 15) / 16 * 16 : t == GROUPED_BF16 ? (K + 7) / 8 * 8 : K;
  const int64_t ldn = t == GROUPED_BF16 ? (N + 7) / 8 * 8 : N;
  int heights[4] = {};
  for (int gated = 0; gated < 2; ++gated) {
    const GroupedTile c = tile_of(t, R, E, N, K, 1, gated, false);
    heights[gated] = c.bm;
    const int on = gated ? c.bn / 2 : c.bn;
    const char* what = gated ? "gated forward" : "linear forward";
    if (t == GROUPED_F32) {
      if (ldk % 4 == 0) by_rows<float, 64, 64, 128, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
      else by_rows<float, 64, 64, 128, 4, false>(what, K, N, ldk, ldk, N * ldk, on);
    } else if (t == GROUPED_BF16) {
      if (c.bm == 320) by_rows<uint16_t, 384, 256, 64, 16, false, 320>(what, K, N, ldk, ldk, N * ldk, on);
      else if (c.bm == 128) by_rows<uint16_t, 128, 256, 64, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
      else if (c.bn == 128) by_rows<uint16_t, 64, 128, 128, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
      else by_rows<uint16_t, 64, 64, 128, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
    } else {
      if (c.bm == 320) by_rows<int8_t, 384, 256, 64, 16, false, 320>(what, K, N, ldk, ldk, N * ldk, on);
      else if (c.bm == 128) by_rows<int8_t, 128, 256, 64, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
      else if (c.bn == 128) by_rows<int8_t, 64, 128, 128, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
      else by_rows<int8_t, 64, 64, 128, 16, false>(what, K, N, ldk, ldk, N * ldk, on);
    }
    if (t == GROUPED_INT8) continue;
    const GroupedTile x = tile_of(t, R, E, K, N, 1 + gated, false, true);
    heights[2] = x.bm;
    DenseJob j{};
    j.M = N; j.N = K;
    j.segs = 1; j.batch = 1 + gated;
    const GroupedTile w = dw_tile_of(j, t, Groups{nullptr, E, R});
    heights[3] = w.bm;
    if (t == GROUPED_F32) {
      if (ldk % 4 == 0 && ldn % 4 == 0) {
        by_rows<float, 64, 64, 128, 16, true>("dx", N, K, ldn, ldk, N * ldk, 64);
        by_experts<float, 64, 64, 128, 16>("dw", ldn, ldk);
      } else {
        by_rows<float, 64, 64, 128, 4, true>("dx", N, K, ldn, ldk, N * ldk, 64);
        by_experts<float, 64, 64, 128, 4>("dw", ldn, ldk);
      }
    } else {
      if (x.bm == 320) by_rows<uint16_t, 384, 256, 64, 16, true, 320>("dx", N, K, ldn, ldk, N * ldk, 256);
      else if (x.bm == 128) by_rows<uint16_t, 128, 256, 64, 16, true>("dx", N, K, ldn, ldk, N * ldk, 256);
      else by_rows<uint16_t, 64, 64, 128, 16, true>("dx", N, K, ldn, ldk, N * ldk, 64);
      if (w.bm == 256) by_experts<uint16_t, 256, 256, 64, 16>("dw", ldn, ldk);
      else if (w.bm == 128) by_experts<uint16_t, 128, 256, 64, 16>("dw", ldn, ldk);
      else by_experts<uint16_t, 64, 64, 128, 16>("dw", ldn, ldk);
    }
  }
  printf("%d %d %d %d\n", heights[0], heights[1], heights[2], heights[3]);
  free(offsets);
  return failures != 0;
}
