// What the dense products may read, checked on the host without running a kernel: every launch that
// a call's products take is replayed tile by tile with the kernel's own address functions, and each
// lane's load that the buffer range lets through has to lie inside its operand, and each load that
// a stored result needs has to be let through.
//
//   dense_bounds bf16|f32 terms T K N ...   prints, a line for each size,
//   "<output columns left of the cut: gated and linear forward, gated and linear dx, dw>" (0: not cut)
#include <stdio.h>
#include <stdlib.h>
#include <string.h>

#include "dense_mm.hip"

using namespace moe;

hipError_t moe::launch_col_sum(const ColSum&, hipStream_t) { return hipSuccess; }

static int failures = 0;

// An operand: its first byte and how many it has.
struct Span { int64_t base, bytes; };

// One side of a tile: `from` its first row or column from p on, `valid` how many of them the product
// has, `column` a column operand's tile's first column in the operand's rows.
template <typename Tile, bool COL, int DB>
static void side(const char* what, const DenseJob& j, const void* p, const Span& span, int64_t ld, int from, int valid,
                 int column, int k0, int BK) {
  constexpr int ES = Tile::ES;
  const int rows = k0 + BK < j.K ? BK : j.K - k0;
  const int64_t at = reinterpret_cast<int64_t>(p) + (COL ? from + k0 * ld : from * ld + k0) * ES;
  const int bytes = COL ? mm_col_bytes(rows, ld, column, ES)
                        : mm_row_bytes(valid, ld, ES) - k0 * ES;
  for (int q = 0; q < Tile::INSTR; ++q)
    for (int lane = 0; lane < 64; ++lane) {
      uint32_t off = Tile::src(q, lane, ld, valid);
      if (!COL && Tile::element(q, lane) >= rows) off = kOutOfRange;
      const bool read = off < (uint32_t)(bytes > 0 ? bytes : 0);
      const int64_t lo = at + off - span.base;
      bool need;
      if (COL) {  // the load's contraction row and its first column in the tile
        const int k = (int)(off / ES / ld), c = (int)(off / ES - k * ld);
        need = k < rows && c < valid;
      } else {
        need = Tile::row(q, lane) < valid && Tile::element(q, lane) < rows;
      }
      if ((read && (lo < 0 || lo + DB > span.bytes)) || (need && !read)) {
        if (++failures < 20)
          fprintf(stderr, "%s: M %d N %d K %d, from %d, k %d: bytes %lld .. of %lld %s\n", what, j.M, j.N, j.K, from, k0,
                  (long long)lo, (long long)span.bytes, read ? "read" : "left out");
        return;
      }
    }
}

template <typename T, int BM, int BN, int SB, int DB, bool A_COL, bool B_COL>
static void tiles(const char* what, const DenseJob& j, const Span* sa, const Span* sb) {
  constexpr int BK = SB / (int)sizeof(T);
  const int on = j.pair ? BN / 2 : BN;
  using TA = MmTile<T, BM, A_COL, SB, DB>;
  using TB = MmTile<T, BN, B_COL, SB, DB>;
  const int last = (j.K - 1) / BK * BK;
  const int b_planes = j.pair ? 2 : j.batch;
  for (int k0 : {0, last})
    for (int seg = 0; seg < j.segs; ++seg) {
      for (int z = 0; z < j.batch; ++z)
        for (int m0 = 0; m0 < j.M; m0 += BM)
          if (m0 == 0 || m0 + 2 * BM >= j.M)
            side<TA, A_COL, DB>(what, j, j.A[z][seg], sa[z], j.lda, m0, j.M - m0 < BM ? j.M - m0 : BM, m0, k0, BK);
      for (int z = 0; z < b_planes; ++z)
        for (int n0 = 0; n0 < j.N; n0 += on)
          if (n0 == 0 || n0 + 2 * on >= j.N)
            side<TB, B_COL, DB>(what, j, j.B[z][seg], sb[z], j.ldb, n0, j.N - n0 < on ? j.N - n0 : on, mm_b_column(j, n0), k0, BK);
    }
}

template <typename T, int BM, int BN, int SB, int DB>
static void layouts(const char* what, const DenseJob& j, const Span* sa, const Span* sb) {
  if (!j.a_col && !j.b_col) tiles<T, BM, BN, SB, DB, false, false>(what, j, sa, sb);
  else if (!j.a_col) tiles<T, BM, BN, SB, DB, false, true>(what, j, sa, sb);
  else if constexpr ((BM & (BM - 1)) == 0) tiles<T, BM, BN, SB, DB, true, true>(what, j, sa, sb);
}

// The tile shapes as launch_planned and launch_dense_grads take them.
static void launch(const char* what, const DenseJob& j, const MmPlan& p, bool bf16, const Span* sa, const Span* sb) {
  const int bm = p.tile.bm, bn = p.tile.bn;
  if (!bf16) {
    if (bn == 64 && whole_chunks(j)) layouts<float, 64, 64, 128, 16>(what, j, sa, sb);
    else if (bn == 64) layouts<float, 64, 64, 128, 4>(what, j, sa, sb);
    else if (whole_chunks(j)) layouts<float, 64, 32, 128, 16>(what, j, sa, sb);
    else layouts<float, 64, 32, 128, 4>(what, j, sa, sb);
  } else if (bn == 256) layouts<uint16_t, 256, 256, 64, 16>(what, j, sa, sb);
  else if (bm == 256) layouts<uint16_t, 256, 128, 128, 16>(what, j, sa, sb);
  else if (bm == 192) layouts<uint16_t, 192, 128, 128, 16>(what, j, sa, sb);
  else if (bm == 128) layouts<uint16_t, 128, 128, 128, 16>(what, j, sa, sb);
  else layouts<uint16_t, 64, 64, 128, 16>(what, j, sa, sb);
}

// A product on its own, and (backward) on the tiles of a joint launch.  Returns its cut.
static int product(const char* what, const DenseJob& j, bool bf16, bool backward) {
  const int es = bf16 ? 2 : 4;
  Span sa[2], sb[2];
  for (int z = 0; z < 2; ++z) {
    sa[z] = {reinterpret_cast<int64_t>(j.A[z][0]), (int64_t)(j.a_col ? j.K : j.M) * j.lda * es};
    sb[z] = {reinterpret_cast<int64_t>(j.B[z][0]), (int64_t)(j.b_col ? j.K : j.N) * j.ldb * es};
  }
  const MmPlan p = plan_of(j, bf16);
  if (p.cut) {
    DenseJob left, right;
    DenseEpi e{}, er;
    cut_product(j, e, p, bf16, left, right, er);
    launch(what, left, p, bf16, sa, sb);
    launch(what, right, plan_of_rest(right, bf16), bf16, sa, sb);
  } else {
    launch(what, j, p, bf16, sa, sb);
  }
  for (int t = 0; backward && t < (bf16 ? 1 : 2); ++t)
    launch(what, j, mm_plan(bf16, j.M, j.N, j.K, j.segs, j.batch, j.pair, j.a_col, false, kTogether[t]), bf16, sa, sb);
  return p.cut;
}

int main(int argc, char** argv) {
  const bool bf16 = !strcmp(argv[1], "bf16");
  const int terms = atoi(argv[2]);
  const void* far[2] = {reinterpret_cast<void*>(1ll << 44), reinterpret_cast<void*>(2ll << 44)};
  const void* away[2] = {reinterpret_cast<void*>(3ll << 44), reinterpret_cast<void*>(4ll << 44)};
  for (int i = 3; i + 2 < argc; i += 3) {
    const int T = atoi(argv[i]), K = atoi(argv[i + 1]), N = atoi(argv[i + 2]);
    const int64_t ldk = bf16 ? (K + 7) / 8 * 8 : K, ldn = bf16 ? (N + 7) / 8 * 8 : N;
    int cut[6];
    for (int gated = 1; gated >= 0; --gated) {
      DenseJob f{}, x{}, w{};
      f.M = T; f.N = N; f.K = K;
      f.segs = f.batch = 1;
      f.pair = gated;
      x.M = T; x.N = K; x.K = N;
      x.segs = 1 + gated; x.batch = 1;
      x.b_col = true;
      w.M = N; w.N = K; w.K = T;
      w.segs = terms; w.batch = 1 + gated;
      w.a_col = w.b_col = true;
      f.lda = f.ldb = x.ldb = w.ldb = ldk;
      x.lda = w.lda = ldn;
      for (int z = 0; z < 2; ++z)
        for (int s = 0; s < 3; ++s) {
          f.A[z][s] = x.A[z][s] = w.A[z][s] = far[z];
          f.B[z][s] = x.B[z][s] = w.B[z][s] = away[z];
        }
      cut[1 - gated] = T <= kDecodeRows ? 0 : product("forward", f, bf16, false);
      cut[3 - gated] = product("dx", x, bf16, true);
      cut[5 - gated] = product("dw", w, bf16, true);
    }
    printf("%d %d %d %d %d %d\n", cut[0], cut[1], cut[2], cut[3], cut[4], cut[5]);
  }
  return failures != 0;
}
