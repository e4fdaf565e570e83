// The tile of a product on the matrix cores (the layouts are described in dense_kernels.h):
// v_mfma_f32_16x16x32_bf16, for fp32 operands v_mfma_f32_16x16x4_f32, for 8-bit integers
// v_mfma_i32_16x16x64_i8.  Shared by the dense products, the products grouped by expert and the
// integer ones.
#pragma once

#include <type_traits>

#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_dst;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr uint32_t kOutOfRange = 0x80000000u;  // a lane offset no buffer of ours reaches: reads 0

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const char*>(((uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32) | (uint32_t)uniform((int)a));
}

// What a tile may read of an operand, in bytes.  A row operand: from its first row on, whole rows and
// none past the last.  A column operand: from column `from` of a contraction step's first row to
// the end of the last of its `rows` rows (tests/host/dense_bounds.hip replays every launch's loads
// against their operands).
__host__ __device__ __forceinline__ int mm_row_bytes(int rows, int64_t ld, int es) { return rows * (int)ld * es; }
__host__ __device__ __forceinline__ int mm_col_bytes(int rows, int64_t ld, int from, int es) {
  return (rows * (int)ld - from) * es;
}
// The column of a column operand B's rows at which the tile at output column n0 starts.
__host__ __device__ __forceinline__ int mm_b_column(const DenseJob& j, int n0) { return j.b_from + n0; }

// A tile of R rows (m or n) by one contraction step in LDS, filled by buffer loads straight into
// LDS (DB = 16 bytes per lane, lane i to byte DB i of the instruction's part; 4 for fp32 rows
// that are no whole number of 16-byte chunks) and read as MFMA operands in
// pieces of 64 bytes of contraction, of which a step has one or two (SB = 64 or 128): lane l
// holds row l % 16, the (l / 16)-th 16 bytes of the piece's contraction elements.
// For bf16 and 8-bit integers that is one instruction's operand; for fp32 the i-th of four instructions takes
// element i of every lane's four, an order of the contraction that both sides share.
//
// Row operands (contraction along memory): LDS row r is SB bytes, its 16-byte chunk c sits at
// slot c ^ swz(r), so the 16 rows one ds_read_b128 touches at one chunk index cover all banks.
//
// bf16 column operands (contraction across memory): LDS row k holds R elements, and
// ds_read_b64_tr_b16 turns 4 x 16 blocks into operand order: of each 16 lanes, lane i reads
// 8 bytes of row i / 4 at 4 (i % 4) and receives element i of rows 0..3.  The 32-byte unit u
// of row k sits at u ^ f(k) with f(k) = (k & 3) | (k >> 1 & 4), which spreads the 16 rows one
// instruction touches over all banks.  fp32 column operands are read a dword per element, 16
// lanes to a 64-byte unit of one row; unit u of row k sits at u ^ (k >> 2 & 3).
template <typename T, int R, bool COL, int SB, int DB>
struct MmTile {
  static constexpr int ES = sizeof(T);
  static constexpr int HALFS = R * SB / 2;       // 16-bit words of the tile
  static constexpr int INSTR = R * SB / (64 * DB);  // fill instructions
  static constexpr int PER = 16 / DB;               // lanes of a 16-byte chunk
  static constexpr int CPR = R * ES / 16;           // column operand: chunks per LDS row
  static constexpr int UC = ES;                     // and chunks per unit (16 elements)
  static constexpr int RC = SB / 16;                // row operand: chunks per LDS row
  static __host__ __device__ __forceinline__ int swz(int r) { return SB == 128 ? r & 7 : (r >> 1) & 3; }
  // Row operand: the row that a lane of fill instruction q fills, and its first element there.
  static __host__ __device__ __forceinline__ int row(int q, int lane) { return (q * 64 + lane) / (RC * PER); }
  static __host__ __device__ __forceinline__ int element(int q, int lane) {
    return ((((lane / PER) % RC) ^ swz(row(q, lane))) * PER + lane % PER) * (DB / ES);
  }
  static_assert(!COL || (R & (R - 1)) == 0, "units are exchanged within a power of two");
  static __host__ __device__ __forceinline__ int f(int k) {
    return (ES == 2 ? (k & 3) | ((k >> 1) & 4) : (k >> 2) & 3) & (R / 16 - 1);
  }

  // Byte offset of lane's DB bytes of fill instruction q, from the tile's first row at
  // contraction 0 (row operand; rows >= valid are out of range) or from the tile's first
  // element of the step's first contraction row (column operand).
  static __host__ __device__ __forceinline__ uint32_t src(int q, int lane, int64_t ld, int valid) {
    if constexpr (COL) {
      const int at = q * 64 + lane, k = at / (CPR * PER), s = at / PER % CPR;
      const int chunk = ((s / UC) ^ f(k)) * UC + s % UC;
      return (uint32_t)(k * ld * ES + chunk * 16 + lane % PER * DB);
    } else {
      const int r = row(q, lane);
      return r < valid ? (uint32_t)((r * ld + element(q, lane)) * ES) : kOutOfRange;
    }
  }

  // Operand of rows row0 + 16 i .. + 16 (row0 a multiple of 16), contraction piece h, of the tile
  // at 16-bit word `at` of a stage.  One pointer addition from the stage's array: the compiler
  // follows only a few when it derives what a read can alias.
  static __device__ __forceinline__ u32x4 read(const uint16_t* stage, int at, int row0, int i, int h, int lane) {
    if constexpr (COL && ES == 4) {
      const int g = lane >> 4, k = 16 * h + 4 * g, u = ((row0 >> 4) + i) ^ f(k);
      const int o = at + 2 * (k * R + u * 16 + (lane & 15));
      u32x4 v;
#pragma unroll
      for (int e = 0; e < 4; ++e) v[e] = *reinterpret_cast<const uint32_t*>(stage + (o + 2 * e * R));
      return v;
    } else if constexpr (COL) {
      const int g = lane >> 4, j = (lane >> 2) & 3;
      const int k = 32 * h + 8 * g + j, u = ((row0 >> 4) + i) ^ f(8 * g + j);
      const int o = at + k * R + u * 16 + (lane & 3) * 4;
      s16x4 v[2];
      v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(stage + o));
      v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(stage + (o + 4 * R)));
      return __builtin_bit_cast(u32x4, v);
    } else {
      const int r = row0 + (lane & 15);
      const int o = at + (r + 16 * i) * (SB / 2) + (((4 * h + (lane >> 4)) ^ swz(lane & 15)) << 3);
      return *reinterpret_cast<const u32x4*>(stage + o);
    }
  }
};

// Eight neighbouring output columns n .. n + 7 of row m (the first `left` of them), from the
// fp32 sums; rows of odd widths are stored at element alignment.  ACT: the activation; PAST: past the caches; bias and
// res: the bias' and the residual's eight, where there are such; o: the first element of row 0.
template <typename T, int KIND, int ACT, bool PAST = false>
__device__ __forceinline__ void mm_out8(const DenseEpi& e, int z, int64_t o, int m, int n, int N, float* a,
                                        const float* b, const Raw8<T>& bias, const Raw8<T>& res) {
  constexpr bool FAST = sizeof(T) == 2;
  const int64_t idx = o + (int64_t)m * e.ldo + n;
  const int left = N - n;
  float y[8];
  if constexpr (KIND == DENSE_STORE) {
    if (e.out_f32) store8<PAST>(static_cast<float*>(e.out[z]) + idx, left, a);
    else store8<PAST>(static_cast<T*>(e.out[z]) + idx, left, a);
  } else if constexpr (KIND == DENSE_LINEAR) {
    if (e.bias) {
      for (int i = 0; i < 8; ++i) a[i] += bias.get(i);
    }
    if (e.save[0]) store8<PAST>(static_cast<T*>(e.save[0]) + idx, left, a);
    for (int i = 0; i < 8; ++i) a[i] = act_value<FAST>(a[i], ACT);
    if (e.residual) {
      for (int i = 0; i < 8; ++i) a[i] += res.get(i);
    }
    store8<PAST>(static_cast<T*>(e.out[0]) + idx, left, a);
  } else {
    if (e.save[0]) {
      store8<PAST>(static_cast<T*>(e.save[0]) + idx, left, a);
      store8<PAST>(static_cast<T*>(e.save[1]) + idx, left, b);
    }
    for (int i = 0; i < 8; ++i) y[i] = act_value<FAST>(a[i], ACT) * b[i];
    store8<PAST>(static_cast<T*>(e.out[0]) + idx, left, y);
  }
}

template <typename T, int KIND>
__device__ __forceinline__ void load_bias(const DenseEpi& e, int n, int N, Raw8<T>* bias) {
  if (KIND == DENSE_LINEAR && e.bias) bias->load(static_cast<const T*>(e.bias) + n, N - n);
}
template <typename T, int KIND>
__device__ __forceinline__ void load_residual(const DenseEpi& e, int m, int n, int M, int N, Raw8<T>* res) {
  if (KIND == DENSE_LINEAR && e.residual)
    res->load(static_cast<const T*>(e.residual) + (int64_t)min(m, M - 1) * e.ldo + n, m < M ? N - n : 0);
}

// f(std::integral_constant<int, act>) for the activation of a launch.
template <int KIND, typename F>
__device__ __forceinline__ void with_act(int act, F&& f) {
  if constexpr (KIND != DENSE_STORE) {
    switch (act) {
      case MOE_ACT_RELU: return f(std::integral_constant<int, MOE_ACT_RELU>{});
      case MOE_ACT_SILU: return f(std::integral_constant<int, MOE_ACT_SILU>{});
      case MOE_ACT_GELU: return f(std::integral_constant<int, MOE_ACT_GELU>{});
      case MOE_ACT_GELU_TANH: return f(std::integral_constant<int, MOE_ACT_GELU_TANH>{});
    }
  }
  f(std::integral_constant<int, MOE_ACT_NONE>{});
}

// Tile (m-tile, n-tile, batch) and contraction slice of a workgroup: work items are dealt to
// the 8 XCDs in contiguous chunks, within which groups of 8 m-tiles run down their n-tiles, so
// that the tiles an XCD works on at a time share rows and columns in its L2.
struct MmWhere { int mt, nt, z, slice; bool ok; };

__device__ __forceinline__ MmWhere mm_where(int block, int tm, int tn, int batch, int slices) {
  const int total = tm * tn * batch * slices, per = ceil_div(total, 8);
  const int slot = block >> 3, L = (block & 7) * per + slot;
  MmWhere w{0, 0, 0, 0, slot < per && L < total};
  const int q = L / (tm * tn);
  w.slice = q / batch;
  w.z = q - w.slice * batch;
  const int t = L - q * (tm * tn), grp = t / (8 * tn), first = grp * 8, r = t - grp * (8 * tn);
  const int gsz = min(8, tm - first);
  w.nt = r / gsz;
  w.mt = first + (r - w.nt * gsz);
  return w;
}

// The product that a tile belongs to: its rows and contraction length and where its operands and its
// output start (elements), as one of those that a grouped launch covers.  row, col: its first row
// and column among the scales of an integer product; row too among those of a grouped launch's slices.
struct MmPart {
  int M, K;
  int64_t a, b, o;
  int64_t row, col;
};

// The fp32 sums of one contraction slice: rows of ldp (N rounded up to 8) columns, a plane per
// batch entry or projection, planes of a slice together.
struct MmSlices {
  float* part;   // NULL: one slice, straight to the epilogue
  int slices, planes, ldp;
  int rows;      // of a plane, in a grouped launch: those of all its products
  __device__ __forceinline__ f32x4* at(int slice, int plane, int m, int n, int M) const {  // n: a multiple of 8
    return reinterpret_cast<f32x4*>(part + (((int64_t)slice * planes + plane) * M + m) * ldp + n);
  }
};

// s_waitcnt immediate: at most n vector-memory operations outstanding (bits [3:0] and
// [15:14]), no LDS operation (bits [11:8]), exports as they are.
constexpr int mm_waitcnt(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }

// Passes of the epilogue: so many that W waves' sums of `tile` bytes find room in S stages of `stage` bytes.
constexpr int mm_passes(int stage, int S, int tile, int W) {
  int p = 1;
  while (stage / (tile / p) * S < W) p *= 2;
  return p;
}
template <int BM, int BN, int SB>
constexpr int kMmStage = (BM + BN) * SB / 2;  // 16-bit words of a stage

// Bound by the matrix cores where the device is full: 8192^3 in bf16 takes 819 us forward, 787 for
// dx and 772 for dw (1.34, 1.40 and 1.43 PFLOP/s on 256 x 256 tiles; the library's products of
// the three layouts run at 1.43, 1.34 and 1.18), 4096^3 in fp32 950 us (145 of the library's
// 154 TFLOP/s).  Smaller products are bound by their tiles' prologues, epilogues and last round.
//
// BM x BN tile by WM x WN waves, S LDS stages: up to S - 1 steps' loads are in flight while one
// stage is multiplied.  With PAIR the tile's first BN / 2 rows of B come from the first weight
// and the rest from the second, for the same BN / 2 output columns.
//
// The stages are separate arrays, used in an unrolled ring: the compiler then knows which
// loads into LDS a read has to wait for, and waits for no later ones.
//
// Steps of 128 bytes: all waves read a stage's operands and multiply at their own pace, one
// barrier per step.  Steps of 64 bytes (8 waves, two per SIMD): the waves of a SIMD take turns,
// one reading a step's operands while the other multiplies, a barrier after each turn.
//
// T: the operands' type; O: that of what the epilogue reads and writes.  GROUPED: a wave with no row of the
// product does not multiply (rows in groups of any number end inside most tiles), and outputs are written past the
// caches, where the operands that other tiles read again stay (32768 rows of 128 experts, 2048 -> 768, a gated backward
// pass: 642 us, 706 with ordinary stores).  A product that reads them next loses nothing by it: a gated product and the
// linear one after it, 2048 / 768, take 393 us (429) for 32768 rows of 128 experts, 250 (251) for 4096 and 23 (23) for 64 of
// 8; in integers, each after its codes, 302 (309), 163 (164) and 29 (29), and 8192 dense rows, 2048 / 7168, 371 (396).
// STREAM: past the caches go B's loads too, for weights that one tile reads.  HEIGHT: rows that the waves share, where A's
// tile in LDS is filled by whole instructions of every wave and has more (the rest reads 0); the 16-row blocks without rows
// are not multiplied then.
template <typename T, typename O, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool A_COL, bool B_COL, bool PAIR,
          int KIND, bool GROUPED = false, bool STREAM = false, int HEIGHT = BM>
__device__ __forceinline__ void mm_body(const DenseJob& j, const DenseEpi& e, const MmSlices& sl, const MmWhere& w,
                                        const MmPart& at, uint16_t* s0, uint16_t* s1, uint16_t* s2, uint16_t* s3) {
  using TA = MmTile<T, BM, A_COL, SB, DB>;
  using TB = MmTile<T, BN, B_COL, SB, DB>;
  constexpr int ES = sizeof(T), BK = SB / ES;
  constexpr int W = WM * WN, TM = HEIGHT / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int QA = TA::INSTR / W, QB = TB::INSTR / W;
  constexpr int ON = PAIR ? BN / 2 : BN;   // output columns of a tile
  static_assert(QA >= 1 && QB >= 1 && !(PAIR && (B_COL || FN % 2)), "tile");
  static_assert(S == 3 || S == 4, "stages");
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  constexpr bool INT8 = ES == 1;
  using Acc = std::conditional_t<INT8, i32x4, f32x4>;

  if (!w.ok) return;
  const int m0 = uniform(w.mt * HEIGHT), n0 = uniform(w.nt * ON), z = uniform(w.z);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = ceil_div(at.K, BK), slice = uniform(w.slice);
  const int first = (int)((int64_t)nk * j.segs * slice / sl.slices);  // this slice's steps
  const int steps = (int)((int64_t)nk * j.segs * (slice + 1) / sl.slices) - first;

  // fill: this wave's instructions are wave * Q .. + Q of each tile
  uint32_t va[QA], vb[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) va[q] = TA::src(wave * QA + q, lane, j.lda, HEIGHT == BM ? at.M - m0 : min(HEIGHT, at.M - m0));
  const bool second = PAIR && wave >= W / 2;
#pragma unroll
  for (int q = 0; q < QB; ++q)
    vb[q] = TB::src((PAIR ? wave % (W / 2) : wave) * QB + q, lane, j.ldb, j.N - n0);
  // of the next step to load: where the tile starts and how many bytes from there are the
  // operand's (whole rows of it, none past its last one)
  const char *pa, *pb;
  int na, nb, left, seg = first / max(nk, 1);                   // left: contraction elements to load of this segment
  auto segment = [&]() __attribute__((always_inline)) {
    const void* b = PAIR ? (second ? j.B[1][0] : j.B[0][0]) : j.B[z][seg];
    pa = uniform(static_cast<const char*>(j.A[z][seg]) + (at.a + (A_COL ? (int64_t)m0 : (int64_t)m0 * j.lda)) * ES);
    pb = uniform(static_cast<const char*>(b) + (at.b + (B_COL ? (int64_t)n0 : (int64_t)n0 * j.ldb)) * ES);
    na = mm_row_bytes(min(HEIGHT, at.M - m0), j.lda, ES);
    nb = mm_row_bytes(min(ON, j.N - n0), j.ldb, ES);
    left = at.K;
  };
  auto advance = [&](int n) __attribute__((always_inline)) {
    left -= n * BK;
    pa += n * (A_COL ? (int64_t)SB * j.lda : SB);
    pb += n * (B_COL ? (int64_t)SB * j.ldb : SB);
    na -= n * SB;
    nb -= n * SB;
  };
  // The next step's loads (cache policy 2: not to be kept).  Past the last step they are issued all the same with an empty
  // buffer (zeros, no memory read), so that the count of loads in flight is the same at every
  // wait, which the compiler's own waits need too.
  int filled = 0;
  auto fill = [&](uint16_t* st) __attribute__((always_inline)) {
    const bool live = filled++ < steps;
    if (left <= 0 && live) {
      ++seg;
      segment();
    }
    const int rows = min(BK, left);
    auto one = [&](const char* p, int n, bool col, const uint32_t* v, int Q, int q0, int dst)
        __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(p), 0, uniform(live ? n : 0), 0x00020000);
#pragma unroll
      for (int q = 0; q < Q; ++q) {
        const uint32_t off = col || TA::element(q0 + q, lane) < rows ? v[q] : kOutOfRange;
        const lds_dst to = (lds_dst)(st + (dst + (q0 + q) * 32 * DB));
        if constexpr (DB == 16) {
          if (STREAM && dst) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, off, 0, 0, 2);
          else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, off, 0, 0, 0);
        }
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 4, off, 0, 0, 0);
      }
    };
    one(pa, A_COL ? mm_col_bytes(rows, j.lda, m0, ES) : na, A_COL, va, QA, wave * QA, 0);
    one(pb, B_COL ? mm_col_bytes(rows, j.ldb, mm_b_column(j, n0), ES) : nb, B_COL, vb, QB, wave * QB, TA::HALFS);
    advance(1);
  };

  const int mine = at.M - m0 - wm * TM;   // rows of this wave, in tiles of rows that no other expert has
  Acc acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = Acc{};
  auto mfma = [&](u32x4 b, u32x4 a, Acc c) __attribute__((always_inline)) {
    if constexpr (INT8) return __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, b), __builtin_bit_cast(i32x4, a), c, 0, 0, 0);
    else return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(b), as_bf16x8(a), c, 0, 0, 0);
  };
  static_assert(HEIGHT == BM || (SB == 64 && W == 8), "only turns leave blocks out");
  auto multiply = [&](const uint16_t* st) __attribute__((always_inline)) {
    if (GROUPED && mine <= 0) return;
#pragma unroll
    for (int h = 0; h < SB / 64; ++h) {
      u32x4 fb[FN];
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        // with PAIR, the wave's first half of columns in the first weight's rows, then the second's
        const int row0 = PAIR ? wn * (TN / 2) + (b / (FN / 2)) * ON : wn * TN;
        fb[b] = TB::read(st, TA::HALFS, row0, PAIR ? b % (FN / 2) : b, h, lane);
      }
      if constexpr (ES <= 2) {
#pragma unroll
        for (int a = 0; a < FM; ++a) {
          const u32x4 fa = TA::read(st, 0, wm * TM, a, h, lane);
#pragma unroll
          for (int b = 0; b < FN; ++b)
            acc[a][b] = mfma(fb[b], fa, acc[a][b]);
        }
      } else {
        u32x4 fa[FM];
#pragma unroll
        for (int a = 0; a < FM; ++a) fa[a] = TA::read(st, 0, wm * TM, a, h, lane);
#pragma unroll
        for (int e = 0; e < 4; ++e)  // FM * FN independent sums between two products of one
#pragma unroll
          for (int a = 0; a < FM; ++a)
#pragma unroll
            for (int b = 0; b < FN; ++b)
              acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(fb[b][e]), __uint_as_float(fa[a][e]),
                                                               acc[a][b], 0, 0, 0);
      }
    }
  };
  // One step: the stage's loads have landed (behind them at most S - 2 later stages' are in
  // flight) and this wave's reads of the stage before are done; then so for every wave, and
  // that earlier stage takes the loads of S - 1 steps on.
  auto step = [&](const uint16_t* cur, uint16_t* last) __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(mm_waitcnt((S - 2) * (QA + QB)));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    fill(last);  // the compiler may move these loads among the products: a ring this deep has the time
    multiply(cur);
  };

  // The same in turns.  In a wave's reading turn of step s it issues the loads of step s + 3 into
  // the stage of step s - 1 (whose readers are done: the other wave's turn ended with the last
  // barrier) and reads its operands; in the next turn it multiplies.  The early waves read step
  // s + 1 two turns after they read s, so every wave's loads of it must have landed (with the 2
  // later steps' in flight) by the end of the turn between: there the early waves multiply and
  // the late ones read.
  const bool late = wave >= W / 2;
  auto turn = [&](const uint16_t* cur, uint16_t* last) __attribute__((always_inline)) {
    constexpr int flight = 2 * (QA + QB);
    u32x4 fa[FM], fb[FN];
    fill(last);
    __builtin_amdgcn_sched_barrier(0);
#pragma unroll
    for (int b = 0; b < FN; ++b)
      fb[b] = TB::read(cur, TA::HALFS, PAIR ? wn * (TN / 2) + (b / (FN / 2)) * ON : wn * TN, PAIR ? b % (FN / 2) : b, 0, lane);
#pragma unroll
    for (int a = 0; a < FM; ++a) fa[a] = TA::read(cur, 0, wm * TM, a, 0, lane);
    __builtin_amdgcn_sched_barrier(0);
    if (late) __builtin_amdgcn_s_waitcnt(mm_waitcnt(flight));
    else __builtin_amdgcn_s_waitcnt(mm_waitcnt(63));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
    __builtin_amdgcn_sched_barrier(0);
    if (!GROUPED || mine > 0) {
      __builtin_amdgcn_s_setprio(1);
#pragma unroll
      for (int a = 0; a < FM; ++a) {
        if (HEIGHT != BM && 16 * a >= mine) continue;
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = mfma(fb[b], fa[a], acc[a][b]);
      }
      __builtin_amdgcn_s_setprio(0);
    }
    __builtin_amdgcn_sched_barrier(0);
    if (!late) __builtin_amdgcn_s_waitcnt(mm_waitcnt(flight));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  segment();
  advance(first - seg * nk);
  fill(s0);
  fill(s1);
  if (S > 3) fill(s2);
  if constexpr (SB == 64 && W == 8) {
    static_assert(S == 4 && ES <= 2, "turns");
    __builtin_amdgcn_s_waitcnt(mm_waitcnt(2 * (QA + QB)));
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    if (late) __builtin_amdgcn_s_barrier();  // a turn behind
    asm volatile("" ::: "memory");
    int s = 0;
    for (; s + S <= steps; s += S) {
      turn(s0, s3);
      turn(s1, s0);
      turn(s2, s1);
      turn(s3, s2);
    }
    if (s < steps) turn(s0, s3);
    if (s + 1 < steps) turn(s1, s0);
    if (s + 2 < steps) turn(s2, s1);
    if (!late) __builtin_amdgcn_s_barrier();
  } else {
    // whole rounds of the ring, then the rest of one: with exits inside the round the compiler
    // merges their states and waits for the newest loads at the loop's head
    int s = 0;
    for (; s + S <= steps; s += S) {
      step(s0, S == 3 ? s2 : s3);
      step(s1, s0);
      step(s2, s1);
      if (S > 3) step(s3, s2);
    }
    if (s < steps) step(s0, S == 3 ? s2 : s3);
    if (s + 1 < steps) step(s1, s0);
    if (S > 3 && s + 2 < steps) step(s2, s1);
  }
  __builtin_amdgcn_s_waitcnt(mm_waitcnt(0));

  // Epilogue through LDS, the stages being free now: a wave's sums go to a region of its own
  // (in passes where they are more than the stages hold), rows of TN columns whose 16-byte chunks are rotated
  // by row, and come back eight columns of a row per lane: whole cache lines per store, and one
  // copy of the epilogue's code in a loop, where straight from the accumulators it would be
  // FM * FN copies (which cost 12 us of a 120 us product, 4096^3, in instruction fetches and
  // scattered stores).
  constexpr int PASSES = mm_passes(STAGE * 2, S, TM * TN * 4, W), PM = TM / PASSES, PF = FM / PASSES;
  constexpr int CH = TN / 4;                       // chunks per row
  constexpr int OC = PAIR ? TN / 2 : TN;           // output columns of the wave
  constexpr int LPR = OC / 8, RPI = 64 / LPR;      // lanes per row, rows per iteration
  constexpr int PER = STAGE * 2 / (PM * TN * 4);   // regions per stage array
  static_assert(PER * S >= W, "epilogue regions");
  uint16_t* stage = wave < PER ? s0 : wave < 2 * PER ? s1 : wave < 3 * PER ? s2 : s3;
  float* reg = reinterpret_cast<float*>(stage) + (wave % PER) * (PM * TN);
  const int nw = n0 + wn * OC, lr = lane / LPR, lc = lane % LPR;
  const int mw = m0 + wm * TM + lr, n = nw + 8 * lc;
  // A residual's rows are all on their way before the first is used: taken one iteration
  // at a time their latency is most of the epilogue (8192 x 2048 x 7168: 40 us of 273).
  constexpr int U = KIND == DENSE_LINEAR && PM > RPI ? PM / RPI : 1;
  Raw8<O> res[PASSES][U], bias;
  // An integer product's scales, of the rows and columns whose sums this lane has: they become fp32 on
  // their way to LDS.
  constexpr int BF = PAIR ? FN / 2 : FN;
  float by_row[INT8 ? FM : 1], by_col[INT8 ? FN : 1][4];
  if constexpr (INT8) {
#pragma unroll
    for (int a = 0; a < FM; ++a) by_row[a] = e.row_scale[at.row + min(m0 + wm * TM + 16 * a + (lane & 15), at.M - 1)];
#pragma unroll
    for (int b = 0; b < FN; ++b)
#pragma unroll
      for (int i = 0; i < 4; ++i)
        by_col[b][i] = e.col_scale[PAIR ? b / BF : 0][at.col + min(nw + 16 * (b % BF) + 4 * (lane >> 4) + i, j.N - 1)];
  }
  if (!sl.part) {
    load_bias<O, KIND>(e, n, j.N, &bias);
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < U; ++i) load_residual<O, KIND>(e, mw + p * PM + i * RPI, n, at.M, j.N, &res[p][i]);
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  // One of the wave's rows has a scale of two factors, the second of which follows on the way back.
  bool wide = false;
  if constexpr (INT8) {
#pragma unroll
    for (int a = 0; a < FM; ++a) {
      wide |= by_row[a] > kWideScale;
      by_row[a] = row_scale_by(by_row[a]);
    }
    wide = __ballot(wide) != 0;
  }
  auto pass = [&](auto which) __attribute__((always_inline)) {
    constexpr int p = which();
#pragma unroll
    for (int a = 0; a < PF; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        f32x4 v;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          v[i] = (float)acc[p * PF + a][b][i];
          if constexpr (INT8) v[i] = v[i] * by_row[p * PF + a] * by_col[b][i];
        }
        *reinterpret_cast<f32x4*>(reg + (16 * a + (lane & 15)) * TN + (((4 * b + (lane >> 4)) ^ (lane & (CH - 1) & 15)) << 2)) = v;
      }
    asm volatile("" ::: "memory");  // the region is this wave's, and its LDS operations stay in order
    __builtin_amdgcn_wave_barrier();
    const int mp = mw + p * PM;
    auto chunk = [&](int r, int c) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4*>(reg + r * TN + ((c ^ (r & (CH - 1) & 15)) << 2));
    };
    if (sl.part) {
      for (int r = lr; r < PM; r += RPI) {
        const int m = mp + r - lr;
        if (m >= at.M || n >= j.N) continue;
        f32x4* o = sl.at(slice, z, GROUPED ? (int)at.row + m : m, n, GROUPED ? sl.rows : at.M);
        o[0] = chunk(r, 2 * lc);
        o[1] = chunk(r, 2 * lc + 1);
        if (PAIR) {
          o = sl.at(slice, 1, GROUPED ? (int)at.row + m : m, n, GROUPED ? sl.rows : at.M);
          o[0] = chunk(r, CH / 2 + 2 * lc);
          o[1] = chunk(r, CH / 2 + 2 * lc + 1);
        }
      }
    } else {
      with_act<KIND>(e.act, [&](auto act) __attribute__((always_inline)) {
        for (int r0 = 0; r0 < PM; r0 += U * RPI) {
#pragma unroll
          for (int i = 0; i < U; ++i) {
            const int r = r0 + i * RPI + lr, m = mp + r - lr;
            if (m >= at.M || n >= j.N || (RPI > PM && r >= PM)) continue;
            f32x4 v[2] = {chunk(r, 2 * lc), chunk(r, 2 * lc + 1)}, u[2] = {v[0], v[1]};
            if (PAIR) u[0] = chunk(r, CH / 2 + 2 * lc), u[1] = chunk(r, CH / 2 + 2 * lc + 1);
            if (INT8 && wide) {
              const float up = row_scale_up(e.row_scale[at.row + m]);
              for (int k = 0; k < 2; ++k) v[k] *= up, u[k] *= up;
            }
            mm_out8<O, KIND, act(), GROUPED>(e, z, at.o, m, n, j.N, reinterpret_cast<float*>(v), reinterpret_cast<const float*>(u),
                                    bias, res[p][i]);
          }
        }
      });
    }
    asm volatile("" ::: "memory");
    __builtin_amdgcn_wave_barrier();
  };
  pass(std::integral_constant<int, 0>{});
  if constexpr (PASSES > 1) pass(std::integral_constant<int, 1>{});
  if constexpr (PASSES > 2) pass(std::integral_constant<int, 2>{}), pass(std::integral_constant<int, 3>{});
}

}  // namespace moe
