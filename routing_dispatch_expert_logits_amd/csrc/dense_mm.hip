// Dense products on the matrix cores, fp32 accumulate (the layouts are described in
// dense_kernels.h): v_mfma_f32_16x16x32_bf16, or for fp32 operands v_mfma_f32_16x16x4_f32.
#include <type_traits>

#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
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
// For bf16 that is one instruction's operand; for fp32 the i-th of four instructions takes
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
// fp32 sums; rows of odd widths are stored at element alignment.  ACT: the activation; bias and
// res: the bias' and the residual's eight, where there are such.
template <typename T, int KIND, int ACT>
__device__ __forceinline__ void mm_out8(const DenseEpi& e, int z, int m, int n, int N, float* a, const float* b,
                                        const Raw8<T>& bias, const Raw8<T>& res) {
  constexpr bool FAST = sizeof(T) == 2;
  const int64_t idx = (int64_t)m * e.ldo + n;
  const int left = N - n;
  float y[8];
  if constexpr (KIND == DENSE_STORE) {
    if (e.out_f32) store8(static_cast<float*>(e.out[z]) + idx, left, a);
    else store8(static_cast<T*>(e.out[z]) + idx, left, a);
  } else if constexpr (KIND == DENSE_LINEAR) {
    if (e.bias) {
      for (int i = 0; i < 8; ++i) a[i] += bias.get(i);
    }
    if (e.save[0]) store8(static_cast<T*>(e.save[0]) + idx, left, a);
    for (int i = 0; i < 8; ++i) a[i] = act_value<FAST>(a[i], ACT);
    if (e.residual) {
      for (int i = 0; i < 8; ++i) a[i] += res.get(i);
    }
    store8(static_cast<T*>(e.out[0]) + idx, left, a);
  } else {
    if (e.save[0]) {
      store8(static_cast<T*>(e.save[0]) + idx, left, a);
      store8(static_cast<T*>(e.save[1]) + idx, left, b);
    }
    for (int i = 0; i < 8; ++i) y[i] = act_value<FAST>(a[i], ACT) * b[i];
    store8(static_cast<T*>(e.out[0]) + idx, left, y);
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

// The fp32 sums of one contraction slice: rows of ldp (N rounded up to 8) columns, a plane per
// batch entry or projection, planes of a slice together.
struct MmSlices {
  float* part;   // NULL: one slice, straight to the epilogue
  int slices, planes, ldp;
  __device__ __forceinline__ f32x4* at(int slice, int plane, int m, int n, int M) const {  // n: a multiple of 8
    return reinterpret_cast<f32x4*>(part + (((int64_t)slice * planes + plane) * M + m) * ldp + n);
  }
};

// s_waitcnt immediate: at most n vector-memory operations outstanding (bits [3:0] and
// [15:14]), no LDS operation (bits [11:8]), exports as they are.
constexpr int mm_waitcnt(int n) { return (n & 0xF) | ((n >> 4) << 14) | (0x7 << 4); }

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
template <int BM, int BN, int SB>
constexpr int kMmStage = (BM + BN) * SB / 2;  // 16-bit words of a stage
template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool A_COL, bool B_COL, bool PAIR, int KIND>
__device__ __forceinline__ void mm_body(const DenseJob& j, const DenseEpi& e, const MmSlices& sl, int block,
                                        uint16_t* s0, uint16_t* s1, uint16_t* s2, uint16_t* s3) {
  using TA = MmTile<T, BM, A_COL, SB, DB>;
  using TB = MmTile<T, BN, B_COL, SB, DB>;
  constexpr int ES = sizeof(T), BK = SB / ES;
  constexpr int W = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int QA = TA::INSTR / W, QB = TB::INSTR / W;
  constexpr int ON = PAIR ? BN / 2 : BN;   // output columns of a tile
  static_assert(QA >= 1 && QB >= 1 && !(PAIR && (B_COL || FN % 2)), "tile");
  static_assert(S == 3 || S == 4, "stages");
  constexpr int STAGE = kMmStage<BM, BN, SB>;

  const MmWhere w = mm_where(block, ceil_div(j.M, BM), ceil_div(j.N, ON), j.batch, sl.slices);
  if (!w.ok) return;
  const int m0 = uniform(w.mt * BM), n0 = uniform(w.nt * ON), z = uniform(w.z);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = ceil_div(j.K, BK), slice = uniform(w.slice);
  const int first = (int)((int64_t)nk * j.segs * slice / sl.slices);  // this slice's steps
  const int steps = (int)((int64_t)nk * j.segs * (slice + 1) / sl.slices) - first;

  // fill: this wave's instructions are wave * Q .. + Q of each tile
  uint32_t va[QA], vb[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) va[q] = TA::src(wave * QA + q, lane, j.lda, j.M - m0);
  const bool second = PAIR && wave >= W / 2;
#pragma unroll
  for (int q = 0; q < QB; ++q)
    vb[q] = TB::src((PAIR ? wave % (W / 2) : wave) * QB + q, lane, j.ldb, j.N - n0);
  // of the next step to load: where the tile starts and how many bytes from there are the
  // operand's (whole rows of it, none past its last one)
  const char *pa, *pb;
  int na, nb, left, seg = first / nk;                   // left: contraction elements to load of this segment
  auto segment = [&]() __attribute__((always_inline)) {
    const void* b = PAIR ? (second ? j.B[1][0] : j.B[0][0]) : j.B[z][seg];
    pa = uniform(static_cast<const char*>(j.A[z][seg]) + (A_COL ? (int64_t)m0 : (int64_t)m0 * j.lda) * ES);
    pb = uniform(static_cast<const char*>(b) + (B_COL ? (int64_t)n0 : (int64_t)n0 * j.ldb) * ES);
    na = mm_row_bytes(min(BM, j.M - m0), j.lda, ES);
    nb = mm_row_bytes(min(ON, j.N - n0), j.ldb, ES);
    left = j.K;
  };
  auto advance = [&](int n) __attribute__((always_inline)) {
    left -= n * BK;
    pa += n * (A_COL ? (int64_t)SB * j.lda : SB);
    pb += n * (B_COL ? (int64_t)SB * j.ldb : SB);
    na -= n * SB;
    nb -= n * SB;
  };
  // The next step's loads.  Past the last step they are issued all the same with an empty
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
        if constexpr (DB == 16) __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 16, off, 0, 0, 0);
        else __builtin_amdgcn_raw_ptr_buffer_load_lds(r, to, 4, off, 0, 0, 0);
      }
    };
    one(pa, A_COL ? mm_col_bytes(rows, j.lda, m0, ES) : na, A_COL, va, QA, wave * QA, 0);
    one(pb, B_COL ? mm_col_bytes(rows, j.ldb, mm_b_column(j, n0), ES) : nb, B_COL, vb, QB, wave * QB, TA::HALFS);
    advance(1);
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const uint16_t* st) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < SB / 64; ++h) {
      u32x4 fb[FN];
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        // with PAIR, the wave's first half of columns in the first weight's rows, then the second's
        const int row0 = PAIR ? wn * (TN / 2) + (b / (FN / 2)) * ON : wn * TN;
        fb[b] = TB::read(st, TA::HALFS, row0, PAIR ? b % (FN / 2) : b, h, lane);
      }
      if constexpr (ES == 2) {
#pragma unroll
        for (int a = 0; a < FM; ++a) {
          const u32x4 fa = TA::read(st, 0, wm * TM, a, h, lane);
#pragma unroll
          for (int b = 0; b < FN; ++b)
            acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fb[b]), as_bf16x8(fa), acc[a][b], 0, 0, 0);
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
    __builtin_amdgcn_s_setprio(1);
#pragma unroll
    for (int a = 0; a < FM; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
        acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(fb[b]), as_bf16x8(fa[a]), acc[a][b], 0, 0, 0);
    __builtin_amdgcn_s_setprio(0);
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
  if constexpr (SB == 64) {
    static_assert(S == 4 && W == 8 && ES == 2, "turns");
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
  // (in two passes where they are more than the stages hold), rows of TN columns whose 16-byte chunks are rotated
  // by row, and come back eight columns of a row per lane: whole cache lines per store, and one
  // copy of the epilogue's code in a loop, where straight from the accumulators it would be
  // FM * FN copies (which cost 12 us of a 120 us product, 4096^3, in instruction fetches and
  // scattered stores).
  constexpr int PASSES = TM * TN * 4 * W > S * STAGE * 2 ? 2 : 1, PM = TM / PASSES, PF = FM / PASSES;
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
  Raw8<T> res[PASSES][U], bias;
  if (!sl.part) {
    load_bias<T, KIND>(e, n, j.N, &bias);
#pragma unroll
    for (int p = 0; p < PASSES; ++p)
#pragma unroll
      for (int i = 0; i < U; ++i) load_residual<T, KIND>(e, mw + p * PM + i * RPI, n, j.M, j.N, &res[p][i]);
  }
  __builtin_amdgcn_s_barrier();
  asm volatile("" ::: "memory");
  auto pass = [&](auto which) __attribute__((always_inline)) {
    constexpr int p = which();
#pragma unroll
    for (int a = 0; a < PF; ++a)
#pragma unroll
      for (int b = 0; b < FN; ++b)
        *reinterpret_cast<f32x4*>(reg + (16 * a + (lane & 15)) * TN +
                                  (((4 * b + (lane >> 4)) ^ (lane & (CH - 1) & 15)) << 2)) = acc[p * PF + a][b];
    asm volatile("" ::: "memory");  // the region is this wave's, and its LDS operations stay in order
    __builtin_amdgcn_wave_barrier();
    const int mp = mw + p * PM;
    auto chunk = [&](int r, int c) __attribute__((always_inline)) {
      return *reinterpret_cast<const f32x4*>(reg + r * TN + ((c ^ (r & (CH - 1) & 15)) << 2));
    };
    if (sl.part) {
      for (int r = lr; r < PM; r += RPI) {
        const int m = mp + r - lr;
        if (m >= j.M || n >= j.N) continue;
        f32x4* o = sl.at(slice, z, m, n, j.M);
        o[0] = chunk(r, 2 * lc);
        o[1] = chunk(r, 2 * lc + 1);
        if (PAIR) {
          o = sl.at(slice, 1, m, n, j.M);
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
            if (m >= j.M || n >= j.N || (RPI > PM && r >= PM)) continue;
            f32x4 v[2] = {chunk(r, 2 * lc), chunk(r, 2 * lc + 1)}, u[2] = {v[0], v[1]};
            if (PAIR) u[0] = chunk(r, CH / 2 + 2 * lc), u[1] = chunk(r, CH / 2 + 2 * lc + 1);
            mm_out8<T, KIND, act()>(e, z, m, n, j.N, reinterpret_cast<float*>(v), reinterpret_cast<const float*>(u),
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
}

template <typename T, int BM, int BN, int WM, int WN, int S, int SB, int DB, bool A_COL, bool B_COL, bool PAIR,
          int KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_dense_mm(DenseJob j, DenseEpi e, MmSlices sl) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  mm_body<T, BM, BN, WM, WN, S, SB, DB, A_COL, B_COL, PAIR, KIND>(j, e, sl, blockIdx.x, s0, s1, s2, s3);
}

// A small backward pass's two products, dx on the first `first` workgroups and dw on the others:
// neither fills the device, and a launch of its own costs each about 5 us.
template <typename T, int BN, int WM, int WN, int S, int DB>
__global__ __launch_bounds__(256, 2) void k_dense_mm_two(DenseJob jx, DenseEpi ex, MmSlices sx, int first, DenseJob jw,
                                                         DenseEpi ew, MmSlices sw) {
  constexpr int STAGE = kMmStage<64, BN, 128>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  if ((int)blockIdx.x < first)
    mm_body<T, 64, BN, WM, WN, S, 128, DB, false, true, false, DENSE_STORE>(jx, ex, sx, blockIdx.x, s0, s1, s2, s3);
  else
    mm_body<T, 64, BN, WM, WN, S, 128, DB, true, true, false, DENSE_STORE>(jw, ew, sw, blockIdx.x - first, s0, s1, s2, s3);
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
    with_act<KIND>(j.e.act, [&](auto act) __attribute__((always_inline)) { mm_out8<T, KIND, act()>(j.e, z, m, n, j.N, a, b, bias, res); });
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
