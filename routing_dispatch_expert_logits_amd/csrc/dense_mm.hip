// bf16 dense products on v_mfma_f32_16x16x32_bf16, fp32 accumulate (the layouts are described
// in dense_kernels.h).
#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

typedef short s16x4 __attribute__((ext_vector_type(4)));
typedef __attribute__((address_space(3))) void* lds_dst;
typedef __attribute__((address_space(3))) s16x4* lds_s16x4;

constexpr int kMBK = 64;                       // contraction step
constexpr uint32_t kOutOfRange = 0x80000000u;  // a lane offset no buffer of ours reaches: reads 0

__device__ __forceinline__ int uniform(int v) { return __builtin_amdgcn_readfirstlane(v); }
__device__ __forceinline__ const char* uniform(const char* p) {
  const uint64_t a = reinterpret_cast<uint64_t>(p);
  return reinterpret_cast<const char*>(((uint64_t)(uint32_t)uniform((int)(a >> 32)) << 32) | (uint32_t)uniform((int)a));
}

// A tile of R rows (m or n) by 64 contraction elements in LDS, filled by 16-byte buffer loads
// straight into LDS (1 KB per instruction, lane i to byte 16 i) and read as MFMA operands: lane
// l holds row l % 16, contraction elements 8 (l / 16) .. + 8 of each 32.
//
// Row operands (contraction along memory): LDS row r is 128 bytes, its 16-byte chunk c sits at
// slot c ^ (r & 7), so the 16 rows one ds_read_b128 touches at one chunk index cover all banks.
//
// Column operands (contraction across memory): LDS row k holds R elements, and
// ds_read_b64_tr_b16 turns 4 x 16 blocks into operand order: of each 16 lanes, lane i reads
// 8 bytes of row i / 4 at 4 (i % 4) and receives element i of rows 0..3.  The 32-byte unit u
// of row k sits at u ^ f(k) with f(k) = (k & 3) | (k >> 1 & 4), which spreads the 16 rows one
// instruction touches over all banks.
template <int R, bool COL>
struct MmTile {
  static constexpr int ELEMS = R * kMBK;
  static constexpr int INSTR = R / 8;           // fill instructions
  static constexpr int CPR = R / 8;             // column operand: 16-byte chunks per LDS row
  static __device__ __forceinline__ int f(int k) { return ((k & 3) | ((k >> 1) & 4)) & (R / 16 - 1); }

  // Byte offset of lane's 16 bytes of fill instruction q, from the tile's first row at
  // contraction 0 (row operand; rows >= valid are out of range) or from the tile's first
  // element of the step's first contraction row (column operand).
  static __device__ __forceinline__ uint32_t src(int q, int lane, int64_t ld, int valid) {
    if constexpr (COL) {
      const int k = q * (64 / CPR) + lane / CPR, s = lane % CPR;
      const int chunk = (((s >> 1) ^ f(k)) << 1) | (s & 1);
      return (uint32_t)(k * ld * 2 + chunk * 16);
    } else {
      const int r = q * 8 + (lane >> 3);
      return r < valid ? (uint32_t)(r * ld * 2 + (((lane & 7) ^ (lane >> 3)) << 4)) : kOutOfRange;
    }
  }

  // Operand of rows row0 + 16 i .. + 16 (row0 a multiple of 16), contraction half h.
  static __device__ __forceinline__ bf16x8 read(const uint16_t* t, int row0, int i, int h, int lane) {
    if constexpr (COL) {
      const int g = lane >> 4, j = (lane >> 2) & 3;
      const int k = 32 * h + 8 * g + j, u = ((row0 >> 4) + i) ^ f(8 * g + j);
      const uint16_t* p = t + k * R + u * 16 + (lane & 3) * 4;
      s16x4 v[2];
      v[0] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)p);
      v[1] = __builtin_amdgcn_ds_read_tr16_b64_v4i16((lds_s16x4)(p + 4 * R));
      return __builtin_bit_cast(bf16x8, v);
    } else {
      const int r = row0 + (lane & 15);
      return as_bf16x8(*reinterpret_cast<const u32x4*>(t + (r + 16 * i) * kMBK +
                                                       (((4 * h + (lane >> 4)) ^ (lane & 7)) << 3)));
    }
  }
};

// Four neighbouring output columns n .. n + 3 of row m.
template <int KIND>
__device__ __forceinline__ void mm_out4(const DenseEpi& e, int z, int m, int n, int N, f32x4 v0, f32x4 v1) {
  const int64_t idx = (int64_t)m * N + n;
  const bool vec = (N & 3) == 0;
  auto put = [&](void* p, const float* v, bool f32) {
    if (f32) {
      if (vec) *reinterpret_cast<f32x4*>(static_cast<float*>(p) + idx) = f32x4{v[0], v[1], v[2], v[3]};
      else for (int i = 0; i < 4; ++i) { if (n + i < N) static_cast<float*>(p)[idx + i] = v[i]; }
    } else {
      uint16_t* o = static_cast<uint16_t*>(p) + idx;
      if (vec)
        *reinterpret_cast<uint2*>(o) = make_uint2(f32_to_bf16(v[0]) | (uint32_t)f32_to_bf16(v[1]) << 16,
                                                  f32_to_bf16(v[2]) | (uint32_t)f32_to_bf16(v[3]) << 16);
      else for (int i = 0; i < 4; ++i) { if (n + i < N) o[i] = f32_to_bf16(v[i]); }
    }
  };
  auto get = [&](const void* p, int64_t at, float* v) {
    const uint16_t* o = static_cast<const uint16_t*>(p) + at;
    if (vec) {
      const uint2 w = *reinterpret_cast<const uint2*>(o);
      v[0] = __uint_as_float(w.x << 16); v[1] = __uint_as_float(w.x & 0xffff0000u);
      v[2] = __uint_as_float(w.y << 16); v[3] = __uint_as_float(w.y & 0xffff0000u);
    } else {
      for (int i = 0; i < 4; ++i) v[i] = n + i < N ? bf16_to_f32(o[i]) : 0.f;
    }
  };
  float a[4] = {v0[0], v0[1], v0[2], v0[3]}, y[4];
  if constexpr (KIND == DENSE_STORE) {
    put(e.out[z], a, e.out_f32);
  } else if constexpr (KIND == DENSE_LINEAR) {
    if (e.bias) {
      get(e.bias, n, y);
      for (int i = 0; i < 4; ++i) a[i] += y[i];
    }
    if (e.save[0]) put(e.save[0], a, false);
    for (int i = 0; i < 4; ++i) y[i] = act_value<true>(a[i], e.act);
    if (e.residual) {
      get(e.residual, idx, a);
      for (int i = 0; i < 4; ++i) y[i] += a[i];
    }
    put(e.out[0], y, false);
  } else {
    const float b[4] = {v1[0], v1[1], v1[2], v1[3]};
    if (e.save[0]) {
      put(e.save[0], a, false);
      put(e.save[1], b, false);
    }
    for (int i = 0; i < 4; ++i) y[i] = act_value<true>(a[i], e.act) * b[i];
    put(e.out[0], y, false);
  }
}

// Tile (m-tile, n-tile, batch) of a workgroup: tiles are dealt to the 8 XCDs in contiguous
// chunks, within which groups of 8 m-tiles run down their n-tiles, so that the tiles an XCD
// works on at a time share rows and columns in its L2.
struct MmWhere { int mt, nt, z; bool ok; };
__device__ __forceinline__ MmWhere mm_where(int tm, int tn, int batch) {
  const int total = tm * tn * batch, per = ceil_div(total, 8);
  const int slot = blockIdx.x >> 3, L = (blockIdx.x & 7) * per + slot;
  MmWhere w{0, 0, 0, slot < per && L < total};
  w.z = L / (tm * tn);
  const int t = L - w.z * (tm * tn), grp = t / (8 * tn), first = grp * 8, r = t - grp * (8 * tn);
  const int gsz = min(8, tm - first);
  w.nt = r / gsz;
  w.mt = first + (r - w.nt * gsz);
  return w;
}

// BM x BN tile by WM x WN waves, two LDS stages: the next step's loads fill one while the
// other is multiplied.  With PAIR the tile's first BN / 2 rows of B come from the first weight
// and the rest from the second, for the same BN / 2 output columns.
template <int BM, int BN, int WM, int WN, bool A_COL, bool B_COL, bool PAIR, int KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_dense_mm(DenseJob j, DenseEpi e) {
  using TA = MmTile<BM, A_COL>;
  using TB = MmTile<BN, B_COL>;
  constexpr int W = WM * WN, TM = BM / WM, TN = BN / WN, FM = TM / 16, FN = TN / 16;
  constexpr int QA = TA::INSTR / W, QB = TB::INSTR / W;
  constexpr int ON = PAIR ? BN / 2 : BN;   // output columns of a tile
  static_assert(QA >= 1 && QB >= 1 && !(PAIR && (B_COL || FN % 2)), "tile");
  __shared__ __attribute__((aligned(1024))) uint16_t sA0[TA::ELEMS], sB0[TB::ELEMS], sA1[TA::ELEMS], sB1[TB::ELEMS];

  const MmWhere w = mm_where(ceil_div(j.M, BM), ceil_div(j.N, ON), j.batch);
  if (!w.ok) return;
  const int m0 = uniform(w.mt * BM), n0 = uniform(w.nt * ON), z = uniform(w.z);
  const int lane = threadIdx.x & 63, wave = __builtin_amdgcn_readfirstlane(threadIdx.x >> 6);
  const int wm = wave / WN, wn = wave % WN;
  const int nk = ceil_div(j.K, kMBK), steps = nk * j.segs;

  // fill: this wave's instructions are wave * Q .. + Q of each tile
  uint32_t va[QA], vb[QB];
#pragma unroll
  for (int q = 0; q < QA; ++q) va[q] = TA::src(wave * QA + q, lane, j.lda, j.M - m0);
  const bool second = PAIR && wave >= W / 2;
#pragma unroll
  for (int q = 0; q < QB; ++q)
    vb[q] = TB::src((PAIR ? wave % (W / 2) : wave) * QB + q, lane, j.ldb, j.N - n0);
  const int kchunk = ((lane & 7) ^ (lane >> 3)) * 8;  // row operands: this lane's first element in a step
  // of the next step to load: where the tile starts and how many bytes from there are the
  // operand's (whole rows of it, none past its last one)
  const char *pa, *pb;
  int na, nb, left = 0, seg = 0;                      // left: contraction elements to load of this segment
  auto segment = [&]() __attribute__((always_inline)) {
    const void* b = PAIR ? (second ? j.B[1][0] : j.B[0][0]) : j.B[z][seg];
    pa = uniform(static_cast<const char*>(j.A[z][seg]) + (A_COL ? (int64_t)m0 : (int64_t)m0 * j.lda) * 2);
    pb = uniform(static_cast<const char*>(b) + (B_COL ? (int64_t)n0 : (int64_t)n0 * j.ldb) * 2);
    na = min(BM, j.M - m0) * (int)j.lda * 2;
    nb = min(ON, j.N - n0) * (int)j.ldb * 2;
    left = j.K;
  };
  auto fill = [&](uint16_t* la, uint16_t* lb) __attribute__((always_inline)) {
    if (left <= 0) {
      ++seg;
      segment();
    }
    const int rows = min(kMBK, left);
    auto one = [&](const char* p, int n, bool col, const uint32_t* v, int Q, uint16_t* dst)
        __attribute__((always_inline)) {
      const __amdgpu_buffer_rsrc_t r = __builtin_amdgcn_make_buffer_rsrc(
          const_cast<char*>(p), 0, __builtin_amdgcn_readfirstlane(n), 0x00020000);
      if (col || rows == kMBK) {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_dst)(dst + q * 512), 16, v[q], 0, 0, 0);
      } else {
#pragma unroll
        for (int q = 0; q < Q; ++q)
          __builtin_amdgcn_raw_ptr_buffer_load_lds(r, (lds_dst)(dst + q * 512), 16,
                                                   kchunk < rows ? v[q] : kOutOfRange, 0, 0, 0);
      }
    };
    one(pa, A_COL ? (rows * (int)j.lda - m0) * 2 : na, A_COL, va, QA, la + wave * QA * 512);
    one(pb, B_COL ? (rows * (int)j.ldb - n0) * 2 : nb, B_COL, vb, QB, lb + wave * QB * 512);
    left -= kMBK;
    pa += A_COL ? (int64_t)kMBK * j.lda * 2 : kMBK * 2;
    pb += B_COL ? (int64_t)kMBK * j.ldb * 2 : kMBK * 2;
    na -= kMBK * 2;
    nb -= kMBK * 2;
  };

  f32x4 acc[FM][FN];
#pragma unroll
  for (int a = 0; a < FM; ++a)
#pragma unroll
    for (int b = 0; b < FN; ++b) acc[a][b] = f32x4{0.f, 0.f, 0.f, 0.f};
  auto multiply = [&](const uint16_t* la, const uint16_t* lb) __attribute__((always_inline)) {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      bf16x8 fb[FN];
#pragma unroll
      for (int b = 0; b < FN; ++b) {
        // with PAIR, the wave's first half of columns in the first weight's rows, then the second's
        const int row0 = PAIR ? wn * (TN / 2) + (b / (FN / 2)) * ON : wn * TN;
        fb[b] = TB::read(lb, row0, PAIR ? b % (FN / 2) : b, h, lane);
      }
#pragma unroll
      for (int a = 0; a < FM; ++a) {
        const bf16x8 fa = TA::read(la, wm * TM, a, h, lane);
#pragma unroll
        for (int b = 0; b < FN; ++b)
          acc[a][b] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(fb[b], fa, acc[a][b], 0, 0, 0);
      }
    }
  };
  // every load into LDS of this wave has landed and every read from it is done; then all waves
  auto hand_over = [&]() __attribute__((always_inline)) {
    __builtin_amdgcn_s_waitcnt(0x0070);  // vmcnt(0) lgkmcnt(0)
    asm volatile("" ::: "memory");
    __builtin_amdgcn_s_barrier();
    asm volatile("" ::: "memory");
  };

  segment();
  fill(sA0, sB0);
  hand_over();
  for (int s = 0; s < steps; s += 2) {
    if (s + 1 < steps) fill(sA1, sB1);
    multiply(sA0, sB0);
    hand_over();
    if (s + 1 < steps) {
      if (s + 2 < steps) fill(sA0, sB0);
      multiply(sA1, sB1);
      hand_over();
    }
  }

#pragma unroll
  for (int a = 0; a < FM; ++a) {
    const int m = m0 + wm * TM + 16 * a + (lane & 15);
#pragma unroll
    for (int b = 0; b < (PAIR ? FN / 2 : FN); ++b) {
      const int n = n0 + wn * (PAIR ? TN / 2 : TN) + 16 * b + 4 * (lane >> 4);
      if (m < j.M && n < j.N) mm_out4<KIND>(e, z, m, n, j.N, acc[a][b], acc[a][PAIR ? b + FN / 2 : b]);
    }
  }
}

template <int BM, int BN, int WM, int WN>
static void mm_go(const DenseJob& j, const DenseEpi& e, hipStream_t st) {
  const int64_t tiles = (int64_t)ceil_div(j.M, BM) * ceil_div(j.N, j.pair ? BN / 2 : BN) * j.batch;
  const dim3 grid((unsigned)((tiles + 7) / 8 * 8)), block(WM * WN * 64);
  if (j.pair) k_dense_mm<BM, BN, WM, WN, false, false, true, DENSE_GATED><<<grid, block, 0, st>>>(j, e);
  else if (e.kind == DENSE_LINEAR) k_dense_mm<BM, BN, WM, WN, false, false, false, DENSE_LINEAR><<<grid, block, 0, st>>>(j, e);
  else if (!j.a_col) k_dense_mm<BM, BN, WM, WN, false, true, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e);
  else k_dense_mm<BM, BN, WM, WN, true, true, false, DENSE_STORE><<<grid, block, 0, st>>>(j, e);
}

hipError_t launch_dense_mm(const DenseJob& j, const DenseEpi& e, hipStream_t st) {
  mm_go<256, 256, 2, 4>(j, e, st);
  return hipGetLastError();
}

}  // namespace moe
