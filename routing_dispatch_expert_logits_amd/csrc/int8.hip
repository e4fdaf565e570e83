// Products in 8-bit integers with a scale for each row and each output column, and the rows' codes.
//
//   scale = max |x| / 127 (fp32),  q = x / scale rounded to the nearest integer, ties to even,
//   y = row_scale col_scale sum q_x q_w
//
// The sums are whole numbers in 32 bits, so exact in any order, while the contraction is no longer than
// 2^17 (127^2 2^17 < 2^31).
#include "dense_tile.h"
#include "grouped_kernels.h"

namespace moe {

template <typename O, int BM, int BN, int WM, int WN, int S, int SB, bool PAIR, int KIND>
__global__ __launch_bounds__(WM* WN * 64, 2) void k_int8_mm(DenseJob j, DenseEpi e) {
  constexpr int STAGE = kMmStage<BM, BN, SB>;
  __shared__ __attribute__((aligned(1024))) uint16_t s0[STAGE], s1[STAGE], s2[STAGE], s3[S > 3 ? STAGE : 1];
  const MmWhere w = mm_where(blockIdx.x, ceil_div(j.M, BM), ceil_div(j.N, PAIR ? BN / 2 : BN), 1, 1);
  mm_body<int8_t, O, BM, BN, WM, WN, S, SB, 16, false, false, PAIR, KIND, true>(
      j, e, MmSlices{nullptr, 1, 1, 0}, w, MmPart{j.M, j.K, 0, 0, 0, 0, 0}, s0, s1, s2, s3);
}

template <typename O, int BM, int BN, int WM, int WN, int S, int SB = 128>
static void go(const DenseJob& j, const DenseEpi& e, hipStream_t st) {
  const int64_t items = (int64_t)ceil_div(j.M, BM) * ceil_div(j.N, j.pair ? BN / 2 : BN);
  const dim3 grid((unsigned)((items + 7) / 8 * 8)), block(WM * WN * 64);
  if (j.pair) k_int8_mm<O, BM, BN, WM, WN, S, SB, true, DENSE_GATED><<<grid, block, 0, st>>>(j, e);
  else k_int8_mm<O, BM, BN, WM, WN, S, SB, false, DENSE_LINEAR><<<grid, block, 0, st>>>(j, e);
}

// Tile by estimated time, from what a kernel takes per round of `at_once` workgroups: us per contraction step of 128
// bytes and besides, measured (MI355X).  8192 x 8192 x 8192 / 8192 x 2048 x 7168 with a residual / 2048 x 4096 x 4096 /
// 512 x 4096 x 4096 take 453 / 157 / 52 / 47 us on 256 x 256 (2.43 POP/s; the library's largest is 2.13), 532 / 177 / 39 / 33 on
// 256 x 128, 812 / 272 / 58 / 17 on 64 x 64.  All of it with bf16 outputs.  With fp32 ones the linear product's 256 x 256 tile
// holds 128 registers of residual ahead and spills 300, also where there is none: with the codes, 8192 x 2048 -> 7168 takes 210 us
// (with a residual 264) where no 256 x 256 tiles would take 190 (229), 8192 x 7168 -> 2048 182 (190) and 189 (200),
// 4096 x 4096 -> 4096 103 (114) and 104 (117), 8192 x 512 -> 2048 52 (56) and 51 (57).
struct Int8Tile {
  int bm, bn, at_once;
  double step, fixed;
};
constexpr Int8Tile kInt8Tiles[] = {{256, 256, 256, 1.7, 10.0}, {256, 128, 256, 1.0, 6.0}, {64, 64, 512, 0.42, 3.0}};

struct Int8Plan {
  int tile;   // of kInt8Tiles
  int cut;    // 256 x 256 tiles for this many output columns, and a launch of its own for the rest; 0: none
  double us;
};
static Int8Plan int8_plan(int M, int N, int K, bool pair, bool whole) {
  Int8Plan best{};
  const int steps = ceil_div(K, 128);
  for (int i = 0; i < 3; ++i) {
    const Int8Tile& c = kInt8Tiles[i];
    const int64_t items = (int64_t)ceil_div(M, c.bm) * ceil_div(N, pair ? c.bn / 2 : c.bn);
    const double us = (double)((items + c.at_once - 1) / c.at_once) * (steps * c.step + c.fixed);
    if (i == 0 || us < best.us) best = {i, 0, us};
  }
  // Whole rounds of 256 x 256 tiles, and smaller ones for the columns that would start another: 8192 x 2048 x 7168 has 896
  // such tiles, three and a half rounds.
  const Int8Tile& c = kInt8Tiles[0];
  const int on = pair ? c.bn / 2 : c.bn, tn = ceil_div(N, on);
  const int64_t column = ceil_div(M, c.bm), rounds = column * tn / c.at_once, n = rounds * c.at_once / column;
  if (!whole && rounds >= 1 && n >= 1 && n < tn) {
    const double us = rounds * (steps * c.step + c.fixed) + 3.0 + int8_plan(M, N - (int)n * on, K, pair, true).us;
    if (us < best.us) best = {0, (int)n * on, us};
  }
  return best;
}

template <typename O>
static void go(const DenseJob& j, const DenseEpi& e, int tile, hipStream_t st) {
  if (tile == 0) go<O, 256, 256, 2, 4, 4, 64>(j, e, st);
  else if (tile == 1) go<O, 256, 128, 4, 2, 3>(j, e, st);
  else go<O, 64, 64, 2, 2, 4>(j, e, st);
}

// Output columns from n on.
template <typename O>
static void from_column(DenseJob& j, DenseEpi& e, int n) {
  auto on = [&](auto* v) { return v ? static_cast<decltype(v)>(const_cast<O*>(static_cast<const O*>(v) + n)) : v; };
  j.N -= n;
  for (int z = 0; z < 2; ++z) {
    if (j.B[z][0]) j.B[z][0] = static_cast<const int8_t*>(j.B[z][0]) + n * j.ldb;
    if (e.col_scale[z]) e.col_scale[z] += n;
  }
  e.bias = on(e.bias);
  e.residual = on(e.residual);
  e.out[0] = on(e.out[0]);
}

hipError_t launch_int8(const DenseJob& j, const DenseEpi& e, bool out_bf16, hipStream_t st) {
  const Int8Plan p = int8_plan(j.M, j.N, j.K, j.pair, false);
  auto by_type = [&](auto* t) {
    using O = std::remove_pointer_t<decltype(t)>;
    DenseJob left = j, right = j;
    DenseEpi er = e;
    if (p.cut) left.N = p.cut;
    go<O>(left, e, p.tile, st);
    if (!p.cut) return;
    from_column<O>(right, er, p.cut);
    go<O>(right, er, int8_plan(right.M, right.N, right.K, right.pair, true).tile, st);
  };
  if (out_bf16) by_type(static_cast<uint16_t*>(nullptr));
  else by_type(static_cast<float*>(nullptr));
  return hipGetLastError();
}

// ---- codes of rows

// The largest magnitude's bits: for finite numbers their order is the magnitudes', infinities and NaN are above.
__device__ __forceinline__ uint32_t magnitude(float v) { return __float_as_uint(v) & 0x7fffffffu; }

// A row's scale and what turns its elements into codes: x / s as x up inv, with up a power of two that keeps
// the smallest scales' reciprocals finite (s up is exact, as x up is: |x| <= 127.5 s or it is clamped).
struct Int8Scale {
  float scale, up, s, inv;
  __device__ __forceinline__ explicit Int8Scale(uint32_t most) {
    const bool finite = most < 0x7f800000u;
    scale = finite ? __uint_as_float(most) / 127.f : __builtin_nanf("");
    up = scale < 0x1p-100f ? 0x1p100f : 1.f;
    s = scale * up;
    inv = scale > 0.f ? 1.f / s : 0.f;   // 0 for rows of zeros and for rows that are not finite: codes 0
  }
  // rint(x / scale) from the exact quotient: n is off only where x inv is within its rounding (2^-16)
  // of a tie, and the remainder x - n s, which an fma has exactly, says on which side of it x / s is.
  __device__ __forceinline__ int code(float x) const {
    if (inv == 0.f) return 0;
    x *= up;
    float n = rintf(x * inv);
    const float r = fmaf(-n, s, x), half = 0.5f * s;
    if (fabsf(r) >= half) {
      const bool odd = (int)n & 1;
      if (fabsf(r) > half || odd) n += r > 0.f ? 1.f : -1.f;
    }
    return (int)fminf(fmaxf(n, -127.f), 127.f);
  }
};

__device__ __forceinline__ uint2 codes8(const Int8Scale& s, const float* f) {
  uint32_t c[2] = {0, 0};
#pragma unroll
  for (int i = 0; i < 8; ++i) c[i >> 2] |= (uint32_t)(s.code(f[i]) & 0xff) << (8 * (i & 3));
  return make_uint2(c[0], c[1]);
}

// Bound by memory.  A row of up to 16384 elements stays in registers between its largest magnitude and its codes: NV
// pieces of eight elements per lane of one wave (WAVES 1, four rows a workgroup) or of four.
template <typename ST, int WAVES, int NV>
__global__ __launch_bounds__(256) void k_quantize_int8(const ST* __restrict__ src, int64_t rows, int cols, int64_t ld,
                                                       int8_t* __restrict__ q, float* __restrict__ scale) {
  constexpr int LANES = 64 * WAVES, ROWS = 4 / WAVES;
  __shared__ uint32_t part[2][4];
  const int at = threadIdx.x % LANES, n8 = (int)(ld / 8);
  int turn = 0;
  for (int64_t r = (int64_t)blockIdx.x * ROWS + threadIdx.x / LANES; r < rows; r += (int64_t)gridDim.x * ROWS, turn ^= 1) {
    const ST* x = src + r * cols;
    Raw8<ST> v[NV];
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const int i = at + h * LANES;
      v[h].load(x + 8 * min(i, n8 - 1), i < n8 ? cols - 8 * i : 0);
    }
    uint32_t most = 0;
#pragma unroll
    for (int h = 0; h < NV; ++h)
#pragma unroll
      for (int k = 0; k < 8; ++k) most = max(most, magnitude(v[h].get(k)));
    most = wave_max_u32(most);
    if constexpr (WAVES > 1) {
      if ((threadIdx.x & 63) == 0) part[turn][threadIdx.x >> 6] = most;
      __syncthreads();   // the next row's maxima go to the other four places
      most = max(max(part[turn][0], part[turn][1]), max(part[turn][2], part[turn][3]));
    }
    const Int8Scale s(most);
    if (at == 0) scale[r] = s.scale;
#pragma unroll
    for (int h = 0; h < NV; ++h) {
      const int i = at + h * LANES;
      if (i >= n8) continue;
      float f[8];
#pragma unroll
      for (int k = 0; k < 8; ++k) f[k] = v[h].get(k);
      reinterpret_cast<uint2*>(q + r * ld)[i] = codes8(s, f);
    }
  }
}

// Longer rows are read twice.
template <typename ST>
__global__ __launch_bounds__(256) void k_quantize_int8_long(const ST* __restrict__ src, int64_t rows, int cols, int64_t ld,
                                                            int8_t* __restrict__ q, float* __restrict__ scale) {
  __shared__ uint32_t part[4];
  const int n8 = (int)(ld / 8);
  for (int64_t r = blockIdx.x; r < rows; r += gridDim.x) {
    const ST* x = src + r * cols;
    uint32_t most = 0;
    for (int i = threadIdx.x; i < n8; i += 256) {
      float f[8];
      load8(x + 8 * i, cols - 8 * i, f);
#pragma unroll
      for (int k = 0; k < 8; ++k) most = max(most, magnitude(f[k]));
    }
    most = wave_max_u32(most);
    if ((threadIdx.x & 63) == 0) part[threadIdx.x >> 6] = most;
    __syncthreads();
    const Int8Scale s(max(max(part[0], part[1]), max(part[2], part[3])));
    __syncthreads();
    if (threadIdx.x == 0) scale[r] = s.scale;
    for (int i = threadIdx.x; i < n8; i += 256) {
      float f[8];
      load8(x + 8 * i, cols - 8 * i, f);
      reinterpret_cast<uint2*>(q + r * ld)[i] = codes8(s, f);
    }
  }
}

template <typename ST>
static void quantize(const ST* src, int64_t rows, int cols, int64_t ld, int8_t* q, float* scale, hipStream_t st) {
  const int n8 = (int)(ld / 8);
  auto go = [&](auto kernel, int per) {
    const int64_t want = (rows + per - 1) / per;
    kernel<<<(unsigned)(want < (1 << 20) ? want : 1 << 20), 256, 0, st>>>(src, rows, cols, ld, q, scale);
  };
  if (n8 <= 64) go(k_quantize_int8<ST, 1, 1>, 4);
  else if (n8 <= 128) go(k_quantize_int8<ST, 1, 2>, 4);
  else if (n8 <= 256) go(k_quantize_int8<ST, 1, 4>, 4);
  else if (n8 <= 512) go(k_quantize_int8<ST, 4, 2>, 1);
  else if (n8 <= 1024) go(k_quantize_int8<ST, 4, 4>, 1);
  else if (n8 <= 2048) go(k_quantize_int8<ST, 4, 8>, 1);
  else go(k_quantize_int8_long<ST>, 1);
}

hipError_t launch_quantize_int8(const void* src, bool bf16, int64_t rows, int cols, int64_t ld, int8_t* q, float* scale,
                                hipStream_t st) {
  if (bf16) quantize(static_cast<const uint16_t*>(src), rows, cols, ld, q, scale, st);
  else quantize(static_cast<const float*>(src), rows, cols, ld, q, scale, st);
  return hipGetLastError();
}

}  // namespace moe
