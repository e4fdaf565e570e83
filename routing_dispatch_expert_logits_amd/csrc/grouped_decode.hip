// Forward products of few rows (decoding steps), grouped by expert, and in 8-bit integers also dense:
// each expert's weights are read once, straight from memory into matrix-core operands, with no table
// of tiles and no launch before the product's own.
#include "dense_device.h"
#include "grouped_kernels.h"

namespace moe {

typedef int i32x4 __attribute__((ext_vector_type(4)));

// Sixteen bytes of one row per lane: lane l holds row l % 16, the (l / 16)-th 16 bytes of a chunk of 64.  One
// v_mfma_f32_16x16x32_bf16 or v_mfma_i32_16x16x64_i8 per chunk; fp32: four v_mfma_f32_16x16x4_f32, the i-th
// taking element i of every lane's four (the contraction's order is the same on both sides).
template <typename T>
struct Bytes16 {
  static constexpr int PER = 16 / sizeof(T), K = 4 * PER;
  u32x4 v;
  // The first n elements, zeros behind (rows of codes are whole 16-byte chunks).
  __device__ __forceinline__ void load(const T* p, int n) {
    v = u32x4{0, 0, 0, 0};
    if (sizeof(T) == 1 ? n > 0 : n >= PER) {
      using Vec = std::conditional_t<sizeof(T) == 1, u32x4, u32x4_of2>;
      v = *reinterpret_cast<const Vec*>(p);
      return;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        else if constexpr (sizeof(T) == 4) v[i] = __float_as_uint(p[i]);
      }
  }
};

// A strip is 16 of an expert's weight rows (with PAIR 8 of each projection).  A workgroup of 8 waves has 8 / SPLIT
// strips of one expert that has rows; SPLIT waves share a strip's contraction, U chunks of loads in flight each,
// and their sums meet in LDS in wave order.  Rows beyond an expert's first 16 meet the same weights again.
// blockIdx.y: the expert, or, where there are fewer rows than experts, the row that an expert's rows begin with.
template <typename T, typename O, int KIND, int SPLIT, int U>
__global__ __launch_bounds__(512) void k_grouped_decode(DenseJob j, DenseEpi e, Groups groups, int64_t w_stride) {
  using C = Bytes16<T>;
  constexpr bool PAIR = KIND == DENSE_GATED, INT8 = sizeof(T) == 1;
  using Acc = std::conditional_t<INT8, i32x4, f32x4>;
  using A = std::conditional_t<INT8, int, float>;
  constexpr int W = 8, ON = PAIR ? 8 : 16, STRIPS = W / SPLIT, WIDE = STRIPS * ON;
  __shared__ A s[W][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  int expert = 0, lo = 0, hi = j.M;
  if (groups.E) {
    expert = blockIdx.y;
    if (groups.E > (int)gridDim.y) {
      // whose rows begin with this one: a look at all experts at once, as the row counts are not known before
      const int row = blockIdx.y;
      uint64_t found = 0;
      for (int i0 = 0; i0 < groups.E && !found; i0 += 64) {
        const int i = min(i0 + lane, groups.E - 1);
        const int2 r = group_rows(groups, i);
        found = __ballot(i == i0 + lane && r.x == row && r.y > row);
        if (found) {
          const int at = __builtin_ctzll(found);
          expert = i0 + at;
          lo = __builtin_amdgcn_readlane(r.x, at);
          hi = __builtin_amdgcn_readlane(r.y, at);
        }
      }
      if (!found) return;
    } else {
      const int2 r = group_rows(groups, expert);
      lo = r.x;
      hi = r.y;
      if (hi == lo) return;
    }
  }
  const int part = wave % SPLIT, first = (int)blockIdx.x * WIDE, n0 = first + wave / SPLIT * ON;  // columns of the workgroup, of this wave
  const T* w = static_cast<const T*>(PAIR && r >= 8 ? j.B[1][0] : j.B[0][0]) + expert * w_stride +
               (int64_t)min(n0 + (r & (ON - 1)), j.N - 1) * j.ldb + g * C::PER;
  const int nc = ceil_div(j.K, C::K), per = ceil_div(nc, SPLIT);
  const int c0 = part * per, c1 = min(nc, c0 + per);
  for (int b = lo; b < hi; b += 16) {
    const T* x = static_cast<const T*>(j.A[0][0]) + (int64_t)min(b + r, hi - 1) * j.lda + g * C::PER;
    Acc acc = {};
    for (int c = c0; c < c1; c += U) {
      C cw[U], cx[U];
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + i < c1) cw[i].load(w + (int64_t)(c + i) * C::K, j.K - (c + i) * C::K - g * C::PER);
#pragma unroll
      for (int i = 0; i < U; ++i)
        if (c + i < c1) cx[i].load(x + (int64_t)(c + i) * C::K, j.K - (c + i) * C::K - g * C::PER);
#pragma unroll
      for (int i = 0; i < U; ++i) {
        if (c + i >= c1) continue;
        if constexpr (INT8) {
          acc = __builtin_amdgcn_mfma_i32_16x16x64_i8(__builtin_bit_cast(i32x4, cw[i].v), __builtin_bit_cast(i32x4, cx[i].v), acc, 0, 0, 0);
        } else if constexpr (sizeof(T) == 2) {
          acc = __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(cw[i].v), as_bf16x8(cx[i].v), acc, 0, 0, 0);
        } else {
#pragma unroll
          for (int k = 0; k < 4; ++k)
            acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(cw[i].v[k]), __uint_as_float(cx[i].v[k]), acc, 0, 0, 0);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) s[wave][r][4 * g + i] = acc[i];  // [row][weight row]
    __syncthreads();
    for (int k = threadIdx.x; k < 16 * WIDE; k += 512) {
      const int t = k / WIDE, col = k % WIDE, n = first + col, row = b + t;
      if (row >= hi || n >= j.N) continue;
      const int q0 = col / ON * SPLIT, i = col % ON;
      A sum[2] = {};
#pragma unroll
      for (int q = q0; q < q0 + SPLIT; ++q) {
        sum[0] += s[q][t][i];
        if (PAIR) sum[1] += s[q][t][8 + i];
      }
      float v[2] = {(float)sum[0], (float)sum[1]};
      if constexpr (INT8) {
        const int64_t at = (int64_t)expert * j.N + n;
        const float by = row_scale_by(e.row_scale[row]), up = row_scale_up(e.row_scale[row]);
        v[0] = v[0] * by * e.col_scale[0][at] * up;
        if (PAIR) v[1] = v[1] * by * e.col_scale[1][at] * up;
      }
      constexpr bool FAST = sizeof(O) == 2;
      const int64_t idx = (int64_t)row * e.ldo + n;
      float y = v[0];
      if constexpr (PAIR) {
        if (e.save[0]) {
          store1(static_cast<O*>(e.save[0]) + idx, v[0]);
          store1(static_cast<O*>(e.save[1]) + idx, v[1]);
        }
        y = act_value<FAST>(v[0], e.act) * v[1];
      } else if constexpr (KIND == DENSE_LINEAR) {
        const float a = e.bias ? v[0] + load1(static_cast<const O*>(e.bias) + n) : v[0];
        y = act_value<FAST>(a, e.act);
        if (e.residual) y += load1(static_cast<const O*>(e.residual) + idx);
      }
      store1(static_cast<O*>(e.out[0]) + idx, y);
    }
    __syncthreads();
  }
}

template <typename T, typename O, int SPLIT>
static void go(const DenseJob& j, const DenseEpi& e, const Groups& g, int64_t w_stride, int strips, int experts, hipStream_t st) {
  // Chunks in flight.  16 take twice the registers, for two waves a SIMD (16 and 8: 8 rows in integers, 8192 -> 8192, 18.4 and
  // 15.9 us, 7168 -> 2048 8.5 and 8.8; 8 bf16 rows of 4 experts, 4096 -> 2048, 16.1 and 14.0; 8 fp32 rows of 2, 7168 -> 4096,
  // 59.8 and 52.6).
  constexpr int U = 8;
  const dim3 grid(ceil_div(strips, 8 / SPLIT), experts);
  if (j.pair) k_grouped_decode<T, O, DENSE_GATED, SPLIT, U><<<grid, 512, 0, st>>>(j, e, g, w_stride);
  else if (e.kind == DENSE_STORE) k_grouped_decode<T, O, DENSE_STORE, SPLIT, U><<<grid, 512, 0, st>>>(j, e, g, w_stride);
  else if constexpr (sizeof(T) == 1) k_grouped_decode<T, O, DENSE_LINEAR, SPLIT, U><<<grid, 512, 0, st>>>(j, e, g, w_stride);
}

// Waves that share a strip: as many as fill the device (4096 waves), while each keeps 4 chunks, half of its loads in
// flight.  2048 -> 7168 in integers, one row by 8 experts: 1 / 2 / 4 waves a strip 25.3 / 26.4 / 29.5 us; one
// row by one weight 4 / 8 waves 8.0 / 7.6.
template <typename T, typename O>
static void go(const DenseJob& j, const DenseEpi& e, const Groups& g, int64_t w_stride, hipStream_t st) {
  const int strips = ceil_div(j.N, j.pair ? 8 : 16), experts = g.E ? (g.R < g.E ? g.R : g.E) : 1;
  const int chunks = ceil_div(j.K, Bytes16<T>::K);
  int split = 1;
  while (split < 8 && (int64_t)strips * experts * split < 4096 && chunks / (2 * split) >= 4) split *= 2;
  if (split == 1) go<T, O, 1>(j, e, g, w_stride, strips, experts, st);
  else if (split == 2) go<T, O, 2>(j, e, g, w_stride, strips, experts, st);
  else if (split == 4) go<T, O, 4>(j, e, g, w_stride, strips, experts, st);
  else go<T, O, 8>(j, e, g, w_stride, strips, experts, st);
}

hipError_t launch_grouped_decode(const DenseJob& j, const DenseEpi& e, GroupedType t, bool out_bf16, const Groups& g,
                                 int64_t w_stride, hipStream_t st) {
  if (t == GROUPED_F32) go<float, float>(j, e, g, w_stride, st);
  else if (t == GROUPED_BF16) go<uint16_t, uint16_t>(j, e, g, w_stride, st);
  else if (out_bf16) go<int8_t, uint16_t>(j, e, g, w_stride, st);
  else go<int8_t, float>(j, e, g, w_stride, st);
  return hipGetLastError();
}

}  // namespace moe
