// Dense forward products of up to 16 rows (decoding steps): the weights are read once, straight
// from memory into matrix-core operands, which bounds them.  Measured (MI355X, bf16): 8 rows by
// two 2048 x 7168 weights 12.9 us, 4.6 TB/s; 1 row by one of 7168 x 2048 8.1 us, 3.6 TB/s with
// its launch.
#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

// Sixteen bytes of one row per lane: lane l holds row l % 16, elements (16 / size) (l / 16) ..
// of a chunk of 64 / size elements.  bf16: one v_mfma_f32_16x16x32_bf16 per chunk; fp32: four
// v_mfma_f32_16x16x4_f32, the i-th taking element i of every lane's four (the contraction's
// order is the same on both sides).
template <typename T>
struct Chunk {
  static constexpr int PER = 16 / sizeof(T), K = 4 * PER;
  u32x4 v;
  __device__ __forceinline__ void load(const T* p) {
    if constexpr (sizeof(T) == 2) {
      const Bytes16of2 b = *reinterpret_cast<const Bytes16of2*>(p);
      v = u32x4{b.v[0], b.v[1], b.v[2], b.v[3]};
    } else {
      const Bytes16of4 b = *reinterpret_cast<const Bytes16of4*>(p);
      v = u32x4{b.v[0], b.v[1], b.v[2], b.v[3]};
    }
  }
  __device__ __forceinline__ void load(const T* p, int n) {  // the first n elements, zeros behind
    if (n >= PER) return load(p);
    v = u32x4{0, 0, 0, 0};
#pragma unroll
    for (int i = 0; i < PER; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        else v[i] = __float_as_uint(p[i]);
      }
  }
};
template <typename T>
__device__ __forceinline__ f32x4 mfma_chunk(const Chunk<T>& w, const Chunk<T>& x, f32x4 acc) {
  if constexpr (sizeof(T) == 2) return __builtin_amdgcn_mfma_f32_16x16x32_bf16(as_bf16x8(w.v), as_bf16x8(x.v), acc, 0, 0, 0);
#pragma unroll
  for (int i = 0; i < 4; ++i)
    acc = __builtin_amdgcn_mfma_f32_16x16x4f32(__uint_as_float(w.v[i]), __uint_as_float(x.v[i]), acc, 0, 0, 0);
  return acc;
}

// One workgroup per 16 weight rows (with PAIR 8 of each projection, so that a narrow gated
// product still spreads over the CUs); its 8 waves take an eighth of the contraction each, 8
// chunks of loads in flight per wave, and their sums meet in LDS in wave order.
template <typename T, bool PAIR>
__global__ __launch_bounds__(512) void k_dense_decode(DenseJob j, DenseEpi e) {
  using C = Chunk<T>;
  constexpr int W = 8, U = 8, ON = PAIR ? 8 : 16;
  __shared__ float s[W][16][17];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6, r = lane & 15, g = lane >> 4;
  const int n0 = (int)blockIdx.x * ON;
  const T* w = static_cast<const T*>(PAIR && r >= 8 ? j.B[1][0] : j.B[0][0]) +
               (int64_t)min(n0 + (r & (ON - 1)), j.N - 1) * j.ldb + g * C::PER;
  const T* x = static_cast<const T*>(j.A[0][0]) + (int64_t)min(r, j.M - 1) * j.lda + g * C::PER;
  const int nc = ceil_div(j.K, C::K), per = ceil_div(nc, W);
  const int c1 = min(nc, (wave + 1) * per);
  int c = wave * per;
  f32x4 acc = {0.f, 0.f, 0.f, 0.f};
  for (; c + U <= c1 && (c + U) * C::K <= j.K; c += U) {
    C cw[U], cx[U];
#pragma unroll
    for (int i = 0; i < U; ++i) cw[i].load(w + (c + i) * C::K);
#pragma unroll
    for (int i = 0; i < U; ++i) cx[i].load(x + (c + i) * C::K);
#pragma unroll
    for (int i = 0; i < U; ++i) acc = mfma_chunk<T>(cw[i], cx[i], acc);
  }
  for (; c < c1; ++c) {
    C cw, cx;
    const int left = j.K - c * C::K - g * C::PER;
    cw.load(w + c * C::K, left);
    cx.load(x + c * C::K, left);
    acc = mfma_chunk<T>(cw, cx, acc);
  }
#pragma unroll
  for (int i = 0; i < 4; ++i) s[wave][r][4 * g + i] = acc[i];  // [token][weight row]
  __syncthreads();
  const int t = threadIdx.x / ON, i = threadIdx.x % ON, n = n0 + i;
  if (t >= j.M || n >= j.N || t >= 16) return;
  float v[2] = {0.f, 0.f};
#pragma unroll
  for (int q = 0; q < W; ++q) {
    v[0] += s[q][t][i];
    if (PAIR) v[1] += s[q][t][8 + i];
  }
  constexpr bool FAST = sizeof(T) == 2;
  const int64_t idx = (int64_t)t * j.N + n;
  float y;
  if constexpr (PAIR) {
    if (e.save[0]) {
      store1(static_cast<T*>(e.save[0]) + idx, v[0]);
      store1(static_cast<T*>(e.save[1]) + idx, v[1]);
    }
    y = act_value<FAST>(v[0], e.act) * v[1];
  } else {
    const float a = e.bias ? v[0] + load1(static_cast<const T*>(e.bias) + n) : v[0];
    if (e.save[0]) store1(static_cast<T*>(e.save[0]) + idx, a);
    y = act_value<FAST>(a, e.act);
    if (e.residual) y += load1(static_cast<const T*>(e.residual) + idx);
  }
  store1(static_cast<T*>(e.out[0]) + idx, y);
}

hipError_t launch_dense_decode(const DenseJob& j, const DenseEpi& e, bool bf16, hipStream_t st) {
  const unsigned grid = ceil_div(j.N, j.pair ? 8 : 16);
  if (bf16) {
    if (j.pair) k_dense_decode<uint16_t, true><<<grid, 512, 0, st>>>(j, e);
    else k_dense_decode<uint16_t, false><<<grid, 512, 0, st>>>(j, e);
  } else {
    if (j.pair) k_dense_decode<float, true><<<grid, 512, 0, st>>>(j, e);
    else k_dense_decode<float, false><<<grid, 512, 0, st>>>(j, e);
  }
  return hipGetLastError();
}

}  // namespace moe
