// fp32 dense products of the gated and linear operators and of their backward passes.
//
// C(m, n) = sum_k A(m, k) B(n, k) for the three layouts these need: y = x w^T (both operands
// with k along their rows), dx = d w (the weight with k across its rows) and dw = d^T x (both).
#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

// What the epilogue does with one output value (and the second projection's, for the
// gated product).
__device__ __forceinline__ void f32_out(const DenseEpi& e, int z, int64_t idx, int n, float v0, float v1) {
  float* out = static_cast<float*>(e.out[z]);
  if (e.kind == DENSE_STORE) {
    out[idx] = v0;
  } else if (e.kind == DENSE_LINEAR) {
    const float a = e.bias ? v0 + static_cast<const float*>(e.bias)[n] : v0;
    if (e.save[0]) static_cast<float*>(e.save[0])[idx] = a;
    float y = act_value<false>(a, e.act);
    if (e.residual) y += static_cast<const float*>(e.residual)[idx];
    out[idx] = y;
  } else {
    if (e.save[0]) {
      static_cast<float*>(e.save[0])[idx] = v0;
      static_cast<float*>(e.save[1])[idx] = v1;
    }
    out[idx] = act_value<false>(v0, e.act) * v1;
  }
}

// Tile 64 x 64, four waves in 2 x 2, K-steps of 16 staged through LDS with k across the
// rows, v_mfma_f32_16x16x4_f32: lane l supplies A[l % 16][l / 16] and B[l / 16][l % 16]
// and receives D[4 (l / 16) + i][l % 16].  B's columns take the A side, so a lane holds four
// neighbouring output columns.
template <bool PAIR>
__global__ __launch_bounds__(256) void k_dense_f32(DenseJob j, DenseEpi e) {
  constexpr int BK = 16, LD = 68, NB = PAIR ? 2 : 1;
  __shared__ float sA[BK * LD];
  __shared__ float sB[NB][BK * LD];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int NT = ceil_div(j.N, 64);
  const int z = blockIdx.y;
  const int m0 = (int)(blockIdx.x / NT) * 64, n0 = (int)(blockIdx.x % NT) * 64;
  const int wm = (wave >> 1) * 32, wn = (wave & 1) * 32;
  f32x4 acc[NB][2][2];
#pragma unroll
  for (int b = 0; b < NB; ++b)
#pragma unroll
    for (int f = 0; f < 4; ++f) acc[b][f >> 1][f & 1] = f32x4{0.f, 0.f, 0.f, 0.f};

  auto fill = [&](float* dst, const float* src, int64_t ld, bool col, int r0, int rows, int k0) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const int q = tid + 256 * i;  // of 64 x 16 elements, the stored-along index fastest
      const int r = col ? q & 63 : q >> 4, k = col ? q >> 6 : q & 15;
      float v = 0.f;
      if (r0 + r < rows && k0 + k < j.K)
        v = src[col ? (int64_t)(k0 + k) * ld + (r0 + r) : (int64_t)(r0 + r) * ld + (k0 + k)];
      dst[k * LD + r] = v;
    }
  };
  for (int s = 0; s < j.segs; ++s)
    for (int k0 = 0; k0 < j.K; k0 += BK) {
      __syncthreads();
      fill(sA, static_cast<const float*>(j.A[z][s]), j.lda, j.a_col, m0, j.M, k0);
#pragma unroll
      for (int b = 0; b < NB; ++b)
        fill(sB[b], static_cast<const float*>(PAIR ? j.B[b][0] : j.B[z][s]), j.ldb, j.b_col, n0, j.N, k0);
      __syncthreads();
#pragma unroll
      for (int kk = 0; kk < BK; kk += 4) {
        const int row = (kk + (lane >> 4)) * LD + (lane & 15);
        const float a0 = sA[row + wm], a1 = sA[row + wm + 16];
#pragma unroll
        for (int b = 0; b < NB; ++b)
#pragma unroll
          for (int f = 0; f < 2; ++f) {
            const float bv = sB[b][row + wn + 16 * f];
            acc[b][0][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv, a0, acc[b][0][f], 0, 0, 0);
            acc[b][1][f] = __builtin_amdgcn_mfma_f32_16x16x4f32(bv, a1, acc[b][1][f], 0, 0, 0);
          }
      }
    }
#pragma unroll
  for (int fm = 0; fm < 2; ++fm)
#pragma unroll
    for (int fn = 0; fn < 2; ++fn)
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int m = m0 + wm + 16 * fm + (lane & 15), n = n0 + wn + 16 * fn + 4 * (lane >> 4) + i;
        if (m < j.M && n < j.N)
          f32_out(e, z, (int64_t)m * j.N + n, n, acc[0][fm][fn][i], acc[NB - 1][fm][fn][i]);
      }
}

hipError_t launch_dense(const DenseJob& j, const DenseEpi& e, bool bf16, float* part, hipStream_t st) {
  if (bf16) return launch_dense_mm(j, e, part, st);
  const dim3 grid((unsigned)((int64_t)ceil_div(j.M, 64) * ceil_div(j.N, 64)), j.batch);
  if (j.pair) k_dense_f32<true><<<grid, 256, 0, st>>>(j, e);
  else k_dense_f32<false><<<grid, 256, 0, st>>>(j, e);
  return hipGetLastError();
}

}  // namespace moe
