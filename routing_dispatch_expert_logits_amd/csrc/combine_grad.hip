// Backward pass of the combine: out[t] = sum_j w[t, j] Y[token_row[t, j]] gives each expert row the
// gradient w[t, j] dout[t], and each routing weight the dot product <dout[t], Y[token_row[t, j]]>.
#include "dense_device.h"
#include "grouped_kernels.h"

namespace moe {

// A workgroup per token (while the grid lasts) and part of its assignments: a token's gradient row is read once into registers, eight
// elements per thread and chunk, and meets JB expert rows at a time; the dot products are summed per thread,
// then over the lanes of a wave, then over the waves in order.
template <typename T, typename G, int JB, int CH>
__global__ __launch_bounds__(256) void k_combine_grad(const G* __restrict__ dout, const T* __restrict__ y,
                                                      const int32_t* __restrict__ token_row,
                                                      const float* __restrict__ topk_w, int D, int tokens,
                                                      int k, T* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float part[4][JB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int n8 = ceil_div(D, 8), per = ceil_div(ceil_div(k, JB), (int)gridDim.y) * JB;
  const int j1 = min(k, ((int)blockIdx.y + 1) * per);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j0 = blockIdx.y * per; j0 < j1; j0 += JB) {
      int64_t row[JB];
      float w[JB], dot[JB];
#pragma unroll
      for (int u = 0; u < JB; ++u) {
        row[u] = j0 + u < j1 ? token_row[t * k + j0 + u] : -1;
        if (row[u] >= (int64_t)tokens * k) row[u] = -1;   // no row of ours
        w[u] = dy && j0 + u < j1 ? topk_w[t * k + j0 + u] : 0.f;
        dot[u] = 0.f;
      }
      for (int c0 = 0; c0 < n8; c0 += 256 * CH) {
#pragma unroll
        for (int h = 0; h < CH; ++h) {
          const int c = c0 + h * 256 + (int)threadIdx.x, left = D - 8 * c;
          if (left <= 0) continue;
          float g[8];
          load8(dout + t * D + 8 * c, left, g);
#pragma unroll
          for (int u = 0; u < JB; ++u) {
            if (row[u] < 0) continue;
            const int64_t at = row[u] * D + 8 * c;
            float v[8];
            if (dw) {
              load8(y + at, left, v);
#pragma unroll
              for (int i = 0; i < 8; ++i) dot[u] = fmaf(g[i], v[i], dot[u]);
            }
            if (dy) {
#pragma unroll
              for (int i = 0; i < 8; ++i) v[i] = w[u] * g[i];
              store8(dy + at, left, v);
            }
          }
        }
      }
      if (!dw) continue;
#pragma unroll
      for (int u = 0; u < JB; ++u) dot[u] = wave_sum_f32(dot[u]);
      if (lane == 0)
#pragma unroll
        for (int u = 0; u < JB; ++u) part[wave][u] = dot[u];
      __syncthreads();
      if ((int)threadIdx.x < JB && j0 + (int)threadIdx.x < j1) {
        const int u = threadIdx.x;
        dw[t * k + j0 + u] = ((part[0][u] + part[1][u]) + part[2][u]) + part[3][u];
      }
      __syncthreads();
    }
  }
}

hipError_t launch_combine_grad(const void* dout, bool dout_f32, const void* y_perm, const int32_t* token_row,
                               const float* topk_w, int D, bool bf16, int T, int k, void* dy_perm, float* dtopk_w,
                               hipStream_t st) {
  auto go = [&](auto* ty, auto* tg) {
    using E = std::remove_pointer_t<decltype(ty)>;
    using G = std::remove_pointer_t<decltype(tg)>;
    k_combine_grad<E, G, 1, 1><<<T < (1 << 22) ? T : 1 << 22, 256, 0, st>>>(static_cast<const G*>(dout), static_cast<const E*>(y_perm),
                                                                        token_row, topk_w, D, T, k, static_cast<E*>(dy_perm), dtopk_w);
  };
  uint16_t* h = nullptr;
  float* f = nullptr;
  if (bf16 && dout_f32) go(h, f);
  else if (bf16) go(h, h);
  else if (dout_f32) go(f, f);
  else go(f, h);
  return hipGetLastError();
}

}  // namespace moe
