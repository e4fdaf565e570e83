// Backward pass of the combine: out[t] = sum_j w[t, j] Y[token_row[t, j]] gives each expert row the
// gradient w[t, j] dout[t], and each routing weight the dot product <dout[t], Y[token_row[t, j]]>.
#include <type_traits>

#include "dense_device.h"
#include "grouped_kernels.h"

namespace moe {

// Bound by memory: each expert row is read once and its gradient written once, past the caches, which nothing will
// read them from.  A workgroup per token (while the grid lasts) and part of its assignments: a token's gradient row is
// read once for JB expert rows, whose loads are in flight together, eight elements per thread; the dot
// products are summed per thread, then over the lanes of a wave, then over the waves in order.  Rows of fewer than 2048
// elements leave lanes idle: 4096 tokens of 8 experts take 17 us for 64 columns, 25 for 256, 31 for 512, 35 for 1024 and 57 for
// 2048, where the bytes are 2, 7, 14, 28 and 56 us.
template <typename T>
struct Piece {   // eight elements of a row of whole 16-byte chunks; fp32 rows may end after four
  u32x4 v[sizeof(T) / 2];
  __device__ __forceinline__ void load(const T* p, int left) {
    v[0] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p));
    if constexpr (sizeof(T) == 4) {
      v[1] = u32x4{0, 0, 0, 0};
      if (left > 4) v[1] = __builtin_nontemporal_load(reinterpret_cast<const u32x4*>(p) + 1);
    }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? v[0][i / 2] & 0xffff0000u : v[0][i / 2] << 16);
    else return __uint_as_float(v[i >> 2][i & 3]);
  }
  __device__ __forceinline__ void set(int i, float a, float b) {   // elements i and i + 1, i even
    if constexpr (sizeof(T) == 2) v[0][i / 2] = f32_to_bf16(a) | (uint32_t)f32_to_bf16(b) << 16;
    else v[i >> 2][i & 3] = __float_as_uint(a), v[i >> 2][(i & 3) + 1] = __float_as_uint(b);
  }
  __device__ __forceinline__ void store(T* p, int left) const {
    __builtin_nontemporal_store(v[0], reinterpret_cast<u32x4*>(p));
    if constexpr (sizeof(T) == 4)
      if (left > 4) __builtin_nontemporal_store(v[1], reinterpret_cast<u32x4*>(p) + 1);
  }
};

template <typename T, typename G, int JB>
__global__ __launch_bounds__(256) void k_combine_grad(const G* __restrict__ dout, const T* __restrict__ y,
                                                      const int32_t* __restrict__ token_row,
                                                      const float* __restrict__ topk_w, int D, int tokens,
                                                      int k, T* __restrict__ dy, float* __restrict__ dw) {
  __shared__ float part[4][JB];
  const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
  const int per = ceil_div(ceil_div(k, JB), (int)gridDim.y) * JB;
  const int j1 = min(k, ((int)blockIdx.y + 1) * per);
  for (int64_t t = blockIdx.x; t < tokens; t += gridDim.x) {
    for (int j0 = blockIdx.y * per; j0 < j1; j0 += JB) {
      int64_t row[JB];
      float w[JB], dot[JB];
#pragma unroll
      for (int u = 0; u < JB; ++u) {
        row[u] = j0 + u < j1 ? token_row[t * k + j0 + u] : -1;
        if (row[u] >= (int64_t)tokens * k) row[u] = -1;   // no row of ours
        w[u] = dy && row[u] >= 0 ? topk_w[t * k + j0 + u] : 0.f;
        dot[u] = 0.f;
      }
      for (int c = 8 * (int)threadIdx.x; c < D; c += 8 * 256) {
        const int left = D - c;
        float g[8];
        load8(dout + t * D + c, left, g);
        Piece<T> v[JB];
        if (dw) {
#pragma unroll
          for (int u = 0; u < JB; ++u)
            if (row[u] >= 0) v[u].load(y + row[u] * D + c, left);
#pragma unroll
          for (int u = 0; u < JB; ++u) {
            if (row[u] < 0) continue;
#pragma unroll
            for (int i = 0; i < 8; ++i) dot[u] = fmaf(g[i], v[u].get(i), dot[u]);
          }
        }
        if (dy) {
#pragma unroll
          for (int u = 0; u < JB; ++u) {
            if (row[u] < 0) continue;
#pragma unroll
            for (int i = 0; i < 8; i += 2) v[u].set(i, w[u] * g[i], w[u] * g[i + 1]);
            v[u].store(dy + row[u] * D + c, left);
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
  constexpr int JB = 2;   // 8192 tokens of 7168, 8 experts: 406 / 404 / 417 / 420 us with 1 / 2 / 4 / 8
  // a token's assignments over several workgroups while there are few tokens
  int parts = 1;
  while (parts < ceil_div(k, JB) && (int64_t)T * parts < 1024) ++parts;
  const dim3 grid(T < (1 << 20) ? T : 1 << 20, parts);
  auto go = [&](auto* ty, auto* tg) {
    using E = std::remove_pointer_t<decltype(ty)>;
    using G = std::remove_pointer_t<decltype(tg)>;
    k_combine_grad<E, G, JB><<<grid, 256, 0, st>>>(static_cast<const G*>(dout), static_cast<const E*>(y_perm), token_row, topk_w,
                                                   D, T, k, static_cast<E*>(dy_perm), dtopk_w);
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
