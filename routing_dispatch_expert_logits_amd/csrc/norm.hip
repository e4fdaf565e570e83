// Layer norm, forward and backward.
#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

// Sum over the 256 threads of a workgroup, in a fixed order, in every thread.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = wave_sum_f32(v);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  return (s[0] + s[1]) + (s[2] + s[3]);
}

// Workgroups of a kernel that takes a row at a time.
static unsigned norm_grid(int T) { return T < (1 << 20) ? T : 1 << 20; }

// One workgroup per row; the variance is taken from the centred row.
template <typename T>
__global__ __launch_bounds__(256) void k_norm_forward(const T* __restrict__ x, const T* __restrict__ w,
                                                      const T* __restrict__ b, T* __restrict__ y,
                                                      float* __restrict__ mean, float* __restrict__ rstd, int rows,
                                                      int H, float eps) {
  __shared__ float s[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const T* xr = x + row * H;
  float v[8], sum = 0.f;
  for (int c = threadIdx.x * 8; c < H; c += 2048) {
    load8(xr + c, H - c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += v[i];
  }
  const float m = block_sum(sum, s) / H;
  sum = 0.f;
  for (int c = threadIdx.x * 8; c < H; c += 2048) {
    load8(xr + c, H - c, v);
#pragma unroll
    for (int i = 0; i < 8; ++i) sum += c + i < H ? (v[i] - m) * (v[i] - m) : 0.f;
  }
  const float r = 1.f / sqrtf(block_sum(sum, s) / H + eps);
  if (threadIdx.x == 0) {
    if (mean) mean[row] = m;
    if (rstd) rstd[row] = r;
  }
  for (int c = threadIdx.x * 8; c < H; c += 2048) {
    float vw[8], vb[8] = {};
    load8(xr + c, H - c, v);
    load8(w + c, H - c, vw);
    if (b) load8(b + c, H - c, vb);
#pragma unroll
    for (int i = 0; i < 8; ++i) v[i] = (v[i] - m) * r * vw[i] + vb[i];
    store8(y + row * H + c, H - c, v);
  }
  }
}

hipError_t launch_norm_forward(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                               int T, int H, float eps, bool bf16, hipStream_t st) {
  if (bf16)
    k_norm_forward<uint16_t><<<norm_grid(T), 256, 0, st>>>(static_cast<const uint16_t*>(x), static_cast<const uint16_t*>(w),
                                                static_cast<const uint16_t*>(b), static_cast<uint16_t*>(y), mean,
                                                rstd, T, H, eps);
  else
    k_norm_forward<float><<<norm_grid(T), 256, 0, st>>>(static_cast<const float*>(x), static_cast<const float*>(w),
                                             static_cast<const float*>(b), static_cast<float*>(y), mean, rstd, T,
                                             H, eps);
  return hipGetLastError();
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_dx(const T* __restrict__ dy, const T* __restrict__ x,
                                                 const T* __restrict__ w, const float* __restrict__ mean,
                                                 const float* __restrict__ rstd, T* __restrict__ dx, int rows, int H) {
  __shared__ float s[4];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
  const float m = mean[row], r = rstd[row];
  float vx[8], vd[8], vw[8], s1 = 0.f, s2 = 0.f;
  for (int c = threadIdx.x * 8; c < H; c += 2048) {
    load8(x + row * H + c, H - c, vx);
    load8(dy + row * H + c, H - c, vd);
    load8(w + c, H - c, vw);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float e = vd[i] * vw[i];
      s1 += e;
      s2 += e * ((vx[i] - m) * r);
    }
  }
  s1 = block_sum(s1, s) / H;
  s2 = block_sum(s2, s) / H;
  for (int c = threadIdx.x * 8; c < H; c += 2048) {
    load8(x + row * H + c, H - c, vx);
    load8(dy + row * H + c, H - c, vd);
    load8(w + c, H - c, vw);
#pragma unroll
    for (int i = 0; i < 8; ++i) vx[i] = r * (vd[i] * vw[i] - s1 - (vx[i] - m) * r * s2);
    store8(dx + row * H + c, H - c, vx);
  }
  }
}

// Column sums of dy n and dy over one block of rows (rows of 2 H partial sums).
template <typename T>
__global__ __launch_bounds__(256) void k_norm_dw(const T* __restrict__ dy, const T* __restrict__ x,
                                                 const float* __restrict__ mean, const float* __restrict__ rstd,
                                                 float* __restrict__ part, int rows, int H) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  const int per = ceil_div(rows, (int)gridDim.y);
  const int r0 = (int)min<int64_t>(rows, (int64_t)blockIdx.y * per), r1 = min(rows, r0 + per);
  float sw = 0.f, sb = 0.f;
  for (int r = r0; r < r1; ++r) {
    const float d = load1(dy + (int64_t)r * H + c);
    sw += d * ((load1(x + (int64_t)r * H + c) - mean[r]) * rstd[r]);
    sb += d;
  }
  part[(int64_t)blockIdx.y * 2 * H + c] = sw;
  part[((int64_t)blockIdx.y * 2 + 1) * H + c] = sb;
}

int norm_row_blocks(int T, int) {
  const int n = ceil_div(T, 32);
  return n < 256 ? n : 256;
}

hipError_t launch_norm_backward(const void* dy, const void* x, const void* w, const float* mean,
                                const float* rstd, void* dx, float* part, int T, int H, bool bf16,
                                hipStream_t st) {
  auto go = [&](auto* t) {
    using E = std::remove_pointer_t<decltype(t)>;
    const E *a = static_cast<const E*>(dy), *b = static_cast<const E*>(x), *c = static_cast<const E*>(w);
    if (dx) k_norm_dx<E><<<norm_grid(T), 256, 0, st>>>(a, b, c, mean, rstd, static_cast<E*>(dx), T, H);
    if (part)
      k_norm_dw<E><<<dim3(ceil_div(H, 256), norm_row_blocks(T, H)), 256, 0, st>>>(a, b, mean, rstd, part, T, H);
  };
  if (bf16) go(static_cast<uint16_t*>(nullptr));
  else go(static_cast<float*>(nullptr));
  return hipGetLastError();
}

}  // namespace moe
