// Gradients before an activation, column sums and zero fills of the dense backward passes.
#include <type_traits>

#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

constexpr int kGradCols = 256;  // columns per workgroup: 32 lanes of 8
constexpr int kGradSub = 8;     // rows in flight per workgroup

// Row blocks of a pass that sums columns: one for up to 32 rows (whose sums then need no second
// launch), else 2048 workgroups or 8 rows each.
int grad_row_blocks(int T, int N) {
  if (T <= 32) return 1;
  const int cb = ceil_div(N, kGradCols), want = ceil_div(2048, cb), most = ceil_div(T, kGradSub);
  return want < most ? want : most;
}

// The first bf16 term of v, v rounded but no infinity in place of a finite v, and in *rest what it
// leaves of v: nothing of an infinity, whose first term says it all.
__device__ __forceinline__ float first_term(float v, float* rest) {
  const bool finite = fabsf(v) < __builtin_inff();
  const float b = bf16_to_f32(f32_to_bf16(v)), t = finite ? copysignf(fminf(fabsf(b), 0x1.fep127f), b) : b;
  *rest = finite ? v - t : 0.f;
  return t;
}

// The finite rows, eight elements of a row in dst per thread.
__device__ __forceinline__ void finite_rows(const FiniteRows& f, int rows) {
  const uint16_t* src = static_cast<const uint16_t*>(f.src);
  uint16_t* dst = static_cast<uint16_t*>(f.dst);
  const int per = (int)(f.ld / 8);
  const int64_t total = (int64_t)rows * per, step = (int64_t)gridDim.x * gridDim.y * blockDim.x;
  for (int64_t i = ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * blockDim.x + threadIdx.x; i < total; i += step) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    float v[8];
    load8(src + r * f.cols + c, f.cols - c, v);
#pragma unroll
    for (int k = 0; k < 8; ++k) v[k] = fabsf(v[k]) < __builtin_inff() ? v[k] : 0.f;  // not so for NaN
    store8(dst + i * 8, v);
  }
}

// Bound by memory in bf16 (4096 x 8192 gated, 3 reads and 2 writes of 64 MB: 60 to 64 us, 5.2 to
// 5.6 TB/s), by the exponentials of fp32 GELU otherwise (545 x 5664: 13 us, 37 MB).
// One pass over dh, g (and u): d0 = dh u act'(g), d1 = dh act(g) in fp32, rounded on store.
// Workgroup (column block, row block); a thread owns 8 columns and every kGradSub-th row of
// its block; the column sums of d0 go through LDS in row-lane order.  A second plane of workgroups
// (blockIdx.z) makes the finite rows, in the same launch.
template <typename T, bool GATED>
__global__ __launch_bounds__(256) void k_act_grad(const T* __restrict__ dh, const T* __restrict__ g,
                                                  const T* __restrict__ u, int act, int rows, int N,
                                                  T* __restrict__ d0, T* __restrict__ d1, int terms, int64_t lo,
                                                  int64_t ld, float* __restrict__ part, void* __restrict__ out,
                                                  bool out_f32, FiniteRows finite) {
  constexpr bool FAST = sizeof(T) == 2;
  if (sizeof(T) == 2 && blockIdx.z) return finite_rows(finite, rows);
  const int tid = threadIdx.x, cl = tid & 31, sub = tid >> 5;
  const int c0 = (int)blockIdx.x * kGradCols + cl * 8;
  const int per = ceil_div(rows, (int)gridDim.y);
  const int r0 = min(rows, (int)blockIdx.y * per), r1 = min(rows, r0 + per);
  const int nc = N - c0;                                          // columns of this thread in N
  const int np = (int)min<int64_t>(8, max<int64_t>(0, ld - c0));  // and in an output row, padding included
  float sum[8] = {};
  if (nc > 0) {
    for (int r = r0 + sub; r < r1; r += kGradSub) {
      const int64_t in = (int64_t)r * N + c0, out = (int64_t)r * ld + c0;
      float vdh[8], vg[8], vu[8], v0[8], v1[8];
      load8(dh + in, nc, vdh);
      if (g) load8(g + in, nc, vg);
      if (GATED) load8(u + in, nc, vu);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        float slope = 1.f, a = 0.f;
        if (g) a = act_value_slope<FAST>(vg[i], act, &slope);
        v0[i] = i < nc ? vdh[i] * (GATED ? vu[i] * slope : slope) : 0.f;
        v1[i] = i < nc ? vdh[i] * a : 0.f;
        sum[i] += v0[i];
      }
      if (sizeof(T) == 4 || terms == 1) {
        if (d0) store8(d0 + out, np, v0);
        if (GATED) store8(d1 + out, np, v1);
        continue;
      }
      float t0[8], t1[8];
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        t0[i] = first_term(v0[i], &v0[i]);
        if (GATED) t1[i] = first_term(v1[i], &v1[i]);
      }
      store8(d0 + out, np, t0);
      if (GATED) store8(d1 + out, np, t1);
      for (int q = 1; q < terms; ++q) {
        store8(d0 + q * lo + out, np, v0);
        if (GATED) store8(d1 + q * lo + out, np, v1);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
          v0[i] -= bf16_to_f32(f32_to_bf16(v0[i]));
          if (GATED) v1[i] -= bf16_to_f32(f32_to_bf16(v1[i]));
        }
      }
    }
  }
  if (part) {
    __shared__ float s[kGradSub][kGradCols];
#pragma unroll
    for (int i = 0; i < 8; ++i) s[sub][cl * 8 + i] = sum[i];
    __syncthreads();
    const int n = (int)blockIdx.x * kGradCols + tid;
    if (n < N) {
      float v = 0.f;
#pragma unroll
      for (int q = 0; q < kGradSub; ++q) v += s[q][tid];
      if (gridDim.y > 1) part[(int64_t)blockIdx.y * N + n] = v;
      else if (out_f32) static_cast<float*>(out)[n] = v;
      else static_cast<uint16_t*>(out)[n] = f32_to_bf16(v);
    }
  }
}

__global__ __launch_bounds__(1024) void k_col_sum(ColSum c) {
  __shared__ float s[16][64];
  col_sum(c, blockIdx.x, blockIdx.y, s);
}

hipError_t launch_col_sum(const ColSum& c, hipStream_t st) {
  if (c.P) k_col_sum<<<dim3(ceil_div(c.N, 64), c.out1 ? 2 : 1), 1024, 0, st>>>(c);
  return hipGetLastError();
}

hipError_t launch_act_grad(const void* dh, const void* g, const void* u, int act, bool bf16, int T, int N,
                           void* d0, void* d1, int terms, int64_t lo, int64_t ld, float* part, void* sum, bool sum_f32,
                           ColSum* later, const FiniteRows& finite, hipStream_t st) {
  const int single = ceil_div(T, kGradSub);  // without sums, a row per thread while the grid lasts
  const dim3 grid(ceil_div(N, kGradCols), sum ? grad_row_blocks(T, N) : single < 32768 ? single : 32768,
                  finite.src ? 2 : 1);
  if (!sum) part = nullptr;
  auto go = [&](auto* t) {
    using E = std::remove_pointer_t<decltype(t)>;
    const E *a = static_cast<const E*>(dh), *b = static_cast<const E*>(g), *c = static_cast<const E*>(u);
    E *p0 = static_cast<E*>(d0), *p1 = static_cast<E*>(d1);
    if (u) k_act_grad<E, true><<<grid, 256, 0, st>>>(a, b, c, act, T, N, p0, p1, terms, lo, ld, part, sum, sum_f32, finite);
    else k_act_grad<E, false><<<grid, 256, 0, st>>>(a, b, c, act, T, N, p0, p1, terms, lo, ld, part, sum, sum_f32, finite);
  };
  if (bf16) go(static_cast<uint16_t*>(nullptr));
  else go(static_cast<float*>(nullptr));
  if (sum && grid.y > 1) *later = ColSum{part, (int)grid.y, N, N, sum, nullptr, sum_f32};
  return hipGetLastError();
}

// Eight elements of a padded row per thread.
__global__ __launch_bounds__(256) void k_pad_rows(PadRows p, int cols, int ld) {
  const uint16_t* src = static_cast<const uint16_t*>(p.src[blockIdx.y]);
  uint16_t* dst = static_cast<uint16_t*>(p.dst[blockIdx.y]);
  if (!src) return;
  const int per = ld / 8;
  const int64_t total = p.rows[blockIdx.y] * per;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < total; i += (int64_t)gridDim.x * 256) {
    const int64_t r = i / per;
    const int c = (int)(i - r * per) * 8;
    float v[8];
    load8(src + r * cols + c, cols - c, v);
    store8(dst + i * 8, v);
  }
}

hipError_t launch_pad_rows(const PadRows& p, int cols, int64_t ld, hipStream_t st) {
  int64_t most = 1;
  for (int64_t r : p.rows) most = r > most ? r : most;
  const int64_t want = (most * (ld / 8) + 255) / 256;
  k_pad_rows<<<dim3((unsigned)(want < 8192 ? want : 8192), 3), 256, 0, st>>>(p, cols, (int)ld);
  return hipGetLastError();
}

__global__ __launch_bounds__(256) void k_fill_zero(uint16_t* p, size_t n) {
  for (size_t i = (size_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (size_t)gridDim.x * 256) p[i] = 0;
}

hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t st) {
  const size_t n = bytes / 2, want = (n + 255) / 256;
  k_fill_zero<<<(unsigned)(want < 4096 ? want : 4096), 256, 0, st>>>(static_cast<uint16_t*>(p), n);
  return hipGetLastError();
}

}  // namespace moe
