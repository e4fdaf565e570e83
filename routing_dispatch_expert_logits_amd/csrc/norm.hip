// Layer norm, forward and backward: y = (x - mean) rstd w + b; with n = (x - mean) rstd and
// e = dy w, dx = rstd (e - mean(e) - n mean(e n)), dw = sum_t dy n, db = sum_t dy.  Both are
// bound by memory: a row is read once, kept in registers while its sums are formed, and written
// once.  Measured (MI355X, 8192 x 7168, bf16): forward 55 us, 4.27 TB/s; backward with all three
// gradients 82 us, 77 of them the pass over the rows and 5 the launch that joins its column sums; a
// copy of 2 GiB runs at 4.9 TB/s.  One row of 4096 takes 6.7 us, a launch; 2049 x 1021 fp32
// backward 13.5 us, two launches and their latencies (25 MB, 5 us at that rate).  Rows too wide for
// registers are read twice or more: 2048 x 16384 fp32 backward 193 us, 2.1 TB/s.
#include "dense_device.h"
#include "dense_kernels.h"

namespace moe {

// Forward rows up to kRowChunks * 8 elements stay in registers.
constexpr int kRowChunks = 2048;

// Sum over a workgroup of up to 16 waves, in a fixed order, in every thread.  s: 16 floats of
// LDS that no earlier sum of the caller still reads.
__device__ __forceinline__ float block_sum(float v, float* s) {
  v = wave_sum_f32(v);
  if ((threadIdx.x & 63) == 0) s[threadIdx.x >> 6] = v;
  __syncthreads();
  const int waves = blockDim.x >> 6;
  v = 0.f;
  for (int i = 0; i < waves; ++i) v += s[i];
  return v;
}

// A row per workgroup at a time (or per wave, blockDim.y of them in a workgroup, where 64
// threads hold it): thread i holds the chunks of 8 elements i, i + blockDim.x, ..  Weight and
// bias stay in registers over all rows of the workgroup: read again for each row they would be
// as many bytes from L2 as the row itself.  The next row's loads are in flight while one is
// worked on; the variance is taken from the centred row.
template <typename T, int NCH, bool WAVE>
__global__ __launch_bounds__(WAVE ? 256 : 1024) void k_norm_forward(const T* __restrict__ x, const T* __restrict__ w,
                                                                    const T* __restrict__ b, T* __restrict__ y,
                                                                    float* __restrict__ mean,
                                                                    float* __restrict__ rstd, int rows, int per,
                                                                    int H, float eps) {
  __shared__ float s[4][16];
  const int first = ((int)blockIdx.x * (int)blockDim.y + (int)threadIdx.y) * per;
  const int last = min(rows, first + per);
  int col[NCH];
  Raw8<T> next[NCH], vw[NCH], vb[NCH];
  auto load = [&](int row) __attribute__((always_inline)) {
#pragma unroll
    for (int i = 0; i < NCH; ++i) next[i].load(x + (int64_t)row * H + col[i], H - col[i]);
  };
#pragma unroll
  for (int i = 0; i < NCH; ++i) col[i] = ((int)threadIdx.x + i * (int)blockDim.x) * 8;
  if (first < last) load(first);
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    vw[i].load(w + col[i], H - col[i]);
    vb[i].load(b + col[i], b ? H - col[i] : 0);
  }
  for (int row = first, q = 0; row < last; ++row, q ^= 2) {
    float v[NCH][8], sum = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] = next[i].get(k);
        sum += v[i][k];
      }
    if (row + 1 < last) load(row + 1);
    // divided by H, not multiplied by 1 / H: a constant row's mean is the constant.  The sums'
    // LDS alternates between rows: its readers are one sync behind the next row's writers.
    const float m = (WAVE ? wave_sum_f32(sum) : block_sum(sum, s[q])) / (float)H;
    sum = 0.f;
#pragma unroll
    for (int i = 0; i < NCH; ++i)
#pragma unroll
      for (int k = 0; k < 8; ++k) {
        v[i][k] -= m;
        sum += col[i] + k < H ? v[i][k] * v[i][k] : 0.f;
      }
    const float r = 1.f / sqrtf((WAVE ? wave_sum_f32(sum) : block_sum(sum, s[q + 1])) / (float)H + eps);
    if (threadIdx.x == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = r;
    }
#pragma unroll
    for (int i = 0; i < NCH; ++i) {
#pragma unroll
      for (int k = 0; k < 8; ++k) v[i][k] = v[i][k] * r * vw[i].get(k) + vb[i].get(k);
      store8(y + (int64_t)row * H + col[i], H - col[i], v[i]);
    }
  }
}

// Longer rows: read three times.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_forward_long(const T* __restrict__ x, const T* __restrict__ w,
                                                            const T* __restrict__ b, T* __restrict__ y,
                                                            float* __restrict__ mean, float* __restrict__ rstd,
                                                            int rows, int H, float eps) {
  __shared__ float s[2][16];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const T* xr = x + row * H;
    float v[8], sum = 0.f;
    for (int c = threadIdx.x * 8; c < H; c += 8192) {
      load8(xr + c, H - c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += v[i];
    }
    const float m = block_sum(sum, s[0]) / H;
    sum = 0.f;
    for (int c = threadIdx.x * 8; c < H; c += 8192) {
      load8(xr + c, H - c, v);
#pragma unroll
      for (int i = 0; i < 8; ++i) sum += c + i < H ? (v[i] - m) * (v[i] - m) : 0.f;
    }
    const float r = 1.f / sqrtf(block_sum(sum, s[1]) / H + eps);
    if (threadIdx.x == 0) {
      if (mean) mean[row] = m;
      if (rstd) rstd[row] = r;
    }
    for (int c = threadIdx.x * 8; c < H; c += 8192) {
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

template <typename T>
static void norm_forward(const void* x_, const void* w_, const void* b_, void* y_, float* mean, float* rstd, int rows,
                         int H, float eps, hipStream_t st) {
  const T *x = static_cast<const T*>(x_), *w = static_cast<const T*>(w_), *b = static_cast<const T*>(b_);
  T* y = static_cast<T*>(y_);
  const int chunks = ceil_div(H, 8);
  if (chunks <= 256) {
    // 8 waves per SIMD of 256 CUs, then several rows each
    const int per = ceil_div(rows, 8192), grid = ceil_div(ceil_div(rows, per), 4);
    const dim3 block(64, 4);
    if (chunks <= 64) k_norm_forward<T, 1, true><<<grid, block, 0, st>>>(x, w, b, y, mean, rstd, rows, per, H, eps);
    else if (chunks <= 128) k_norm_forward<T, 2, true><<<grid, block, 0, st>>>(x, w, b, y, mean, rstd, rows, per, H, eps);
    else k_norm_forward<T, 4, true><<<grid, block, 0, st>>>(x, w, b, y, mean, rstd, rows, per, H, eps);
  } else if (chunks <= kRowChunks) {
    // two chunks a thread; up to four workgroups per CU
    const int threads = ceil_div(ceil_div(chunks, 2), 64) * 64;
    const int per = ceil_div(rows, 1024), grid = ceil_div(rows, per);
    k_norm_forward<T, 2, false><<<grid, threads, 0, st>>>(x, w, b, y, mean, rstd, rows, per, H, eps);
  } else {
    k_norm_forward_long<T><<<rows < 4096 ? rows : 4096, 1024, 0, st>>>(x, w, b, y, mean, rstd, rows, H, eps);
  }
}

hipError_t launch_norm_forward(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                               int T, int H, float eps, bool bf16, hipStream_t st) {
  if (bf16) norm_forward<uint16_t>(x, w, b, y, mean, rstd, T, H, eps, st);
  else norm_forward<float>(x, w, b, y, mean, rstd, T, H, eps, st);
  return hipGetLastError();
}

// Backward in one pass over dy and x.  A workgroup takes a block of consecutive rows, RB at a
// time; a thread owns NCH chunks of 8 columns, whose dw and db sums it keeps in registers over
// all its rows (rows in order), while the two sums of a row that dx needs meet in LDS.  The
// next rows' loads are in flight while these are worked on.  Behind a row's end dy and w are zeros,
// and n is made 0: a mean times rstd that overflows would enter the row's sums as 0 times infinity.
template <typename T, int NCH, int RB, int MAXT>
__global__ __launch_bounds__(MAXT) void k_norm_backward(const T* __restrict__ dy, const T* __restrict__ x,
                                                        const T* __restrict__ w, const float* __restrict__ mean,
                                                        const float* __restrict__ rstd, T* __restrict__ dx,
                                                        float* __restrict__ part, int rows, int per, int H, void* __restrict__ dw,
                                                        void* __restrict__ db, bool grad_f32) {
  __shared__ float s[2][16][2 * RB];
  const int r0 = (int)blockIdx.x * per, r1 = min(rows, r0 + per);
  const int wave = threadIdx.x >> 6, waves = blockDim.x >> 6;
  const float inv = 1.f / (float)H;
  // whether the wave holds columns behind the row's end
  const bool beyond = __builtin_amdgcn_readfirstlane(8 * ((int)threadIdx.x + 64 + (NCH - 1) * (int)blockDim.x) > H);
  float vw[NCH][8], sw[NCH][8] = {}, sb[NCH][8] = {};
  int col[NCH];
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    col[i] = ((int)threadIdx.x + i * (int)blockDim.x) * 8;
    load8(w + col[i], H - col[i], vw[i]);
  }
  Raw8<T> nx[RB][NCH], nd[RB][NCH];
  float nm[RB], nr[RB];
  auto load = [&](int r) __attribute__((always_inline)) {
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      const bool in = r + q < r1;
      const int64_t at = (int64_t)min(r + q, r1 - 1) * H;
      nm[q] = mean[min(r + q, r1 - 1)];
      nr[q] = in ? rstd[r + q] : 0.f;
#pragma unroll
      for (int i = 0; i < NCH; ++i) {
        nx[q][i].load(x + at + col[i], H - col[i]);
        nd[q][i].load(dy + at + col[i], in ? H - col[i] : 0);
      }
    }
  };
  load(r0);
  for (int r = r0, odd = 0; r < r1; r += RB, odd ^= 1) {
    float n[RB][NCH][8], d[RB][NCH][8], rs[RB], s1[RB], s2[RB];
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      rs[q] = nr[q];
      s1[q] = s2[q] = 0.f;
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          n[q][i][k] = (nx[q][i].get(k) - nm[q]) * rs[q];
          d[q][i][k] = nd[q][i].get(k);
        }
      if (beyond)
#pragma unroll
        for (int i = 0; i < NCH; ++i)
#pragma unroll
          for (int k = 0; k < 8; ++k) n[q][i][k] = col[i] + k < H ? n[q][i][k] : 0.f;
    }
    if (r + RB < r1) load(r + RB);
#pragma unroll
    for (int q = 0; q < RB; ++q) {
#pragma unroll
      for (int i = 0; i < NCH; ++i)
#pragma unroll
        for (int k = 0; k < 8; ++k) {
          sw[i][k] += d[q][i][k] * n[q][i][k];
          sb[i][k] += d[q][i][k];
          d[q][i][k] *= vw[i][k];
          s1[q] += d[q][i][k];
          s2[q] += d[q][i][k] * n[q][i][k];
        }
      s1[q] = wave_sum_f32(s1[q]);
      s2[q] = wave_sum_f32(s2[q]);
    }
    if (!dx) continue;  // the same for every thread of the launch
    if ((threadIdx.x & 63) == 0)
#pragma unroll
      for (int q = 0; q < RB; ++q) {
        s[odd][wave][2 * q] = s1[q];
        s[odd][wave][2 * q + 1] = s2[q];
      }
    __syncthreads();  // the other buffer's readers are past the sync before this one
#pragma unroll
    for (int q = 0; q < RB; ++q) {
      s1[q] = s2[q] = 0.f;
      for (int v = 0; v < waves; ++v) {
        s1[q] += s[odd][v][2 * q];
        s2[q] += s[odd][v][2 * q + 1];
      }
      s1[q] *= inv;
      s2[q] *= inv;
      if (r + q < r1) {
#pragma unroll
        for (int i = 0; i < NCH; ++i) {
          float o[8];
#pragma unroll
          for (int k = 0; k < 8; ++k) o[k] = rs[q] * (d[q][i][k] - s1[q] - n[q][i][k] * s2[q]);
          store8(dx + (int64_t)(r + q) * H + col[i], H - col[i], o);
        }
      }
    }
  }
  if (!part) return;
  float* p = part + (int64_t)blockIdx.x * 2 * H;
#pragma unroll
  for (int i = 0; i < NCH; ++i) {
    const int c = col[i], n = H - c;
    auto out = [&](void* o, const float* v) {
      if (o && grad_f32) store8(static_cast<float*>(o) + c, n, v);
      else if (o) store8(static_cast<uint16_t*>(o) + c, n, v);
    };
    if (gridDim.x == 1) {  // all rows are here: these are the gradients
      out(dw, sw[i]);
      out(db, sb[i]);
    } else {
      store8(p + c, n, sw[i]);
      store8(p + H + c, n, sb[i]);
    }
  }
}

// Rows of more than 16384 elements (fp32: 8192): dx by a workgroup per row, the column sums by a second kernel.
template <typename T>
__global__ __launch_bounds__(1024) void k_norm_dx_long(const T* __restrict__ dy, const T* __restrict__ x,
                                                       const T* __restrict__ w, const float* __restrict__ mean,
                                                       const float* __restrict__ rstd, T* __restrict__ dx, int rows,
                                                       int H) {
  __shared__ float s[2][16];
  for (int64_t row = blockIdx.x; row < rows; row += gridDim.x) {
    const float m = mean[row], r = rstd[row];
    float vx[8], vd[8], vw[8], s1 = 0.f, s2 = 0.f;
    for (int c = threadIdx.x * 8; c < H; c += 8192) {
      load8(x + row * H + c, H - c, vx);
      load8(dy + row * H + c, H - c, vd);
      load8(w + c, H - c, vw);
#pragma unroll
      for (int i = 0; i < 8; ++i) {
        const float e = vd[i] * vw[i];
        s1 += e;
        s2 += c + i < H ? e * ((vx[i] - m) * r) : 0.f;
      }
    }
    s1 = block_sum(s1, s[0]) / H;
    s2 = block_sum(s2, s[1]) / H;
    for (int c = threadIdx.x * 8; c < H; c += 8192) {
      load8(x + row * H + c, H - c, vx);
      load8(dy + row * H + c, H - c, vd);
      load8(w + c, H - c, vw);
#pragma unroll
      for (int i = 0; i < 8; ++i) vx[i] = r * (vd[i] * vw[i] - s1 - (vx[i] - m) * r * s2);
      store8(dx + row * H + c, H - c, vx);
    }
  }
}

template <typename T>
__global__ __launch_bounds__(256) void k_norm_dw_long(const T* __restrict__ dy, const T* __restrict__ x,
                                                      const float* __restrict__ mean, const float* __restrict__ rstd,
                                                      float* __restrict__ part, int rows, int per, int H) {
  const int c = (int)blockIdx.x * 256 + threadIdx.x;
  if (c >= H) return;
  const int r0 = (int)blockIdx.y * per, r1 = min(rows, r0 + per);
  float sw = 0.f, sb = 0.f;
  for (int r = r0; r < r1; ++r) {
    const float d = load1(dy + (int64_t)r * H + c);
    sw += d * ((load1(x + (int64_t)r * H + c) - mean[r]) * rstd[r]);
    sb += d;
  }
  part[(int64_t)blockIdx.y * 2 * H + c] = sw;
  part[((int64_t)blockIdx.y * 2 + 1) * H + c] = sb;
}

// Chunks of 8 columns per thread and threads per workgroup of the one-pass kernel.
static void backward_shape(int H, int* nch, int* threads) {
  const int chunks = ceil_div(H, 8);
  *nch = chunks <= 1024 ? 1 : 4;
  *threads = ceil_div(ceil_div(chunks, *nch), 64) * 64;
}
static bool one_pass(int H, bool bf16) {
  int nch, threads;
  backward_shape(H, &nch, &threads);
  return nch == 1 || (bf16 && threads <= 512);  // fp32 rows of four chunks a thread would not fit the registers
}
// Consecutive rows of one workgroup: no more blocks than the device holds at a time.  The column
// sums of a block cost 8 H bytes twice over, a row of it 2 H bytes or more three times, so at least 8
// rows from 4096 rows on, where the blocks fill the device all the same; below, 4, for more of them
// at a time (8 instead of 4: 300 x 7168 bf16 18.1 and 13.3 us, 1000 x 7168 20.9 and 18.2, 2049 x 1021
// fp32 15.2 and 13.5; 3500 x 2048 17.9 and 18.4).  Up to 16 rows in one block, which needs no second
// launch.
static int rows_per_block(int T, int H) {
  int nch, threads;
  backward_shape(H, &nch, &threads);
  const int blocks = 256 * (threads >= 512 ? 1 : 512 / threads);
  const int per = ceil_div(T, blocks), least = T <= 16 && H <= 8192 ? 16 : T < 4096 ? 4 : 8;
  return per > least ? per : least;
}
int norm_row_blocks(int T, int H) { return ceil_div(T, rows_per_block(T, H)); }

template <typename T>
static void norm_backward(const void* dy_, const void* x_, const void* w_, const float* mean, const float* rstd,
                          void* dx_, float* part, int rows, int H, void* dw, void* db, bool grad_f32, hipStream_t st) {
  const T *dy = static_cast<const T*>(dy_), *x = static_cast<const T*>(x_), *w = static_cast<const T*>(w_);
  T* dx = static_cast<T*>(dx_);
  const int per = rows_per_block(rows, H);
  int nch, threads;
  backward_shape(H, &nch, &threads);
  const int grid = ceil_div(rows, per);
  if (nch == 1 && threads <= 256) {
    k_norm_backward<T, 1, 4, 256><<<grid, threads, 0, st>>>(dy, x, w, mean, rstd, dx, part, rows, per, H, dw, db, grad_f32);
    return;
  }
  if (nch == 1) {
    k_norm_backward<T, 1, sizeof(T) == 2 ? 2 : 1, 1024><<<grid, threads, 0, st>>>(dy, x, w, mean, rstd, dx, part, rows, per, H, dw, db, grad_f32);
    return;
  }
  if constexpr (sizeof(T) == 2) {
    if (one_pass(H, true)) {
      k_norm_backward<T, 4, 1, 512><<<grid, threads, 0, st>>>(dy, x, w, mean, rstd, dx, part, rows, per, H, dw, db, grad_f32);
      return;
    }
  }
  if (dx) k_norm_dx_long<T><<<rows < 4096 ? rows : 4096, 1024, 0, st>>>(dy, x, w, mean, rstd, dx, rows, H);
  if (part)
    k_norm_dw_long<T><<<dim3(ceil_div(H, 256), ceil_div(rows, per)), 256, 0, st>>>(dy, x, mean, rstd, part, rows, per, H);
}

hipError_t launch_norm_backward(const void* dy, const void* x, const void* w, const float* mean,
                                const float* rstd, void* dx, void* dw, void* db, bool grad_f32, float* part, int T,
                                int H, bool bf16, hipStream_t st) {
  if (!dw && !db) part = nullptr;
  if (bf16) norm_backward<uint16_t>(dy, x, w, mean, rstd, dx, part, T, H, dw, db, grad_f32, st);
  else norm_backward<float>(dy, x, w, mean, rstd, dx, part, T, H, dw, db, grad_f32, st);
  const hipError_t r = hipGetLastError();
  const int blocks = norm_row_blocks(T, H);
  if (r != hipSuccess || !part || (blocks == 1 && one_pass(H, bf16))) return r;
  return launch_col_sum(ColSum{part, blocks, H, 2 * (int64_t)H, dw, db, grad_f32}, st);
}

}  // namespace moe
