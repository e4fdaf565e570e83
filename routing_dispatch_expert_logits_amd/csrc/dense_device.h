// Device helpers of the dense operators: activations, their slopes and guarded loads.
#pragma once

#include "moe.h"
#include "dense_kernels.h"
#include "moe_device.h"

namespace moe {

// e^a through the hardware exp2 (about one fp32 ulp of the argument's scale), or the
// library's correctly scaled one.
template <bool FAST>
__device__ __forceinline__ float exp_of(float a) {
  if constexpr (FAST) return __builtin_amdgcn_exp2f(a * 1.4426950408889634f);
  else return expf(a);
}
template <bool FAST>
__device__ __forceinline__ float recip(float a) {
  if constexpr (FAST) return __builtin_amdgcn_rcpf(a);
  else return 1.f / a;
}

// Phi(a), the normal distribution's mass left of a, and in *gauss e^(-a^2 / 2), which its slope
// takes too.  FAST: Phi(-|a|) = (c1 t + .. + c6 t^6) e^(-a^2 / 2) with t = 1 / (1 + p |a|), the form
// of Hastings' approximations; p and the c are a minimax fit over |a| <= 13.5 (where e^(-a^2 / 2)
// leaves the normal numbers) of the relative error below 2^-13 and the absolute one below 7.5e-8
// at once, since for negative a the result is the small tail itself (evaluated in fp32: within 9.2e-5
// of itself and 2e-7).  13 operations, where the library's erfc takes several times that and a
// 256 x 256 tile's epilogue spends about 1000 cycles for each operation per value (8192 x 2048 x
// 7168 with GELU: 241.3 us; 240.3 with one term less, which cannot hold both bounds).
template <bool FAST>
__device__ __forceinline__ float normal_mass(float a, float* gauss) {
  if constexpr (!FAST) {
    *gauss = expf(-0.5f * a * a);
    return 0.5f * erfcf(a * -0.70710678118654752f);
  } else {
    *gauss = __builtin_amdgcn_exp2f(a * a * (-0.5f * 1.4426950408889634f));
    const float t = recip<true>(1.f + 0.291f * fabsf(a));
    const float p = t * (0.117190704f + t * (0.101976506f + t * (0.176354036f + t * (-0.0864994004f +
                    t * (0.279152215f + t * -0.0881741270f)))));
    const float h = p * *gauss;
    return a >= 0.f ? 1.f - h : h;
  }
}

constexpr float kInvSqrt2Pi = 0.39894228040143268f;
constexpr float kTanhC = 1.5957691216057308f;  // 2 sqrt(2 / pi)
constexpr float kTanhA = 0.044715f;

// act(a).  ReLU keeps NaN.  The tanh form uses (1 + tanh q) / 2 = 1 / (1 + e^(-2 q)).
template <bool FAST>
__device__ __forceinline__ float act_value(float a, int act) {
  switch (act) {
    case MOE_ACT_RELU: return a < 0.f ? 0.f : a;
    case MOE_ACT_SILU: return a * recip<FAST>(1.f + exp_of<FAST>(-a));
    case MOE_ACT_GELU: {
      float gauss;
      return a * normal_mass<FAST>(a, &gauss);
    }
    case MOE_ACT_GELU_TANH:
      return a * recip<FAST>(1.f + exp_of<FAST>(-kTanhC * (a + kTanhA * a * a * a)));
    default: return a;
  }
}

// act(a) and act'(a).
template <bool FAST>
__device__ __forceinline__ float act_value_slope(float a, int act, float* slope) {
  switch (act) {
    case MOE_ACT_RELU: *slope = a > 0.f ? 1.f : 0.f; return a < 0.f ? 0.f : a;
    case MOE_ACT_SILU: {
      const float s = recip<FAST>(1.f + exp_of<FAST>(-a));
      *slope = s * (1.f + a * (1.f - s));
      return a * s;
    }
    case MOE_ACT_GELU: {
      float gauss;
      const float p = normal_mass<FAST>(a, &gauss);
      *slope = p + a * kInvSqrt2Pi * gauss;
      return a * p;
    }
    case MOE_ACT_GELU_TANH: {
      // e^(-2q) overflows to inf for very negative a: p = 0, and p (1 - p) = 0 from |a| = 16 on,
      // whose factors are held there lest a square overflows and 0 times it is NaN
      const float p = recip<FAST>(1.f + exp_of<FAST>(-kTanhC * (a + kTanhA * a * a * a)));
      const float b = fminf(fmaxf(a, -16.f), 16.f);
      *slope = p + b * p * (1.f - p) * kTanhC * (1.f + 3.f * kTanhA * b * b);
      return a * p;
    }
    default: *slope = 1.f; return a;
  }
}

// One element of the layer's type as fp32.
template <typename T>
__device__ __forceinline__ float load1(const T* p) {
  if constexpr (sizeof(T) == 2) return bf16_to_f32(*p);
  else return *p;
}
template <typename T>
__device__ __forceinline__ void store1(T* p, float v) {
  if constexpr (sizeof(T) == 2) *p = f32_to_bf16(v);
  else *p = v;
}

// Eight consecutive elements at any element-aligned address (rows of odd widths).
struct __attribute__((packed, aligned(2))) Bytes16of2 { uint32_t v[4]; };
struct __attribute__((packed, aligned(4))) Bytes16of4 { uint32_t v[4]; };
template <typename T>
__device__ __forceinline__ void load8(const T* p, float* f) {
  if constexpr (sizeof(T) == 2) {
    const Bytes16of2 b = *reinterpret_cast<const Bytes16of2*>(p);
    unpack_bf16x8(make_uint4(b.v[0], b.v[1], b.v[2], b.v[3]), f);
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      const Bytes16of4 b = reinterpret_cast<const Bytes16of4*>(p)[h];
#pragma unroll
      for (int i = 0; i < 4; ++i) f[4 * h + i] = __uint_as_float(b.v[i]);
    }
  }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const float* f) {
  if constexpr (sizeof(T) == 2) {
    Bytes16of2 b;
#pragma unroll
    for (int i = 0; i < 4; ++i)
      b.v[i] = f32_to_bf16(f[2 * i]) | (static_cast<uint32_t>(f32_to_bf16(f[2 * i + 1])) << 16);
    *reinterpret_cast<Bytes16of2*>(p) = b;
  } else {
#pragma unroll
    for (int h = 0; h < 2; ++h) {
      Bytes16of4 b;
#pragma unroll
      for (int i = 0; i < 4; ++i) b.v[i] = __float_as_uint(f[4 * h + i]);
      reinterpret_cast<Bytes16of4*>(p)[h] = b;
    }
  }
}
// The first n of eight elements (n may be <= 0 or >= 8); the others read as 0 / stay as they are.
template <typename T>
__device__ __forceinline__ void load8(const T* p, int n, float* f) {
  if (n >= 8) return load8(p, f);
#pragma unroll
  for (int i = 0; i < 8; ++i) f[i] = i < n ? load1(p + i) : 0.f;
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int n, const float* f) {
  if (n >= 8) return store8(p, f);
#pragma unroll
  for (int i = 0; i < 8; ++i)
    if (i < n) store1(p + i, f[i]);
}


// Eight elements as they are in memory: what a load in flight costs in registers.
template <typename T>
struct Raw8 {
  uint32_t v[2 * sizeof(T)];
  __device__ __forceinline__ void load(const T* p, int n) {  // the first n, zeros behind
    if (n >= 8) {
#pragma unroll
      for (int h = 0; h < (int)sizeof(T) / 2; ++h) {
        if constexpr (sizeof(T) == 2) {
          const Bytes16of2 b = *reinterpret_cast<const Bytes16of2*>(p);
#pragma unroll
          for (int i = 0; i < 4; ++i) v[i] = b.v[i];
        } else {
          const Bytes16of4 b = reinterpret_cast<const Bytes16of4*>(p)[h];
#pragma unroll
          for (int i = 0; i < 4; ++i) v[4 * h + i] = b.v[i];
        }
      }
      return;
    }
#pragma unroll
    for (int i = 0; i < (int)(2 * sizeof(T)); ++i) v[i] = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i)
      if (i < n) {
        if constexpr (sizeof(T) == 2) v[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
        else v[i] = __float_as_uint(p[i]);
      }
  }
  __device__ __forceinline__ float get(int i) const {
    if constexpr (sizeof(T) == 2) return __uint_as_float(i & 1 ? v[i / 2] & 0xffff0000u : v[i / 2] << 16);
    else return __uint_as_float(v[i]);
  }
};

// COLS columns of waiting column sums by 16 COLS threads: 16 groups of the P rows (each in
// ascending order, four loads at a time), then the groups.  half: 0 for out0, 1 for out1.
template <int COLS>
__device__ __forceinline__ void col_sum(const ColSum& c, int block, int half, float (*s)[COLS]) {
  void* out = half ? c.out1 : c.out0;
  if (!out) return;
  const int tid = threadIdx.x % COLS, q = threadIdx.x / COLS, n = block * COLS + tid;
  const float* src = c.part + (int64_t)half * c.N + min(n, c.N - 1);
  float v = 0.f;
  int p = q;
  for (; p + 48 < c.P; p += 64) {
    const float a = src[p * c.stride], b = src[(p + 16) * c.stride], d = src[(p + 32) * c.stride],
                e = src[(p + 48) * c.stride];
    v = (((v + a) + b) + d) + e;
  }
  for (; p < c.P; p += 16) v += src[p * c.stride];
  s[q][tid] = v;
  __syncthreads();
  if (q == 0 && n < c.N) {
    v = 0.f;
#pragma unroll
    for (int g = 0; g < 16; ++g) v += s[g][tid];
    if (c.out_f32) static_cast<float*>(out)[n] = v;
    else static_cast<uint16_t*>(out)[n] = f32_to_bf16(v);
  }
}

}  // namespace moe
