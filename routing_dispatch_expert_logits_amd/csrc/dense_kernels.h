// Internal launchers of the dense operators' kernels (layer norm, gated product, linear
// projection and their backward passes; not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "moe_device.h"

namespace moe {

// One dense product: for z < batch, C_z[m][n] = sum_{s < segs} sum_{k < K} A_zs(m, k) B_zs(n, k).
// An operand stored with the contraction index along its rows' length (A(m, k) = A[m * ld + k])
// is a row operand; one stored the other way (A(m, k) = A[k * ld + m]) is a column operand.
// With pair, batch is 1 and B[0][0], B[1][0] are the two projections of one output.
struct DenseJob {
  int M, N, K;
  int segs, batch;
  bool pair;
  bool a_col, b_col;
  const void* A[2][3];
  const void* B[2][3];
  int64_t lda, ldb;
  int b_from;   // of a column operand B: columns of its rows that lie before B (a cut's first part)
};

enum DenseEpiKind {
  DENSE_STORE = 0,   // out[z] = acc, fp32 or the layer's type
  DENSE_LINEAR = 1,  // z = acc + bias, out[0] = act(z) + residual
  DENSE_GATED = 2    // out[0] = act(acc0) * acc1
};
struct DenseEpi {
  int kind, act;
  bool out_f32;          // DENSE_STORE: fp32 output
  const void* bias;      // [N], nullable
  const void* residual;  // [M x N], nullable
  void* out[2];
  void* save[2];         // z, or g and u; nullable
  int64_t ldo;           // row length of outputs, residual and saved values
  const float* row_scale;     // integer products: a factor for each row and for each column
  const float* col_scale[2];
};

// Column sums by row blocks, not joined yet: out0[n] = sum_p part[p * stride + n] and out1[n] =
// sum_p part[p * stride + N + n] for p < P, n < N (each output nullable), in a fixed order; in
// fp32 or bf16.  P == 0: none.
struct ColSum {
  const float* part;
  int P, N;
  int64_t stride;
  void *out0, *out1;
  bool out_f32;
};

// bf16: element type of the operands and of what the epilogue reads and writes (else fp32).
// bf16: lda and ldb are whole 16-byte chunks, row operands zero from the contraction length on.
//
// Forward products of at most kDecodeRows rows read each weight once, straight into operands,
// and take rows of any length.
constexpr int kDecodeRows = 16;
hipError_t launch_dense_decode(const DenseJob& j, const DenseEpi& e, bool bf16, hipStream_t st);
//
// Products whose tiles are too few for the device are cut along the contraction; the slices'
// sums meet in `part`, dense_part_bytes of scratch for the same sizes.
size_t dense_part_bytes(bool bf16, int M, int N, int K, int segs, int batch, bool pair, bool a_col, bool backward);
hipError_t launch_dense(const DenseJob& j, const DenseEpi& e, bool bf16, float* part, hipStream_t st);
// A backward pass's dx and dw products (either NULL), in one launch where both are small; each
// with its scratch.  Their slices and the column sums that wait meet in one last launch.
struct DenseProduct {
  DenseJob j;
  DenseEpi e;
  float* part;
};
hipError_t launch_dense_grads(const DenseProduct* dx, const DenseProduct* dw, const ColSum& sum, bool bf16,
                              hipStream_t st);

// The gradient before an activation, [T x N]:
//   linear (dh == dy, u == NULL): d0 = dy act'(g);  gated: d0 = dh u act'(g), d1 = dh act(g).
// d0, d1 (nullable) get them in the layer's type with rows of ld elements.  With terms of 2
// or 3 (bf16) the second and third bf16 terms of each value follow at d + lo and d + 2 lo: three
// hold its 24 bits exactly, two a product of two bf16 numbers.  sum (nullable) receives the column
// sums of the unrounded d0 (fp32 or bf16): at once where there is one row block, else *later says what is to be joined
// (part: a row of N floats for each of the grad_row_blocks(T, N) row blocks).
// finite (bf16; src NULL: none): the T rows of src with zeros in place of infinities and NaN, in rows of
// ld elements, zeros behind the first cols: what the terms after the first are multiplied with.
struct FiniteRows {
  const void* src;
  void* dst;
  int cols;
  int64_t ld;
};
int grad_row_blocks(int T, int N);
hipError_t launch_act_grad(const void* dh, const void* g, const void* u, int act, bool bf16, int T, int N,
                           void* d0, void* d1, int terms, int64_t lo, int64_t ld, float* part, void* sum, bool sum_f32,
                           ColSum* later, const FiniteRows& finite, hipStream_t st);
hipError_t launch_col_sum(const ColSum& sum, hipStream_t st);
// dst[r][0 .. ld) = src[r][0 .. cols) and zeros for up to three bf16 operands of the same width
// (src NULL: none) in one launch; ld: cols rounded up to 8.
struct PadRows {
  const void* src[3];
  void* dst[3];
  int64_t rows[3];
};
hipError_t launch_pad_rows(const PadRows& p, int cols, int64_t ld, hipStream_t st);
hipError_t launch_fill_zero(void* p, size_t bytes, hipStream_t st);

hipError_t launch_norm_forward(const void* x, const void* w, const void* b, void* y, float* mean, float* rstd,
                               int T, int H, float eps, bool bf16, hipStream_t st);
// dx, dw and db each nullable; part: norm_row_blocks(T, H) rows of 2 H fp32 column sums.
int norm_row_blocks(int T, int H);
hipError_t launch_norm_backward(const void* dy, const void* x, const void* w, const float* mean,
                                const float* rstd, void* dx, void* dw, void* db, bool grad_f32, float* part, int T,
                                int H, bool bf16, hipStream_t st);

}  // namespace moe
