// Internal launchers of the products grouped by expert, the 8-bit integer products and the combine's
// gradients (not part of the C ABI).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "dense_kernels.h"

namespace moe {

// Rows sorted by expert: those of expert e are [offsets[e], offsets[e + 1]) of R, read on the device and
// clamped to what there is, so that no offsets reach past the rows.
struct Groups {
  const int32_t* offsets;
  int E, R;
};

// Expert e's rows: first, end.
__device__ __forceinline__ int2 group_rows(const Groups& g, int e) {
  const int lo = min(max(g.offsets[e], 0), g.R);
  return make_int2(lo, min(max(g.offsets[e + 1], lo), g.R));
}

// Element types of a grouped product's operands.
enum GroupedType { GROUPED_F32 = 0, GROUPED_BF16 = 1, GROUPED_INT8 = 2 };

// Rows by their expert's weight: job j of one expert (M unused), whose weights are w_stride elements apart and whose
// row operands and outputs are those of its rows; j.b_col: the gradient's product, across the weights' rows.
// scratch: grouped_scratch_bytes, for the table of tiles and a cut contraction's sums.  out_bf16: what an integer product's epilogue writes.
size_t grouped_scratch_bytes(GroupedType t, int R, int E, int N, int K, int segs, bool pair, bool b_col);
hipError_t launch_grouped(const DenseJob& j, const DenseEpi& e, GroupedType t, bool out_bf16, const Groups& g,
                          int64_t w_stride, void* scratch, hipStream_t st);
// Forward products of at most kDecodeRows rows, whose operands may have rows of any length (codes: whole 16-byte
// chunks): no table.  (32 rows of 8 experts, 2048 -> 768 gated: 13.0 us, 12.1 by launch_grouped; 64 of 54 of 128: 87.9 and 76.2.)  g.E == 0: dense rows, j.M of them (integers).
hipError_t launch_grouped_decode(const DenseJob& j, const DenseEpi& e, GroupedType t, bool out_bf16, const Groups& g,
                                 int64_t w_stride, hipStream_t st);
// bf16 weights [E x N x cols] (the second may be NULL) in rows of ld elements with zeros behind, ld: cols rounded up to 8;
// those of experts without rows are left out.
hipError_t launch_pad_weights(const void* w0, const void* w1, void* p0, void* p1, const Groups& g, int N, int cols, int64_t ld,
                              hipStream_t st);
// A backward pass's products, either NULL: dx as launch_grouped's with b_col, and for every expert dw's out[z][e] = sum of its
// rows' A_z x B_z, M x N (j.K unused), zeros without rows.
struct GroupedProduct {
  DenseJob j;
  DenseEpi e;
};
hipError_t launch_grouped_grads(const GroupedProduct* dx, const GroupedProduct* dw, GroupedType t, const Groups& g,
                                int64_t w_stride, void* scratch, hipStream_t st);

// Integer products of dense rows; row operands of whole 16-byte chunks, zero from the contraction length on.
hipError_t launch_int8(const DenseJob& j, const DenseEpi& e, bool out_bf16, hipStream_t st);
// Codes and scales of rows; ld: row length of q.
hipError_t launch_quantize_int8(const void* src, bool bf16, int64_t rows, int cols, int64_t ld, int8_t* q, float* scale,
                                hipStream_t st);

// dy_perm[token_row[t, j]] = topk_w[t, j] dout[t] and dtopk_w[t, j] = <dout[t], y_perm[token_row[t, j]]>, either NULL.
hipError_t launch_combine_grad(const void* dout, bool dout_f32, const void* y_perm, const int32_t* token_row,
                               const float* topk_w, int D, bool bf16, int T, int k, void* dy_perm, float* dtopk_w,
                               hipStream_t st);

}  // namespace moe
