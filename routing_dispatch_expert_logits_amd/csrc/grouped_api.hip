// Host side of the C ABI of the products grouped by expert and of the 8-bit integer products: argument
// validation, workspace carve-up and the launch sequence of each call.  No call allocates,
// synchronises or reads device memory.
#include "dense_host.h"
#include "grouped_kernels.h"

using namespace moe;

namespace {

constexpr int64_t kMaxInt8Width = 1ll << 17;  // 127^2 times this is below 2^31
// Columns of all experts: with the limits of the dense products, fewer than 2^24 tiles of 64 x 32 of any product, so
// that every grid stays below 2^32 threads.
constexpr int64_t kMaxExpertWidth = 1ll << 27;

struct GroupedDims {
  int R, K, N, E, act;
  bool bf16, grad_f32;
  size_t es, ges;   // element bytes of the layer, of the weight gradients
};

moe_status check_grouped(const moe_grouped_shape* s, bool gated, GroupedDims& d) {
  if (!s || s->R < 0 || s->K < 1 || s->N < 1 || s->E < 1 || s->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (!gated && s->act != MOE_ACT_NONE) return MOE_ERR_INVALID_ARG;
  if (check_types(s->dtype, s->grad_dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (s->E > kMaxE || s->R > kMaxRows || s->K > kMaxWidth || s->N > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (s->R * s->K > kMaxElems || s->R * s->N > kMaxElems || s->N * s->K > kMaxElems / s->E) return MOE_ERR_UNSUPPORTED;
  if (s->E * s->N > kMaxExpertWidth || s->E * s->K > kMaxExpertWidth) return MOE_ERR_UNSUPPORTED;
  d.R = (int)s->R; d.K = (int)s->K; d.N = (int)s->N; d.E = (int)s->E; d.act = s->act;
  d.bf16 = s->dtype == MOE_BF16;
  d.grad_f32 = s->grad_dtype == MOE_F32;
  d.es = d.bf16 ? 2 : 4;
  d.ges = d.grad_f32 ? 4 : 2;
  return MOE_OK;
}

moe_status check_dense_int8(const moe_dense_shape* s) {
  if (!s || s->T < 0 || s->K < 1 || s->N < 1 || s->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (check_types(s->dtype, s->grad_dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (s->T > kMaxRows || s->K > kMaxInt8Width || s->N > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (s->T * s->K > kMaxElems || s->T * s->N > kMaxElems || s->N * s->K > kMaxElems) return MOE_ERR_UNSUPPORTED;
  return MOE_OK;
}

int64_t padded(bool bf16, int cols) { return bf16 ? ((int64_t)cols + 7) / 8 * 8 : cols; }
int64_t code_bytes(int64_t cols) { return (cols + 15) / 16 * 16; }

// x, w[2]: padded copies (0 bytes where the operand is read in place); d0, d1: the gradient before the
// activation as operand of the products, lo elements between its terms; finite: x with zeros for infinities
// and NaN, for the terms after the first; scratch: the row tiles and a cut contraction's sums.
struct GroupedWs {
  size_t x, w[2], d0, d1, finite, scratch, total;
  int terms;
  int64_t lo, ldk, ldn;
};

GroupedWs grouped_ws(const GroupedDims& d, bool gated, bool backward, bool int8) {
  Carve c; GroupedWs w{};
  const GroupedType t = int8 ? GROUPED_INT8 : d.bf16 ? GROUPED_BF16 : GROUPED_F32;
  w.ldk = int8 ? code_bytes(d.K) : padded(d.bf16, d.K);
  w.ldn = padded(d.bf16, d.N);
  const bool decode = !backward && d.R <= kDecodeRows;
  if (decode && !int8) w.ldk = d.K;  // its kernel takes rows of any length
  const bool pad_k = !int8 && w.ldk != d.K;
  w.x = c.take(pad_k ? (size_t)d.R * w.ldk * d.es : 0);
  for (int i = 0; i < (gated ? 2 : 1); ++i) w.w[i] = c.take(pad_k ? (size_t)d.E * d.N * w.ldk * d.es : 0);
  if (backward) {
    w.terms = d.bf16 && d.grad_f32 ? grad_terms(d.act, gated) : 1;
    w.lo = (int64_t)(align_up((size_t)d.R * w.ldn * d.es) / d.es);
    const size_t bytes = gated || w.ldn != d.N ? (size_t)w.lo * d.es * w.terms : 0;
    w.d0 = c.take(bytes);
    w.d1 = c.take(gated ? bytes : 0);
    w.finite = c.take(w.terms > 1 ? (size_t)d.R * w.ldk * d.es : 0);
  }
  w.scratch = c.take(d.R == 0 || decode ? 0
                   : backward ? grouped_scratch_bytes(t, d.R, d.E, d.K, d.N, gated ? 2 : 1, false, true)
                              : grouped_scratch_bytes(t, d.R, d.E, d.N, d.K, 1, gated, false));
  w.total = c.cur;
  return w;
}

// x and the weights (each nullable) at row length w.ldk: in place, or copied to the workspace.
moe_status in_rows(const GroupedDims& d, const GroupedWs& w, const Groups& g, const void** x, const void** w0, const void** w1,
                   void* ws, hipStream_t st) {
  if (w.ldk == d.K) return MOE_OK;
  if (x) {
    const PadRows p{{*x}, {at<void>(ws, w.x)}, {d.R}};
    MOE_HIP(launch_pad_rows(p, d.K, w.ldk, st));
    *x = p.dst[0];
  }
  if (w0) {
    void *p0 = at<void>(ws, w.w[0]), *p1 = at<void>(ws, w.w[1]);
    MOE_HIP(launch_pad_weights(*w0, *w1, p0, p1, g, d.N, d.K, w.ldk, st));
    *w0 = p0;
    if (*w1) *w1 = p1;
  }
  return MOE_OK;
}

moe_status forward(const GroupedDims& d, const GroupedWs& w, GroupedType t, const void* x, const int32_t* offsets,
                   const void* w0, const void* w1, DenseEpi e, void* ws, hipStream_t st) {
  const Groups g{offsets, d.E, d.R};
  if (t != GROUPED_INT8) MOE_TRY(in_rows(d, w, g, &x, &w0, &w1, ws, st));
  DenseJob j{};
  j.N = d.N; j.K = d.K;
  j.segs = 1; j.batch = 1;
  j.pair = w1 != nullptr;
  j.A[0][0] = x; j.lda = w.ldk;
  j.B[0][0] = w0; j.B[1][0] = w1; j.ldb = w.ldk;
  e.kind = j.pair ? DENSE_GATED : DENSE_STORE;
  e.act = d.act;
  e.ldo = d.N;
  e.out_f32 = !d.bf16;
  const int64_t w_stride = (int64_t)d.N * w.ldk;
  MOE_HIP(d.R <= kDecodeRows ? launch_grouped_decode(j, e, t, d.bf16, g, w_stride, st)
                                    : launch_grouped(j, e, t, d.bf16, g, w_stride, at<void>(ws, w.scratch), st));
  return MOE_OK;
}

// dx = d0 w0 (+ d1 w1) by rows and dw_z[e] = (sum of d_z's terms)^T x over the rows of e; dx or dw0 may be NULL.
moe_status gradients(const GroupedDims& d, const GroupedWs& w, const void* d0, const void* d1, int terms, const void* x,
                     const int32_t* offsets, const void* w0, const void* w1, void* dx, void* dw0, void* dw1, void* ws,
                     hipStream_t st) {
  const GroupedType t = d.bf16 ? GROUPED_BF16 : GROUPED_F32;
  const Groups g{offsets, d.E, d.R};
  MOE_TRY(in_rows(d, w, g, dw0 ? &x : nullptr, dx ? &w0 : nullptr, dx ? &w1 : nullptr, ws, st));
  GroupedProduct px{}, pw{};
  DenseJob &jx = px.j, &jw = pw.j;
  px.e.kind = pw.e.kind = DENSE_STORE;
  px.e.ldo = pw.e.ldo = d.K;
  jx.N = d.K; jx.K = d.N;
  jx.segs = d1 ? 2 : 1; jx.batch = 1;
  jx.b_col = true;
  jx.A[0][0] = d0; jx.A[0][1] = d1; jx.lda = w.ldn;
  jx.B[0][0] = w0; jx.B[0][1] = w1; jx.ldb = w.ldk;
  px.e.out_f32 = !d.bf16;
  px.e.out[0] = dx;
  jw.M = d.N; jw.N = d.K;
  jw.segs = terms; jw.batch = d1 ? 2 : 1;
  jw.a_col = jw.b_col = true;
  for (int q = 0; q < terms; ++q) {
    jw.A[0][q] = static_cast<const char*>(d0) + q * w.lo * d.es;
    if (d1) jw.A[1][q] = static_cast<const char*>(d1) + q * w.lo * d.es;
    jw.B[0][q] = jw.B[1][q] = q ? at<void>(ws, w.finite) : x;
  }
  jw.lda = w.ldn;
  jw.ldb = w.ldk;
  pw.e.out_f32 = d.grad_f32;
  pw.e.out[0] = dw0; pw.e.out[1] = dw1;
  MOE_HIP(launch_grouped_grads(dx ? &px : nullptr, dw0 ? &pw : nullptr, t, g, (int64_t)d.N * w.ldk, at<void>(ws, w.scratch), st));
  return MOE_OK;
}

FiniteRows finite_x(const GroupedDims& d, const GroupedWs& w, int terms, const void* x, void* ws) {
  return terms > 1 ? FiniteRows{x, at<void>(ws, w.finite), d.K, w.ldk} : FiniteRows{};
}

size_t offset_bytes(const GroupedDims& d) { return (size_t)(d.E + 1) * 4; }
size_t weight_elems(const GroupedDims& d) { return (size_t)d.E * d.N * d.K; }

}  // namespace

extern "C" {

size_t moe_grouped_workspace_bytes(const moe_grouped_shape* s, int call) {
  const bool gated = call == MOE_CALL_GROUPED_GATED_FORWARD || call == MOE_CALL_GROUPED_GATED_BACKWARD ||
                     call == MOE_CALL_GROUPED_GATED_INT8;
  const bool int8 = call == MOE_CALL_GROUPED_LINEAR_INT8 || call == MOE_CALL_GROUPED_GATED_INT8;
  const bool backward = call == MOE_CALL_GROUPED_LINEAR_BACKWARD || call == MOE_CALL_GROUPED_GATED_BACKWARD;
  GroupedDims d;
  if (call < MOE_CALL_GROUPED_LINEAR_FORWARD || call > MOE_CALL_GROUPED_GATED_INT8) return 0;
  if (check_grouped(s, gated, d) != MOE_OK || (int8 && d.K > kMaxInt8Width)) return 0;
  return grouped_ws(d, gated, backward, int8).total;
}

moe_status moe_grouped_linear_forward(const void* x, const int32_t* offsets, const void* w, void* y,
                                      const moe_grouped_shape* s, void* ws, size_t ws_bytes, void* stream) {
  GroupedDims d;
  MOE_TRY(check_grouped(s, false, d));
  Buffers b;
  b.in(x, (size_t)d.R * d.K * d.es, d.R > 0);
  b.in(offsets, offset_bytes(d));
  b.in(w, weight_elems(d) * d.es);
  b.out(y, (size_t)d.R * d.N * d.es, d.R > 0);
  const GroupedWs p = grouped_ws(d, false, false, false);
  MOE_TRY(check_ws(b, ws, ws_bytes, p.total));
  if (d.R == 0) return MOE_OK;
  DenseEpi e{};
  e.out[0] = y;
  return forward(d, p, d.bf16 ? GROUPED_BF16 : GROUPED_F32, x, offsets, w, nullptr, e, ws, (hipStream_t)stream);
}

moe_status moe_grouped_linear_backward(const void* dy, const void* x, const int32_t* offsets, const void* w, void* dx,
                                       void* dw, const moe_grouped_shape* s, void* ws, size_t ws_bytes, void* stream) {
  GroupedDims d;
  MOE_TRY(check_grouped(s, false, d));
  const size_t gb = weight_elems(d) * d.ges, xb = (size_t)d.R * d.K * d.es;
  Buffers b;
  b.in(dy, (size_t)d.R * d.N * d.es, d.R > 0);
  b.in(x, xb, d.R > 0 && dw);
  b.in(offsets, offset_bytes(d));
  b.in(w, weight_elems(d) * d.es, d.R > 0 && dx);
  b.out(dx, xb, false);
  b.out(dw, gb, false);
  if (!dx && !dw) return MOE_ERR_INVALID_ARG;
  const GroupedWs p = grouped_ws(d, false, true, false);
  MOE_TRY(check_ws(b, ws, ws_bytes, p.total));
  const hipStream_t st = (hipStream_t)stream;
  if (d.R == 0) {
    if (dw) MOE_HIP(launch_fill_zero(dw, gb, st));
    return MOE_OK;
  }
  const void* d0 = dy;
  if (p.ldn != d.N) {
    void* rows = at<void>(ws, p.d0);
    MOE_HIP(launch_act_grad(dy, nullptr, nullptr, MOE_ACT_NONE, d.bf16, d.R, d.N, rows, nullptr, 1, p.lo, p.ldn, nullptr,
                            nullptr, false, nullptr, FiniteRows{}, st));
    d0 = rows;
  }
  return gradients(d, p, d0, nullptr, 1, x, offsets, w, nullptr, dx, dw, nullptr, ws, st);
}

moe_status moe_grouped_gated_forward(const void* x, const int32_t* offsets, const void* w1, const void* w3, void* h,
                                     void* g, void* u, const moe_grouped_shape* s, void* ws, size_t ws_bytes,
                                     void* stream) {
  GroupedDims d;
  MOE_TRY(check_grouped(s, true, d));
  const size_t wide = (size_t)d.R * d.N * d.es;
  Buffers b;
  b.in(x, (size_t)d.R * d.K * d.es, d.R > 0);
  b.in(offsets, offset_bytes(d));
  b.in(w1, weight_elems(d) * d.es);
  b.in(w3, weight_elems(d) * d.es);
  b.out(h, wide, d.R > 0);
  b.out(g, wide, false);
  b.out(u, wide, false);
  if (!g != !u) return MOE_ERR_INVALID_ARG;
  const GroupedWs p = grouped_ws(d, true, false, false);
  MOE_TRY(check_ws(b, ws, ws_bytes, p.total));
  if (d.R == 0) return MOE_OK;
  DenseEpi e{};
  e.out[0] = h; e.save[0] = g; e.save[1] = u;
  return forward(d, p, d.bf16 ? GROUPED_BF16 : GROUPED_F32, x, offsets, w1, w3, e, ws, (hipStream_t)stream);
}

moe_status moe_grouped_gated_backward(const void* dh, const void* x, const int32_t* offsets, const void* w1,
                                      const void* w3, const void* g, const void* u, void* dx, void* dw1, void* dw3,
                                      const moe_grouped_shape* s, void* ws, size_t ws_bytes, void* stream) {
  GroupedDims d;
  MOE_TRY(check_grouped(s, true, d));
  const size_t wide = (size_t)d.R * d.N * d.es, xb = (size_t)d.R * d.K * d.es;
  const size_t wb = weight_elems(d) * d.es, gb = weight_elems(d) * d.ges;
  Buffers b;
  b.in(dh, wide, d.R > 0);
  b.in(x, xb, d.R > 0 && dw1);
  b.in(offsets, offset_bytes(d));
  b.in(w1, wb, d.R > 0 && dx);
  b.in(w3, wb, d.R > 0 && dx);
  b.in(g, wide, d.R > 0);
  b.in(u, wide, d.R > 0);
  b.out(dx, xb, false);
  b.out(dw1, gb, false);
  b.out(dw3, gb, false);
  if (!dw1 != !dw3 || (!dx && !dw1)) return MOE_ERR_INVALID_ARG;
  const GroupedWs p = grouped_ws(d, true, true, false);
  MOE_TRY(check_ws(b, ws, ws_bytes, p.total));
  const hipStream_t st = (hipStream_t)stream;
  if (d.R == 0) {
    if (dw1) MOE_HIP(launch_fill_zero(dw1, gb, st));
    if (dw3) MOE_HIP(launch_fill_zero(dw3, gb, st));
    return MOE_OK;
  }
  // dg and du enter the bf16 products rounded to bf16, as in the dense gated backward pass: a gradient is sqrt(2) of one
  // rounding's error from its definition.  A second bf16 term of each would leave its own rounding alone, at twice the
  // products (32768 rows of 128 experts, 2048 -> 768: 2.35e-3 of the gradients' norm in 634 us, 1.66e-3 in 1055).  Weight
  // gradients asked for in fp32 take the terms that hold dg and du exactly; dx is rounded to bf16 in any case.
  const int terms = dw1 ? p.terms : 1;
  void *d0 = at<void>(ws, p.d0), *d1 = at<void>(ws, p.d1);
  MOE_HIP(launch_act_grad(dh, g, u, d.act, d.bf16, d.R, d.N, d0, d1, terms, p.lo, p.ldn, nullptr, nullptr, false, nullptr,
                          finite_x(d, p, terms, x, ws), st));
  return gradients(d, p, d0, d1, terms, x, offsets, w1, w3, dx, dw1, dw3, ws, st);
}

// ---- 8-bit integers

int64_t moe_int8_row_bytes(int64_t cols) { return cols < 1 || cols > kMaxWidth ? 0 : code_bytes(cols); }

moe_status moe_quantize_int8(const void* src, int src_dtype, int64_t rows, int64_t cols, int8_t* q, float* scale,
                             void* stream) {
  if ((src_dtype != MOE_F32 && src_dtype != MOE_BF16) || rows < 0 || cols < 1) return MOE_ERR_INVALID_ARG;
  if (cols > kMaxWidth || rows > kMaxElems / cols) return MOE_ERR_UNSUPPORTED;
  const int64_t ld = code_bytes(cols);
  Buffers b;
  b.in(src, (size_t)rows * cols * (src_dtype == MOE_BF16 ? 2 : 4), rows > 0);
  b.out(q, (size_t)rows * ld, rows > 0);
  b.out(scale, (size_t)rows * 4, rows > 0);
  MOE_TRY(b.status());
  if (rows == 0) return MOE_OK;
  MOE_HIP(launch_quantize_int8(src, src_dtype == MOE_BF16, rows, (int)cols, ld, q, scale, (hipStream_t)stream));
  return MOE_OK;
}

static moe_status int8_forward(const int8_t* x, const float* x_scale, const int8_t* w0, const float* w0_scale,
                               const int8_t* w1, const float* w1_scale, bool gated, const void* bias, const void* residual,
                               void* y, const moe_dense_shape* s, void* stream) {
  MOE_TRY(check_dense_int8(s));
  const size_t es = s->dtype == MOE_BF16 ? 2 : 4, T = (size_t)s->T, N = (size_t)s->N, ld = (size_t)code_bytes(s->K);
  Buffers b;
  b.in(x, T * ld, T > 0);
  b.in(x_scale, T * 4, T > 0);
  b.in(w0, N * ld);
  b.in(w0_scale, N * 4);
  if (gated) {
    b.in(w1, N * ld);
    b.in(w1_scale, N * 4);
  }
  b.in(bias, N * es, false);
  if (residual != y) b.in(residual, T * N * es, false);  // y in place of its residual
  b.out(y, T * N * es, T > 0);
  MOE_TRY(b.status());
  if (T == 0) return MOE_OK;
  DenseJob j{};
  j.M = (int)s->T; j.N = (int)s->N; j.K = (int)s->K;
  j.segs = 1; j.batch = 1;
  j.pair = gated;
  j.A[0][0] = x;
  j.B[0][0] = w0; j.B[1][0] = w1;
  j.lda = j.ldb = (int64_t)ld;
  DenseEpi e{};
  e.kind = gated ? DENSE_GATED : DENSE_LINEAR;
  e.act = s->act;
  e.ldo = s->N;
  e.bias = bias; e.residual = residual;
  e.out[0] = y;
  e.row_scale = x_scale; e.col_scale[0] = w0_scale; e.col_scale[1] = w1_scale;
  const hipStream_t st = (hipStream_t)stream;
  const bool bf16 = s->dtype == MOE_BF16;
  MOE_HIP(T <= (size_t)kDecodeRows ? launch_grouped_decode(j, e, GROUPED_INT8, bf16, Groups{}, 0, st) : launch_int8(j, e, bf16, st));
  return MOE_OK;
}

moe_status moe_linear_int8_forward(const int8_t* x, const float* x_scale, const int8_t* w, const float* w_scale,
                                   const void* bias, const void* residual, void* y, const moe_dense_shape* s,
                                   void* stream) {
  return int8_forward(x, x_scale, w, w_scale, nullptr, nullptr, false, bias, residual, y, s, stream);
}

moe_status moe_gated_int8_forward(const int8_t* x, const float* x_scale, const int8_t* w1, const float* w1_scale,
                                  const int8_t* w3, const float* w3_scale, void* h, const moe_dense_shape* s,
                                  void* stream) {
  return int8_forward(x, x_scale, w1, w1_scale, w3, w3_scale, true, nullptr, nullptr, h, s, stream);
}

static moe_status grouped_int8(const int8_t* x, const float* x_scale, const int32_t* offsets, const int8_t* w0,
                               const float* w0_scale, const int8_t* w1, const float* w1_scale, bool gated, void* y,
                               const moe_grouped_shape* s, void* ws, size_t ws_bytes, void* stream) {
  GroupedDims d;
  MOE_TRY(check_grouped(s, gated, d));
  if (d.K > kMaxInt8Width) return MOE_ERR_UNSUPPORTED;
  const size_t ld = (size_t)code_bytes(d.K), wn = (size_t)d.E * d.N;
  Buffers b;
  b.in(x, (size_t)d.R * ld, d.R > 0);
  b.in(x_scale, (size_t)d.R * 4, d.R > 0);
  b.in(offsets, offset_bytes(d));
  b.in(w0, wn * ld);
  b.in(w0_scale, wn * 4);
  if (gated) {
    b.in(w1, wn * ld);
    b.in(w1_scale, wn * 4);
  }
  b.out(y, (size_t)d.R * d.N * d.es, d.R > 0);
  const GroupedWs p = grouped_ws(d, gated, false, true);
  MOE_TRY(check_ws(b, ws, ws_bytes, p.total));
  if (d.R == 0) return MOE_OK;
  DenseEpi e{};
  e.out[0] = y;
  e.row_scale = x_scale; e.col_scale[0] = w0_scale; e.col_scale[1] = w1_scale;
  return forward(d, p, GROUPED_INT8, x, offsets, w0, w1, e, ws, (hipStream_t)stream);
}

moe_status moe_grouped_linear_int8_forward(const int8_t* x, const float* x_scale, const int32_t* offsets,
                                           const int8_t* w, const float* w_scale, void* y, const moe_grouped_shape* s,
                                           void* ws, size_t ws_bytes, void* stream) {
  return grouped_int8(x, x_scale, offsets, w, w_scale, nullptr, nullptr, false, y, s, ws, ws_bytes, stream);
}

moe_status moe_grouped_gated_int8_forward(const int8_t* x, const float* x_scale, const int32_t* offsets,
                                          const int8_t* w1, const float* w1_scale, const int8_t* w3,
                                          const float* w3_scale, void* h, const moe_grouped_shape* s, void* ws,
                                          size_t ws_bytes, void* stream) {
  return grouped_int8(x, x_scale, offsets, w1, w1_scale, w3, w3_scale, true, h, s, ws, ws_bytes, stream);
}

}  // extern "C"
