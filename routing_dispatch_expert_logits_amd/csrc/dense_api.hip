// Host side of the dense operators' C ABI: argument validation, workspace carve-up and the
// launch sequence of each call.  No call allocates, synchronises or reads device memory.
#include <cmath>

#include "dense_kernels.h"
#include "moe.h"
#include "moe_host.h"

using namespace moe;

namespace {

// tiles of 64 rows and 16 columns: at most 2^23 of them by the elements and 2^22 more by the
// rows, so that every grid stays below 2^32 threads
constexpr int64_t kMaxRows = 1ll << 28, kMaxWidth = 1ll << 21, kMaxElems = 1ll << 33;

struct DenseDims {
  int T, K, N, act;
  bool bf16, grad_f32;
  size_t es, ges;   // element bytes of the layer, of the weight gradients
};

moe_status check_types(int dtype, int grad_dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (grad_dtype != dtype && grad_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
  return MOE_OK;
}

moe_status check_dense(const moe_dense_shape* s, DenseDims& d) {
  if (!s || s->T < 0 || s->K < 1 || s->N < 1 || s->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (s->act < MOE_ACT_NONE || s->act > MOE_ACT_GELU_TANH) return MOE_ERR_INVALID_ARG;
  if (check_types(s->dtype, s->grad_dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (s->T > kMaxRows || s->K > kMaxWidth || s->N > kMaxWidth) return MOE_ERR_UNSUPPORTED;
  if (s->T * s->K > kMaxElems || s->T * s->N > kMaxElems || s->N * s->K > kMaxElems)
    return MOE_ERR_UNSUPPORTED;
  d.T = (int)s->T; d.K = (int)s->K; d.N = (int)s->N; d.act = s->act;
  d.bf16 = s->dtype == MOE_BF16;
  d.grad_f32 = s->grad_dtype == MOE_F32;
  d.es = d.bf16 ? 2 : 4;
  d.ges = d.grad_f32 ? 4 : 2;
  return MOE_OK;
}

struct NormDims {
  int T, H;
  bool bf16, grad_f32;
  size_t es, ges;
};

moe_status check_norm(const moe_norm_shape* s, NormDims& d) {
  if (!s || s->T < 0 || s->H < 1 || s->reserved != 0) return MOE_ERR_INVALID_ARG;
  if (!(s->eps >= 0.f) || std::isinf(s->eps)) return MOE_ERR_INVALID_ARG;
  if (check_types(s->dtype, s->grad_dtype) != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (s->T > kMaxRows || s->H > kMaxWidth || s->T * s->H > kMaxElems) return MOE_ERR_UNSUPPORTED;
  d.T = (int)s->T; d.H = (int)s->H;
  d.bf16 = s->dtype == MOE_BF16;
  d.grad_f32 = s->grad_dtype == MOE_F32;
  d.es = d.bf16 ? 2 : 4;
  d.ges = d.grad_f32 ? 4 : 2;
  return MOE_OK;
}

// The buffers of one call: every one given is 16-byte aligned, and no output overlaps
// another buffer.
struct Buffers {
  struct One { uintptr_t lo, hi; bool out; } v[12];
  int n = 0;
  bool ok = true;
  void add(const void* p, size_t bytes, bool out, bool required) {
    if (!p) { ok = ok && !required; return; }
    ok = ok && al16(p);
    const uintptr_t a = reinterpret_cast<uintptr_t>(p);
    v[n++] = One{a, a + bytes, out};
  }
  void in(const void* p, size_t bytes, bool required = true) { add(p, bytes, false, required); }
  void out(const void* p, size_t bytes, bool required = true) { add(p, bytes, true, required); }
  moe_status status() const {
    if (!ok) return MOE_ERR_INVALID_ARG;
    for (int a = 0; a < n; ++a)
      for (int b = a + 1; b < n; ++b)
        if ((v[a].out || v[b].out) && v[a].lo < v[b].hi && v[b].lo < v[a].hi) return MOE_ERR_INVALID_ARG;
    return MOE_OK;
  }
};

moe_status check_ws(Buffers& b, const void* ws, size_t ws_bytes, size_t need) {
  if (b.status() != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (need == 0) return MOE_OK;
  if (!ws || ws_bytes < need) return MOE_ERR_WORKSPACE;
  b.out(ws, need);
  return b.status();
}

// ---- workspaces

// The bf16 products read rows of whole 16-byte chunks; operands with other widths are copied to
// such rows first.
int64_t padded(const DenseDims& d, int cols) { return d.bf16 ? ((int64_t)cols + 7) / 8 * 8 : cols; }

// Backward: the gradient before the activation as operand of the products (in bf16 terms of
// each value, lo elements apart, where fp32 weight gradients are asked for), and the row
// blocks' column sums.  finite: x with zeros for infinities and NaN, which the terms after the first
// are multiplied with: a zero or a term of the other sign would make NaN of what an infinite x has
// already made infinite in the first term's product.  slices, slices_w: the products' contraction
// slices (dw's in slices_w).  x, w[2]: padded copies (0 bytes where the operand is read in place).
struct DenseWs {
  size_t x, w[2], d0, d1, finite, part, slices, slices_w, total;
  int terms;
  int64_t lo, ldk, ldn;
};
// bf16 terms that hold the fp32 gradient before the activation exactly: with a slope of 0 or 1
// it is dy itself, or in a gated product one of two bf16 numbers (16 significant bits).
int grad_terms(int act, bool gated) {
  const bool slope01 = act == MOE_ACT_NONE || act == MOE_ACT_RELU;
  return slope01 ? (gated ? 2 : 1) : 3;
}

DenseWs dense_ws(const DenseDims& d, bool gated, bool backward) {
  Carve c; DenseWs w{};
  w.ldk = padded(d, d.K);
  w.ldn = padded(d, d.N);
  const bool decode = !backward && d.T <= kDecodeRows;
  if (decode) w.ldk = d.K;  // its kernel takes rows of any length
  const bool pad_k = w.ldk != d.K;
  w.x = c.take(pad_k ? (size_t)d.T * w.ldk * d.es : 0);
  w.w[0] = c.take(pad_k ? (size_t)d.N * w.ldk * d.es : 0);
  w.w[1] = c.take(pad_k && gated ? (size_t)d.N * w.ldk * d.es : 0);
  if (backward) {
    const bool through = gated || d.act != MOE_ACT_NONE;
    w.terms = d.bf16 && d.grad_f32 ? grad_terms(d.act, gated) : 1;
    w.lo = (int64_t)(align_up((size_t)d.T * w.ldn * d.es) / d.es);
    const size_t bytes = through || w.ldn != d.N ? (size_t)w.lo * d.es * w.terms : 0;
    w.d0 = c.take(bytes);
    w.d1 = c.take(gated ? bytes : 0);
    w.finite = c.take(w.terms > 1 ? (size_t)d.T * w.ldk * d.es : 0);
    w.part = c.take(gated || d.T == 0 ? 0 : (size_t)grad_row_blocks(d.T, d.N) * d.N * 4);
  }
  if (d.T > 0 && !decode) {
    const int z = gated ? 2 : 1;
    w.slices = c.take(backward ? dense_part_bytes(d.bf16, d.T, d.K, d.N, z, 1, false, false, true)
                               : dense_part_bytes(d.bf16, d.T, d.N, d.K, 1, 1, gated, false, false));
    w.slices_w = c.take(backward ? dense_part_bytes(d.bf16, d.N, d.K, d.T, w.terms, z, false, true, true) : 0);
  }
  w.total = c.cur;
  return w;
}

// x and the weights (each nullable) at row length w.ldk: in place, or copied to the workspace.
moe_status in_rows(const DenseDims& d, const DenseWs& w, const void** x, const void** w0, const void** w1, void* ws,
                   hipStream_t st) {
  if (w.ldk == d.K) return MOE_OK;
  PadRows p{};
  auto one = [&](int i, const void** v, int64_t rows, size_t off) {
    if (!v || !*v) return;
    p.src[i] = *v;
    p.dst[i] = at<void>(ws, off);
    p.rows[i] = rows;
    *v = p.dst[i];
  };
  one(0, x, d.T, w.x);
  one(1, w0, d.N, w.w[0]);
  one(2, w1, d.N, w.w[1]);
  MOE_HIP(launch_pad_rows(p, d.K, w.ldk, st));
  return MOE_OK;
}

FiniteRows finite_x(const DenseDims& d, const DenseWs& w, int terms, const void* x, void* ws) {
  return terms > 1 ? FiniteRows{x, at<void>(ws, w.finite), d.K, w.ldk} : FiniteRows{};
}

size_t norm_ws(const NormDims& d) {
  return d.T == 0 ? 0 : align_up((size_t)norm_row_blocks(d.T, d.H) * 2 * d.H * 4);
}

#define MOE_TRY(call)                                         \
  do {                                                        \
    if (const moe_status r = (call); r != MOE_OK) return r;   \
  } while (0)

// z = x w0^T (and x w1^T) with epilogue e.
moe_status forward(const DenseDims& d, const DenseWs& w, const void* x, const void* w0, const void* w1,
                   const DenseEpi& e, void* ws, hipStream_t st) {
  MOE_TRY(in_rows(d, w, &x, &w0, &w1, ws, st));
  DenseJob j{};
  j.M = d.T; j.N = d.N; j.K = d.K;
  j.segs = 1; j.batch = 1;
  j.pair = w1 != nullptr;
  j.A[0][0] = x; j.lda = w.ldk;
  j.B[0][0] = w0; j.B[1][0] = w1; j.ldb = w.ldk;
  MOE_HIP(d.T <= kDecodeRows ? launch_dense_decode(j, e, d.bf16, st)
                                : launch_dense(j, e, d.bf16, at<float>(ws, w.slices), st));
  return MOE_OK;
}

// dx = d0 w0 (+ d1 w1), the contraction over N, across the weights' rows, and dw_z = (sum of
// d_z's terms)^T x, the contraction over the tokens, across both operands' rows.  dx or dw0
// may be NULL.  sum: column sums still to be joined.
moe_status gradients(const DenseDims& d, const DenseWs& w, const void* d0, const void* d1, int terms, const void* x,
                     const void* w0, const void* w1, void* dx, void* dw0, void* dw1, const ColSum& sum, void* ws,
                     hipStream_t st) {
  MOE_TRY(in_rows(d, w, dw0 ? &x : nullptr, dx ? &w0 : nullptr, dx ? &w1 : nullptr, ws, st));
  DenseProduct px{}, pw{};
  DenseJob &jx = px.j, &jw = pw.j;
  DenseEpi &ex = px.e, &ew = pw.e;
  jx.M = d.T; jx.N = d.K; jx.K = d.N;
  jx.segs = d1 ? 2 : 1; jx.batch = 1;
  jx.b_col = true;
  jx.A[0][0] = d0; jx.A[0][1] = d1; jx.lda = w.ldn;
  jx.B[0][0] = w0; jx.B[0][1] = w1; jx.ldb = w.ldk;
  ex.kind = DENSE_STORE;
  ex.out_f32 = !d.bf16;
  ex.out[0] = dx;
  ex.ldo = ew.ldo = d.K;
  jw.M = d.N; jw.N = d.K; jw.K = d.T;
  jw.segs = terms; jw.batch = d1 ? 2 : 1;
  jw.a_col = jw.b_col = true;
  for (int q = 0; q < terms; ++q) {
    jw.A[0][q] = static_cast<const char*>(d0) + q * w.lo * d.es;
    if (d1) jw.A[1][q] = static_cast<const char*>(d1) + q * w.lo * d.es;
    jw.B[0][q] = jw.B[1][q] = q ? at<void>(ws, w.finite) : x;
  }
  jw.lda = w.ldn;
  jw.ldb = w.ldk;
  ew.kind = DENSE_STORE;
  ew.out_f32 = d.grad_f32;
  ew.out[0] = dw0; ew.out[1] = dw1;
  px.part = at<float>(ws, w.slices);
  pw.part = at<float>(ws, w.slices_w);
  MOE_HIP(launch_dense_grads(dx ? &px : nullptr, dw0 ? &pw : nullptr, sum, d.bf16, st));
  return MOE_OK;
}

}  // namespace

extern "C" {

size_t moe_dense_workspace_bytes(const moe_dense_shape* s, int call) {
  DenseDims d;
  if (check_dense(s, d) != MOE_OK) return 0;
  switch (call) {
    case MOE_CALL_GATED_FORWARD: return dense_ws(d, true, false).total;
    case MOE_CALL_GATED_BACKWARD: return dense_ws(d, true, true).total;
    case MOE_CALL_LINEAR_FORWARD: return dense_ws(d, false, false).total;
    case MOE_CALL_LINEAR_BACKWARD: return dense_ws(d, false, true).total;
    default: return 0;
  }
}

size_t moe_norm_workspace_bytes(const moe_norm_shape* s) {
  NormDims d;
  return check_norm(s, d) == MOE_OK ? norm_ws(d) : 0;
}

moe_status moe_layer_norm_forward(const void* x, const void* w, const void* b, void* y, float* mean,
                                  float* rstd, const moe_norm_shape* s, void* stream) {
  NormDims d;
  MOE_TRY(check_norm(s, d));
  const size_t rows = (size_t)d.T * d.H * d.es;
  Buffers bufs;
  bufs.in(x, rows, d.T > 0);
  bufs.in(w, d.H * d.es);
  bufs.in(b, d.H * d.es, false);
  bufs.out(y, rows, d.T > 0);
  bufs.out(mean, (size_t)d.T * 4, false);
  bufs.out(rstd, (size_t)d.T * 4, false);
  if (bufs.status() != MOE_OK) return MOE_ERR_INVALID_ARG;
  if (d.T == 0) return MOE_OK;
  MOE_HIP(launch_norm_forward(x, w, b, y, mean, rstd, d.T, d.H, s->eps, d.bf16, (hipStream_t)stream));
  return MOE_OK;
}

moe_status moe_layer_norm_backward(const void* dy, const void* x, const void* w, const float* mean,
                                   const float* rstd, void* dx, void* dw, void* db,
                                   const moe_norm_shape* s, void* ws, size_t ws_bytes, void* stream) {
  NormDims d;
  MOE_TRY(check_norm(s, d));
  const size_t rows = (size_t)d.T * d.H * d.es;
  Buffers bufs;
  bufs.in(dy, rows, d.T > 0);
  bufs.in(x, rows, d.T > 0);
  bufs.in(w, d.H * d.es);
  bufs.in(mean, (size_t)d.T * 4, d.T > 0);
  bufs.in(rstd, (size_t)d.T * 4, d.T > 0);
  bufs.out(dx, rows, false);
  bufs.out(dw, d.H * d.ges, false);
  bufs.out(db, d.H * d.ges, false);
  if (!dx && !dw && !db) return MOE_ERR_INVALID_ARG;
  MOE_TRY(check_ws(bufs, ws, ws_bytes, norm_ws(d)));
  const hipStream_t st = (hipStream_t)stream;
  if (d.T == 0) {
    if (dw) MOE_HIP(launch_fill_zero(dw, d.H * d.ges, st));
    if (db) MOE_HIP(launch_fill_zero(db, d.H * d.ges, st));
    return MOE_OK;
  }
  MOE_HIP(launch_norm_backward(dy, x, w, mean, rstd, dx, dw, db, d.grad_f32, static_cast<float*>(ws), d.T, d.H, d.bf16,
                               st));
  return MOE_OK;
}

moe_status moe_gated_forward(const void* x, const void* w1, const void* w3, void* h, void* g, void* u,
                             const moe_dense_shape* s, void* ws, size_t ws_bytes, void* stream) {
  DenseDims d;
  MOE_TRY(check_dense(s, d));
  const size_t wide = (size_t)d.T * d.N * d.es, wb = (size_t)d.N * d.K * d.es;
  Buffers bufs;
  bufs.in(x, (size_t)d.T * d.K * d.es, d.T > 0);
  bufs.in(w1, wb);
  bufs.in(w3, wb);
  bufs.out(h, wide, d.T > 0);
  bufs.out(g, wide, false);
  bufs.out(u, wide, false);
  if (!g != !u) return MOE_ERR_INVALID_ARG;
  const DenseWs w = dense_ws(d, true, false);
  MOE_TRY(check_ws(bufs, ws, ws_bytes, w.total));
  if (d.T == 0) return MOE_OK;
  DenseEpi e{};
  e.kind = DENSE_GATED;
  e.act = d.act;
  e.ldo = d.N;
  e.out[0] = h; e.save[0] = g; e.save[1] = u;
  return forward(d, w, x, w1, w3, e, ws, (hipStream_t)stream);
}

moe_status moe_gated_backward(const void* dh, const void* x, const void* w1, const void* w3, const void* g,
                              const void* u, void* dx, void* dw1, void* dw3, const moe_dense_shape* s,
                              void* ws, size_t ws_bytes, void* stream) {
  DenseDims d;
  MOE_TRY(check_dense(s, d));
  const size_t wide = (size_t)d.T * d.N * d.es, wb = (size_t)d.N * d.K * d.es;
  const size_t gb = (size_t)d.N * d.K * d.ges, xb = (size_t)d.T * d.K * d.es;
  Buffers bufs;
  bufs.in(dh, wide, d.T > 0);
  bufs.in(x, xb, d.T > 0);
  bufs.in(w1, wb);
  bufs.in(w3, wb);
  bufs.in(g, wide, d.T > 0);
  bufs.in(u, wide, d.T > 0);
  bufs.out(dx, xb, false);
  bufs.out(dw1, gb, false);
  bufs.out(dw3, gb, false);
  if (!dw1 != !dw3 || (!dx && !dw1)) return MOE_ERR_INVALID_ARG;
  const DenseWs w = dense_ws(d, true, true);
  MOE_TRY(check_ws(bufs, ws, ws_bytes, w.total));
  const hipStream_t st = (hipStream_t)stream;
  if (d.T == 0) {
    if (dw1) MOE_HIP(launch_fill_zero(dw1, gb, st));
    if (dw3) MOE_HIP(launch_fill_zero(dw3, gb, st));
    return MOE_OK;
  }
  const int terms = dw1 ? w.terms : 1;
  void *d0 = at<void>(ws, w.d0), *d1 = at<void>(ws, w.d1);
  MOE_HIP(launch_act_grad(dh, g, u, d.act, d.bf16, d.T, d.N, d0, d1, terms, w.lo, w.ldn, nullptr, nullptr,
                          false, nullptr, finite_x(d, w, terms, x, ws), st));
  return gradients(d, w, d0, d1, terms, x, w1, w3, dx, dw1, dw3, ColSum{}, ws, st);
}

moe_status moe_linear_forward(const void* x, const void* w, const void* bias, const void* residual, void* y,
                              void* z, const moe_dense_shape* s, void* ws, size_t ws_bytes, void* stream) {
  DenseDims d;
  MOE_TRY(check_dense(s, d));
  const size_t wide = (size_t)d.T * d.N * d.es;
  Buffers bufs;
  bufs.in(x, (size_t)d.T * d.K * d.es, d.T > 0);
  bufs.in(w, (size_t)d.N * d.K * d.es);
  bufs.in(bias, d.N * d.es, false);
  if (residual != y) bufs.in(residual, wide, false);  // y in place of its residual
  bufs.out(y, wide, d.T > 0);
  bufs.out(z, wide, false);
  const DenseWs p = dense_ws(d, false, false);
  MOE_TRY(check_ws(bufs, ws, ws_bytes, p.total));
  if (d.T == 0) return MOE_OK;
  DenseEpi e{};
  e.kind = DENSE_LINEAR;
  e.act = d.act;
  e.ldo = d.N;
  e.bias = bias; e.residual = residual;
  e.out[0] = y; e.save[0] = z;
  return forward(d, p, x, w, nullptr, e, ws, (hipStream_t)stream);
}

moe_status moe_linear_backward(const void* dy, const void* x, const void* w, const void* z, void* dx, void* dw,
                               void* dbias, const moe_dense_shape* s, void* ws, size_t ws_bytes,
                               void* stream) {
  DenseDims d;
  MOE_TRY(check_dense(s, d));
  const size_t wide = (size_t)d.T * d.N * d.es, gb = (size_t)d.N * d.K * d.ges, xb = (size_t)d.T * d.K * d.es;
  const bool through = d.act != MOE_ACT_NONE;
  Buffers bufs;
  bufs.in(dy, wide, d.T > 0);
  bufs.in(x, xb, d.T > 0 && dw);
  bufs.in(w, (size_t)d.N * d.K * d.es, d.T > 0 && dx);
  bufs.in(z, wide, d.T > 0 && through);
  bufs.out(dx, xb, false);
  bufs.out(dw, gb, false);
  bufs.out(dbias, d.N * d.ges, false);
  if ((!dx && !dw && !dbias) || (!through && z)) return MOE_ERR_INVALID_ARG;
  const DenseWs p = dense_ws(d, false, true);
  MOE_TRY(check_ws(bufs, ws, ws_bytes, p.total));
  const hipStream_t st = (hipStream_t)stream;
  if (d.T == 0) {
    if (dw) MOE_HIP(launch_fill_zero(dw, gb, st));
    if (dbias) MOE_HIP(launch_fill_zero(dbias, d.N * d.ges, st));
    return MOE_OK;
  }
  // the operand of the products: dy itself, or dz (or padded rows of dy) in the workspace
  const bool operand = (through || p.ldn != d.N) && (dx || dw);
  void* d0 = operand ? at<void>(ws, p.d0) : nullptr;
  const int terms = dw ? p.terms : 1;
  ColSum sum{};
  if (operand || dbias)
    MOE_HIP(launch_act_grad(dy, through ? z : nullptr, nullptr, d.act, d.bf16, d.T, d.N, d0, nullptr, terms, p.lo,
                            p.ldn, at<float>(ws, p.part), dbias, d.grad_f32, &sum, finite_x(d, p, terms, x, ws), st));
  if (!dx && !dw) {
    MOE_HIP(launch_col_sum(sum, st));
    return MOE_OK;
  }
  return gradients(d, p, operand ? d0 : dy, nullptr, terms, x, w, nullptr, dx, dw, nullptr, sum, ws, st);
}

}  // extern "C"
