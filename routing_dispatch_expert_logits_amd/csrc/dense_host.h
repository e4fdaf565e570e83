// Host helpers of the dense and the grouped operators' C ABI: limits, types, buffers and workspaces.
#pragma once

#include "moe.h"
#include "moe_host.h"

namespace {

// tiles of 64 rows and 16 columns: at most 2^23 of them by the elements and 2^22 more by the
// rows, so that every grid stays below 2^32 threads
constexpr int64_t kMaxRows = 1ll << 28, kMaxWidth = 1ll << 21, kMaxElems = 1ll << 33;

moe_status check_types(int dtype, int grad_dtype) {
  if (dtype != MOE_F32 && dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
  if (grad_dtype != dtype && grad_dtype != MOE_F32) return MOE_ERR_INVALID_ARG;
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

#define MOE_TRY(call)                                         \
  do {                                                        \
    if (const moe_status r = (call); r != MOE_OK) return r;   \
  } while (0)

// bf16 terms that hold the fp32 gradient before the activation exactly: with a slope of 0 or 1
// it is dy itself, or in a gated product one of two bf16 numbers (16 significant bits).
int grad_terms(int act, bool gated) {
  const bool slope01 = act == MOE_ACT_NONE || act == MOE_ACT_RELU;
  return slope01 ? (gated ? 2 : 1) : 3;
}

}  // namespace
