// Host helpers shared by the C ABI's sources: workspace carve-up, pointer checks and the
// status of a launch.
#pragma once

#include <hip/hip_runtime.h>
#include <cstddef>
#include <cstdint>

namespace {

constexpr size_t kAlign = 256;

size_t align_up(size_t x) { return (x + kAlign - 1) & ~(kAlign - 1); }

struct Carve {
  size_t cur = 0;
  size_t take(size_t bytes) {
    const size_t o = cur;
    cur = align_up(cur + bytes);
    return o;
  }
};

bool al16(const void* p) { return p && (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
bool al16_or_null(const void* p) { return !p || al16(p); }

template <typename P>
P* at(void* ws, size_t off) {
  return reinterpret_cast<P*>(static_cast<char*>(ws) + off);
}

#define MOE_HIP(call)                             \
  do {                                            \
    if ((call) != hipSuccess) return MOE_ERR_HIP; \
  } while (0)

}  // namespace
