// Host-side argument checks shared by the C-ABI entry points.
#pragma once
#include <cmath>
#include <cstddef>
#include <cstdint>

#include "fa2.h"

namespace fa2 {

inline bool aligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) == 0; }

struct Range {
  uintptr_t lo, hi;
};
inline bool overlap(Range a, Range b) { return a.lo < b.hi && b.lo < a.hi; }
inline Range range_of(const void* p, size_t bytes) {
  const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
  return {lo, lo + bytes};
}

inline int check_scale(float scale) { return (std::isfinite(scale) && scale > 0.f) ? FA2_OK : FA2_ERR_SCALE; }

inline bool head_dim_ok(int d) { return d == 16 || d == 32 || d == 64 || d == 128; }

constexpr size_t kWsAlign = 256;
inline size_t round_up(size_t x) { return (x + kWsAlign - 1) / kWsAlign * kWsAlign; }

// Whether `count` steps of `stride` (both >= 0) stay within 2^46: products of
// sizes and strides that pass this do not overflow.
inline bool stride_ok(long long stride, long long count) {
  return stride >= 0 && (count <= 0 || stride <= (1LL << 46) / count);
}

// Query heads H, key/value heads Hkv (H a multiple of Hkv).
inline int check_heads(int H, int Hkv) { return (Hkv >= 1 && Hkv <= H && H % Hkv == 0) ? FA2_OK : FA2_ERR_SHAPE; }

}  // namespace fa2
