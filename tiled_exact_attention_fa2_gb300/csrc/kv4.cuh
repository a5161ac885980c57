// The 4-bit key-value cache: layout, number formats and the register-level
// pieces that its kernels share.
//
// Format.  A value is an e2m1 code (0, 0.5, 1, 1.5, 2, 3, 4, 6 and a sign)
// times an e4m3 scale, one scale per 16 columns of a token's head, times the
// cache's factor (k_scale, v_scale: a power of two): 4.5 bits a value.  A
// code has at most 2 significant bits and a scale 4, so a value has at most 6
// and is exact in fp16 and bf16: reading the cache rounds nothing.
//
// Layout.  16 consecutive tokens of one K/V head are one tile of 18 d bytes;
// a page of P tokens is P / 16 tiles per head, the cache
// [pages, H_kv, P / 16, 18 d].  A tile is ordered as one warp's
// mma.m16n8k16 operands, so that the attention kernel loads it straight into
// registers, lane (g, c) = (lane / 4, lane % 4), with full-width coalesced
// loads:
//   0 .. 8d     K codes [key 16][d / 2]: lane (g, c) takes columns
//               c d/4 .. of keys g and g + 8
//   8d .. 16d   V codes [t 2][g 8][c 4][p 2][d / 16]: columns g d/8 .. of
//               key 8 t + 2 c + p
//   16d .. 17d  K scales [key mod 8][column / 16][key / 8]
//   17d .. 18d  V scales [column / 16][c 4][t 2][p 2]
// A byte belongs to one token, so tokens are written without reading.
#pragma once
#include <cstdint>

#include "ptx.cuh"

namespace fa2 {

constexpr int kCacheTile = 16;  // tokens of a tile

template <int D>
struct Kv4 {
  static constexpr int kTileBytes = 18 * D;
  static constexpr int kV = 8 * D, kKS = 16 * D, kVS = 17 * D;
  static constexpr int kGroups = D / 16;  // scales of a token's head

  static __device__ __forceinline__ int k_scale_at(int key, int grp) {
    return kKS + ((key & 7) * kGroups + grp) * 2 + (key >> 3);
  }
  // (the key's place in a quad's order: t, p innermost)
  static __device__ __forceinline__ int v_scale_at(int key, int grp) {
    return kVS + (grp * 4 + ((key >> 1) & 3)) * 4 + (key >> 3) * 2 + (key & 1);
  }
  // First byte of the D / 16 code bytes of V columns g D/8 .. of a key.
  static __device__ __forceinline__ int v_piece_at(int key, int g) {
    return kV + ((((key >> 3) * 8 + g) * 4 + ((key >> 1) & 3)) * 2 + (key & 1)) * (D / 16);
  }
};

// The 8 values of four code bytes as fp16 pairs (even column low).
__device__ __forceinline__ void e2m1x8_to_f16(uint32_t w, uint32_t (&h)[4]) {
  asm("{\n .reg .b8 a, b, c, d;\n mov.b32 {a, b, c, d}, %4;\n"
      " cvt.rn.f16x2.e2m1x2 %0, a;\n cvt.rn.f16x2.e2m1x2 %1, b;\n"
      " cvt.rn.f16x2.e2m1x2 %2, c;\n cvt.rn.f16x2.e2m1x2 %3, d;\n}"
      : "=r"(h[0]), "=r"(h[1]), "=r"(h[2]), "=r"(h[3])
      : "r"(w));
}
// Two e4m3 scales (the low 16 bits) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
// The codes of 8 values given as fp16 pairs, a byte per pair: round to nearest
// even, saturating, the low half of a pair in the low half of its byte.
__device__ __forceinline__ uint32_t f16_to_e2m1x8(const uint32_t (&h)[4]) {
  uint32_t r;
  asm("{\n .reg .b8 a, b, c, d;\n cvt.rn.satfinite.e2m1x2.f16x2 a, %1;\n cvt.rn.satfinite.e2m1x2.f16x2 b, %2;\n"
      " cvt.rn.satfinite.e2m1x2.f16x2 c, %3;\n cvt.rn.satfinite.e2m1x2.f16x2 d, %4;\n mov.b32 %0, {a, b, c, d};\n}"
      : "=r"(r)
      : "r"(h[0]), "r"(h[1]), "r"(h[2]), "r"(h[3]));
  return r;
}
__device__ __forceinline__ uint32_t e4m3_of(float x) {
  uint16_t r;
  asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(0.f), "f"(x));
  return r & 0xffu;
}
// Larger of bf16 pairs, a NaN if either is one.
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ uint32_t hmul2(uint32_t a, uint32_t b) {
  uint32_t r;
  asm("mul.rn.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
__device__ __forceinline__ float2 f16x2_to_f32(uint32_t v) {
  float2 f;
  asm("{\n .reg .b16 l, h;\n mov.b32 {l, h}, %2;\n cvt.f32.f16 %0, l;\n cvt.f32.f16 %1, h;\n}"
      : "=f"(f.x), "=f"(f.y)
      : "r"(v));
  return f;
}

// The cache as its kernels see it.
struct PagedCache {
  char* base;
  long long page_stride;  // bytes
  int num_pages, shift;   // pages of 1 << shift tokens
  int heads;              // H_kv
};

// Host side (kv4_cache.cu): the checks of a cache's arguments (an fa2_status),
// of its factors, and the bytes it spans.
int check_cache(const void* cache, long long page_stride, int num_pages, int page_size, int H_kv, int d);
bool power_of_two(float x);
PagedCache paged_cache(const void* cache, long long page_stride, int num_pages, int page_size, int H_kv);
size_t cache_span(long long page_stride, int num_pages, int page_size, int H_kv, int d);

}  // namespace fa2
