// Writing keys and values into the 4-bit paged cache, and reading them back
// as bf16.
//
// Both are bound by HBM: the append reads 2 bytes a value and writes 4.5
// bits (and 2 bytes more where the caller wants the stored values), the
// gather reads 4.5 bits and writes 2 bytes.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>

#include "args.h"
#include "fa2.h"
#include "kv4.cuh"
#include "launch.h"

namespace fa2 {
namespace {

__device__ int g_cache_status;

struct AppendProblem {
  const __nv_bfloat16* x[2];  // k, v [T, H_kv, d]
  long long token_stride[2], head_stride[2];
  __nv_bfloat16* out[2];  // stored values [T, H_kv, d], or NULL
  float factor[2];
  const long long* slots;
  PagedCache cache;
  long long groups;  // T * H_kv * d / 16
};

// One thread per group of 16 columns (K: blockIdx.y = 0, V: 1).  The scale is
// e4m3(max |x| / (6 f)) and a code e2m1(x / (f s)), f the cache's factor: the
// quotients are IEEE divisions, whose rounding cannot cross a border of the
// two formats (the borders have few bits, and x is bf16), so a value is
// always the nearest one, ties to even.  A group whose scale rounds to zero
// is stored as zeros; one that holds a NaN gets the NaN scale.
template <int D>
__global__ void __launch_bounds__(256) fa2_kv4_append_kernel(const AppendProblem p) {
  using L = Kv4<D>;
  griddep_wait();
  griddep_launch_dependents();
  const long long i = static_cast<long long>(blockIdx.x) * 256 + threadIdx.x;
  if (i >= p.groups) return;
  const int which = blockIdx.y;
  const int grp = static_cast<int>(i % L::kGroups);
  const long long row = i / L::kGroups;
  const long long t = row / p.cache.heads;
  const int h = static_cast<int>(row - t * p.cache.heads);
  const long long slot = __ldg(p.slots + t);
  // (selected, not indexed: an indexed parameter array is copied to the stack)
  const __nv_bfloat16* x = which ? p.x[1] : p.x[0];
  const long long token_stride = which ? p.token_stride[1] : p.token_stride[0];
  const long long head_stride = which ? p.head_stride[1] : p.head_stride[0];
  const uint4* src = reinterpret_cast<const uint4*>(x + t * token_stride + h * head_stride + grp * 16);
  const uint4 u0 = __ldg(src), u1 = __ldg(src + 1);
  const uint32_t w[8] = {u0.x, u0.y, u0.z, u0.w, u1.x, u1.y, u1.z, u1.w};
  const float f = which ? p.factor[1] : p.factor[0], inv = 1.f / f;  // a power of two: exact
  float y[16];
  float mx = 0.f;
  bool nan = false;
#pragma unroll
  for (int j = 0; j < 8; ++j) {
    const float2 v = unpack_bf16x2(w[j]);
    y[2 * j] = v.x * inv;
    y[2 * j + 1] = v.y * inv;
    nan |= isnan(v.x) || isnan(v.y);
    mx = fmaxf(mx, fmaxf(fabsf(y[2 * j]), fabsf(y[2 * j + 1])));
  }
  const uint32_t scale = nan ? 0x7fu : e4m3_of(__fdiv_rn(mx, 6.f));
  const float s = f16lo_to_f32(e4m3x2_to_f16(scale));
  uint32_t code[2] = {0, 0};
  if (s > 0.f) {  // (false for the NaN scale)
#pragma unroll
    for (int j = 0; j < 8; ++j)
      code[j >> 2] |= e2m1x2_of(__fdiv_rn(y[2 * j], s), __fdiv_rn(y[2 * j + 1], s)) << (8 * (j & 3));
  }
  if (__nv_bfloat16* out = which ? p.out[1] : p.out[0]) {
    uint4 o[2];
    uint32_t* ow = reinterpret_cast<uint32_t*>(o);
    const float sf = s * f;
#pragma unroll
    for (int j = 0; j < 2; ++j) {
      uint32_t hv[4];
      e2m1x8_to_f16(code[j], hv);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = f16x2_to_f32(hv[m]);
        ow[4 * j + m] = pack_bf16x2(v.x * sf, v.y * sf);
      }
    }
    uint4* dst = reinterpret_cast<uint4*>(out + row * D + grp * 16);
    dst[0] = o[0];
    dst[1] = o[1];
  }
  if (slot < 0) return;  // a padding token
  if (slot >= static_cast<long long>(p.cache.num_pages) << p.cache.shift) {
    atomicCAS(&g_cache_status, kDevOk, kDevBadIndex);
    return;
  }
  const long long page = slot >> p.cache.shift;
  const int off = static_cast<int>(slot) & ((1 << p.cache.shift) - 1), key = off & 15;
  char* tile = p.cache.base + page * p.cache.page_stride +
               (static_cast<long long>(h) * (1 << (p.cache.shift - 4)) + (off >> 4)) * L::kTileBytes;
  if (which == 0) {
    *reinterpret_cast<uint2*>(tile + key * (D / 2) + grp * 8) = make_uint2(code[0], code[1]);
    tile[L::k_scale_at(key, grp)] = static_cast<char>(scale);
  } else {
    // the 16 columns are 128 / D lanes' pieces of D / 16 bytes
    constexpr int kPiece = D / 16;
    if constexpr (kPiece == 8) {
      *reinterpret_cast<uint2*>(tile + L::v_piece_at(key, grp)) = make_uint2(code[0], code[1]);
    } else if constexpr (kPiece == 4) {
#pragma unroll
      for (int j = 0; j < 2; ++j) *reinterpret_cast<uint32_t*>(tile + L::v_piece_at(key, grp * 2 + j)) = code[j];
    } else if constexpr (kPiece == 2) {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        *reinterpret_cast<uint16_t*>(tile + L::v_piece_at(key, grp * 4 + j)) =
            static_cast<uint16_t>(code[j >> 1] >> (16 * (j & 1)));
    } else {
#pragma unroll
      for (int j = 0; j < 8; ++j) tile[L::v_piece_at(key, j)] = static_cast<char>(code[j >> 2] >> (8 * (j & 3)));
    }
    tile[L::v_scale_at(key, grp)] = static_cast<char>(scale);
  }
}

struct GatherProblem {
  PagedCache cache;
  const int* table;
  long long table_stride;
  int width;
  const int* cu;
  int B, total;
  __nv_bfloat16* out[2];
  float factor[2];
};

constexpr int kGatherTokens = 16;

// A CTA reads kGatherTokens packed rows back: each row's sequence is found by
// bisection of the offsets once per CTA and followed from there.  One thread
// per 8 columns (a 16-byte store), K and V in turn.
template <int D>
__global__ void __launch_bounds__(256) fa2_kv4_gather_kernel(const GatherProblem p) {
  using L = Kv4<D>;
  griddep_wait();
  griddep_launch_dependents();
  __shared__ const char* s_tile[kGatherTokens];  // the token's tile of head 0, or NULL
  __shared__ int s_key[kGatherTokens];
  const int t0 = blockIdx.x * kGatherTokens;
  if (threadIdx.x < kGatherTokens) {
    const int t = t0 + threadIdx.x;
    const char* tile = nullptr;
    int key = 0;
    if (t < p.total) {
      int lo = 0, hi = p.B;  // the last b with cu[b] <= t
      while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu + mid) <= t)
          lo = mid;
        else
          hi = mid;
      }
      const int a = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
      if (a >= 0 && a <= t && t < e) {
        const int pos = t - a, pg = pos >> p.cache.shift, off = pos & ((1 << p.cache.shift) - 1);
        if (pg >= p.width) {
          atomicCAS(&g_cache_status, kDevOk, kDevBadSeqlens);
        } else {
          const int id = __ldg(p.table + lo * p.table_stride + pg);
          if (id < 0 || id >= p.cache.num_pages) {
            atomicCAS(&g_cache_status, kDevOk, kDevBadIndex);
          } else {
            tile = p.cache.base + id * p.cache.page_stride + static_cast<long long>(off >> 4) * L::kTileBytes;
            key = off & 15;
          }
        }
      } else if (a > t || a < 0 || e < a) {  // (a row past the last sequence is no error)
        atomicCAS(&g_cache_status, kDevOk, kDevBadSeqlens);
      }
    }
    s_tile[threadIdx.x] = tile;
    s_key[threadIdx.x] = key;
  }
  __syncthreads();
  constexpr int kPer = D / 8;  // threads of a head
  const int row_threads = p.cache.heads * kPer;
  const long long head_bytes = static_cast<long long>(L::kTileBytes) << (p.cache.shift - 4);
  for (int i = threadIdx.x; i < row_threads * kGatherTokens; i += 256) {
    const int tok = i / row_threads, r = i - tok * row_threads;
    const char* tile = s_tile[tok];
    if (!tile) continue;
    const int h = r / kPer, c8 = r % kPer, key = s_key[tok];
    tile += h * head_bytes;
    const long long dst = (static_cast<long long>(t0 + tok) * p.cache.heads + h) * D + c8 * 8;
#pragma unroll
    for (int which = 0; which < 2; ++which) {
      uint32_t code;
      int scale_at;
      if (which == 0) {
        code = *reinterpret_cast<const uint32_t*>(tile + key * (D / 2) + c8 * 4);
        scale_at = L::k_scale_at(key, c8 >> 1);
      } else {
        constexpr int kPiece = D / 16;
        if constexpr (kPiece == 8) {
          code = *reinterpret_cast<const uint32_t*>(tile + L::v_piece_at(key, c8 >> 1) + (c8 & 1) * 4);
        } else if constexpr (kPiece == 4) {
          code = *reinterpret_cast<const uint32_t*>(tile + L::v_piece_at(key, c8));
        } else if constexpr (kPiece == 2) {
          code = *reinterpret_cast<const uint16_t*>(tile + L::v_piece_at(key, c8 * 2)) |
                 static_cast<uint32_t>(*reinterpret_cast<const uint16_t*>(tile + L::v_piece_at(key, c8 * 2 + 1))) << 16;
        } else {
          code = 0;
#pragma unroll
          for (int j = 0; j < 4; ++j)
            code |= static_cast<uint32_t>(static_cast<uint8_t>(tile[L::v_piece_at(key, c8 * 4 + j)])) << (8 * j);
        }
        scale_at = L::v_scale_at(key, c8 >> 1);
      }
      const float s = f16lo_to_f32(e4m3x2_to_f16(static_cast<uint8_t>(tile[scale_at]))) * p.factor[which];
      uint32_t hv[4], o[4];
      e2m1x8_to_f16(code, hv);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 v = f16x2_to_f32(hv[m]);
        o[m] = pack_bf16x2(v.x * s, v.y * s);
      }
      *reinterpret_cast<uint4*>(p.out[which] + dst) = make_uint4(o[0], o[1], o[2], o[3]);
    }
  }
}

template <int D>
int launch_append_d(const AppendProblem& p, cudaStream_t st) {
  return launch_pdl(fa2_kv4_append_kernel<D>, dim3(static_cast<unsigned>((p.groups + 255) / 256), 2), dim3(256), 0, st, p);
}
template <int D>
int launch_gather_d(const GatherProblem& p, cudaStream_t st) {
  return launch_pdl(fa2_kv4_gather_kernel<D>, dim3(static_cast<unsigned>((p.total + kGatherTokens - 1) / kGatherTokens)),
                    dim3(256), 0, st, p);
}

}  // namespace

bool power_of_two(float x) {
  int e;
  return std::isfinite(x) && x > 0.f && std::frexp(x, &e) == 0.5f && e >= -63 && e <= 65;
}

size_t kv4_page_bytes(int H_kv, int page_size, int d) {
  return static_cast<size_t>(H_kv) * (page_size / kCacheTile) * 18 * d;
}

int check_cache(const void* cache, long long page_stride, int num_pages, int page_size, int H_kv, int d) {
  if (H_kv < 1 || num_pages < 1) return FA2_ERR_SHAPE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FA2_ERR_SHAPE;
  if (!head_dim_ok(d)) return FA2_ERR_HEADDIM;
  if (!cache) return FA2_ERR_NULL;
  if (H_kv > (1 << 20) || page_stride < static_cast<long long>(kv4_page_bytes(H_kv, page_size, d)) ||
      page_stride > (1LL << 40))
    return FA2_ERR_SHAPE;
  if (!aligned(cache, 16) || page_stride % 16 != 0) return FA2_ERR_ALIGN;
  return FA2_OK;
}

PagedCache paged_cache(const void* cache, long long page_stride, int num_pages, int page_size, int H_kv) {
  PagedCache c{static_cast<char*>(const_cast<void*>(cache)), page_stride, num_pages, 4, H_kv};
  while ((1 << c.shift) < page_size) ++c.shift;
  return c;
}

// The bytes a cache can span (its pages may have others' between them).
size_t cache_span(long long page_stride, int num_pages, int page_size, int H_kv, int d) {
  return static_cast<size_t>(num_pages - 1) * page_stride + kv4_page_bytes(H_kv, page_size, d);
}

int read_cache_status(int* value, bool reset) {
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_cache_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_cache_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

extern "C" {

size_t fa2_kv4_page_bytes(int H_kv, int page_size, int d) {
  if (H_kv < 1 || !head_dim_ok(d)) return 0;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return 0;
  return kv4_page_bytes(H_kv, page_size, d);
}

int fa2_kv4_append(const void* k, const void* v, const long long* strides, void* cache, long long page_stride,
                   const long long* slots, void* k_out, void* v_out, int num_tokens, int H_kv, int num_pages,
                   int page_size, int d, float k_scale, float v_scale, void* stream) {
  if (int rc = check_cache(cache, page_stride, num_pages, page_size, H_kv, d)) return rc;
  if (num_tokens < 0 || num_tokens > (1 << 30)) return FA2_ERR_SHAPE;
  if (!power_of_two(k_scale) || !power_of_two(v_scale)) return FA2_ERR_SCALE;
  if (num_tokens == 0) return FA2_OK;
  if (!k || !v || !slots) return FA2_ERR_NULL;
  if (!aligned(k, 16) || !aligned(v, 16) || !aligned(slots, 8) || !aligned(k_out, 16) || !aligned(v_out, 16))
    return FA2_ERR_ALIGN;
  AppendProblem p{};
  p.groups = static_cast<long long>(num_tokens) * H_kv * (d / 16);
  if ((p.groups + 255) / 256 > 0x7fffffffLL) return FA2_ERR_SHAPE;
  size_t span[2];
  for (int i = 0; i < 2; ++i) {
    p.token_stride[i] = num_tokens > 1 && strides ? strides[2 * i] : static_cast<long long>(H_kv) * d;
    p.head_stride[i] = H_kv > 1 && strides ? strides[2 * i + 1] : d;
    if (p.token_stride[i] < 0 || p.head_stride[i] < 0 || p.token_stride[i] > (1LL << 40) || p.head_stride[i] > (1LL << 40))
      return FA2_ERR_SHAPE;
    if (p.token_stride[i] % 8 != 0 || p.head_stride[i] % 8 != 0) return FA2_ERR_ALIGN;
    span[i] = static_cast<size_t>((num_tokens - 1) * p.token_stride[i] + (H_kv - 1) * p.head_stride[i] + d) * 2;
  }
  const size_t ob = static_cast<size_t>(num_tokens) * H_kv * d * 2;
  const Range outs[] = {range_of(cache, cache_span(page_stride, num_pages, page_size, H_kv, d)),
                        range_of(k_out, k_out ? ob : 0), range_of(v_out, v_out ? ob : 0)};
  const Range ins[] = {range_of(k, span[0]), range_of(v, span[1]), range_of(slots, static_cast<size_t>(num_tokens) * 8)};
  for (int i = 0; i < 3; ++i) {
    if (outs[i].lo == outs[i].hi) continue;
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return FA2_ERR_ALIAS;
    for (int j = i + 1; j < 3; ++j)
      if (outs[j].lo != outs[j].hi && overlap(outs[i], outs[j])) return FA2_ERR_ALIAS;
  }
  p.x[0] = static_cast<const __nv_bfloat16*>(k);
  p.x[1] = static_cast<const __nv_bfloat16*>(v);
  p.out[0] = static_cast<__nv_bfloat16*>(k_out);
  p.out[1] = static_cast<__nv_bfloat16*>(v_out);
  p.factor[0] = k_scale;
  p.factor[1] = v_scale;
  p.slots = slots;
  p.cache = paged_cache(cache, page_stride, num_pages, page_size, H_kv);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int e = d == 16    ? launch_append_d<16>(p, st)
                : d == 32  ? launch_append_d<32>(p, st)
                : d == 64  ? launch_append_d<64>(p, st)
                           : launch_append_d<128>(p, st);
  return e ? record_cuda_failure(e, "kv4 append launch") : FA2_OK;
}

int fa2_kv4_gather(const void* cache, long long page_stride, const int* block_table, long long table_stride,
                   const int* cu_seqlens, void* k, void* v, int B, int H_kv, int total, int num_pages, int page_size,
                   int table_width, int d, float k_scale, float v_scale, void* stream) {
  if (int rc = check_cache(cache, page_stride, num_pages, page_size, H_kv, d)) return rc;
  if (B < 1 || total < 0 || total > (1 << 30) || table_width < 1 || (B > 1 && table_stride < table_width))
    return FA2_ERR_SHAPE;
  if (H_kv > (1 << 16)) return FA2_ERR_SHAPE;
  if (!power_of_two(k_scale) || !power_of_two(v_scale)) return FA2_ERR_SCALE;
  if (total == 0) return FA2_OK;
  if (!block_table || !cu_seqlens || !k || !v) return FA2_ERR_NULL;
  if (!aligned(block_table, 4) || !aligned(cu_seqlens, 4) || !aligned(k, 16) || !aligned(v, 16)) return FA2_ERR_ALIGN;
  const size_t ob = static_cast<size_t>(total) * H_kv * d * 2;
  const size_t tb = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
  const Range ins[] = {range_of(cache, cache_span(page_stride, num_pages, page_size, H_kv, d)), range_of(block_table, tb),
                       range_of(cu_seqlens, static_cast<size_t>(B + 1) * 4)};
  const Range rk = range_of(k, ob), rv = range_of(v, ob);
  for (const Range& r : ins)
    if (overlap(rk, r) || overlap(rv, r)) return FA2_ERR_ALIAS;
  if (overlap(rk, rv)) return FA2_ERR_ALIAS;
  const GatherProblem p{paged_cache(cache, page_stride, num_pages, page_size, H_kv), block_table, table_stride, table_width,
                        cu_seqlens, B, total,
                        {static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v)}, {k_scale, v_scale}};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const int e = d == 16    ? launch_gather_d<16>(p, st)
                : d == 32  ? launch_gather_d<32>(p, st)
                : d == 64  ? launch_gather_d<64>(p, st)
                           : launch_gather_d<128>(p, st);
  return e ? record_cuda_failure(e, "kv4 gather launch") : FA2_OK;
}

}  // extern "C"
