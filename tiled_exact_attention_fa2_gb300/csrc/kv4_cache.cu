// Writing keys and values into the 4-bit paged cache, and reading them back
// as bf16.
//
// Both are bound by HBM: the append reads 2 bytes a value and writes 4.5
// bits (and 2 bytes more where the caller wants the stored values), the
// gather reads 4.5 bits and writes 2 bytes.  Measured on a GB300 (device
// time): append of 16385 tokens x 8 heads of 128 columns with the stored
// values 25.5 us (6.0 TB/s, 88 % of a copy's rate), gather of 20000 tokens of
// the same 21.4 us (5.4 TB/s; 1258 CTAs in 2.8 waves).
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "args.h"
#include "fa2.h"
#include "kv4.cuh"
#include "launch.h"

namespace fa2 {
namespace {

__device__ int g_cache_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

struct AppendProblem {
  const __nv_bfloat16 *k, *v;  // [T, H_kv, d]
  long long token_stride[2], head_stride[2];
  __nv_bfloat16 *k_out, *v_out;  // stored values [T, H_kv, d], or NULL
  float k_scale, v_scale;
  const long long* slots;
  PagedCache cache;
  int tokens, block_heads, block_tokens;  // K/V heads and tokens of a CTA
};

// The values of four code bytes as bf16 (exact: 6 significant bits).
__device__ __forceinline__ uint4 expand(uint32_t code, float scale) {
  uint32_t hv[4], o[4];
  e2m1x8_to_f16(code, hv);
  const uint64_t s2 = f2_pack(scale, scale);
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 v = f16x2_to_f32(hv[i]), u = f2_unpack(fmul2(f2_pack(v.x, v.y), s2));
    o[i] = pack_bf16x2(u.x, u.y);
  }
  return make_uint4(o[0], o[1], o[2], o[3]);
}
__device__ __forceinline__ float scale_of(uint32_t byte) { return f16lo_to_f32(e4m3x2_to_f16(byte)); }

// 8 columns of a group of 16, the other 8 in the neighbouring lane: the
// group's scale byte, the columns' four code bytes, and the stored values in
// place of x.  The scale is e4m3(max |x| / (6 f)), a code e2m1(x / (f s)), f
// the cache's factor.  Both quotients are products with a rounded reciprocal,
// off by less than 2^-22; that does not move a value across a border of its
// format or off it: x is bf16 (8 significant bits), a border times a scale
// has at most 9, so a quotient that is not on a border is at least 2^-9
// away; one that is on it comes out exact (a scale's borders) or is rounded
// back onto it (a code's: fp16 keeps 11 bits).  So every value is the nearest
// one, ties to even, as an exact division would give it.
__device__ __forceinline__ void quantize(uint4& x, float f, uint32_t& scale, uint32_t& code, bool want_values) {
  const uint32_t w[4] = {x.x, x.y, x.z, x.w};
  constexpr uint32_t kAbs = 0x7fff7fffu;
  uint32_t top = max_bf16x2(max_bf16x2(w[0] & kAbs, w[1] & kAbs), max_bf16x2(w[2] & kAbs, w[3] & kAbs));
  top = max_bf16x2(top, __shfl_xor_sync(0xffffffffu, top, 1));
  top = max_bf16x2(top, top >> 16);  // (its low half)
  const float mx = __uint_as_float(top << 16), inv_f = 1.f / f;  // a power of two: exact
  // a NaN in the group: the NaN scale
  scale = isnan(mx) ? 0x7fu : e4m3_of(mx * inv_f * (1.f / 6.f));
  const float s = scale_of(scale);
  code = 0;  // of a group whose scale is 0 or NaN
  if (s > 0.f) {
    const float inv = __frcp_rn(s) * inv_f;
    const uint64_t inv2 = f2_pack(inv, inv);
    uint32_t q[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 v = unpack_bf16x2(w[i]), u = f2_unpack(fmul2(f2_pack(v.x, v.y), inv2));
      q[i] = pack_f16x2(u.x, u.y);
    }
    code = f16_to_e2m1x8(q);
  }
  if (want_values) {
    x = expand(code, s * f);
  }
}

// One thread per 8 columns of a token's head, for K and for V: 16-byte loads
// and stores side by side, two of each in flight.  (One thread per group of
// 16 with IEEE divisions was bound by instructions: 36 us against 23 of
// memory for 16385 tokens of 8 heads of 128 columns.)
template <int D, int TOKENS>
__global__ void __launch_bounds__(256, 5) fa2_kv4_append_kernel(const AppendProblem p) {
  using L = Kv4<D>;
  griddep_wait();
  griddep_launch_dependents();
  // thread -> (token, head, columns), a group's pair of lanes together.  Rows
  // of 16 and 32 columns go through the tokens before the heads: a byte store
  // of a warp then falls into a few sectors of a tile, not into one of every
  // head (39000 tokens of 16 heads of 32 columns 44 us else).
  const int c8 = threadIdx.x % (D / 8), grp = c8 >> 1, at = threadIdx.x / (D / 8);
  const int slow = at / (D <= 32 ? p.block_tokens : p.block_heads), fast = at - slow * (D <= 32 ? p.block_tokens : p.block_heads);
  const int local = D <= 32 ? fast : slow, head = D <= 32 ? slow : fast;
  const int h = blockIdx.y * p.block_heads + head;
  const bool fits = local < p.block_tokens && head < p.block_heads && h < p.cache.heads;
  uint4 k[TOKENS], v[TOKENS];
  long long slot[TOKENS];
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    const int t = (blockIdx.x * TOKENS + i) * p.block_tokens + local;
    k[i] = v[i] = make_uint4(0, 0, 0, 0);
    slot[i] = -1;
    if (fits && t < p.tokens) {
      slot[i] = __ldg(p.slots + t);
      k[i] = __ldg(reinterpret_cast<const uint4*>(p.k + t * p.token_stride[0] + h * p.head_stride[0] + c8 * 8));
      v[i] = __ldg(reinterpret_cast<const uint4*>(p.v + t * p.token_stride[1] + h * p.head_stride[1] + c8 * 8));
    }
  }
#pragma unroll
  for (int i = 0; i < TOKENS; ++i) {
    const int t = (blockIdx.x * TOKENS + i) * p.block_tokens + local;
    uint32_t k_scale, k_code, v_scale, v_code;
    quantize(k[i], p.k_scale, k_scale, k_code, p.k_out != nullptr);
    quantize(v[i], p.v_scale, v_scale, v_code, p.v_out != nullptr);
    if (!fits || t >= p.tokens) continue;
    const long long out = (static_cast<long long>(t) * p.cache.heads + h) * D + c8 * 8;
    if (p.k_out) *reinterpret_cast<uint4*>(p.k_out + out) = k[i];
    if (p.v_out) *reinterpret_cast<uint4*>(p.v_out + out) = v[i];
    if (slot[i] < 0) continue;  // a padding token
    if (slot[i] >= static_cast<long long>(p.cache.num_pages) << p.cache.shift) {
      atomicCAS(&g_cache_status, kDevOk, kDevBadIndex);
      continue;
    }
    const int off = static_cast<int>(slot[i]) & ((1 << p.cache.shift) - 1), key = off & 15;
    char* tile = p.cache.base + (slot[i] >> p.cache.shift) * p.cache.page_stride +
                 ((static_cast<long long>(h) << (p.cache.shift - 4)) + (off >> 4)) * L::kTileBytes;
    *reinterpret_cast<uint32_t*>(tile + key * (D / 2) + c8 * 4) = k_code;
    constexpr int kPiece = D / 16;  // bytes of a lane's V columns
    if constexpr (kPiece >= 4) {
      constexpr int kPer = kPiece / 4;  // threads of a piece
      *reinterpret_cast<uint32_t*>(tile + L::v_piece_at(key, c8 / kPer) + c8 % kPer * 4) = v_code;
    } else if constexpr (kPiece == 2) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
        *reinterpret_cast<uint16_t*>(tile + L::v_piece_at(key, c8 * 2 + j)) = static_cast<uint16_t>(v_code >> (16 * j));
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j) tile[L::v_piece_at(key, c8 * 4 + j)] = static_cast<char>(v_code >> (8 * j));
    }
    if (c8 & 1)
      tile[L::v_scale_at(key, grp)] = static_cast<char>(v_scale);
    else
      tile[L::k_scale_at(key, grp)] = static_cast<char>(k_scale);
  }
}

struct GatherProblem {
  PagedCache cache;
  const int* table;
  long long table_stride;
  int width;
  const int* cu;
  int B, total;
  __nv_bfloat16 *k, *v;
  float k_scale, v_scale;
  int head_warps;  // of a CTA's 8 warps on one group of tokens
};

constexpr int kGatherTokens = 16;  // of a warp

// Where a packed row's values lie: head 0's tile and the key in it, or NULL
// for a row outside every sequence or not to be found.
__device__ __forceinline__ const char* find_row(const GatherProblem& p, int t, int tile_bytes, int& key) {
  if (t >= p.total) return nullptr;
  int lo = 0, hi = p.B;  // the last b with cu[b] <= t
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (__ldg(p.cu + mid) <= t)
      lo = mid;
    else
      hi = mid;
  }
  const int a = __ldg(p.cu + lo), e = __ldg(p.cu + lo + 1);
  if (a < 0 || t < a || t >= e) return nullptr;  // (before the first sequence, behind the last)
  const int pos = t - a, pg = pos >> p.cache.shift, off = pos & ((1 << p.cache.shift) - 1);
  if (pg >= p.width) {
    atomicCAS(&g_cache_status, kDevOk, kDevBadSeqlens);
    return nullptr;
  }
  const int id = __ldg(p.table + lo * p.table_stride + pg);
  if (id < 0 || id >= p.cache.num_pages) {
    atomicCAS(&g_cache_status, kDevOk, kDevBadIndex);
    return nullptr;
  }
  key = off & 15;
  return p.cache.base + id * p.cache.page_stride + static_cast<long long>(off >> 4) * tile_bytes;
}

// A warp reads kGatherTokens packed rows of one head after another back: a
// lane takes 8 columns (a 16-byte store) of every (D / 8)-th row, all loads
// of the rows first.  Where the rows lie is found once per CTA, a thread per
// row.
template <int D>
__global__ void __launch_bounds__(256) fa2_kv4_gather_kernel(const GatherProblem p) {
  using L = Kv4<D>;
  constexpr int kLanes = D / 8, kAtOnce = 32 / kLanes, kIters = kGatherTokens / kAtOnce;
  __shared__ const char* s_tile[8 * kGatherTokens];
  __shared__ int s_key[8 * kGatherTokens];
  griddep_wait();
  griddep_launch_dependents();
  const int groups = 8 / p.head_warps;  // of tokens
  const int t0 = blockIdx.x * groups * kGatherTokens;
  if (threadIdx.x < groups * kGatherTokens) {
    int key = 0;
    s_tile[threadIdx.x] = find_row(p, t0 + threadIdx.x, L::kTileBytes, key);
    s_key[threadIdx.x] = key;
  }
  // Offsets out of order would give rows to the wrong sequences unnoticed: the
  // last CTA, which has the fewest rows, looks at all of them.
  if (blockIdx.x == gridDim.x - 1)
    for (int b = threadIdx.x; b < p.B; b += 256) {
      const int a = __ldg(p.cu + b);
      if (a < 0 || __ldg(p.cu + b + 1) < a) atomicCAS(&g_cache_status, kDevOk, kDevBadSeqlens);
    }
  __syncthreads();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int group = warp / p.head_warps;
  if (group >= groups) return;
  const int c8 = lane % kLanes, grp = c8 >> 1;
  const long long head_bytes = static_cast<long long>(L::kTileBytes) << (p.cache.shift - 4);
  for (int h = warp - group * p.head_warps; h < p.cache.heads; h += p.head_warps) {
    uint32_t kc[kIters], vc[kIters], ks[kIters], vs[kIters];
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = group * kGatherTokens + i * kAtOnce + lane / kLanes;
      kc[i] = vc[i] = ks[i] = vs[i] = 0;
      if (const char* tile = s_tile[row]) {
        const int key = s_key[row];
        tile += h * head_bytes;
        kc[i] = __ldg(reinterpret_cast<const uint32_t*>(tile + key * (D / 2) + c8 * 4));
        ks[i] = __ldg(reinterpret_cast<const uint8_t*>(tile + L::k_scale_at(key, grp)));
        vs[i] = __ldg(reinterpret_cast<const uint8_t*>(tile + L::v_scale_at(key, grp)));
        constexpr int kPiece = D / 16;
        if constexpr (kPiece >= 4) {
          constexpr int kPer = kPiece / 4;
          vc[i] = __ldg(reinterpret_cast<const uint32_t*>(tile + L::v_piece_at(key, c8 / kPer) + c8 % kPer * 4));
        } else if constexpr (kPiece == 2) {
#pragma unroll
          for (int j = 0; j < 2; ++j)
            vc[i] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint16_t*>(tile + L::v_piece_at(key, c8 * 2 + j)))) << (16 * j);
        } else {
#pragma unroll
          for (int j = 0; j < 4; ++j)
            vc[i] |= static_cast<uint32_t>(__ldg(reinterpret_cast<const uint8_t*>(tile + L::v_piece_at(key, c8 * 4 + j)))) << (8 * j);
        }
      }
    }
#pragma unroll
    for (int i = 0; i < kIters; ++i) {
      const int row = group * kGatherTokens + i * kAtOnce + lane / kLanes;
      if (!s_tile[row]) continue;
      const long long dst = (static_cast<long long>(t0 + row) * p.cache.heads + h) * D + c8 * 8;
      *reinterpret_cast<uint4*>(p.k + dst) = expand(kc[i], scale_of(ks[i]) * p.k_scale);
      *reinterpret_cast<uint4*>(p.v + dst) = expand(vc[i], scale_of(vs[i]) * p.v_scale);
    }
  }
}

template <int D>
int launch_append_d(AppendProblem p, cudaStream_t st) {
  // (token, head) pairs of a CTA: whole tokens where they fit (16 of them for
  // short rows), else equal parts of the heads over blockIdx.y
  constexpr int kPairs = 256 / (D / 8), kHeads = D <= 32 ? kPairs / 16 : kPairs;
  const unsigned parts = (p.cache.heads + kHeads - 1) / kHeads;
  p.block_heads = (p.cache.heads + parts - 1) / parts;
  p.block_tokens = kPairs / p.block_heads;
  // Many tokens: two to a thread, for twice the loads in flight.
  const long long ctas = (p.tokens + p.block_tokens - 1LL) / p.block_tokens;
  if (ctas * parts >= 152 * 16)
    return launch_pdl(fa2_kv4_append_kernel<D, 2>, dim3(static_cast<unsigned>((ctas + 1) / 2), parts), dim3(256), 0, st, p);
  return launch_pdl(fa2_kv4_append_kernel<D, 1>, dim3(static_cast<unsigned>(ctas), parts), dim3(256), 0, st, p);
}
template <int D>
int launch_gather_d(GatherProblem p, cudaStream_t st) {
  p.head_warps = p.cache.heads < 8 ? p.cache.heads : 8;
  const int per = 8 / p.head_warps * kGatherTokens;
  return launch_pdl(fa2_kv4_gather_kernel<D>, dim3(static_cast<unsigned>((p.total + per - 1) / per)), dim3(256), 0, st, p);
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
  if (H_kv > (1 << 16) || page_stride < static_cast<long long>(kv4_page_bytes(H_kv, page_size, d)) ||
      !stride_ok(page_stride, num_pages))
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
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
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
  p.tokens = num_tokens;
  size_t span[2];
  for (int i = 0; i < 2; ++i) {
    p.token_stride[i] = num_tokens > 1 && strides ? strides[2 * i] : static_cast<long long>(H_kv) * d;
    p.head_stride[i] = H_kv > 1 && strides ? strides[2 * i + 1] : d;
    if (!stride_ok(p.token_stride[i], num_tokens - 1) || !stride_ok(p.head_stride[i], H_kv - 1)) return FA2_ERR_SHAPE;
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
  p.k = static_cast<const __nv_bfloat16*>(k);
  p.v = static_cast<const __nv_bfloat16*>(v);
  p.k_out = static_cast<__nv_bfloat16*>(k_out);
  p.v_out = static_cast<__nv_bfloat16*>(v_out);
  p.k_scale = k_scale;
  p.v_scale = v_scale;
  p.slots = slots;
  p.cache = paged_cache(cache, page_stride, num_pages, page_size, H_kv);
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  g_launched = true;
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
  if (B < 1 || total < 0 || total > (1 << 30) || table_width < 1 ||
      (B > 1 && (table_stride < table_width || !stride_ok(table_stride, B))))
    return FA2_ERR_SHAPE;
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
                        cu_seqlens, B, total, static_cast<__nv_bfloat16*>(k), static_cast<__nv_bfloat16*>(v), k_scale, v_scale, 0};
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  g_launched = true;
  const int e = d == 16    ? launch_gather_d<16>(p, st)
                : d == 32  ? launch_gather_d<32>(p, st)
                : d == 64  ? launch_gather_d<64>(p, st)
                           : launch_gather_d<128>(p, st);
  return e ? record_cuda_failure(e, "kv4 gather launch") : FA2_OK;
}

}  // extern "C"
