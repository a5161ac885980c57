// Attention of new query tokens over a paged key-value cache in bf16 or e4m3, for
// many requests of few keys: one, two or four warps take a whole unit (request, K/V
// head, up to 32 query rows).
//
// A unit of 100 keys is 50 KB (128 columns, bf16), 2300 cycles of an SM's share of
// the memory; to divide it among a CTA's warps and join their results takes longer.
// Here eight warps of a CTA work on eight, four or two units, and no warp waits for
// another but the few of its group, at a unit's end.  Each has a ring of shared memory
// and copies the next slots itself after each one that it has read, into the next unit
// too; lengths and page ids of the unit after that are on their way meanwhile.  Bound by
// reading the cache once, or, with few units, by a warp's chain of slots (some 1400
// cycles each with 8 rows, 2500 with 32).  Measured (8 K/V heads of 128 columns, bf16):
// 1000 requests of up to 100 keys 58 us (4.8 TB/s; the CTA-wide way 163), 300 of up to
// 512 74 us (5.4 TB/s; 81), 40 of up to 250 11 us (15).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>

#include "args.h"
#include "fa2.h"
#include "kv_attn.cuh"
#include "launch.h"

namespace fa2 {
namespace {

using namespace kv_attn;

__device__ int g_kv_short_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

template <int D, int E, int NT>
struct ShortSmem {
  static constexpr int kBytes = NT == 4 ? 16384 : 24576;  // of a warp's ring
  static constexpr int kRing = kBytes / Tile<D, E>::kSlot < 8 ? kBytes / Tile<D, E>::kSlot : 8;
  alignas(1024) char ring[kWarps][kRing][Tile<D, E>::kSlot];
  uint32_t q[kWarps][NT * (D / 16) * 64];
  float factor[kWarps][8 * NT];
  float2 ml[kWarps][8 * NT];
  uint64_t full[kWarps][kRing];
};

// What a unit's lengths and pages are read to, a lane's share of the pages: those of
// the warp's slot number `lane`, slot rank + group lane of the unit (32-key slots of
// 16-key pages have two).
struct Raw {
  int Lk, q0, q1, page[2];
};
template <int D, int E>
__device__ __forceinline__ void ask_unit(Raw& r, const AttnProblem& p, int unit, int units, int slot) {
  constexpr int kKeys = Tile<D, E>::kKeys;
  r = Raw{0, 0, 0, {-1, -1}};
  if (unit >= units) return;
  const int b = unit / p.heads, key = slot * kKeys;
  r.Lk = __ldg(p.lens + b);
  if (p.cu_q) {
    r.q0 = __ldg(p.cu_q + b);
    r.q1 = __ldg(p.cu_q + b + 1);
  } else {
    r.q0 = b * p.max_q;
    r.q1 = r.q0 + p.max_q;
  }
  // (the table has room for max_k keys, whatever the length)
  const int* const table = p.table + b * p.table_stride + (key >> p.shift);
  if (key < p.max_k) r.page[0] = __ldg(table);
  if (kKeys == 32 && p.shift == 4 && key + 16 < p.max_k) r.page[1] = __ldg(table + 1);
}

struct ShortUnit {
  int q0, Lq, Lk, h, slots, copied;  // slots: of this warp
  int page[2];    // of its slot `lane`; the last page + 1 gives zeros
  uint32_t mark;  // bit i: its 16-key half i has a page id out of range
};
template <int D, int E>
__device__ __forceinline__ ShortUnit known_unit(const Raw& r, const AttnProblem& p, int unit, int units, int group, int rank, int lane) {
  constexpr int kKeys = Tile<D, E>::kKeys;
  ShortUnit u{};
  if (unit >= units) return u;
  u.q0 = r.q0, u.Lq = r.q1 - r.q0, u.Lk = r.Lk;
  u.h = unit % p.heads;
  const bool ok = u.q0 >= 0 && u.Lq >= 0 && u.Lq <= p.max_q && u.q0 <= p.total_q - u.Lq && u.Lk >= 0 && u.Lk <= p.max_k;
  if (!ok) {
    if (lane == 0) atomicCAS(&g_kv_short_status, kDevOk, kDevBadSeqlens);
    u.Lq = u.Lk = 0;
  }
  const int all = u.Lq > 0 ? (u.Lk + kKeys - 1) / kKeys : 0, slot = rank + group * lane;
  u.slots = (all - rank + group - 1) / group;
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    const bool there = slot < all && (i == 0 || (kKeys == 32 && p.shift == 4 && slot * kKeys + 16 < u.Lk));
    u.page[i] = p.num_pages;
    if (there) {
      if (static_cast<uint32_t>(r.page[i]) < static_cast<uint32_t>(p.num_pages))
        u.page[i] = r.page[i];
      else
        u.mark |= 1u << i;
    }
  }
  if (p.shift > 4 && u.mark) u.mark = 3;  // (both halves lie in one page)
  if (u.mark) atomicCAS(&g_kv_short_status, kDevOk, kDevBadIndex);
  return u;
}

// The group's warps.
__device__ __forceinline__ void sync_group(int which, int warps) { asm volatile("bar.sync %0, %1;" ::"r"(which + 1), "r"(warps * 32) : "memory"); }

// The results of a group's warps, joined in their order by the first.  They lie in the
// same lanes, so they are handed over lane to lane, a half at a time, through the place
// of the queries, which are done with.
template <int D, int E, int NT>
__device__ __forceinline__ void join_group(Rows<D, NT>& s, ShortSmem<D, E, NT>& sm, int group, int warp, int lane) {
  const int rank = warp % group, which = warp / group, g = lane >> 2, c = lane & 3;
  float w0[NT][2];
#pragma unroll
  for (int half = 0; half < 2; ++half) {
    if (rank > 0) {
      float2* const to = reinterpret_cast<float2*>(sm.q[warp]) + lane;
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int t = 0; t < D / 16; ++t) to[(j * (D / 16) + t) * 32] = make_float2(s.o[j][t][2 * half], s.o[j][t][2 * half + 1]);
      if (half == 0 && g == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) sm.ml[warp][8 * j + 2 * c + u] = make_float2(-s.off[j][u], s.l[j][u]);
      }
    }
    sync_group(which, group);
    if (rank == 0) {
      if (half == 0) {
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int u = 0; u < 2; ++u) {
            const float m = -s.off[j][u];
            float top = m;
            for (int i = 1; i < group; ++i) top = fmaxf(top, sm.ml[warp + i][8 * j + 2 * c + u].x);
            w0[j][u] = ex2_approx(m - top);
            s.l[j][u] *= w0[j][u];
            s.off[j][u] = -top;
          }
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int t = 0; t < D / 16; ++t) {
          s.o[j][t][2 * half] *= w0[j][0];
          s.o[j][t][2 * half + 1] *= w0[j][1];
        }
#pragma unroll 1
      for (int i = 1; i < group; ++i) {
        const float2* const from = reinterpret_cast<const float2*>(sm.q[warp + i]) + lane;
#pragma unroll
        for (int j = 0; j < NT; ++j) {
          const float2 a = sm.ml[warp + i][8 * j + 2 * c], b = sm.ml[warp + i][8 * j + 2 * c + 1];
          const float wa = ex2_approx(a.x + s.off[j][0]), wb = ex2_approx(b.x + s.off[j][1]);
          if (half == 0) {
            s.l[j][0] = fmaf(wa, a.y, s.l[j][0]);
            s.l[j][1] = fmaf(wb, b.y, s.l[j][1]);
          }
#pragma unroll
          for (int t = 0; t < D / 16; ++t) {
            const float2 v = from[(j * (D / 16) + t) * 32];
            s.o[j][t][2 * half] = fmaf(wa, v.x, s.o[j][t][2 * half]);
            s.o[j][t][2 * half + 1] = fmaf(wb, v.y, s.o[j][t][2 * half + 1]);
          }
        }
      }
    }
    sync_group(which, group);  // (the half has been read)
  }
}

// A unit's rows, finished.  Transposed 8 by 8, a lane has neighbouring columns of row
// g of each tile.
template <int D, int E, int NT>
__device__ __forceinline__ void write_rows(Rows<D, NT>& s, const AttnProblem& p, const ShortUnit& u, int lane) {
  const int g = lane >> 2, c = lane & 3, rows = p.G * u.Lq;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    float f[2];
#pragma unroll
    for (int k = 0; k < 2; ++k) {
      const float l = s.l[j][k];
      f[k] = l == 0.f ? 0.f : p.v_scale / l;
      const int r = 8 * j + 2 * c + k;
      if (g == 0 && r < rows) {
        const int i = query_of(p, r), head = u.h * p.G + (r - i * p.G);
        p.lse[static_cast<long long>(head) * p.total_q + u.q0 + i] = l == 0.f ? -INFINITY : row_lse(-s.off[j][k], l);
      }
    }
    const int r = 8 * j + g, i = query_of(p, r), head = u.h * p.G + (r - i * p.G);
    __nv_bfloat16* const dst = p.o + (static_cast<long long>(u.q0 + i) * p.H + head) * D;
#pragma unroll
    for (int t = 0; t < D / 16; ++t) {
      const float(&o)[4] = s.o[j][t];
      const uint32_t a = transpose8x8(pack_bf16x2(o[0] * f[0], o[1] * f[1])), b = transpose8x8(pack_bf16x2(o[2] * f[0], o[3] * f[1]));
      if (r < rows) {
        if constexpr (E == 2) {  // columns 16 t + 2 c, + 1 and 16 t + 8 + 2 c, + 1
          *reinterpret_cast<uint32_t*>(dst + 16 * t + 2 * c) = a;
          *reinterpret_cast<uint32_t*>(dst + 16 * t + 8 + 2 * c) = b;
        } else {  // 16 t + 4 c, + 2 and 16 t + 4 c + 1, + 3
          *reinterpret_cast<uint2*>(dst + 16 * t + 4 * c) = make_uint2(__byte_perm(a, b, 0x5410), __byte_perm(a, b, 0x7632));
        }
      }
    }
  }
}

// ONE: a unit has one warp (else p.group; what is known then saves 2 to 7 %).
template <int D, int E, int NT, bool ONE>
__global__ void __launch_bounds__(kWarps * 32, 1)
    fa2_kv_attn_short_kernel(const __grid_constant__ CacheMaps maps, const __grid_constant__ AttnProblem p) {
  using T = Tile<D, E>;
  using S = ShortSmem<D, E, NT>;
  constexpr int kKeys = T::kKeys;
  extern __shared__ __align__(1024) char raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (smem_u32(raw) & 1023u) {  // (the copies' swizzle goes by the address)
    if (threadIdx.x == 0) atomicCAS(&g_kv_short_status, kDevOk, kDevSmemMisaligned);
    return;
  }
  if (lane < S::kRing) mbar_init(&sm.full[warp][lane], 1);
  fence_mbar_init();
  if (threadIdx.x < 2) tma_prefetch_desc(&maps.kv[threadIdx.x]);
  __syncwarp();
  griddep_wait();
  griddep_launch_dependents();
  // (neighbouring units on neighbouring SMs)
  const int units = p.B * p.heads, group = ONE ? 1 : p.group, stride = gridDim.x * (kWarps / group), rank = warp % group;
  int unit = blockIdx.x + warp / group * gridDim.x;
  const int slot = rank + group * lane;
  Raw r0, r1, r2;
  ask_unit<D, E>(r0, p, unit, units, slot);
  ask_unit<D, E>(r1, p, unit + stride, units, slot);
  ask_unit<D, E>(r2, p, unit + 2 * stride, units, slot);
  if (p.cu_q) {  // offsets out of order: nothing is written
    bool mixed = false;
    for (int b = threadIdx.x; b < p.B; b += kWarps * 32) mixed |= out_of_order(p, b);
    if (__syncthreads_or(mixed)) {
      if (threadIdx.x == 0) atomicCAS(&g_kv_short_status, kDevOk, kDevBadSeqlens);
      return;
    }
  }
  ShortUnit now = known_unit<D, E>(r0, p, unit, units, group, rank, lane), next = known_unit<D, E>(r1, p, unit + stride, units, group, rank, lane);
  uint32_t asked = 0, taken = 0;  // slots
  bool alive = true;
  // The next slots of this unit and the one after it, while the ring has room.
  auto copy = [&](ShortUnit& u) {
    for (; alive && asked - taken < S::kRing && u.copied < u.slots; ++u.copied, ++asked) {
      const int page0 = __shfl_sync(0xffffffffu, u.page[0], u.copied), page1 = __shfl_sync(0xffffffffu, u.page[1], u.copied);
      if (lane < 2) {  // keys, values
        const int place = asked % S::kRing, tok = (rank + group * u.copied) * kKeys & ((1 << p.shift) - 1);
        uint64_t* const bar = &sm.full[warp][place];
        const uint32_t dst = smem_u32(sm.ring[warp][place]) + lane * T::kHalf;
        if (lane == 0) mbar_arrive_expect_tx(bar, T::kSlot);
        __syncwarp(3);  // (no byte arrives before it is expected)
        tma_load_5d(dst, maps.kv + lane, bar, tok, u.h, page0);
        if (kKeys == 32 && p.shift == 4)  // (a page's 16 keys are a copy)
          tma_load_5d(dst + 16 * T::kRow, maps.kv + lane, bar, 0, u.h, page1);
      }
    }
  };
  copy(now);
  copy(next);
  Queries<D, NT, 32> queries;
  Rows<D, NT> s;
  for (; unit < units; unit += stride) {
    if (now.Lq > 0) {
      ask_queries(queries, p, now.q0, now.Lq, now.h, 0, lane);
      put_queries<D, E>(sm.q[warp], sm.factor[warp], queries, p.scale_log2, now.Lk, lane);
      start_rows<D, E, NT>(s, p, now.Lq, now.Lk, 0, lane);
      __syncwarp();
      for (int i = 0; alive && i < now.slots; ++i) {
        const int place = taken % S::kRing;
        if (!mbar_wait_warp(&sm.full[warp][place], taken / S::kRing & 1, &g_kv_short_status)) {
          // a copy that never came: rows are wrong from here on, with the status word set
          // (no more is copied; those under way are waited for)
          alive = false;
          for (; taken != asked; ++taken) mbar_wait_warp(&sm.full[warp][taken % S::kRing], taken / S::kRing & 1, &g_kv_short_status);
          break;
        }
        const uint32_t half = smem_u32(sm.ring[warp][place]), out = __shfl_sync(0xffffffffu, now.mark, i);
        constexpr int kAtOnce = T::kTiles < 2 || D * NT > 256 ? 1 : 2;  // (32 rows of 128 columns have no registers for two)
#pragma unroll 1
        for (int tile = 0; tile < T::kTiles; tile += kAtOnce) {
          const int k0 = (rank + group * i) * kKeys + 16 * tile;
          if (k0 >= now.Lk) break;
          if (k0 + 16 * kAtOnce <= s.min_vis && out == 0)
            step<D, E, NT, kAtOnce, false>(s, sm.q[warp], sm.factor[warp], p.scale_log2, half, tile, k0, 0, 0, lane);
          else
            step<D, E, NT, kAtOnce, true>(s, sm.q[warp], sm.factor[warp], p.scale_log2, half, tile, k0, now.Lk - k0, out >> tile, lane);
        }
        __syncwarp();  // every lane has read the slot
        ++taken;
        copy(now);
        copy(next);
      }
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u)
#pragma unroll
          for (int sh = 4; sh < 32; sh <<= 1) s.l[j][u] += __shfl_xor_sync(0xffffffffu, s.l[j][u], sh);
      __syncwarp();  // (the queries' place is free)
      if constexpr (!ONE) join_group<D, E, NT>(s, sm, group, warp, lane);
      if (rank == 0) write_rows<D, E, NT>(s, p, now, lane);
    }
    now = next;
    next = known_unit<D, E>(r2, p, unit + 2 * stride, units, group, rank, lane);
    ask_unit<D, E>(r2, p, unit + 3 * stride, units, slot);
    copy(now);
    copy(next);
  }
}

template <int D, int E, int NT>
int launch_nt(const CacheMaps& maps, const AttnProblem& p, cudaStream_t st) {
  static_assert(kShortKeys <= 32 * 16, "a lane has the page of one of the warp's slots");
  constexpr int kSmem = sizeof(ShortSmem<D, E, NT>);
  static_assert(kSmem <= 232448, "shared memory of a CTA");
  const auto kernel = p.group == 1 ? fa2_kv_attn_short_kernel<D, E, NT, true> : fa2_kv_attn_short_kernel<D, E, NT, false>;
  if (int e = ensure_max_smem(reinterpret_cast<const void*>(kernel), kSmem)) return e;
  const long long units = static_cast<long long>(p.B) * p.heads;
  return launch_pdl(kernel, dim3(units < kCtas ? static_cast<unsigned>(units) : kCtas), dim3(kWarps * 32), kSmem, st, maps, p);
}
template <int D, int E>
int launch_d(const CacheMaps& maps, const AttnProblem& p, cudaStream_t st) {
  switch (tiles_of(static_cast<long long>(p.max_q) * p.G)) {
    case 1: return launch_nt<D, E, 1>(maps, p, st);
    case 2: return launch_nt<D, E, 2>(maps, p, st);
    default: return launch_nt<D, E, 4>(maps, p, st);
  }
}
template <int E>
int launch_e(const CacheMaps& maps, const AttnProblem& p, int d, cudaStream_t st) {
  return d == 16 ? launch_d<16, E>(maps, p, st) : d == 32 ? launch_d<32, E>(maps, p, st) : d == 64 ? launch_d<64, E>(maps, p, st)
                                                                                                 : launch_d<128, E>(maps, p, st);
}

}  // namespace

namespace kv_attn {
int launch_short(const CacheMaps& maps, const AttnProblem& p, int d, int elem, cudaStream_t st) {
  g_launched = true;
  return elem == 2 ? launch_e<2>(maps, p, d, st) : launch_e<1>(maps, p, d, st);
}
}  // namespace kv_attn

int read_kv_short_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_kv_short_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_kv_short_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2
