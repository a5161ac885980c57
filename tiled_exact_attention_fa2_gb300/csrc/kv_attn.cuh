// What the attention kernels over a paged cache in bf16 or e4m3 share: the problem,
// and a warp's work on tiles of 16 keys.
//
// Operands (lane (g, c) = (lane / 4, lane % 4)).  S^T = K Q^T: a tile's 16 keys
// are the rows of the instruction and 8 query rows its columns, which wastes
// none of it on a group of 8 heads; K comes by ldmatrix.  O^T = V^T P^T: V comes
// by transposing ldmatrix, P^T from S^T's registers by 8x8 transposes
// (movmatrix).  The TMA copies swizzle rows as wide as 128 bytes, so ldmatrix
// has no bank conflicts.  e4m3 comes by the same loads as pairs of bytes and is
// made fp16 in registers; which columns a lane then holds is another order of
// the contraction (of S, Q has the same) or of O's columns.
//
// Precision.  P is split into two numbers of the cache's 16-bit type, high and low
// part, for two instructions instead of one: 16 significant bits of bf16, 22 of
// fp16.  With one fp16 number (11 bits) outputs in bf16 would differ from an fp32 P's by
// 4 to 8 in 10^4 of their norm, and sums that nearly cancel by more than bf16's
// rounding.  The second number's time (e4m3, 128 columns, one / two, us): 2 x
// 131072 keys, 16 rows a head 50.5 / 50.5, 32 rows 64.5 / 75.9; 64 requests of up to 1024,
// 4 rows 21.1 / 22.5; 300 of up to 512 41.5 / 43.1.
// bf16: scores are exact products summed in fp32.  e4m3 is exact in
// fp16; Q (8 bits) is divided by a power of two per row so that its largest
// value is in [1, 2), exact in fp16 down to 2^-14 of it (2^-25 absolute below);
// P is held 2^11 up so that weights down to 2^-25 of the largest keep all bits of
// the high part.  The running maximum is raised only when a score
// passes it by kLag, which saves the tile's maximum and the rescaling of O for
// nearly every tile.  Maximum, sum and O are fp32; the quotient removes the
// common factor exactly.  Any finite V gives a finite O: see lift().
#pragma once
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cstdint>

#include "ptx.cuh"
#include "tiles.cuh"

namespace fa2 {
namespace kv_attn {

constexpr int kWarps = 8;   // that compute, of a CTA
constexpr int kCtas = 152;  // one wave, one CTA an SM
constexpr float kNoMax = -1.7e38f;  // running maximum of a row that has seen no key (finite: no inf - inf)

struct CacheMaps {
  CUtensorMap kv[2];  // keys, values
};

struct AttnProblem {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  const int* table;
  long long table_stride;
  const int* lens;
  const int* cu_q;    // or NULL: every request has max_q queries
  size_t table_bytes, q_bytes;
  float* part;        // [kPlaces][rows][d] unnormalised O
  float2* part_ml;    // [kPlaces][rows] maximum - lift (log2), sum
  unsigned long long* arrived;  // [2][kPlaces]: this call's number in the upper 48 bits, parts that are there in the lower
  unsigned long long* queue;    // the number, and runs of items that have been taken
  unsigned long long call;      // the number, in the upper 48 bits
  uint32_t g_mul, g_shift;      // r / G = (umulhi(r, g_mul) + r) >> g_shift
  int num_pages, shift, heads;  // pages of 1 << shift tokens
  int B, H, G, total_q, max_q, max_k;
  float scale_log2, v_scale;
  int causal;
  int group;              // warps of a unit, where it has no more
  int direct, max_tiles;  // not 0: every unit has so many CTAs, a cluster; row tiles of a K/V head's grid
};

// Geometry of a cache of element size E and d columns.
template <int D, int E>
struct Tile {
  static constexpr int kRow = D * E;                      // bytes of a key
  static constexpr int kBoxRow = kRow > 128 ? 128 : kRow; // bytes of a copy's row
  static constexpr int kKeys = kRow > 128 ? 16 : 32;      // of a slot
  static constexpr int kHalf = kKeys * kRow;              // bytes of a slot's K, and of its V
  static constexpr int kSlot = 2 * kHalf;
  static constexpr int kTiles = kKeys / 16;

  // Byte of 16-byte chunk j of key `key` of a half (as TMA's swizzle lays it out).
  static __device__ __forceinline__ uint32_t at(uint32_t key, uint32_t j) {
    constexpr uint32_t kMask = kBoxRow == 128 ? 7u : kBoxRow == 64 ? 3u : kBoxRow == 32 ? 1u : 0u;
    constexpr uint32_t kPer = kBoxRow / 16;
    const uint32_t off = key * kBoxRow + (j % kPer) * 16;
    return (j / kPer) * (kKeys * kBoxRow) + (off ^ (((off >> 7) & kMask) << 4));
  }
};

struct Request {
  int q0, Lq, Lk;
  bool ok;
};

// A request with impossible lengths is left out (its rows are not written).
__device__ __forceinline__ Request request(const AttnProblem& p, int b) {
  Request r;
  r.Lk = __ldg(p.lens + b);
  if (p.cu_q) {
    r.q0 = __ldg(p.cu_q + b);
    r.Lq = __ldg(p.cu_q + b + 1) - r.q0;
  } else {
    r.q0 = b * p.max_q;
    r.Lq = p.max_q;
  }
  r.ok = r.q0 >= 0 && r.Lq >= 0 && r.Lq <= p.max_q && r.q0 <= p.total_q - r.Lq && r.Lk >= 0 && r.Lk <= p.max_k;
  return r;
}
// Whether the offsets begin below 0 or go down at request b.
__device__ __forceinline__ bool out_of_order(const AttnProblem& p, int b) {
  const int q0 = __ldg(p.cu_q + b);
  return q0 < 0 || __ldg(p.cu_q + b + 1) < q0;
}

// Row tiles of a K/V head, slots of a unit, slots of a request.
template <int ROWS>
__device__ __forceinline__ int row_tiles(const AttnProblem& p, const Request& r) {
  return static_cast<int>((static_cast<long long>(p.G) * r.Lq + ROWS - 1) / ROWS);
}
template <int KEYS>
__device__ __forceinline__ int key_slots(const Request& r) { return static_cast<int>((r.Lk + (KEYS - 1LL)) / KEYS); }
template <int ROWS, int KEYS>
__device__ __forceinline__ long long slots_of(const AttnProblem& p, const Request& r) {
  return r.ok ? static_cast<long long>(p.heads) * row_tiles<ROWS>(p, r) * key_slots<KEYS>(r) : 0;
}

__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// r / G of a row.
__device__ __forceinline__ int query_of(const AttnProblem& p, int r) {
  return static_cast<int>((__umulhi(static_cast<uint32_t>(r), p.g_mul) + static_cast<uint32_t>(r)) >> p.g_shift);
}

// ---------------------------------------------------------------- instructions
template <bool F16>
__device__ __forceinline__ void mma(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  if constexpr (F16)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
template <bool TRANS, int N>
__device__ __forceinline__ void load_matrices(uint32_t (&r)[4], uint32_t at) {
  if constexpr (N == 4 && TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else if constexpr (N == 4)
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(at) : "memory");
  else if constexpr (TRANS)
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.trans.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
  else
    asm volatile("ldmatrix.sync.aligned.m8n8.x2.shared.b16 {%0, %1}, [%2];" : "=r"(r[0]), "=r"(r[1]) : "r"(at) : "memory");
}
// The larger magnitudes of two pairs (their signs mean nothing), NaN where one is.
template <bool F16>
__device__ __forceinline__ uint32_t max_abs(uint32_t a, uint32_t b) {
  uint32_t r;
  if constexpr (F16)
    asm("max.NaN.xorsign.abs.f16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  else
    asm("max.NaN.xorsign.abs.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
  return r;
}
// Two numbers as a pair of fp16 or bf16, and back.
template <bool F16>
__device__ __forceinline__ uint32_t pack(float lo, float hi) { return F16 ? pack_f16x2(lo, hi) : pack_bf16x2(lo, hi); }
template <bool F16>
__device__ __forceinline__ float2 unpack(uint32_t v) {
  if constexpr (!F16) return unpack_bf16x2(v);
  return make_float2(f16lo_to_f32(v), f16lo_to_f32(v >> 16));
}
// Two e4m3 numbers (the low 16 bits) as an fp16 pair.
__device__ __forceinline__ uint32_t e4m3x2_to_f16(uint32_t w) {
  uint32_t r;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(r) : "h"(static_cast<uint16_t>(w)));
  return r;
}
// A slot's keys or values: from column 0 of token c1 of a page on (c2 and c3: the
// 128-byte half of a row, always from the first on; head, page).
__device__ __forceinline__ void tma_load_5d(uint32_t dst, const CUtensorMap* map, uint64_t* bar, int tok, int head, int page) {
  asm volatile(
      "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4, %3, %5, %6}], [%2];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(smem_u32(bar)), "r"(0), "r"(tok), "r"(head), "r"(page)
      : "memory");
}

// The A operands of a 16-key tile at `half` in shared memory, for steps (of K:
// columns 16 t ..) or row blocks (of V^T: columns 16 t ..) t and, of e4m3, t + 1.
// e4m3: a lane's word holds columns 4 c .. 4 c + 3 of a key of K, or columns 2 g,
// 2 g + 1 of keys 2 c, 2 c + 1 of V.
template <int D, int E>
__device__ __forceinline__ void load_k(uint32_t (*a)[4], uint32_t half, int tile, int t, int lane) {
  using T = Tile<D, E>;
  const int r = lane & 7, m = lane >> 3;
  if constexpr (E == 2) {
    load_matrices<false, 4>(a[0], half + T::at(tile * 16 + r + 8 * (m & 1), 2 * t + (m >> 1)));
  } else {
    uint32_t w[4];
    constexpr bool kBoth = D >= 32;
    load_matrices<false, kBoth ? 4 : 2>(w, half + T::at(tile * 16 + r + 8 * (m & 1), kBoth ? t + (m >> 1) : t));
#pragma unroll
    for (int i = 0; i < (kBoth ? 2 : 1); ++i) {
      a[i][0] = e4m3x2_to_f16(w[2 * i]), a[i][1] = e4m3x2_to_f16(w[2 * i + 1]);
      a[i][2] = e4m3x2_to_f16(w[2 * i] >> 16), a[i][3] = e4m3x2_to_f16(w[2 * i + 1] >> 16);
    }
  }
}
// V of keys from `keys` of the tile on counts as zeros.
template <int D, int E, bool MASKED>
__device__ __forceinline__ void load_v(uint32_t (*a)[4], uint32_t half, int tile, int t, int keys, int lane) {
  using T = Tile<D, E>;
  const int r = lane & 7, m = lane >> 3, c = lane & 3;
  uint32_t keep[2] = {0xffffffffu, 0xffffffffu};  // of keys 2 c, 2 c + 1; 2 c + 8, 2 c + 9
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      const int n = keys - 8 * i - 2 * c;
      keep[i] = n >= 2 ? 0xffffffffu : n == 1 ? 0x0000ffffu : 0u;
    }
  }
  if constexpr (E == 2) {
    load_matrices<true, 4>(a[0], half + T::at(tile * 16 + r + 8 * (m >> 1), 2 * t + (m & 1)));
    if constexpr (MASKED) a[0][0] &= keep[0], a[0][1] &= keep[0], a[0][2] &= keep[1], a[0][3] &= keep[1];
  } else {
    uint32_t w[4];
    constexpr bool kBoth = D >= 32;
    load_matrices<true, kBoth ? 4 : 2>(w, half + T::at(tile * 16 + r + 8 * (m & 1), kBoth ? t + (m >> 1) : t));
#pragma unroll
    for (int i = 0; i < (kBoth ? 2 : 1); ++i) {
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        uint32_t x = w[2 * i + k];
        if constexpr (MASKED) x &= keep[k];
        x = __byte_perm(x, 0, 0x3120);  // columns 2 g of both keys, then 2 g + 1
        a[i][2 * k] = e4m3x2_to_f16(x), a[i][2 * k + 1] = e4m3x2_to_f16(x >> 16);
      }
    }
  }
}
// ---------------------------------------------------------------- a warp's state of a unit
template <int D, int NT>
struct Rows {
  float o[NT][D / 16][4];
  float off[NT][2], l[NT][2];  // lift - maximum, sum, of query rows 2c, 2c + 1: a weight is 2^(score + off)
  int vis[NT][2];              // keys they see
  int min_vis;                 // least of all the unit's rows
};

// A score may pass the maximum by 2^kLag.  e4m3: weights are held 2^11 up (fp16 ones
// reach 2^15).  bf16: they are held down by 2^kLag and the number of keys, so that
// their sum is at most 1 and O stays within the largest value of V, whatever that is,
// at the price of bits of values below 2^-118 times the number of keys
// (7 requests of up to 3527 keys, 40 rows a head, a lag of 2^4 / 2^8: 44.4 / 43.6 us).
// That number's logarithm lies in shared memory: 32-row kernels have no register for it.
template <int E>
constexpr float kLag = E == 2 ? 8.f : 4.f;
template <int E>
__device__ __forceinline__ float lift(const float* factor) { return E == 1 ? 11.f : *factor; }

template <int D, int E, int NT>
__device__ __forceinline__ void start_rows(Rows<D, NT>& s, const AttnProblem& p, int Lq, int Lk, int row0, int lane) {
  const int c = lane & 3, rows = p.G * Lq;
  s.min_vis = Lk;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s.off[j][u] = -kNoMax;
      s.l[j][u] = 0.f;
      const int r = row0 + 8 * j + 2 * c + u;
      int vis = Lk;
      if (p.causal && r < rows) vis = min(max(Lk - Lq + query_of(p, r) + 1, 0), Lk);
      s.vis[j][u] = vis;
      s.min_vis = min(s.min_vis, vis);
    }
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int u = 0; u < 4; ++u) s.o[j][t][u] = 0.f;
  }
  s.min_vis = __reduce_min_sync(0xffffffffu, s.min_vis);
}

// The unit's queries, 16 bytes a thread and place (whole warps, or, of 16 columns
// and 8 rows, half of one), on their way to registers: they are asked for long
// before they are needed, since behind the copies that are under way a load takes
// some microseconds.
template <int D, int NT, int THREADS>
struct Queries {
  static constexpr int kLanes = D / 8, kPieces = 8 * NT * kLanes, kPer = (kPieces + THREADS - 1) / THREADS;
  uint4 u[kPer];
};
template <int D, int NT, int THREADS>
__device__ __forceinline__ void ask_queries(Queries<D, NT, THREADS>& s, const AttnProblem& p, int q0, int Lq, int h, int row0,
                                            int thread) {
  using Q = Queries<D, NT, THREADS>;
#pragma unroll
  for (int k = 0; k < Q::kPer; ++k) {
    const int i = k * THREADS + thread, r = row0 + i / Q::kLanes;
    uint4& u = s.u[k];
    u = make_uint4(0, 0, 0, 0);
    if (i < Q::kPieces && r < p.G * Lq) {
      const int tok = query_of(p, r);
      const __nv_bfloat16* src =
          p.q + (static_cast<long long>(q0 + tok) * p.H + h * p.G + (r - tok * p.G)) * D + i % Q::kLanes * 8;
      asm volatile("ld.global.nc.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(u.x), "=r"(u.y), "=r"(u.z), "=r"(u.w) : "l"(src));
    }
  }
}
// The same as B operands in shared memory: lane (g, c)'s two words of row tile j
// and step t at (j D / 16 + t) 256 + 8 lane.  e4m3: in fp16, each row divided by a
// power of two, whose product with the scale goes to `factor`.  bf16: lift() goes there.
template <int D, int E, int NT, int THREADS>
__device__ __forceinline__ void put_queries(uint32_t* sq, float* factor, const Queries<D, NT, THREADS>& s, float scale, int Lk, int thread) {
  using Q = Queries<D, NT, THREADS>;
  if (E == 2 && thread == 0) *factor = -kLag<E> - static_cast<float>(32 - __clz(Lk - 1));
#pragma unroll
  for (int k = 0; k < Q::kPer; ++k) {
    const int i = k * THREADS + thread;
    if (i >= Q::kPieces) break;
    const int local = i / Q::kLanes, x = i % Q::kLanes;
    uint32_t w[4] = {s.u[k].x, s.u[k].y, s.u[k].z, s.u[k].w};
    uint32_t* const to = sq + ((local >> 3) * (D / 16) + (x >> 1)) * 64 + (local & 7) * 8;
    if constexpr (E == 2) {
#pragma unroll
      for (int c = 0; c < 4; ++c) to[2 * c + (x & 1)] = w[c];
    } else {
      // the power of two at or below the row's largest finite magnitude (1 for a row
      // without one but 0): beside an infinity the others stay finite, too
      float mx = 0.f;
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 f = unpack_bf16x2(w[m]);
        mx = fmaxf(mx, fmaxf(finite_abs(f.x), finite_abs(f.y)));
      }
      constexpr uint32_t kMask = Q::kPieces >= 32 ? 0xffffffffu : (1u << (Q::kPieces & 31)) - 1u;
#pragma unroll
      for (int sh = 1; sh < Q::kLanes; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(kMask, mx, sh));
      const int e = mx == 0.f ? 0 : min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -126), 126);
      const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
#pragma unroll
      for (int m = 0; m < 4; ++m) {
        const float2 f = unpack_bf16x2(w[m]);
        w[m] = pack_f16x2(f.x * down, f.y * down);
      }
      // columns 4 c ..: lanes 2 (x & 1) and 2 (x & 1) + 1 of the row's four
      *reinterpret_cast<uint2*>(to + 4 * (x & 1)) = make_uint2(w[0], w[1]);
      *reinterpret_cast<uint2*>(to + 4 * (x & 1) + 2) = make_uint2(w[2], w[3]);
      // (kept off zero and infinity: the score of a masked key is -inf times it)
      if (x == 0) factor[local] = fminf(fmaxf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23) * scale, 1e-37f), 3e38f);
    }
  }
}

// P is a sum of two numbers.
constexpr int kParts = 2;

// Keys of a slot's tile i: its first `end` keys less those of the tiles before,
// none where its bit of `bad` is set (a page id out of range).
__device__ __forceinline__ int tile_keys(int end, uint32_t bad, int i) { return bad >> i & 1 ? 0 : min(max(end - 16 * i, 0), 16); }

// The products of a group of column blocks (t0 ..) with a tile's V where that has
// an infinity or NaN: rows that see the same number n of the tile's keys are taken
// together, V of later keys as zeros.
template <int D, int E, int NT>
__device__ __forceinline__ void odd_values(Rows<D, NT>& s, const uint32_t (&pb)[NT][kParts][2], uint32_t v_half, int tile, int t0,
                                           int key0, int keys, int lane) {
  constexpr int kSteps = D / 16, kPer = E == 1 && D >= 32 ? 2 : 1, kGroup = kSteps < 4 ? kSteps : 4;
#pragma unroll 1
  for (int n = 1; n <= keys; ++n) {
    bool mine = false;
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) mine |= min(s.vis[j][u] - key0, keys) == n;
    if (!__any_sync(0xffffffffu, mine)) continue;
    uint32_t a[kGroup][4];
#pragma unroll
    for (int t = 0; t < kGroup; t += kPer) load_v<D, E, true>(a + t, v_half, tile, t0 + t, n, lane);
#pragma unroll
    for (int t = 0; t < kGroup; ++t)
#pragma unroll
      for (int j = 0; j < NT; ++j) {
        float add[4] = {0.f, 0.f, 0.f, 0.f};
        mma<E == 1>(add, a[t], pb[j][0][0], pb[j][0][1]);
        if constexpr (E == 2) {  // (an infinity has met the high part)
          uint32_t v[4];
#pragma unroll
          for (int u = 0; u < 4; ++u) {
            v[u] = a[t][u];
            if ((v[u] & 0x7f80u) == 0x7f80u) v[u] &= 0xffff0000u;
            if ((v[u] >> 16 & 0x7f80u) == 0x7f80u) v[u] &= 0x0000ffffu;
          }
          mma<false>(add, v, pb[j][1][0], pb[j][1][1]);
        } else {
          mma<true>(add, a[t], pb[j][1][0], pb[j][1][1]);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u)
          if (min(s.vis[j][u & 1] - key0, keys) == n) s.o[j][t0 + t][u] += add[u];
      }
  }
}

// A slot's TILES 16-key tiles from `tile` on, keys key0 .., into the unit's state
// (two where they are there: their products are independent chains, and the
// step's fixed costs are shared).  Where some row does not see all their keys
// (MASKED), a tile's keys are tile_keys(end, bad, i); what shared memory holds past
// them has no influence.
template <int D, int E, int NT, int TILES, bool MASKED>
__device__ __forceinline__ void step(Rows<D, NT>& s, const uint32_t* sq, const float* factor, float scale, uint32_t k_half,
                                     int tile, int key0, int end, uint32_t bad, int lane) {
  using T = Tile<D, E>;
  constexpr int kSteps = D / 16, kPer = E == 1 && D >= 32 ? 2 : 1;
  const int g = lane >> 2, c = lane & 3;
  // (one tile of 8 rows: its sums in two halves, so that an instruction does not wait for
  // the one before it)
  constexpr bool kTwo = TILES * NT == 1 && kSteps > 1;
  float x[TILES][NT][4], cs[NT][2], odd[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int i = 0; i < TILES; ++i)
#pragma unroll
      for (int u = 0; u < 4; ++u) x[i][j][u] = 0.f;
    if constexpr (E == 1) {
      const float2 f = *reinterpret_cast<const float2*>(factor + 8 * j + 2 * c);
      cs[j][0] = f.x, cs[j][1] = f.y;
    } else {
      cs[j][0] = cs[j][1] = scale;
    }
  }
#pragma unroll
  for (int t = 0; t < kSteps; t += kPer) {
    uint2 b[NT][kPer];
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int k = 0; k < kPer; ++k) b[j][k] = *reinterpret_cast<const uint2*>(sq + (j * kSteps + t + k) * 64 + lane * 2);
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      uint32_t a[kPer][4];
      load_k<D, E>(a, k_half, tile + i, t, lane);
#pragma unroll
      for (int k = 0; k < kPer; ++k)
#pragma unroll
        for (int j = 0; j < NT; ++j) mma<E == 1>(kTwo && (t + k) % 2 ? odd : x[i][j], a[k], b[j][k].x, b[j][k].y);
    }
  }
  if constexpr (kTwo) {
#pragma unroll
    for (int u = 0; u < 4; ++u) x[0][0][u] += odd[u];
  }
  // x[i][j][0], [1]: key g, query rows 2c, 2c + 1; [2], [3]: key g + 8.
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int keys = tile_keys(end, bad, i);
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = g + (u >> 1) * 8;
          if (key >= keys || key0 + 16 * i + key >= s.vis[j][u & 1]) x[i][j][u] = -INFINITY;
        }
    }
  }
  float y[TILES][NT][4], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) y[i][j][u] = fmaf(x[i][j][u], cs[j][u & 1], s.off[j][u & 1]);
      top = fmax3(fmax3(top, y[i][j][0], y[i][j][1]), y[i][j][2], y[i][j][3]);
    }
  if (__builtin_expect(__any_sync(0xffffffffu, top > lift<E>(factor) + kLag<E>), 0)) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float mx = -INFINITY;
#pragma unroll
        for (int i = 0; i < TILES; ++i) mx = fmaxf(mx, fmaxf(x[i][j][u], x[i][j][u + 2]));
        mx *= cs[j][u];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        const float off = fminf(s.off[j][u], lift<E>(factor) - mx), down = ex2_approx(off - s.off[j][u]);
        s.off[j][u] = off;
        s.l[j][u] *= down;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
          s.o[j][t][u] *= down;
          s.o[j][t][u + 2] *= down;
        }
#pragma unroll
        for (int i = 0; i < TILES; ++i) {
          y[i][j][u] = fmaf(x[i][j][u], cs[j][u], s.off[j][u]);
          y[i][j][u + 2] = fmaf(x[i][j][u + 2], cs[j][u], s.off[j][u]);
        }
      }
  }
  uint32_t pb[TILES][NT][kParts][2];
#pragma unroll
  for (int i = 0; i < TILES; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float e[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) e[u] = ex2_approx(y[i][j][u]);
      s.l[j][0] += e[0] + e[2];
      s.l[j][1] += e[1] + e[3];
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        const uint32_t hi = pack<E == 1>(e[2 * k], e[2 * k + 1]);
        const float2 f = unpack<E == 1>(hi);
        pb[i][j][0][k] = transpose8x8(hi);
        pb[i][j][1][k] = transpose8x8(pack<E == 1>(e[2 * k] - f.x, e[2 * k + 1] - f.y));
      }
    }
  // O in groups of up to four blocks of columns.  An infinity or NaN in V takes
  // another way: 0 times it would reach rows that do not see its key, and the
  // low part of P times an infinity can be NaN.
  const uint32_t v_half = k_half + T::kHalf;
  constexpr int kGroup = kSteps < 4 ? kSteps : 4;
#pragma unroll
  for (int t0 = 0; t0 < kSteps; t0 += kGroup) {
#pragma unroll
    for (int i = 0; i < TILES; ++i) {
      const int keys = MASKED ? tile_keys(end, bad, i) : 16;
      uint32_t a[kGroup][4];
#pragma unroll
      for (int t = 0; t < kGroup; t += kPer) load_v<D, E, MASKED>(a + t, v_half, tile + i, t0 + t, keys, lane);
      if constexpr (MASKED || E == 2) {
        uint32_t bigs[4] = {0, 0, 0, 0};
#pragma unroll
        for (int t = 0; t < kGroup; ++t)
#pragma unroll
          for (int u = 0; u < 4; ++u) bigs[u] = max_abs<E == 1>(bigs[u], a[t][u]);
        const uint32_t big = max_abs<E == 1>(max_abs<E == 1>(bigs[0], bigs[1]), max_abs<E == 1>(bigs[2], bigs[3]));
        constexpr uint32_t kExp = E == 2 ? 0x7f80u : 0x7c00u;
        if (__builtin_expect(__any_sync(0xffffffffu, (big & kExp) == kExp || (big >> 16 & kExp) == kExp), 0)) {
          odd_values<D, E, NT>(s, pb[i], v_half, tile + i, t0, key0 + 16 * i, keys, lane);
          continue;
        }
      }
#pragma unroll
      for (int t = 0; t < kGroup; ++t)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
          for (int k = 0; k < kParts; ++k) mma<E == 1>(s.o[j][t0 + t], a[t], pb[i][j][k][0], pb[i][j][k][1]);
    }
  }
}

// Of a sum of weights 2^(score - m).
__device__ __forceinline__ float row_lse(float m, float l) { return (m + log2f(l)) * 0.69314718055994531f; }

// Row tiles of a unit, 8 rows each: as many as the K/V head has rows, up to 4.
inline int tiles_of(long long max_rows) { return max_rows <= 8 ? 1 : max_rows <= 16 ? 2 : 4; }


// For up to kShortKeys keys a request and warp, and 32 rows a K/V head: p.group (1, 2
// or 4) warps for each of the B * H_kv units.
constexpr int kShortKeys = 512;
int launch_short(const CacheMaps& maps, const AttnProblem& p, int d, int elem, cudaStream_t st);

}  // namespace kv_attn
}  // namespace fa2
