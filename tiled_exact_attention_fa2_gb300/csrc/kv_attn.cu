// Attention of new query tokens over a paged key-value cache in bf16 or e4m3.
//
// O = softmax(scale Q K^T) V over each request's cached keys, the queries
// being its last positions (causal: query i of Lq sees key j iff
// j <= i + Lk - Lq).  Bound by reading the cache once: 4 d bytes (2 d of e4m3)
// a key and K/V head against 4 d flops for each query head of its group; up to
// 32 query rows a K/V head stay below what mma.sync.m16n8k16 does in the time
// of the bytes, so the products are warp-level ones, and the design is about
// keeping copies in flight.
//
// Work.  A unit is (request, K/V head, 8 NT query rows); its keys are cut into
// slots of 16 keys (32 where a row of d values has at most 128 bytes).  All units
// lie on one line, numbered from the lengths by every CTA for itself, and are cut
// into items (layout() has the rule), the parts of a unit equally long.  A CTA (one
// an SM, 152) has eight warps that compute, one that finds items, one after the
// other, from an atomic queue, and three that start the TMA copies of the items'
// slots, each computing warp's into a ring of its own, several items ahead: no warp
// waits for another but at an item's end.  There the eight warps' results
// (unnormalised O, running maximum, sum) are joined in shared memory; those of a
// unit's part go to the workspace, and the CTA whose part is counted last joins them
// in the parts' order, with its next item.  Which warp reads which slot, and what is
// joined in which order, is the same whoever does it, so results do not vary.
// Few units of few keys have a cluster of CTAs each, whose results are joined
// through their shared memory (cluster_ctas() has the rule); many units of few keys
// have up to four warps each (kv_attn_short.cu).
//
// Measured (128 columns): 48 requests of up to 8191 keys, 8 K/V heads, bf16 149 us
// (6.8 TB/s, a copy's rate); 64 of up to 1024 36 us (4.8 TB/s); 2 of 131072 keys, 4 K/V
// heads, 4 queries each, e4m3 50.5 us (5 TB/s: the join of 19 parts of 16 rows takes
// some 7 us); 1 of 1000 keys, 8 heads, bf16 7.4 us (latency).  With 32 rows the products
// bound: 2 of up to 131072 keys, 8 queries each, 4 K/V heads, e4m3 76 us (bf16 alike, 7 of up to
// 3527 keys, 8 heads, 40 rows: 43.6 us, e4m3 43.8).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <chrono>
#include <climits>
#include <cmath>
#include <random>

#include "args.h"
#include "fa2.h"
#include "kv_attn.cuh"
#include "kv_cache.h"
#include "launch.h"

namespace fa2 {
namespace {

using namespace kv_attn;

__device__ int g_kv_attn_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

// ---------------------------------------------------------------- items
// The work in items, numbered along the line of all units: a unit, or one of the
// equal parts that it is cut into.
// Places for partial results, as many as layout() may ask for: a unit of s slots that is
// cut has at most 4/3 s / cut parts; with cuts of total / 608 and, of at most a quarter,
// total / 2432, that is 811 + 608 at most.
constexpr int kPlaces = 1440;
constexpr int kFewUnits = kCtas / 2;

struct Layout {
  int items, mine;         // items of this lane's requests and of those before; of its own
  int places;              // partial results of the requests before
  int per;                 // requests of a lane
  int cut, tail_cut;       // slots of an item at most (`up`), or about
  bool tail;               // this lane's requests are cut finer: they lie at the line's end
  bool up;                 // parts are counted by rounding up
  int total;               // items of all
};
__device__ __forceinline__ int parts_of(int slots, int cut, bool up) {
  const int c = static_cast<int>((static_cast<unsigned>(slots) + static_cast<unsigned>(up ? cut - 1 : cut / 2)) / static_cast<unsigned>(cut));
  return max(c, 1);
}
__device__ __forceinline__ int warp_upto(int v, int lane) {
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, v, i);
    if (lane >= i) v += u;
  }
  return v;
}

// What an item is.
struct Item {
  Request rq;
  int b, h, row0;         // request, K/V head, first row of the unit
  int first, len;         // its slots of the unit
  int parts, part, place; // parts of the unit, which of them it is, where its first one's result goes
};

// How the work is cut; a lane adds up its share of the requests.
// Few units: each into equal parts, as many as there are CTAs, so that all work is
// one wave.  Else units are cut where they are long, and handed out as CTAs become
// free: the SMs do not get their bytes at one rate (48 requests of up to 8191 keys,
// equal shares: 120 to 155 us by SM), finer towards the line's end.
template <int ROWS, int KEYS, int MIN_ITEM>
__device__ __forceinline__ Layout layout(const AttnProblem& p, bool& fine, bool& mixed, int lane) {
  Layout y;
  y.per = (p.B + 31) / 32;
  const int lo = min(lane * y.per, p.B), hi = min(lo + y.per, p.B);
  long long sum = 0;
  int units = 0;  // (total_q H fits 31 bits, and a unit has a row of it)
  Request r{};
  // (loops are not unrolled: one warp runs this once, so the instructions' way to the
  // SM counts)
#pragma unroll 1
  for (int b = lo; b < hi; ++b) {
    r = request(p, b);
    fine &= r.ok;
    if (p.cu_q) mixed |= out_of_order(p, b);
    sum += slots_of<ROWS, KEYS>(p, r);
    if (r.ok && r.Lk > 0) units += p.heads * row_tiles<ROWS>(p, r);
  }
  fine = __all_sync(0xffffffffu, fine);
  mixed = __any_sync(0xffffffffu, mixed);
  // (all lanes' sums together fit 31 bits: of very many slots they are counted by 2^shift)
  int shift = 0;
  while (__any_sync(0xffffffffu, sum >> shift >= 1 << 26)) ++shift;
  const int slots = static_cast<int>(sum >> shift);
  const int total = __reduce_add_sync(0xffffffffu, slots), all = __reduce_add_sync(0xffffffffu, units);
  auto full = [&](int n) { return static_cast<int>(min(static_cast<long long>(n) << shift, static_cast<long long>(INT_MAX / 4))); };
  const int share = full((total + kCtas - 1) / kCtas);
  y.tail = false;
  int places;
  // Of few units the least cut of kTries that gives a wave at most (total / (kCtas - all)
  // does), if it is not far above a share; else parts of shares; or (it does not happen,
  // kPlaces is enough) no cut at all.  Measured (128 columns, bf16; us, the queue's items and a
  // wave): 64 units of up to 20000 keys, 1.1 shares 64.9 and 60.4, 1.3 42.6 and 35.0; 72 units
  // of up to 60000, 1.9 shares 88.6 and 89.6 or (one more uneven) 120.3 and 119.7.  Nearer than
  // the rule goes, 1.7 shares, a wave is still ahead (64 units of up to 60000, 84.4 and 71.5).
  constexpr int kTries = 5;
  int attempt = all <= kFewUnits && total > 0 ? 0 : kTries;
#pragma unroll 1
  for (;; ++attempt) {
    y.up = attempt < kTries;
    if (y.up) {
      const int ctas = kCtas - all * attempt / (kTries - 1);
      y.cut = max(full((total + ctas - 1) / ctas), kWarps);
      if (y.cut < 8 * kWarps) y.cut = (y.cut + kWarps - 1) / kWarps * kWarps;  // (the same for the warps, fewer parts)
      y.tail_cut = y.cut;
    } else if (attempt == kTries) {
      y.cut = max((share + 3) / 4, MIN_ITEM);
      y.tail_cut = max((share + 15) / 16, MIN_ITEM);
      y.tail = warp_upto(slots, lane) - slots >= total - total / 4;
    } else {
      y.cut = y.tail_cut = INT_MAX / 4;
    }
    // items and places of this lane's requests
    const int cut = y.tail ? y.tail_cut : y.cut;
    y.mine = places = 0;
#pragma unroll 1
    for (int b = lo; b < hi; ++b) {
      if (y.per > 1) r = request(p, b);
      if (!r.ok || r.Lk == 0) continue;
      const int n = p.heads * row_tiles<ROWS>(p, r), c = parts_of(key_slots<KEYS>(r), cut, y.up);
      const int held = static_cast<int>(min(static_cast<long long>(n) * c, static_cast<long long>(kPlaces) + 1));
      y.mine += c > 1 ? held : n;
      if (c > 1) places = min(places + held, kPlaces + 1);
    }
    if (y.up) {
      if (__reduce_add_sync(0xffffffffu, y.mine) <= kCtas) {
        if (y.cut <= share + share / 2 || share <= 2 * MIN_ITEM) break;
        attempt = kTries - 1;
      }
    } else if (__reduce_add_sync(0xffffffffu, places) <= kPlaces) {
      break;
    }
  }
  y.items = y.mine;
  y.places = places;
#pragma unroll
  for (int i = 1; i < 32; i <<= 1) {
    const int u = __shfl_up_sync(0xffffffffu, y.items, i), v = __shfl_up_sync(0xffffffffu, y.places, i);
    if (lane >= i) y.items += u, y.places += v;
  }
  y.total = __shfl_sync(0xffffffffu, y.items, 31);
  y.places -= places;
  return y;
}

template <int ROWS, int KEYS>
__device__ __forceinline__ Item find_item(const Layout& y, const AttnProblem& p, int id, int lane) {
  const int owner = __ffs(__ballot_sync(0xffffffffu, y.items > id)) - 1;
  int before = __shfl_sync(0xffffffffu, y.items - y.mine, owner);
  int places = __shfl_sync(0xffffffffu, y.places, owner);
  const int cut = __ballot_sync(0xffffffffu, y.tail) >> owner & 1 ? y.tail_cut : y.cut;
  Item it;
  it.b = owner * y.per;
  if (y.per > 1) {  // which of the lane's requests: 32 at a time
    const int end = min(it.b + y.per, p.B);
    for (;; it.b += 32) {
      int items = 0, held = 0;
      if (it.b + lane < end) {
        const Request r = request(p, it.b + lane);
        if (r.ok && r.Lk > 0) {
          const int c = parts_of(key_slots<KEYS>(r), cut, y.up);
          items = p.heads * row_tiles<ROWS>(p, r) * c;
          held = c > 1 ? items : 0;
        }
      }
      const int upto = warp_upto(items, lane), held_upto = warp_upto(held, lane);
      const uint32_t past = __ballot_sync(0xffffffffu, before + upto > id);
      if (past || it.b + 32 >= end) {
        const int at = past ? __ffs(past) - 1 : 0;
        before += __shfl_sync(0xffffffffu, upto - items, at);
        places += __shfl_sync(0xffffffffu, held_upto - held, at);
        it.b += at;
        break;
      }
      before += __shfl_sync(0xffffffffu, upto, 31);
      places += __shfl_sync(0xffffffffu, held_upto, 31);
    }
  }
  it.rq = request(p, it.b);
  const int np = key_slots<KEYS>(it.rq), rt = row_tiles<ROWS>(p, it.rq);
  it.parts = parts_of(np, cut, y.up);
  int unit = id - before;
  it.part = it.place = it.first = 0;
  it.len = np;
  if (it.parts > 1) {
    const int rel = unit;
    unit = rel / it.parts;
    it.part = rel - unit * it.parts;
    it.place = places + unit * it.parts;
    it.first = static_cast<int>(quotient(static_cast<long long>(np) * it.part, it.parts));
    it.len = static_cast<int>(quotient(static_cast<long long>(np) * (it.part + 1), it.parts)) - it.first;
  }
  it.h = rt > 1 ? unit / rt : unit;
  it.row0 = (unit - it.h * rt) * ROWS;
  return it;
}

// ---------------------------------------------------------------- the kernel
// Slots below which a part of a unit costs more than it gives.
// (64 requests of up to 1024 keys, 8 heads of 128 columns, bf16, 32 / 64 / 128: 39.4 /
// 36.0 / 36.1 us; of up to 2048 66.4 / 63.5 / 61.6; 7 of up to 3527, 40 rows a head 58.0 /
// 48.5 / 44.9; joining more rows takes longer)
template <int D, int E, int NT>
constexpr int kMinItem = Tile<D, E>::kSlot >= 8192 ? (NT == 4 ? 128 : 64) : Tile<D, E>::kSlot >= 4096 ? 48 : 64;

template <int D>
constexpr int kJoinCols = D < 128 ? D : 64;  // columns of a round of the join

// Shared memory.  Slot i of an item is read by warp i mod kWarps (always, so that
// sums do not depend on what the CTA did before), from the warp's own ring, which is
// filled by the same copying warp always: a barrier's parity tells a round of a place
// from the one before it only.
constexpr int kDescs = 4;  // items that are described at a time, at most
constexpr int kAhead = 32; // slots: with fewer than these to come more than two items are described
constexpr int kMaxSmem = 232448;
struct Unit {
  int q0, Lq, h, row0;    // first query row and queries of its request, K/V head, first row
  int parts, place;       // parts that it is cut into, where the first one's result goes
};
// An item, or none (len 0).  Before it, the parts of another unit to be joined
// (join.parts 0: none), of which `group` is the one whose last part came.
struct Desc {
  Unit unit, join;
  int b, Lk, first, len, part, group;
  bool end, skip;         // no more follow; no rows are to be written at all
  bool live;              // of a cluster: there is a unit (this CTA's part of it may have no slot)
};
template <int D, int E, int NT>
struct Fixed {
  float join[kWarps][8][kJoinCols<D>];
  uint32_t q[NT * (D / 16) * 64];
  float2 ml[kWarps][8];
  float factor[8 * NT];
  Desc desc[kDescs];
  uint64_t desc_full[kDescs], desc_empty[kDescs];
  int last;
};
template <int D, int E, int NT>
struct Smem {
  static constexpr int kRing = 24576 / Tile<D, E>::kSlot < 8 ? 24576 / Tile<D, E>::kSlot : 8;  // slots of a warp
  alignas(1024) char ring[kWarps][kRing][Tile<D, E>::kSlot];
  uint64_t full[kWarps][kRing], empty[kWarps][kRing];
  uint32_t marks[kWarps][kRing];  // bit i: 16-key half i has a page id out of range
  Fixed<D, E, NT> f;
};

// The warps that compute.
__device__ __forceinline__ void sync_warps() { asm volatile("bar.sync 1, %0;" ::"n"(kWarps * 32) : "memory"); }

// Columns of a finished row: `n` consecutive ones from `col` on.
template <int N>
__device__ __forceinline__ void write_columns(__nv_bfloat16* dst, const float (&o)[N], float f) {
  if constexpr (N == 4) {
    *reinterpret_cast<uint2*>(dst) = make_uint2(pack_bf16x2(o[0] * f, o[1] * f), pack_bf16x2(o[2] * f, o[3] * f));
  } else if constexpr (N == 2) {
    *reinterpret_cast<uint32_t*>(dst) = pack_bf16x2(o[0] * f, o[1] * f);
  } else {
    dst[0] = __float2bfloat16_rn(o[0] * f);
  }
}

// The warps' results of an item joined: every warp takes one of eight rows.
// `part`, `ml`: where a part's result goes, or NULL for a unit that is whole.
template <int D, int E, int NT>
__device__ __forceinline__ void join_unit(Rows<D, NT>& s, Fixed<D, E, NT>& sm, const AttnProblem& p, const Unit& it, float* part,
                                          float2* ml, int warp, int lane) {
  constexpr int kCols = kJoinCols<D>, kLane = kCols >= 32 ? kCols / 32 : 1, kSteps = kCols / 16;
  const int g = lane >> 2, c = lane & 3;
#pragma unroll
  for (int j = 0; j < NT; ++j) {
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = s.l[j][u];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
      s.l[j][u] = l;
    }
    float top = 0.f, l = 0.f, w = 0.f;
#pragma unroll
    for (int round = 0; round < D / kCols; ++round) {
      if (j > 0 || round > 0) sync_warps();  // (the round before has been read)
      // (columns are stored with bits 3 and 4 turned by the row: no bank conflicts)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float* const row = sm.join[warp][2 * c + u];
        const int turn = (c << 3) & (kCols - 1) & 24;
#pragma unroll
        for (int t = 0; t < kSteps; ++t) {
          const float a = s.o[j][round * kSteps + t][u], b = s.o[j][round * kSteps + t][u + 2];
          if constexpr (E == 1) {
            *reinterpret_cast<float2*>(row + ((16 * t + 2 * g) ^ turn)) = make_float2(a, b);
          } else {
            row[(16 * t + g) ^ turn] = a;
            row[(16 * t + 8 + g) ^ turn] = b;
          }
        }
        if (round == 0 && g == 0) sm.ml[warp][2 * c + u] = make_float2(-s.off[j][u], s.l[j][u]);
      }
      sync_warps();
      if (round == 0) {
        const float2 v = lane < kWarps ? sm.ml[lane][warp] : make_float2(kNoMax, 0.f);
        top = v.x;
#pragma unroll
        for (int sh = 4; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
        top = __shfl_sync(0xffffffffu, top, 0);
        w = ex2_approx(v.x - top);
        l = w * v.y;
#pragma unroll
        for (int sh = 4; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
        l = __shfl_sync(0xffffffffu, l, 0);
      }
      const int turn = ((warp >> 1) << 3) & (kCols - 1) & 24, col = lane * kLane;
      float o[kLane];
#pragma unroll
      for (int k = 0; k < kLane; ++k) o[k] = 0.f;
#pragma unroll
      for (int i = 0; i < kWarps; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
        if (col < kCols) {
          const float* const src = &sm.join[i][warp][col ^ turn];
          float v[kLane];
          if constexpr (kLane == 4) {
            const float4 f = *reinterpret_cast<const float4*>(src);
            v[0] = f.x, v[1] = f.y, v[2] = f.z, v[3] = f.w;
          } else if constexpr (kLane == 2) {
            const float2 f = *reinterpret_cast<const float2*>(src);
            v[0] = f.x, v[1] = f.y;
          } else {
            v[0] = *src;
          }
#pragma unroll
          for (int k = 0; k < kLane; ++k) o[k] = fmaf(wi, v[k], o[k]);
        }
      }
      const int local = 8 * j + warp, r = it.row0 + local;
      if (r < p.G * it.Lq) {
        const int i0 = query_of(p, r), head = it.h * p.G + (r - i0 * p.G);
        const long long tok = it.q0 + i0;
        if (col < kCols) {
          const int at = round * kCols + col;
          if (part) {
            float* const dst = part + local * D + at;
            if constexpr (kLane == 4)
              *reinterpret_cast<float4*>(dst) = make_float4(o[0], o[1], o[2], o[3]);
            else if constexpr (kLane == 2)
              *reinterpret_cast<float2*>(dst) = make_float2(o[0], o[1]);
            else
              *dst = o[0];
          } else {
            write_columns<kLane>(p.o + (tok * p.H + head) * D + at, o, l == 0.f ? 0.f : p.v_scale / l);
          }
        }
        if (round == 0 && lane == 0) {
          if (part)
            ml[local] = make_float2(top, l);
          else
            p.lse[static_cast<long long>(head) * p.total_q + tok] = l == 0.f ? -INFINITY : row_lse(top, l);
        }
      }
    }
  }
}

// `count` <= 32 partial results of an item's unit (or of groups of them), at places
// from, from + step, ..., joined in that order by the CTA: into the first place if
// there are more, or to the outputs.
template <int D, int E, int ROWS>
__device__ __forceinline__ void join_parts(const AttnProblem& p, const Unit& it, int from, int step, int count, bool more, int warp, int lane) {
  constexpr int kCols = D >= 32 ? D / 32 : 1, kBatch = 20;  // (a wave's few units have 19 or 20 parts)
  const bool active = lane * kCols < D;
  for (int local = warp; local < ROWS && it.row0 + local < p.G * it.Lq; local += kWarps) {
    const float* const src = p.part + (static_cast<size_t>(from) * ROWS + local) * D + lane * kCols;
    const size_t apart = static_cast<size_t>(step) * ROWS * D;
    float v[kBatch][kCols];
    auto ask = [&](int i0) {  // (rows that are not there: zeros)
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float* const row = src + (i0 + i) * apart;
#pragma unroll
        for (int k = 0; k < kCols; ++k) v[i][k] = 0.f;
        if (i0 + i < count && active) {
          if constexpr (kCols == 4) {
            const float4 t = __ldcg(reinterpret_cast<const float4*>(row));
            v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
          } else if constexpr (kCols == 2) {
            const float2 t = __ldcg(reinterpret_cast<const float2*>(row));
            v[i][0] = t.x, v[i][1] = t.y;
          } else {
            v[i][0] = __ldcg(row);
          }
        }
      }
    };
    float2 ml = make_float2(kNoMax, 0.f);
    if (lane < count) ml = __ldcg(p.part_ml + (from + lane * step) * ROWS + local);
    ask(0);  // (on their way together)
    float top = ml.x, o[kCols];
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
    const float wt = ex2_approx(ml.x - top);
    float l = wt * ml.y;
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[k] = 0.f;
    for (int i0 = 0; i0 < count; i0 += kBatch) {
      if (i0 > 0) ask(i0);
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float wi = __shfl_sync(0xffffffffu, wt, (i0 + i) & 31);
        if (i0 + i < count) {
#pragma unroll
          for (int k = 0; k < kCols; ++k) o[k] = fmaf(wi, v[i][k], o[k]);
        }
      }
    }
    if (more) {
      float* const dst = p.part + (static_cast<size_t>(from) * ROWS + local) * D + lane * kCols;
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (active) dst[k] = o[k];
      if (lane == 0) p.part_ml[from * ROWS + local] = make_float2(top, l);
    } else {
      const int r = it.row0 + local, i = query_of(p, r), head = it.h * p.G + (r - i * p.G);
      const long long tok = it.q0 + i;
      if (active) write_columns<kCols>(p.o + (tok * p.H + head) * D + lane * kCols, o, l == 0.f ? 0.f : p.v_scale / l);
      if (lane == 0) p.lse[static_cast<long long>(head) * p.total_q + tok] = l == 0.f ? -INFINITY : row_lse(top, l);
    }
  }
}

// Counters.  A workspace may hold anything, so a counter counts only where it
// carries the call's number (in its upper 48 bits): a CTA sees to that for its
// share of them when it begins, or whoever adds before.  The last to add sets it
// back, so a graph may be replayed with the same number.
constexpr int kMaxRuns = 0xffff - kCtas;  // (each CTA asks once more than it is given)
__device__ __forceinline__ void claim(unsigned long long* counter, unsigned long long call) {
  const unsigned long long old = *static_cast<volatile unsigned long long*>(counter);
  if ((old ^ call) >> 16 != 0) atomicCAS(counter, old, call);  // (if another was faster, it is done)
}
// One more, and the count before (releases what the CTA has written, acquires what
// those before it have).
__device__ __forceinline__ unsigned long long add_one(unsigned long long* counter) {
  unsigned long long old;
  asm volatile("atom.add.acq_rel.gpu.global.u64 %0, [%1], 1;" : "=l"(old) : "l"(counter) : "memory");
  return old;
}
// The count before, of what add_one returned.
__device__ __forceinline__ unsigned long long counted(unsigned long long* counter, unsigned long long old, unsigned long long call) {
  while ((old ^ call) >> 16 != 0) {  // it was not this call's yet
    const unsigned long long seen = *static_cast<volatile unsigned long long*>(counter);
    if ((seen ^ call) >> 16 == 0) {
      old = add_one(counter);
    } else {
      unsigned long long got;
      asm volatile("atom.cas.acq_rel.gpu.global.b64 %0, [%1], %2, %3;"
                   : "=l"(got) : "l"(counter), "l"(seen), "l"(call + 1) : "memory");
      if (got == seen) old = call;  // (the first)
    }
  }
  return old - call;
}
// Whether all `count` parts are there with this one (the same for the CTA, whose
// threads have written theirs).
__device__ __forceinline__ bool arrive(unsigned long long* counter, unsigned long long call, int count, int* flag) {
  sync_warps();
  if (threadIdx.x == 0) {
    const bool last = static_cast<int>(counted(counter, add_one(counter), call)) + 1 == count;
    if (last) atomicExch(counter, call);
    *flag = last;
  }
  sync_warps();
  return *flag != 0;
}
// Parts of a unit that are joined at once; of more, each group of so many has a
// joined result first, so that no CTA reads the rows of all of them.
constexpr int kJoin = 32;

// Rows of requests without keys: zeros and -inf.
template <int D>
__device__ __forceinline__ void empty_rows(const AttnProblem& p, int warp, int lane) {
  for (int b0 = (blockIdx.x * kWarps + warp) * 32; b0 < p.B; b0 += kCtas * kWarps * 32) {
    Request rq{};
    if (b0 + lane < p.B) rq = request(p, b0 + lane);
    uint32_t left = __ballot_sync(0xffffffffu, rq.ok && rq.Lk == 0 && rq.Lq > 0);
    while (left) {
      const int from = __ffs(left) - 1;
      left &= left - 1;
      const long long q0 = __shfl_sync(0xffffffffu, rq.q0, from);
      const int Lq = __shfl_sync(0xffffffffu, rq.Lq, from);
      uint4* const dst = reinterpret_cast<uint4*>(p.o + q0 * p.H * D);
      for (long long i = lane; i < static_cast<long long>(Lq) * p.H * (D / 8); i += 32) dst[i] = make_uint4(0, 0, 0, 0);
      for (int h = 0; h < p.H; ++h)
        for (int i = lane; i < Lq; i += 32) p.lse[static_cast<long long>(h) * p.total_q + q0 + i] = -INFINITY;
    }
  }
}

// The finding warp: the CTA's items, one after the other, described to the other
// warps, and the count of their parts.  The first two items are the CTA's own, the
// others are taken from a queue.
template <int D, int E, int NT>
__device__ __forceinline__ void find_items(Fixed<D, E, NT>& sm, const AttnProblem& p, int lane) {
  constexpr int kRows = 8 * NT, kKeys = Tile<D, E>::kKeys;
  bool fine = true, mixed = false;
  // One join waits for the next description, no more: with a part of kAhead slots open, no third
  // item is described, so a second part is not done before.  (Parts of a wave may be
  // shorter; a CTA has one item of it.  A part is at least three quarters of the cut.)
  static_assert(kMinItem<D, E, NT> / 4 * 3 >= kAhead, "parts that are done before a finished unit's join is described");
  const Layout y = layout<kRows, kKeys, kMinItem<D, E, NT>>(p, fine, mixed, lane);
  if (blockIdx.x == 0 && lane == 0 && (!fine || mixed)) atomicCAS(&g_kv_attn_status, kDevOk, kDevBadSeqlens);
  int id = mixed ? INT_MAX : static_cast<int>(blockIdx.x);  // (offsets out of order: nothing is written)
  bool there = id < y.total;
  // The queue hands out runs of items, of one each unless they are more than its counter can count.
  const int left = max(y.total - 2 * kCtas, 0), run = left / kMaxRuns + 1, runs = (left + run - 1) / run;
  int until = 0;  // where the run that was taken ends
  int described = 0, done = 0, open = 0, ahead = 0;  // descriptions, those that are done; items and slots that are not done
  Unit join{};  // to be joined, of its group `group`
  int group = 0;
  auto describe = [&](Desc& d) {
    d.join = join;
    d.group = group;
    d.skip = mixed;
    join.parts = 0;
    if (lane == 0) {
      sm.desc[described % kDescs] = d;
      mbar_arrive(&sm.desc_full[described % kDescs]);
    }
    ++described;
  };
  for (;;) {
    if (there && (open < 2 || (described - done < kDescs && ahead < kAhead))) {
      if (id == INT_MIN) {  // (an item is better taken by a CTA that is free)
        if (lane == 0) {
          // (every CTA asks until it is told that there is no more; the last to hear so sets the queue back)
          const int n = static_cast<int>(counted(p.queue, add_one(p.queue), p.call));
          if (n == runs + min(kCtas, y.total - kCtas) - 1) atomicExch(p.queue, p.call);
          id = n < runs ? 2 * kCtas + n * run : INT_MAX;
        }
        id = __shfl_sync(0xffffffffu, id, 0);
        there = id < y.total;
        if (!there) continue;
        until = min(id + run, y.total);
      }
      Desc d{};
      const Item it = find_item<kRows, kKeys>(y, p, id, lane);
      d.unit = Unit{it.rq.q0, it.rq.Lq, it.h, it.row0, it.parts, it.place};
      d.b = it.b, d.Lk = it.rq.Lk, d.first = it.first, d.len = it.len, d.part = it.part;
      describe(d);
      ++open;
      ahead += it.len;
      if (described == 1) {
        // (counters that this CTA claims)
        for (int i = blockIdx.x + lane * kCtas; i < 2 * kPlaces; i += 32 * kCtas) claim(p.arrived + i, p.call);
        if (blockIdx.x == 0 && lane == 31) claim(p.queue, p.call);
        id += kCtas;
        there = id < y.total;
      } else {
        id = id + 1 < until ? id + 1 : INT_MIN;  // (the latter: from the queue, when there is room for it)
      }
      continue;
    }
    if (!there && open == 0) {
      Desc d{};
      d.end = true;
      describe(d);
      return;
    }
    if (!there && join.parts > 0) {
      Desc d{};
      describe(d);
      continue;
    }
    // What was described first and is not done yet.
    const int at = done % kDescs;
    if (!mbar_wait_warp(&sm.desc_empty[at], (done / kDescs) & 1, &g_kv_attn_status)) return;
    ++done;
    const int len = sm.desc[at].len, part = sm.desc[at].part;
    const Unit u = sm.desc[at].unit;
    __syncwarp();
    if (len == 0) continue;
    --open;
    ahead -= len;
    // The last part of a unit (of its group) to be counted has the unit joined.
    if (u.parts > 1) {
      int last = 0;
      if (lane == 0) {
        const bool one = u.parts <= kJoin;
        const int from = part / kJoin * kJoin, size = one ? u.parts : min(kJoin, u.parts - from);
        unsigned long long* const counter = p.arrived + (one ? u.place : kPlaces + u.place + from);
        last = static_cast<int>(counted(counter, add_one(counter), p.call)) + 1 == size;
        if (last) atomicExch(counter, p.call);
      }
      if (__shfl_sync(0xffffffffu, last, 0)) join = u, group = part / kJoin;
    }
  }
}

// The same where every unit has a cluster of CTAs: one item, its part of a unit.
template <int D, int E, int NT>
__device__ __forceinline__ void find_part(Fixed<D, E, NT>& sm, const AttnProblem& p, int lane) {
  constexpr int kRows = 8 * NT, kKeys = Tile<D, E>::kKeys;
  bool fine = true, mixed = false;
  for (int b = lane; b < p.B; b += 32) {
    fine &= request(p, b).ok;
    if (p.cu_q) mixed |= out_of_order(p, b);
  }
  mixed = __any_sync(0xffffffffu, mixed);
  if (blockIdx.x == 0 && (!fine || mixed)) atomicCAS(&g_kv_attn_status, kDevOk, kDevBadSeqlens);
  if (lane == 0) {
    const int unit = blockIdx.x / p.direct, rank = static_cast<int>(blockIdx.x) - unit * p.direct;
    const int head = unit / p.max_tiles, b = head / p.heads;
    const Request rq = request(p, b);
    Desc d{};
    d.unit = Unit{rq.q0, rq.Lq, head - b * p.heads, (unit - head * p.max_tiles) * kRows, 1, 0};
    d.b = b, d.Lk = rq.Lk;
    d.end = true, d.skip = mixed;
    d.live = !mixed && rq.ok && rq.Lk > 0 && d.unit.row0 < static_cast<long long>(p.G) * rq.Lq;
    if (d.live) {
      const int np = key_slots<kKeys>(rq);
      d.first = np * rank / p.direct;
      d.len = np * (rank + 1) / p.direct - d.first;
    }
    sm.desc[0] = d;
    mbar_arrive(&sm.desc_full[0]);
  }
}

// The parts of a cluster's CTAs, which lie at `part` (and `ml`) in their shared
// memory, joined in the CTAs' order: each CTA takes every p.direct-th row.
template <int D, int E, int ROWS>
__device__ __forceinline__ void join_cluster(const AttnProblem& p, const Unit& it, const float* part, const float2* ml, int rank, int warp,
                                             int lane) {
  constexpr int kLane = D >= 32 ? D / 32 : 1;
  const int col = lane * kLane;
  for (int local = warp * p.direct + rank; local < ROWS && it.row0 + local < p.G * it.Lq; local += kWarps * p.direct) {
    float m = kNoMax, l = 0.f, o[kLane];
    if (lane < p.direct) {
      m = load_cluster_f32(smem_u32(ml + local), lane);
      l = load_cluster_f32(smem_u32(ml + local) + 4, lane);
    }
    float top = m;
#pragma unroll
    for (int sh = 4; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
    top = __shfl_sync(0xffffffffu, top, 0);
    const float wt = ex2_approx(m - top);
    l *= wt;
#pragma unroll
    for (int sh = 4; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
    l = __shfl_sync(0xffffffffu, l, 0);
#pragma unroll
    for (int k = 0; k < kLane; ++k) o[k] = 0.f;
#pragma unroll 4
    for (int i = 0; i < p.direct; ++i) {
      const float wi = __shfl_sync(0xffffffffu, wt, i);
      if (col < D) {
#pragma unroll
        for (int k = 0; k < kLane; ++k) o[k] = fmaf(wi, load_cluster_f32(smem_u32(part + local * D + col + k), i), o[k]);
      }
    }
    const int r = it.row0 + local, i0 = query_of(p, r), head = it.h * p.G + (r - i0 * p.G);
    const long long tok = it.q0 + i0;
    if (col < D) write_columns<kLane>(p.o + (tok * p.H + head) * D + col, o, l == 0.f ? 0.f : p.v_scale / l);
    if (lane == 0) p.lse[static_cast<long long>(head) * p.total_q + tok] = l == 0.f ? -INFINITY : row_lse(top, l);
  }
}

// The next item's description, or none in time: the finding warp gives up, and ends,
// within one of its waits; this is longer.
__device__ __forceinline__ bool described(uint64_t* full, int k) {
  return mbar_wait_warp(&full[k % kDescs], (k / kDescs) & 1, &g_kv_attn_status, 4 * FA2_WAIT_TIMEOUT_NS);
}

// A copying warp: starts the copies for every kCopyWarps-th warp, as far ahead as
// their rings have room.  (One warp for all takes 560 cycles a slot of
// two copies, where 340 are there.)
constexpr int kCopyWarps = 3;
template <int D, int E, int NT>
__device__ __forceinline__ void copy_slots(Smem<D, E, NT>& sm, const CUtensorMap* maps, const AttnProblem& p, int which, int lane) {
  using T = Tile<D, E>;
  using S = Smem<D, E, NT>;
  constexpr int kKeys = T::kKeys;
  const int group = (kWarps - which + kCopyWarps - 1) / kCopyWarps;  // warps which + kCopyWarps m that this one copies for
  int copied[(kWarps + kCopyWarps - 1) / kCopyWarps] = {};           // slots of each so far
  for (int k = 0; described(sm.f.desc_full, k); ++k) {
    const Desc& d = sm.f.desc[k % kDescs];
    const int len = d.len, first = d.first, head = d.unit.h, Lk = d.Lk;
    const int* const table = p.table + d.b * p.table_stride;
    const bool end = d.end;
    for (int j0 = 0; j0 * kWarps < len * group; j0 += 32) {
      // a lane looks one of the next 32 slots up
      const int row = (j0 + lane) / group, m = j0 + lane - row * group, warp = which + kCopyWarps * m;
      const int mine = row * kWarps + warp, key = (first + mine) * kKeys;
      int count = row;
#pragma unroll
      for (int i = 0; i < static_cast<int>(sizeof(copied) / sizeof(int)); ++i) count += m == i ? copied[i] : 0;
      const int round = count / S::kRing, place = warp * S::kRing + count - round * S::kRing;
      int page[2] = {p.num_pages, p.num_pages};  // (a page past the last: the copy gives zeros)
      const bool there = mine < len, two = kKeys == 32 && p.shift == 4 && there && key + 16 < Lk;
      const int n = __popc(__ballot_sync(0xffffffffu, there));
      if (there) page[0] = __ldg(table + (key >> p.shift));
      if (two) page[1] = __ldg(table + (key >> p.shift) + 1);
      const int tok = key & ((1 << p.shift) - 1);
      uint32_t mark = 0;
#pragma unroll
      for (int i = 0; i < 2; ++i) {
        const bool bad = (i == 0 ? there : two) && static_cast<uint32_t>(page[i]) >= static_cast<uint32_t>(p.num_pages);
        if (bad) page[i] = p.num_pages, mark |= 1u << i;
      }
      if (p.shift > 4 && mark) mark = 3;  // (both halves lie in one page)
      if (mark) atomicCAS(&g_kv_attn_status, kDevOk, kDevBadIndex);
      for (int i = 0; i < n; ++i) {
        const int to = __shfl_sync(0xffffffffu, place, i), at = __shfl_sync(0xffffffffu, round, i);
        // (the round before has been read; of a fresh barrier that phase counts as complete)
        if (!mbar_wait_warp(&sm.empty[0][0] + to, (at & 1) ^ 1, &g_kv_attn_status)) return;
        if (lane == i) {
          uint64_t* const bar = &sm.full[0][0] + to;
          const uint32_t dst = smem_u32(sm.ring) + to * T::kSlot;
          (&sm.marks[0][0])[to] = mark;
          mbar_arrive_expect_tx(bar, T::kSlot);
#pragma unroll
          for (int kv = 0; kv < 2; ++kv) {
            tma_load_5d(dst + kv * T::kHalf, maps + kv, bar, tok, head, page[0]);
            if (kKeys == 32 && p.shift == 4)  // (a page's 16 keys are a copy)
              tma_load_5d(dst + kv * T::kHalf + 16 * T::kRow, maps + kv, bar, 0, head, page[1]);
          }
        }
      }
    }
#pragma unroll
    for (int i = 0; i < static_cast<int>(sizeof(copied) / sizeof(int)); ++i)
      copied[i] += max(len - (which + kCopyWarps * i) + kWarps - 1, 0) / kWarps;
    if (end) return;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.f.desc_empty[k % kDescs]);
  }
}

// Threads of a CTA: two warpgroups that compute, one that finds and copies.  32 rows
// of a unit need more than the 168 registers that 384 threads can have: the
// warpgroups then take 216, 216 and 72 (128 times their sum are the 384 x 168 that
// the block starts with).
constexpr int kThreads = (kWarps + 1 + kCopyWarps) * 32;

template <int D, int E, int NT>
__global__ void __launch_bounds__(kThreads, 1)
    fa2_kv_attn_kernel(const __grid_constant__ CacheMaps maps, const __grid_constant__ AttnProblem p) {
  using T = Tile<D, E>;
  using S = Smem<D, E, NT>;
  constexpr int kRows = 8 * NT, kKeys = T::kKeys;
  extern __shared__ __align__(1024) char raw[];
  S& sm = *reinterpret_cast<S*>(raw);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  if (smem_u32(raw) & 1023u) {  // (the copies' swizzle goes by the address)
    if (threadIdx.x == 0) atomicCAS(&g_kv_attn_status, kDevOk, kDevSmemMisaligned);
    return;
  }
  for (int i = threadIdx.x; i < kWarps * S::kRing; i += blockDim.x) {
    mbar_init(&sm.full[0][0] + i, 1);
    mbar_init(&sm.empty[0][0] + i, 1);
  }
  if (threadIdx.x < kDescs) {
    mbar_init(&sm.f.desc_full[threadIdx.x], 1);
    mbar_init(&sm.f.desc_empty[threadIdx.x], kWarps + kCopyWarps);
  }
  fence_mbar_init();
  if (threadIdx.x < 2) tma_prefetch_desc(&maps.kv[threadIdx.x]);
  __syncthreads();
  griddep_wait();
  griddep_launch_dependents();
  // A CTA needs, one after the other, the lengths, then page ids and queries: the
  // lines of the latter two start on their way to L2 while the first is read.
  {
    const size_t line = (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 128;
    if (line < p.table_bytes) prefetch_l2(reinterpret_cast<const char*>(p.table) + line);
    if (line < p.q_bytes) prefetch_l2(reinterpret_cast<const char*>(p.q) + line);
  }
  if (warp >= kWarps) {
    if constexpr (NT == 4) asm volatile("setmaxnreg.dec.sync.aligned.u32 72;");
    if (warp == kWarps && p.direct)
      find_part<D, E, NT>(sm.f, p, lane);
    else if (warp == kWarps)
      find_items<D, E, NT>(sm.f, p, lane);
    else
      copy_slots<D, E, NT>(sm, maps.kv, p, warp - kWarps - 1, lane);
    return;
  }
  if constexpr (NT == 4) asm volatile("setmaxnreg.inc.sync.aligned.u32 216;");
  Queries<D, NT, kWarps * 32> queries;
  Rows<D, NT> s;
  bool alive = true;
  uint32_t slot = 0, phase = 0;
  if (!described(sm.f.desc_full, 0)) return;
  auto ask = [&](const Desc& d) {
    if (d.len > 0 || d.live) ask_queries(queries, p, d.unit.q0, d.unit.Lq, d.unit.h, d.unit.row0, threadIdx.x);
  };
  ask(sm.f.desc[0]);
  for (int k = 0;; ++k) {
    const Desc& it = sm.f.desc[k % kDescs];
    const Desc& next = sm.f.desc[(k + 1) % kDescs];
    if (it.join.parts > 0) {
      const Unit u = it.join;
      if (u.parts <= kJoin) {
        join_parts<D, E, kRows>(p, u, u.place, 1, u.parts, false, warp, lane);
      } else {
        const int from = it.group * kJoin;
        join_parts<D, E, kRows>(p, u, u.place + from, 1, min(kJoin, u.parts - from), true, warp, lane);
        const int groups = (u.parts + kJoin - 1) / kJoin;
        if (arrive(p.arrived + u.place, p.call, groups, &sm.f.last)) join_parts<D, E, kRows>(p, u, u.place, kJoin, groups, false, warp, lane);
      }
    }
    bool known = false;  // the next is described
    if (it.len > 0 || it.live) {
      const int first = it.first, len = it.len, Lk = it.Lk;
      put_queries<D, E>(sm.f.q, sm.f.factor, queries, p.scale_log2, Lk, threadIdx.x);
      start_rows<D, E, NT>(s, p, it.unit.Lq, Lk, it.unit.row0, lane);
      known = !it.end && __all_sync(0xffffffffu, mbar_test_wait(&sm.f.desc_full[(k + 1) % kDescs], ((k + 1) / kDescs) & 1));
      if (known) ask(next);
      sync_warps();
      for (int i = warp; i < len; i += kWarps) {
        if (alive && !mbar_wait_warp(&sm.full[warp][slot], phase, &g_kv_attn_status)) {
          alive = false;  // a copy that never came: the unit's rows are wrong, with the status word set
          mbar_wait_warp(&sm.full[warp][slot], phase, &g_kv_attn_status);
        }
        if (!alive) break;
        const uint32_t half = smem_u32(sm.ring[warp][slot]), out = sm.marks[warp][slot];
        constexpr int kAtOnce = T::kTiles < 2 || D * NT > 256 ? 1 : 2;  // (32 rows of 128 columns have no registers for two)
#pragma unroll 1
        for (int tile = 0; tile < T::kTiles; tile += kAtOnce) {
          const int k0 = (first + i) * kKeys + 16 * tile;
          if (k0 >= Lk) break;
          if (k0 + 16 * kAtOnce <= s.min_vis && out == 0)
            step<D, E, NT, kAtOnce, false>(s, sm.f.q, sm.f.factor, p.scale_log2, half, tile, k0, 0, 0, lane);
          else
            step<D, E, NT, kAtOnce, true>(s, sm.f.q, sm.f.factor, p.scale_log2, half, tile, k0, Lk - k0, out >> tile, lane);
        }
        __syncwarp();  // every lane has read the slot
        if (lane == 0) mbar_arrive(&sm.empty[warp][slot]);
        if (++slot == S::kRing) slot = 0, phase ^= 1;
      }
      const size_t place = static_cast<size_t>(it.unit.place + it.part) * kRows;
      float* part = it.unit.parts == 1 ? nullptr : p.part + place * D;
      float2* ml = it.unit.parts == 1 ? nullptr : p.part_ml + place;
      if (p.direct > 1) {  // (the ring has been read to its end)
        part = reinterpret_cast<float*>(sm.ring);
        ml = reinterpret_cast<float2*>(part + kRows * D);
      }
      join_unit<D, E, NT>(s, sm.f, p, it.unit, part, ml, warp, lane);
    }
    if (p.direct > 1) {
      cluster_sync();
      const float* const part = reinterpret_cast<const float*>(sm.ring);
      if (it.live)
        join_cluster<D, E, kRows>(p, it.unit, part, reinterpret_cast<const float2*>(part + kRows * D), static_cast<int>(cluster_rank()), warp, lane);
      cluster_sync();  // (no CTA leaves while another reads its rows)
    }
    if (it.end) break;
    __syncwarp();
    if (lane == 0) mbar_arrive(&sm.f.desc_empty[k % kDescs]);  // (releases the part, too)
    if (!known) {
      if (!described(sm.f.desc_full, k + 1)) return;
      ask(next);
    }
  }
  if (!sm.f.desc[0].skip) empty_rows<D>(p, warp, lane);
}

// ---------------------------------------------------------------- host
// Few units whose keys are few get a cluster of CTAs each: no line to lay out, no
// queue, no workspace.  How many CTAs a unit may have, 0 for the line.  Measured
// (8 K/V heads of 128 columns, bf16; us, the line and the cluster): 1 request of 128
// keys 6.1 and 4.7, 1000: 8.6 and 7.4, 4000: 9.8 and 9.6, 8000: 12.1 and 13.1; 4 of
// up to 2000: 10.7 and 9.4; 8 of up to 1024: 11.9 and 9.2; 16 of up to 512: 9.2 and
// 7.4, 2048: 25.9 and 20.4, 4096: 40.3 and 35.4, but one long request among short ones
// would wait for its one CTA.  (Not by type and columns: they were not measured.)
inline int cluster_ctas(int B, int H_kv, long long max_rows, int max_keys) {
  const int rows = 8 * tiles_of(max_rows);
  const long long units = static_cast<long long>(B) * H_kv * ((max_rows + rows - 1) / rows);
  // (a cluster's CTAs lie in one GPC: 32 clusters of 4 find room at once, 16 of 8 do not, 8.9 and 13.3 us)
  const int most = units <= 8 ? 8 : units <= 32 ? 4 : units <= 64 ? 2 : units <= kCtas ? 1 : 0;
  return max_keys <= (most == 1 ? 2048 : 448 * (most + 1)) ? most : 0;
}

// Many units of few keys, one a K/V head and request, have four warps, two or one each
// (launch_short): as many as make about a wave of 152 x 8.  0: the line, where a warp's
// chain of slots would be longer, or units too many for what more than one warp gives.
// Measured (8 K/V heads of 128 columns, bf16; us, the line and one / two / four warps):
// 20 requests of up to 120 keys 9.6 and 9.0 / 7.3 / 6.6, 512: 13.0 and 26.6 / 16.0 / 11.6,
// 1000: 21.5 and - / 27.5 / 19.9, 2000: 28.2 and - / - / 33.3; 40 of 120: 12.7 and 9.3 / 8.1 /
// 9.7, 512: 19.8 and 26.9 / 19.5 / 22.0, 1000: 27.2 and - / 30.9 / 31.2; 64 of 1000: 36.8 and
// - / 36.2 / 39.2; 100 of 120: 22.0 and 11.7 / 14.5 / 16.9,
// 512: 33.9 and 31.9 / 33.5 / 31.8, 1000: 49.6 and - / 59.6 / 52.5; 300 of 1000: 127 and - /
// 135 / 129, with 16 rows a unit 152 and - / 145 / 147, 32 rows 246 and - / 205 / 218.
// e4m3: 20 of 120 9.9 and 7.1 / 6.5 / 6.0, 512: 11.5 and 16.0 / 10.7 / 9.0; 40 of 120 14.2 and
// 6.6 / 6.4 / 9.1, 512: 16.3 and 15.8 / 11.9 / 13.4; 64 of 1000 28.1 and - / 23.3 / 24.8; 100 of
// 120 25.2 and 7.9 / 10.6 / 14.3, 512: 30.4 and 21.4 / 22.7 / 23.8; 300 of 1000 with 16 rows 138
// and - / 120 / 125.  64 columns: 64 of 1000 24.4 and - / 19.8 / 21.6 (e4m3 21.2 and - / 18.0 /
// 19.7), 40 of 512, 4 rows 13.4 and 14.3 / 10.1 / 11.7; 32 columns: 100 of 512, 4 rows 21.2 and
// 14.8 / 16.3 / 16.6.  The rule does not go by type, and so takes the slower for 300 of 1000 in
// e4m3, 8 rows or fewer (93.5 and - / 73.0 / 82.6) and, by 3 %, 32 (236 and - / 244 / 264).
inline int warps_each(int B, int H_kv, long long max_rows, int max_keys) {
  const long long units = static_cast<long long>(B) * H_kv;
  if (max_rows > 32 || units > 1 << 30 || cluster_ctas(B, H_kv, max_rows, max_keys)) return 0;
  if (units <= 2 * kCtas) return max_keys <= 2 * kShortKeys ? 4 : 0;
  if (units <= 4 * kCtas) return max_keys <= 2 * kShortKeys && max_keys <= 2 * units ? 2 : 0;
  if (max_keys <= kShortKeys) return 1;
  return max_rows > 8 && units >= 8 * kCtas && max_keys <= 2 * kShortKeys ? 2 : 0;
}

template <int D, int E, int NT>
int launch_attn_nt(const CacheMaps& maps, const AttnProblem& p, cudaStream_t st) {
  constexpr int kSmem = sizeof(Smem<D, E, NT>);
  static_assert(kSmem <= kMaxSmem, "shared memory of a CTA");
  static_assert(sizeof(Smem<D, E, NT>::ring) >= 8 * NT * (D * 4 + 8), "a part's rows fit the ring");
  const auto kernel = fa2_kv_attn_kernel<D, E, NT>;
  if (int e = ensure_max_smem(reinterpret_cast<const void*>(kernel), kSmem)) return e;
  if (p.direct) {
    const dim3 grid(static_cast<unsigned>(p.B) * p.heads * p.max_tiles * p.direct);
    return p.direct > 1 ? launch_pdl_cluster(kernel, grid, dim3(kThreads), kSmem, st, p.direct, maps, p)
                        : launch_pdl(kernel, grid, dim3(kThreads), kSmem, st, maps, p);
  }
  return launch_pdl(kernel, dim3(kCtas), dim3(kThreads), kSmem, st, maps, p);
}

template <int D, int E>
int launch_attn(const CacheMaps& maps, const AttnProblem& p, cudaStream_t st) {
  switch (tiles_of(static_cast<long long>(p.max_q) * p.G)) {
    case 1: return launch_attn_nt<D, E, 1>(maps, p, st);
    case 2: return launch_attn_nt<D, E, 2>(maps, p, st);
    default: return launch_attn_nt<D, E, 4>(maps, p, st);
  }
}

// A number for a call's counters, from a random one on: a word that a workspace
// happens to hold has it by a chance of 2^-48, one of those that a call may count in
// by 2^-36.
unsigned long long first_call() {
  try {
    std::random_device r;
    return static_cast<unsigned long long>(r()) << 32 ^ r();
  } catch (...) {  // (no source of random numbers: the clock)
    return static_cast<unsigned long long>(std::chrono::steady_clock::now().time_since_epoch().count()) * 0xd1342543de82ef95ull;
  }
}
unsigned long long next_call() {
  static std::atomic<unsigned long long> number{first_call()};
  return number.fetch_add(0x9e3779b97f4a7c15ull, std::memory_order_relaxed) & ~0xffffull;
}

size_t part_rows(int nt) { return static_cast<size_t>(kPlaces) * 8 * nt; }

constexpr int kMaxKeys = 1 << 30;  // of a request: positions, rounded up, in 32 bits

int check_attn_sizes(int B, int H, int H_kv, int total_q, int max_q, int d) {
  if (B < 1 || H < 1 || total_q < 0 || max_q < 0 || total_q > (1 << 30)) return FA2_ERR_SHAPE;
  if (total_q == 0) max_q = 0;  // (a step without queries, whatever the bound)
  if (max_q > total_q || (total_q > 0 && max_q < 1)) return FA2_ERR_SHAPE;
  if (!head_dim_ok(d)) return FA2_ERR_HEADDIM;
  if (int rc = check_heads(H, H_kv)) return rc;
  if (static_cast<long long>(H / H_kv) * max_q > (1LL << 30) || static_cast<long long>(total_q) * H > 0x7fffffffLL) return FA2_ERR_SHAPE;
  return FA2_OK;
}

}  // namespace

int read_kv_attn_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_kv_attn_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_kv_attn_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

extern "C" {

size_t fa2_kv_attn_workspace_bytes(int B, int H, int H_kv, int max_seqlen_q, int max_seqlen_k, int d) {
  if (max_seqlen_q < 1 || max_seqlen_k < 1 || check_attn_sizes(B, H, H_kv, max_seqlen_q, max_seqlen_q, d) != FA2_OK) return 0;
  const long long max_rows = static_cast<long long>(H / H_kv) * max_seqlen_q;
  if (cluster_ctas(B, H_kv, max_rows, max_seqlen_k) || warps_each(B, H_kv, max_rows, max_seqlen_k)) return 0;
  const size_t rows = part_rows(tiles_of(max_rows));
  return round_up(rows * d * sizeof(float)) + round_up(rows * sizeof(float2)) + round_up((2 * kPlaces + 1) * sizeof(long long));
}

int fa2_kv_attn(const void* q, const void* k_cache, const void* v_cache, const long long* cache_strides, int cache_type,
                const int* block_table, long long table_stride, const int* lens, const int* cu_seqlens_q, void* o, float* lse, int B,
                int H, int H_kv, int total_q, int max_seqlen_q, int max_seqlen_k, int num_pages, int page_size, int table_width, int d,
                float scale, float k_scale, float v_scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_attn_sizes(B, H, H_kv, total_q, max_seqlen_q, d)) return rc;
  Strided c[2];
  if (int rc = check_kv(c, k_cache, v_cache, cache_strides, cache_type, num_pages, page_size, H_kv, d, k_scale, v_scale)) return rc;
  if (table_width < 1 || (B > 1 && (table_stride < table_width || !stride_ok(table_stride, B)))) return FA2_ERR_SHAPE;
  if (max_seqlen_k < 1) return FA2_ERR_SHAPE;
  if (max_seqlen_k > kMaxKeys) max_seqlen_k = kMaxKeys;
  if (static_cast<long long>(table_width) * page_size < max_seqlen_k) max_seqlen_k = table_width * page_size;
  if (!cu_seqlens_q && total_q > 0 && static_cast<long long>(B) * max_seqlen_q != total_q) return FA2_ERR_SHAPE;
  if (check_scale(scale) || check_scale(scale * k_scale)) return FA2_ERR_SCALE;
  if (total_q == 0) return FA2_OK;
  if (!q || !block_table || !lens || !o || !lse) return FA2_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(lse, 4))
    return FA2_ERR_ALIGN;
  const size_t need = fa2_kv_attn_workspace_bytes(B, H, H_kv, max_seqlen_q, max_seqlen_k, d);
  if (need > 0 && (!workspace || !aligned(workspace, kWsAlign) || workspace_bytes < need)) return FA2_ERR_WORKSPACE;
  const size_t qb = static_cast<size_t>(total_q) * H * d * 2;
  const size_t tb = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
  const Range outs[] = {range_of(o, qb), range_of(lse, static_cast<size_t>(total_q) * H * 4), range_of(workspace, need)};
  const Range ins[] = {range_of(q, qb),
                       span_of(c[0]),
                       span_of(c[1]),
                       range_of(block_table, tb),
                       range_of(lens, static_cast<size_t>(B) * 4),
                       range_of(cu_seqlens_q, cu_seqlens_q ? static_cast<size_t>(B + 1) * 4 : 0)};
  for (int i = 0; i < (need > 0 ? 3 : 2); ++i) {
    for (const Range& r : ins)
      if (r.lo != r.hi && overlap(outs[i], r)) return FA2_ERR_ALIAS;
    for (int j = i + 1; j < (need > 0 ? 3 : 2); ++j)
      if (overlap(outs[i], outs[j])) return FA2_ERR_ALIAS;
  }
  CacheMaps maps;
  for (int i = 0; i < 2; ++i)
    if (!make_tmap_paged(&maps.kv[i], c[i], d > 128 / c[i].elem ? 16 : page_size < 32 ? 16 : 32))
      return record_cuda_failure(static_cast<int>(cudaErrorInvalidValue), "tensor map of the cache");
  AttnProblem p{};
  const size_t rows = part_rows(tiles_of(static_cast<long long>(H / H_kv) * max_seqlen_q));
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.table = block_table;
  p.table_stride = table_stride;
  p.lens = lens;
  p.cu_q = cu_seqlens_q;
  if (need > 0) {
    char* ws = static_cast<char*>(workspace);
    p.part = reinterpret_cast<float*>(ws);
    ws += round_up(rows * d * sizeof(float));
    p.part_ml = reinterpret_cast<float2*>(ws);
    ws += round_up(rows * sizeof(float2));
    p.arrived = reinterpret_cast<unsigned long long*>(ws);
    p.queue = p.arrived + 2 * kPlaces;
    p.call = next_call();
  }
  const long long max_rows = static_cast<long long>(H / H_kv) * max_seqlen_q;
  p.group = warps_each(B, H_kv, max_rows, max_seqlen_k);
  p.direct = cluster_ctas(B, H_kv, max_rows, max_seqlen_k);
  // (of 24 slots one CTA is through as soon as several have met: 500 keys 7.1 us both)
  if (p.direct > 1 && max_seqlen_k <= 24 * (d * c[0].elem > 128 ? 16 : 32)) p.direct = 1;
  p.max_tiles = static_cast<int>((max_rows + 8 * tiles_of(max_rows) - 1) / (8 * tiles_of(max_rows)));
  // (r / G by a product: the usual multiplier one bit longer than the word, whose top bit is the addition)
  while ((1u << p.g_shift) < static_cast<uint32_t>(H / H_kv)) ++p.g_shift;
  p.g_mul = static_cast<uint32_t>(((1ull << 32) * ((1ull << p.g_shift) - H / H_kv)) / (H / H_kv) + 1);
  p.table_bytes = tb;
  p.q_bytes = qb;
  p.num_pages = num_pages;
  while ((1 << p.shift) < page_size) ++p.shift;
  p.heads = H_kv;
  p.B = B;
  p.H = H;
  p.G = H / H_kv;
  p.total_q = total_q;
  p.max_q = max_seqlen_q;
  p.max_k = max_seqlen_k;
  p.scale_log2 = scale * k_scale * 1.44269504088896341f;
  p.v_scale = v_scale;
  p.causal = causal != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  g_launched = true;
  int e;
  if (p.group)
    e = launch_short(maps, p, d, c[0].elem, st);
  else if (cache_type == FA2_KV_E4M3)
    e = d == 16 ? launch_attn<16, 1>(maps, p, st) : d == 32 ? launch_attn<32, 1>(maps, p, st) : d == 64 ? launch_attn<64, 1>(maps, p, st)
                                                                                                       : launch_attn<128, 1>(maps, p, st);
  else
    e = d == 16 ? launch_attn<16, 2>(maps, p, st) : d == 32 ? launch_attn<32, 2>(maps, p, st) : d == 64 ? launch_attn<64, 2>(maps, p, st)
                                                                                                       : launch_attn<128, 2>(maps, p, st);
  return e ? record_cuda_failure(e, "kv attention launch") : FA2_OK;
}

}  // extern "C"
