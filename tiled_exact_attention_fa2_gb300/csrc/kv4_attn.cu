// Attention of new query tokens over a paged key-value cache held in 4 bits.
//
// O = softmax(scale Q K^T) V over each request's cached keys, the queries
// being its last positions (causal: query i of Lq sees key j iff
// j <= i + Lk - Lq).  Bound by reading the cache once: 9 d / 8 bytes a key
// and K/V head against 4 d flops for each query head of its group, far below
// the balance of even the warp-level matrix instructions (1024 fp16
// multiply-adds a clock and SM, measured), so the products are
// mma.sync.m16n8k16 on operands decoded in registers.  A tcgen05 operand in
// shared memory would have to be written there in 16 bits first, 3.6 times the
// bytes that come in; keys decoded into TMEM (as the A operand, 128 of them)
// would not, but pay only where a K/V head has more rows than the 8 or 16 of a
// unit here: a unit reads and decodes its keys for itself, so the time grows
// with every 16 rows.
//
// Work.  A unit is (request, K/V head, 8 NT query rows), its keys pairs of
// 16-key tiles; row r of a unit is query r / G, head r % G of the group.  All
// units' pairs form one line, which is cut into equal spans, one for each
// warp: every warp reads as many bytes as any other, whatever the lengths.
// A unit inside one span is finished by its warp; one that spans share leaves
// a partial result per span (unnormalised O, running maximum and sum), which
// the combine kernel joins in span order (where very many share a unit, each
// CTA's warps first).  Warps share nothing on the way, and the result does not
// depend on the order they run in.  Units
// of short requests take one CTA each instead, whose warps share the unit's
// keys and join in shared memory.
//
// Operands (lane (g, c) = (lane / 4, lane % 4)).  The first product is
// S^T = K Q^T: a tile's 16 keys are the rows of the instruction and the 8
// query rows its columns, which wastes none of it on a group of 8 heads.  The
// columns of K are a contraction index, so their order is free as long as Q
// has the same: lane c holds columns c d/4 .. of keys g and g + 8, contiguous
// in the cache.  The second is O^T = V^T P^T, columns of V as rows: lane g
// holds columns g d/8 .. of keys 2c, 2c+1, 2c+8, 2c+9, and one
// byte-interleave of two keys' codes makes the pairs along the contraction
// that the instruction wants before they are decoded.  P^T comes from S^T's
// registers by two 8x8 transposes (movmatrix).
//
// Measured on a GB300 (device time, 8 and 4 K/V heads of 128 columns): 48
// requests of up to 8191 keys, one query and 4 heads a group, 55.6 us (5.14
// TB/s of cache; between two lengths the marginal rate is 6.9 TB/s, a copy's:
// the rest is 6 us until the first tiles arrive, about 4 us for the combine
// kernel and as much between the first and the last warp's end); two requests
// of 131072 keys, four queries and 4 heads a group (16 rows), 45.7 us, of which
// about 14 do not depend on the length (262144 and 524288 keys: 79 and 142 us)
// and the others are 72.5 ns, about 145 cycles, an SM and tile.  Of these its
// bytes would take 100 cycles and its 32 matrix instructions, 64 decodes and 64
// scalings 107 if nothing waited; with 12 warps an SM (168 registers) the
// schedulers issue in half of the cycles, and their three warps wait most for
// fixed latencies (1.8 of the 6 cycles between two instructions of a warp) and
// for the matrix and ALU pipes (0.9): as much latency as issue.  One request of
// 1000 keys 8.0 us, bound by latency.
//
// Precision.  Cache values are exact in fp16 (6 significant bits), Q (8 bits)
// is divided by a power of two per row so that its largest value is in
// [1, 2), which is exact in fp16 down to 2^-14 of it (2^-25 absolute below),
// so S is exact up to its fp32 sums.  P is rounded to fp16 (11 bits against
// bf16's 8), held 2^11 up so that weights down to 2^-25 of the largest keep
// all 11.  The running maximum is raised only when a score passes it by 2^4
// (weights then reach 2^15, inside fp16), which saves the tile's maximum
// (three shuffles per column) and the rescaling of O for nearly every tile;
// maximum, sum, O are fp32 and the final quotient removes the common factor
// exactly.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <climits>
#include <cmath>

#include "args.h"
#include "fa2.h"
#include "kv4.cuh"
#include "launch.h"

namespace fa2 {
namespace {

__device__ int g_attn4_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

// Warps of a CTA (one CTA per SM): as many as the registers of 8 and of 16
// rows allow.
template <int NT>
constexpr int kWarps = NT == 1 ? 16 : 12;
constexpr int kCtas = 152;  // one wave
// From this many spans of a unit on its CTAs join theirs before the combine
// kernel, whose time else grows with them.  Measured, 128 columns, joined /
// not, in us: one unit of 131072 keys 15.6 / 36, 8 of up to 131072 (304 spans)
// 34.5 / 38.0, 24 of 40000 (101) 30.2 / 30.9, 32 of 32768 (76) 27.0 / 27.2, 64
// of 16384 (38) 30.0 / 29.5; 16 rows a unit, 8 of 65536 (228) 30.5 / 32.0, 64
// of 8192 (28) 34.1 / 31.3.
constexpr int kJoinSpans = 96;
template <int NT>
constexpr int kSpans = kCtas * kWarps<NT>;
constexpr int kFew = 4;  // warps of a CTA that takes one of many short units
constexpr float kNoMax = -1.7e38f;  // running maximum of a row that has seen no key (finite: no inf - inf)
constexpr float kLift = 11.f;   // weights are held 2^11 up
constexpr float kLag = 4.f;     // a score may pass the running maximum by 2^4
constexpr int kMinPairs = 2;    // shortest span: below, a partial result costs more than its keys
constexpr int kPair = 2, kPairKeys = kPair * kCacheTile;  // tiles and keys of a step

struct Attn4Problem {
  const __nv_bfloat16* q;
  __nv_bfloat16* o;
  float* lse;
  PagedCache cache;
  const int* table;
  long long table_stride;
  size_t table_bytes, q_bytes;
  const int* lens;
  const int* cu_q;    // or NULL: every request has uniform_q queries
  float* part;        // [2 * spans][rows][d] unnormalised O
  float2* part_ml;    // [2 * spans][rows] maximum (log2), sum
  long long* start;   // [B + 1] first tile pair of each request on the line; then, for the search, whether offsets are out of order
  int B, H, G, total_q, uniform_q, max_q, max_k;
  float scale_log2, v_scale;
  int causal;
  int ragged;         // the grids count row tiles (below) instead of requests times the most of one
};

struct Request {
  int q0, Lq, Lk;
  bool ok;
};

// The query rows of request b; false where they are out of range.
__device__ __forceinline__ bool queries(const Attn4Problem& p, int b, int& q0, int& Lq) {
  if (p.cu_q) {
    q0 = __ldg(p.cu_q + b);
    Lq = __ldg(p.cu_q + b + 1) - q0;
  } else {
    q0 = b * p.uniform_q;
    Lq = p.uniform_q;
  }
  return q0 >= 0 && Lq >= 0 && Lq <= p.max_q && q0 <= p.total_q - Lq;
}

// Whether the offsets go down at request b or begin below 0; if they do at
// none, all are in order.
__device__ __forceinline__ bool out_of_order(const Attn4Problem& p, int b) {
  const int q0 = __ldg(p.cu_q + b);
  return q0 < 0 || __ldg(p.cu_q + b + 1) < q0;
}

// A request with impossible lengths is left out (its rows are not written).
__device__ __forceinline__ Request request(const Attn4Problem& p, int b) {
  Request r;
  r.Lk = __ldg(p.lens + b);
  r.ok = queries(p, b, r.q0, r.Lq) && r.Lk >= 0 && r.Lk <= p.max_k;
  return r;
}

template <int ROWS>
__device__ __forceinline__ int row_tiles(const Attn4Problem& p, const Request& r) {
  return static_cast<int>((static_cast<long long>(p.G) * r.Lq + ROWS - 1) / ROWS);
}
__device__ __forceinline__ int key_pairs(const Request& r) { return (r.Lk + kPairKeys - 1) / kPairKeys; }

// Row tiles of a K/V head's grid are numbered.  Where the grid has
// `max_row_tiles` for every request, t is tile t mod max_row_tiles of request
// t / max_row_tiles.  Where a few requests have most of the queries it has as
// many as total_q and B allow, and request b's are numbers G cu_q[b] / ROWS + b
// on: past those of the one before if the offsets are in order, since its
// G Lq rows touch at most that many tiles.
template <int ROWS>
__device__ __forceinline__ long long first_tile(const Attn4Problem& p, int q0, int b) {
  return static_cast<long long>(p.G) * q0 / ROWS + b;
}

// The request and the tile of it that number t stands for, found by a search
// 32 wide; right where the offsets are in order.  False where no request has
// it.
template <int ROWS>
__device__ __forceinline__ bool search_tile(const Attn4Problem& p, int t, int lane, int& b, int& rt) {
  auto number = [&](int i) { return first_tile<ROWS>(p, __ldg(p.cu_q + i), i); };
  b = 0;
  for (int n = p.B; n > 0;) {
    const int step = (n + 31) / 32, i = lane * step;
    const uint32_t below = __ballot_sync(0xffffffffu, i < n && number(b + i) <= t);
    if (below == 0) return false;  // (only in the first round)
    const int at = (31 - __clz(below)) * step;
    b += at;
    n = step > 1 ? min(step, n - at) : 0;
  }
  const long long rel = t - number(b);
  rt = static_cast<int>(min(max(rel, 0LL), 0x7fffffffLL / ROWS));
  return true;
}

// The same by asking every request from `from` on, a lane each, whether the
// number is one of its own: right whatever the offsets are, so that a wrong one
// costs no request but those it belongs to.  (Offsets out of order can give a
// number to several requests: `more`.)
template <int ROWS>
__device__ __forceinline__ bool scan_tile(const Attn4Problem& p, int t, int from, int lane, int& b, int& rt, bool& more) {
  int mine = INT_MAX, tile = 0, count = 0;
#pragma unroll 4
  for (int i = from + lane; i < p.B; i += 32) {  // (unrolled: the loads of four requests at once)
    int q0, Lq;
    const bool there = queries(p, i, q0, Lq);
    const long long rel = t - first_tile<ROWS>(p, q0, i);
    if (there && rel >= 0 && rel * ROWS < static_cast<long long>(p.G) * Lq && count++ == 0)
      mine = i, tile = static_cast<int>(rel);
  }
  b = __reduce_min_sync(0xffffffffu, mine);
  rt = __shfl_sync(0xffffffffu, tile, (b - from) & 31);
  more = __reduce_add_sync(0xffffffffu, count) > 1;
  return b < INT_MAX;
}

template <int ROWS>
__device__ __forceinline__ long long pairs_of(const Attn4Problem& p, const Request& r) {
  return r.ok ? static_cast<long long>(p.cache.heads) * row_tiles<ROWS>(p, r) * key_pairs(r) : 0;
}

// The next unit, from unit k of request b on (k: its row tile times H_kv plus
// its head), whose number the search takes for another's.
template <int ROWS>
__device__ __forceinline__ bool next_lost(const Attn4Problem& p, int& b, int& k, int lane) {
  for (; b < p.B; ++b, k = 0) {
    const Request r = request(p, b);
    for (const int units = r.ok ? row_tiles<ROWS>(p, r) * p.cache.heads : 0; k < units; ++k) {
      const int t = static_cast<int>(first_tile<ROWS>(p, r.q0, b)) + k / p.cache.heads;
      int found, rt;
      if (!search_tile<ROWS>(p, t, lane, found, rt) || found != b) return true;
    }
  }
  return false;
}

__device__ __forceinline__ long long quotient(long long a, long long b) {
  return (a | b) >> 32 ? a / b : static_cast<uint32_t>(a) / static_cast<uint32_t>(b);
}

// The line of all units' pairs cut into equal spans, of which a CTA's `warps`
// take consecutive ones: all of a CTA's on a long line, few on a short one, so
// that it spreads over the SMs.  With JOIN a CTA whose spans lie in one unit
// joins them to one partial result, in the place of its first span's.
template <int NT>
struct Line {
  int warps;
  long long len;
  __device__ __forceinline__ explicit Line(long long total)
      : warps(static_cast<int>(min(static_cast<long long>(kWarps<NT>), quotient(total + kCtas * kMinPairs - 1, kCtas * kMinPairs)))),
        len(max(quotient(total + kSpans<NT> - 1, kSpans<NT>), static_cast<long long>(kMinPairs))) {}
  __device__ __forceinline__ long long share() const { return len * warps; }  // of a CTA
  __device__ __forceinline__ int span_of(long long pair) const { return static_cast<int>(quotient(pair, len)); }
};

__device__ __forceinline__ void mma_f16(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}
__device__ __forceinline__ void mma_f16_first(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
  asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%10, %10, %10, %10};"
      : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1), "f"(0.f));
}
__device__ __forceinline__ uint32_t transpose8x8(uint32_t v) {
  uint32_t r;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}

template <int N>
__device__ __forceinline__ void load_words(uint32_t (&w)[N], uint32_t p) {
  if constexpr (N == 4) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(p));
  } else if constexpr (N == 2) {
    asm volatile("ld.shared.v2.b32 {%0, %1}, [%2];" : "=r"(w[0]), "=r"(w[1]) : "r"(p));
  } else {
    asm volatile("ld.shared.b32 %0, [%1];" : "=r"(w[0]) : "r"(p));
  }
}
__device__ __forceinline__ uint32_t load_half(uint32_t p) {
  uint16_t h;
  asm volatile("ld.shared.b16 %0, [%1];" : "=h"(h) : "r"(p));
  return h;
}

// A lane's codes (of K at 0, of V at kV) and scales of a tile in shared
// memory, as the tile lies in the cache: every load takes consecutive lanes'
// consecutive pieces, so none has a bank conflict.
template <int D>
constexpr int kWords = D >= 32 ? D / 32 : 1;  // of one load

template <int D>
__device__ __forceinline__ void load_codes(uint32_t (&w)[2][kWords<D>], uint32_t at, int lane) {
  constexpr int kB = D / 8;  // bytes of a lane's piece
#pragma unroll
  for (int i = 0; i < 2; ++i) {
    if constexpr (kB == 2)
      w[i][0] = load_half(at + i * 32 * kB + lane * kB);
    else
      load_words(w[i], at + i * 32 * kB + lane * kB);
  }
}
template <int D>
__device__ __forceinline__ uint32_t load_k_scales(uint32_t tile, int lane) {
  using L = Kv4<D>;
  const int g = lane >> 2, c = lane & 3;
  if constexpr (D == 128) {  // groups 2 c, 2 c + 1 of keys g, g + 8
    uint32_t w[1];
    load_words(w, tile + L::kKS + lane * 4);
    return w[0];
  } else {
    return load_half(tile + L::kKS + (g * L::kGroups + c * L::kGroups / 4) * 2);
  }
}
template <int D>
__device__ __forceinline__ uint32_t load_v_scales(uint32_t tile, int lane) {
  using L = Kv4<D>;
  uint32_t w[1];
  load_words(w, tile + L::kVS + (((lane >> 2) * L::kGroups / 8) * 4 + (lane & 3)) * 4);
  return w[0];
}

// One warp's running state of a unit.
template <int D, int NT>
struct Rows {
  uint32_t q;  // shared address of the lane's Q^T operand: 8 bytes at (row tile, step) x 256
  float o[NT][D / 16][4];
  float cs[NT][2], off[NT][2], l[NT][2];  // score factor, kLift - maximum, sum, of columns 2c, 2c + 1
  int vis[NT][2];                         // keys they see
  int min_vis;                            // least of all the unit's rows
};

template <int D, int NT>
__device__ __forceinline__ void start_unit(Rows<D, NT>& s, const Attn4Problem& p, const Request& rq, int h, int row0,
                                           int lane) {
  constexpr int kPer = D / 4;  // columns of a lane
  const int g = lane >> 2, c = lane & 3;
  const int rows = p.G * rq.Lq;
  s.min_vis = rq.Lk;
  uint32_t raw[NT][kPer / 2];
#pragma unroll
  for (int j = 0; j < NT; ++j) {  // (all rows' loads at once)
    const int r = row0 + 8 * j + g;
    uint32_t (&w)[kPer / 2] = raw[j];
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) w[i] = 0;
    if (r < rows) {
      const int i = r / p.G;
      const __nv_bfloat16* src =
          p.q + (static_cast<long long>(rq.q0 + i) * p.H + h * p.G + (r - i * p.G)) * D + c * kPer;
      if constexpr (kPer >= 8) {
#pragma unroll
        for (int v = 0; v < kPer / 8; ++v) {
          const uint4 u = __ldg(reinterpret_cast<const uint4*>(src) + v);
          w[4 * v] = u.x, w[4 * v + 1] = u.y, w[4 * v + 2] = u.z, w[4 * v + 3] = u.w;
        }
      } else {
        const uint2 u = __ldg(reinterpret_cast<const uint2*>(src));
        w[0] = u.x, w[1] = u.y;
      }
    }
  }
#pragma unroll
  for (int j = 0; j < NT; ++j) {
    uint32_t (&w)[kPer / 2] = raw[j];
    // the power of two at or below the row's largest magnitude (1 for a row
    // of zeros, infinities or NaN)
    float mx = 0.f;
#pragma unroll
    for (int i = 0; i < kPer / 2; ++i) {
      const float2 f = unpack_bf16x2(w[i]);
      mx = fmaxf(mx, fmaxf(fabsf(f.x), fabsf(f.y)));
    }
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 1));
    mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, 2));
    const bool plain = mx == 0.f || isinf(mx);
    const int e = plain ? 0 : min(max(static_cast<int>(__float_as_uint(mx) >> 23) - 127, -126), 126);
    const float down = __uint_as_float(static_cast<uint32_t>(127 - e) << 23);
    // (kept off zero and infinity: the score of a masked key is -inf times it)
    const float up = fminf(fmaxf(__uint_as_float(static_cast<uint32_t>(127 + e) << 23) * p.scale_log2, 1e-37f), 3e38f);
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        const float2 f = unpack_bf16x2(w[2 * t + u]);
        w[2 * t + u] = pack_f16x2(f.x * down, f.y * down);
      }
#pragma unroll
    for (int t = 0; t < D / 16; ++t)
      asm volatile("st.shared.v2.b32 [%0], {%1, %2};" ::"r"(s.q + (j * (D / 16) + t) * 256), "r"(w[2 * t]), "r"(w[2 * t + 1])
                   : "memory");
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      s.cs[j][u] = __shfl_sync(0xffffffffu, up, (2 * c + u) * 4);
      s.off[j][u] = kLift - kNoMax;
      s.l[j][u] = 0.f;
      const int col = row0 + 8 * j + 2 * c + u;
      int vis = rq.Lk;
      if (p.causal && col < rows) vis = min(max(rq.Lk - rq.Lq + col / p.G + 1, 0), rq.Lk);
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

// e4m3 NaN bytes of a word, one bit per byte.
__device__ __forceinline__ uint32_t nan_bytes(uint32_t w) {
  uint32_t m = 0;
#pragma unroll
  for (int i = 0; i < 4; ++i) m |= static_cast<uint32_t>(((w >> (8 * i)) & 0x7fu) == 0x7fu) << i;
  return m;
}

// Two 16-key tiles, keys key0 .., at `tiles` in shared memory, into the
// unit's state: two, because their products are independent chains and the
// step's fixed costs (wait, vote, branches) are shared.  Where some row does
// not see all 32 keys (MASKED), a tile's keys are those below `end`, and none
// where its bit of `bad` is set (a page id out of range); what shared memory
// holds past them has no influence.
template <int D, int NT, bool MASKED>
__device__ __forceinline__ void step(Rows<D, NT>& s, uint32_t tiles, int key0, int end, uint32_t bad, int lane) {
  using L = Kv4<D>;
  constexpr int kSteps = D / 16;
  const int g = lane >> 2, c = lane & 3;
  auto keys = [&](int i) { return bad >> i & 1 ? 0 : min(max(end - key0 - i * kCacheTile, 0), kCacheTile); };

  float x[kPair][NT][4];
  {
    uint32_t k[kPair][2][kWords<D>], sa[kPair][2], sb[kPair][2];  // codes; scales of keys g and g + 8 for the lane's columns
#pragma unroll
    for (int i = 0; i < kPair; ++i) {
      load_codes<D>(k[i], tiles + i * L::kTileBytes, lane);
      const uint32_t ks = load_k_scales<D>(tiles + i * L::kTileBytes, lane);
      const uint32_t s0 = e4m3x2_to_f16(ks), s1 = D == 128 ? e4m3x2_to_f16(ks >> 16) : s0;
      sa[i][0] = __byte_perm(s0, 0, 0x1010), sb[i][0] = __byte_perm(s0, 0, 0x3232);
      sa[i][1] = __byte_perm(s1, 0, 0x1010), sb[i][1] = __byte_perm(s1, 0, 0x3232);
    }
#pragma unroll
    for (int w = 0; w < (kSteps + 1) / 2; ++w) {
      uint32_t q[NT][2][2];
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 2 && 2 * w + u < kSteps; ++u) load_words(q[j][u], s.q + (j * kSteps + 2 * w + u) * 256);
#pragma unroll
      for (int i = 0; i < kPair; ++i) {
        uint32_t lo[4], hi[4];
        e2m1x8_to_f16(k[i][0][w], lo);
        e2m1x8_to_f16(k[i][1][w], hi);
        const uint32_t a_s = sa[i][w >= 2], b_s = sb[i][w >= 2];
#pragma unroll
        for (int u = 0; u < 2 && 2 * w + u < kSteps; ++u) {
          const uint32_t a[4] = {hmul2(lo[2 * u], a_s), hmul2(hi[2 * u], b_s), hmul2(lo[2 * u + 1], a_s),
                                 hmul2(hi[2 * u + 1], b_s)};
#pragma unroll
          for (int j = 0; j < NT; ++j) {
            if (w == 0 && u == 0)
              mma_f16_first(x[i][j], a, q[j][u][0], q[j][u][1]);
            else
              mma_f16(x[i][j], a, q[j][u][0], q[j][u][1]);
          }
        }
      }
    }
  }
  // x[i][j][0], [1]: key g, columns 2c, 2c + 1; [2], [3]: key g + 8.
  if constexpr (MASKED) {
#pragma unroll
    for (int i = 0; i < kPair; ++i)
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 4; ++u) {
          const int key = g + (u >> 1) * 8;
          if (key >= keys(i) || key0 + i * kCacheTile + key >= s.vis[j][u & 1]) x[i][j][u] = -INFINITY;
        }
  }
  float y[kPair][NT][4], top = -INFINITY;
#pragma unroll
  for (int i = 0; i < kPair; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
#pragma unroll
      for (int u = 0; u < 4; ++u) y[i][j][u] = fmaf(x[i][j][u], s.cs[j][u & 1], s.off[j][u & 1]);
      top = fmax3(fmax3(top, y[i][j][0], y[i][j][1]), y[i][j][2], y[i][j][3]);
    }
  if (__builtin_expect(__any_sync(0xffffffffu, top > kLift + kLag), 0)) {
#pragma unroll
    for (int j = 0; j < NT; ++j)
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        float mx = fmaxf(x[0][j][u], x[0][j][u + 2]);
        mx = fmaxf(mx, fmaxf(x[1][j][u], x[1][j][u + 2])) * s.cs[j][u];
#pragma unroll
        for (int sh = 4; sh < 32; sh <<= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, sh));
        const float old = kLift - s.off[j][u], m = fmaxf(old, mx);
        const float down = ex2_approx(old - m);
        s.off[j][u] = kLift - m;
        s.l[j][u] *= down;
#pragma unroll
        for (int i = 0; i < kSteps; ++i) {
          s.o[j][i][u] *= down;
          s.o[j][i][u + 2] *= down;
        }
#pragma unroll
        for (int i = 0; i < kPair; ++i) {
          y[i][j][u] = fmaf(x[i][j][u], s.cs[j][u], s.off[j][u]);
          y[i][j][u + 2] = fmaf(x[i][j][u + 2], s.cs[j][u], s.off[j][u]);
        }
      }
  }
  uint32_t pb[kPair][NT][2];
#pragma unroll
  for (int i = 0; i < kPair; ++i)
#pragma unroll
    for (int j = 0; j < NT; ++j) {
      float e[4];
#pragma unroll
      for (int u = 0; u < 4; ++u) e[u] = ex2_approx(y[i][j][u]);
      s.l[j][0] += e[0] + e[2];
      s.l[j][1] += e[1] + e[3];
      pb[i][j][0] = transpose8x8(pack_f16x2(e[0], e[1]));
      pb[i][j][1] = transpose8x8(pack_f16x2(e[2], e[3]));
    }
#pragma unroll
  for (int i = 0; i < kPair; ++i) {
    uint32_t v[2][kWords<D>];
    load_codes<D>(v, tiles + i * L::kTileBytes + L::kV, lane);
    uint32_t vs = load_v_scales<D>(tiles + i * L::kTileBytes, lane);
    uint32_t nan_keys = 0;  // keys of the tile with a NaN in this lane's columns of V
    if constexpr (MASKED) {
      // V of keys past the end counts as zeros, whatever the page holds; a NaN
      // that some rows see is taken out of the product (0 x NaN would reach the
      // rows that do not) and put into those rows afterwards.
      uint32_t drop = 0, nan = nan_bytes(vs);
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        const int key = (u >> 1) * 8 + 2 * c + (u & 1);
        if (key >= keys(i)) drop |= 1u << u;
        else if (nan >> u & 1) nan_keys |= 1u << key, drop |= 1u << u;
      }
#pragma unroll
      for (int u = 0; u < 4; ++u)
        if (drop >> u & 1) vs &= ~(0xffu << (8 * u));
      nan_keys |= __shfl_xor_sync(0xffffffffu, nan_keys, 1);
      nan_keys |= __shfl_xor_sync(0xffffffffu, nan_keys, 2);
    }
    const uint32_t s0 = e4m3x2_to_f16(vs), s1 = e4m3x2_to_f16(vs >> 16);  // keys 2c, 2c + 1; 2c + 8, 2c + 9
    constexpr int kPiece = D >= 64 ? D / 64 : 1;  // words of one key's piece
#pragma unroll
    for (int w = 0; w < kPiece; ++w) {
      // low / high codes of the two keys' bytes side by side
      uint32_t even[2][4], odd[2][4];
#pragma unroll
      for (int u = 0; u < 2; ++u) {
        uint32_t a, b;
        if constexpr (D >= 64) {
          a = v[u][w], b = v[u][kPiece + w];
        } else {
          a = v[u][0], b = v[u][0] >> (D / 2);
        }
        e2m1x8_to_f16((a & 0x0f0f0f0fu) | ((b << 4) & 0xf0f0f0f0u), even[u]);
        e2m1x8_to_f16(((a >> 4) & 0x0f0f0f0fu) | (b & 0xf0f0f0f0u), odd[u]);
      }
#pragma unroll
      for (int u = 0; u < 4; ++u) {
        if (4 * w + u < kSteps) {
          const uint32_t a[4] = {hmul2(even[0][u], s0), hmul2(odd[0][u], s0), hmul2(even[1][u], s1),
                                 hmul2(odd[1][u], s1)};
#pragma unroll
          for (int j = 0; j < NT; ++j) mma_f16(s.o[j][4 * w + u], a, pb[i][j][0], pb[i][j][1]);
        }
      }
    }
    if (MASKED && __any_sync(0xffffffffu, nan_keys != 0)) {
#pragma unroll
      for (int j = 0; j < NT; ++j)
#pragma unroll
        for (int u = 0; u < 2; ++u) {
          const int n = min(max(s.vis[j][u] - key0 - i * kCacheTile, 0), kCacheTile);
          if (nan_keys & ((1u << n) - 1u)) {
#pragma unroll
            for (int t = 0; t < kSteps; ++t) s.o[j][t][u] = s.o[j][t][u + 2] = __uint_as_float(0x7fffffffu);
          }
        }
    }
  }
}

// o and lse of a row from its sums (a row that saw no key: zeros, -inf).
__device__ __forceinline__ float row_lse(float m, float l) { return (m - kLift + log2f(l)) * 0.69314718055994531f; }

// The end of a unit's keys: its rows go out, or, where `part` is given, leave
// a partial result there ([rows][D]) and in `ml`.
template <int D, int NT>
__device__ __forceinline__ void end_unit(Rows<D, NT>& s, const Attn4Problem& p, const Request& rq, int h, int row0,
                                         float* part, float2* ml, int lane) {
  constexpr int kPer = D / 8;
  const int g = lane >> 2, c = lane & 3;
  const int rows = p.G * rq.Lq;
#pragma unroll
  for (int j = 0; j < NT; ++j)
#pragma unroll
    for (int u = 0; u < 2; ++u) {
      float l = s.l[j][u];
#pragma unroll
      for (int sh = 4; sh < 32; sh <<= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
      const int local = 8 * j + 2 * c + u, r = row0 + local;
      if (r >= rows) continue;
      const float m = kLift - s.off[j][u];
      float v[kPer];
#pragma unroll
      for (int i = 0; i < D / 16; ++i) {
        v[2 * i] = s.o[j][i][u];
        v[2 * i + 1] = s.o[j][i][u + 2];
      }
      if (part) {
        float* dst = part + local * D + g * kPer;
#pragma unroll
        for (int i = 0; i < kPer; i += (kPer >= 4 ? 4 : 2)) {
          if constexpr (kPer >= 4)
            *reinterpret_cast<float4*>(dst + i) = make_float4(v[i], v[i + 1], v[i + 2], v[i + 3]);
          else
            *reinterpret_cast<float2*>(dst + i) = make_float2(v[i], v[i + 1]);
        }
        if (g == 0) ml[local] = make_float2(m, l);
        continue;
      }
      const float k = l == 0.f ? 0.f : p.v_scale / l;
      const int i0 = r / p.G;
      const long long tok = rq.q0 + i0;
      const int head = h * p.G + (r - i0 * p.G);
      uint32_t w[kPer / 2];
#pragma unroll
      for (int i = 0; i < kPer / 2; ++i) w[i] = pack_bf16x2(v[2 * i] * k, v[2 * i + 1] * k);
      char* dst = reinterpret_cast<char*>(p.o + (tok * p.H + head) * D + g * kPer);
      if constexpr (kPer == 16) {
        reinterpret_cast<uint4*>(dst)[0] = make_uint4(w[0], w[1], w[2], w[3]);
        reinterpret_cast<uint4*>(dst)[1] = make_uint4(w[4], w[5], w[6], w[7]);
      } else if constexpr (kPer == 8) {
        *reinterpret_cast<uint4*>(dst) = make_uint4(w[0], w[1], w[2], w[3]);
      } else if constexpr (kPer == 4) {
        *reinterpret_cast<uint2*>(dst) = make_uint2(w[0], w[1]);
      } else {
        *reinterpret_cast<uint32_t*>(dst) = w[0];
      }
      if (g == 0) p.lse[static_cast<long long>(head) * p.total_q + tok] = l == 0.f ? -INFINITY : row_lse(m, l);
    }
}

// A warp's ring of two tile pairs in shared memory, filled by bulk copies, a
// pair completing on its slot's mbarrier.  Every 32 pairs each lane looks one
// of the next 32 up in the block table and keeps where it lies, so that a
// pair's copy is one instruction of its lane (two where pages hold 16 tokens;
// a larger page holds whole pairs, the last of a request perhaps with a tile
// that has no key).
struct Ring {
  uint32_t tiles;        // shared address of slot 0
  uint64_t* full;        // the two mbarriers
  uint32_t slot, phase;  // next to be read, parity of its phase
  // the request's pages and the lanes' pairs
  const int* row;
  const char* head;      // this head's part of page 0
  int pages, first;      // first: the pair of lane 0
  const char *a, *b;     // the lane's pair: its first (or only) copy, its second or NULL
  uint32_t bytes;        // of both copies
  uint32_t bad_a, bad_b; // lanes whose first / second tile has a page id out of range (copied from page 0, its keys left out)
  uint32_t bad;          // the slots' bits: first and second tile of slot 0, of slot 1
};

template <int D>
__device__ __forceinline__ void look_up(Ring& r, const Attn4Problem& p, int pair, int lane) {
  constexpr int kBytes = Kv4<D>::kTileBytes;
  const int per = p.cache.shift - 4, tile = (pair + lane) * kPair, idx = tile >> per;
  const bool there = idx < r.pages, more = per == 0 && idx + 1 < r.pages;
  int id = there ? __ldg(r.row + idx) : 0, id2 = more ? __ldg(r.row + idx + 1) : 0;
  const bool bad = static_cast<uint32_t>(id) >= static_cast<uint32_t>(p.cache.num_pages);
  const bool bad2 = static_cast<uint32_t>(id2) >= static_cast<uint32_t>(p.cache.num_pages);
  if (bad) id = 0;
  if (bad2) id2 = 0;
  r.first = pair;
  r.a = r.head + id * p.cache.page_stride + (tile & ((1 << per) - 1)) * kBytes;
  r.b = more ? r.head + id2 * p.cache.page_stride : nullptr;
  r.bytes = per == 0 && !more ? kBytes : kPair * kBytes;
  r.bad_a = __ballot_sync(0xffffffffu, bad);
  r.bad_b = per == 0 ? __ballot_sync(0xffffffffu, bad2) : r.bad_a;
  if (lane == 0 && (r.bad_a | r.bad_b)) atomicCAS(&g_attn4_status, kDevOk, kDevBadIndex);
}

// Start the copy of a pair into a slot.
template <int D>
__device__ __forceinline__ void fetch(Ring& r, const Attn4Problem& p, int pair, uint32_t slot, int lane) {
  constexpr int kBytes = Kv4<D>::kTileBytes;
  int at = pair - r.first;
  if (at >= 32) {
    look_up<D>(r, p, pair, lane);
    at = 0;
  }
  if (r.bad | r.bad_a | r.bad_b)
    r.bad = (r.bad & ~(3u << 2 * slot)) | ((r.bad_a >> at & 1u) | (r.bad_b >> at & 1u) << 1) << 2 * slot;
  if (lane == at) {
    const uint32_t dst = r.tiles + slot * (kPair * kBytes);
    mbar_arrive_expect_tx(&r.full[slot], r.bytes);
    bulk_load(dst, r.a, r.b ? kBytes : r.bytes, &r.full[slot]);
    if (r.b) bulk_load(dst + kBytes, r.b, kBytes, &r.full[slot]);
  }
}

template <int D, int NT>
struct __align__(128) WarpSmem {
  char tiles[2 * kPair * Kv4<D>::kTileBytes];
  uint64_t q[NT * (D / 16) * 32];
  float2 ml[8 * NT];  // of a partial result (its rows are put into `tiles`)
  uint64_t full[2];
};
static_assert(sizeof(WarpSmem<16, 2>::tiles) >= 16 * 16 * 4 && sizeof(WarpSmem<128, 2>::tiles) >= 16 * 128 * 4, "rows fit");

template <int D, int NT>
__device__ __forceinline__ void start_warp(WarpSmem<D, NT>* ws, Rows<D, NT>& s, Ring& ring, int lane) {
  // (a warp's barriers are its own: no other warp waits for this)
  if (lane == 0) {
    for (int i = 0; i < 2; ++i) mbar_init(&ws->full[i], 1);
    fence_mbar_init();
  }
  __syncwarp();
  s.q = smem_u32(ws->q) + lane * 8;
  ring.tiles = smem_u32(ws->tiles);
  ring.full = ws->full;
  ring.slot = ring.phase = ring.bad = 0;
}

// Pairs first .. first + n - 1 (n > 0) of a unit's keys into fresh row states.
// False (and a status word) if a copy did not come in time.
template <int D, int NT>
__device__ __forceinline__ bool run_pairs(Rows<D, NT>& s, Ring& ring, const Attn4Problem& p, const Request& rq, int b, int h,
                                          int row0, int first, int n, int lane) {
  ring.row = p.table + b * p.table_stride;
  ring.pages = static_cast<int>((rq.Lk + ((1LL << p.cache.shift) - 1)) >> p.cache.shift);
  ring.head = p.cache.base + (static_cast<long long>(h) << (p.cache.shift - 4)) * Kv4<D>::kTileBytes;
  // (both slots are free here: the part before has been read to its end)
  look_up<D>(ring, p, first, lane);
  fetch<D>(ring, p, first, ring.slot, lane);
  if (n > 1) fetch<D>(ring, p, first + 1, ring.slot ^ 1, lane);
  start_unit<D, NT>(s, p, rq, h, row0, lane);
  const int whole = s.min_vis / kPairKeys;  // every row sees all keys of the pairs below
  for (int pair = first; pair < first + n; ++pair) {
    if (!mbar_wait_warp(&ring.full[ring.slot], ring.phase, &g_attn4_status)) {
      // a copy that never came: wait (as long again) for the other, then give up
      if (pair + 1 < first + n) mbar_wait_warp(&ring.full[ring.slot ^ 1], ring.phase ^ ring.slot, &g_attn4_status);
      return false;
    }
    const uint32_t tiles = ring.tiles + ring.slot * (kPair * Kv4<D>::kTileBytes);
    if (__builtin_expect(pair < whole && !ring.bad, 1))
      step<D, NT, false>(s, tiles, 0, 0, 0, lane);
    else
      step<D, NT, true>(s, tiles, pair * kPairKeys, rq.Lk, ring.bad >> 2 * ring.slot & 3u, lane);
    __syncwarp();  // every lane has read the slot
    if (pair + 2 < first + n) fetch<D>(ring, p, pair + 2, ring.slot, lane);
    ring.phase ^= ring.slot;  // (the parity changes when the ring has gone round)
    ring.slot ^= 1;
  }
  return true;
}

// A joined row: `o` the lane's columns of the sum of weighted partial rows, l
// and top of the same.
template <int D>
__device__ __forceinline__ void write_row(const Attn4Problem& p, const Request& rq, int h, int r, const float* o, float l,
                                          float top, int lane) {
  constexpr int kCols = D >= 32 ? D / 32 : 1;
  const int i = r / p.G;
  const long long tok = rq.q0 + i;
  const int head = h * p.G + (r - i * p.G);
  const float f = l == 0.f ? 0.f : p.v_scale / l;
  __nv_bfloat16* dst = p.o + (tok * p.H + head) * D + lane * kCols;
#pragma unroll
  for (int k = 0; k < kCols; ++k)
    if (lane * kCols < D) dst[k] = __float2bfloat16_rn(o[k] * f);
  if (lane == 0) p.lse[static_cast<long long>(head) * p.total_q + tok] = l == 0.f ? -INFINITY : row_lse(top, l);
}

// A row of the partial results that `parts` <= 32 warps of the CTA left in
// shared memory: the lane's columns, sum and maximum.
template <int D, int NT>
__device__ __forceinline__ void join_row(const WarpSmem<D, NT>* all, int parts, int local, float* o, float& l, float& top,
                                         int lane) {
  constexpr int kCols = D >= 32 ? D / 32 : 1;
  const float2 ml = lane < parts ? all[lane].ml[local] : make_float2(kNoMax, 0.f);
  top = ml.x;
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
  const float w = ex2_approx(ml.x - top);
  l = w * ml.y;
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
#pragma unroll
  for (int k = 0; k < kCols; ++k) o[k] = 0.f;
  for (int i = 0; i < parts; ++i) {
    const float wi = __shfl_sync(0xffffffffu, w, i);
    const float* row = reinterpret_cast<const float*>(all[i].tiles) + local * D + lane * kCols;
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      if (lane * kCols < D) o[k] = fmaf(wi, row[k], o[k]);
  }
}

template <int D, int NT, bool JOIN>
__global__ void __launch_bounds__(kWarps<NT> * 32, 1) fa2_kv4_attn_kernel(const Attn4Problem p) {
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) char smem[];
  WarpSmem<D, NT>* const ws = reinterpret_cast<WarpSmem<D, NT>*>(smem) + (threadIdx.x >> 5);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Rows<D, NT> s;
  Ring ring;
  start_warp(ws, s, ring, lane);
  griddep_wait();
  griddep_launch_dependents();
  // Every warp needs, one after the other, the lengths, its request's page
  // ids and its queries: the lines of the latter two start on their way to
  // L2 while the first is being read.
  {
    const size_t line = (static_cast<size_t>(blockIdx.x) * blockDim.x + threadIdx.x) * 128;
    if (line < p.table_bytes) prefetch_l2(reinterpret_cast<const char*>(p.table) + line);
    if (line < p.q_bytes) prefetch_l2(reinterpret_cast<const char*>(p.q) + line);
  }
  // Each lane adds up the pairs of its share of the requests.
  const int per = (p.B + 31) / 32;
  const int b_lo = min(lane * per, p.B), b_hi = min(b_lo + per, p.B);
  long long mine = 0;
  bool fine = true;
#pragma unroll 4
  for (int b = b_lo; b < b_hi; ++b) {  // (unrolled: the loads of four requests at once)
    const Request r = request(p, b);
    fine &= r.ok;
    mine += pairs_of<kRows>(p, r);
  }
  long long upto = mine;
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long v = __shfl_up_sync(0xffffffffu, upto, s);
    if (lane >= s) upto += v;
  }
  const long long total = __shfl_sync(0xffffffffu, upto, 31);
  if (blockIdx.x == 0 && warp == 0) {  // for the combine kernel
    long long at = upto - mine;
    for (int b = b_lo; b < b_hi; ++b) {
      p.start[b] = at;
      at += pairs_of<kRows>(p, request(p, b));
    }
    if (lane == 31) p.start[p.B] = total;
    if (!fine) atomicCAS(&g_attn4_status, kDevOk, kDevBadSeqlens);
  }
  if (!JOIN && p.ragged && blockIdx.x == kCtas - 1 && warp == kWarps<NT> - 1) {  // (the warp with the least to do)
    bool mixed = false;
#pragma unroll 4
    for (int b = lane; b < p.B; b += 32) mixed |= out_of_order(p, b);
    mixed = __any_sync(0xffffffffu, mixed);
    if (lane == 0) p.start[p.B + 1] = mixed;
  }
  const Line<NT> line(total);
  if (warp >= line.warps) return;
  const int span = blockIdx.x * line.warps + warp;
  const long long begin = span * line.len, end = min(begin + line.len, total);
  long long at = begin;
  if (at >= end) return;
  // the request that holds pair `at`
  const uint32_t holds = __ballot_sync(0xffffffffu, upto > at);
  const int owner = __ffs(holds) - 1;
  int b = __shfl_sync(0xffffffffu, b_lo, owner);
  long long base = __shfl_sync(0xffffffffu, upto - mine, owner);
  Request rq = request(p, b);
  long long size = pairs_of<kRows>(p, rq);

  while (at < end) {
    while (at >= base + size) {
      base += size;
      rq = request(p, ++b);
      size = pairs_of<kRows>(p, rq);
    }
    const int np = key_pairs(rq), rt = row_tiles<kRows>(p, rq);
    // (a request's units are at most H_kv times its row tiles: 32 bits, as its
    // pairs are; their product may not be)
    const long long rel = at - base;
    const int unit = static_cast<int>(quotient(rel, np));
    const int first = static_cast<int>(rel - static_cast<long long>(unit) * np);
    const int h = unit / rt, row0 = (unit - h * rt) * kRows;
    const int n = static_cast<int>(min(static_cast<long long>(np - first), end - at));
    // (the same for all warps of the CTA: it is about all their spans)
    const long long cta = blockIdx.x * line.share(), start = at - first;
    const bool whole = JOIN && start <= cta && cta + line.share() <= start + np;
    if (run_pairs<D, NT>(s, ring, p, rq, b, h, row0, first, n, lane)) {
      // A unit that is whole goes out; else slot 0 of the span if the part
      // began at the span's start, slot 1 if within it.
      const long long slot = (2LL * span + (at == begin ? 0 : 1)) * kRows;
      float* const part = whole ? reinterpret_cast<float*>(ws->tiles) : n == np ? nullptr : p.part + slot * D;
      end_unit<D, NT>(s, p, rq, h, row0, part, whole ? ws->ml : p.part_ml + slot, lane);
    } else if (!whole) {
      return;
    }
    if (whole) {
      // (a warp whose copy did not come leaves the rows wrong, with the status
      // word set: the others must not wait for it)
      asm volatile("bar.sync 1, %0;" ::"r"(line.warps * 32) : "memory");
      constexpr int kCols = D >= 32 ? D / 32 : 1;
      const long long to = 2LL * blockIdx.x * line.warps * kRows;
      for (int local = warp; local < kRows && row0 + local < p.G * rq.Lq; local += line.warps) {
        float o[kCols], l, top;
        join_row<D, NT>(reinterpret_cast<const WarpSmem<D, NT>*>(smem), line.warps, local, o, l, top, lane);
        if (np == line.share()) {
          write_row<D>(p, rq, h, row0 + local, o, l, top, lane);
          continue;
        }
#pragma unroll
        for (int k = 0; k < kCols; ++k)
          if (lane * kCols < D) p.part[(to + local) * D + lane * kCols + k] = o[k];
        if (lane == 0) p.part_ml[to + local] = make_float2(top, l);
      }
      return;
    }
    at += n;
  }
}

// One row of a unit in the combine kernel below, for warp `part` of its WPR.
template <int D, int ROWS, int WPR, bool JOIN>
__device__ __forceinline__ void combine_row(const Attn4Problem& p, int b, int h, int rt, int local, int part,
                                            float (*s_o)[D], float* s_m, float* s_l, int lane, int warp) {
  constexpr int kCols = D >= 32 ? D / 32 : 1, kBatch = 8;
  const long long start = p.start[b], total = p.start[p.B];
  const Request rq = request(p, b);
  const long long row = static_cast<long long>(rt) * ROWS + local;
  const bool live = rq.ok && row < p.G * rq.Lq;
  const int r = static_cast<int>(row);
  const int np = key_pairs(rq);
  // The unit's partial results: `head` spans from s0 on, `mid` CTAs from span
  // s1 on that joined theirs, spans from s2 on.
  int count = 0, s0 = 0, head = 0, mid = 0, s1 = 0, s2 = 0, warps = 0;
  long long slot0 = 0;
  if (live && np > 0) {
    const Line<ROWS / 8> line(total);
    const long long first = start + (static_cast<long long>(h) * row_tiles<ROWS>(p, rq) + rt) * np;
    warps = line.warps;
    s0 = line.span_of(first);
    const int last = line.span_of(first + np - 1);
    // the CTAs of the whole spans: from, to
    const int lo = (s0 + (first != s0 * line.len ? 1 : 0) + warps - 1) / warps;
    const int hi = (last + (first + np == (last + 1) * line.len ? 1 : 0)) / warps;
    count = head = last - s0 + 1;
    if (JOIN && hi > lo) {
      s1 = lo * warps, s2 = hi * warps;
      head = s1 - s0, mid = hi - lo;
      count = head + mid + last - s2 + 1;
    }
    // slot 0 of a span, but slot 1 where the unit begins within it
    slot0 = (2LL * s0 + (first != s0 * line.len ? 1 : 0)) * ROWS + local;
  }
  // (the same for all warps of a row; rows of one warp need no barrier)
  if (WPR == 1 && (!live || count == 1)) return;
  auto at = [&](int i) {
    const int span = i < head ? s0 + i : i < head + mid ? s1 + (i - head) * warps : s2 + i - head - mid;
    return i == 0 ? slot0 : 2LL * span * ROWS + local;
  };
  float l = 0.f, top = kNoMax, o[kCols];
#pragma unroll
  for (int k = 0; k < kCols; ++k) o[k] = 0.f;
  const bool active = lane * kCols < D;
  // warp `part` takes results part, part + WPR, ..., 32 at a time
  for (int i0 = part; count > 1 && i0 < count; i0 += WPR * 32) {
    float2 ml = make_float2(kNoMax, 0.f);
    if (i0 + lane * WPR < count) ml = p.part_ml[at(i0 + lane * WPR)];
    float m = fmaxf(top, ml.x);
#pragma unroll
    for (int sh = 16; sh > 0; sh >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, sh));
    const float down = ex2_approx(top - m), w = ex2_approx(ml.x - m);
    top = m;
    l = l * down + w * ml.y;
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[k] *= down;
    const int n = min((count - i0 + WPR - 1) / WPR, 32);
    const float* src = p.part + lane * kCols;
    for (int c = 0; c < n; c += kBatch) {
      float v[kBatch][kCols];
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        const float* row = src + at(i0 + (c + i) * WPR) * D;
        if constexpr (kCols == 4) {
          const float4 t = c + i < n ? *reinterpret_cast<const float4*>(row) : make_float4(0.f, 0.f, 0.f, 0.f);
          v[i][0] = t.x, v[i][1] = t.y, v[i][2] = t.z, v[i][3] = t.w;
        } else {
#pragma unroll
          for (int k = 0; k < kCols; ++k) v[i][k] = c + i < n && active ? row[k] : 0.f;
        }
      }
#pragma unroll
      for (int i = 0; i < kBatch; ++i) {
        // (lanes past the last span have weight 0)
        const float wi = __shfl_sync(0xffffffffu, w, (c + i) & 31);
#pragma unroll
        for (int k = 0; k < kCols; ++k) o[k] = fmaf(wi, v[i][k], o[k]);
      }
    }
  }
#pragma unroll
  for (int sh = 16; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
  if (WPR > 1) {
#pragma unroll
    for (int k = 0; k < kCols; ++k)
      if (active) s_o[warp][lane * kCols + k] = o[k];
    if (lane == 0) s_m[warp] = top, s_l[warp] = l;
    __syncthreads();
    if (part != 0 || !live || count == 1) return;
    for (int w = 1; w < WPR; ++w) top = fmaxf(top, s_m[warp + w]);
    float down = ex2_approx(s_m[warp] - top);
    l *= down;
#pragma unroll
    for (int k = 0; k < kCols; ++k) o[k] *= down;
#pragma unroll
    for (int w = 1; w < WPR; ++w) {
      down = ex2_approx(s_m[warp + w] - top);
      l += s_l[warp + w] * down;
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (active) o[k] = fmaf(s_o[warp + w][lane * kCols + k], down, o[k]);
    }
  }
  write_row<D>(p, rq, h, r, o, l, top, lane);
}

// Join the partial results of the units that several spans share, in span
// order, and write the rows that see no key.  A CTA of 8 warps takes 8 / WPR
// rows of a unit, WPR warps each.  Bound by the latency of what it reads one
// after the other (where the unit's spans are, their maxima and sums, their
// rows), so each of the three is one round of loads: a lane per span for the
// maxima, then the rows of kBatch spans at once.
template <int D, int ROWS, int WPR, bool JOIN>
__global__ void __launch_bounds__(256) fa2_kv4_combine_kernel(const Attn4Problem p, int max_row_tiles) {
  constexpr int kRowsCta = 8 / WPR;
  __shared__ float s_o[WPR > 1 ? 8 : 1][D];
  __shared__ float s_m[8], s_l[8];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  int id = blockIdx.x;
  const int local = (id % (ROWS / kRowsCta)) * kRowsCta + warp / WPR, part = warp % WPR;
  id /= ROWS / kRowsCta;
  const int h = id % p.cache.heads;
  griddep_wait();
  griddep_launch_dependents();
  const int t = id / p.cache.heads;
  int b = t, rt = 0;
  bool there = true, more = false;
  if (max_row_tiles > 0) {
    b = t / max_row_tiles;
    rt = t - b * max_row_tiles;
  } else if (WPR == 1) {  // (many units)
    const long long mixed = p.start[p.B + 1];
    there = search_tile<ROWS>(p, t, lane, b, rt);
    if (mixed) there = scan_tile<ROWS>(p, t, 0, lane, b, rt, more);
  } else {
    there = scan_tile<ROWS>(p, t, 0, lane, b, rt, more);
  }
  while (there) {  // (of a call as it should be: once)
    combine_row<D, ROWS, WPR, JOIN>(p, b, h, rt, local, part, s_o, s_m, s_l, lane, warp);
    if (!more) return;
    if (WPR > 1) __syncthreads();  // (what the row's warps left has been read)
    there = scan_tile<ROWS>(p, t, b + 1, lane, b, rt, more);
  }
}

// A unit in the kernel below.  `fine`: the warp's copies have all come.
template <int D, int NT, int W, bool CLUSTER>
__device__ __forceinline__ void run_unit(Rows<D, NT>& s, Ring& ring, bool& fine, WarpSmem<D, NT>* all, const Attn4Problem& p,
                                         const Request& rq, int b, int h, int rt, int rank, int ctas, int lane, int warp) {
  constexpr int kRows = 8 * NT, kCols = D >= 32 ? D / 32 : 1;
  WarpSmem<D, NT>* const ws = all + warp;
  const int row0 = rt * kRows, rows = p.G * rq.Lq;
  const int np = key_pairs(rq);
  // the CTA's pairs, and each warp's
  const int from = CLUSTER ? static_cast<int>(static_cast<long long>(np) * rank / ctas) : 0;
  const int size = CLUSTER ? static_cast<int>(static_cast<long long>(np) * (rank + 1) / ctas) - from : np;
  const int each = (size + W - 1) / W, n = min(each, size - warp * each);
  // (a warp whose copy did not come leaves the unit's rows wrong, with the
  // status word set: the others must not wait for it)
  if (n > 0 && fine) {
    fine = run_pairs<D, NT>(s, ring, p, rq, b, h, row0, from + warp * each, n, lane);
    if (fine) end_unit<D, NT>(s, p, rq, h, row0, reinterpret_cast<float*>(ws->tiles), ws->ml, lane);
  }
  __syncthreads();
  const int parts = each > 0 ? (size + each - 1) / each : 0;
  // (a row joined in the CTA goes where the queries were, its maximum and sum behind it)
  auto joined = [&](int local) { return reinterpret_cast<float*>(all[local % W].q) + local / W * (D + 2); };
  static_assert((kRows + W - 1) / W * (D + 2) * sizeof(float) <= sizeof(ws->q), "rows fit");
  for (int local = warp; local < kRows && row0 + local < rows; local += W) {
    float o[kCols], l, top;
    join_row<D, NT>(all, parts, local, o, l, top, lane);
    if constexpr (!CLUSTER) {
      write_row<D>(p, rq, h, row0 + local, o, l, top, lane);
    } else {
      float* const row = joined(local);
#pragma unroll
      for (int k = 0; k < kCols; ++k)
        if (lane * kCols < D) row[lane * kCols + k] = o[k];
      if (lane == 0) row[D] = top, row[D + 1] = l;
    }
  }
  if constexpr (CLUSTER) {
    cluster_sync();
    for (int local = rank + ctas * warp; local < kRows && row0 + local < rows; local += ctas * W) {
      const uint32_t row = smem_u32(joined(local));
      const float m = lane < ctas ? load_cluster_f32(row + D * 4, lane) : kNoMax;
      float l = lane < ctas ? load_cluster_f32(row + D * 4 + 4, lane) : 0.f, top = m, o[kCols];
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, sh));
      const float w = ex2_approx(m - top);
      l *= w;
#pragma unroll
      for (int sh = 16; sh > 0; sh >>= 1) l += __shfl_xor_sync(0xffffffffu, l, sh);
#pragma unroll
      for (int k = 0; k < kCols; ++k) o[k] = 0.f;
      for (int i = 0; i < ctas; ++i) {
        const float wi = __shfl_sync(0xffffffffu, w, i);
#pragma unroll
        for (int k = 0; k < kCols; ++k)
          if (lane * kCols < D) o[k] = fmaf(wi, load_cluster_f32(row + (lane * kCols + k) * 4, i), o[k]);
      }
      write_row<D>(p, rq, h, row0 + local, o, l, top, lane);
    }
    cluster_sync();  // (no CTA leaves while another reads its rows)
  }
}

// Short requests: one CTA of W warps per unit, which take equal parts of its
// keys and join their partial results in shared memory, in the order of the
// keys: one launch, no line to lay out first, no workspace.  CLUSTER: `ctas`
// CTAs per unit, which take equal parts of its keys and join what their warps
// joined through distributed shared memory.
template <int D, int NT, int W, bool CLUSTER>
__global__ void __launch_bounds__(W * 32, kWarps<NT> / W) fa2_kv4_attn_unit_kernel(const Attn4Problem p, int max_row_tiles,
                                                                                   int ctas) {
  constexpr int kRows = 8 * NT;
  extern __shared__ __align__(128) char smem[];
  WarpSmem<D, NT>* const all = reinterpret_cast<WarpSmem<D, NT>*>(smem);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  Rows<D, NT> s;
  Ring ring;
  start_warp(all + warp, s, ring, lane);
  griddep_wait();
  griddep_launch_dependents();
  const int unit = CLUSTER ? blockIdx.x / ctas : blockIdx.x, rank = CLUSTER ? static_cast<int>(cluster_rank()) : 0;
  // (a request that is left out may have no CTA: all are looked at)
  const long long first = static_cast<long long>(blockIdx.x) * (W * 32), mine = first + threadIdx.x;
  bool mixed = false;
  if (mine < p.B) {
    if (!request(p, static_cast<int>(mine)).ok) atomicCAS(&g_attn4_status, kDevOk, kDevBadSeqlens);
    mixed = max_row_tiles == 0 && out_of_order(p, static_cast<int>(mine));
  }
  // Which unit this is.  With a full CTA for each, requests are few (one an SM
  // at most) and all asked.  Else the number is searched for, and a CTA that
  // has found offsets out of order takes the units that no search finds too.
  constexpr bool kSearch = W == kFew;
  const int t = unit / p.cache.heads;
  int h = unit % p.cache.heads, b = t, rt = 0;
  bool there = true, more = false, fine = true;
  if (max_row_tiles > 0) {
    b = t / max_row_tiles;
    rt = t - b * max_row_tiles;
  } else {
    there = kSearch ? search_tile<kRows>(p, t, lane, b, rt) : scan_tile<kRows>(p, t, 0, lane, b, rt, more);
    if (kSearch && first < p.B) more = __syncthreads_or(mixed);
  }
  for (int lost = 0;;) {  // (of a call as it should be: once)
    if (there) {
      const Request rq = request(p, b);
      if (rq.ok && static_cast<long long>(rt) * kRows < p.G * rq.Lq)
        run_unit<D, NT, W, CLUSTER>(s, ring, fine, all, p, rq, b, h, rt, rank, ctas, lane, warp);
    }
    if (!more) return;
    __syncthreads();  // (what the unit's warps left has been read)
    if (kSearch) {
      if (lost == 0) b = 0;  // from the first request's first unit on
      more = there = next_lost<kRows>(p, b, lost, lane);
      rt = lost / p.cache.heads;
      h = lost % p.cache.heads;
      ++lost;
    } else {
      there = scan_tile<kRows>(p, t, b + 1, lane, b, rt, more);
    }
  }
}

// 16 rows a unit when 8 would read the cache twice.
inline bool wide_rows(long long rows) { return rows > 8; }

// Units of the largest size the call allows.
inline long long max_units(int B, int H_kv, long long max_rows) {
  const int rows = wide_rows(max_rows) ? 16 : 8;
  return static_cast<long long>(B) * H_kv * ((max_rows + rows - 1) / rows);
}

// Warps of a CTA where each unit takes a CTA, 0 where the line is cut instead.
// One unit a SM: a full CTA, where the longest request is short for the number
// of units.  More units than SMs: kFew warps, of which three or four CTAs share
// an SM, where the longest request is short.  Measured, lengths from a quarter
// of the longest to it, 128 columns, a full CTA / kFew warps / the line in us:
//   8 rows a unit:
//   8 units     1024 keys   7.8 / 9.4 / 8.6     2048  11.0 / 15.3 / 8.9   4096  17.1 / 26.8 / 9.3
//   64 units    1024 keys   8.1 / 9.8 / 11.7    2048  11.3 / 15.7 / 12.3  4096  17.5 / 27.4 / 15.4
//   152 units   1024 keys   8.4 / 10.1 / 15.3   4096  19.7 / 28.3 / 24.0  8192  32.6 / 52.0 / 32.0
//   304 units    128 keys   9.5 / 5.6 / 11.3    2048  23.4 / 20.2 / 21.9  4096  35.7 / 34.8 / 30.3
//   2432 units   128 keys  66.5 / 22.1 / 28.0   2048 147.1 / 91.4 / 93.2  4096 213.7 / 158.9 / 153.4
//   16 rows a unit:
//   304 units    128 keys  14.8 / 10.2 / 16.4   1024  23.5 / 21.2 / 24.4  2048  35.5 / 35.3 / 32.1
//   760 units    128 keys  34.7 / 18.5 / 22.6   1024  53.5 / 37.7 / 40.6  2048  71.6 / 55.1 / 53.1
//   3040 units    32 keys 116.5 / 50.0 / 31.7    128 126.3 / 59.8 / 59.8  1024 212.9 / 118.2 / 123.6
// (the line spreads the bytes over all SMs but has its layout, its partial
// results and a second launch to pay for: the few units' bound is set where
// that launch's host time is still saved.  Very many units of a few keys leave
// most of a CTA's warps without any.  Up to 64 units of more than 1024 keys no
// longer take one CTA each, as in the first two lines, but a cluster: below.)
// The rule goes by the bound on the lengths, so one long request among short
// ones keeps it to few SMs where the line would spread it.  8 rows a unit, 8
// K/V heads, one request of the longest length and the others of 100 keys, this
// rule's form / the line in us (even lengths in brackets):
//   24 units    1024 keys   8.2 / 11.0 (8.2 / 10.3)     2048   8.5 / 10.9 (8.6 / 10.5)
//   152 units   1024 keys   8.1 / 12.3 (8.7 / 15.6)     2048  11.5 / 12.3 (11.8 / 18.6)   8192  30.1 / 13.5 (32.6 / 32.4)
//   304 units   1024 keys  10.5 / 10.3 (11.8 / 16.1)    2048  16.6 / 11.5 (19.9 / 20.8)
//   760 units   1024 keys  11.7 / 13.5 (24.8 / 26.4)    2048  17.6 / 13.8 (37.4 / 37.3)
// (a caller who knows of such a mix can give a longer bound, up to the table's
// room, which takes the line.)
inline int unit_warps(int B, int H_kv, long long max_rows, long long max_keys) {
  const long long units = max_units(B, H_kv, max_rows);
  const bool wide = wide_rows(max_rows);
  if (units <= 152) return max_keys <= (54 * units > 2048 ? 54 * units : 2048) ? (wide ? kWarps<2> : kWarps<1>) : 0;
  return max_keys <= (wide ? 1024 : 2048) && (units <= 152 * 8 || max_keys >= 128) ? kFew : 0;
}

// CTAs of a unit: a cluster of them where the keys are enough to make up for
// what the cluster costs (about 2 us) and its CTAs find SMs side by side
// (not 16 clusters of 8).  Measured as above, one CTA / two / four / eight:
//   8 units    512 keys   6.2 / 6.9 / 6.7 / 6.9   1000   8.1 / 8.3 / 7.4 / 7.1   2048  11.1 / 9.9 / 8.5 / 7.4
//   16 units  1000 keys   8.2 / 8.3 / 7.5 / 13.1  2048  11.4 / 9.8 / 8.5 / 13.4
//   32 units  1000 keys   8.3 / 8.3 / 7.5         2048  11.4 / 9.9 / 8.6
//   64 units  1000 keys   8.3 / 8.4               2048  11.4 / 10.1              4096  17.7 / 13.3
//   16 rows a unit, 4 units 512 keys 9.0 / 9.7 / 9.0 / 9.0, 1000 12.2 / 11.0 / 10.4 / 9.5, 2048 17.2 / 14.0 / 11.7 / 10.7
//   64 units   512 keys   9.6 / 10.3              1000  12.4 / 11.5              2048  17.5 / 14.4
// (max_keys is a bound: the thresholds leave room for shorter requests).
inline int unit_ctas(long long units, bool wide, int max_keys) {
  if (max_keys <= (wide ? 512 : 1024) || units > 64) return 1;
  if (units > 32) return max_keys > (wide ? 768 : 1536) ? 2 : 1;
  return units > 8 ? 4 : 8;
}

template <int D, int NT>
int launch_attn_d(Attn4Problem p, long long max_rows, cudaStream_t st) {
  constexpr int kRows = 8 * NT, kSmem = kWarps<NT> * sizeof(WarpSmem<D, NT>);
  int row_tiles = static_cast<int>((max_rows + kRows - 1) / kRows);
  long long units = max_units(p.B, p.cache.heads, max_rows);
  // Ragged queries: the grid counts tiles instead of requests times the most
  // of one (63 requests of one query and one of 256, 4 heads a group, 8 K/V
  // heads: 45.7 against 79 us with up to 1000 keys, 110 / 190 with 4000).
  const long long tiles = static_cast<long long>(p.total_q) * p.G / kRows + p.B;
  if (p.cu_q && tiles < static_cast<long long>(p.B) * row_tiles / 2) {
    row_tiles = 0;
    units = tiles * p.cache.heads;
    p.ragged = 1;
  }
  if (const int w = unit_warps(p.B, p.cache.heads, max_rows, p.max_k)) {
    const int smem = w * static_cast<int>(sizeof(WarpSmem<D, NT>));
    const int ctas = w == kFew ? 1 : unit_ctas(units, NT == 2, p.max_k);
    const auto kernel = w == kFew  ? fa2_kv4_attn_unit_kernel<D, NT, kFew, false>
                        : ctas > 1 ? fa2_kv4_attn_unit_kernel<D, NT, kWarps<NT>, true>
                                   : fa2_kv4_attn_unit_kernel<D, NT, kWarps<NT>, false>;
    if (int e = ensure_max_smem(reinterpret_cast<const void*>(kernel), smem)) return e;
    const dim3 grid(static_cast<unsigned>(units * ctas)), block(w * 32);
    return ctas > 1 ? launch_pdl_cluster(kernel, grid, block, smem, st, ctas, p, row_tiles, ctas)
                    : launch_pdl(kernel, grid, block, smem, st, p, row_tiles, ctas);
  }
  // Spans of a unit, were all requests of one length: with few, a warp of the
  // combine kernel joins a row alone; with more a CTA's eight do; with many the
  // CTAs of the first kernel join theirs before.
  const long long spans = kSpans<NT> / units;
  const bool join = spans >= kJoinSpans;
  const auto kernel = join ? fa2_kv4_attn_kernel<D, NT, true> : fa2_kv4_attn_kernel<D, NT, false>;
  if (int e = ensure_max_smem(reinterpret_cast<const void*>(kernel), kSmem)) return e;
  if (int e = launch_pdl(kernel, dim3(kCtas), dim3(kWarps<NT> * 32), kSmem, st, p)) return e;
  if (spans < 16)
    return launch_pdl(fa2_kv4_combine_kernel<D, kRows, 1, false>, dim3(static_cast<unsigned>(units * (kRows / 8))), dim3(256), 0, st, p,
                      row_tiles);
  return launch_pdl(join ? fa2_kv4_combine_kernel<D, kRows, 8, true> : fa2_kv4_combine_kernel<D, kRows, 8, false>,
                    dim3(static_cast<unsigned>(units * kRows)), dim3(256), 0, st, p, row_tiles);
}

template <int D>
int launch_attn(const Attn4Problem& p, long long max_rows, cudaStream_t st) {
  return wide_rows(max_rows) ? launch_attn_d<D, 2>(p, max_rows, st) : launch_attn_d<D, 1>(p, max_rows, st);
}

size_t attn_slots(bool wide) { return wide ? static_cast<size_t>(kSpans<2>) * 2 * 16 : static_cast<size_t>(kSpans<1>) * 2 * 8; }

constexpr int kMaxKeys = 1 << 30;  // of a request: positions, rounded up, in 32 bits

int check_attn_sizes(int B, int H, int H_kv, int total_q, int max_q, int d) {
  if (B < 1 || H < 1 || total_q < 0 || max_q < 0 || total_q > (1 << 30)) return FA2_ERR_SHAPE;
  if (total_q == 0) max_q = 0;  // (a step without queries, whatever the bound)
  if (max_q > total_q || (total_q > 0 && max_q < 1)) return FA2_ERR_SHAPE;
  if (!head_dim_ok(d)) return FA2_ERR_HEADDIM;
  if (int rc = check_heads(H, H_kv)) return rc;
  // combine grid: a CTA per row, rounded up to whole units
  const long long rows = (static_cast<long long>(H / H_kv) * max_q + 15) / 16 * 16;
  if (rows > (1LL << 30) || static_cast<double>(B) * H_kv * rows > 2147483647.0) return FA2_ERR_SHAPE;
  return FA2_OK;
}

}  // namespace

int read_attn4_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_attn4_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_attn4_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

extern "C" {

size_t fa2_kv4_attn_workspace_bytes(int B, int H, int H_kv, int max_seqlen_q, int max_seqlen_k, int d) {
  if (max_seqlen_k > kMaxKeys) max_seqlen_k = kMaxKeys;
  if (max_seqlen_q < 1 || max_seqlen_k < 1 || check_attn_sizes(B, H, H_kv, max_seqlen_q, max_seqlen_q, d) != FA2_OK) return 0;
  const long long max_rows = static_cast<long long>(H / H_kv) * max_seqlen_q;
  if (unit_warps(B, H_kv, max_rows, max_seqlen_k)) return 0;
  const size_t rows = attn_slots(wide_rows(max_rows));
  return round_up(rows * d * sizeof(float)) + round_up(rows * sizeof(float2)) +
         round_up((static_cast<size_t>(B) + 2) * sizeof(long long));
}

int fa2_kv4_attn(const void* q, const void* cache, long long page_stride, const int* block_table, long long table_stride,
                 const int* lens, const int* cu_seqlens_q, void* o, float* lse, int B, int H, int H_kv, int total_q,
                 int max_seqlen_q, int max_seqlen_k, int num_pages, int page_size, int table_width, int d, float scale,
                 float k_scale, float v_scale, int causal, void* workspace, size_t workspace_bytes, void* stream) {
  if (int rc = check_attn_sizes(B, H, H_kv, total_q, max_seqlen_q, d)) return rc;
  if (int rc = check_cache(cache, page_stride, num_pages, page_size, H_kv, d)) return rc;
  if (table_width < 1 || (B > 1 && (table_stride < table_width || !stride_ok(table_stride, B)))) return FA2_ERR_SHAPE;
  if (max_seqlen_k < 1) return FA2_ERR_SHAPE;
  if (max_seqlen_k > kMaxKeys) max_seqlen_k = kMaxKeys;
  if (static_cast<long long>(table_width) * page_size < max_seqlen_k) max_seqlen_k = table_width * page_size;
  if (!cu_seqlens_q && total_q > 0 && static_cast<long long>(B) * max_seqlen_q != total_q) return FA2_ERR_SHAPE;
  if (check_scale(scale) || !power_of_two(k_scale) || !power_of_two(v_scale) || check_scale(scale * k_scale))
    return FA2_ERR_SCALE;
  if (total_q == 0) return FA2_OK;
  if (!q || !block_table || !lens || !o || !lse) return FA2_ERR_NULL;
  if (!aligned(q, 16) || !aligned(o, 16) || !aligned(block_table, 4) || !aligned(lens, 4) || !aligned(cu_seqlens_q, 4) ||
      !aligned(lse, 4))
    return FA2_ERR_ALIGN;
  const size_t need = fa2_kv4_attn_workspace_bytes(B, H, H_kv, max_seqlen_q, max_seqlen_k, d);
  if (need > 0 && (!workspace || !aligned(workspace, kWsAlign) || workspace_bytes < need)) return FA2_ERR_WORKSPACE;
  const size_t qb = static_cast<size_t>(total_q) * H * d * 2;
  const size_t tb = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
  const Range outs[] = {range_of(o, qb), range_of(lse, static_cast<size_t>(total_q) * H * 4), range_of(workspace, need)};
  const Range ins[] = {range_of(q, qb), range_of(cache, cache_span(page_stride, num_pages, page_size, H_kv, d)),
                       range_of(block_table, tb), range_of(lens, static_cast<size_t>(B) * 4),
                       range_of(cu_seqlens_q, cu_seqlens_q ? static_cast<size_t>(B + 1) * 4 : 0)};
  for (int i = 0; i < (need > 0 ? 3 : 2); ++i) {
    for (const Range& r : ins)
      if (r.lo != r.hi && overlap(outs[i], r)) return FA2_ERR_ALIAS;
    for (int j = i + 1; j < (need > 0 ? 3 : 2); ++j)
      if (overlap(outs[i], outs[j])) return FA2_ERR_ALIAS;
  }
  const long long max_rows = static_cast<long long>(H / H_kv) * max_seqlen_q;
  const size_t rows = attn_slots(wide_rows(max_rows));  // (not touched where need is 0)
  Attn4Problem p{};
  p.q = static_cast<const __nv_bfloat16*>(q);
  p.o = static_cast<__nv_bfloat16*>(o);
  p.lse = lse;
  p.cache = paged_cache(cache, page_stride, num_pages, page_size, H_kv);
  p.table = block_table;
  p.table_stride = table_stride;
  p.table_bytes = tb;
  p.q_bytes = qb;
  p.lens = lens;
  p.cu_q = cu_seqlens_q;
  char* ws = static_cast<char*>(workspace);
  p.part = reinterpret_cast<float*>(ws);
  ws += round_up(rows * d * sizeof(float));
  p.part_ml = reinterpret_cast<float2*>(ws);
  ws += round_up(rows * sizeof(float2));
  p.start = reinterpret_cast<long long*>(ws);
  p.B = B;
  p.H = H;
  p.G = H / H_kv;
  p.total_q = total_q;
  p.uniform_q = max_seqlen_q;
  p.max_q = max_seqlen_q;
  p.max_k = max_seqlen_k;
  p.scale_log2 = scale * k_scale * 1.44269504088896341f;
  p.v_scale = v_scale;
  p.causal = causal != 0;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  g_launched = true;
  const int e = d == 16    ? launch_attn<16>(p, max_rows, st)
                : d == 32  ? launch_attn<32>(p, max_rows, st)
                : d == 64  ? launch_attn<64>(p, max_rows, st)
                           : launch_attn<128>(p, max_rows, st);
  return e ? record_cuda_failure(e, "kv4 attention launch") : FA2_OK;
}

}  // extern "C"
