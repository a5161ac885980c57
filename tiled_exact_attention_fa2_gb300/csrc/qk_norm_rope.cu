// Per-head norm of queries and keys with the position rotation in the same
// pass, and its gradient: what a transformer layer does to q and k between
// the projection and the attention kernels.
//
// For a row x of d values (one head of one token), gain w and
// r = 1 / sqrt(mean x^2 + eps):
//   y_i = x_i r w_i
//   out_a = y_a c - y_b s,  out_b = y_b c + y_a s   for the pairs (a, b) of
//   the first rot columns, (i, i + rot/2) or (2 i, 2 i + 1), with the cosine
//   c and sine s of the token's position from an fp32 table;
//   the columns from rot on are y.
// Gradient: with g = the pairs of dout turned back (s -> -s) and h = g w,
//   dx = r h - x r^3 mean(h x),   dw = sum over rows of g x r.
//
// Both passes are bound by HBM (4 and 6 bytes per element against about 10
// and 20 flops): one read of every input, one write of every output, nothing
// kept in between (r is recomputed by the backward pass).  A row is held by
// d / 8 lanes, 8 columns (16 bytes) each, so a warp covers 32 * 8 / d rows
// with whole 32-byte sectors; a row's sums are butterfly shuffles within its
// lanes.  With a partner column's value (of a half-split pair one shuffle of
// the packed bf16 words away, of an interleaved one in the same word) a
// rotated value is x c' + x_partner s', so gain and rotation are folded into
// two factors per column that a lane makes once per token and uses for
// several heads; the arithmetic is on packed pairs of fp32.
//
// Measured on a GB300 (device time): 4 x 1023 tokens x 32 heads of 64 columns
// forward 5.8 us (5.8 TB/s); the gradient for 16384 tokens x 40 heads of 128
// 87.6 us (5.84 TB/s, 86 % of a copy's rate; the same bytes through an
// elementwise sum take 74 us), of which the sums of the gains' gradients are
// about 3 us, forward 53.9 us (6.2 TB/s, 92 %); 48 tokens x 40 heads 2.2 us.
// A form of the gradient with 16 columns a lane took 84 of its 89.5 us without
// its arithmetic (loads, one addition, stores): what is left is how the rows
// come and go, not what is done with them.
//
// All sums and the arithmetic are fp32; the one rounding to bf16 is at the
// store.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>
#include <utility>

#include "args.h"
#include "fa2.h"
#include "launch.h"
#include "ptx.cuh"

namespace fa2 {
namespace {

__device__ int g_norm_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

struct View {  // [B, heads, N, d] with the last dimension contiguous; strides in elements
  char* p;
  long long sb, sh, sn;
};

struct NormProblem {
  View x[2], y[2], g[2];  // of q and k: input, output (dx in the backward pass), dout (backward only)
  const void* w[2];
  float* partial;  // backward: [CTA][d] sums for dw (a CTA works for q or for k), or NULL
  const float* rope;
  const int* positions;
  int heads[2], chunks[2];  // heads, and lane-group items per token, of q and k
  unsigned items[2];        // B * N * chunks
  unsigned tokens;          // B * N
  unsigned ctas_q;          // CTAs below this one work for q
  int N, rot, max_pos, w_fp32;
  float eps;
};

// The gains of 8 columns (16-byte aligned).
__device__ __forceinline__ void gains(float (&f)[8], const void* w, int fp32, int col) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (fp32) {
    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(w) + col);
    const float4 a = __ldg(p), b = __ldg(p + 1);
    f[0] = a.x, f[1] = a.y, f[2] = a.z, f[3] = a.w, f[4] = b.x, f[5] = b.y, f[6] = b.z, f[7] = b.w;
  } else {
    const uint4 u = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(w) + col));
    const uint32_t v[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float2 t = unpack_bf16x2(v[i]);
      f[2 * i] = t.x, f[2 * i + 1] = t.y;
    }
  }
}

template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int s = LANES / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// The two bf16 of a word as a packed pair of fp32.
__device__ __forceinline__ uint64_t widen2(uint32_t w) {
  return f2_pack(__uint_as_float(w << 16), __uint_as_float(w & 0xffff0000u));
}

// The rotation partners of a lane's 8 columns `col` ..: which lane holds them
// (half split; of an interleaved pair the other half of the word), whether
// these columns turn at all, and the sign of their sine.
struct Partner {
  int lane;
  bool turns, low;
  uint32_t keep, flip;  // for the partners' packed words
};
template <bool INTER>
__device__ __forceinline__ Partner partner_of(int rot, int col, bool back) {
  Partner t;
  t.lane = threadIdx.x & 31;
  t.turns = col < rot;
  t.low = col < rot / 2;
  if (!INTER && t.turns) t.lane += t.low ? rot / 16 : -(rot / 16);
  t.keep = t.turns ? 0xffffffffu : 0u;
  // forward: the first of a pair takes minus its partner's sine, the second plus
  t.flip = !t.turns ? 0u : INTER ? (back ? 0x80000000u : 0x00008000u) : (t.low != back ? 0x80008000u : 0u);
  return t;
}

// The partners' words, signed (zeros where nothing turns: their factor is 0,
// and an infinity must not meet it).
template <bool INTER>
__device__ __forceinline__ uint32_t partner_word(const Partner& t, uint32_t w) {
  const uint32_t v = INTER ? __byte_perm(w, 0, 0x1032) : __shfl_sync(0xffffffffu, w, t.lane);
  return (v & t.keep) ^ t.flip;
}

// Cosines and sines of the lane's 8 columns at a position: rotated_j =
// x_j c_j + partner_j s_j.
template <bool INTER>
__device__ __forceinline__ void load_turn(float (&c)[8], float (&s)[8], const Partner& t, const NormProblem& p, int pos,
                                          int col) {
  if (!t.turns) {
#pragma unroll
    for (int i = 0; i < 8; ++i) c[i] = 1.f, s[i] = 0.f;
    return;
  }
  const int half = p.rot >> 1;
  const float* row = p.rope + static_cast<long long>(pos) * p.rot;
  if (INTER) {
    const float4 a = __ldg(reinterpret_cast<const float4*>(row + (col >> 1)));
    const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + (col >> 1)));
    const float cc[4] = {a.x, a.y, a.z, a.w}, ss[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) c[2 * i] = c[2 * i + 1] = cc[i], s[2 * i] = s[2 * i + 1] = ss[i];
  } else {
    row += t.low ? col : col - half;
#pragma unroll
    for (int i = 0; i < 8; i += 4) {
      const float4 a = __ldg(reinterpret_cast<const float4*>(row + i));
      const float4 b = __ldg(reinterpret_cast<const float4*>(row + half + i));
      c[i] = a.x, c[i + 1] = a.y, c[i + 2] = a.z, c[i + 3] = a.w;
      s[i] = b.x, s[i + 1] = b.y, s[i + 2] = b.z, s[i + 3] = b.w;
    }
  }
}

// A lane group's item: `count` heads from h0 on of token (b, n), number tok of
// B * N; none for an item past the end or at a bad position (it does its
// arithmetic on nothing: shuffles are warp-wide).
struct Item {
  unsigned tok, chunk;
  int b, n, h0, pos, count;
};

// The item's heads, and its position as it stands in memory.
template <int ROWS>
__device__ __forceinline__ void place(Item& it, const NormProblem& p, int which) {
  const bool live = it.tok < p.tokens;
  it.h0 = static_cast<int>(it.chunk) * ROWS;
  it.count = live ? min(ROWS, p.heads[which] - it.h0) : 0;
  it.pos = it.n;
  if (p.rot > 0 && p.positions && live) it.pos = __ldg(p.positions + it.tok);
}
// Whether the position is one; if not the item has no rows.
__device__ __forceinline__ bool check_position(Item& it, const NormProblem& p) {
  bool fine = true;
  if (p.rot > 0) {
    if (it.count > 0 && (it.pos < 0 || it.pos >= p.max_pos)) {
      atomicCAS(&g_norm_status, kDevOk, kDevBadIndex);
      it.count = 0;
      fine = false;
    }
    if (it.count == 0) it.pos = 0;
  }
  return fine;
}

template <int ROWS>
__device__ __forceinline__ Item find_item(const NormProblem& p, int which, unsigned id) {
  Item it;
  it.tok = id / static_cast<unsigned>(p.chunks[which]);
  it.chunk = id - it.tok * p.chunks[which];
  it.b = static_cast<int>(it.tok / static_cast<unsigned>(p.N));
  it.n = static_cast<int>(it.tok - static_cast<unsigned>(it.b) * p.N);
  place<ROWS>(it, p, which);
  return it;
}

__device__ __forceinline__ char* row_at(const View& v, const Item& it, int col) {
  return it.count > 0 ? v.p + 2 * (it.b * v.sb + it.n * v.sn + it.h0 * v.sh + col) : v.p;
}

template <int D, bool INTER, int ROWS>
__global__ void __launch_bounds__(256, ROWS == 8 ? 3 : 0) fa2_qk_norm_rope_kernel(const NormProblem p) {
  constexpr int kLanes = D / 8;
  griddep_wait();
  griddep_launch_dependents();
  const int col = (threadIdx.x % kLanes) * 8;
  const int which = blockIdx.x >= p.ctas_q;
  const unsigned cta = which ? blockIdx.x - p.ctas_q : blockIdx.x;
  Item it = find_item<ROWS>(p, which, cta * (256u / kLanes) + threadIdx.x / kLanes);
  check_position(it, p);
  const char* src = row_at(p.x[which], it, col);
  const long long sx = 2 * p.x[which].sh;
  uint4 raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    raw[i] = make_uint4(0, 0, 0, 0);
    if (i < it.count) raw[i] = *reinterpret_cast<const uint4*>(src + i * sx);
  }
  const Partner partner = partner_of<INTER>(p.rot, col, false);
  uint64_t wc[4], ws[4];  // gain times cosine; the partner's gain times sine
  {
    float c[8], s[8];
    load_turn<INTER>(c, s, partner, p, it.pos, col);
    float w[8], pw[8];
    gains(w, p.w[which], p.w_fp32, col);
    if (!INTER) gains(pw, p.w[which], p.w_fp32, col + (partner.lane - static_cast<int>(threadIdx.x & 31)) * 8);
#pragma unroll
    for (int j = 0; j < 8; ++j) {
      c[j] *= w[j];
      s[j] *= INTER ? w[j ^ 1] : pw[j];
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) wc[j] = f2_pack(c[2 * j], c[2 * j + 1]), ws[j] = f2_pack(s[2 * j], s[2 * j + 1]);
  }
  char* dst = row_at(p.y[which], it, col);
  const long long sy = 2 * p.y[which].sh;
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const uint32_t w[4] = {raw[i].x, raw[i].y, raw[i].z, raw[i].w};
    uint64_t x[4], o[4], sq = 0;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      x[j] = widen2(w[j]);
      sq = ffma2(x[j], x[j], sq);
      o[j] = ffma2(widen2(partner_word<INTER>(partner, w[j])), ws[j], fmul2(x[j], wc[j]));
    }
    const float2 q = f2_unpack(sq);
    const float r = rsqrtf(sum_lanes<kLanes>(q.x + q.y) * (1.f / D) + p.eps);
    const uint64_t rr = f2_pack(r, r);
    uint32_t out[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      const float2 f = f2_unpack(fmul2(o[j], rr));
      out[j] = pack_bf16x2(f.x, f.y);
    }
    if (i < it.count) *reinterpret_cast<uint4*>(dst + i * sy) = make_uint4(out[0], out[1], out[2], out[3]);
  }
}

__device__ __forceinline__ void load16(uint32_t (&w)[4], uint32_t at) {
  asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w[0]), "=r"(w[1]), "=r"(w[2]), "=r"(w[3]) : "r"(at) : "memory");
}

// Backward: persistent CTAs, each for q or for k (in proportion to their
// heads), so that a lane sums dw of its 8 columns in registers over all its
// rows; the CTA's sums are joined in shared memory and written to its own
// slot, which the dw kernel adds up in a fixed order (the result does not
// depend on the order CTAs run in).  The next item's rows are on their way
// into shared memory, each thread's own pieces, while this one's are worked
// on, so no registers wait for memory (without this 90.6 us; 20 warps an SM
// with it, since 16 columns a lane, three stages, the angles fetched the same
// way or the partners read from shared memory all cost more: 89-116).
constexpr int kBwdThreads = 128, kBwdPerSm = 5;
template <int D, bool INTER, int ROWS>
__global__ void __launch_bounds__(kBwdThreads, kBwdPerSm) fa2_qk_norm_rope_bwd_kernel(const NormProblem p) {
  constexpr int kLanes = D / 8, kGroups = kBwdThreads / kLanes;
  __shared__ uint4 ring[2 * 2 * ROWS * kBwdThreads];  // [stage][row][x, dout][thread]
  __shared__ float red[kGroups][D];
  griddep_wait();
  griddep_launch_dependents();
  const int col = (threadIdx.x % kLanes) * 8, group = threadIdx.x / kLanes;
  const int which = blockIdx.x >= p.ctas_q;
  const unsigned cta = which ? blockIdx.x - p.ctas_q : blockIdx.x;
  const unsigned step = (which ? gridDim.x - p.ctas_q : p.ctas_q) * kGroups;
  const Partner partner = partner_of<INTER>(p.rot, col, true);
  const long long sx = 2 * p.x[which].sh, sg = 2 * p.g[which].sh, sy = 2 * p.y[which].sh;
  uint64_t w[4], dw[4];
  {
    float f[8];
    gains(f, p.w[which], p.w_fp32, col);
#pragma unroll
    for (int j = 0; j < 4; ++j) w[j] = f2_pack(f[2 * j], f[2 * j + 1]), dw[j] = 0;
  }
  const uint32_t mine = smem_u32(ring) + threadIdx.x * 16;
  constexpr uint32_t kPiece = kBwdThreads * 16, kStage = 2 * ROWS * kPiece;
  auto fetch = [&](const Item& it, uint32_t at) {
    const char* px = row_at(p.x[which], it, col);
    const char* pg = row_at(p.g[which], it, col);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const bool there = i < it.count;
      copy16_async(at + 2 * i * kPiece, there ? px + i * sx : px, there);
      copy16_async(at + (2 * i + 1) * kPiece, there ? pg + i * sg : pg, there);
    }
  };
  // (the loop bound is the same for every lane of a warp: shuffles inside)
  const unsigned rounds = (p.items[which] + step - 1) / step;
  Item next = find_item<ROWS>(p, which, cta * kGroups + group);
  fetch(next, mine);
  copy_async_commit();
  // a round is `step` items further: so many tokens and chunks, sequences and tokens
  const unsigned chunks = p.chunks[which], d_tok = step / chunks, d_chunk = step - d_tok * chunks;
  const int d_b = static_cast<int>(d_tok / static_cast<unsigned>(p.N)), d_n = static_cast<int>(d_tok) - d_b * p.N;
  for (unsigned k = 0; k < rounds; ++k) {
    Item it = next;
    const uint32_t at = mine + (k & 1) * kStage;
    if (k + 1 < rounds) {
      const unsigned c = next.chunk + d_chunk, carry = c >= chunks;
      next.chunk = carry ? c - chunks : c;
      next.tok += d_tok + carry;
      next.b += d_b;
      next.n += d_n + static_cast<int>(carry);
      if (next.n >= p.N) {
        next.n -= p.N;
        ++next.b;
      }
      place<ROWS>(next, p, which);
      fetch(next, mine + (~k & 1) * kStage);
    }
    copy_async_commit();
    const bool fine = check_position(it, p);
    char* py = row_at(p.y[which], it, col);
    uint64_t c[4], s[4];
    {
      float cf[8], sf[8];
      load_turn<INTER>(cf, sf, partner, p, it.pos, col);
#pragma unroll
      for (int j = 0; j < 4; ++j) c[j] = f2_pack(cf[2 * j], cf[2 * j + 1]), s[j] = f2_pack(sf[2 * j], sf[2 * j + 1]);
    }
    copy_async_wait<1>();
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      uint32_t wx[4], wg[4];
      load16(wx, at + 2 * i * kPiece);
      load16(wg, at + (2 * i + 1) * kPiece);
      if (!fine) wx[0] = wx[1] = wx[2] = wx[3] = wg[0] = wg[1] = wg[2] = wg[3] = 0;
      uint64_t x[4], g[4], h[4], sq = 0, hx = 0;
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        x[j] = widen2(wx[j]);
        g[j] = ffma2(widen2(partner_word<INTER>(partner, wg[j])), s[j], fmul2(widen2(wg[j]), c[j]));
        h[j] = fmul2(g[j], w[j]);
        sq = ffma2(x[j], x[j], sq);
        hx = ffma2(h[j], x[j], hx);
      }
      const float2 q = f2_unpack(sq), v = f2_unpack(hx);
      const float r = rsqrtf(sum_lanes<kLanes>(q.x + q.y) * (1.f / D) + p.eps);
      // (a row left out has x = dout = 0 and adds nothing)
      const float along = -r * r * (sum_lanes<kLanes>(v.x + v.y) * (1.f / D));
      const uint64_t rr = f2_pack(r, r), aa = f2_pack(along, along);
      uint32_t out[4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        dw[j] = ffma2(g[j], fmul2(x[j], rr), dw[j]);
        const float2 f = f2_unpack(fmul2(ffma2(x[j], aa, h[j]), rr));
        out[j] = pack_bf16x2(f.x, f.y);
      }
      if (i < it.count) *reinterpret_cast<uint4*>(py + i * sy) = make_uint4(out[0], out[1], out[2], out[3]);
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int j = 0; j < 4; ++j) {
    const float2 f = f2_unpack(dw[j]);
    red[group][col + 2 * j] = f.x;
    red[group][col + 2 * j + 1] = f.y;
  }
  __syncthreads();
  for (int i = threadIdx.x; i < D; i += kBwdThreads) {
    float t = 0.f;
#pragma unroll 8
    for (int k = 0; k < kGroups; ++k) t += red[k][i];
    p.partial[static_cast<size_t>(blockIdx.x) * D + i] = t;
  }
}

// dw of q (blockIdx.y = 0) and k: the sums of their CTAs' slots, 32 columns
// per block; each of the 32 warps adds every 32nd slot (so the loads of all
// of a warp's slots are in flight at once), then warp w adds column w's 32
// sums by a butterfly, whose order is fixed.
__global__ void __launch_bounds__(1024) fa2_qk_norm_dw_kernel(const float* __restrict__ partial, int slots_q, int slots, int d,
                                                              float* dwq, float* dwk) {
  __shared__ float red[32][33];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  const int first = blockIdx.y ? slots_q : 0, last = blockIdx.y ? slots : slots_q;
  float* out = blockIdx.y ? dwk : dwq;
  if (!out) return;
  float s = 0.f;
  if (c < d)
#pragma unroll 8
    for (int i = first + warp; i < last; i += 32) s += partial[static_cast<size_t>(i) * d + c];
  red[warp][lane] = s;
  __syncthreads();
  s = sum_lanes<32>(red[lane][warp]);
  if (lane == 0 && blockIdx.x * 32 + warp < d) out[blockIdx.x * 32 + warp] = s;
}


constexpr int kBwdCtas = 152 * kBwdPerSm;  // one wave
// Rows of q and k that lane groups of `rows` heads have room for, per token.
inline long long room(int hq, int hk, int rows) { return rows * ((hq + rows - 1LL) / rows + (hk + rows - 1) / rows); }

// Heads a lane group of the forward pass takes: one where the call is small
// (shorter chains of loads: 0.3 million elements 2.1 us against 2.5 with four,
// 1 million 3.3 / 2.7) or nearly all rows of a group would be missing, else
// four.  With eight the angles and the addresses are made half as often: of
// half-split pairs, 128 columns, 53.9 against 57.0 us for 16384 tokens x 40
// heads, 15.9 / 16.8 for 4096, 9.7 / 9.6 for 2048 (1.4 rounds of CTAs: so from
// two rounds on, and where at most one row in nine is missing); interleaved
// pairs, whose angles are half the bytes, gain nothing (54.6 / 54.4), rows of
// 16 columns neither.
template <int D, bool INTER>
int forward_rows(long long tokens, int hq, int hk) {
  const int n = hq + hk;
  if (tokens * n * D < 152 * 4096 || room(hq, hk, 4) >= 3 * n) return 1;
  return !INTER && D >= 32 && 8 * room(hq, hk, 8) <= 9 * n && tokens * room(hq, hk, 8) * D >= 152LL * 3 * 256 * 2 * 64 ? 8 : 4;
}

// The same for the gradient.  Measured, 128 columns, one / two / four heads a
// group in us: 0.1 million elements of 32 + 8 heads 4.0 / 3.7 / 3.8, 0.3
// million 5.0 / 4.6 / 4.3, 40 million 66.7 / 50.4 / 45.3; 40 million of 4 + 1
// heads 70.2 / 59.1 / 60.9, 2 + 2 69.4 / 53.6 / 72.4, 2 + 1 69.9 / 64.6 / 93.9:
// with four the missing rows cost the most.
inline int backward_rows(long long tokens, int hq, int hk, int d) {
  const int n = hq + hk;
  if (tokens * n * d < 152 * 1024) return 1;
  if (5 * room(hq, hk, 4) <= 6 * room(hq, hk, 2)) return 4;
  return 2 * room(hq, hk, 2) < 3 * n ? 2 : 1;
}

// Items of `rows` heads, and the CTAs they fill.
void divide(NormProblem* p, long long tokens, int rows, int d, int threads, unsigned (&ctas)[2]) {
  const unsigned per = threads / (d / 8);
  p->tokens = static_cast<unsigned>(tokens);
  for (int i = 0; i < 2; ++i) {
    p->chunks[i] = (p->heads[i] + rows - 1) / rows;
    p->items[i] = static_cast<unsigned>(tokens * p->chunks[i]);
    ctas[i] = (p->items[i] + per - 1) / per;
  }
}

template <int D, bool INTER>
int launch_fwd_d(NormProblem p, long long tokens, cudaStream_t st) {
  const int rows = forward_rows<D, INTER>(tokens, p.heads[0], p.heads[1]);
  unsigned ctas[2];
  divide(&p, tokens, rows, D, 256, ctas);
  p.ctas_q = ctas[0];
  const dim3 grid(ctas[0] + ctas[1]);
  if constexpr (!INTER && D >= 32)
    if (rows == 8) return launch_pdl(fa2_qk_norm_rope_kernel<D, INTER, 8>, grid, dim3(256), 0, st, p);
  return rows == 4 ? launch_pdl(fa2_qk_norm_rope_kernel<D, INTER, 4>, grid, dim3(256), 0, st, p)
                   : launch_pdl(fa2_qk_norm_rope_kernel<D, INTER, 1>, grid, dim3(256), 0, st, p);
}

template <int D, bool INTER>
int launch_bwd_d(NormProblem p, long long tokens, float* dwq, float* dwk, cudaStream_t st) {
  const int rows = backward_rows(tokens, p.heads[0], p.heads[1], D);
  unsigned ctas[2];
  divide(&p, tokens, rows, D, kBwdThreads, ctas);
  if (ctas[0] + ctas[1] > kBwdCtas) {  // q's and k's shares of the persistent CTAs
    const unsigned q = static_cast<unsigned>(static_cast<unsigned long long>(kBwdCtas) * p.items[0] /
                                             (static_cast<unsigned long long>(p.items[0]) + p.items[1]));
    ctas[0] = q < 1 ? 1 : (q > kBwdCtas - 1 ? kBwdCtas - 1 : q);
    ctas[1] = kBwdCtas - ctas[0];
  }
  p.ctas_q = ctas[0];
  const unsigned grid = ctas[0] + ctas[1];
  const auto kernel = rows == 4   ? fa2_qk_norm_rope_bwd_kernel<D, INTER, 4>
                      : rows == 2 ? fa2_qk_norm_rope_bwd_kernel<D, INTER, 2>
                                  : fa2_qk_norm_rope_bwd_kernel<D, INTER, 1>;
  const int e = launch_pdl(kernel, dim3(grid), dim3(kBwdThreads), 0, st, p);
  if (e || !p.partial) return e;
  return launch_pdl(fa2_qk_norm_dw_kernel, dim3((D + 31) / 32, 2), dim3(1024), 0, st, static_cast<const float*>(p.partial),
                    static_cast<int>(ctas[0]), static_cast<int>(grid), D, dwq, dwk);
}

// Where the elements of a strided [B, heads, N, d] tensor can lie, and
// whether its rows are apart from one another.
struct Layout {
  const void* p;
  int heads;
  long long s[3];  // batch, head, token
};

bool rows_apart(const Layout& t, int B, int N, int d) {
  long long size[3] = {B, t.heads, N}, stride[3] = {t.s[0], t.s[1], t.s[2]};
  for (int i = 0; i < 3; ++i)
    for (int j = i + 1; j < 3; ++j)
      if (stride[j] < stride[i]) {
        std::swap(stride[i], stride[j]);
        std::swap(size[i], size[j]);
      }
  long long span = d;
  for (int i = 0; i < 3; ++i)
    if (size[i] > 1) {
      if (stride[i] < span) return false;
      span += stride[i] * (size[i] - 1);
    }
  return true;
}

Range span_of(const Layout& t, int B, int N, int d) {
  const long long last = (B - 1) * t.s[0] + (t.heads - 1) * t.s[1] + (N - 1) * t.s[2] + d;
  return range_of(t.p, static_cast<size_t>(last) * 2);
}

bool same(const Layout& a, const Layout& b) {
  return a.p == b.p && a.heads == b.heads && a.s[0] == b.s[0] && a.s[1] == b.s[1] && a.s[2] == b.s[2];
}

// Whether two tensors may share an element.  Spans that overlap are still
// apart when both are heads of one token-major buffer (same token stride,
// batch stride a multiple of it) and take different parts of a token's row.
bool may_share(const Layout& a, const Layout& b, int B, int N, int d) {
  if (!overlap(span_of(a, B, N, d), span_of(b, B, N, d))) return false;
  const int step = N > 1 ? 2 : 0;  // the dimension that walks over tokens
  if (N == 1 && B == 1) return true;
  const long long sn = a.s[step];
  if (sn != b.s[step] || sn < 1) return true;
  if (N > 1 && B > 1 && (a.s[0] % sn != 0 || b.s[0] % sn != 0)) return true;
  const long long ea = (a.heads - 1) * a.s[1] + d, eb = (b.heads - 1) * b.s[1] + d;
  const long long bytes = static_cast<const char*>(b.p) - static_cast<const char*>(a.p);
  const long long off = ((bytes / 2) % sn + sn) % sn;
  return !(off >= ea && off + eb <= sn);
}

struct NormArgs {
  const void *q_weight, *k_weight;
  int weight_fp32;
  const float* rope;
  const int* positions;
  int B, H, H_kv, N, d, rot, interleaved, max_positions;
  float eps;
};

// `ins` and `outs`: the call's bf16 tensors, q's and k's in turn.
int validate_norm(const NormArgs& a, Layout* t, int count, int outs, const long long* strides) {
  if (a.B < 1 || a.H < 1 || a.N < 0) return FA2_ERR_SHAPE;
  if (!head_dim_ok(a.d)) return FA2_ERR_HEADDIM;
  if (int rc = check_heads(a.H, a.H_kv)) return rc;
  if (a.rot < 0 || a.rot > a.d || a.rot % 16 != 0 || (a.interleaved != 0 && a.interleaved != 1)) return FA2_ERR_SHAPE;
  const long long tokens = static_cast<long long>(a.B) * a.N;
  if (tokens * (static_cast<long long>(a.H) + a.H_kv) > 0x7fffffffLL) return FA2_ERR_SHAPE;
  if (!(std::isfinite(a.eps) && a.eps > 0.f)) return FA2_ERR_SCALE;
  if (a.rot > 0) {
    if (!a.rope) return FA2_ERR_NULL;
    if (a.max_positions < 1 || (!a.positions && a.N > a.max_positions)) return FA2_ERR_SHAPE;
    if (!aligned(a.rope, 16) || !aligned(a.positions, 4)) return FA2_ERR_ALIGN;
  }
  if (!aligned(a.q_weight, 16) || !aligned(a.k_weight, 16)) return FA2_ERR_ALIGN;
  if (tokens == 0) return FA2_OK;
  for (int i = 0; i < count; ++i) {
    if (!t[i].p) return FA2_ERR_NULL;
    t[i].heads = i % 2 ? a.H_kv : a.H;
    const long long size[3] = {a.B, t[i].heads, a.N};
    const long long own[3] = {static_cast<long long>(t[i].heads) * a.N * a.d, static_cast<long long>(a.N) * a.d, a.d};
    for (int j = 0; j < 3; ++j) {
      t[i].s[j] = size[j] == 1 ? own[j] : (strides ? strides[3 * i + j] : own[j]);
      if (!stride_ok(t[i].s[j], size[j] - 1)) return FA2_ERR_SHAPE;
      if (t[i].s[j] % 8 != 0) return FA2_ERR_ALIGN;
    }
    if (!aligned(t[i].p, 16)) return FA2_ERR_ALIGN;
  }
  for (int i = count - outs; i < count; ++i) {
    if (!rows_apart(t[i], a.B, a.N, a.d)) return FA2_ERR_ALIAS;
    for (int j = 0; j < i; ++j) {
      // An input may be overwritten row by row by the output of the same rows.
      if (j % 2 == i % 2 && j < count - outs && same(t[i], t[j])) continue;
      if (may_share(t[i], t[j], a.B, a.N, a.d)) return FA2_ERR_ALIAS;
    }
    const Range r = span_of(t[i], a.B, a.N, a.d);
    const size_t wb = static_cast<size_t>(a.d) * (a.weight_fp32 ? 4 : 2);
    if ((a.q_weight && overlap(r, range_of(a.q_weight, wb))) || (a.k_weight && overlap(r, range_of(a.k_weight, wb))))
      return FA2_ERR_ALIAS;
    if (a.rot > 0 && (overlap(r, range_of(a.rope, static_cast<size_t>(a.max_positions) * a.rot * 4)) ||
                      (a.positions && overlap(r, range_of(a.positions, static_cast<size_t>(tokens) * 4)))))
      return FA2_ERR_ALIAS;
  }
  return FA2_OK;
}

View view_of(const Layout& t) {
  return View{static_cast<char*>(const_cast<void*>(t.p)), t.s[0], t.s[1], t.s[2]};
}

NormProblem problem_of(const NormArgs& a) {
  NormProblem p{};
  p.w[0] = a.q_weight;
  p.w[1] = a.k_weight;
  p.rope = a.rope;
  p.positions = a.positions;
  p.heads[0] = a.H;
  p.heads[1] = a.H_kv;
  p.N = a.N;
  p.rot = a.rot;
  p.max_pos = a.max_positions;
  p.w_fp32 = a.weight_fp32;
  p.eps = a.eps;
  return p;
}

}  // namespace

int read_norm_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_norm_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_norm_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

#define FA2_NORM_DISPATCH(CALL)                                  \
  switch (d) {                                                   \
    case 16: e = interleaved ? CALL(16, true) : CALL(16, false); break;    \
    case 32: e = interleaved ? CALL(32, true) : CALL(32, false); break;    \
    case 64: e = interleaved ? CALL(64, true) : CALL(64, false); break;    \
    default: e = interleaved ? CALL(128, true) : CALL(128, false); break;  \
  }

extern "C" {

int fa2_qk_norm_rope(const void* q, const void* k, const void* q_weight, const void* k_weight, int weight_fp32,
                     const float* rope, const int* positions, void* q_out, void* k_out, int B, int H, int H_kv, int N,
                     int d, int rot_dim, int interleaved, int max_positions, float eps, const long long* strides,
                     void* stream) {
  const NormArgs a{q_weight, k_weight, weight_fp32, rope, positions, B, H, H_kv, N, d, rot_dim, interleaved,
                   max_positions, eps};
  Layout t[4] = {{q, 0, {}}, {k, 0, {}}, {q_out, 0, {}}, {k_out, 0, {}}};
  if (int rc = validate_norm(a, t, 4, 2, strides)) return rc;
  if (N == 0) return FA2_OK;
  NormProblem p = problem_of(a);
  g_launched = true;
  for (int i = 0; i < 2; ++i) {
    p.x[i] = view_of(t[i]);
    p.y[i] = view_of(t[2 + i]);
  }
  const long long tokens = static_cast<long long>(B) * N;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  int e;
#define FA2_CALL(D, I) launch_fwd_d<D, I>(p, tokens, st)
  FA2_NORM_DISPATCH(FA2_CALL)
#undef FA2_CALL
  return e ? record_cuda_failure(e, "qk norm rope launch") : FA2_OK;
}

size_t fa2_qk_norm_rope_bwd_workspace_bytes(int d) {
  return head_dim_ok(d) ? round_up(static_cast<size_t>(kBwdCtas) * d * sizeof(float)) : 0;
}

int fa2_qk_norm_rope_bwd(const void* dq_out, const void* dk_out, const void* q, const void* k, const void* q_weight,
                         const void* k_weight, int weight_fp32, const float* rope, const int* positions, void* dq,
                         void* dk, float* dq_weight, float* dk_weight, int B, int H, int H_kv, int N, int d,
                         int rot_dim, int interleaved, int max_positions, float eps, const long long* strides,
                         void* workspace, size_t workspace_bytes, void* stream) {
  const NormArgs a{q_weight, k_weight, weight_fp32, rope, positions, B, H, H_kv, N, d, rot_dim, interleaved,
                   max_positions, eps};
  Layout t[6] = {{dq_out, 0, {}}, {dk_out, 0, {}}, {q, 0, {}}, {k, 0, {}}, {dq, 0, {}}, {dk, 0, {}}};
  if (int rc = validate_norm(a, t, 6, 2, strides)) return rc;
  if (!aligned(dq_weight, 4) || !aligned(dk_weight, 4)) return FA2_ERR_ALIGN;
  const cudaStream_t st = static_cast<cudaStream_t>(stream);
  const size_t db = static_cast<size_t>(d) * 4;
  const bool wants = dq_weight || dk_weight;
  const size_t need = fa2_qk_norm_rope_bwd_workspace_bytes(d);
  if (N == 0) {  // no rows: the gains' gradients are zero
    for (float* w : {dq_weight, dk_weight})
      if (w)
        if (cudaError_t e = cudaMemsetAsync(w, 0, db, st)) return record_cuda_failure(static_cast<int>(e), "memset dw");
    return FA2_OK;
  }
  if (wants) {
    if (!workspace || !aligned(workspace, kWsAlign) || workspace_bytes < need) return FA2_ERR_WORKSPACE;
    // the gains' gradients and the workspace against everything else
    const size_t wb = static_cast<size_t>(d) * (weight_fp32 ? 4 : 2);
    const Range own[] = {range_of(dq_weight, dq_weight ? db : 0), range_of(dk_weight, dk_weight ? db : 0),
                         range_of(workspace, need)};
    const Range fixed[] = {range_of(q_weight, q_weight ? wb : 0), range_of(k_weight, k_weight ? wb : 0),
                           range_of(rope, rot_dim > 0 ? static_cast<size_t>(max_positions) * rot_dim * 4 : 0),
                           range_of(positions, positions && rot_dim > 0 ? static_cast<size_t>(B) * N * 4 : 0)};
    for (int i = 0; i < 3; ++i) {
      if (own[i].lo == own[i].hi) continue;
      for (const Layout& l : t)
        if (overlap(own[i], span_of(l, B, N, d))) return FA2_ERR_ALIAS;
      for (const Range& r : fixed)
        if (r.lo != r.hi && overlap(own[i], r)) return FA2_ERR_ALIAS;
      for (int j = i + 1; j < 3; ++j)
        if (own[j].lo != own[j].hi && overlap(own[i], own[j])) return FA2_ERR_ALIAS;
    }
  }
  NormProblem p = problem_of(a);
  g_launched = true;
  for (int i = 0; i < 2; ++i) {
    p.g[i] = view_of(t[i]);
    p.x[i] = view_of(t[2 + i]);
    p.y[i] = view_of(t[4 + i]);
  }
  p.partial = wants ? static_cast<float*>(workspace) : nullptr;
  const long long tokens = static_cast<long long>(B) * N;
  int e;
#define FA2_CALL(D, I) launch_bwd_d<D, I>(p, tokens, dq_weight, dk_weight, st)
  FA2_NORM_DISPATCH(FA2_CALL)
#undef FA2_CALL
  return e ? record_cuda_failure(e, "qk norm rope bwd launch") : FA2_OK;
}

}  // extern "C"
