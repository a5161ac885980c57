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
// with whole 32-byte sectors; the two sums of a row are butterfly shuffles
// within its lanes and a half-split pair's partner columns come by one
// shuffle.  A lane group takes several heads of one token, which loads the
// token's cosines and sines once (they are twice a head's bytes).
//
// All sums and the arithmetic are fp32; the one rounding to bf16 is at the
// store.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <cmath>
#include <utility>

#include "args.h"
#include "fa2.h"
#include "launch.h"
#include "ptx.cuh"

namespace fa2 {
namespace {

__device__ int g_norm_status;

struct View {  // [B, heads, N, d] with the last dimension contiguous; strides in elements
  char* p;
  long long sb, sh, sn;
};

struct NormProblem {
  View x[2], y[2], g[2];  // of q and k: input, output (dx in the backward pass), dout (backward only)
  const void* w[2];
  float* partial;  // backward: [CTA][2][d] sums for dw, or NULL
  const float* rope;
  const int* positions;
  int heads[2];  // H, H_kv
  int N, rot, max_pos, w_fp32;
  int chunks;     // lane-group items per token
  unsigned items;  // B * N * chunks
  float eps;
};

__device__ __forceinline__ void load8(const View& v, long long b, int h, int n, int col, uint4* out) {
  const __nv_bfloat16* p = reinterpret_cast<const __nv_bfloat16*>(v.p) + b * v.sb + h * v.sh + n * v.sn + col;
  *out = *reinterpret_cast<const uint4*>(p);
}
__device__ __forceinline__ void store8(const View& v, long long b, int h, int n, int col, const float (&f)[8]) {
  __nv_bfloat16* p = reinterpret_cast<__nv_bfloat16*>(v.p) + b * v.sb + h * v.sh + n * v.sn + col;
  *reinterpret_cast<uint4*>(p) = make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]),
                                            pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}
__device__ __forceinline__ void widen8(const uint4& u, float (&f)[8]) {
  const uint32_t w[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    const float2 t = unpack_bf16x2(w[i]);
    f[2 * i] = t.x;
    f[2 * i + 1] = t.y;
  }
}
__device__ __forceinline__ void load_gain(const void* w, int fp32, int col, float (&f)[8]) {
  if (!w) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = 1.f;
  } else if (fp32) {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = static_cast<const float*>(w)[col + i];
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) f[i] = __bfloat162float(static_cast<const __nv_bfloat16*>(w)[col + i]);
  }
}

template <int LANES>
__device__ __forceinline__ float sum_lanes(float v) {
#pragma unroll
  for (int s = LANES / 2; s > 0; s >>= 1) v += __shfl_xor_sync(0xffffffffu, v, s);
  return v;
}

// What one lane needs of its token's rotation: the cosines and signed sines
// of its 8 columns.  Half split: one pair per column, out = y c + partner s
// (s is negative in the low half).  Interleaved: 4 pairs.  Columns past the
// rotated part get c = 1, s = 0.
template <bool INTER>
struct Turn {
  float c[INTER ? 4 : 8], s[INTER ? 4 : 8];
  int partner;  // lane that holds the partner columns (half split)
};

template <int D, bool INTER>
__device__ __forceinline__ void load_turn(Turn<INTER>& t, const NormProblem& p, int pos, int col, bool back) {
  constexpr int kN = INTER ? 4 : 8;
  const int half = p.rot >> 1;
  const int lane = threadIdx.x & 31;
  t.partner = lane;
  if (col < p.rot) {
    int at;
    float sign;
    if (INTER) {
      at = col >> 1;
      sign = 1.f;
    } else {
      const bool low = col < half;
      at = low ? col : col - half;
      sign = low ? -1.f : 1.f;
      t.partner = lane + (low ? half : -half) / 8;
    }
    if (back) sign = -sign;
    const float* row = p.rope + static_cast<long long>(pos) * p.rot + at;
#pragma unroll
    for (int i = 0; i < kN; i += 4) {
      const float4 c = __ldg(reinterpret_cast<const float4*>(row + i));
      const float4 s = __ldg(reinterpret_cast<const float4*>(row + half + i));
      t.c[i] = c.x, t.c[i + 1] = c.y, t.c[i + 2] = c.z, t.c[i + 3] = c.w;
      t.s[i] = sign * s.x, t.s[i + 1] = sign * s.y, t.s[i + 2] = sign * s.z, t.s[i + 3] = sign * s.w;
    }
  } else {
#pragma unroll
    for (int i = 0; i < kN; ++i) t.c[i] = 1.f, t.s[i] = 0.f;
  }
}

// Columns past the rotated part are their own partner with s = 0; an
// infinity there would turn into NaN through inf * 0, so they are selected.
template <bool INTER>
__device__ __forceinline__ void rotate(const Turn<INTER>& t, bool turns, const float (&y)[8], float (&o)[8]) {
  if (INTER) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float a = y[2 * i], b = y[2 * i + 1];
      o[2 * i] = turns ? a * t.c[i] - b * t.s[i] : a;
      o[2 * i + 1] = turns ? b * t.c[i] + a * t.s[i] : b;
    }
  } else {
#pragma unroll
    for (int i = 0; i < 8; ++i) {
      const float q = __shfl_sync(0xffffffffu, y[i], t.partner);
      o[i] = turns ? y[i] * t.c[i] + q * t.s[i] : y[i];
    }
  }
}

// The lane group's item: heads [h0, h0 + ROWS) of token (b, n).  Heads past
// the last are left out by `h < total`; an item past the end, or at a bad
// position, does the arithmetic on nothing (shuffles are warp-wide).
struct Item {
  long long b;
  int n, h0, pos;
  bool live;
};

template <int ROWS>
__device__ __forceinline__ Item find_item(const NormProblem& p, unsigned id) {
  Item it;
  it.live = id < p.items;
  const unsigned tok = it.live ? id / p.chunks : 0;
  it.h0 = it.live ? static_cast<int>(id - tok * p.chunks) * ROWS : 0;
  it.b = tok / static_cast<unsigned>(p.N);
  it.n = static_cast<int>(tok - static_cast<unsigned>(it.b) * p.N);
  it.pos = it.n;
  if (p.rot > 0) {
    if (p.positions && it.live) it.pos = __ldg(p.positions + tok);
    if (it.live && (it.pos < 0 || it.pos >= p.max_pos)) {
      atomicCAS(&g_norm_status, kDevOk, kDevBadIndex);
      it.live = false;
    }
    if (!it.live) it.pos = 0;
  }
  return it;
}

template <int D, bool INTER, int ROWS>
__global__ void __launch_bounds__(256) fa2_qk_norm_rope_kernel(const NormProblem p) {
  constexpr int kLanes = D / 8;
  griddep_wait();
  griddep_launch_dependents();
  const int col = (threadIdx.x % kLanes) * 8;
  const Item it = find_item<ROWS>(p, blockIdx.x * (256u / kLanes) + threadIdx.x / kLanes);
  const int total = p.heads[0] + p.heads[1];
  uint4 raw[ROWS];
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = it.h0 + i, which = h >= p.heads[0];
    raw[i] = make_uint4(0, 0, 0, 0);
    if (it.live && h < total) load8(p.x[which], it.b, h - (which ? p.heads[0] : 0), it.n, col, &raw[i]);
  }
  Turn<INTER> turn;
  load_turn<D, INTER>(turn, p, it.pos, col, false);
#pragma unroll
  for (int i = 0; i < ROWS; ++i) {
    const int h = it.h0 + i, which = h >= p.heads[0];
    float x[8], w[8], o[8];
    widen8(raw[i], x);
    load_gain(p.w[which], p.w_fp32, col, w);
    float ss = 0.f;
#pragma unroll
    for (int j = 0; j < 8; ++j) ss = fmaf(x[j], x[j], ss);
    const float r = rsqrtf(sum_lanes<kLanes>(ss) * (1.f / D) + p.eps);
#pragma unroll
    for (int j = 0; j < 8; ++j) x[j] = x[j] * r * w[j];
    rotate<INTER>(turn, col < p.rot, x, o);
    if (it.live && h < total) store8(p.y[which], it.b, h - (which ? p.heads[0] : 0), it.n, col, o);
  }
}

// Backward: persistent CTAs, so that each lane sums dw of its 8 columns (of
// q and of k) in registers over all its rows; the CTA's sums are joined in
// shared memory and written to its own slot, which dw_kernel adds up in a
// fixed order (the result does not depend on the order CTAs run in).
template <int D, bool INTER, int ROWS>
__global__ void __launch_bounds__(256) fa2_qk_norm_rope_bwd_kernel(const NormProblem p) {
  constexpr int kLanes = D / 8, kGroups = 256 / kLanes;
  __shared__ float red[kGroups][D];
  griddep_wait();
  griddep_launch_dependents();
  const int col = (threadIdx.x % kLanes) * 8, group = threadIdx.x / kLanes;
  const int total = p.heads[0] + p.heads[1];
  float dw[2][8] = {};
  float w[2][8];
  load_gain(p.w[0], p.w_fp32, col, w[0]);
  load_gain(p.w[1], p.w_fp32, col, w[1]);
  const unsigned step = gridDim.x * kGroups;
  // (the loop bound is the same for every lane of a warp: shuffles inside)
  const unsigned rounds = (p.items + step - 1) / step;
  for (unsigned k = 0; k < rounds; ++k) {
    const Item it = find_item<ROWS>(p, k * step + blockIdx.x * kGroups + group);
    uint4 rx[ROWS], rg[ROWS];
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int h = it.h0 + i, which = h >= p.heads[0];
      rx[i] = rg[i] = make_uint4(0, 0, 0, 0);
      if (it.live && h < total) {
        load8(p.x[which], it.b, h - (which ? p.heads[0] : 0), it.n, col, &rx[i]);
        load8(p.g[which], it.b, h - (which ? p.heads[0] : 0), it.n, col, &rg[i]);
      }
    }
    Turn<INTER> turn;
    load_turn<D, INTER>(turn, p, it.pos, col, true);
#pragma unroll
    for (int i = 0; i < ROWS; ++i) {
      const int h = it.h0 + i, which = h >= p.heads[0];
      const bool real = it.live && h < total;
      float x[8], o[8], g[8];
      widen8(rx[i], x);
      widen8(rg[i], o);
      rotate<INTER>(turn, col < p.rot, o, g);
      float ss = 0.f, hx = 0.f;
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        ss = fmaf(x[j], x[j], ss);
        o[j] = g[j] * (which ? w[1][j] : w[0][j]);
        hx = fmaf(o[j], x[j], hx);
      }
      ss = sum_lanes<kLanes>(ss);
      hx = sum_lanes<kLanes>(hx);
      const float r = rsqrtf(ss * (1.f / D) + p.eps);
      const float along = r * r * (hx * (1.f / D));
#pragma unroll
      for (int j = 0; j < 8; ++j) {
        const float t = real ? g[j] * x[j] * r : 0.f;
        if (which)
          dw[1][j] += t;
        else
          dw[0][j] += t;
        o[j] = r * (o[j] - x[j] * along);
      }
      if (real) store8(p.y[which], it.b, h - (which ? p.heads[0] : 0), it.n, col, o);
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int which = 0; which < 2; ++which) {
    __syncthreads();
#pragma unroll
    for (int j = 0; j < 8; ++j) red[group][col + j] = dw[which][j];
    __syncthreads();
    for (int c = threadIdx.x; c < D; c += 256) {
      float s = 0.f;
#pragma unroll 8
      for (int i = 0; i < kGroups; ++i) s += red[i][c];
      p.partial[(static_cast<size_t>(blockIdx.x) * 2 + which) * D + c] = s;
    }
  }
}

// dw[which][c] = sum over the CTAs' slots: 32 columns per block, 8 warps that
// each add every eighth slot, then the 8 sums in order.
__global__ void __launch_bounds__(256) fa2_qk_norm_dw_kernel(const float* __restrict__ partial, int slots, int d,
                                                             float* dwq, float* dwk) {
  __shared__ float red[8][32];
  griddep_wait();
  griddep_launch_dependents();
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;  // of 2 d
  float s = 0.f;
  if (c < 2 * d)
    for (int i = warp; i < slots; i += 8) s += partial[static_cast<size_t>(i) * 2 * d + c];
  red[warp][lane] = s;
  __syncthreads();
  if (warp == 0 && c < 2 * d) {
    float t = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i) t += red[i][lane];
    float* out = c < d ? dwq : dwk;
    if (out) out[c < d ? c : c - d] = t;
  }
}

constexpr int kBwdCtas = 152 * 4;
// From this many lane groups of four heads on, four heads a group fill the
// GPU (152 SMs, 2048 threads each); below, one head a group gives shorter
// chains of loads.
inline bool many(long long tokens, int heads, int d) {
  return tokens * ((heads + 3) / 4) * (d / 8) >= 152LL * 2048;
}

template <int D, bool INTER>
int launch_fwd_d(NormProblem p, long long tokens, cudaStream_t st) {
  const int heads = p.heads[0] + p.heads[1];
  const bool big = many(tokens, heads, D);
  p.chunks = big ? (heads + 3) / 4 : heads;
  p.items = static_cast<unsigned>(tokens * p.chunks);
  const unsigned per = 256 / (D / 8);
  const dim3 grid((p.items + per - 1) / per);
  return big ? launch_pdl(fa2_qk_norm_rope_kernel<D, INTER, 4>, grid, dim3(256), 0, st, p)
             : launch_pdl(fa2_qk_norm_rope_kernel<D, INTER, 1>, grid, dim3(256), 0, st, p);
}

template <int D, bool INTER>
int launch_bwd_d(NormProblem p, long long tokens, float* dwq, float* dwk, cudaStream_t st) {
  const int heads = p.heads[0] + p.heads[1];
  const bool big = many(tokens, heads, D);
  p.chunks = big ? (heads + 3) / 4 : heads;
  p.items = static_cast<unsigned>(tokens * p.chunks);
  const unsigned per = 256 / (D / 8);
  unsigned grid = (p.items + per - 1) / per;
  if (grid > kBwdCtas) grid = kBwdCtas;
  int e = big ? launch_pdl(fa2_qk_norm_rope_bwd_kernel<D, INTER, 4>, dim3(grid), dim3(256), 0, st, p)
              : launch_pdl(fa2_qk_norm_rope_bwd_kernel<D, INTER, 1>, dim3(grid), dim3(256), 0, st, p);
  if (e || !p.partial) return e;
  return launch_pdl(fa2_qk_norm_dw_kernel, dim3((2 * D + 31) / 32), dim3(256), 0, st,
                    static_cast<const float*>(p.partial), static_cast<int>(grid), D, dwq, dwk);
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
  if (!aligned(a.q_weight, a.weight_fp32 ? 4 : 2) || !aligned(a.k_weight, a.weight_fp32 ? 4 : 2)) return FA2_ERR_ALIGN;
  if (tokens == 0) return FA2_OK;
  for (int i = 0; i < count; ++i) {
    if (!t[i].p) return FA2_ERR_NULL;
    t[i].heads = i % 2 ? a.H_kv : a.H;
    const long long size[3] = {a.B, t[i].heads, a.N};
    const long long own[3] = {static_cast<long long>(t[i].heads) * a.N * a.d, static_cast<long long>(a.N) * a.d, a.d};
    for (int j = 0; j < 3; ++j) {
      t[i].s[j] = size[j] == 1 ? own[j] : (strides ? strides[3 * i + j] : own[j]);
      if (t[i].s[j] < 0 || t[i].s[j] > (1LL << 40)) return FA2_ERR_SHAPE;
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
  return head_dim_ok(d) ? static_cast<size_t>(kBwdCtas) * 2 * d * sizeof(float) : 0;
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
