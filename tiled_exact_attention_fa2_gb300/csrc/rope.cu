// The rotation of queries and keys by their positions, its gradient, and the
// table of cosines and sines, also for contexts longer than the trained one.
//
// Rotation: out_a = a c - b s, out_b = b c + a s for the pairs of the first rot
// columns; the gradient turns back (s -> -s).  Bound by HBM: 4 bytes an element
// against 3 flops, and the table's rows once.  A lane has both columns of its
// pairs (rope.cuh) and takes several heads of one token, so cosines and sines
// are loaded once for all of them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include <atomic>
#include <cmath>

#include "args.h"
#include "fa2.h"
#include "launch.h"
#include "rope.cuh"
#include "views.h"

namespace fa2 {
namespace {

__device__ int g_rope_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

struct RopeView {  // [B, heads, N, d], strides in bytes
  char* p;
  long long sb, sh, sn;
};

struct RopeProblem {
  RopeView x[2], y[2];  // of q and k
  RopeTable table;
  int heads[2];
  unsigned chunks, chunks_q;  // lane-group items of a token, and those of q
  unsigned tokens;            // B * N
  int N, shift;               // 1 << shift slots a row
};

template <bool INTER, int ROWS>
__global__ void __launch_bounds__(256) fa2_rope_kernel(const RopeProblem p) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned long long id = blockIdx.x * 256ull + threadIdx.x;
  const int slot = static_cast<int>(id) & ((1 << p.shift) - 1);
  const unsigned item = static_cast<unsigned>(id >> p.shift), tok = item / p.chunks, chunk = item - tok * p.chunks;
  if (tok >= p.tokens) return;
  const int which = chunk >= p.chunks_q;
  const int h0 = static_cast<int>(which ? chunk - p.chunks_q : chunk) * ROWS;
  const int count = min(ROWS, p.heads[which] - h0);
  const unsigned b = tok / static_cast<unsigned>(p.N), n = tok - b * p.N;
  const int pos = p.table.positions ? __ldg(p.table.positions + tok) : static_cast<int>(n);
  int first, second;
  slot_columns(p.table, slot, first, second);
  const RopeView &x = p.x[which], &y = p.y[which];
  const char* src = x.p + b * x.sb + n * x.sn + h0 * x.sh;
  uint4 u[ROWS][2];
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < count) {
      u[i][0] = *reinterpret_cast<const uint4*>(src + i * x.sh + 2 * first);
      u[i][1] = *reinterpret_cast<const uint4*>(src + i * x.sh + 2 * second);
    }
  if (pos < 0 || pos >= p.table.max_pos) {
    atomicCAS(&g_rope_status, kDevOk, kDevBadIndex);
    return;
  }
  char* dst = y.p + b * y.sb + n * y.sn + h0 * y.sh;
  const bool turns = slot * 16 < p.table.rot;
  Turn t;
  if (turns) load_turn(t, p.table, slot, pos);
#pragma unroll
  for (int i = 0; i < ROWS; ++i)
    if (i < count) {
      if (turns) {
        float f[8], g[8];
        widen8(f, u[i][0]);
        widen8(g, u[i][1]);
        turn16<INTER>(f, g, t);
        u[i][0] = narrow8(f);
        u[i][1] = narrow8(g);
      }
      *reinterpret_cast<uint4*>(dst + i * y.sh + 2 * first) = u[i][0];
      *reinterpret_cast<uint4*>(dst + i * y.sh + 2 * second) = u[i][1];
    }
}

// ---------------------------------------------------------------- the table
constexpr int kMaxHalf = 64;  // rot <= 128
constexpr int kTableCtas = 6;  // an SM, at most

struct TableProblem {
  float* out;
  unsigned long long turns[kMaxHalf];  // of a position, modulo 1, in 2^-64
  unsigned first;
  int n, half;
  float amplitude;
};

// (cos, sin) of `phase` 2^-64 turns.  The phase is a quadrant and a remainder of
// at most an eighth of a turn, which becomes an fp32 angle x of its first 24 bits
// (exact) and the 32 behind them; then, with z = x^2, sin x = x + x z S(z) and
// cos x = 1 - z / 2 + z^2 C(z), S and C the quadratics that meet the functions in
// the Chebyshev nodes of [0, (pi/4)^2] (off by 2^-26.8 and 2^-30.6 at most).
__device__ __forceinline__ void cos_sin(unsigned long long phase, float& c, float& s) {
  constexpr float kHigh = 6.283185307179586f * 0x1p-26f;                                   // 2 pi 2^-26
  constexpr float kRest = static_cast<float>(6.283185307179586 * 0x1p-26 - static_cast<double>(kHigh));
  const unsigned long long turned = phase + (1ull << 61);
  const unsigned quarter = static_cast<unsigned>(turned >> 62);
  const long long r = static_cast<long long>((turned & ((1ull << 62) - 1)) - (1ull << 61));
  const float high = static_cast<float>(static_cast<int>(r >> 38));
  const float low = static_cast<float>(static_cast<unsigned>(r >> 6));
  const float x = fmaf(high, kHigh, fmaf(high, kRest, low * (kHigh * 0x1p-32f)));
  const float z = x * x;
  const float sn = fmaf(x * z, fmaf(z, fmaf(z, -0.00019587638962548226f, 0.008332747034728527f), -0.166666641831398f), x);
  const float cs = fmaf(z, fmaf(z, fmaf(z, fmaf(z, 2.4547689463361166e-05f, -0.0013888301327824593f), 0.0416666641831398f), -0.5f), 1.f);
  // by quadrants: (c, s), (-s, c), (-c, -s), (s, -c)
  const float u = quarter & 1 ? sn : cs, v = quarter & 1 ? cs : sn;
  c = __uint_as_float(__float_as_uint(u) ^ (((quarter + 1) & 2) << 30));
  s = __uint_as_float(__float_as_uint(v) ^ ((quarter & 2) << 30));
}

// A thread takes four columns of every gridDim.x blockDim.y-th position.  The
// angle p theta_i in turns is an integer product modulo 2^64 of the position and
// the column's 64-bit share of a turn.  That share comes from fp64 (off by about 2^-55
// turns where theta is at most 1); the product adds nothing to p times its error, at any
// position, where fp32 angles lose all digits and fp64 ones would run at a
// hundredth of the rate.  Every second row is the one before it turned by the step
// between them (four products in place of some thirty instructions a column).
// Bound by the writes: 131072 positions x 128 columns 10.3 us (6.5 TB/s, 96 % of a
// copy's rate); 11.8 with the polynomials for every row, 46.8 with conversions of
// 64-bit phases and sincospif, 12.4 with lanes that index the parameters.
__global__ void __launch_bounds__(256) fa2_rope_table_kernel(const __grid_constant__ TableProblem p) {
  griddep_wait();
  griddep_launch_dependents();
  const unsigned i0 = threadIdx.x * 4, step = gridDim.x * blockDim.y;
  unsigned row = blockIdx.x * blockDim.y + threadIdx.y;
  // (through a pointer: lanes that index the parameters directly are served one by one)
  const unsigned long long* from = p.turns + i0;
  asm("" : "+l"(from));
  unsigned long long turns[4];
  float cr[4], sr[4];
#pragma unroll
  for (int i = 0; i < 4; ++i) {
    turns[i] = from[i];
    cos_sin(step * turns[i], cr[i], sr[i]);
  }
  auto write = [&](unsigned r, const float (&c)[4], const float (&s)[4]) {
    float* out = p.out + static_cast<long long>(r) * (2 * p.half) + i0;
    *reinterpret_cast<float4*>(out) = make_float4(c[0], c[1], c[2], c[3]);
    *reinterpret_cast<float4*>(out + p.half) = make_float4(s[0], s[1], s[2], s[3]);
  };
  for (unsigned n = p.n; row < n;) {
    float c[4], s[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      cos_sin((p.first + row) * turns[i], c[i], s[i]);
      c[i] *= p.amplitude;
      s[i] *= p.amplitude;
    }
    write(row, c, s);
    if (n - row <= step) break;
    row += step;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
      const float x = fmaf(c[i], cr[i], -s[i] * sr[i]);
      s[i] = fmaf(s[i], cr[i], c[i] * sr[i]);
      c[i] = x;
    }
    write(row, c, s);
    if (n - row <= step) break;
    row += step;
  }
}

template <bool INTER, int ROWS>
int launch_rope_rows(RopeProblem p, int d, cudaStream_t st) {
  p.chunks_q = (p.heads[0] + ROWS - 1) / ROWS;
  p.chunks = p.chunks_q + (p.heads[1] + ROWS - 1) / ROWS;
  const long long threads = static_cast<long long>(p.tokens) * p.chunks * (d / 16);
  return launch_pdl(fa2_rope_kernel<INTER, ROWS>, dim3(static_cast<unsigned>((threads + 255) / 256)), dim3(256), 0, st, p);
}
// Heads a lane takes: one where the call is small (shorter chains of loads), rows are
// short (a warp's lanes then lie side by side) or there is no other, else two.  Measured, one / two
// / four / eight in us: 48 tokens x 40 heads x 128 columns 1.7 / 1.8 / 2.0 / 2.7, 400
// 3.1 / 2.3 / 2.1 / 2.8, 16000 57.6 / 51.3 / 49.8 / 50.3; 16000 x 5 heads 7.9 / 7.3 / 8.2
// / 9.9; 400 x 40 heads x 64 2.0 / 1.9 / 2.2 / 3.0; 16000 x 40 heads x 16 7.4 / 8.6 /
// 14.3 / 14.9; 13914 x 24 heads x 32 8.0 / 9.3 / 9.6; 92910 x 1 head of q and of k x 128
// 18.0 / 19.6 / 23.9.  Those of 16 and 32 columns are packed rows, whose heads lie side by
// side; the rule does not look at that, and where they do not it takes the slowest: 6 x
// 16384 tokens x 40 heads x 16 as [B, H, N, d] 78.6 / 64.3 / 55.3.
template <bool INTER>
int launch_rope(const RopeProblem& p, int d, cudaStream_t st) {
  const long long elements = static_cast<long long>(p.tokens) * (p.heads[0] + p.heads[1]) * d;
  return d <= 32 || p.heads[0] == 1 || elements < 800000 ? launch_rope_rows<INTER, 1>(p, d, st) : launch_rope_rows<INTER, 2>(p, d, st);
}

// Both directions.
int rope(const void* q, const void* k, const float* table, const int* positions, void* q_out, void* k_out, int B, int H,
         int H_kv, int N, int d, int rot, int inter, int max_pos, const long long* strides, bool back, cudaStream_t st) {
  const int tensors = k || k_out || H_kv != 0 ? 2 : 1;
  if (B < 1 || H < 1 || H_kv < 0 || N < 0) return FA2_ERR_SHAPE;
  if (!head_dim_ok(d)) return FA2_ERR_HEADDIM;
  if (tensors == 2)
    if (int rc = check_heads(H, H_kv)) return rc;
  const long long tokens = static_cast<long long>(B) * N;
  if (rot < 16 || rot > d || rot % 16 != 0 || (inter != 0 && inter != 1) || max_pos < 1) return FA2_ERR_SHAPE;
  if (tokens * (static_cast<long long>(H) + H_kv) > 0x7fffffffLL || (!positions && N > max_pos)) return FA2_ERR_SHAPE;
  if (!table) return FA2_ERR_NULL;
  if (!aligned(table, 16) || !aligned(positions, 4)) return FA2_ERR_ALIGN;
  if (tokens == 0) return FA2_OK;
  const void* const ptr[4] = {q, k, q_out, k_out};
  Strided t[4];
  for (int i = 0; i < 4; ++i) {
    if (i % 2 >= tensors) continue;
    if (!ptr[i]) return FA2_ERR_NULL;
    const long long heads = i % 2 ? H_kv : H, row = d;
    t[i] = Strided{ptr[i], 2, {B, heads, N}, {0, 0, 0}, d};
    if (int rc = check_strides(&t[i], strides ? strides + 3 * i : nullptr, {heads * N * row, N * row, row})) return rc;
  }
  const Range fixed[] = {range_of(table, static_cast<size_t>(max_pos) * rot * 4),
                         range_of(positions, positions ? static_cast<size_t>(tokens) * 4 : 0)};
  for (int i = 2; i < 2 + tensors; ++i) {
    if (!rows_apart(t[i])) return FA2_ERR_ALIAS;
    for (int j = 0; j < i; ++j) {
      if (j % 2 >= tensors) continue;
      // an input may be overwritten row by row by the output of the same rows
      if (j == i - 2 && t[i].p == t[j].p && t[i].stride[0] == t[j].stride[0] && t[i].stride[1] == t[j].stride[1] &&
          t[i].stride[2] == t[j].stride[2])
        continue;
      if (!apart(t[i], t[j], 1)) return FA2_ERR_ALIAS;
    }
    for (const Range& r : fixed)
      if (r.lo != r.hi && overlap(span_of(t[i]), r)) return FA2_ERR_ALIAS;
  }
  RopeProblem p{};
  for (int i = 0; i < tensors; ++i) {
    auto view = [](const Strided& v) {
      return RopeView{static_cast<char*>(const_cast<void*>(v.p)), 2 * v.stride[0], 2 * v.stride[1], 2 * v.stride[2]};
    };
    p.x[i] = view(t[i]);
    p.y[i] = view(t[2 + i]);
    p.heads[i] = i ? H_kv : H;
  }
  p.table = RopeTable{table, positions, rot, max_pos, inter, back};
  p.tokens = static_cast<unsigned>(tokens);
  p.N = N;
  while ((16 << p.shift) < d) ++p.shift;
  g_launched = true;
  const int e = inter ? launch_rope<true>(p, d, st) : launch_rope<false>(p, d, st);
  return e ? record_cuda_failure(e, "rope launch") : FA2_OK;
}

}  // namespace

int read_rope_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_rope_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_rope_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

extern "C" {

int fa2_rope(const void* q, const void* k, const float* rope_table, const int* positions, void* q_out, void* k_out, int B, int H,
             int H_kv, int N, int d, int rot_dim, int interleaved, int max_positions, const long long* strides, void* stream) {
  return rope(q, k, rope_table, positions, q_out, k_out, B, H, H_kv, N, d, rot_dim, interleaved, max_positions, strides, false,
              static_cast<cudaStream_t>(stream));
}

int fa2_rope_bwd(const void* dq_out, const void* dk_out, const float* rope_table, const int* positions, void* dq, void* dk, int B,
                 int H, int H_kv, int N, int d, int rot_dim, int interleaved, int max_positions, const long long* strides,
                 void* stream) {
  return rope(dq_out, dk_out, rope_table, positions, dq, dk, B, H, H_kv, N, d, rot_dim, interleaved, max_positions, strides, true,
              static_cast<cudaStream_t>(stream));
}

int fa2_rope_table(float* rope_table, long long first_position, int num_positions, int rot_dim, double base, double factor,
                   double trained_positions, double low_turns, double high_turns, double amplitude, void* stream) {
  constexpr double kTwoPi = 6.283185307179586476925;
  if (rot_dim < 16 || rot_dim > 2 * kMaxHalf || rot_dim % 16 != 0 || num_positions < 0 || first_position < 0 ||
      first_position > 0x80000000LL - num_positions)
    return FA2_ERR_SHAPE;
  auto positive = [](double x) { return std::isfinite(x) && x > 0; };
  if (!positive(base) || !positive(factor) || !positive(amplitude) || !std::isnormal(static_cast<float>(amplitude))) return FA2_ERR_SCALE;
  if (!(std::isfinite(trained_positions) && trained_positions >= 0)) return FA2_ERR_SCALE;
  if (trained_positions > 0 && !(std::isfinite(low_turns) && std::isfinite(high_turns) && low_turns < high_turns)) return FA2_ERR_SCALE;
  TableProblem p{};
  p.half = rot_dim / 2;
  for (int i = 0; i < p.half; ++i) {
    // (the exponent's own rounding, times the logarithm of the base, would be most of the error of a base far below 1)
    const double exponent = -2.0 * i / rot_dim, rest = std::fma(-exponent, rot_dim, -2.0 * i) / rot_dim;
    double theta = std::pow(base, exponent);
    theta += theta * (rest * std::log(base));
    double keep = 0;
    if (trained_positions > 0)
      keep = std::fmin(1.0, std::fmax(0.0, (trained_positions * theta / kTwoPi - low_turns) / (high_turns - low_turns)));
    const double turns = theta * (keep + (1 - keep) / factor) / kTwoPi;
    if (!(turns < 0x1p52)) return FA2_ERR_SCALE;  // (a base or factor far below 1: no fraction of a turn is left)
    p.turns[i] = static_cast<unsigned long long>(std::ldexp(turns - std::floor(turns), 64));
  }
  if (num_positions == 0) return FA2_OK;
  if (!rope_table) return FA2_ERR_NULL;
  if (!aligned(rope_table, 16)) return FA2_ERR_ALIGN;
  p.out = rope_table;
  p.first = static_cast<unsigned>(first_position);
  p.n = num_positions;
  p.amplitude = static_cast<float>(amplitude);
  const unsigned quads = p.half / 4, rows = 256 / quads;
  const unsigned ctas = static_cast<unsigned>((num_positions - 1LL) / rows + 1), most = 152 * kTableCtas;
  const int e = launch_pdl(fa2_rope_table_kernel, dim3(ctas < most ? ctas : most), dim3(quads, rows), 0,
                           static_cast<cudaStream_t>(stream), p);
  return e ? record_cuda_failure(e, "rope table launch") : FA2_OK;
}

}  // extern "C"
