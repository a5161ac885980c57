// The page plan of one step over a paged key-value cache, made on the GPU
// from the requests' lengths: which pages each request's new tokens need
// (taken from a list of free pages in request order), every new token's slot
// and position, and the offsets of the packed batch.  The host needs none of
// the lengths, so the step can be captured in a graph and replayed.
//
// With c_b tokens of request b in the cache, n_b new ones and pages of P
// tokens, request b takes f_b = ceil((c_b + n_b) / P) - ceil(c_b / P) pages;
// its first is number sum_{a < b} f_a of the free list, and its token at
// position x has slot table[b][x / P] * P + x mod P.
//
// Bound by latency (a few hundred bytes to a few MB of integers), so it is
// one launch: every CTA makes the prefix sums over the requests for itself in
// shared memory (two reads of B integers, which L2 serves) instead of waiting
// for another's, and then writes its share of the tokens and table entries,
// finding each one's request by bisection.  A new token's page comes from the
// free list directly, never from the table entry another CTA writes.
// Measured on a GB300 (device time): 64 requests with one new token each 2.9
// us, 333 requests with 132 thousand new tokens 4.9 us.
#include <cuda_runtime.h>

#include <atomic>
#include <climits>

#include "args.h"
#include "fa2.h"
#include "launch.h"
#include "ptx.cuh"

namespace fa2 {
namespace {

__device__ int g_plan_status;
std::atomic<bool> g_launched{false};  // some call of this process has: the word may be set

constexpr int kThreads = 512;
// From here on a thread's lengths no longer stay in L1 between its reads: 4000
// requests 11.5 us read directly, 11.8 staged, 16000 87 and 33.
constexpr int kStagedRequests = 4096;
constexpr int kMaxRequests = 16384;  // two 4-byte prefix sums each in shared memory

struct PlanProblem {
  const int* cached;
  const int* fresh;
  const int* free_pages;
  int* table;
  int* lens;
  int* cu_new;
  int* cu_total;
  long long* slots;
  int* positions;
  int* pages_needed;
  long long table_stride;
  int B, num_free, width, shift, max_tokens;
};

// Tokens in the cache and new ones of request b; a request that is not
// possible (a negative length, more tokens than its table row has room for)
// counts as empty.
__device__ __forceinline__ bool check(const PlanProblem& p, int& c, int& n) {
  const long long room = static_cast<long long>(p.width) << p.shift;
  if (c >= 0 && n >= 0 && static_cast<long long>(c) + n <= room) return true;
  c = n = 0;
  return false;
}
__device__ __forceinline__ bool request(const PlanProblem& p, int b, int& c, int& n) {
  c = __ldg(p.cached + b);
  n = __ldg(p.fresh + b);
  return check(p, c, n);
}

__device__ __forceinline__ int pages(int n, int shift) {
  return static_cast<int>((static_cast<long long>(n) + (1 << shift) - 1) >> shift);
}

__device__ __forceinline__ long long warp_scan(long long v, int lane) {
#pragma unroll
  for (int s = 1; s < 32; s <<= 1) {
    const long long o = __shfl_up_sync(0xffffffffu, v, s);
    if (lane >= s) v += o;
  }
  return v;
}

// The last b with first[b] <= x (first[0] = 0 <= x).
__device__ __forceinline__ int find(const int* first, int B, int x) {
  int lo = 0, hi = B;  // first[lo] <= x < first[hi], where first[B] counts as above
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (first[mid] <= x)
      lo = mid;
    else
      hi = mid;
  }
  return lo;
}

template <bool STAGED>
__global__ void __launch_bounds__(kThreads) fa2_page_plan_kernel(const PlanProblem p) {
  extern __shared__ int sm[];
  int* const s_tok = sm;               // [B + 1] new tokens before request b
  int* const s_page = sm + p.B + 1;    // [B + 1] new pages before request b
  __shared__ long long part[3][kThreads / 32];
  griddep_wait();
  griddep_launch_dependents();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  // Each thread adds up `per` consecutive requests; STAGED: the lengths are
  // first read in order to where their prefix sums will be.
  if constexpr (STAGED) {
#pragma unroll 4
    for (int b = tid; b < p.B; b += kThreads) {
      s_tok[b] = __ldg(p.cached + b);
      s_page[b] = __ldg(p.fresh + b);
    }
    __syncthreads();
  }
  auto lengths = [&](int b, int& c, int& n) {
    if (!STAGED) return request(p, b, c, n);
    c = s_tok[b];
    n = s_page[b];
    return check(p, c, n);
  };
  const int per = ((p.B + kThreads - 1) / kThreads) | (STAGED ? 1 : 0);  // (odd: no bank conflicts)
  const int b0 = min(tid * per, p.B), b1 = min(b0 + per, p.B);
  long long sum[3] = {0, 0, 0};  // new tokens, new pages, all tokens
  bool fine = true;
  for (int b = b0; b < b1; ++b) {
    int c, n;
    fine &= lengths(b, c, n);
    sum[0] += n;
    sum[1] += pages(c + n, p.shift) - pages(c, p.shift);
    sum[2] += static_cast<long long>(c) + n;
  }
  long long run[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    run[i] = warp_scan(sum[i], lane);
    if (lane == 31) part[i][warp] = run[i];
    run[i] -= sum[i];
  }
  __syncthreads();
  long long total[3];
#pragma unroll
  for (int i = 0; i < 3; ++i) {
    long long before = 0, all = 0;
#pragma unroll
    for (int w = 0; w < kThreads / 32; ++w) {
      if (w < warp) before += part[i][w];
      all += part[i][w];
    }
    run[i] += before;
    total[i] = all;
  }
  // More tokens than 32-bit offsets count: every request is left out.
  const bool overflow = total[2] > INT_MAX;
  if (overflow) {
    fine = false;
#pragma unroll
    for (int i = 0; i < 3; ++i) run[i] = total[i] = 0;
  }
  const bool first_cta = blockIdx.x == 0;
  if (first_cta && (!fine || total[0] > p.max_tokens)) atomicCAS(&g_plan_status, kDevOk, kDevBadSeqlens);
  for (int b = b0; b < b1; ++b) {
    int c, n;
    lengths(b, c, n);
    if (overflow) c = n = 0;
    s_tok[b] = static_cast<int>(run[0]);
    s_page[b] = static_cast<int>(run[1]);
    if (first_cta) {
      p.lens[b] = c + n;
      p.cu_new[b] = static_cast<int>(run[0]);
      p.cu_total[b] = static_cast<int>(run[2]);
    }
    run[0] += n;
    run[1] += pages(c + n, p.shift) - pages(c, p.shift);
    run[2] += static_cast<long long>(c) + n;
  }
  if (tid == 0) {
    s_tok[p.B] = static_cast<int>(total[0]);
    s_page[p.B] = static_cast<int>(total[1]);
    if (first_cta) {
      p.cu_new[p.B] = static_cast<int>(total[0]);
      p.cu_total[p.B] = static_cast<int>(total[2]);
      *p.pages_needed = static_cast<int>(total[1]);
    }
  }
  __syncthreads();
  const int step = gridDim.x * kThreads, at = blockIdx.x * kThreads + tid;
  const int n_tok = static_cast<int>(total[0]), n_page = static_cast<int>(total[1]);
  for (long long i = at; i < n_page; i += step) {
    const int e = static_cast<int>(i), b = find(s_page, p.B, e);
    int c, n;
    request(p, b, c, n);
    p.table[b * p.table_stride + pages(c, p.shift) + (e - s_page[b])] = e < p.num_free ? __ldg(p.free_pages + e) : -1;
  }
  for (long long i = at; i < p.max_tokens; i += step) {
    const int t = static_cast<int>(i);
    long long slot = -1;
    int pos = 0;
    if (t < n_tok) {
      const int b = find(s_tok, p.B, t);
      int c, n;
      request(p, b, c, n);
      pos = c + (t - s_tok[b]);
      const int pg = pos >> p.shift, have = pages(c, p.shift);
      int id;
      if (pg < have) {
        id = p.table[b * p.table_stride + pg];  // an entry that was there before: nobody writes it
      } else {
        const int e = s_page[b] + (pg - have);
        id = e < p.num_free ? __ldg(p.free_pages + e) : -1;
      }
      if (id >= 0) slot = (static_cast<long long>(id) << p.shift) + (pos & ((1 << p.shift) - 1));
    }
    p.slots[i] = slot;
    p.positions[i] = pos;
  }
}

}  // namespace

int read_plan_status(int* value, bool reset) {
  if (!g_launched.load()) {
    *value = 0;
    return 0;
  }
  if (cudaError_t e = cudaMemcpyFromSymbol(value, g_plan_status, sizeof(int))) return static_cast<int>(e);
  if (reset) {
    const int zero = 0;
    if (cudaError_t e = cudaMemcpyToSymbol(g_plan_status, &zero, sizeof(int))) return static_cast<int>(e);
  }
  return 0;
}

}  // namespace fa2

using namespace fa2;

extern "C" int fa2_page_plan(const int* cached_lens, const int* new_lens, const int* free_pages, int* block_table,
                             int* lens, int* cu_new, int* cu_total, long long* slots, int* positions,
                             int* pages_needed, int B, int num_free, int table_width, long long table_stride,
                             int page_size, int max_tokens, void* stream) {
  if (B < 1 || B > kMaxRequests || num_free < 0 || table_width < 1 || max_tokens < 0) return FA2_ERR_SHAPE;
  if (B > 1 && (table_stride < table_width || !stride_ok(table_stride, B))) return FA2_ERR_SHAPE;
  if (page_size != 16 && page_size != 32 && page_size != 64 && page_size != 128) return FA2_ERR_SHAPE;
  if (!cached_lens || !new_lens || !block_table || !lens || !cu_new || !cu_total || !pages_needed) return FA2_ERR_NULL;
  if ((num_free > 0 && !free_pages) || (max_tokens > 0 && (!slots || !positions))) return FA2_ERR_NULL;
  const void* words[] = {cached_lens, new_lens, free_pages, block_table, lens, cu_new, cu_total, positions, pages_needed};
  for (const void* w : words)
    if (!aligned(w, 4)) return FA2_ERR_ALIGN;
  if (!aligned(slots, 8)) return FA2_ERR_ALIGN;
  const size_t bb = static_cast<size_t>(B) * 4;
  const size_t tb = (static_cast<size_t>(B - 1) * (B > 1 ? table_stride : 0) + table_width) * 4;
  const Range ins[] = {range_of(cached_lens, bb), range_of(new_lens, bb), range_of(free_pages, static_cast<size_t>(num_free) * 4)};
  const Range outs[] = {range_of(block_table, tb), range_of(lens, bb), range_of(cu_new, bb + 4), range_of(cu_total, bb + 4),
                        range_of(slots, static_cast<size_t>(max_tokens) * 8), range_of(positions, static_cast<size_t>(max_tokens) * 4),
                        range_of(pages_needed, 4)};
  for (int i = 0; i < 7; ++i) {
    for (const Range& r : ins)
      if (overlap(outs[i], r)) return FA2_ERR_ALIAS;
    for (int j = i + 1; j < 7; ++j)
      if (overlap(outs[i], outs[j])) return FA2_ERR_ALIAS;
  }
  PlanProblem p{cached_lens, new_lens, free_pages, block_table, lens, cu_new, cu_total, slots, positions, pages_needed,
                table_stride, B, num_free, table_width, 0, max_tokens};
  while ((1 << p.shift) < page_size) ++p.shift;
  const size_t smem = (static_cast<size_t>(B) + 1) * 8;
  const auto kernel = B > kStagedRequests ? fa2_page_plan_kernel<true> : fa2_page_plan_kernel<false>;
  if (smem > 48 * 1024)
    if (int e = ensure_max_smem(reinterpret_cast<const void*>(kernel), (kMaxRequests + 1) * 8))
      return record_cuda_failure(e, "page plan shared memory");
  // One token per thread, at most one CTA per SM (measured with 2048 / 1024 /
  // 512 tokens a CTA: 333 requests with 143220 new tokens 6.3 / 5.3 / 5.0 us,
  // 113 with 8439 5.9 / 4.8 / 3.9; with two CTAs per SM 5.2 / 3.9).
  long long grid = (static_cast<long long>(max_tokens) + kThreads - 1) / kThreads;
  grid = grid < 1 ? 1 : (grid > 152 ? 152 : grid);
  g_launched = true;
  if (int e = launch_pdl(kernel, dim3(static_cast<unsigned>(grid)), dim3(kThreads), smem,
                         static_cast<cudaStream_t>(stream), p))
    return record_cuda_failure(e, "page plan launch");
  return FA2_OK;
}
