// ssv_page_plan: page table, free stack, sequence table and slot map of a
// pass from the lengths of its requests.
//
// Everything follows from four exclusive sums over the requests: rows N + 2B
// (q_off), slots B (tau_off), pages released and pages wanted.  Page i of
// those wanted (in request, page order) is stack entry A - 1 - i, where the
// stack is the old free list with the released pages on top and A its
// height; a request is granted iff its last wanted page is still on the
// stack, which one comparison of the inclusive sum with A decides.
//
// One launch, no communication between CTAs: every CTA forms the sums itself
// (at most 4096 requests: eight per thread) into shared memory and then fills
// its share of the outputs, finding a row's request by binary search there.
// That is possible because nothing read is written: table entries are read
// below held[] and written from it on, the free list is read below n_free and
// written from it on, and the counters are written to arrays of their own.
// Bound by latency (two dependent rounds of loads around the sums): 5.0 us for 8
// requests, 12.8 us for 1000 of which half are admitted (2.3 MB).
#include "ssv_internal.cuh"
#include "paged.cuh"

#include <atomic>

namespace ssv {
namespace {

constexpr int kPlanThreads = 512;
constexpr int kPlanMaxBatch = 4096;
constexpr int kPlanPer = kPlanMaxBatch / kPlanThreads;  // requests per thread
constexpr int kPlanRows = 2048;                         // rows of the slot map per CTA before a further CTA is launched

struct PlanParams {
  const int32_t *cache_len, *new_len, *block, *held;
  int32_t *pages, *free_list;
  const int32_t* n_free;
  ssv_seq* seqs;
  int32_t *slot_map, *slot_off, *held_out, *n_free_out, *dev_status;
  int batch, max_pages, ps_log2, n_pages, total_rows;
};

// Exclusive sums of (a, b) over the CTA's threads, and the totals.
__device__ __forceinline__ void block_scan2(long long& a, long long& b, long long& ta, long long& tb,
                                            long long (*s)[2]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  long long ia = a, ib = b;
#pragma unroll
  for (int o = 1; o < 32; o <<= 1) {
    const long long xa = __shfl_up_sync(0xffffffffu, ia, o), xb = __shfl_up_sync(0xffffffffu, ib, o);
    if (lane >= o) { ia += xa; ib += xb; }
  }
  __syncthreads();  // s may still be read from an earlier scan
  if (lane == 31) { s[warp][0] = ia; s[warp][1] = ib; }
  __syncthreads();
  long long ca = 0, cb = 0;
  ta = tb = 0;
#pragma unroll
  for (int w = 0; w < kPlanThreads / 32; ++w) {
    if (w < warp) { ca += s[w][0]; cb += s[w][1]; }
    ta += s[w][0];
    tb += s[w][1];
  }
  a = ca + ia - a;
  b = cb + ib - b;
}

// last index b in [0, n) with x[b] <= v (x[0] <= v)
__device__ __forceinline__ int last_le(const int* x, int n, int v) {
  int lo = 0, hi = n - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (x[mid] <= v) lo = mid; else hi = mid - 1;
  }
  return lo;
}

__global__ void __launch_bounds__(kPlanThreads) page_plan_kernel(const PlanParams p) {
  extern __shared__ int s_tab[];  // six tables of `batch` ints
  __shared__ long long s_scan[kPlanThreads / 32][2];
  const int n = p.batch;
  int* s_q = s_tab;          // first row
  int* s_w = s_q + n;        // pages wanted before
  int* s_r = s_w + n;        // pages released before
  int* s_c = s_r + n;        // C
  int* s_nb = s_c + n;       // N + B of a granted request, else 0
  int* s_held = s_nb + n;
  pdl_wait();  // lengths may come from the kernel before this one
  pdl_trigger();
  const bool first = blockIdx.x == 0;
  const int per = (n + kPlanThreads - 1) / kPlanThreads, b0 = threadIdx.x * per;
  int n_free = p.n_free[0];
  if (n_free < 0 || n_free > p.n_pages) {
    if (first && threadIdx.x == 0) report(p.dev_status, SSV_ERR_INVALID);
    n_free = 0;
  }
  // ---- the requests: rows and slots first (whether its rows fit decides what a request may want)
  int C[kPlanPer], N[kPlanPer], B[kPlanPer], H[kPlanPer], want[kPlanPer], rel[kPlanPer];
  bool ok[kPlanPer];
  long long rows = 0, slots = 0, tr, ts;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    C[k] = N[k] = B[k] = H[k] = want[k] = rel[k] = 0;
    ok[k] = false;
    if (k >= per || b >= n) continue;
    C[k] = p.cache_len[b]; N[k] = p.new_len[b]; B[k] = p.block[b]; H[k] = p.held[b];
    const bool held_ok = H[k] >= 0 && H[k] <= p.max_pages;
    if (C[k] < 0) {
      if (held_ok) rel[k] = H[k];
      else if (first) report(p.dev_status, SSV_ERR_INVALID);
      N[k] = B[k] = 0;
      continue;
    }
    const long long len = (long long)C[k] + N[k] + B[k], need = (len + (1 << p.ps_log2) - 1) >> p.ps_log2;
    ok[k] = held_ok && N[k] >= 0 && B[k] >= 1 && B[k] <= 64 && len <= 0x7fffffffLL && need <= p.max_pages;
    if (!ok[k]) {
      if (first) report(p.dev_status, SSV_ERR_INVALID);
      N[k] = B[k] = 0;
      continue;
    }
    want[k] = max((int)need - H[k], 0);
    rows += (long long)N[k] + 2 * B[k];
    slots += B[k];
  }
  block_scan2(rows, slots, tr, ts, s_scan);
  long long w = 0, r = 0, tw, trel;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    if (k >= per || b >= n) continue;
    s_q[b] = (int)min(rows, 0x7fffffffLL);
    if (first) p.slot_off[b] = (int)min(slots, 0x7fffffffLL);
    if (first) p.seqs[b].tau_off = (int)min(slots, 0x7fffffffLL);
    rows += (long long)N[k] + 2 * B[k];
    slots += B[k];
    if (ok[k] && rows > p.total_rows) {
      ok[k] = false;
      want[k] = 0;
      if (first) report(p.dev_status, SSV_ERR_INVALID);
    }
    w += want[k];
    r += rel[k];
  }
  block_scan2(w, r, tw, trel, s_scan);
  long long height = n_free + trel;
  if (height > p.n_pages) {
    if (first && threadIdx.x == 0) report(p.dev_status, SSV_ERR_INVALID);
    height = p.n_pages;
  }
  const int A = (int)height;
  int taken = 0;
#pragma unroll
  for (int k = 0; k < kPlanPer; ++k) {
    const int b = b0 + k;
    if (k >= per || b >= n) continue;
    s_w[b] = (int)min(w, 0x7fffffffLL);
    s_r[b] = (int)min(r, 0x7fffffffLL);
    s_c[b] = C[k];
    s_held[b] = H[k];
    w += want[k];
    r += rel[k];
    const bool granted = ok[k] && (want[k] == 0 || w <= A);
    if (granted && want[k] > 0) taken = (int)w;
    s_nb[b] = granted ? N[k] + B[k] : 0;
    if (first) {
      if (ok[k] && !granted) report(p.dev_status, SSV_ERR_NO_PAGES);
      ssv_seq& o = p.seqs[b];
      o.cache_len = granted ? C[k] : 0;
      o.new_len = granted ? N[k] : 0;
      o.block = granted ? B[k] : 0;
      o.q_off = s_q[b];
      o.kv_off = b * p.max_pages;
      p.held_out[b] = C[k] < 0 && H[k] == rel[k] ? 0 : (granted ? H[k] + want[k] : H[k]);
    }
  }
  // pages taken: the inclusive sum at the last granted request that wants any
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) taken = max(taken, __shfl_xor_sync(0xffffffffu, taken, o));
  __syncthreads();
  if ((threadIdx.x & 31) == 0) s_scan[threadIdx.x >> 5][0] = taken;
  __syncthreads();
#pragma unroll
  for (int i = 0; i < kPlanThreads / 32; ++i) taken = max(taken, (int)s_scan[i][0]);
  if (first && threadIdx.x == 0) p.n_free_out[0] = A - taken;

  // entry i < A of the stack
  auto stack = [&](int i) -> int {
    if (i < n_free) return p.free_list[i];
    const int b = last_le(s_r, n, i - n_free);
    return p.pages[(size_t)b * p.max_pages + (i - n_free - s_r[b])];
  };
  const int tid = blockIdx.x * kPlanThreads + threadIdx.x, step = gridDim.x * kPlanThreads;
  for (int i = tid; i < taken; i += step) {
    const int b = last_le(s_w, n, i);
    p.pages[(size_t)b * p.max_pages + s_held[b] + (i - s_w[b])] = stack(A - 1 - i);
  }
  for (int i = n_free + tid; i < A - taken; i += step) p.free_list[i] = stack(i);
  // the slot map: one row per thread while that covers it, else four per thread and step (one search, then along
  // the requests), so that their loads are in flight together.  Rows are unsigned: the step behind the last of 2^31 - 1
  // stays in range.
  const int mask = (1 << p.ps_log2) - 1, per_row = p.total_rows > step ? 4 : 1;
  const uint32_t total = p.total_rows;
  for (uint32_t row = per_row * tid; row < total; row += per_row * step) {
    int b = last_le(s_q, n, row), slot[4];
#pragma unroll
    for (int k = 0; k < 4; ++k) {
      if (k >= per_row || row + k >= total) break;
      const int r = row + k;
      while (b + 1 < n && s_q[b + 1] <= r) ++b;
      const int j = r - s_q[b];
      slot[k] = -1;
      if (j < s_nb[b]) {
        const int t = s_c[b] + j, idx = t >> p.ps_log2;
        const int page = idx < s_held[b] ? p.pages[(size_t)b * p.max_pages + idx]
                                         : stack(A - 1 - (s_w[b] + idx - s_held[b]));
        slot[k] = (page << p.ps_log2) + (t & mask);
      }
    }
#pragma unroll
    for (int k = 0; k < 4; ++k)
      if (k < per_row && row + k < total) p.slot_map[row + k] = slot[k];
  }
}

bool any_overlap(const void* a, size_t an, const void* b, size_t bn) {
  const uintptr_t x = (uintptr_t)a, y = (uintptr_t)b;
  return an > 0 && bn > 0 && x < y + bn && y < x + an;
}

}  // namespace
}  // namespace ssv

extern "C" ssv_status ssv_page_plan(const ssv_page_plan_args* a, void* stream) {
  using namespace ssv;
  if (!a) return SSV_ERR_INVALID;
  if (a->batch < 0 || a->max_pages < 0 || a->n_pages < 0 || a->total_rows < 0 || !page_size_ok(a->page_size))
    return SSV_ERR_INVALID;
  if ((long long)a->n_pages * a->page_size > 0x7fffffffLL || (long long)a->batch * a->max_pages > 0x7fffffffLL)
    return SSV_ERR_INVALID;
  if (a->batch > kPlanMaxBatch) return SSV_ERR_UNSUPPORTED;
  if (a->batch == 0) return SSV_OK;
  if (!a->cache_len || !a->new_len || !a->block || !a->held || !a->n_free || !a->seqs || !a->slot_off ||
      !a->held_out || !a->n_free_out || (a->max_pages > 0 && !a->pages) || (a->n_pages > 0 && !a->free_list) ||
      (a->total_rows > 0 && !a->slot_map))
    return SSV_ERR_INVALID;
  // no output may overlap an input or another output (every CTA reads the inputs while others write)
  const size_t bb = sizeof(int32_t) * (size_t)a->batch;
  const void* r[] = {a->cache_len, a->new_len, a->block, a->held, a->n_free, a->pages, a->free_list,
                     a->seqs, a->slot_map, a->slot_off, a->held_out, a->n_free_out};
  const size_t rn[] = {bb, bb, bb, bb, 4, 4 * (size_t)a->batch * a->max_pages, 4 * (size_t)a->n_pages,
                       sizeof(ssv_seq) * (size_t)a->batch, 4 * (size_t)a->total_rows, bb, bb, 4};
  for (int o = 5; o < 12; ++o)
    for (int i = 0; i < o; ++i)
      if (any_overlap(r[i], rn[i], r[o], rn[o])) return SSV_ERR_INVALID;
  PlanParams p{a->cache_len, a->new_len, a->block, a->held, a->pages, a->free_list, a->n_free, a->seqs,
               a->slot_map, a->slot_off, a->held_out, a->n_free_out, a->dev_status, a->batch, a->max_pages,
               ilog2(a->page_size), a->n_pages, a->total_rows};
  const size_t smem = sizeof(int) * 6 * (size_t)a->batch;
  static std::atomic<unsigned long long> ready{0};  // bit per device
  int dev = 0;
  SSV_CUDA_CHECK(cudaGetDevice(&dev));
  if (dev >= 64 || !(ready.load() >> dev & 1)) {
    SSV_CUDA_CHECK(cudaFuncSetAttribute(page_plan_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                        (int)(sizeof(int) * 6 * kPlanMaxBatch)));
    if (dev < 64) ready |= 1ull << dev;
  }
  const int grid = min(152, max(1, a->total_rows / kPlanRows + (a->total_rows % kPlanRows > 0)));
  const cudaError_t e =
      launch_pdl(page_plan_kernel, dim3(grid), dim3(kPlanThreads), smem, static_cast<cudaStream_t>(stream), p);
  return e == cudaSuccess ? SSV_OK : SSV_ERR_CUDA;
}
