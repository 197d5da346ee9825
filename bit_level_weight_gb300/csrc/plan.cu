// plan.cu - block tables and slot maps of a serving step, made on the device
// from the lengths of the requests (cas_paged_plan in cas.h states the rules).
//
// Three prefix sums over the sequences decide everything: pages that go back,
// pages that are wanted, rows. What goes back is on the stack before anything is
// taken, so the first is summed over the whole batch before the others begin.
//
// What bounds it: the launches, in a launch the chain of dependent loads
// (lengths, tables, stack) of a few hundred ns each, and the sums: a CTA of 1024 threads
// adds up five numbers of 64 bits over itself, also for one request, which makes most of
// the 30 000 instructions of its warps and keeps 48 % of its SM's issue slots busy
// (44 bytes a thread are spilled). Its bytes are a few KB (one request 9.4 us, 61 with drafts
// 10.7, 1021 with 34000 rows and 5000 pages that move 17.0, less than the call takes on the
// host).
//   plan_seq_kernel   one CTA: the sums, the pages that go back, kv_len, row_start
//   plan_rows_kernel  pages taken and the rows' places, over the grid
// A step of few rows does the second part in the first kernel's CTA.
#include <cuda_runtime.h>

#include <algorithm>

#include "common.cuh"

namespace cas {
namespace {

constexpr int kThreads = 1024;      // sequences a round of the scans
constexpr int kRowThreads = 256;
constexpr int kRowsOfOneCta = 2048;  // rows up to which one CTA does all

// What the second part needs of a sequence: pages behind the kept tokens', pages
// taken by the ones before it, pages it takes.
struct SeqPlan {
  int hold, before, want, kept;
};
struct PlanArgs {
  int32_t *pages, *kv_len, *free_pages, *n_free;
  const int32_t *keep, *add;
  int32_t *row_start, *granted, *pos;
  int64_t* slot;
  SeqPlan* seq;  // workspace: [batch], then the stack's height before pages are taken
  int* height;
  int batch, max_pages, shift, n_pages, rows;
};

// Inclusive sums over the CTA (kThreads threads), and their total.
__device__ __forceinline__ int64_t cta_sum(int64_t v, int64_t* sm, int64_t& total) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int d = 1; d < 32; d <<= 1) {
    const int64_t u = __shfl_up_sync(CAS_FULL, v, d);
    if (lane >= d) v += u;
  }
  __syncthreads();
  if (lane == 31) sm[warp] = v;
  __syncthreads();
  int64_t before = 0;
  total = 0;
#pragma unroll
  for (int i = 0; i < kThreads / 32; ++i) {
    if (i < warp) before += sm[i];
    total += sm[i];
  }
  return v + before;
}

struct Want {
  int held, kept, add, hold, freed, want;
  bool fits;
};
__device__ __forceinline__ Want want_of(const PlanArgs& a, int b) {
  Want w;
  const int cap = a.max_pages << a.shift, up = (1 << a.shift) - 1;
  w.held = min(max(a.kv_len[b], 0), cap);
  w.kept = a.keep ? min(max(a.keep[b], 0), w.held) : w.held;
  const int add = max(a.add[b], 0);
  w.fits = add <= cap - w.kept;
  w.add = w.fits ? add : 0;
  // (lengths up to 2^31 - 1: rounding up may not add to them)
  auto pages = [&](int n) { return (n >> a.shift) + ((n & up) != 0); };
  w.hold = pages(w.kept);
  w.freed = pages(w.held) - w.hold;
  w.want = pages(w.kept + w.add) - w.hold;
  return w;
}

// The sequence of row r, or of the r-th page taken: the last whose rows (pages) start at or before it.
template <class F>
__device__ __forceinline__ int last_at(int n, int64_t r, F start) {
  int lo = 0, hi = n;  // start(lo) <= r
  while (hi - lo > 1) {
    const int mid = (lo + hi) >> 1;
    if (start(mid) <= r) lo = mid; else hi = mid;
  }
  return lo;
}

// Pages taken and rows, by the threads i of n.
__device__ void plan_rows(const PlanArgs& a, int64_t i0, int64_t n, int used, int height) {
  const int mask = (1 << a.shift) - 1;
  auto from_stack = [&](int64_t k) {  // the k-th page taken
    const int64_t at = height - 1 - k;
    return at >= 0 ? a.free_pages[at] : 0;  // (the sums keep k below the height)
  };
  const int rows = a.pos || a.slot ? a.rows : used;  // (else those behind them are nowhere written)
  for (int64_t r = i0; r < rows; r += n) {
    int pos = -1;
    int64_t slot = -1;
    if (r < used) {
      const int b = last_at(a.batch, r, [&](int k) { return a.row_start[k]; });
      const SeqPlan s = a.seq[b];
      pos = s.kept + (int)(r - a.row_start[b]);
      const int p = pos >> a.shift;
      // a new page's id comes from the stack, and its first token's row writes the table (new pages
      // begin behind the kept tokens, so each has that row)
      int id;
      if (p < s.hold) {
        id = a.pages[(int64_t)b * a.max_pages + p];
      } else {
        id = from_stack((int64_t)s.before + p - s.hold);
        if ((pos & mask) == 0) a.pages[(int64_t)b * a.max_pages + p] = id;
      }
      slot = ((int64_t)id << a.shift) + (pos & mask);
    }
    if (a.pos) a.pos[r] = pos;
    if (a.slot) a.slot[r] = slot;
  }
}

__global__ void __launch_bounds__(kThreads) plan_seq_kernel(const __grid_constant__ PlanArgs a, bool rows_too) {
  __shared__ int64_t sm[kThreads / 32];
  __shared__ int starts[kThreads], firsts[kThreads];
  pdl_wait();
  pdl_trigger();
  const int t = threadIdx.x;
  const int n_free = min(max(*a.n_free, 0), a.n_pages);
  // ---- pages that go back
  int64_t back = 0, total;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + t, here = min(kThreads, a.batch - b0);
    Want w{};
    if (b < a.batch) w = want_of(a, b);
    const int64_t incl = cta_sum(w.freed, sm, total);
    if (total > 0) {
      starts[t] = (int)min(incl - w.freed, (int64_t)0x7FFFFFFF);  // (what lies behind the stack's end is dropped)
      firsts[t] = w.hold;
      __syncthreads();
      for (int64_t i = t; i < total; i += kThreads) {
        const int64_t at = n_free + back + i;
        if (at >= a.n_pages) break;
        const int k = last_at(here, i, [&](int j) { return starts[j]; });
        a.free_pages[at] = a.pages[(int64_t)(b0 + k) * a.max_pages + firsts[k] + (i - starts[k])];
      }
      __syncthreads();
    }
    back += total;
  }
  const int height = (int)min(n_free + back, (int64_t)a.n_pages);
  // ---- who is granted what
  int64_t wants = 0, asked = 0, rows = 0, taken = 0;
  for (int b0 = 0; b0 < a.batch; b0 += kThreads) {
    const int b = b0 + t;
    Want w{};
    if (b < a.batch) w = want_of(a, b);
    const int64_t pages = wants + cta_sum(w.want, sm, total);
    wants += total;
    const int64_t upto = asked + cta_sum(w.add, sm, total);
    asked += total;
    const bool ok = w.fits && (w.want == 0 || pages <= height) && upto <= a.rows;
    const int add = ok ? w.add : 0, want = ok ? w.want : 0;
    const int64_t end = rows + cta_sum(add, sm, total);
    rows += total;
    taken += want;
    if (b < a.batch) {
      a.seq[b] = SeqPlan{w.hold, (int)min(pages - w.want, (int64_t)0x7FFFFFFF), want, w.kept};
      a.kv_len[b] = w.kept + add;
      a.row_start[b] = (int)(end - add);
      if (a.granted) a.granted[b] = add;
    }
  }
  cta_sum(taken, sm, total);
  if (t == 0) {
    a.row_start[a.batch] = (int)rows;
    *a.n_free = height - (int)total;
    *a.height = height;
  }
  if (rows_too) {
    __syncthreads();
    plan_rows(a, t, kThreads, (int)rows, height);
  }
}

__global__ void __launch_bounds__(kRowThreads) plan_rows_kernel(const __grid_constant__ PlanArgs a) {
  pdl_wait();
  pdl_trigger();
  plan_rows(a, (int64_t)blockIdx.x * kRowThreads + threadIdx.x, (int64_t)gridDim.x * kRowThreads, a.row_start[a.batch],
            *a.height);
}

}  // namespace
}  // namespace cas

using namespace cas;

extern "C" uint64_t cas_paged_plan_workspace_bytes(int batch) {
  return batch < 0 ? 16 : 16 + (uint64_t)batch * sizeof(SeqPlan);
}

extern "C" int cas_paged_plan(const cas_page_pool* pool, const int32_t* keep, const int32_t* add, int rows,
                              int32_t* row_start, int32_t* granted, int32_t* pos, int64_t* slot, void* workspace,
                              uint64_t workspace_bytes, void* stream) {
  if (!pool || rows < 0 || pool->batch < 0 || pool->batch > CAS_MAX_BATCH || pool->max_pages < 1 || pool->n_pages < 1) return CAS_ERR_INVALID;
  const int S = pool->page_size;
  if (S < 8 || S > 1024 || (S & (S - 1)) || (int64_t)pool->max_pages * S > 0x7FFFFFFF) return CAS_ERR_INVALID;
  if (!row_start || !pool->n_free || !pool->free_pages || (pool->batch > 0 && (!pool->pages || !pool->kv_len || !add)))
    return CAS_ERR_INVALID;
  if (!workspace || !aligned16(workspace) || workspace_bytes < cas_paged_plan_workspace_bytes(pool->batch))
    return CAS_ERR_BUFFER;
  PlanArgs a{};
  a.pages = pool->pages, a.kv_len = pool->kv_len, a.free_pages = pool->free_pages, a.n_free = pool->n_free;
  a.keep = keep, a.add = add, a.row_start = row_start, a.granted = granted, a.pos = pos, a.slot = slot;
  a.height = (int*)workspace;
  a.seq = (SeqPlan*)((uint8_t*)workspace + 16);
  a.batch = pool->batch, a.max_pages = pool->max_pages, a.n_pages = pool->n_pages, a.rows = rows;
  while ((1 << a.shift) < S) ++a.shift;
  const cudaStream_t st = (cudaStream_t)stream;
  const bool one = rows <= kRowsOfOneCta;
  if (const int e = launch_k(plan_seq_kernel, 1, kThreads, 0, st, a, one)) return e;
  if (one) return CAS_OK;
  const int blocks = (int)std::min<int64_t>(((int64_t)rows + kRowThreads - 1) / kRowThreads, sm_count() * 8);
  // directly behind our own kernel: its launch may overlap that kernel's tail
  return launch_with(true, plan_rows_kernel, dim3(blocks), kRowThreads, 0, st, a);
}
