// A step's plan for the paged key-value cache: sequences are cut back, their
// pages return to the pool, the pages that the new rows miss are handed out, and
// the rows' sequences, slots and positions are written. Defined in include/qmoe.h.
#include <climits>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

constexpr int PL_THREADS = 1024, PL_WARPS = 32, PF_THREADS = 256, PF_ROWS = 1024, PF_MAX_CTAS = 2048;

// What the first kernel leaves for the second: the state of the pool before the
// call, and arrays over the sequences.
struct PlanHead {
  int n_free, back, taken, pad;
};

struct PlanWs {
  PlanHead* head;
  int32_t *first;     // the rows before the sequence
  int32_t *back_end;  // pages that came back up to and with the sequence
  int32_t *need_end;  // pages asked for up to and with it
  int32_t *need;      // pages that it asks for (0: none, or refused for its size)
  int32_t *len;       // entries that it keeps
  int32_t *from;      // first table entry without a page
  int32_t *back;      // [pages] the pages that came back, in order
};

__host__ __device__ inline size_t plan_up(size_t v) { return (v + 255) & ~size_t(255); }

__host__ PlanWs plan_ws(const PagedView& c, void* ws, size_t* total) {
  char* p = static_cast<char*>(ws);
  const size_t seqs = plan_up(sizeof(int32_t) * (size_t)c.n_seqs);
  size_t o = 256;
  PlanWs w{};
  w.head = reinterpret_cast<PlanHead*>(p);
  int32_t** const arrays[] = {&w.first, &w.back_end, &w.need_end, &w.need, &w.len, &w.from};
  for (int32_t** a : arrays) {
    *a = reinterpret_cast<int32_t*>(p + o);
    o += seqs;
  }
  w.back = reinterpret_cast<int32_t*>(p + o);
  o += plan_up(sizeof(int32_t) * (size_t)c.n_pages);
  *total = o;
  return w;
}

__device__ __forceinline__ bool plan_page(const PagedView& c, int page) { return (unsigned)page < (unsigned)c.n_pages; }

// Inclusive sums over the block of three numbers each thread, with 32 words of
// shared memory each; the totals come back in ``total``.
__device__ __forceinline__ void plan_scan(long long (&v)[3], long long (&total)[3], long long (*part)[PL_WARPS]) {
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
  for (int k = 0; k < 3; ++k) {
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long o = __shfl_up_sync(0xffffffffu, v[k], d);
      if (lane >= d) v[k] += o;
    }
    if (lane == 31) part[k][warp] = v[k];
  }
  __syncthreads();
#pragma unroll
  for (int k = 0; k < 3; ++k) {
    long long p = part[k][lane];
#pragma unroll
    for (int d = 1; d < 32; d *= 2) {
      const long long o = __shfl_up_sync(0xffffffffu, p, d);
      if (lane >= d) p += o;
    }
    const long long before = __shfl_sync(0xffffffffu, p, (warp + 31) & 31);
    v[k] += warp > 0 ? before : 0;
    total[k] = __shfl_sync(0xffffffffu, p, 31);
  }
  __syncthreads();
}

__device__ __forceinline__ int plan_int(long long v) { return v > INT_MAX ? INT_MAX : (int)v; }

// The sequence ``b``'s rows are granted: they fit, and its pages are there.
__device__ __forceinline__ bool plan_granted(const PagedView& c, const PlanArgs& a, const PlanWs& w, const PlanHead& h,
                                             int b, int n) {
  return n > 0 && (long long)w.first[b] + n <= a.n_rows && (long long)w.len[b] + n <= paged_slots(c) &&
         (w.need[b] == 0 || w.need_end[b] <= h.n_free + h.back);
}

// One CTA: each sequence's pages that come back and that it misses, and their sums
// over the sequences. A thread has a sequence; runs of pages are walked by its warp.
__device__ __forceinline__ void plan_count(const PagedView& c, const PlanArgs& a, const PlanWs& w) {
  __shared__ long long part[3][PL_WARPS];
  const int tid = threadIdx.x, lane = tid & 31;
  const long long cap = paged_slots(c);
  long long rows0 = 0, back0 = 0, need0 = 0;
  for (int b0 = 0; b0 < c.n_seqs; b0 += PL_THREADS) {
    const int b = b0 + tid;
    const bool mine = b < c.n_seqs;
    int len = 0, n = 0, keep = -1, cut = 0, have = 0, want = 0;
    if (mine) {
      len = paged_len(c, b);
      n = max(a.count[b], 0);
      keep = a.keep ? a.keep[b] : -1;
      if (keep >= 0) {
        len = min(len, keep);
        c.lens[b] = len;
      }
      const long long end = min((long long)len + n, cap);
      cut = (int)((len + (1ll << c.page_log2) - 1) >> c.page_log2);
      want = (int)((end + (1ll << c.page_log2) - 1) >> c.page_log2);
      have = len >> c.page_log2;  // a page that is begun may be missing too
    }
    // how far the sequence's pages go: where they come back all of them, else as far as the rows need
    const int32_t* row = c.table + (long long)(mine ? b : 0) * c.max_pages;
    const int stop = !mine ? 0 : keep >= 0 ? c.max_pages : n > 0 ? want : 0;
    bool open = mine && have < stop && plan_page(c, row[have]);
    if (open) ++have;
    for (unsigned m = __ballot_sync(0xffffffffu, open); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      const int32_t* r = c.table + (long long)(b - lane + src) * c.max_pages;
      int at = __shfl_sync(0xffffffffu, have, src);
      const int to = __shfl_sync(0xffffffffu, stop, src);
      while (at < to) {
        const bool page = at + lane < to && plan_page(c, r[at + lane]);
        const unsigned gone = __ballot_sync(0xffffffffu, !page);
        if (gone) {
          at += __ffs(gone) - 1;
          break;
        }
        at += 32;
      }
      if (lane == src) have = min(at, to);
    }
    const int back = keep >= 0 ? max(have - cut, 0) : 0;
    const int from = keep >= 0 ? min(have, cut) : have;
    long long v[3] = {n, back, 0}, total[3];
    plan_scan(v, total, part);
    const long long first = rows0 + v[0] - n, back_end = back0 + v[1];
    const bool fits = n > 0 && first + n <= a.n_rows && (long long)len + n <= cap;
    const int need = fits ? max(want - from, 0) : 0;
    long long u[3] = {need, 0, 0}, need_total[3];
    plan_scan(u, need_total, part);
    if (mine) {
      w.first[b] = plan_int(first);
      w.back_end[b] = plan_int(back_end);
      w.need_end[b] = plan_int(need0 + u[0]);
      w.need[b] = need;
      w.len[b] = len;
      w.from[b] = from;
      a.first[b] = plan_int(first);
    }
    // the pages that come back, in order, leave the table
    for (unsigned m = __ballot_sync(0xffffffffu, back > 0); m; m &= m - 1) {
      const int src = __ffs(m) - 1;
      int32_t* r = const_cast<int32_t*>(c.table) + (long long)(b - lane + src) * c.max_pages +
                   __shfl_sync(0xffffffffu, cut, src);
      const int many = __shfl_sync(0xffffffffu, back, src);
      const long long to = __shfl_sync(0xffffffffu, back_end, src) - many;
      for (int i = lane; i < many; i += 32) {
        if (to + i < c.n_pages) w.back[to + i] = r[i];
        r[i] = -1;
      }
    }
    rows0 += total[0];
    back0 += total[1];
    need0 += need_total[0];
  }
  // more pages than there are come back only where the table names one twice
  if (back0 > c.n_pages) {
    if (tid == 0) record_status(a.status, QMOE_ERR_DEVICE_ARG);
    back0 = c.n_pages;
  }
  int n_free = *a.n_free;
  if (n_free < 0 || n_free + back0 > c.n_pages) {
    if (tid == 0) record_status(a.status, QMOE_ERR_DEVICE_ARG);
    n_free = n_free < 0 ? 0 : (int)(c.n_pages - back0);
  }
  __syncthreads();  // everybody has read the pool's count
  const long long pool = n_free + back0;
  __shared__ int taken;
  if (tid == 0) taken = 0;
  __syncthreads();
  for (int b = tid; b < c.n_seqs; b += PL_THREADS) {
    const int n = max(a.count[b], 0);
    const PlanHead h{n_free, (int)back0, 0, 0};
    const bool ok = plan_granted(c, a, w, h, b, n);
    a.granted[b] = ok ? n : 0;
    if (ok && w.need[b] > 0) atomicMax(&taken, w.need_end[b]);
  }
  __syncthreads();
  if (tid == 0) {
    *w.head = PlanHead{n_free, (int)back0, taken, 0};
    *a.n_free = (int)pool - taken;
  }
}

// The first index in [0, n) whose entry is above v (n: none); entries do not fall.
__device__ __forceinline__ int plan_above(const int32_t* end, int n, int v) {
  int lo = 0, hi = n;
  while (lo < hi) {
    const int mid = (lo + hi) >> 1;
    if (end[mid] > v)
      hi = mid;
    else
      lo = mid + 1;
  }
  return lo;
}

// Table, stack and row maps, over ``threads`` threads of the grid.
__device__ __forceinline__ void plan_fill(const PagedView& c, const PlanArgs& a, const PlanWs& w, long long tid,
                                          long long threads) {
  const PlanHead h = *w.head;
  const int pool = h.n_free + h.back, left = pool - h.taken;
  // pages that came back and that the rows leave are pushed
  for (long long i = tid; h.n_free + i < left; i += threads) a.free_pages[h.n_free + i] = w.back[i];
  // pages off the top: first the last that came back
  for (long long i = tid; i < h.taken; i += threads) {
    const int b = plan_above(w.need_end, c.n_seqs, (int)i);
    const int before = b ? w.need_end[b - 1] : 0, from = pool - 1 - (int)i;
    int page = from >= h.n_free ? w.back[from - h.n_free] : a.free_pages[from];
    if (!plan_page(c, page)) {
      record_status(a.status, QMOE_ERR_DEVICE_ARG);
      page = -1;
    }
    const_cast<int32_t*>(c.table)[(long long)b * c.max_pages + w.from[b] + (int)i - before] = page;
  }
  for (long long i = tid; i < a.n_rows; i += threads) {
    // the last sequence that begins at or before the row (those without rows begin where the next one does)
    const int b = plan_above(w.first, c.n_seqs, (int)i) - 1;
    const int r = (int)i - w.first[b], n = max(a.count[b], 0);
    const bool somebodys = r < n;
    a.seq[i] = somebodys ? b : -1;
    a.slot[i] = somebodys && a.granted[b] > 0 ? w.len[b] + r : -1;
    a.pos[i] = !somebodys ? 0 : (a.next_pos ? a.next_pos[b] : w.len[b]) + r;
  }
}

__global__ void __launch_bounds__(PL_THREADS) plan_count_kernel(const PagedView c, const PlanArgs a, const PlanWs w,
                                                                bool fill) {
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  plan_count(c, a, w);
  if (!fill) return;
  __syncthreads();
  plan_fill(c, a, w, threadIdx.x, PL_THREADS);
}

__global__ void __launch_bounds__(PF_THREADS) plan_fill_kernel(const PagedView c, const PlanArgs a, const PlanWs w) {
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  plan_fill(c, a, w, (long long)blockIdx.x * PF_THREADS + threadIdx.x, (long long)gridDim.x * PF_THREADS);
}

// One CTA does it all where there are few rows.
bool plan_alone(const PlanArgs& a) { return a.n_rows <= PF_ROWS; }

}  // namespace

size_t paged_plan_ws_bytes(const PagedView& c) {
  size_t total = 0;
  plan_ws(c, nullptr, &total);
  return total;
}

int paged_plan_launches(const PagedView&, const PlanArgs& a) { return plan_alone(a) ? 1 : 2; }

cudaError_t launch_paged_plan(const PagedView& c, const PlanArgs& a, cudaStream_t st) {
  size_t total = 0;
  const PlanWs w = plan_ws(c, a.ws, &total);
  cudaError_t e = launch_overlapped(plan_count_kernel, dim3(1), PL_THREADS, 0, 0, st, c, a, w, plan_alone(a));
  if (e != cudaSuccess || plan_alone(a)) return e;
  long long ctas = ((long long)a.n_rows + PF_THREADS - 1) / PF_THREADS;
  if (ctas > PF_MAX_CTAS) ctas = PF_MAX_CTAS;
  return launch_overlapped(plan_fill_kernel, dim3((unsigned)ctas), PF_THREADS, 0, 0, st, c, a, w);
}

}  // namespace qmoe
