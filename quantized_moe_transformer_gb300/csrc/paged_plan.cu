// A step's plan for the paged key-value cache: sequences are cut back, their
// pages return to the pool, the pages that the new rows miss are handed out, and
// the rows' sequences, slots and positions are written. Defined in include/qmoe.h.
#include <climits>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

constexpr int PL_THREADS = 1024, PL_WARPS = 32, PF_THREADS = 256, PF_ROWS = 4, PF_MAX_CTAS = 2048;
constexpr int PL_SEQS = 1024;   // as many sequences' arrays fit in shared memory
constexpr int PL_ALONE = 1024;  // up to as many rows are written by the kernel that counts

// What the first kernel leaves for the second: the state of the pool before the
// call, and arrays over the sequences.
struct PlanHead {
  int n_free, back, taken, pad;
};

struct PlanWs {
  PlanHead* head;
  int32_t *first;     // the rows before the sequence
  int32_t *need_end;  // pages asked for up to and with it
  int32_t *len;       // entries that it keeps
  int32_t *from;      // first table entry without a page
  int32_t *granted;   // rows that the sequence is granted
  int32_t *need;      // pages that it asks for (0: none, or refused for its size); for the first kernel alone
  int32_t *back;      // [pages] the pages that came back, in order
};
constexpr int PL_ARRAYS = 6, PF_ARRAYS = 5;

__host__ __device__ inline size_t plan_up(size_t v) { return (v + 255) & ~size_t(255); }

__host__ PlanWs plan_ws(const PagedView& c, void* ws, size_t* total) {
  char* p = static_cast<char*>(ws);
  const size_t seqs = plan_up(sizeof(int32_t) * (size_t)c.n_seqs);
  size_t o = 256;
  PlanWs w{};
  w.head = reinterpret_cast<PlanHead*>(p);
  int32_t** const arrays[PL_ARRAYS] = {&w.first, &w.need_end, &w.len, &w.from, &w.granted, &w.need};
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

// The sequence ``b``'s rows are granted: they fit, and its pages are among the first ``pages`` off the stack.
__device__ __forceinline__ bool plan_granted(const PagedView& c, const PlanArgs& a, const PlanWs& w, int pages, int b,
                                             int n) {
  return n > 0 && (long long)w.first[b] + n <= a.n_rows && (long long)w.len[b] + n <= paged_slots(c) &&
         (w.need[b] == 0 || w.need_end[b] <= pages);
}

// The threads with ``mine`` in ``list`` (in any order), and how many; all threads of the CTA.
__device__ __forceinline__ int plan_list(bool mine, int* list, int* listed) {
  if (threadIdx.x == 0) *listed = 0;
  __syncthreads();
  if (mine) list[atomicAdd(listed, 1)] = threadIdx.x;
  __syncthreads();
  return *listed;
}

// What bounds it: a chain of dependent loads and barriers in one CTA (lengths, table entries, sums, pages), 8 us for 96
// sequences with a row each; 256 sequences, 256 thousand rows and 13 thousand pages given back and handed out 17 us, of which
// the second kernel's maps take 4 (3 MB).
// One CTA: each sequence's pages that come back and that it misses, and their sums
// over the sequences. A thread has a sequence; long runs of pages are walked and moved by the warps.
__device__ __forceinline__ void plan_count(const PagedView& c, const PlanArgs& a, const PlanWs& w) {
  __shared__ long long part[3][PL_WARPS];
  __shared__ int list[PL_THREADS], one_of[3][PL_THREADS], listed;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
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
    // (most have the page that is begun and none behind it: two entries at once by the thread itself)
    const bool one = have < stop && plan_page(c, row[have]);
    const bool two = have + 1 < stop && plan_page(c, row[have + 1]);
    if (one) have += two ? 2 : 1;
    const bool open = one && two;
    const int n_open = plan_list(open, list, &listed);
    one_of[0][tid] = have;
    one_of[1][tid] = stop;
    __syncthreads();
    for (int i = warp; i < n_open; i += PL_WARPS) {
      const int src = list[i], to = one_of[1][src];
      const int32_t* r = c.table + (long long)(b0 + src) * c.max_pages;
      int at = one_of[0][src];
      while (at < to) {  // 128 entries at once, the last of them that is a page, and the first that is none
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) page[k] = at + 32 * k + lane < to ? r[at + 32 * k + lane] : -1;
        unsigned gone = 0;
        int k = 0;
#pragma unroll
        for (int e = 0; e < 4; ++e) {
          const unsigned g = __ballot_sync(0xffffffffu, !plan_page(c, page[e]));
          if (gone == 0 && g != 0) {
            gone = g;
            k = e;
          }
        }
        if (gone) {
          at += 32 * k + __ffs(gone) - 1;
          break;
        }
        at += 128;
      }
      if (lane == 0) one_of[0][src] = min(at, to);
    }
    __syncthreads();
    have = one_of[0][tid];
    __syncthreads();
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
      w.need_end[b] = plan_int(need0 + u[0]);
      w.need[b] = need;
      w.len[b] = len;
      w.from[b] = from;
      a.first[b] = plan_int(first);
    }
    // the pages that come back, in order, leave the table
    const int n_back = plan_list(back > 0, list, &listed);
    one_of[0][tid] = cut;
    one_of[1][tid] = back;
    one_of[2][tid] = (int)min(back_end - back, (long long)c.n_pages);
    __syncthreads();
    for (int i = warp; i < n_back; i += PL_WARPS) {
      const int src = list[i], many = one_of[1][src];
      int32_t* r = const_cast<int32_t*>(c.table) + (long long)(b0 + src) * c.max_pages + one_of[0][src];
      const long long to = one_of[2][src];
      for (int i0 = 0; i0 < many; i0 += 128) {
        int page[4];
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = i0 + 32 * k + lane;
          if (x < many) page[k] = r[x];
        }
#pragma unroll
        for (int k = 0; k < 4; ++k) {
          const int x = i0 + 32 * k + lane;
          if (x >= many) continue;
          if (to + x < c.n_pages) w.back[to + x] = page[k];
          r[x] = -1;
        }
      }
    }
    __syncthreads();
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
  __shared__ int taken, pages;
  const int pool = (int)(n_free + back0);
  if (tid == 0) {
    taken = 0;
    pages = pool;
  }
  __syncthreads();  // (everybody has read the pool's count too)
  // a number on the stack that is no page ends what can be handed out: a sequence's pages have no hole
  const int asked = (int)min(need0, (long long)pool);
  for (int i = (int)back0 + tid; i < asked; i += PL_THREADS) {
    if (plan_page(c, a.free_pages[pool - 1 - i])) continue;
    record_status(a.status, QMOE_ERR_DEVICE_ARG);
    atomicMin(&pages, i);
  }
  __syncthreads();
  for (int b = tid; b < c.n_seqs; b += PL_THREADS) {
    const int n = max(a.count[b], 0);
    const bool ok = plan_granted(c, a, w, pages, b, n);
    a.granted[b] = w.granted[b] = ok ? n : 0;
    if (ok && w.need[b] > 0) atomicMax(&taken, w.need_end[b]);
  }
  __syncthreads();
  if (tid == 0) {
    *w.head = PlanHead{n_free, (int)back0, taken, 0};
    *a.n_free = pool - taken;
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

// Table, stack and row maps, over ``threads`` threads of the grid (a multiple of 32).
__device__ __forceinline__ void plan_fill(const PagedView& c, const PlanArgs& a, const PlanWs& w, const PlanHead& h,
                                          long long tid, long long threads) {
  const int pool = h.n_free + h.back, left = pool - h.taken;
  // pages that came back and that the rows leave are pushed
  for (long long i = tid; h.n_free + i < left; i += threads) a.free_pages[h.n_free + i] = w.back[i];
  // pages off the top: first the last that came back
  for (long long i = tid; i < h.taken; i += threads) {
    const int b = plan_above(w.need_end, c.n_seqs, (int)i);
    const int before = b ? w.need_end[b - 1] : 0, from = pool - 1 - (int)i;
    const_cast<int32_t*>(c.table)[(long long)b * c.max_pages + w.from[b] + (int)i - before] =
        from >= h.n_free ? w.back[from - h.n_free] : a.free_pages[from];
  }
  // four rows a thread, 16 bytes of each map where they lie so
  const bool wide = ((reinterpret_cast<uintptr_t>(a.seq) | reinterpret_cast<uintptr_t>(a.slot) |
                      reinterpret_cast<uintptr_t>(a.pos)) & 15) == 0;
  for (long long i0 = PF_ROWS * tid; i0 < a.n_rows; i0 += PF_ROWS * threads) {
    // the last sequence that begins at or before the row (those without rows begin where the next one does)
    int b = plan_above(w.first, c.n_seqs, (int)i0) - 1;
    int seq[PF_ROWS], slot[PF_ROWS], pos[PF_ROWS];
    int next = b + 1 < c.n_seqs ? w.first[b + 1] : INT_MAX, r0 = w.first[b], n = max(a.count[b], 0), granted = w.granted[b],
        len = w.len[b], at = a.next_pos ? a.next_pos[b] : len;
#pragma unroll
    for (int k = 0; k < PF_ROWS; ++k) {
      const int i = (int)i0 + k;
      if (i >= next) {
        b = plan_above(w.first, c.n_seqs, i) - 1;
        next = b + 1 < c.n_seqs ? w.first[b + 1] : INT_MAX;
        r0 = w.first[b];
        n = max(a.count[b], 0);
        granted = w.granted[b];
        len = w.len[b];
        at = a.next_pos ? a.next_pos[b] : len;
      }
      const int r = i - r0;
      const bool somebodys = r < n;
      seq[k] = somebodys ? b : -1;
      slot[k] = somebodys && granted > 0 ? len + r : -1;
      pos[k] = somebodys ? at + r : 0;
    }
    if (wide && i0 + PF_ROWS <= a.n_rows) {
      *reinterpret_cast<int4*>(a.seq + i0) = make_int4(seq[0], seq[1], seq[2], seq[3]);
      *reinterpret_cast<int4*>(a.slot + i0) = make_int4(slot[0], slot[1], slot[2], slot[3]);
      *reinterpret_cast<int4*>(a.pos + i0) = make_int4(pos[0], pos[1], pos[2], pos[3]);
    } else {
#pragma unroll
      for (int k = 0; k < PF_ROWS; ++k) {
        if (i0 + k >= a.n_rows) break;
        a.seq[i0 + k] = seq[k];
        a.slot[i0 + k] = slot[k];
        a.pos[i0 + k] = pos[k];
      }
    }
  }
}

// The arrays over the sequences in shared memory (all but ``need``).
__device__ __forceinline__ PlanWs plan_shared(PlanWs w, int32_t (*arrays)[PL_SEQS]) {
  w.first = arrays[0];
  w.need_end = arrays[1];
  w.len = arrays[2];
  w.from = arrays[3];
  w.granted = arrays[4];
  return w;
}

// The pages are counted by one CTA: sums over the sequences decide who gets which. With few rows it writes all the
// rest too; a second launch costs 2 us more than 1024 rows do here.
__global__ void __launch_bounds__(PL_THREADS) plan_count_kernel(const PagedView c, const PlanArgs a, PlanWs w, bool fill) {
  __shared__ int32_t arrays[PL_ARRAYS][PL_SEQS];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  if (fill && c.n_seqs <= PL_SEQS) {
    w = plan_shared(w, arrays);
    w.need = arrays[PF_ARRAYS];
  }
  plan_count(c, a, w);
  if (!fill) return;
  __syncthreads();
  plan_fill(c, a, w, *w.head, threadIdx.x, PL_THREADS);
}

__global__ void __launch_bounds__(PF_THREADS) plan_fill_kernel(const PagedView c, const PlanArgs a, PlanWs w) {
  __shared__ int32_t arrays[PF_ARRAYS][PL_SEQS];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const PlanHead h = *w.head;
  if (c.n_seqs <= PL_SEQS) {
    const PlanWs s = plan_shared(w, arrays);
    for (int b = threadIdx.x; b < c.n_seqs; b += PF_THREADS) {
      s.first[b] = w.first[b];
      s.need_end[b] = w.need_end[b];
      s.len[b] = w.len[b];
      s.from[b] = w.from[b];
      s.granted[b] = w.granted[b];
    }
    w = s;
    __syncthreads();
  }
  plan_fill(c, a, w, h, (long long)blockIdx.x * PF_THREADS + threadIdx.x, (long long)gridDim.x * PF_THREADS);
}

bool plan_alone(const PlanArgs& a) { return a.n_rows <= PL_ALONE; }

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
  long long ctas = ((long long)a.n_rows + PF_ROWS * PF_THREADS - 1) / (PF_ROWS * PF_THREADS);
  if (ctas > PF_MAX_CTAS) ctas = PF_MAX_CTAS;
  return launch_overlapped(plan_fill_kernel, dim3((unsigned)ctas), PF_THREADS, 0, 0, st, c, a, w);
}

}  // namespace qmoe
