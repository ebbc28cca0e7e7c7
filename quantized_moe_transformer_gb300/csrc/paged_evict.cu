// Eviction from a paged key-value cache by accumulated attention weight.
//
// For each (sequence, KV head) the m entries that stay are the first m in the
// order (newest positions first, then larger weight, then lower slot). What
// stays in a slot below m is not touched; the i-th staying entry of the slots
// from m on moves into the i-th slot below m whose entry goes. Attention does
// not depend on the order of a cache's entries, so this is the least that has
// to move, and sources (slots from m on) and destinations (below m) never meet.
#include "paged.cuh"

namespace qmoe {

namespace {

constexpr int EV_THREADS = 1024;

// Order of an entry as an unsigned key: 0xFFFFFFFF for the protected newest
// positions, otherwise the weight's bits made monotone (NaN as the least,
// -0 as 0). No weight maps to 0xFFFFFFFF.
__device__ __forceinline__ uint32_t evict_key(float w, bool young) {
  uint32_t u = __float_as_uint(w);
  if ((u << 1) > 0xFF000000u) u = 0xFF800000u;  // NaN: as -infinity
  if ((u << 1) == 0u) u = 0u;
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return young ? 0xFFFFFFFFu : u;
}

__device__ __forceinline__ int block_sum(int v, int* red) {
  v = __reduce_add_sync(0xffffffffu, v);
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  int s = 0;
  for (int w = 0; w < EV_THREADS / 32; ++w) s += red[w];
  return s;
}

// Exclusive rank of this thread among the threads with ``f``; ``total``: all.
__device__ __forceinline__ int block_rank(bool f, int* red, int* total) {
  const unsigned m = __ballot_sync(0xffffffffu, f);
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  __syncthreads();
  if (lane == 0) red[warp] = __popc(m);
  __syncthreads();
  int before = 0, all = 0;
  for (int w = 0; w < EV_THREADS / 32; ++w) {
    if (w < warp) before += red[w];
    all += red[w];
  }
  *total = all;
  return before + __popc(m & ((1u << lane) - 1u));
}

struct EvictLists {
  int32_t *count, *keep, *hole, *mover;  // [pairs], [pairs], [pairs][slots], [pairs][slots]
};

__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const PagedView c, const EvictArgs a,
                                                                  const EvictLists ls) {
  __shared__ int red[EV_THREADS / 32];
  const int b = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
  const long long slots = paged_slots(c), pair = (long long)b * c.n_kv + g, base = pair * slots;
  const int n = paged_len(c, b), m = min(n, a.budget);
  const int young_from = a.recent > 0 ? a.next_pos[b] - a.recent : 0;
  auto key = [&](int j) {
    return evict_key(c.weight[base + j], a.recent > 0 && c.pos[base + j] >= young_from);
  };
  if (tid == 0) ls.keep[pair] = m;
  if (m == n || m == 0) {
    if (tid == 0) ls.count[pair] = 0;
    return;
  }
  // the m-th largest key, a bit at a time
  uint32_t t = 0;
  for (int bit = 31; bit >= 0; --bit) {
    const uint32_t u = t | (1u << bit);
    int cnt = 0;
    for (int j = tid; j < n; j += EV_THREADS) cnt += key(j) >= u;
    if (block_sum(cnt, red) >= m) t = u;
  }
  int cnt = 0;
  for (int j = tid; j < n; j += EV_THREADS) cnt += key(j) > t;
  const int ties = m - block_sum(cnt, red);  // of the entries equal to it, the first stay
  int eq0 = 0, hole0 = 0, mover0 = 0;
  for (int j0 = 0; j0 < n; j0 += EV_THREADS) {
    const int j = j0 + tid;
    const uint32_t k = j < n ? key(j) : 0u;
    int total;
    const bool eq = j < n && k == t;
    const int er = block_rank(eq, red, &total) + eq0;  // (a barrier: every thread takes part)
    const bool kept = (j < n && k > t) || (eq && er < ties);
    eq0 += total;
    const bool hole = j < m && !kept, mover = j >= m && kept;
    int r = block_rank(hole, red, &total) + hole0;
    if (hole) ls.hole[base + r] = j;
    hole0 += total;
    r = block_rank(mover, red, &total) + mover0;
    if (mover) ls.mover[base + r] = j;
    mover0 += total;
  }
  if (tid == 0) ls.count[pair] = mover0;
}

__global__ void __launch_bounds__(256) evict_move_kernel(const PagedView c, const EvictArgs a, const EvictLists ls) {
  const int b = blockIdx.x, g = blockIdx.y, tid = threadIdx.x;
  const long long slots = paged_slots(c), pair = (long long)b * c.n_kv + g, base = pair * slots;
  const int m = ls.keep[pair], moves = ls.count[pair], hd = c.head_dim;
  if (a.weight_out != c.weight)
    for (int j = tid; j < m; j += 256) a.weight_out[base + j] = c.weight[base + j];
  if (c.pos && a.pos_out != c.pos)
    for (int j = tid; j < m; j += 256) a.pos_out[base + j] = c.pos[base + j];
  __syncthreads();
  for (int i = tid >> 5; i < moves; i += 8) {
    const int src = ls.mover[base + i], dst = ls.hole[base + i];
    const long long so = paged_offset(c, b, src), to = paged_offset(c, b, dst);
    if ((tid & 31) == 0) {
      a.weight_out[base + dst] = c.weight[base + src];
      if (c.pos) a.pos_out[base + dst] = c.pos[base + src];
    }
    if (so < 0 || to < 0) {
      record_status(a.status, QMOE_ERR_DEVICE_ARG);
      continue;
    }
    const long long hs = (long long)g * c.head_stride;
    for (int d = tid & 31; d < hd; d += 32) {
      c.k[to + hs + d] = c.k[so + hs + d];
      c.v[to + hs + d] = c.v[so + hs + d];
    }
  }
  if (g == 0 && tid == 0) a.lens_out[b] = m;
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

}  // namespace

size_t cache_evict_ws_bytes(const PagedView& c) {
  const size_t pairs = (size_t)c.n_seqs * c.n_kv, slots = (size_t)paged_slots(c);
  return 2 * up256(4 * pairs) + 2 * up256(4 * pairs * slots);
}
int cache_evict_launches() { return 2; }

cudaError_t launch_cache_evict(const PagedView& c, const EvictArgs& a, cudaStream_t st) {
  const size_t pairs = (size_t)c.n_seqs * c.n_kv, slots = (size_t)paged_slots(c);
  char* p = static_cast<char*>(a.ws);
  EvictLists ls;
  ls.count = reinterpret_cast<int32_t*>(p);
  ls.keep = reinterpret_cast<int32_t*>(p + up256(4 * pairs));
  ls.hole = reinterpret_cast<int32_t*>(p + 2 * up256(4 * pairs));
  ls.mover = reinterpret_cast<int32_t*>(p + 2 * up256(4 * pairs) + up256(4 * pairs * slots));
  evict_select_kernel<<<dim3(c.n_seqs, c.n_kv), EV_THREADS, 0, st>>>(c, a, ls);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess) return e;
  evict_move_kernel<<<dim3(c.n_seqs, c.n_kv), 256, 0, st>>>(c, a, ls);
  return cudaGetLastError();
}

}  // namespace qmoe
