// Eviction from a paged key-value cache by accumulated attention weight.
//
// For each (sequence, KV head) the m entries that stay are the first m in the
// order (newest positions first, then larger weight, then lower slot). What
// stays in a slot below m is not touched; the i-th staying entry of the slots
// from m on moves into the i-th slot below m whose entry goes. Attention does
// not depend on the order of a cache's entries, so this is the least that has
// to move, and sources (slots from m on) and destinations (below m) never meet.
#include <cooperative_groups.h>

#include "paged.cuh"

namespace qmoe {

namespace {

namespace cg = cooperative_groups;

constexpr int EV_THREADS = 1024, EV_WARPS = EV_THREADS / 32;
static_assert(EV_WARPS == 32, "a warp adds up the warps' counts");
constexpr int EV_MAX_KEYS = 40960;   // keys a CTA holds in shared memory (160 KB); it re-reads what is behind
constexpr int MV_THREADS = 256, MV_MOVES = 64;

// Order of an entry as an unsigned key: 0xFFFFFFFF for the protected newest
// positions, otherwise the weight's bits made monotone (NaN as -infinity, -0
// as 0). No weight maps to 0xFFFFFFFF.
__device__ __forceinline__ uint32_t evict_key(float w, bool young) {
  uint32_t u = __float_as_uint(w);
  if ((u << 1) > 0xFF000000u) u = 0xFF800000u;
  if ((u << 1) == 0u) u = 0u;
  u = (u & 0x80000000u) ? ~u : u | 0x80000000u;
  return young ? 0xFFFFFFFFu : u;
}

struct EvictLists {
  int32_t *count, *keep;  // [pairs] entries that move, entries that stay
  int32_t *hole, *mover;  // [pairs][list] slots, in order
  long long list;
};

// Up to MV_MOVES moves from the ``i0``-th of a pair on: weights and positions,
// then the rows in units of 16 bytes, all of a thread's loads before its stores.
template <int U>
__device__ __forceinline__ void evict_move(const PagedView& c, const EvictArgs& a, const EvictLists& ls, int b, int g,
                                           int i0, int moves, int threads, long long (*off)[2]) {
  const long long pair = (long long)b * c.n_kv + g, base = pair * paged_slots(c), lb = pair * ls.list;
  const int tid = threadIdx.x, n = min(MV_MOVES, moves - i0);
  if (tid < n) {
    const int src = ls.mover[lb + i0 + tid], dst = ls.hole[lb + i0 + tid];
    long long so = paged_offset(c, b, src), to = paged_offset(c, b, dst);
    a.weight_out[base + dst] = c.weight[base + src];
    if (c.pos) a.pos_out[base + dst] = c.pos[base + src];
    if (so < 0 || to < 0) {
      record_status(a.status, QMOE_ERR_DEVICE_ARG);
      so = -1;
    }
    off[tid][0] = so;
    off[tid][1] = to;
  }
  __syncthreads();
  const int row = c.head_dim / 8, units = n * 2 * row;
  const long long hs = (long long)g * c.head_stride;
  for (int u0 = tid; u0 < units; u0 += U * threads) {
    uint4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + k * threads, mv = u / (2 * row), r = u - mv * 2 * row;
      if (u < units && off[mv][0] >= 0)
        x[k] = *reinterpret_cast<const uint4*>((r < row ? c.k + 8 * r : c.v + 8 * (r - row)) + hs + off[mv][0]);
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int u = u0 + k * threads, mv = u / (2 * row), r = u - mv * 2 * row;
      if (u < units && off[mv][0] >= 0)
        *reinterpret_cast<uint4*>((r < row ? c.k + 8 * r : c.v + 8 * (r - row)) + hs + off[mv][1]) = x[k];
    }
  }
  __syncthreads();
}

// One cluster per (sequence, KV head); CTA r of it holds the keys of the r-th
// slice of the slots in shared memory, warp w the w-th part of the slice. The m-th
// largest key is found 8 bits at a time from the top: each CTA counts its keys by
// digit, every CTA adds the counts up over the cluster through distributed
// shared memory and picks the digit, until the entries that share the digits so
// far all stay. Then the staying entries' ranks (counts over warps and CTAs)
// give each of them its place in the list of holes or movers. The weights are
// read once; what bounds it is the latency of the 2 to 6 cluster barriers.
template <bool INLINE>
__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const PagedView c, const EvictArgs a,
                                                                     const EvictLists ls, int smem_keys) {
  extern __shared__ uint32_t ev_keys[];
  __shared__ int hist[2][256], warp_cnt[2][EV_WARPS], cta_cnt[2][2], scan[8], pick[3];
  __shared__ long long off[MV_MOVES][2];
  cg::cluster_group cluster = cg::this_cluster();
  const int C = (int)cluster.num_blocks(), rank = (int)cluster.block_rank();
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const long long pair = blockIdx.x / C, base = pair * paged_slots(c), lb = pair * ls.list;
  const int b = (int)(pair / c.n_kv), g = (int)(pair % c.n_kv);
  const int n = paged_len(c, b), m = min(n, a.budget);
  const long long young_from = a.recent > 0 ? (long long)a.next_pos[b] - a.recent : 0;
  if (rank == 0 && tid == 0) {
    ls.keep[pair] = m;
    if (m == n || m == 0) ls.count[pair] = 0;
  }
  const bool copy_w = a.weight_out != c.weight, copy_p = c.pos != nullptr && a.pos_out != c.pos;
  if (m == n || m == 0) {  // (the whole cluster)
    for (int j = rank * EV_THREADS + tid; j < m; j += C * EV_THREADS) {
      if (copy_w) a.weight_out[base + j] = c.weight[base + j];
      if (copy_p) a.pos_out[base + j] = c.pos[base + j];
    }
    if (INLINE && rank == 0 && g == 0 && tid == 0) a.lens_out[b] = m;
    return;
  }
  const int per = ((n + C - 1) / C + EV_THREADS - 1) / EV_THREADS * EV_THREADS;  // slots of a slice
  const long long lo = (long long)rank * per;
  const int size = lo < n ? (int)(n - lo < per ? n - lo : per) : 0;
  const int w0 = warp * (per / EV_WARPS), w1 = min(size, w0 + per / EV_WARPS);    // this warp's part of it
  auto fresh = [&](int i) {
    return evict_key(c.weight[base + lo + i], a.recent > 0 && c.pos[base + lo + i] >= young_from);
  };
  auto key = [&](int i) { return i < smem_keys ? ev_keys[i] : fresh(i); };
#pragma unroll 4
  for (int i = w0 + lane; i < min(w1, smem_keys); i += 32) ev_keys[i] = fresh(i);

  // ---- the m-th largest key
  uint32_t t = 0, known = 0;  // its digits so far, and which bits those are
  int need = m, equal = 0;    // of the ``equal`` keys with these digits, ``need`` stay
  for (int shift = 24; shift >= 0; shift -= 8) {
    int* h = hist[(shift >> 3) & 1];
    if (tid < 256) h[tid] = 0;
    __syncthreads();
    for (int i0 = w0; i0 < w1; i0 += 32) {
      const int i = i0 + lane;
      const uint32_t k = i < w1 ? key(i) : 0u;
      const bool in = i < w1 && (k & known) == t;
      const uint32_t digit = (k >> shift) & 255u;
      // lanes with one digit (equal weights, the first digits) add up first
      const unsigned active = __ballot_sync(0xffffffffu, in);
      if (in) {
        const int lead = __ffs(active) - 1;
        const unsigned same = __ballot_sync(active, digit == __shfl_sync(active, digit, lead));
        if (same == active) {
          if (lane == lead) atomicAdd(&h[digit], __popc(active));
        } else {
          atomicAdd(&h[digit], 1);
        }
      }
    }
    cluster.sync();
    int cnt = 0, incl = 0;
    if (tid < 256) {  // from the largest digit down
#pragma unroll
      for (int r = 0; r < 8; ++r) cnt += cluster.map_shared_rank(h, r < C ? r : rank)[255 - tid] * (r < C);
      incl = cnt;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int x = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o) incl += x;
      }
      if (lane == 31) scan[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
      for (int w = 0; w < warp; ++w) incl += scan[w];
      if (incl >= need && incl - cnt < need) {
        pick[0] = 255 - tid;
        pick[1] = need - (incl - cnt);
        pick[2] = cnt;
      }
    }
    __syncthreads();
    t |= (uint32_t)pick[0] << shift;
    known |= 255u << shift;
    need = pick[1];
    equal = pick[2];
    if (need == equal) break;
  }
  // ---- ranks: of the equal keys the lowest slots stay
  int eq_before = 0;
  const bool rank_equal = need < equal;
  if (rank_equal) {
    int cnt = 0;
    for (int i = w0 + lane; i < w1; i += 32) cnt += key(i) == t;
    cnt = __reduce_add_sync(0xffffffffu, cnt);
    if (lane == 0) warp_cnt[0][warp] = cnt;
    __syncthreads();
    const int v = warp_cnt[0][lane], all = __reduce_add_sync(0xffffffffu, v);
    eq_before = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
    if (tid == 0) cta_cnt[0][0] = all;
    cluster.sync();
#pragma unroll
    for (int r = 0; r < 8; ++r) eq_before += cluster.map_shared_rank(&cta_cnt[0][0], r < rank ? r : rank)[0] * (r < rank);
    __syncthreads();
  }
  // which of 32 entries stay; ``eq`` runs over the equal ones before them
  auto stays = [&](int i, int& eq) {
    const uint32_t k = i < w1 ? key(i) : 0u;
    bool kept = i < w1 && k >= t;
    if (rank_equal) {
      const bool same = i < w1 && k == t;
      const unsigned mk = __ballot_sync(0xffffffffu, same);
      if (same) kept = eq + __popc(mk & ((1u << lane) - 1u)) < need;
      eq += __popc(mk);
    }
    return kept;
  };
  int holes = 0, movers = 0, eq = eq_before;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool kept = stays(i, eq);
    holes += __popc(__ballot_sync(0xffffffffu, i < w1 && !kept && lo + i < m));
    movers += __popc(__ballot_sync(0xffffffffu, kept && lo + i >= m));
  }
  if (lane == 0) {
    warp_cnt[0][warp] = holes;
    warp_cnt[1][warp] = movers;
  }
  __syncthreads();
  {
    const int h = warp_cnt[0][lane], v = warp_cnt[1][lane];
    const int hs = __reduce_add_sync(0xffffffffu, h), vs = __reduce_add_sync(0xffffffffu, v);
    if (tid == 0) {
      cta_cnt[1][0] = hs;
      cta_cnt[1][1] = vs;
    }
    holes = __reduce_add_sync(0xffffffffu, lane < warp ? h : 0);
    movers = __reduce_add_sync(0xffffffffu, lane < warp ? v : 0);
  }
  cluster.sync();
  int all = 0;
#pragma unroll
  for (int r = 0; r < 8; ++r) {  // (all loads at once: one after the other they cost their latency each)
    const int* x = cluster.map_shared_rank(&cta_cnt[1][0], r < C ? r : rank);
    const int x0 = x[0], x1 = x[1];
    if (r < rank) {
      holes += x0;
      movers += x1;
    }
    if (r < C) all += x1;
  }
  eq = eq_before;
  for (int i0 = w0; i0 < w1; i0 += 32) {
    const int i = i0 + lane;
    const bool kept = stays(i, eq);
    const int j = (int)lo + i;
    const bool hole = i < w1 && !kept && j < m, mover = kept && j >= m;
    const unsigned mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    const unsigned below = (1u << lane) - 1u;
    if (hole) ls.hole[lb + holes + __popc(mh & below)] = j;
    if (mover) ls.mover[lb + movers + __popc(mm & below)] = j;
    holes += __popc(mh);
    movers += __popc(mm);
    if (kept && j < m) {
      if (copy_w) a.weight_out[base + j] = c.weight[base + j];
      if (copy_p) a.pos_out[base + j] = c.pos[base + j];
    }
  }
  if (rank == 0 && tid == 0) ls.count[pair] = all;
  cluster.sync();  // the lists are written, and no CTA ends while another reads its counts
  if (!INLINE) return;
  if (rank == 0 && g == 0 && tid == 0) a.lens_out[b] = m;  // (every CTA of the cluster has read the old length)
  for (int i0 = rank * MV_MOVES; i0 < all; i0 += C * MV_MOVES)
    evict_move<4>(c, a, ls, b, g, i0, all, EV_THREADS, off);
}

// 64 moves a CTA.
__global__ void __launch_bounds__(MV_THREADS, 4) evict_move_kernel(const PagedView c, const EvictArgs a,
                                                                const EvictLists ls) {
  __shared__ long long off[MV_MOVES][2];
  asm volatile("griddepcontrol.wait;" ::: "memory");
  const long long pair = blockIdx.x;
  const int b = (int)(pair / c.n_kv), g = (int)(pair % c.n_kv), all = ls.count[pair];
  if (blockIdx.y == 0 && g == 0 && threadIdx.x == 0) a.lens_out[b] = ls.keep[pair];
  for (long long i0 = (long long)blockIdx.y * MV_MOVES; i0 < all; i0 += (long long)gridDim.y * MV_MOVES)
    evict_move<8>(c, a, ls, b, g, (int)i0, all, MV_THREADS, off);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Moves of a pair: at most half its slots.
size_t list_len(const PagedView& c) { return (size_t)paged_slots(c) / 2 + 1; }

}  // namespace

size_t cache_evict_ws_bytes(const PagedView& c) {
  const size_t pairs = (size_t)c.n_seqs * c.n_kv;
  return 2 * up256(4 * pairs) + 2 * up256(4 * pairs * list_len(c));
}

// One kernel where a CTA of the select kernel has at most 64 moves, and no
// cluster that starts later reads a length that another has replaced: a second
// launch costs more than the moves. Else the moves get a grid of their own.
static bool evict_inline(const PagedView& c, const EvictArgs& a) {
  const long long slots = paged_slots(c), most = a.budget < slots - a.budget ? a.budget : slots - a.budget;
  return most <= MV_MOVES && (c.n_kv == 1 || a.lens_out != c.lens);
}

int cache_evict_launches(const PagedView& c, const EvictArgs& a) { return evict_inline(c, a) ? 1 : 2; }

cudaError_t launch_cache_evict(const PagedView& c, const EvictArgs& a, cudaStream_t st) {
  const long long pairs = (long long)c.n_seqs * c.n_kv, slots = paged_slots(c);
  char* p = static_cast<char*>(a.ws);
  EvictLists ls;
  ls.list = (long long)list_len(c);
  ls.count = reinterpret_cast<int32_t*>(p);
  ls.keep = reinterpret_cast<int32_t*>(p + up256(4 * pairs));
  ls.hole = reinterpret_cast<int32_t*>(p + 2 * up256(4 * pairs));
  ls.mover = reinterpret_cast<int32_t*>(p + 2 * up256(4 * pairs) + up256(4 * pairs * ls.list));
  // CTAs of a cluster: slices of at most 8192 slots (8 keys a thread; a barrier of the cluster costs more than
  // those), while the CTAs fit the SMs
  int C = 1;
  while (C < 8 && slots > 8192ll * C && pairs * C * 2 <= device_sm_count()) C *= 2;
  const long long slice = ((slots + C - 1) / C + EV_THREADS - 1) / EV_THREADS * EV_THREADS;
  const int keys = slice < EV_MAX_KEYS ? (int)slice : EV_MAX_KEYS;
  const bool in = evict_inline(c, a);
  if (pairs * C > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  auto* select = in ? evict_select_kernel<true> : evict_select_kernel<false>;
  cudaError_t e = ensure_kernel_smem(reinterpret_cast<const void*>(select), sizeof(uint32_t) * keys);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = dim3((unsigned)(pairs * C));
  cfg.blockDim = dim3(EV_THREADS);
  cfg.dynamicSmemBytes = sizeof(uint32_t) * keys;
  cfg.stream = st;
  cudaLaunchAttribute attr{};
  attr.id = cudaLaunchAttributeClusterDimension;
  attr.val.clusterDim.x = C;
  attr.val.clusterDim.y = attr.val.clusterDim.z = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  e = cudaLaunchKernelEx(&cfg, select, c, a, ls, keys);
  if (e != cudaSuccess || in) return e;
  const long long most = a.budget < slots - a.budget ? a.budget : slots - a.budget;
  long long parts = (most + MV_MOVES - 1) / MV_MOVES;
  if (parts < 1) parts = 1;
  if (parts > 65535) parts = 65535;
  cfg = cudaLaunchConfig_t{};
  cfg.gridDim = dim3((unsigned)pairs, (unsigned)parts);
  cfg.blockDim = dim3(MV_THREADS);
  cfg.stream = st;
  attr.id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr.val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = &attr;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, evict_move_kernel, c, a, ls);
}

}  // namespace qmoe
