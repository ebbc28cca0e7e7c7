// Eviction from a paged key-value cache by accumulated attention weight.
//
// For each (sequence, KV head) the m entries that stay are the first m in the
// order (newest positions first, by lower slot; then larger weight, then lower slot). What
// stays in a slot below m is not touched; the i-th staying entry of the slots
// from m on moves into the i-th slot below m whose entry goes. Attention does
// not depend on the order of a cache's entries, so this is the least that has
// to move, and sources (slots from m on) and destinations (below m) never meet.
#include <cooperative_groups.h>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

namespace cg = cooperative_groups;

constexpr int EV_THREADS = 1024, EV_WARPS = 32, EV_CLUSTER = 8;
constexpr int EV_MAX_KEYS = 40960;  // 160 KB
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
  int2 *hole, *mover;     // [pairs][list] (slot, page), in the slots' order
  long long list;
};

__device__ __forceinline__ long long row_offset(const PagedView& c, int2 at) {
  if ((unsigned)at.y >= (unsigned)c.n_pages) return -1;
  return (long long)at.y * c.page_stride + (long long)(at.x & ((1 << c.page_log2) - 1)) * c.slot_stride;
}

// Up to MV_MOVES moves from the ``i0``-th of a pair on: weights and positions,
// then the rows in units of 16 bytes, U loads of a thread before their stores.
// (``count``: the pair's moves; the lists are read while it is still on its way.)
template <int U>
__device__ __forceinline__ void evict_move(const PagedView& c, const EvictArgs& a, const EvictLists& ls, int b, int g,
                                           int i0, const int32_t* count, int threads, long long (*off)[2]) {
  const long long pair = (long long)b * c.n_kv + g, base = pair * paged_slots(c), at = pair * ls.list + i0;
  const int tid = threadIdx.x;
  int2 src = make_int2(0, 0), dst = src;
  if (tid < MV_MOVES && i0 + tid < ls.list) {
    src = ls.mover[at + tid];
    dst = ls.hole[at + tid];
  }
  const int n = min(MV_MOVES, *count - i0);
  if (tid < n) {
    long long so = row_offset(c, src);
    const long long to = row_offset(c, dst);
    if (so < 0 || to < 0) {
      record_status(a.status, QMOE_ERR_DEVICE_ARG);
      so = -1;
    }
    off[tid][0] = so;
    off[tid][1] = to;
    a.weight_out[base + dst.x] = c.weight[base + src.x];
    if (c.pos) a.pos_out[base + dst.x] = c.pos[base + src.x];
  }
  __syncthreads();
  // a lane keeps its place r in a row pair (the key's units, then the value's); a warp has 32 / (2 row) moves at once
  // where a pair fits it, else it walks one pair
  const int row = c.head_dim / 8, pair_units = 2 * row, lane = tid & 31, warp = tid >> 5, warps = threads / 32;
  const int at_once = pair_units <= 32 ? 32 / pair_units : 1, sub = pair_units <= 32 ? lane / pair_units : 0;
  const long long hs = (long long)g * c.head_stride;
  for (int r = lane - sub * pair_units; r < pair_units && sub < at_once; r += 32) {
    __nv_bfloat16* pool = (r < row ? c.k + 8 * r : c.v + 8 * (r - row)) + hs;
    for (int mv = warp * at_once + sub; mv < n; mv += U * warps * at_once) {
      uint4 x[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = mv + k * warps * at_once;
        if (i < n && off[i][0] >= 0) x[k] = *reinterpret_cast<const uint4*>(pool + off[i][0]);
      }
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int i = mv + k * warps * at_once;
        if (i < n && off[i][0] >= 0) *reinterpret_cast<uint4*>(pool + off[i][1]) = x[k];
      }
    }
  }
  __syncthreads();
}

// One cluster of C CTAs per (sequence, KV head). CTA r takes the r-th slice of
// the slots, warp w the w-th part of the slice, 32 slots at a time; the keys
// stay in shared memory (slices beyond EV_MAX_KEYS are read again for each step). The m-th largest key is
// found 11 bits at a time from the top: the keys that share the digits so far
// are counted by their next digit in shared memory, summed over the cluster
// through distributed shared memory, until all that share the digits stay (two or three
// digits; of 8 bits it took one more, which is 1 to 2 us). The staying
// entries' ranks (counts over warps and CTAs) give each its place in the list
// of holes or movers. Weights and positions are read once; what bounds it is a
// chain of short steps: barriers (0.1 us in a CTA, 0.8 us in a cluster) and code
// that runs once, whose fetch shows (keys in registers with every loop unrolled
// over 8 of them ran longer, 16.5 against 12.0 us for 1 x 4112). 1 x 4112 takes 8.9 us
// with its 16 moves, 64 sequences of 1500 to 8190 11 us, 3 x 65537 (8 CTAs each) 17 us.
template <bool LONG, bool INLINE>
__global__ void __launch_bounds__(EV_THREADS) evict_select_kernel(const PagedView c, const EvictArgs a,
                                                                  const EvictLists ls) {
  extern __shared__ uint32_t ev_keys[];
  __shared__ __align__(16) int2 hist[3][EV_THREADS];  // counts of 2048 digits, two of a thread, for each digit
  __shared__ __align__(16) int2 mine[EV_THREADS];     // a cluster's CTA: its own counts
  __shared__ int4 warp_cnt[EV_WARPS], cta_cnt;
  __shared__ int above_warp[EV_WARPS], pick[3];
  __shared__ long long off[INLINE ? MV_MOVES : 1][2];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
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
  auto all_sync = [&]() {
    if (C > 1)
      cluster.sync();
    else
      __syncthreads();
  };
  // this CTA's slots from lo on; its warp's are [w0, w1) of them
  const int part = ((n + C - 1) / C + EV_THREADS - 1) / EV_THREADS * 32;
  const int lo = (int)min((long long)rank * part * EV_WARPS, (long long)n), size = min(part * EV_WARPS, n - lo);
  const int w0 = warp * part, w1 = min(size, w0 + part);
  const float* weights = c.weight + base + lo;
  const int32_t* positions = c.pos + base + lo;
  auto key = [&](int i) {
    if (!LONG || i < EV_MAX_KEYS) return ev_keys[i];
    return evict_key(weights[i], a.recent > 0 && positions[i] >= young_from);
  };
  hist[0][tid] = hist[1][tid] = hist[2][tid] = mine[tid] = make_int2(0, 0);
  if (C > 1) cluster.barrier_arrive();
  // read once; what stays in place goes to the outputs now (what moves into the holes is written over it later)
  // (eight loads ahead of their stores, which the compiler could not tell from the inputs)
#pragma unroll 1
  for (int i0 = w0 + lane; i0 < w1; i0 += 256) {
    float w[8];
    int p[8];
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + 32 * k;
      w[k] = i < w1 ? weights[i] : 0.f;
      p[k] = i < w1 && c.pos != nullptr ? positions[i] : 0;
    }
#pragma unroll
    for (int k = 0; k < 8; ++k) {
      const int i = i0 + 32 * k;
      if (i >= w1) continue;
      if (!LONG || i < EV_MAX_KEYS) ev_keys[i] = evict_key(w[k], a.recent > 0 && p[k] >= young_from);
      if (copy_w && lo + i < m) a.weight_out[base + lo + i] = w[k];
      if (copy_p && lo + i < m) a.pos_out[base + lo + i] = p[k];
    }
  }
  __syncthreads();

  // ---- the m-th largest key
  uint32_t t = 0, known = 0;  // its digits so far, and which bits those are
  int need = m, equal = 0;    // of the ``equal`` keys with these digits, ``need`` stay
#pragma unroll 1
  for (int pass = 0; pass < 3; ++pass) {
    const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0;  // digits of 11, 11 and 10 bits
    const uint32_t digits = pass == 2 ? 1023u : 2047u;
    int2* h = C > 1 ? mine : hist[pass];
#pragma unroll 2
    for (int i = w0 + lane; i < w1; i += 32) {
      const uint32_t k = key(i);
      if ((k & known) == t) atomicAdd(reinterpret_cast<int*>(h) + ((k >> shift) & digits), 1);
    }
    if (C > 1) {
      // every CTA adds its counts (of few digits but the first) to those of all
      __syncthreads();
      const int2 v = mine[tid];
      mine[tid] = make_int2(0, 0);
      if (pass == 0) cluster.barrier_wait();  // (the others' counts start at zero)
      if (v.x | v.y)
        for (int r = 0; r < C; ++r) {
          int2* to = cluster.map_shared_rank(hist[pass], r) + tid;
          if (v.x) atomicAdd(&to->x, v.x);
          if (v.y) atomicAdd(&to->y, v.y);
        }
    }
    all_sync();
    // this thread's digits 2 tid and 2 tid + 1, and the keys with higher ones
    const int2 d = hist[pass][tid];
    const int own = d.x + d.y;
    int above = own;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int x = __shfl_down_sync(0xffffffffu, above, o);
      if (lane + o < 32) above += x;
    }
    if (lane == 0) above_warp[warp] = above;
    __syncthreads();
    above += __reduce_add_sync(0xffffffffu, lane > warp ? above_warp[lane] : 0) - own;
    if (above < need && above + own >= need) {
      const bool upper = above + d.y >= need;
      pick[0] = 2 * tid + upper;
      pick[1] = upper ? need - above : need - above - d.y;
      pick[2] = upper ? d.y : d.x;
    }
    __syncthreads();
    t |= (uint32_t)pick[0] << shift;
    known |= digits << shift;
    need = pick[1];
    equal = pick[2];
    if (need == equal) break;
  }
  // ---- ranks. Entries above t stay, those below go, of the equal ones the first ``need`` stay (in the slots'
  // order, so those in slots below m first). With the counts x, y of entries below t in slots below m and above t in
  // slots from m on, z, w of equal ones in slots below m and from m on, a stretch of slots with ``before`` equal
  // entries ahead of it has
  auto ranked = [&](int4 c4, int before) {  // (holes, movers)
    const int kept = max(0, min(need - before, c4.z + c4.w)), low = min(kept, c4.z);
    return make_int2(c4.x + c4.z - low, c4.y + kept - low);
  };
  auto scan_equal = [&](int4 c4) {  // equal entries of the lanes below
    int x = c4.z + c4.w;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int y = __shfl_up_sync(0xffffffffu, x, o);
      if (lane >= o) x += y;
    }
    return x - c4.z - c4.w;
  };
  auto sum4 = [&](int4 c4) {
    return make_int4(__reduce_add_sync(0xffffffffu, c4.x), __reduce_add_sync(0xffffffffu, c4.y),
                     __reduce_add_sync(0xffffffffu, c4.z), __reduce_add_sync(0xffffffffu, c4.w));
  };
  int4 cnt = make_int4(0, 0, 0, 0);
#pragma unroll 2
  for (int i = w0 + lane; i < w1; i += 32) {
    const uint32_t k = key(i);
    const bool low = lo + i < m;
    cnt.x += k < t && low;
    cnt.y += k > t && !low;
    cnt.z += k == t && low;
    cnt.w += k == t && !low;
  }
  cnt = sum4(cnt);
  if (lane == 0) warp_cnt[warp] = cnt;
  __syncthreads();
  const int4 of_warp = warp_cnt[lane];
  int eq_before = 0, holes = 0, movers = 0, all;
  {
    const int4 mine4 = sum4(of_warp);
    if (C > 1) {
      if (tid == 0) cta_cnt = mine4;
      cluster.sync();
      const int4 of_cta = *cluster.map_shared_rank(&cta_cnt, lane < C ? lane : rank);
      const int4 c4 = lane < C ? of_cta : make_int4(0, 0, 0, 0);
      const int before = scan_equal(c4);
      const int2 r = ranked(c4, before);
      eq_before = __shfl_sync(0xffffffffu, before, rank);
      holes = __reduce_add_sync(0xffffffffu, lane < rank ? r.x : 0);
      movers = __reduce_add_sync(0xffffffffu, lane < rank ? r.y : 0);
      all = __reduce_add_sync(0xffffffffu, r.y);
    } else {
      all = ranked(mine4, 0).y;
    }
    const int before = eq_before + scan_equal(of_warp);
    const int2 r = ranked(of_warp, before);
    eq_before = __shfl_sync(0xffffffffu, before, warp);
    holes += __reduce_add_sync(0xffffffffu, lane < warp ? r.x : 0);
    movers += __reduce_add_sync(0xffffffffu, lane < warp ? r.y : 0);
  }
  // whether the entry stays (the whole warp asks for 32 in a row); ``eq`` runs over the equal ones before
  const bool rank_equal = need < equal;
  const unsigned lower = (1u << lane) - 1u;
  auto stays = [&](int i, int& eq) {
    const uint32_t k = i < w1 ? key(i) : 0u;
    bool s = i < w1 && k >= t;
    if (rank_equal) {
      const bool same = s && k == t;
      const unsigned mk = __ballot_sync(0xffffffffu, same);
      if (same) s = eq + __popc(mk & lower) < need;
      eq += __popc(mk);
    }
    return s;
  };
  int eq = eq_before;
  const int32_t* table = c.table + (long long)b * c.max_pages;
#pragma unroll 2
  for (int i = w0 + lane; i - lane < w1; i += 32) {
    const bool s = stays(i, eq);
    const int j = lo + i;
    const bool hole = i < w1 && !s && j < m, mover = s && j >= m;
    const unsigned mh = __ballot_sync(0xffffffffu, hole), mm = __ballot_sync(0xffffffffu, mover);
    if (hole || mover) {
      int2* to = hole ? ls.hole + holes + __popc(mh & lower) : ls.mover + movers + __popc(mm & lower);
      to[lb] = make_int2(j, __ldg(table + (j >> c.page_log2)));
    }
    holes += __popc(mh);
    movers += __popc(mm);
  }
  if (rank == 0 && tid == 0) ls.count[pair] = all;
  all_sync();  // the lists are written, and no CTA ends while another reads its counts
  if (!INLINE) return;
  if (rank == 0 && g == 0 && tid == 0) a.lens_out[b] = m;  // (every CTA of the cluster has read the old length)
  for (int i0 = rank * MV_MOVES; i0 < all; i0 += C * MV_MOVES)
    evict_move<2>(c, a, ls, b, g, i0, &all, EV_THREADS, off);
}

// 64 moves a CTA. 110 thousand moves of 512 bytes (64 sequences) take 20 us, 5.6 TB/s
// of reads and writes in pieces of 256 bytes.
__global__ void __launch_bounds__(MV_THREADS, 5) evict_move_kernel(const PagedView c, const EvictArgs a,
                                                                   const EvictLists ls) {
  __shared__ long long off[MV_MOVES][2];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const long long pair = blockIdx.x;
  const int b = (int)(pair / c.n_kv), g = (int)(pair % c.n_kv);
  const int32_t* count = ls.count + pair;
  if (blockIdx.y == 0 && g == 0 && threadIdx.x == 0) a.lens_out[b] = ls.keep[pair];
  for (long long i0 = (long long)blockIdx.y * MV_MOVES; i0 < *count; i0 += (long long)gridDim.y * MV_MOVES)
    evict_move<8>(c, a, ls, b, g, (int)i0, count, MV_THREADS, off);
}

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

// Moves of a pair: at most half its slots.
size_t list_len(const PagedView& c) { return (size_t)paged_slots(c) / 2 + 1; }

}  // namespace

size_t cache_evict_ws_bytes(const PagedView& c) {
  const size_t pairs = (size_t)c.n_seqs * c.n_kv;
  return 2 * up256(4 * pairs) + 2 * up256(sizeof(int2) * pairs * list_len(c));
}

namespace {

struct EvictPlan {
  int cluster, keys;  // CTAs of a cluster, keys of a CTA in shared memory
  bool long_slices, inline_moves;
  long long moves;    // of one pair, at most
};

// One CTA for up to 8192 slots (1 x 4112: 9.4 us, with a cluster of 2 11.1; 16 x
// 8100: 12.1 and with 4 11.8; all figures of this rule from one build); beyond, clusters of 8 where they fit the SMs at once
// (1 x 16000: 12.3 us, of 2 15.3; 1 x 32000: 13.6, of 4 15.7), else as small as
// keeps a slice to 8192 slots. The moves are made by the select kernel where a
// CTA has at most 128 of them and no cluster that starts later reads a length that
// another has replaced (1 x 4112 to 4048: 9.6 us, 10.9 with a launch of their own; at
// 256 moves 14.7 and 11.3), else by a grid of their own. All of it goes by the
// table's width: one entry over a budget of 4096 takes 7.8 us for one sequence
// with a table of 8192 slots and outputs of its own, 8.6 in place; 64 sequences
// 15.4 us, but 74 in place with tables of 131072 slots, whose slices and grids
// are sized for them.
EvictPlan evict_plan(const PagedView& c, const EvictArgs& a) {
  EvictPlan p{};
  const long long slots = paged_slots(c);
  p.cluster = 1;
  const long long pairs = (long long)c.n_seqs * c.n_kv;
  if (slots > 8 * EV_THREADS && pairs * EV_CLUSTER <= device_sm_count())
    p.cluster = EV_CLUSTER;
  else
    while (p.cluster < EV_CLUSTER && slots > 8ll * EV_THREADS * p.cluster) p.cluster *= 2;
  const long long per = ((slots + p.cluster - 1) / p.cluster + EV_THREADS - 1) / EV_THREADS * EV_THREADS;
  p.keys = per < EV_MAX_KEYS ? (int)per : EV_MAX_KEYS;
  p.long_slices = per > EV_MAX_KEYS;
  p.moves = a.budget < slots - a.budget ? a.budget : slots - a.budget;
  p.inline_moves = p.moves <= 2 * MV_MOVES * p.cluster && (c.n_kv == 1 || a.lens_out != c.lens);
  return p;
}

}  // namespace

int cache_evict_launches(const PagedView& c, const EvictArgs& a) { return evict_plan(c, a).inline_moves ? 1 : 2; }

cudaError_t launch_cache_evict(const PagedView& c, const EvictArgs& a, cudaStream_t st) {
  const long long pairs = (long long)c.n_seqs * c.n_kv;
  char* p = static_cast<char*>(a.ws);
  EvictLists ls;
  ls.list = (long long)list_len(c);
  const size_t head = up256(4 * pairs), lists = up256(sizeof(int2) * pairs * ls.list);
  ls.count = reinterpret_cast<int32_t*>(p);
  ls.keep = reinterpret_cast<int32_t*>(p + head);
  ls.hole = reinterpret_cast<int2*>(p + 2 * head);
  ls.mover = reinterpret_cast<int2*>(p + 2 * head + lists);
  const EvictPlan pl = evict_plan(c, a);
  if (pairs * pl.cluster > 0x7FFFFFFFll) return cudaErrorInvalidValue;
  auto* select = pl.long_slices ? (pl.inline_moves ? evict_select_kernel<true, true> : evict_select_kernel<true, false>)
                                : (pl.inline_moves ? evict_select_kernel<false, true> : evict_select_kernel<false, false>);
  const size_t smem = sizeof(uint32_t) * pl.keys;
  cudaError_t e = ensure_kernel_smem(reinterpret_cast<const void*>(select), smem);
  if (e != cudaSuccess) return e;
  e = launch_overlapped(select, dim3((unsigned)(pairs * pl.cluster)), EV_THREADS, smem, pl.cluster, st, c, a, ls);
  if (e != cudaSuccess || pl.inline_moves) return e;
  long long parts = (pl.moves + MV_MOVES - 1) / MV_MOVES;
  if (parts < 1) parts = 1;
  if (parts > 65535) parts = 65535;
  return launch_overlapped(evict_move_kernel, dim3((unsigned)pairs, (unsigned)parts), MV_THREADS, 0, 0, st, c, a, ls);
}

}  // namespace qmoe
