// Attention of one new token for each sequence over a paged key-value cache.
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": 16 query heads over 2 KV heads, query head h reads KV head
// h / 8. "Distributed CPU: Zip Fusion Beyond Tensor Parallelism",
// "Two-Dimensional Attention at Long Context": the softmax over parts of the
// context carried by (max, normaliser, weighted output) and joined exactly.
#include <cuda.h>
#include <cudaTypedefs.h>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

// What bounds it: each cached byte is read once and serves the G query heads of
// its KV head, 8 flops a byte at G = 8, so HBM bounds it. 256 sequences of about
// 4054 entries, 16 heads over 2 KV heads of 128, fp32 rows: 167 us, 6.40 TB/s (0.96
// of the measured copy rate); one of 131075: 30.5 us, 4.4 TB/s, of which 20 are the
// copy's, 4 the way to the first copies and 5 the merges and the join; 1 x 4096
// 9.1 us, a chain of latencies.
//
// Work. A row is (sequence, KV head, tile of at most 8 NT query heads); its
// slots are cut into tiles of KT. The tiles of all rows in order are dealt out
// evenly, a contiguous range to each CTA (one CTA per SM) and of that to each
// of its warps, so that a batch of unequal sequences and one long sequence both
// keep every SM busy. A warp finishes the rows that lie inside its range by
// itself; what it has of others it leaves in shared memory (the end of a row
// that began earlier in the merge area, the beginning of one that goes on in
// its own ring), and after the CTA's only barrier these are merged. A row over
// several CTAs leaves a partial in each, which the join kernel finishes: a CTA
// has at most one of a row that began earlier (slot 0) and one of a row that
// begins in it (slot 1).
//
// Loads. Every warp has its own ring of STAGES tiles. It issues its first tiles'
// copies itself; then one more warp, whose lane w serves warp w, looks pages up
// a tile ahead and issues tensor copies (boxes of 64 head dims x up to KT slots
// of a page, 128-byte swizzled) as stages come free, across rows. (With every
// warp issuing its own copies a tile took 438 instructions of a warp, and the
// kernel stopped at 6.5 TB/s even out of L2.)
//
// Products. Scores are S^T = K Q^T with the slots as the rows of a 16 x 8
// fragment and the G heads as its 8 columns, so that a group of 8 heads fills
// the instruction; the output is O^T = V^T P^T with the head dims as rows. The
// instructions are mma.sync: at 8 flops a byte the whole cache needs a tenth of
// their rate, and a fragment's scores are in registers at once.
// fp32 queries are split into three bf16 parts (exact), the probabilities of both
// types of rows into three, and a tile's products are added to the output by a
// rounded fp32 sum: fp32 rows come out at fp32 accuracy, and bf16 rows are what
// fp32 rows of the same queries would be, rounded once. (bf16 rows with two parts,
// up to 2^-17 of a probability, and sums inside the instruction, which are cut
// off: 24 x 1..1025 at 8/8 heads of 64 11.9 instead of 12.7 us, 64 x 4096 with 16
// heads on one KV head 36.3 instead of 37.9, 32 heads of 256 on two 103 instead of
// 122, the other cases within 1 %.)
template <int HDP_, int NT_, bool F32_>
struct PaCfg {
  static constexpr int HDP = HDP_, NT = NT_, QP = F32_ ? 3 : 1, PP = 3;
  static constexpr bool F32 = F32_;
  static constexpr int CHAINS = NT == 1 ? 4 : 2;           // sums of a score side by side (2: the same time, 1.5 times the error)
  static constexpr int KT = HDP == 64 ? 32 : 16;           // slots of a tile: 4 or 8 KB of keys
  // Warps that compute, and one more that feeds them (8 in all have 255 registers a thread), with a ring of at most
  // 192 KB an SM. fp32 rows of 256 are bound by their products: 5 warps with 2 stages 64 x 4096 in 101 us, 4 with 3
  // in 110.
  static constexpr bool WIDE = HDP == 256, WIDE_F32 = WIDE && F32_;
  static constexpr int WARPS = WIDE_F32 ? 5 : WIDE ? 4 : 7;
  static constexpr int STAGES = NT == 1 && !WIDE_F32 ? 3 : 2;
  static constexpr int HALF = KT * 128;                    // 64 head dims of a tile
  static constexpr int KBYTES = HALF * (HDP / 64);
  static constexpr int RING = WARPS * STAGES * 2 * KBYTES;
  static constexpr int HT = 8 * NT;                        // heads of a row
  static constexpr int MROW = HDP + 4;                     // a head's output in shared memory: rows apart by 4 banks
  static constexpr int MERGE = WARPS * HT * MROW * 4;
  static constexpr int SMEM = 1024 + RING + MERGE + 2 * WARPS * HT * 8 + WARPS * STAGES * 20;
  static_assert(HT * MROW * 4 <= STAGES * 2 * KBYTES, "a warp's output fits its ring");
};

struct PaSplit {
  PagedView c;
  const void* q;
  void* out;
  float scale_log2;  // scores in units of log2(e)
  int n_heads, group, head_tiles, box_rows;
  bool at_once;      // a copy brings all head dims (else 64)
  int whole_rows;    // CTAs begin at rows (nothing is joined)
  int4* desc;        // [CTAs] the row that begins there and is joined: (sequence, row, CTAs, 1 if the CTA gave up), or -1
  float2* part_ml;   // [CTAs][2][heads]
  float* part_o;     // [CTAs][2][heads][HDP]
  float* lse;        // [sequences][heads] log2 of the softmax's denominator, with accumulate
  float* scores;     // [sequences][KV heads][slots][group], with accumulate
  int* status;
  unsigned long long wait_ns;
  bool fault;
};

// ``part``: the 64 head dims from 64 part on, or with a box of all parts the first of them.
__device__ __forceinline__ void pa_tma(uint32_t dst, const CUtensorMap* map, int row, int part, int head, int page,
                                       bool at_once, uint64_t* bar) {
  if (at_once)
    asm volatile(
        "cp.async.bulk.tensor.5d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5, "
        "%6}], [%7];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(0), "r"(row), "r"(part), "r"(head), "r"(page), "r"(tc::smem_u32(bar))
        : "memory");
  else
    asm volatile(
        "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
        "[%6];" ::"r"(dst),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(64 * part), "r"(row), "r"(head), "r"(page), "r"(tc::smem_u32(bar))
        : "memory");
}

__device__ __forceinline__ void pa_ldsm(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ void pa_ldsm_t(uint32_t* r, uint32_t addr) {
  asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
               : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
               : "r"(addr)
               : "memory");
}
__device__ __forceinline__ uint32_t pa_transpose(uint32_t v) {
  uint32_t r;
  asm volatile("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(r) : "r"(v));
  return r;
}
__device__ __forceinline__ void pa_mma(float* d, const uint32_t* a, uint32_t b0, uint32_t b1) {
  asm volatile(
      "mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
      : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
      : "r"(a[0]), "r"(a[1]), "r"(a[2]), "r"(a[3]), "r"(b0), "r"(b1));
}

__device__ __forceinline__ float bf_lo(uint32_t u) { return __uint_as_float(u << 16); }
__device__ __forceinline__ float bf_hi(uint32_t u) { return __uint_as_float(u & 0xFFFF0000u); }

__device__ __forceinline__ int pa_tiles(const PagedView& c, int b, int kt) {
  const int n = (paged_len(c, b) + kt - 1) / kt;
  return n > 0 ? n : 1;  // an empty sequence has one tile without entries, which writes its zeros
}

// A walk over tiles: row ``vh`` of sequence ``b``, its tile ``t`` of ``nt``.
struct PaWalk {
  int b, vh, t, nt, len;
};

template <int KT>
__device__ __forceinline__ void pa_seq(const PagedView& c, PaWalk& w) {
  w.len = paged_len(c, w.b);
  w.nt = w.len > 0 ? (w.len + KT - 1) / KT : 1;
}

template <int KT>
__device__ __forceinline__ void pa_step(const PagedView& c, int rows, int by, PaWalk& w) {
  w.t += by;
  if (w.t < w.nt) return;
  w.t = 0;
  if (++w.vh < rows) return;
  w.vh = 0;
  if (++w.b < c.n_seqs) pa_seq<KT>(c, w);  // (behind the last tile the walk is not used)
}

// floor(a * b / d) for b <= d (a share of ``a``): 32-bit division where it does.
__device__ __forceinline__ long long pa_share(long long a, int b, int d) {
  const unsigned long long x = (unsigned long long)a * (unsigned)b;
  return (x >> 32) == 0 ? (long long)((unsigned)x / (unsigned)d) : (long long)(x / (unsigned)d);
}

template <class C>
__global__ void __launch_bounds__(32 * (C::WARPS + 1), 1)
    paged_split_kernel(const PaSplit p, const __grid_constant__ CUtensorMap kmap,
                       const __grid_constant__ CUtensorMap vmap) {
  constexpr int KT = C::KT, W = C::WARPS, ST = C::STAGES, NT = C::NT, HDP = C::HDP, KS = HDP / 16, HT = C::HT;
  constexpr int THREADS = 32 * (W + 1), KB = KT / 16;
  extern __shared__ uint8_t pa_smem_raw[];
  __shared__ int4 s_head[W], s_tail[W];  // what a warp left: (sequence, row, 1 if there, 1 if the row goes on)
  __shared__ long long s_last[W];      // the last tile of the row that a warp's tail begins
  __shared__ int4 s_walk[W];           // a warp's next tile to copy: (sequence, row, tile, tiles left)
  __shared__ int s_abort;
  const uint32_t s0 = tc::smem_u32(pa_smem_raw);
  uint8_t* smem = pa_smem_raw + (((s0 + 1023u) & ~1023u) - s0);
  float* merge_o = reinterpret_cast<float*>(smem + C::RING);                    // [W][HT][MROW]
  float2* merge_ml = reinterpret_cast<float2*>(smem + C::RING + C::MERGE);      // [2: head, tail][W][HT]
  uint64_t* bars = reinterpret_cast<uint64_t*>(merge_ml + 2 * W * HT);          // [W][ST]
  uint64_t* empties = bars + W * ST;                                            // [W][ST]
  uint32_t* masks = reinterpret_cast<uint32_t*>(empties + W * ST);              // [W][ST]
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, tid = threadIdx.x;
  const PagedView& c = p.c;
  const int rows = c.n_kv * p.head_tiles;
  tc::grid_dep_launch();

  if (tid < 2 * W * ST) tc::mbar_init(&bars[tid], 1);
  if (tid == 0) {
    s_abort = 0;
    tc::fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  if (tid < W) s_head[tid] = s_tail[tid] = make_int4(0, 0, 0, 0);
  tc::grid_dep_wait();
  // ---- this CTA's and this warp's share of the tiles, found by every warp for itself: a lane has the sequences
  // lane * q .. lane * q + q - 1, and the tiles ahead of them
  const int q = (c.n_seqs + 31) / 32;
  long long ahead_of = 0;
  for (int b = lane * q; b < min(c.n_seqs, (lane + 1) * q); ++b) ahead_of += pa_tiles(c, b, KT);
  const long long own_tiles = ahead_of;
  long long total;
  if (c.n_seqs == 1) {
    total = __shfl_sync(0xffffffffu, (int)own_tiles, 0);  // (a sequence's tiles are few enough)
    ahead_of = lane > 0 ? total : 0;
  } else {
#pragma unroll
    for (int off = 1; off < 32; off <<= 1) {
      const long long x = __shfl_up_sync(0xffffffffu, ahead_of, off);
      if (lane >= off) ahead_of += x;
    }
    total = __shfl_sync(0xffffffffu, ahead_of, 31);
    ahead_of -= own_tiles;
  }
  total *= rows;
  ahead_of *= rows;
  // CTAs: one for each W tiles (a tile for each warp) as far as there are; those of a single sequence then begin at its rows
  const long long fit = c.n_seqs != 1 ? (total + W - 1) / W : p.whole_rows ? rows : (total / rows + W - 1) / W * rows;
  const int n_ctas = (int)(fit < gridDim.x ? fit : gridDim.x);
  if (blockIdx.x >= n_ctas) {
    if (tid == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);
    return;
  }
  // the row of tile ``x`` (below the total): sequence, row, tile, and the row's first tile
  auto locate = [&](long long x, PaWalk& w) {
    const int holder = __popc(__ballot_sync(0xffffffffu, ahead_of <= x)) - 1;
    long long base = __shfl_sync(0xffffffffu, ahead_of, holder);
    w.b = holder * q;
    pa_seq<KT>(c, w);
    while (x >= base + (long long)w.nt * rows) {
      base += (long long)w.nt * rows;
      ++w.b;
      pa_seq<KT>(c, w);
    }
    x -= base;
    w.vh = (int)((x >> 32) == 0 ? (unsigned)x / (unsigned)w.nt : x / w.nt);
    w.t = (int)(x - (long long)w.vh * w.nt);
  };
  long long C0 = pa_share(total, blockIdx.x, n_ctas), C1 = pa_share(total, blockIdx.x + 1, n_ctas);
  if (p.whole_rows && (c.n_seqs > 1 || n_ctas < rows)) {  // (one sequence's rows, where each has a CTA, begin there already)
    PaWalk w;
    locate(C0, w);
    C0 -= w.t;
    if (C1 < total) {
      locate(C1, w);
      C1 -= w.t;
    }
  }
  const long long T0 = C0 + pa_share(C1 - C0, min(warp, W - 1), W);
  const int count = warp < W ? (int)(C0 + pa_share(C1 - C0, warp + 1, W) - T0) : 0;  // this warp's tiles
  PaWalk seg{};
  if (count > 0) locate(T0, seg);
  __syncthreads();  // the barriers are set up
  if (tid == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 0);

  // ---- loads
  uint8_t* ring = smem + warp * ST * 2 * C::KBYTES;
  uint64_t* full = bars + warp * ST;
  uint32_t* mask_of = masks + warp * ST;
  const int boxes = p.at_once ? 1 : HDP / 64, pieces = KT / p.box_rows, page_mask = (1 << c.page_log2) - 1;
  int left = count;  // tiles still to look up
  PaWalk ahead = seg;
  // a row's queries as B fragments hold them: head lane / 4, dims 2 (lane % 4) + {0, 1, 8, 9} of each 16
  float2 qx[C::F32 ? KS : 1][NT][2];
  uint32_t qf[KS][NT][C::QP][2];
  auto load_q = [&](const PaWalk& w) {
    const int g = w.vh / p.head_tiles, h0 = g * p.group + (w.vh % p.head_tiles) * HT;
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      const int hh = 8 * n + (lane >> 2);
      const long long qo = ((long long)w.b * p.n_heads + h0 + hh) * c.head_dim;
      const bool head = h0 + hh < (g + 1) * p.group;
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int half = 0; half < 2; ++half) {
          const int d = 16 * i + 8 * half + 2 * (lane & 3);
          const bool in = head && d < c.head_dim;
          if constexpr (C::F32)
            qx[i][n][half] = in ? *reinterpret_cast<const float2*>(static_cast<const float*>(p.q) + qo + d)
                                : make_float2(0.f, 0.f);
          else
            qf[i][n][0][half] =
                in ? *reinterpret_cast<const uint32_t*>(static_cast<const __nv_bfloat16*>(p.q) + qo + d) : 0u;
        }
    }
  };
  // The copies of piece i of the tile at ``w`` into stage st of a warp's ring.
  constexpr int PIECES = KT / 8;
  auto copy = [&](const PaWalk& w, int to_warp, int st, int i, int page) {
    const uint32_t dst = tc::smem_u32(smem + (to_warp * ST + st) * 2 * C::KBYTES) + (uint32_t)(i * p.box_rows) * 128u;
    const int row = (w.t * KT + i * p.box_rows) & page_mask, g = w.vh / p.head_tiles;
    uint64_t* bar = &bars[to_warp * ST + st];
#pragma unroll 1
    for (int h = 0; h < boxes; ++h) {
      pa_tma(dst + h * C::HALF, &kmap, row, h, g, page, p.at_once, bar);
      pa_tma(dst + C::KBYTES + h * C::HALF, &vmap, row, h, g, page, p.at_once, bar);
    }
  };
  // which of a tile's slots hold entries: their piece has a page (bits of ``ok``) and they lie below the length
  auto held_of = [&](unsigned ok, int n_in) {
    uint32_t held = 0;
#pragma unroll
    for (int i = 0; i < PIECES; ++i)
      if ((ok >> i) & 1u) held |= (p.box_rows == 32 ? 0xffffffffu : (1u << p.box_rows) - 1u) << (i * p.box_rows);
    return n_in >= 32 ? held : held & (n_in > 0 ? (1u << n_in) - 1u : 0u);
  };
  if (count > 0) {
    // this warp's first ST tiles: lane 8 s + i copies piece i of the s-th
    const int s = lane >> 3, piece = lane & 7;
    PaWalk w{};
#pragma unroll 1
    for (int k = 0; k < ST; ++k) {
      if (k == s) w = ahead;
      if (--left > 0) pa_step<KT>(c, rows, 1, ahead);
    }
    const bool some = s < ST && s < count;
    const int n_in = min(KT, w.len - w.t * KT), slot = w.t * KT + piece * p.box_rows;
    const bool want = some && piece < pieces && piece * p.box_rows < n_in;
    int page = -1;
    if (want) page = __ldg(c.table + (long long)w.b * c.max_pages + (slot >> c.page_log2));
    load_q(seg);
    const bool there = want && (unsigned)page < (unsigned)c.n_pages;
    if (want && !there) record_status(p.status, QMOE_ERR_DEVICE_ARG);
    const unsigned ok = (__ballot_sync(0xffffffffu, there) >> (8 * s)) & 255u;
    const bool dropped = p.fault && blockIdx.x == 0 && warp == 0 && s == 0;  // (the test-only fault)
    if (some && piece == 0 && !dropped) {
      masks[warp * ST + s] = held_of(ok, n_in);
      tc::mbar_expect_tx(&bars[warp * ST + s], (uint32_t)__popc(ok) * (uint32_t)p.box_rows * 4u * HDP);
    }
    __syncwarp();
    if (there && !dropped) copy(w, warp, s, piece, page);
  }
  if (warp < W && lane == 0) s_walk[warp] = make_int4(ahead.b, ahead.vh, ahead.t, left);
  __syncthreads();

  if (warp == W) {
    // ---- the copies of the other warps' later tiles: lane w feeds warp w
    const int4 from = lane < W ? s_walk[lane] : make_int4(0, 0, 0, 0);
    PaWalk w{};
    w.b = from.x;
    if (from.w > 0) pa_seq<KT>(c, w);
    w.vh = from.y;
    w.t = from.z;
    left = from.w;
    int pages[PIECES];
    auto pages_of = [&]() {
#pragma unroll
      for (int i = 0; i < PIECES; ++i) {
        const int slot = w.t * KT + i * p.box_rows;
        pages[i] = left > 0 && i < pieces && slot < w.len
                       ? __ldg(c.table + (long long)w.b * c.max_pages + (slot >> c.page_log2)) : -1;
      }
    };
    pages_of();
    const int to = lane < W ? lane : 0, bar0 = to * ST;
    int st = 0;
    uint32_t ph = 0;
    uint64_t since = tc::global_ns();
    for (int spin = 0; __any_sync(0xffffffffu, left > 0); ++spin) {
      const bool ready = left > 0 && tc::mbar_test_wait(&empties[bar0 + st], ph);
      if (ready) {
        const int n_in = min(KT, w.len - w.t * KT);
        unsigned there = 0;
#pragma unroll
        for (int i = 0; i < PIECES; ++i) {
          const bool want = i < pieces && i * p.box_rows < n_in;
          if (want && (unsigned)pages[i] < (unsigned)c.n_pages)
            there |= 1u << i;
          else if (want)
            record_status(p.status, QMOE_ERR_DEVICE_ARG);
        }
        masks[bar0 + st] = held_of(there, n_in);
        tc::mbar_expect_tx(&bars[bar0 + st], (uint32_t)__popc(there) * (uint32_t)p.box_rows * 4u * HDP);
#pragma unroll
        for (int i = 0; i < PIECES; ++i)
          if ((there >> i) & 1u) copy(w, to, st, i, pages[i]);
        if (--left > 0) pa_step<KT>(c, rows, 1, w);
        pages_of();
        if (++st == ST) {
          st = 0;
          ph ^= 1u;
        }
      }
      if (__any_sync(0xffffffffu, ready)) {
        since = tc::global_ns();
      } else if ((spin & 255) == 0) {
        // (the lanes read their clocks apart and leave together: one that went on would wait for the others' votes)
        const bool over = *(volatile int*)&s_abort || tc::global_ns() - since > p.wait_ns;
        if (__any_sync(0xffffffffu, over)) {
          if (lane == 0) {
            record_status(p.status, QMOE_ERR_TIMEOUT);
            *(volatile int*)&s_abort = 1;
          }
          break;
        }
      }
    }
  }

  // ---- rows
  int stage = 0, done = 0;
  uint32_t phase = 0;
  bool ok = true;
  while (done < count) {
    const int n_tiles = min(count - done, seg.nt - seg.t);
    const int g = seg.vh / p.head_tiles, h0 = g * p.group + (seg.vh % p.head_tiles) * HT;
    const int n_h = min(HT, (g + 1) * p.group - h0);  // heads of this row
    if constexpr (C::F32) {
#pragma unroll
      for (int i = 0; i < KS; ++i)
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            float x0 = qx[i][n][half].x, x1 = qx[i][n][half].y;
#pragma unroll
            for (int part = 0; part < C::QP; ++part) {
              const uint32_t u = tc::pack_bf16x2(x0, x1);
              qf[i][n][part][half] = u;
              x0 -= bf_lo(u);
              x1 -= bf_hi(u);
            }
          }
    }
    float m[NT][2], l[NT][2], o[KS][NT][4];
#pragma unroll
    for (int n = 0; n < NT; ++n) {
      m[n][0] = m[n][1] = -INFINITY;
      l[n][0] = l[n][1] = 0.f;
#pragma unroll
      for (int i = 0; i < KS; ++i) o[i][n][0] = o[i][n][1] = o[i][n][2] = o[i][n][3] = 0.f;
    }
    const int row_t = seg.t;
    float* row_scores = p.scores + ((long long)seg.b * c.n_kv + g) * paged_slots(c) * p.group + (h0 - g * p.group);
#pragma unroll 1
    for (int turn = 0; turn < n_tiles; ++turn) {
      if (ok && !__all_sync(0xffffffffu, tc::mbar_wait(&full[stage], phase, &s_abort, p.wait_ns))) {
        ok = false;
        if (lane == 0) record_status(p.status, QMOE_ERR_TIMEOUT);
      }
      if (!ok) continue;
      const uint32_t held = mask_of[stage];
      uint8_t* tile = ring + stage * 2 * C::KBYTES;
      const uint32_t kt = tc::smem_u32(tile), vt = kt + C::KBYTES;
      constexpr uint32_t FULL = KT == 32 ? 0xffffffffu : (1u << (KT & 31)) - 1u;
      if (held != FULL) {
        // values of slots that hold nothing are set to zero: 0 times whatever lay there need not be 0
        for (int i = lane; i < KT * (HDP / 8); i += 32) {
          const int r = i / (HDP / 8), ch = i % (HDP / 8);
          if (!((held >> r) & 1u))
            *reinterpret_cast<uint4*>(tile + C::KBYTES + (ch >> 3) * C::HALF + r * 128 + (ch & 7) * 16) =
                make_uint4(0, 0, 0, 0);
        }
        tc::fence_proxy_async_smem();  // before a later copy into the same bytes
        __syncwarp();
      }
      // S^T: slots x heads
      float s[KB][NT][4];
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        float sc[C::CHAINS][NT][4];  // sums over every CHAINS-th 16 head dims: dependent products would wait for one another
#pragma unroll
        for (int h = 0; h < C::CHAINS; ++h)
#pragma unroll
          for (int n = 0; n < NT; ++n)
#pragma unroll
            for (int e = 0; e < 4; ++e) sc[h][n][e] = 0.f;
        const int r = 16 * kb + (lane & 15);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint32_t a[4];
          const int ch = 2 * (i & 3) + (lane >> 4);
          pa_ldsm(a, kt + (i >> 2) * C::HALF + tc::sw128_offset(r, ch));
#pragma unroll
          for (int part = C::QP - 1; part >= 0; --part)
#pragma unroll
            for (int n = 0; n < NT; ++n)
              pa_mma(sc[i % C::CHAINS][n], a, qf[i][n][part][0], qf[i][n][part][1]);
        }
#pragma unroll
        for (int n = 0; n < NT; ++n)
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            float x = sc[0][n][e];
#pragma unroll
            for (int h = 1; h < C::CHAINS; ++h) x += sc[h][n][e];
            s[kb][n][e] = x * p.scale_log2;
          }
        if (held != FULL) {
#pragma unroll
          for (int e = 0; e < 4; e += 2)
            if (!((held >> (16 * kb + (lane >> 2) + 4 * e)) & 1u))
#pragma unroll
              for (int n = 0; n < NT; ++n) s[kb][n][e] = s[kb][n][e + 1] = -INFINITY;
        }
      }
      if (p.scores != nullptr) {
        // kept until the denominators are known
        const int j0 = (row_t + turn) * KT + (lane >> 2);
        float* at = row_scores + (long long)j0 * p.group + 2 * (lane & 3);
#pragma unroll
        for (int kb = 0; kb < KB; ++kb)
#pragma unroll
          for (int e = 0; e < 4; e += 2) {
            const int j = 16 * kb + 4 * e;
            if (j0 + j >= seg.len) continue;
#pragma unroll
            for (int n = 0; n < NT; ++n) {
              const int hh = 8 * n + 2 * (lane & 3);
              float* to = at + (long long)j * p.group + 8 * n;
              if ((p.group & 1) == 0) {
                if (hh < n_h) *reinterpret_cast<float2*>(to) = make_float2(s[kb][n][e], s[kb][n][e + 1]);
              } else {
                if (hh < n_h) to[0] = s[kb][n][e];
                if (hh + 1 < n_h) to[1] = s[kb][n][e + 1];
              }
            }
          }
      }
      // running maximum; the output is rescaled where one grew
      uint32_t pf[KB][NT][C::PP][2];  // P^T as B fragments: bf16 parts, slots 0-7 and 8-15
      bool grew = false;
      float mn[NT][2];
#pragma unroll
      for (int n = 0; n < NT; ++n)
#pragma unroll
        for (int e = 0; e < 2; ++e) {
          float x = fmaxf(s[0][n][e], s[0][n][e + 2]);
#pragma unroll
          for (int kb = 1; kb < KB; ++kb) x = fmaxf(x, fmaxf(s[kb][n][e], s[kb][n][e + 2]));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 4));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 8));
          x = fmaxf(x, __shfl_xor_sync(0xffffffffu, x, 16));
          mn[n][e] = fmaxf(m[n][e], x);
          grew |= mn[n][e] > m[n][e];
        }
      if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
        for (int n = 0; n < NT; ++n) {
          float al[2];
#pragma unroll
          for (int e = 0; e < 2; ++e) {
            al[e] = m[n][e] == mn[n][e] ? 1.f : exp2f(m[n][e] - mn[n][e]);
            m[n][e] = mn[n][e];
            l[n][e] *= al[e];
          }
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            o[i][n][0] *= al[0];
            o[i][n][1] *= al[1];
            o[i][n][2] *= al[0];
            o[i][n][3] *= al[1];
          }
        }
      }
#pragma unroll
      for (int n = 0; n < NT; ++n) {
        const float r0 = m[n][0] == -INFINITY ? 0.f : m[n][0], r1 = m[n][1] == -INFINITY ? 0.f : m[n][1];
#pragma unroll
        for (int kb = 0; kb < KB; ++kb) {
          const float p0 = exp2f(s[kb][n][0] - r0), p1 = exp2f(s[kb][n][1] - r1);
          const float p2 = exp2f(s[kb][n][2] - r0), p3 = exp2f(s[kb][n][3] - r1);
          l[n][0] += p0 + p2;
          l[n][1] += p1 + p3;
          float r[4] = {p0, p1, p2, p3};
#pragma unroll
          for (int part = 0; part < C::PP; ++part) {
            const uint32_t ua = tc::pack_bf16x2(r[0], r[1]), ub = tc::pack_bf16x2(r[2], r[3]);
            pf[kb][n][part][0] = pa_transpose(ua);
            pf[kb][n][part][1] = pa_transpose(ub);
            r[0] -= bf_lo(ua);
            r[1] -= bf_hi(ua);
            r[2] -= bf_lo(ub);
            r[3] -= bf_hi(ub);
          }
        }
      }
      // O^T += V^T P^T: head dims x heads
#pragma unroll
      for (int kb = 0; kb < KB; ++kb) {
        const int r = 16 * kb + (lane & 7) + 8 * (lane >> 4);
#pragma unroll
        for (int i = 0; i < KS; ++i) {
          uint32_t a[4];
          const int ch = 2 * (i & 3) + ((lane >> 3) & 1);
          pa_ldsm_t(a, vt + (i >> 2) * C::HALF + tc::sw128_offset(r, ch));
#pragma unroll
          for (int n = 0; n < NT; ++n) {
            // a tile's products apart, added by a rounded sum: the instruction's own sums are cut off, which adds up
            // over a long row
            float x[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
            for (int part = C::PP - 1; part >= 0; --part) pa_mma(x, a, pf[kb][n][part][0], pf[kb][n][part][1]);
#pragma unroll
            for (int e = 0; e < 4; ++e) o[i][n][e] += x[e];
          }
        }
      }
      __syncwarp();  // every lane has read the stage
      if (lane == 0) tc::mbar_arrive(&empties[warp * ST + stage]);
      if (++stage == ST) {
        stage = 0;
        phase ^= 1u;
      }
    }
    const PaWalk row = seg;
    done += n_tiles;
    if (done < count) {
      pa_step<KT>(c, rows, n_tiles, seg);
      load_q(seg);
    }
    // ---- the row's result, or what this warp leaves of it
    const bool begins = row.t == 0, goes_on = row.t + n_tiles < row.nt;
    const bool whole = begins && !goes_on;
    float* left_o = begins ? reinterpret_cast<float*>(ring) : merge_o + warp * HT * C::MROW;
    float2* left_ml = merge_ml + (begins ? W + warp : warp) * HT;
#pragma unroll
    for (int n = 0; n < NT; ++n)
#pragma unroll
      for (int e = 0; e < 2; ++e) {
        float x = l[n][e];
        x += __shfl_xor_sync(0xffffffffu, x, 4);
        x += __shfl_xor_sync(0xffffffffu, x, 8);
        x += __shfl_xor_sync(0xffffffffu, x, 16);
        const int hh = 8 * n + 2 * (lane & 3) + e;
        if (!whole) {
          if (lane < 4) left_ml[hh] = make_float2(m[n][e], x);
#pragma unroll
          for (int i = 0; i < KS; ++i) {
            left_o[hh * C::MROW + 16 * i + (lane >> 2)] = o[i][n][e];
            left_o[hh * C::MROW + 16 * i + 8 + (lane >> 2)] = o[i][n][e + 2];
          }
          continue;
        }
        if (hh >= n_h) continue;
        const long long head = (long long)row.b * p.n_heads + h0 + hh;
        const float il = x == 0.f ? 0.f : 1.f / x;
        if (lane < 4 && p.lse != nullptr) p.lse[head] = x == 0.f ? 0.f : m[n][e] + log2f(x);
#pragma unroll
        for (int i = 0; i < KS; ++i)
#pragma unroll
          for (int half = 0; half < 2; ++half) {
            const int d = 16 * i + 8 * half + (lane >> 2);
            if (d >= c.head_dim) continue;
            const float y = o[i][n][e + 2 * half] * il;
            if (C::F32)
              static_cast<float*>(p.out)[head * c.head_dim + d] = y;
            else
              static_cast<__nv_bfloat16*>(p.out)[head * c.head_dim + d] = __float2bfloat16_rn(y);
          }
      }
    if (!whole && lane == 0) {
      (begins ? s_tail : s_head)[warp] = make_int4(row.b, row.vh, 1, goes_on);
      if (begins) s_last[warp] = T0 + done - n_tiles + row.nt - 1;
    }
  }
  __syncthreads();
  if (*(volatile int*)&s_abort) {
    // a wait ran out: nothing is issued any more; the copies still in flight land before the CTA leaves
    if (tid == 0) p.desc[blockIdx.x] = make_int4(-1, 0, 0, 1);
    if (warp < W && lane == 0) {
      volatile int never = 0;
      for (int s = stage; s < stage + ST; ++s)
        tc::mbar_wait(&full[s % ST], s < ST ? phase : phase ^ 1u, &never, 1000000ull);
    }
    return;
  }

  // ---- rows over several warps: the beginning that a warp left, then the ends that the next ones did
  const unsigned heads = __ballot_sync(0xffffffffu, lane < W && s_head[lane < W ? lane : 0].z);
  const unsigned ends = __ballot_sync(0xffffffffu, lane < W && s_head[lane < W ? lane : 0].z && !s_head[lane < W ? lane : 0].w);
  const unsigned tails = __ballot_sync(0xffffffffu, lane < W && s_tail[lane < W ? lane : 0].z);
  auto merge = [&](int first, bool began) {  // first: the warp of the row's first part; began: that is its tail
    const unsigned after = heads & ~((1u << first) - 1u) & (began ? ~(1u << first) : ~0u);
    const unsigned end = ends & after;
    const bool over = end != 0;  // the row ends in this CTA
    const unsigned mine = over ? after & ((end & (0u - end)) * 2u - 1u) : after;  // warps with another part of it
    const int4 at = began ? s_tail[first] : s_head[first];
    const int g = at.y / p.head_tiles, h0 = g * p.group + (at.y % p.head_tiles) * HT;
    const int n_h = min(HT, (g + 1) * p.group - h0);
    const long long part = ((long long)blockIdx.x * 2 + (began ? 1 : 0)) * HT;
    const float* tail_o = reinterpret_cast<const float*>(smem + first * ST * 2 * C::KBYTES);
    for (int i = tid; i < n_h * (HDP / 4); i += THREADS) {
      const int hh = i / (HDP / 4), d = 4 * (i % (HDP / 4));
      float2 ml[W + 1];
      float4 x[W + 1];
#pragma unroll
      for (int w = 0; w <= W; ++w) {  // the tail last
        ml[w] = make_float2(-INFINITY, 0.f);
        x[w] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (w < W ? (mine >> w) & 1u : began) {
          ml[w] = merge_ml[(w < W ? w : W + first) * HT + hh];
          x[w] = *reinterpret_cast<const float4*>((w < W ? merge_o + w * HT * C::MROW : tail_o) + hh * C::MROW + d);
        }
      }
      float M = -INFINITY, L = 0.f;
#pragma unroll
      for (int w = 0; w <= W; ++w) M = fmaxf(M, ml[w].x);
      const float ref = M == -INFINITY ? 0.f : M;
      float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
      for (int w = 0; w <= W; ++w) {
        const float f = exp2f(ml[w].x - ref);
        L = fmaf(ml[w].y, f, L);
        acc.x = fmaf(x[w].x, f, acc.x);
        acc.y = fmaf(x[w].y, f, acc.y);
        acc.z = fmaf(x[w].z, f, acc.z);
        acc.w = fmaf(x[w].w, f, acc.w);
      }
      if (!began || !over) {
        if (d == 0) p.part_ml[part + hh] = make_float2(M, L);
        *reinterpret_cast<float4*>(&p.part_o[(part + hh) * HDP + d]) = acc;
        continue;
      }
      const float il = L == 0.f ? 0.f : 1.f / L;
      const long long head = (long long)at.x * p.n_heads + h0 + hh;
      if (d == 0 && p.lse != nullptr) p.lse[head] = L == 0.f ? 0.f : M + log2f(L);
      if (d < c.head_dim) {
        if (C::F32)
          *reinterpret_cast<float4*>(static_cast<float*>(p.out) + head * c.head_dim + d) =
              make_float4(acc.x * il, acc.y * il, acc.z * il, acc.w * il);
        else
          *reinterpret_cast<uint2*>(static_cast<__nv_bfloat16*>(p.out) + head * c.head_dim + d) =
              make_uint2(tc::pack_bf16x2(acc.x * il, acc.y * il), tc::pack_bf16x2(acc.z * il, acc.w * il));
      }
    }
    if (began && !over && tid == 0) {
      // the last CTA whose share begins at or before the row's last tile
      const int owner = (int)(((unsigned long long)(s_last[first] + 1) * (unsigned)n_ctas - 1) / (unsigned long long)total);
      p.desc[blockIdx.x] = make_int4(at.x, at.y, owner - (int)blockIdx.x + 1, 0);
    }
  };
  // a row from the CTA before comes first (no warp ahead of its part has begun one), then each that a warp began
  const int first_head = __ffs(heads) - 1;
  bool from_before = heads != 0 && (tails & ((1u << (first_head & 31)) - 1u)) == 0;
#pragma unroll 1
  for (unsigned left_tails = tails; from_before || left_tails != 0;) {
    const int first = from_before ? first_head : __ffs(left_tails) - 1;
    merge(first, !from_before);
    if (!from_before) left_tails &= left_tails - 1u;
    from_before = false;
  }
}

// Joins the partials of a row over several CTAs: one CTA per (CTA in which a
// row may begin, head of the row). out = sum O_i 2^(m_i - M) / sum l_i 2^(m_i - M).
// A latency of about 3 us behind the split kernel (it starts while that ends).
struct PaJoin {
  const int4* desc;
  const float2* part_ml;
  const float* part_o;
  void* out;
  float* lse;
  int n_heads, group, head_tiles, head_tile, head_dim, hdp;
  bool f32;
};

constexpr int PJ_THREADS = 256;

__global__ void __launch_bounds__(PJ_THREADS) paged_join_kernel(const PaJoin p) {
  __shared__ float fs[PJ_THREADS], red[PJ_THREADS / 32], acc_s[PJ_THREADS * 4];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int4 d = p.desc[blockIdx.x];
  if (d.x < 0) return;
  const int hh = blockIdx.y, tid = threadIdx.x, g = d.y / p.head_tiles;
  const int h0 = g * p.group + (d.y % p.head_tiles) * p.head_tile;
  if (h0 + hh >= (g + 1) * p.group) return;
  // partial i: the beginning in slot 1 of the first CTA, then slot 0 of the next ones
  auto at = [&](int i) { return ((long long)(blockIdx.x + i) * 2 + (i == 0 ? 1 : 0)) * p.head_tile + hh; };
  const int lanes = p.hdp / 4, groups = PJ_THREADS / lanes;  // lanes over the head dims, groups over the partials
  const int grp = tid / lanes, col = 4 * (tid % lanes);
  float M = -INFINITY, L = 0.f;
  float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
  constexpr int U = 8;
  for (int i0 = 0; i0 < d.z; i0 += U * groups) {
    // the partials are on their way while their maxima are compared
    const int n = min(U * groups, d.z - i0);
    const float2 ml = tid < n ? p.part_ml[at(i0 + tid)] : make_float2(-INFINITY, 0.f);
    float4 x[U];
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = grp + k * groups;
      x[k] = i < n ? *reinterpret_cast<const float4*>(&p.part_o[at(i0 + i) * p.hdp + col]) : make_float4(0.f, 0.f, 0.f, 0.f);
    }
    float mx = ml.x;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, off));
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = mx;
    __syncthreads();
    mx = M;
#pragma unroll
    for (int w = 0; w < PJ_THREADS / 32; ++w) mx = fmaxf(mx, red[w]);
    const float ref = mx == -INFINITY ? 0.f : mx;
    const float old = exp2f(M - ref), f = exp2f(ml.x - ref);
    M = mx;
    fs[tid] = f;
    float sum = ml.y * f;
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, off);
    __syncthreads();
    if ((tid & 31) == 0) red[tid >> 5] = sum;
    __syncthreads();
    L *= old;
#pragma unroll
    for (int w = 0; w < PJ_THREADS / 32; ++w) L += red[w];
    acc.x *= old;
    acc.y *= old;
    acc.z *= old;
    acc.w *= old;
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const float fi = fs[min(grp + k * groups, PJ_THREADS - 1)];  // (0 behind the last partial)
      acc.x = fmaf(x[k].x, fi, acc.x);
      acc.y = fmaf(x[k].y, fi, acc.y);
      acc.z = fmaf(x[k].z, fi, acc.z);
      acc.w = fmaf(x[k].w, fi, acc.w);
    }
  }
  __syncthreads();
  *reinterpret_cast<float4*>(&acc_s[4 * tid]) = acc;
  __syncthreads();
  const long long head = (long long)d.x * p.n_heads + h0 + hh;
  const float il = L == 0.f ? 0.f : 1.f / L;
  if (tid == 0 && p.lse != nullptr) p.lse[head] = L == 0.f ? 0.f : M + log2f(L);
  if (tid < p.head_dim) {
    float x = 0.f;
    for (int k = 0; k < groups; ++k) x += acc_s[k * p.hdp + tid];
    if (p.f32)
      static_cast<float*>(p.out)[head * p.head_dim + tid] = x * il;
    else
      static_cast<__nv_bfloat16*>(p.out)[head * p.head_dim + tid] = __float2bfloat16_rn(x * il);
  }
}

// weight[b][g][j] += sum over the group's heads of 2^(score - lse). The scores
// (4 bytes a head and slot, 1/16 of the cache at 8 heads of 128) come back out of
// L2: 64 sequences of up to 8191 entries, 25 MB in 8 us, with its start. Where one
// of the ``ctas`` CTAs gave up, scores and denominators are missing and no weight
// is touched (asking costs 0.4 us; behind the loads instead of ahead of them 0.5).
// (Plain pointers: the kernel that writes scores and lse still runs when this one starts.)
__global__ void __launch_bounds__(256) paged_weight_kernel(const PagedView c, const float* scores, const float* lse,
                                                           int n_heads, int group, const int4* desc, int ctas) {
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int pair = blockIdx.x, b = pair / c.n_kv, g = pair % c.n_kv;
  const int n = paged_len(c, b);
  const long long base = (long long)pair * paged_slots(c);
  const float* ls = lse + (long long)b * n_heads + (long long)g * group;
  float ls8[8];  // (the compiler cannot keep them: a store might change them)
#pragma unroll
  for (int h = 0; h < 8; ++h) ls8[h] = group == 8 ? ls[h] : 0.f;
  int gave_up = 0;
  for (int i = threadIdx.x; i < ctas; i += 256) gave_up |= desc[i].w;
  if (__syncthreads_or(gave_up)) return;
  constexpr int U = 4;  // slots of a thread at a time: all loads ahead of the stores
  for (int j0 = blockIdx.y * 256 * U + threadIdx.x; j0 < n; j0 += gridDim.y * 256 * U) {
    float w[U], old[U];
    if (group == 8) {
      float4 x[U], y[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int j = min(j0 + 256 * k, n - 1);
        const float4* s = reinterpret_cast<const float4*>(scores + (base + j) * 8);
        x[k] = s[0];
        y[k] = s[1];
        old[k] = c.weight[base + j];
      }
#pragma unroll
      for (int k = 0; k < U; ++k)
        w[k] = ((exp2f(x[k].x - ls8[0]) + exp2f(x[k].y - ls8[1])) + (exp2f(x[k].z - ls8[2]) + exp2f(x[k].w - ls8[3]))) +
               ((exp2f(y[k].x - ls8[4]) + exp2f(y[k].y - ls8[5])) + (exp2f(y[k].z - ls8[6]) + exp2f(y[k].w - ls8[7])));
    } else {
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int j = min(j0 + 256 * k, n - 1);
        old[k] = c.weight[base + j];
        w[k] = 0.f;
        for (int h = 0; h < group; ++h) w[k] += exp2f(scores[(base + j) * group + h] - ls[h]);
      }
    }
#pragma unroll
    for (int k = 0; k < U; ++k)
      if (j0 + 256 * k < n) c.weight[base + j0 + 256 * k] = old[k] + w[k];
  }
}

struct PaPlan {
  int hdp, nt, head_tile, head_tiles, ctas;
  size_t desc, ml, o, lse, scores, total;
};

size_t up256(size_t v) { return (v + 255) & ~size_t(255); }

PaPlan pa_plan(const PagedView& c, int n_heads, bool f32, bool accumulate, int ctas) {
  PaPlan p{};
  const int group = n_heads / c.n_kv;
  p.hdp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  // A group of more than 8 heads is cut into rows of 8, or of 16 for bf16 queries over 32 MB and more: rows of 8
  // read the cache once each, the second time out of L2 where it is not too large, and take less code, fewer
  // registers and a stage more. bf16, G = 16: 1 x 4096 8.9 us with 8 against 11.2 with 16, 8 x 3000 11.6 against
  // 12.9, 32 x 4096 of one KV head of 64 (32 MB) 19.2 against 17.5, 64 x 4096 of two KV heads of 128 78.7 against
  // 62.4 and of 256 171 against 122 (16 x 2000 of one of 256, at the border, 20.0 against 22.6); G = 10, 64 x 4096
  // 77.0 against 59.0. fp32, whose queries are three parts, 64 x 4096: 79.5 against 77.5 with spills, 1 x 4096 8.8
  // against 13.7, so fp32 has rows of 8 only.
  const double bytes = 4.0 * c.n_seqs * c.n_kv * (double)paged_slots(c) * c.head_dim;
  p.nt = !f32 && group > 8 && bytes >= 32.0 * (1 << 20) ? 2 : 1;
  p.head_tile = 8 * p.nt;
  p.head_tiles = (group + p.head_tile - 1) / p.head_tile;
  p.ctas = ctas;
  size_t o = 0;
  p.desc = o;   o += up256(sizeof(int4) * ctas);
  p.ml = o;     o += up256(sizeof(float2) * ctas * 2 * p.head_tile);
  p.o = o;      o += up256(sizeof(float) * ctas * 2 * p.head_tile * (size_t)p.hdp);
  p.lse = o;    o += accumulate ? up256(sizeof(float) * (size_t)c.n_seqs * n_heads) : 0;
  p.scores = o; o += accumulate ? up256(sizeof(float) * (size_t)c.n_seqs * n_heads * (size_t)paged_slots(c)) : 0;
  p.total = o;
  return p;
}

constexpr int PA_MAX_CTAS = 256;  // the workspace does not depend on the device

// A pool as a tensor map. With ``hdp`` == hd, [64 head dims][slot of a page][hd /
// 64][KV head][page] and boxes of all head dims, 64 by 64; else [head dim][slot
// of a page][KV head][page] and boxes of 64, where head dims from hd on read as
// zero (split in 64s, the last box would read what lies behind the head).
bool pa_encode(CUtensorMap* m, const void* base, const PagedView& c, int box_rows, int hdp) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const bool at_once = hdp == c.head_dim;
  const cuuint64_t page = (cuuint64_t)1 << c.page_log2, kv = (cuuint64_t)c.n_kv, pages = (cuuint64_t)c.n_pages;
  // (a dimension of one element never steps: its stride may be anything that is valid)
  const cuuint64_t ss = (cuuint64_t)c.slot_stride * 2, hs = (cuuint64_t)(c.n_kv > 1 ? c.head_stride : c.slot_stride) * 2,
                   ps = (cuuint64_t)(c.n_pages > 1 ? c.page_stride : c.slot_stride) * 2;
  const cuuint64_t dims5[5] = {64, page, (cuuint64_t)hdp / 64, kv, pages}, dims4[4] = {(cuuint64_t)c.head_dim, page, kv, pages};
  const cuuint64_t strides5[4] = {ss, 128, hs, ps}, strides4[3] = {ss, hs, ps};
  const cuuint32_t box5[5] = {64, (cuuint32_t)box_rows, (cuuint32_t)hdp / 64, 1, 1}, box4[4] = {64, (cuuint32_t)box_rows, 1, 1};
  const cuuint32_t estr[5] = {1, 1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, at_once ? 5 : 4, const_cast<void*>(base), at_once ? dims5 : dims4,
            at_once ? strides5 : strides4, at_once ? box5 : box4, estr, CU_TENSOR_MAP_INTERLEAVE_NONE,
            CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B, CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_split(PaSplit& s, int ctas, cudaStream_t st) {
  s.box_rows = 1 << s.c.page_log2;
  if (s.box_rows > C::KT) s.box_rows = C::KT;
  CUtensorMap km, vm;
  // (with a page smaller than a tile the parts of a box would not land where the tile has them)
  s.at_once = s.c.head_dim == C::HDP && s.box_rows == C::KT;
  const int parts = s.at_once ? C::HDP : 0;
  if (!pa_encode(&km, s.c.k, s.c, s.box_rows, parts) || !pa_encode(&vm, s.c.v, s.c, s.box_rows, parts))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_kernel_smem(reinterpret_cast<const void*>(paged_split_kernel<C>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(paged_split_kernel<C>, dim3(ctas), 32 * (C::WARPS + 1), C::SMEM, 0, st, s, km, vm);
}

template <bool F32, int NT>
cudaError_t pick_split(PaSplit& s, const PaPlan& pl, cudaStream_t st) {
  if (pl.hdp == 64) return launch_split<PaCfg<64, NT, F32>>(s, pl.ctas, st);
  if (pl.hdp == 128) return launch_split<PaCfg<128, NT, F32>>(s, pl.ctas, st);
  return launch_split<PaCfg<256, NT, F32>>(s, pl.ctas, st);
}

}  // namespace

size_t paged_attention_ws_bytes(const PagedView& c, int n_heads, bool accumulate) {
  return pa_plan(c, n_heads, false, accumulate, PA_MAX_CTAS).total;
}

// Rows of at most 512 slots are not cut between CTAs: a row more or less for a
// CTA costs no more than the second launch that joins (bf16, 64 sequences of 300 to
// 500 entries: 12.0 us whole, 15.6 cut; 256: 27.1 and 31.4; 8: 9.3 and 9.4; at 1024
// slots 8 sequences take 14.0 and 9.8).
static bool pa_whole_rows(const PagedView& c) { return paged_slots(c) <= 512; }

int paged_attention_launches(const PagedView& c, int, bool accumulate) {
  return 1 + (pa_whole_rows(c) ? 0 : 1) + (accumulate ? 1 : 0);
}

cudaError_t launch_paged_attention(const PagedView& c, const PagedAttnArgs& a, cudaStream_t st) {
  int ctas = device_sm_count();
  if (ctas > PA_MAX_CTAS) ctas = PA_MAX_CTAS;
  const PaPlan pl = pa_plan(c, a.n_heads, a.f32, a.accumulate, PA_MAX_CTAS);
  char* ws = static_cast<char*>(a.ws);
  PaSplit s{};
  s.c = c;
  s.q = a.q;
  s.out = a.out;
  s.scale_log2 = a.scale * 1.4426950408889634f;
  s.n_heads = a.n_heads;
  s.group = a.n_heads / c.n_kv;
  s.head_tiles = pl.head_tiles;
  s.whole_rows = pa_whole_rows(c);
  s.desc = reinterpret_cast<int4*>(ws + pl.desc);
  s.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
  s.part_o = reinterpret_cast<float*>(ws + pl.o);
  s.lse = a.accumulate ? reinterpret_cast<float*>(ws + pl.lse) : nullptr;
  s.scores = a.accumulate ? reinterpret_cast<float*>(ws + pl.scores) : nullptr;
  s.status = a.status;
  s.wait_ns = a.wait_ns;
  s.fault = a.fault;
  PaPlan run = pl;
  run.ctas = ctas;
  cudaError_t e = a.f32 ? pick_split<true, 1>(s, run, st)
                        : run.nt == 1 ? pick_split<false, 1>(s, run, st) : pick_split<false, 2>(s, run, st);
  if (e != cudaSuccess) return e;
  PaJoin j{};
  j.desc = s.desc;
  j.part_ml = s.part_ml;
  j.part_o = s.part_o;
  j.out = a.out;
  j.lse = s.lse;
  j.n_heads = a.n_heads;
  j.group = s.group;
  j.head_tiles = pl.head_tiles;
  j.head_tile = pl.head_tile;
  j.head_dim = c.head_dim;
  j.hdp = pl.hdp;
  j.f32 = a.f32;
  if (!s.whole_rows)
    e = launch_overlapped(paged_join_kernel, dim3(ctas, pl.head_tile < s.group ? pl.head_tile : s.group), PJ_THREADS, 0,
                          0, st, j);
  if (e != cudaSuccess || !a.accumulate) return e;
  // about 8 CTAs an SM over all (sequence, KV head) pairs
  const long long pairs = (long long)c.n_seqs * c.n_kv;
  long long parts = (paged_slots(c) + 1023) / 1024, most = (8ll * ctas + pairs - 1) / pairs;
  if (parts > most) parts = most;
  return launch_overlapped(paged_weight_kernel, dim3((unsigned)pairs, (unsigned)parts), 256, 0, 0, st, c, s.scores,
                           s.lse, a.n_heads, s.group, s.desc, ctas);
}

}  // namespace qmoe
