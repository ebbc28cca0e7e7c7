// Causal attention of packed rows (prompts, parts of prompts, single tokens of
// many sequences) over a paged key-value cache. Defined in include/qmoe.h.
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": 16 query heads over 2 KV heads, causal. Pages and packed rows have
// no counterpart there.
#include <cuda.h>
#include <cudaTypedefs.h>

#include <cfloat>
#include <cmath>

#include "paged.cuh"
#include "rope.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

struct PrefillView {
  PagedView c;
  PrefillArgs a;
  float scale_log2;  // scores in units of log2(e)
  int group;         // query heads of a KV head
};

// The rows of sequence b: (first row, rows, entries, entries before the first row), no
// rows where they do not lie in the call's.
struct PrefillRows {
  int first, count, len, before;
};
__device__ __forceinline__ PrefillRows prefill_rows(const PrefillView& p, int b) {
  PrefillRows r{p.a.first[b], p.a.count[b], paged_len(p.c, b), 0};
  if (r.count < 0) r.count = 0;
  if (r.count > 0 && (r.first < 0 || (long long)r.first + r.count > p.a.n_rows)) {
    record_status(p.a.status, QMOE_ERR_DEVICE_ARG);
    r.count = 0;
  }
  r.before = r.len - r.count;
  return r;
}

// ---------------------------------------------------------------- work of a CTA
// A tile is ``span`` positions of a sequence for the query heads of one "head
// row" (a KV head's heads, or 128 of them at most). All tiles in order, head row by
// head row, sequence by sequence, are dealt out evenly over the CTAs by their cost,
// the entries that they see and ``tile_cost`` more; a cut inside a tile falls between
// key blocks, at least PF_MIN_BLOCKS from its ends. So a CTA has whole tiles, and at
// most one part of a tile that began in an earlier CTA (slot 0) and one of a tile that
// goes on in a later one (slot 1); the join kernel puts those together.
constexpr int PF_KEYS = 64, PF_MIN_BLOCKS = 4, PF_ITEMS = 4;

struct PfTiling {
  int span, head_rows, row_heads;  // positions of a tile; head rows in all, of a KV head's heads row_heads each
  int ctas, tile_cost, v_parts;    // v_parts: head rows that share their query heads, with 128 head dims of the values each
  int4* desc;  // [CTAs][2] a part of a tile: (sequence or -1, tile, head row, 1 if it is the tile's last)
};

struct PfItem {
  int b, t, row, kb0, kb1, first, count, len, before, slot;  // b -1: no more; slot -1: a whole tile
};

__device__ __forceinline__ long long pf_cost(long long tiles, long long each, int span) {
  return tiles * each + span * (tiles * (tiles + 1) / 2);
}
__device__ __forceinline__ int pf_blocks(const PrefillRows& r, int t, int span) {
  const int end = r.before + min((t + 1) * span, r.count);
  return end > 0 ? (end + PF_KEYS - 1) / PF_KEYS : 0;
}

struct PfCut {
  int row, b, t, kb;
};

// The place ``x`` (in units of cost, inside sequence b) cuts the sequence's tiles at.
__device__ __forceinline__ PfCut pf_cut(const PrefillRows& r, int row, int b, long long x, int span, int tile_cost) {
  const long long before = (long long)max(r.before, 0) + tile_cost;
  // the tile whose sum of costs reaches x: near the root of the quadratic, then exactly
  const float half = (float)before + 0.5f * span, xf = (float)x;
  long long t = (long long)(2.f * xf / (half + sqrtf(half * half + 2.f * span * xf)));
  const int tiles = (r.count + span - 1) / span;
  t = max(0ll, min(t, (long long)tiles - 1));
  while (t > 0 && pf_cost(t, before, span) > x) --t;
  while (t + 1 < tiles && pf_cost(t + 1, before, span) <= x) ++t;
  const int blocks = pf_blocks(r, (int)t, span);
  const long long off = x - pf_cost(t, before, span) - tile_cost + PF_KEYS / 2;
  int kb = off > 0 ? (int)(off / PF_KEYS) : 0;
  if (kb < PF_MIN_BLOCKS) kb = 0;
  if (blocks - kb < PF_MIN_BLOCKS && kb > 0) return PfCut{row, b, (int)t + 1, 0};
  return PfCut{row, b, (int)t, kb};
}

__device__ __forceinline__ long long pf_sequence_cost(const PrefillRows& r, int span, int tile_cost) {
  return r.count > 0 ? pf_cost((r.count + span - 1) / span, (long long)max(r.before, 0) + tile_cost, span) : 0;
}
__device__ __forceinline__ long long pf_warp_sum(long long v) {  // inclusive, over the lanes
#pragma unroll
  for (int d = 1; d < 32; d *= 2) {
    const long long o = __shfl_up_sync(0xffffffffu, v, d);
    if ((int)(threadIdx.x & 31) >= d) v += o;
  }
  return v;
}

// Where this CTA's work begins and ends, by one warp: a lane sums a run of sequences, the run that a cut falls
// into is looked at again, a lane a sequence.
__device__ __forceinline__ void pf_share(const PrefillView& p, const PfTiling& w, PfCut (&cuts)[2]) {
  const int lane = threadIdx.x & 31, run = (p.c.n_seqs + 31) / 32;
  long long mine = 0;
#pragma unroll 4
  for (int i = 0; i < run; ++i) {
    const int b = lane * run + i;
    if (b < p.c.n_seqs) mine += pf_sequence_cost(prefill_rows(p, b), w.span, w.tile_cost);
  }
  const long long end = pf_warp_sum(mine), total = __shfl_sync(0xffffffffu, end, 31);
  cuts[0] = cuts[1] = PfCut{w.head_rows, 0, 0, 0};
  if (total == 0) return;
  // (where the shares are cut need not be exact, only the same in both CTAs and in order; fp32 products are)
  const long long all = total * w.head_rows;
  const float per = (float)all / (float)w.ctas;
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    const int i = blockIdx.x + k;
    if (i >= w.ctas) break;
    const long long x = min((long long)(per * (float)i), all - 1);
    int row = (int)((float)x / (float)total);
    while (row > 0 && row * total > x) --row;
    while ((row + 1) * total <= x) ++row;
    long long at = x - row * total;  // inside the sequences' costs
    const int src = __ffs(__ballot_sync(0xffffffffu, end > at)) - 1;
    at -= __shfl_sync(0xffffffffu, end - mine, src);
    const int first = src * run, behind = min(first + run, p.c.n_seqs);
    for (int b0 = first; b0 < behind; b0 += 32) {
      const PrefillRows r = b0 + lane < behind ? prefill_rows(p, b0 + lane) : PrefillRows{0, 0, 0, 0};
      const long long cost = pf_sequence_cost(r, w.span, w.tile_cost), sum = pf_warp_sum(cost);
      const unsigned over = __ballot_sync(0xffffffffu, sum > at);
      if (over) {
        const int l = __ffs(over) - 1;
        PrefillRows s;
        s.first = 0;
        s.count = __shfl_sync(0xffffffffu, r.count, l);
        s.len = __shfl_sync(0xffffffffu, r.len, l);
        s.before = s.len - s.count;
        cuts[k] = pf_cut(s, row, b0 + l, at - __shfl_sync(0xffffffffu, sum - cost, l), w.span, w.tile_cost);
        break;
      }
      at -= __shfl_sync(0xffffffffu, sum, 31);
    }
  }
}

// Walks a CTA's share; one warp, whose lanes hold the rows of 32 sequences.
struct PfWalk {
  PfCut at, end;
  PrefillRows mine;
  int window;
  bool whole;  // the tile is taken from its first block on

  __device__ __forceinline__ void look(const PrefillView& p, int b) {
    window = b & ~31;
    const int s = window + (int)(threadIdx.x & 31);
    mine = s < p.c.n_seqs ? prefill_rows(p, s) : PrefillRows{0, 0, 0, 0};
  }
  __device__ __forceinline__ PrefillRows rows(int b) const {
    PrefillRows r;
    r.first = __shfl_sync(0xffffffffu, mine.first, b & 31);
    r.count = __shfl_sync(0xffffffffu, mine.count, b & 31);
    r.len = __shfl_sync(0xffffffffu, mine.len, b & 31);
    r.before = r.len - r.count;
    return r;
  }
  // On to the first tile of the next sequence with rows.
  __device__ __forceinline__ void next_sequence(const PrefillView& p) {
    at.t = at.kb = 0;
    unsigned left = __ballot_sync(0xffffffffu, mine.count > 0) & ~(0xffffffffu >> (31 - (at.b & 31)));
    while (left == 0) {
      if (at.row > end.row || (at.row == end.row && window >= end.b)) {  // behind the end already
        at.row = end.row + 1;
        return;
      }
      int to = window + 32;
      if (to >= p.c.n_seqs) {
        to = 0;
        ++at.row;
      }
      look(p, to);
      left = __ballot_sync(0xffffffffu, mine.count > 0);
      if (at.row > end.row) return;
    }
    at.b = window + __ffs(left) - 1;
  }
  __device__ __forceinline__ void begin(const PrefillView& p, const PfTiling& w) {
    PfCut cuts[2];
    pf_share(p, w, cuts);
    at = cuts[0];
    end = cuts[1];
    look(p, at.b);
  }
  // The next item; false: no more.
  __device__ __forceinline__ bool next(const PrefillView& p, const PfTiling& w, PfItem* item) {
    for (;;) {
      if (at.row >= w.head_rows || at.row > end.row) return false;
      const PrefillRows r = rows(at.b);
      if ((long long)at.t * w.span >= r.count) {
        next_sequence(p);
        continue;
      }
      if (at.row == end.row && (at.b > end.b || (at.b == end.b && at.t > end.t))) return false;
      const bool last = at.row == end.row && at.b == end.b && at.t == end.t;
      if (last && end.kb == 0) return false;
      const int blocks = pf_blocks(r, at.t, w.span), to = last ? end.kb : blocks;
      *item = PfItem{at.b, at.t, at.row, at.kb, to, r.first, r.count, r.len, r.before, -1};
      if (at.kb > 0)
        item->slot = 0;
      else if (to < blocks)
        item->slot = 1;
      const bool some = to > at.kb || blocks == 0;
      if (last)
        at.row = end.row + 1;
      else
        ++at.t;
      at.kb = 0;
      if (some) return true;
    }
  }
};

// ---------------------------------------------------------------- tensor cores
// A block is 128 query rows: positions x the heads of one KV head, so that short parts of
// prompts fill it too.
//   S_j = Q K_j^T   128 rows x 64 keys, Q and K_j in shared memory (128-byte swizzled,
//                   K-major), fp32 S in tensor memory, two buffers a block of rows in turn.
//   P_j             exp2(s - m), a thread a row, back to tensor memory: the A operand of
//   O += P_j V_j    V_j as an MN-major operand, fp32 O in tensor memory.
// m is a reference: O and l are rescaled only where a row's maximum exceeds it by more than 2^8.
// bf16 rows: a tile is two blocks of rows that share the copies of K and V. P_j, two bf16 parts that leave 2^-17 of a
// probability (one part would leave 2^-8: outputs 2.1e-3 to 2.4e-3 of their norm off 64 bits, of which their own rounding is
// 1.65e-3; 1 x 16384 674 us), lies in S_j's own columns; S_{j+2} takes them again when P_j V_j is done. While one block's
// softmax runs, the tensor core has the other's products and the same block's next S. O stays in tensor memory, whose fp32
// sums are cut off, not rounded: with the parts, 0.2 % of outputs (0.9 % behind 65000 entries) are the bf16 number next to the
// one that plain fp32 operations give.
// fp32 rows: a tile is one block; q and each probability are three bf16 parts (24 bits), so S and P V
// take three products each, small parts first. P V of a key block goes into a fresh accumulator and is added, rounded, to
// the output in registers, so nothing is cut off over a long axis. With more than 128 head dims the three parts of 128 rows do
// not fit: a block is 64 rows (the instruction's other 64 read what follows in shared memory and are masked), and a tile
// has half of the values' head dims, so that S is formed twice.
// Warps: 0-7 the softmax; then one that walks the CTA's work and copies K (and bf16 Q), one that issues S, one that copies V,
// one that issues P V, and for bf16's second block of rows one more of each of the issuers. Every wait is bounded.
//
// What bounds it. bf16, 16 heads on 2 of 128, 1 x 16384: 859 us at burst clocks (933 under the power cap of a warm GPU), 1280
// TFLOP/s, 1920 with both parts' products: the tensor pipe is busy 90 % of the time (64-key products read the queries' 4 KB for
// each 2 KB of keys, which holds it at 40 cycles an MMA of 32), issue slots are 54 % used, MUFU 28 %. fp32 rows, 1 x
// 4096: 156 us (171 warm), 440 TFLOP/s of the attention's own and 1310 of the three products', tensor pipe 73 %. 64 head dims,
// 256 rows behind 65000 entries: 104 us, tensor pipe 55 %: as many exponentials for half the products, and the softmax of a
// block of rows is one chain in each of its warps: see the scores, load them, form weights, store them, arrive. Short
// calls wait on the chain launch - lengths - cut - pages - copies - S - softmax - P V - store, and on code that runs once: 1 x 37
// 11.5 us.
// bf16 rows: the maximum of a key block ahead of its weights. Formed together, and the weights again where the reference moved,
// the scores stay in registers beside all the weights, and a warp has too few left for exponentials in flight (1 x 16384
// 943 us against 862, 32 sequences 220 against 205, 256 head dims 1 x 4096 99 against 94; with one part of a probability
// 704 against 680, 181 against 172, and 256 head dims, whose four warps have registers enough, 80 against 84).
// Tried and not kept, with one part: key blocks of 128 with one score buffer (the block waits for its scores to be read: 1 x 8192 362 against
// 325 us at that stage); one warp issuing both blocks' products (222 against 216); four groups of softmax warps that take a
// block's key blocks in turn and pass the reference on (308 against 214); sixteen warps of 16 rows, four lanes a row, 80
// registers each (the chain stays as long: 746 against 703); the next key block's scores fetched by halves while this one's are
// worked on (886 against 703); the two warps of an SM partition forming weights in turn (679 against 684, the others 1 to 3 %
// slower); seeing the next scores ahead, waits voted on at once, predicated arrivals (none faster by 1 %).
template <int HDP_, bool F32_>
struct PfCfg {
  static constexpr bool F32 = F32_;
  static constexpr int HDP = HDP_, NH = HDP / 64;         // head dims of queries and keys, padded
  static constexpr int HDV = F32 && HDP == 256 ? 128 : HDP;  // of a tile's values: 256 of fp32 rows are two tiles
  static constexpr int QROWS = F32 && HDP == 256 ? 64 : 128; // rows of a block that are used
  static constexpr int BLOCKS = F32 || HDP == 256 ? 1 : 2;
  static constexpr int PARTS = F32 ? 3 : 1, P_PARTS = F32 ? 3 : 2;  // bf16 parts of a query and of a probability
  static constexpr int SOFT = F32 ? 8 : 4 * BLOCKS;       // warps of the softmax (of 8; the others have none)
  static constexpr int THREADS = BLOCKS == 1 ? 384 : 512; // (two blocks: two warps more, so that warps give registers up by fours)
  static constexpr int QT = HDP == 256 && !F32 ? 1 : 3;   // bf16: a ring of blocks of queries; fp32: their parts
  static constexpr int QHALF = QROWS * 128;               // 64 head dims of the query rows
  static constexpr int QTILE = NH * QHALF;
  static constexpr int HALF = PF_KEYS * 128;              // 64 head dims of a key block
  static constexpr int TILE = NH * HALF, VTILE = HDV / 64 * HALF;
  static constexpr int KST = HDP == 256 ? 2 : 4, VST = HDP == 64 ? 6 : F32 ? 3 : HDP == 128 ? 4 : 2;
  // Key blocks' words on missing pages. A word is read by the softmax of both blocks of rows, but where a tile has rows in
  // the first block alone, only the rings bound how far the copies run ahead of the second block's softmax: it
  // holds back the values of VST blocks on, those hold back S of two more, and that the keys of KST more.
  static constexpr int RING = 16;
  static_assert(RING > KST + VST + 1, "a word may be overwritten before it is read");
  static constexpr int SMEM = 1024 + QT * QTILE + KST * TILE + VST * VTILE;
  static constexpr uint32_t P_COL = 128, O_COL = F32 ? 320 : 256;
  // tensor memory: S of (block, buffer), P of (block, part, buffer), O of a block
  static __device__ __forceinline__ uint32_t s_col(int blk, int buf) { return 64u * (2 * blk + buf); }
  static __device__ __forceinline__ uint32_t p_col(int blk, int part, int buf) {
    return F32 ? P_COL + 96u * buf + 32u * part : s_col(blk, buf) + 32u * part;
  }
  static __device__ __forceinline__ uint32_t o_col(int blk) { return O_COL + (uint32_t)HDV * blk; }
};
constexpr int PF_KWARP = 8, PF_SWARP = 9, PF_VWARP = 10;  // 11 P V; block 1's S and P V 12 and 13
constexpr float PF_RESCALE_LOG2 = 8.f;

struct PfArgs {
  PrefillView p;
  PfTiling w;
  float scale;       // of scores, in units of log2(e), at least FLT_MIN
  uint32_t flip;     // the sign bit where the scale is negative
  int box_rows;      // slots of a copy
  int block_pos;     // positions of a block of 128 query rows
  bool wide;         // rows of out are 32-byte aligned
  float2* part_ml;   // [CTAs][2 slots][blocks][128 rows]
  float* part_o;     // as pf_part has it
};

struct PfBars {
  uint64_t k_full[6], v_full[6], k_empty[6], v_empty[6];
  uint64_t it_full[PF_ITEMS], it_empty[PF_ITEMS];
  uint64_t q_full[3], q_empty[3];                      // bf16: of the ring; fp32: q_full[0]
  uint64_t s_full[2][2], p_full[2][2], pv_done[2][2];  // [block][buffer]
  uint64_t o_read, drain[4];
};

__device__ __forceinline__ void pf_tma(uint32_t dst, const CUtensorMap* map, int dim, int row, int head, int page,
                                       uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.4d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4, %5}], "
      "[%6];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(dim), "r"(row), "r"(head), "r"(page), "r"(tc::smem_u32(bar))
      : "memory");
}

// 32 lanes x 32 consecutive 32-bit columns of tensor memory, without the wait.
__device__ __forceinline__ void pf_ld32(uint32_t ta, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
      "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]),
        "=r"(v[8]), "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]),
        "=r"(v[16]), "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]),
        "=r"(v[24]), "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31])
      : "r"(ta)
      : "memory");
}
// 32 lanes x 64 columns and the wait, in one statement: the registers come out of it as they
// are (loads and wait apart, with the registers passing through the wait, cost a move each).
__device__ __forceinline__ void pf_ld64(uint32_t ta, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x64.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,%19,"
      "%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31,%32,%33,%34,%35,%36,%37,%38,%39,"
      "%40,%41,%42,%43,%44,%45,%46,%47,%48,%49,%50,%51,%52,%53,%54,%55,%56,%57,%58,%59,"
      "%60,%61,%62,%63}, [%64];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15]), "=r"(v[16]),
        "=r"(v[17]), "=r"(v[18]), "=r"(v[19]), "=r"(v[20]), "=r"(v[21]), "=r"(v[22]), "=r"(v[23]), "=r"(v[24]),
        "=r"(v[25]), "=r"(v[26]), "=r"(v[27]), "=r"(v[28]), "=r"(v[29]), "=r"(v[30]), "=r"(v[31]), "=r"(v[32]),
        "=r"(v[33]), "=r"(v[34]), "=r"(v[35]), "=r"(v[36]), "=r"(v[37]), "=r"(v[38]), "=r"(v[39]), "=r"(v[40]),
        "=r"(v[41]), "=r"(v[42]), "=r"(v[43]), "=r"(v[44]), "=r"(v[45]), "=r"(v[46]), "=r"(v[47]), "=r"(v[48]),
        "=r"(v[49]), "=r"(v[50]), "=r"(v[51]), "=r"(v[52]), "=r"(v[53]), "=r"(v[54]), "=r"(v[55]), "=r"(v[56]),
        "=r"(v[57]), "=r"(v[58]), "=r"(v[59]), "=r"(v[60]), "=r"(v[61]), "=r"(v[62]), "=r"(v[63])
      : "r"(ta)
      : "memory");
}
// 16 columns and the wait.
__device__ __forceinline__ void pf_ld16(uint32_t ta, uint32_t* v) {
  asm volatile(
      "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];\n\t"
      "tcgen05.wait::ld.sync.aligned;"
      : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
        "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
      : "r"(ta)
      : "memory");
}
// Waits for this thread's loads from tensor memory; the registers pass through, so
// that no use of them moves ahead of the wait.
__device__ __forceinline__ void pf_wait_ld(uint32_t* v) {
  asm volatile("tcgen05.wait::ld.sync.aligned;"
               : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7]),
                 "+r"(v[8]), "+r"(v[9]), "+r"(v[10]), "+r"(v[11]), "+r"(v[12]), "+r"(v[13]), "+r"(v[14]), "+r"(v[15]),
                 "+r"(v[16]), "+r"(v[17]), "+r"(v[18]), "+r"(v[19]), "+r"(v[20]), "+r"(v[21]), "+r"(v[22]),
                 "+r"(v[23]), "+r"(v[24]), "+r"(v[25]), "+r"(v[26]), "+r"(v[27]), "+r"(v[28]), "+r"(v[29]),
                 "+r"(v[30]), "+r"(v[31])
               :
               : "memory");
}

// Shared-memory matrix descriptors with 128-byte swizzle, low words: address and
// leading byte offset. K-major operands (rows of 128 bytes, 64 values along K) do not
// use the offset; MN-major ones (rows of 64 values along N for consecutive K) step by it to
// the next 64 values along N. 8-row atoms of 1024 bytes lie one after the other.
__device__ __forceinline__ uint32_t pf_desc(uint32_t smem_addr, uint32_t lbo_bytes) {
  return ((smem_addr >> 4) & 0x3FFFu) | ((lbo_bytes >> 4) << 16);
}

__device__ __forceinline__ void pf_tma_q(uint32_t dst, const CUtensorMap* map, int dim, int head, int row, uint64_t* bar) {
  asm volatile(
      "cp.async.bulk.tensor.3d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], "
      "[%5];" ::"r"(dst),
      "l"(reinterpret_cast<uint64_t>(map)), "r"(dim), "r"(head), "r"(row), "r"(tc::smem_u32(bar))
      : "memory");
}

// Waits for an mbarrier's phase; false: given up, after ``limit_ns`` or because another
// warp has (tc::mbar_wait in fewer instructions: the kernel's loops take turns in the instruction
// cache, and with it the same loops ran 1 x 16384 in 710 to 910 us, by where the compiler put them).
__device__ __forceinline__ uint32_t pf_now() {
  uint32_t t;
  asm volatile("mov.u32 %0, %%globaltimer_lo;" : "=r"(t));
  return t;
}
__device__ __forceinline__ bool pf_wait(uint64_t* bar, uint32_t parity, volatile int* abort, uint32_t limit_ns) {
  if (tc::mbar_try_wait(bar, parity)) return true;
  const uint32_t t0 = pf_now();
  while (!tc::mbar_try_wait(bar, parity)) {
    if (*abort || pf_now() - t0 > limit_ns) {
      *abort = 1;
      return false;
    }
  }
  return true;
}

// MMAs and their commits by one lane of a whole warp: predicated instead of branched
// around, so that descriptors stay in uniform registers (in a branch of one lane every operand is moved there
// first, about 70 cycles an MMA).
__device__ __forceinline__ uint32_t pf_leader() {
  uint32_t one;
  asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(one));
  return one;
}
// (descriptors by their low words; the high word, stride and swizzle, is the same for all)
constexpr uint32_t PF_DESC_HI = (1024u >> 4) | (1u << 14) | (2u << 29);
__device__ __forceinline__ void pf_mma(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 x, y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 x, {%1, %6};\n\tmov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], x, y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader), "n"(PF_DESC_HI)
      : "memory");
}
__device__ __forceinline__ void pf_mma_ts(uint32_t leader, uint32_t d, uint32_t a, uint32_t b, uint32_t idesc, bool add) {
  asm volatile(
      "{\n\t.reg .pred p, q;\n\t.reg .b64 y;\n\t"
      "setp.ne.b32 p, %4, 0;\n\tsetp.ne.b32 q, %5, 0;\n\t"
      "mov.b64 y, {%2, %6};\n\t"
      "@q tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], y, %3, p;\n\t}" ::"r"(d),
      "r"(a), "r"(b), "r"(idesc), "r"((uint32_t)add), "r"(leader), "n"(PF_DESC_HI)
      : "memory");
}
__device__ __forceinline__ void pf_commit(uint32_t leader, uint64_t* bar) {
  asm volatile(
      "{\n\t.reg .pred q;\n\tsetp.ne.b32 q, %1, 0;\n\t"
      "@q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n\t}" ::"r"(tc::smem_u32(bar)),
      "r"(leader)
      : "memory");
}
__device__ __forceinline__ int pf_same(int x) { return __shfl_sync(0xffffffffu, x, 0); }

// A key block of K or V: this lane's copy (a page, or as many slots of one as a block has).
struct PfPages {
  int page, row;   // ``page`` n_pages: out of range, reads zeros
  uint32_t there;  // bit i: keys 8 i .. 8 i + 7 of the block lie in a page that exists
};
__device__ __forceinline__ PfPages pf_pages(const PfArgs& a, const PfItem& it, int kb) {
  const int lane = threadIdx.x & 31, boxes = PF_KEYS / a.box_rows, slot = kb * PF_KEYS + lane * a.box_rows;
  const PagedView& c = a.p.c;
  PfPages r{c.n_pages, 0, 0xFFu};
  bool ok = true;
  if (lane < boxes && slot < it.len) {
    const int page = paged_entry(c, it.b, slot);
    ok = (unsigned)page < (unsigned)c.n_pages;
    if (ok)
      r.page = page;
    else
      record_status(a.p.a.status, QMOE_ERR_DEVICE_ARG);
    r.row = slot & ((1 << c.page_log2) - 1);
  }
  const unsigned gone = __ballot_sync(0xffffffffu, !ok);
  if (gone) {
    const int per = a.box_rows / 8;
    for (int i = 0; i < boxes; ++i)
      if ((gone >> i) & 1u) r.there &= ~(((1u << per) - 1u) << (i * per));
  }
  return r;
}

template <int NH, int HALF>
__device__ __forceinline__ void pf_copy(const PfArgs& a, int g, int dim, const PfPages& pg, const CUtensorMap* map,
                                        uint8_t* stage, uint64_t* bar) {
  const int lane = threadIdx.x & 31, boxes = PF_KEYS / a.box_rows;
  if (lane == 0) tc::mbar_expect_tx(bar, NH * HALF);
  __syncwarp();
  if (lane < boxes) {
    const uint32_t dst = tc::smem_u32(stage) + lane * a.box_rows * 128;
#pragma unroll
    for (int h = 0; h < NH; ++h) pf_tma(dst + h * HALF, map, dim + 64 * h, pg.row, g, pg.page, bar);
  }
  __syncwarp();
}

// The KV head of a head row, its first query head and how many there are, and its first head dim of the values.
struct PfHeads {
  int g, h0, n, dv;
};
__host__ __device__ __forceinline__ PfHeads pf_heads(const PfTiling& w, int n_kv, int group, int row) {
  if (w.head_rows == n_kv) return PfHeads{row, row * group, group, 0};
  const int rows = w.head_rows / n_kv, g = row / rows, in = row - g * rows, tile = in / w.v_parts, at = tile * w.row_heads;
  return PfHeads{g, g * group + at, min(w.row_heads, group - at), 128 * (in - tile * w.v_parts)};
}
__device__ __forceinline__ PfHeads pf_heads(const PfArgs& a, int row) {
  return pf_heads(a.w, a.p.c.n_kv, a.p.group, row);
}

// Row r of a block of 128: position ``place``, head ``head`` of the block's.
struct PfRow {
  int vis;  // entries that it sees (0 where the row is none)
  bool valid;
  long long at;  // element of q and out
};
__device__ __forceinline__ PfRow pf_row(const PfArgs& a, const PfItem& it, const PfHeads& hs, int blk, int place, int head) {
  const int pos = it.t * a.w.span + blk * a.block_pos + place;
  PfRow x;
  x.valid = place < a.block_pos && pos < it.count && head < hs.n;
  x.vis = x.valid ? max(it.before + pos + 1, 0) : 0;
  x.at = ((long long)(it.first + pos) * a.p.a.n_heads + hs.h0 + head) * a.p.c.head_dim;
  return x;
}

// Scores that a row does not see: those from ``seen`` on, and those of missing pages.
__device__ __forceinline__ void pf_mask(uint32_t* v, int seen, uint32_t exist) {
  if (__any_sync(0xffffffffu, seen < PF_KEYS)) {
#pragma unroll
    for (int i = 0; i < PF_KEYS; ++i)
      if (i >= seen) v[i] = 0xFF800000u;
  }
  if (exist != 0xFFu) {
#pragma unroll
    for (int i = 0; i < PF_KEYS; ++i)
      if (!((exist >> (i / 8)) & 1u)) v[i] = 0xFF800000u;
  }
}

__device__ __forceinline__ float pf_max3(float a, uint32_t b, uint32_t c) {
  float m;
  asm("max.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(__uint_as_float(b)), "f"(__uint_as_float(c)));
  return m;
}
__device__ __forceinline__ float pf_max(const uint32_t* v) {
  float m[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
  for (int i = 0; i < PF_KEYS; i += 2) m[(i >> 1) & 3] = pf_max3(m[(i >> 1) & 3], v[i], v[i + 1]);
  return fmaxf(fmaxf(m[0], m[1]), fmaxf(m[2], m[3]));
}

// 32 or 16 bytes of a row. (A row's bytes in pieces of 32, whole sectors, by its own thread: 8 of
// them take a warp less time than 16 pieces of 16, and than pieces exchanged between lanes.)
__device__ __forceinline__ void pf_store32(void* p, const uint32_t* w) {
  asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(w[0]), "r"(w[1]), "r"(w[2]), "r"(w[3]),
               "r"(w[4]), "r"(w[5]), "r"(w[6]), "r"(w[7])
               : "memory");
}
__device__ __forceinline__ void pf_store16(void* p, const uint32_t* w) {
  *reinterpret_cast<uint4*>(p) = make_uint4(w[0], w[1], w[2], w[3]);
}
// 8 words of a row of which ``bytes`` exist.
__device__ __forceinline__ void pf_store_row(char* p, const uint32_t* w, int bytes, bool wide) {
  if (bytes >= 32 && wide) {
    pf_store32(p, w);
  } else {
    if (bytes >= 16) pf_store16(p, w);
    if (bytes >= 32) pf_store16(p + 16, w + 4);
  }
}

// A part's O: [part][block][4 columns][128 rows], so that a warp's rows lie side by side.
__device__ __forceinline__ float4* pf_part(float* base, long long part, int blk, int blocks, int hdp, int col4, int r) {
  return reinterpret_cast<float4*>(base) + ((part * blocks + blk) * (hdp / 4) + col4) * 128 + r;
}

// Warps 0-7 of tiles of bf16 rows.
template <class C, class Take>
__device__ __forceinline__ void prefill_bf16_rows(const PfArgs& a, Take& take, const PfItem& it, uint32_t tmem,
                                                  const uint32_t* there, PfBars& bar, volatile int* abort_flag) {
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hd = a.p.c.head_dim;
  const uint32_t lim = (uint32_t)min(a.p.a.wait_ns, 4000000000ull);
  const int blk = warp >> 2, r = threadIdx.x & 127;
  const int place = r / a.w.row_heads, head = r - place * a.w.row_heads;
  const uint32_t tq = tmem + ((uint32_t)(32 * (warp & 3)) << 16), tO = tq + C::o_col(blk);
  const float c = a.scale;
  const uint64_t c2 = pack2(__float_as_uint(c), __float_as_uint(c)), one2 = pack2(0x3F800000u, 0x3F800000u),
                 minus2 = pack2(0xBF800000u, 0xBF800000u);
  int j = 0;   // key blocks of this block of rows so far
  int ring = 0;  // the key block's place in the ring of ``there``
  for (int n = 0; take(n); ++n) {
    if (blk * a.block_pos >= it.count - it.t * a.w.span) {  // no rows in this block
      ring = (ring + it.kb1 - it.kb0) % C::RING;
      continue;
    }
    const PfRow row = pf_row(a, it, pf_heads(a, it.row), blk, place, head);
    // key blocks that all rows of the warp see whole (with a negative scale all are gone through)
    const int whole = a.flip ? 0 : __reduce_min_sync(0xffffffffu, row.valid ? row.vis : 0x7FFFFFFF) / PF_KEYS;
    float m = -INFINITY, l = 0.f;
#pragma unroll 1
    for (int kb = it.kb0; kb < it.kb1; ++kb, ++j) {
      const int buf = j & 1;
      if (!__all_sync(0xffffffffu, pf_wait(&bar.s_full[blk][buf], (j >> 1) & 1, abort_flag, lim))) return;
      tc::tc_fence_after();
      const uint32_t tS = tq + C::s_col(blk, buf);
      uint32_t v[PF_KEYS], w[PF_KEYS / 2];
      const uint32_t exist = there[ring];
      ring = (ring + 1) % C::RING;
      pf_ld64(tS, v);
      if (__builtin_expect(kb >= whole || exist != 0xFFu, 0)) {
        if (a.flip) {
#pragma unroll
          for (int i = 0; i < PF_KEYS; ++i) v[i] ^= a.flip;
        }
        pf_mask(v, row.vis - kb * PF_KEYS, exist);
      }
      const float mx = pf_max(v) * c;
      const bool need = mx > m + PF_RESCALE_LOG2;
      if (__builtin_expect(__any_sync(0xffffffffu, need), 0)) {
        const float alpha = need ? exp2f(m - mx) : 1.f;
        if (need) m = mx;
        l *= alpha;
        if (kb > it.kb0) {
          // O holds P V of the block before once that is done
          if (!__all_sync(0xffffffffu, pf_wait(&bar.pv_done[blk][buf ^ 1], ((j - 1) >> 1) & 1, abort_flag, lim)))
            return;
          tc::tc_fence_after();
#pragma unroll 1
          for (int i = 0; i < C::HDP / 16; ++i) {
            uint32_t o[16];
            pf_ld16(tO + 16 * i, o);
#pragma unroll
            for (int e = 0; e < 16; ++e) o[e] = __float_as_uint(__uint_as_float(o[e]) * alpha);
            tc::tmem_st16(tO + 16 * i, o);
          }
        }
      }
      // p = exp2(c s - m) as two bf16 parts, their sum in fp32
      const float mref = m == -INFINITY ? 0.f : m;
      const uint64_t negm2 = pack2(__float_as_uint(-mref), __float_as_uint(-mref));
      uint64_t l2[2] = {0, 0};
#pragma unroll
      for (int i = 0; i < PF_KEYS / 2; ++i) {
        const float2 d = unpack2(ffma2(pack2(v[2 * i], v[2 * i + 1]), c2, negm2));
        const float p0 = exp2f(d.x), p1 = exp2f(d.y);
        const uint64_t p = pack2(__float_as_uint(p0), __float_as_uint(p1));
        l2[i & 1] = ffma2(p, one2, l2[i & 1]);
        const uint32_t hi = tc::pack_bf16x2(p0, p1);
        const float2 rest = unpack2(ffma2(pack2(hi << 16, hi & 0xFFFF0000u), minus2, p));
        w[i & 15] = hi;
        w[16 + (i & 15)] = tc::pack_bf16x2(rest.x, rest.y);
        if ((i & 15) == 15) {
          tc::tmem_st16(tS + (i - 15), w);
          tc::tmem_st16(tS + 32 + (i - 15), w + 16);
        }
      }
      const float2 la = unpack2(l2[0]), lc = unpack2(l2[1]);
      l += (la.x + la.y) + (lc.x + lc.y);
      tc::tmem_wait_st();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.p_full[blk][buf]);
    }
    // out = O / l, or the part's O, m and l
    const bool some = it.kb1 > it.kb0;
    if (some) {
      if (!__all_sync(0xffffffffu, pf_wait(&bar.pv_done[blk][(j - 1) & 1], ((j - 1) >> 1) & 1, abort_flag, lim)))
        return;
      tc::tc_fence_after();
    }
    const float il = l > 0.f ? 1.f / l : 0.f;
    const long long part = (long long)blockIdx.x * 2 + it.slot;
    if (it.slot >= 0 && row.valid) a.part_ml[(part * C::BLOCKS + blk) * 128 + r] = make_float2(m, l);
    char* out = reinterpret_cast<char*>(static_cast<__nv_bfloat16*>(a.p.a.out) + row.at);
#pragma unroll 1
    for (int i = 0; i < C::HDP / 32; ++i) {
      uint32_t o[32];
      if (some) {
        pf_ld32(tO + 32 * i, o);
        pf_wait_ld(o);
      } else {
#pragma unroll
        for (int e = 0; e < 32; ++e) o[e] = 0u;
      }
      if (it.slot >= 0) {
        if (row.valid) {
          float4* to = pf_part(a.part_o, part, blk, C::BLOCKS, C::HDP, 8 * i, r);
#pragma unroll
          for (int e = 0; e < 8; ++e)
            to[128 * e] = make_float4(__uint_as_float(o[4 * e]), __uint_as_float(o[4 * e + 1]), __uint_as_float(o[4 * e + 2]),
                                      __uint_as_float(o[4 * e + 3]));
        }
      } else if (row.valid) {
#pragma unroll
        for (int e = 0; e < 16; ++e)
          o[e] = tc::pack_bf16x2(__uint_as_float(o[2 * e]) * il, __uint_as_float(o[2 * e + 1]) * il);
#pragma unroll
        for (int e = 0; e < 2; ++e) pf_store_row(out + 64 * i + 32 * e, o + 8 * e, 2 * hd - 64 * i - 32 * e, a.wide);
      }
      __syncwarp();
    }
    tc::tc_fence_before();
  }
}

// What the two warps of 32 fp32 rows (a half of the columns each) tell one another.
struct PfHalves {
  uint64_t max_there[4][2], l_there[4];  // [quarter][key block parity]
  float max[2][2][128], l[2][128];       // [parity][half][row]
};

// Tiles of fp32 rows: warps w and w + 4 have the same 32 rows, each half of a key block's scores and half
// of the head dims of their output, which is in registers. The reference is settled with the partner's maximum
// ahead of the weights (formed while that is on its way, and again where the reference moves, they need registers beside
// the scores: 1 x 4096 163 against 157 us, 256 head dims 488 against 456). P V of a key block is added once
// the next one's weights are out; a tile's last one, after the next tile's queries.
template <class C, class Take>
__device__ __forceinline__ void prefill_f32_rows(const PfArgs& a, Take& take, const PfItem& it, uint32_t tmem, uint8_t* sQ,
                                                 const uint32_t* there, PfBars& bar, PfHalves& halves,
                                                 volatile int* abort_flag) {
  constexpr int KH = PF_KEYS / 2, DH = C::HDV / 2;  // scores and head dims of a warp
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, r = threadIdx.x & 127, hd = a.p.c.head_dim;
  const int half = warp >> 2, quarter = warp & 3;
  const uint32_t lim = (uint32_t)min(a.p.a.wait_ns, 4000000000ull);
  const int place = r / a.w.row_heads, head = r - place * a.w.row_heads;
  const uint32_t tq = tmem + ((uint32_t)(32 * quarter) << 16), tO = tq + C::o_col(0) + DH * half;
  const float c = a.scale;
  const auto wait = [&](uint64_t* b, int phase) -> bool {
    return __all_sync(0xffffffffu, pf_wait(b, (uint32_t)phase & 1u, abort_flag, lim));
  };
  int j = 0, tiles = 0;      // key blocks, and tiles with key blocks, so far
  float m = -INFINITY, l = 0.f, alpha = 0.f;
  float acc[DH];
  PfRow row{}, old{};
  int slot = -1, dv = 0;     // of the tile before
  bool open = false;         // the tile before waits for its last P V
  // acc = acc alpha + P V of key block k
  const auto add = [&](int k) -> bool {
    if (!wait(&bar.pv_done[0][k & 1], k >> 1)) return false;
    tc::tc_fence_after();
#pragma unroll
    for (int i = 0; i < DH / 32; ++i) {
      uint32_t o[32];
      pf_ld32(tO + 32 * i, o);
      pf_wait_ld(o);
#pragma unroll
      for (int e = 0; e < 32; ++e) acc[32 * i + e] = fmaf(acc[32 * i + e], alpha, __uint_as_float(o[e]));
    }
    tc::tc_fence_before();
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bar.o_read);
    return true;
  };
  const auto store = [&](const PfRow& to, float il) {
    if (!to.valid) return;
    if (slot >= 0) {
      float4* p = pf_part(a.part_o, (long long)blockIdx.x * 2 + slot, 0, 1, C::HDV, DH / 4 * half, r);
#pragma unroll
      for (int e = 0; e < DH / 4; ++e)
        p[128 * e] = make_float4(acc[4 * e], acc[4 * e + 1], acc[4 * e + 2], acc[4 * e + 3]);
    } else {
      char* p = reinterpret_cast<char*>(static_cast<float*>(a.p.a.out) + to.at + dv + DH * half);
#pragma unroll
      for (int e = 0; e < DH / 8; ++e) {
        uint32_t x[8];
#pragma unroll
        for (int k = 0; k < 8; ++k) x[k] = __float_as_uint(acc[8 * e + k] * il);
        pf_store_row(p + 32 * e, x, 4 * (hd - dv - DH * half) - 32 * e, a.wide);
      }
    }
  };
  for (int n = 0;; ++n) {
    const bool more = take(n);
    if (more) row = pf_row(a, it, pf_heads(a, it.row), 0, place, head);
    if (more && it.kb1 > it.kb0) {
      // q as three bf16 parts, which hold all its bits, where the S products of the tile before no longer read (this
      // warp has taken their results): 16 rows of the quarter, a row's head dims over HDP / 4 lanes, the next
      // rows' loads ahead
      constexpr int LANES = C::HDP < 128 ? C::HDP / 4 : 32, ROWS = 32 / LANES, PER = C::HDP / (4 * LANES), STEP = 4;
      constexpr int STEPS = 16 / ROWS * PER;
      const int sub = lane / LANES, d0 = 4 * (lane - sub * LANES), r0 = 16 * half;
      const auto load = [&](int i) {
        const int src = r0 + (i % STEPS / PER) * ROWS + sub, d = d0 + 128 * (i % PER);
        const long long at = __shfl_sync(0xffffffffu, row.at, src);
        const bool real = __shfl_sync(0xffffffffu, (int)row.valid, src);
        float4 x = make_float4(0.f, 0.f, 0.f, 0.f);
        if (real && d < hd) x = *reinterpret_cast<const float4*>(static_cast<const float*>(a.p.a.q) + at + d);
        return x;
      };
      float4 x[STEP];
#pragma unroll
      for (int i = 0; i < STEP; ++i) x[i] = load(i);
#pragma unroll 1
      for (int i0 = 0; i0 < STEPS && 32 * quarter < C::QROWS; i0 += STEP) {
        float4 y[STEP];
#pragma unroll
        for (int i = 0; i < STEP; ++i) y[i] = load(i0 + STEP + i);  // (behind the last: the first again)
#pragma unroll
        for (int i = 0; i < STEP; ++i) {
          const int rr = 32 * quarter + r0 + (i0 + i) / PER * ROWS + sub, d = d0 + 128 * ((i0 + i) % PER), ch = d >> 3;
          const uint32_t to = (ch >> 3) * C::QHALF + tc::sw128_offset(rr, ch & 7) + 2 * (d & 4);
#pragma unroll
          for (int part = 0; part < 3; ++part) {
            const uint32_t w0 = tc::pack_bf16x2(x[i].x, x[i].y), w1 = tc::pack_bf16x2(x[i].z, x[i].w);
            x[i].x -= __uint_as_float(w0 << 16);
            x[i].y -= __uint_as_float(w0 & 0xFFFF0000u);
            x[i].z -= __uint_as_float(w1 << 16);
            x[i].w -= __uint_as_float(w1 & 0xFFFF0000u);
            *reinterpret_cast<uint2*>(sQ + part * C::QTILE + to) = make_uint2(w0, w1);
          }
          x[i] = y[i];
        }
      }
      tc::fence_proxy_async_smem();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.q_full[0]);
    }
    if (open) {
      // the tile before: its last P V, then out = O / l, or the part's O, m and l
      if (!add(j - 1)) return;
      halves.l[half][r] = l;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&halves.l_there[quarter]);
      if (!wait(&halves.l_there[quarter], tiles)) return;
      ++tiles;
      l = halves.l[0][r] + halves.l[1][r];
      if (slot >= 0 && old.valid && half == 0) a.part_ml[((long long)blockIdx.x * 2 + slot) * 128 + r] = make_float2(m, l);
      store(old, l > 0.f ? 1.f / l : 0.f);
    }
    if (!more) return;
#pragma unroll
    for (int i = 0; i < DH; ++i) acc[i] = 0.f;
    m = -INFINITY;
    l = alpha = 0.f;
    slot = it.slot;
    dv = pf_heads(a, it.row).dv;
    old = row;
    open = it.kb1 > it.kb0;
    if (!open) store(row, 0.f);
#pragma unroll 1
    for (int kb = it.kb0; kb < it.kb1; ++kb, ++j) {
      const int buf = j & 1;
      if (!wait(&bar.s_full[0][buf], j >> 1)) return;
      tc::tc_fence_after();
      const uint32_t exist = there[j % C::RING];
      uint32_t v[KH];
      pf_ld32(tq + C::s_col(0, buf) + KH * half, v);
      pf_wait_ld(v);
      const int seen = row.vis - kb * PF_KEYS - KH * half;
      if (__builtin_expect(a.flip || exist != 0xFFu || __any_sync(0xffffffffu, seen < KH), 0)) {
#pragma unroll
        for (int i = 0; i < KH; ++i) v[i] = i >= seen || !((exist >> (4 * half + i / 8)) & 1u) ? 0xFF800000u : v[i] ^ a.flip;
      }
      float mx = __uint_as_float(v[0]);
#pragma unroll
      for (int i = 1; i + 1 < KH; i += 2) mx = pf_max3(mx, v[i], v[i + 1]);
      mx = fmaxf(mx, __uint_as_float(v[KH - 1])) * c;
      halves.max[buf][half][r] = mx;
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&halves.max_there[quarter][buf]);
      const float before = alpha;  // the factor that goes with P V of the block before
      alpha = 1.f;
      if (!wait(&halves.max_there[quarter][buf], j >> 1)) return;
      mx = fmaxf(mx, halves.max[buf][half ^ 1][r]);
      if (mx > m + PF_RESCALE_LOG2) {
        alpha = exp2f(m - mx);
        m = mx;
        l *= alpha;
      }
      const float mref = m == -INFINITY ? 0.f : m;
      float p[KH], l4[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
      for (int i = 0; i < KH; ++i) {
        p[i] = exp2f(fmaf(__uint_as_float(v[i]), c, -mref));
        l4[i & 3] += p[i];
      }
      l += (l4[0] + l4[1]) + (l4[2] + l4[3]);
      // (P's buffer is free: this warp has added P V of two blocks before)
#pragma unroll
      for (int part = 0; part < 3; ++part) {
        uint32_t w[16];
#pragma unroll
        for (int e = 0; e < 16; ++e) {
          w[e] = tc::pack_bf16x2(p[2 * e], p[2 * e + 1]);
          if (part < 2) {
            p[2 * e] -= __uint_as_float(w[e] << 16);
            p[2 * e + 1] -= __uint_as_float(w[e] & 0xFFFF0000u);
          }
        }
        tc::tmem_st16(tq + C::p_col(0, part, buf) + KH / 2 * half, w);
      }
      tc::tmem_wait_st();
      tc::tc_fence_before();
      __syncwarp();
      if (lane == 0) tc::mbar_arrive(&bar.p_full[0][buf]);
      if (kb > it.kb0) {
        const float now = alpha;
        alpha = before;
        if (!add(j - 1)) return;
        alpha = now;
      }
    }
  }
}

template <class C>
__global__ void __launch_bounds__(C::THREADS, 1)
    prefill_tc_kernel(const PfArgs a, const __grid_constant__ CUtensorMap kmap, const __grid_constant__ CUtensorMap vmap,
                      const __grid_constant__ CUtensorMap qmap) {
  extern __shared__ uint8_t pf_smem_raw[];
  __shared__ PfItem items[PF_ITEMS];
  __shared__ uint32_t there[C::RING];
  __shared__ __align__(8) PfBars bar;
  __shared__ __align__(8) PfHalves halves;
  __shared__ uint32_t tmem_slot;
  __shared__ int abort_word;
  const uint32_t s0 = tc::smem_u32(pf_smem_raw);
  uint8_t* smem = pf_smem_raw + (((s0 + 1023u) & ~1023u) - s0);
  uint8_t* sQ = smem;                       // [QT]
  uint8_t* sK = sQ + C::QT * C::QTILE;      // [KST]
  uint8_t* sV = sK + C::KST * C::TILE;      // [VST]
  volatile int* abort_flag = &abort_word;
  const int warp = pf_same(threadIdx.x >> 5), lane = threadIdx.x & 31;
  const uint32_t lim = (uint32_t)min(a.p.a.wait_ns, 4000000000ull);

  if (threadIdx.x == 0) {
    const auto init = [](uint64_t* b, int n, uint32_t count) {
#pragma unroll 1
      for (int i = 0; i < n; ++i) tc::mbar_init(b + i, count);
    };
    init(bar.k_full, 12, 1);               // and v_full
    init(bar.k_empty, 12, C::BLOCKS);      // and v_empty
    init(bar.it_full, PF_ITEMS, 1);
    init(bar.it_empty, PF_ITEMS, C::SOFT + 1 + 2 * C::BLOCKS);
    init(bar.q_full, 3, C::F32 ? 8 : 1);
    init(bar.q_empty, 3, 1);
    init(&bar.s_full[0][0], 4, 1);
    init(&bar.p_full[0][0], 4, C::F32 ? 8 : 4);
    init(&bar.pv_done[0][0], 4, 1);
    init(&bar.o_read, 1, 8);
    if constexpr (C::F32) init(&halves.max_there[0][0], 12, 2);  // and l_there
    init(bar.drain, 4, 1);
    abort_word = 0;
    tc::fence_barrier_init();
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&kmap)) : "memory");
    asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&vmap)) : "memory");
  }
  if (warp == PF_SWARP) tc::tmem_alloc(&tmem_slot, 512);
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const uint32_t tmem = tmem_slot;
  const int hd = a.p.c.head_dim;
  const uint32_t leader = pf_leader();

  // The next item for a consumer warp (n: items taken so far); false: none, or given up.
  PfItem it;
  auto take = [&](int n) -> bool {
    if (!__all_sync(0xffffffffu, pf_wait(&bar.it_full[n % PF_ITEMS], (n / PF_ITEMS) & 1, abort_flag, lim))) return false;
    it = items[n % PF_ITEMS];
    __syncwarp();
    if (lane == 0) tc::mbar_arrive(&bar.it_empty[n % PF_ITEMS]);
    return it.b >= 0;
  };
  auto blocks_of = [&]() { return C::BLOCKS == 2 && it.count - it.t * a.w.span > a.block_pos ? 2 : 1; };

  // registers of 512 threads go from the others to the softmax, which holds 64 scores and 32 weights: 256 x 168 + 256 x 80
  if constexpr (C::BLOCKS == 2) {
    if (warp < 8)
      asm volatile("setmaxnreg.inc.sync.aligned.u32 168;");
    else
      asm volatile("setmaxnreg.dec.sync.aligned.u32 80;");
  }
  if (warp < 8) {
    if constexpr (C::F32)
      prefill_f32_rows<C>(a, take, it, tmem, sQ, there, bar, halves, abort_flag);
    else if (warp < C::SOFT)
      prefill_bf16_rows<C>(a, take, it, tmem, there, bar, abort_flag);
  } else if (warp == PF_KWARP) {
    // ------------------------------------------------------------ the CTA's work, copies of K and bf16 Q
    int4* desc = a.w.desc + 2 * blockIdx.x;
    if (lane < 2) desc[lane] = make_int4(-1, 0, 0, 0);
    __syncwarp();
    PfWalk walk;
    walk.begin(a.p, a.w);
    int k = 0, q_n = 0;
    bool ok = true;
    const bool withhold = a.p.a.fault == 1;
    for (int n = 0; ok; ++n) {
      const bool more = walk.next(a.p, a.w, &it);
      if (!more) it.b = -1;
      if (n >= PF_ITEMS &&
          !__all_sync(0xffffffffu, pf_wait(&bar.it_empty[n % PF_ITEMS], (n / PF_ITEMS - 1) & 1, abort_flag, lim)))
        break;
      if (lane == 0) {
        items[n % PF_ITEMS] = it;
        if (more && it.slot >= 0) {
          const PrefillRows rr{it.first, it.count, it.len, it.before};
          desc[it.slot] = make_int4(it.b, it.t, it.row, it.kb1 == pf_blocks(rr, it.t, a.w.span) ? 1 : 0);
        }
        tc::mbar_arrive(&bar.it_full[n % PF_ITEMS]);
      }
      __syncwarp();
      if (!more) break;
      if (it.kb1 <= it.kb0) continue;
      const PfHeads hs = pf_heads(a, it.row);
      const int blocks = blocks_of();
      // A block's queries go into the space of the third block before (of the one before, with 256 head dims), once S
      // no longer reads that; what lies behind the rows (other sequences' rows, zeros from n_rows on) is masked. The
      // second block's wait for the item before: it comes behind the first keys.
      const auto queries = [&](int blk) -> bool {
        const int qs = q_n % C::QT;
        if (q_n >= C::QT &&
            !__all_sync(0xffffffffu, pf_wait(&bar.q_empty[qs], (q_n / C::QT - 1) & 1, abort_flag, lim)))
          return false;
        ++q_n;
        if (lane == 0) {
          tc::mbar_expect_tx(&bar.q_full[qs], C::NH * 128 * a.w.row_heads * a.block_pos);
#pragma unroll
          for (int h = 0; h < C::NH; ++h)
            pf_tma_q(tc::smem_u32(sQ) + qs * C::QTILE + h * C::QHALF, &qmap, 64 * h, hs.h0,
                     it.first + it.t * a.w.span + blk * a.block_pos, &bar.q_full[qs]);
        }
        __syncwarp();
        return true;
      };
      if (!C::F32 && !queries(0)) break;
      const int second = it.kb0 + min(C::KST - 1, it.kb1 - it.kb0 - 1);
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1; ++kb, ++k) {
        const PfPages pg = pf_pages(a, it, kb);
        const int st = k % C::KST;
        if (k >= C::KST &&
            !__all_sync(0xffffffffu, pf_wait(&bar.k_empty[st], (k / C::KST - 1) & 1, abort_flag, lim))) {
          ok = false;
          break;
        }
        if (withhold && k == 0) {
          // test-only: never copied
          volatile int late = 0;
          pf_wait(&bar.k_full[0], 0, &late, lim);
          *abort_flag = 1;
          ok = false;
          break;
        }
        if (lane == 0) there[k % C::RING] = pg.there;
        pf_copy<C::NH, C::HALF>(a, hs.g, 0, pg, &kmap, sK + st * C::TILE, &bar.k_full[st]);
        if (!C::F32 && kb == second && blocks == 2 && !queries(1)) {
          ++k;
          ok = false;
          break;
        }
      }
    }
    // copies in flight land before the CTA leaves
    volatile int never = 0;
#pragma unroll 1
    for (int i = max(0, k - C::KST); i < k; ++i) pf_wait(&bar.k_full[i % C::KST], (i / C::KST) & 1, &never, lim);
    if (!C::F32) {
#pragma unroll 1
      for (int i = max(0, q_n - C::QT); i < q_n; ++i) pf_wait(&bar.q_full[i % C::QT], (i / C::QT) & 1, &never, lim);
    }
    __syncwarp();
  } else if (warp == PF_VWARP) {
    // ------------------------------------------------------------ copies of V
    int k = 0;
    bool ok = true;
    for (int n = 0; ok && take(n); ++n) {
      const PfHeads hs = pf_heads(a, it.row);
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1; ++kb, ++k) {
        const PfPages pg = pf_pages(a, it, kb);
        const int st = k % C::VST;
        if (k >= C::VST &&
            !__all_sync(0xffffffffu, pf_wait(&bar.v_empty[st], (k / C::VST - 1) & 1, abort_flag, lim))) {
          ok = false;
          break;
        }
        pf_copy<C::HDV / 64, C::HALF>(a, hs.g, hs.dv, pg, &vmap, sV + st * C::VTILE, &bar.v_full[st]);
      }
    }
    volatile int never = 0;
#pragma unroll 1
    for (int i = max(0, k - C::VST); i < k; ++i) pf_wait(&bar.v_full[i % C::VST], (i / C::VST) & 1, &never, lim);
    __syncwarp();
  } else if (warp == PF_SWARP || warp == 12) {
    // ------------------------------------------------------------ S = Q K^T
    const int blk = C::BLOCKS == 2 && warp == 12 ? 1 : 0;
    const uint32_t idesc = tc::idesc_bf16_f32(128, PF_KEYS);
    const int steps = (hd + 15) / 16;
    int k = 0, j = 0, q_n = 0;  // j: S products so far; q_n: bf16 blocks of queries (fp32: tiles) of the items before
    bool ok = true;
    for (int n = 0; ok && take(n); ++n) {
      const int blocks = blocks_of(), q = q_n + blk, qs = C::F32 ? 0 : q % C::QT;
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1; ++kb, ++k) {
        const int st = k % C::KST, buf = j & 1;
        ok = pf_wait(&bar.k_full[st], (k / C::KST) & 1, abort_flag, lim);
        if (blk >= blocks) {  // no rows in this block: the stage is free as far as this warp goes
          ok = __all_sync(0xffffffffu, ok);
          if (!ok) break;
          if (lane == 0) tc::mbar_arrive(&bar.k_empty[st]);
          continue;
        }
        if (kb == it.kb0) ok = ok && pf_wait(&bar.q_full[qs], (C::F32 ? q : q / C::QT) & 1, abort_flag, lim);
        // the buffer is free again: bf16 once P V of two blocks before, which reads P there, is done; fp32 once
        // the softmax has taken S of two blocks before
        uint64_t* free_bar = C::F32 ? &bar.p_full[0][buf] : &bar.pv_done[blk][buf];
        ok = ok && (j < 2 || pf_wait(free_bar, ((j >> 1) - 1) & 1, abort_flag, lim));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++j;
        tc::tc_fence_after();
        const uint32_t kd = pf_same(pf_desc(tc::smem_u32(sK) + (uint32_t)(st * C::TILE), 16));
        const uint32_t d = pf_same(tmem + C::s_col(blk, buf));
#pragma unroll
        for (int part = C::PARTS - 1; part >= 0; --part) {
          const uint32_t qd = pf_same(pf_desc(tc::smem_u32(sQ) + (uint32_t)((qs + part) * C::QTILE), 16));
#pragma unroll
          for (int kk = 0; kk < C::HDP / 16; ++kk)
            if (kk < steps)
              pf_mma(leader, d, qd + (uint32_t)((kk >> 2) * (C::QHALF >> 4) + 2 * (kk & 3)),
                     kd + (uint32_t)((kk >> 2) * (C::HALF >> 4) + 2 * (kk & 3)), idesc,
                     part != C::PARTS - 1 || kk != 0);
        }
        pf_commit(leader, &bar.s_full[blk][buf]);
        pf_commit(leader, &bar.k_empty[st]);
        if (!C::F32 && kb == it.kb1 - 1) pf_commit(leader, &bar.q_empty[qs]);
      }
      if (it.kb1 > it.kb0) q_n += blocks;
    }
    pf_commit(leader, &bar.drain[blk]);
    volatile int never = 0;
    pf_wait(&bar.drain[blk], 0, &never, lim);
    __syncwarp();
  } else if (warp == 11 || warp == 13) {
    // ------------------------------------------------------------ O += P V
    const int blk = C::BLOCKS == 2 && warp == 13 ? 1 : 0;
    int k = 0, j = 0;  // j: P V products so far
    bool ok = true;
    for (int n = 0; ok && take(n); ++n) {
      const int blocks = blocks_of(), dims = min(hd - pf_heads(a, it.row).dv, C::HDV);
      const uint32_t idesc = tc::idesc_bf16_f32(128, (dims + 15) / 16 * 16) | (1u << 16);  // B (V) MN-major
#pragma unroll 1
      for (int kb = it.kb0; kb < it.kb1; ++kb, ++k) {
        const int st = k % C::VST, buf = j & 1;
        ok = __all_sync(0xffffffffu, pf_wait(&bar.v_full[st], (k / C::VST) & 1, abort_flag, lim));
        if (!ok) break;
        if (blk >= blocks) {
          if (lane == 0) tc::mbar_arrive(&bar.v_empty[st]);
          continue;
        }
        uint8_t* vs = sV + st * C::VTILE;
        // rows behind the sequence's last entry may hold anything, NaN too: zero weights need zero values (both
        // blocks' warps write the zeros, each ahead of its own products)
        if (it.len - kb * PF_KEYS < PF_KEYS) {
          const int r0 = it.len - kb * PF_KEYS;
#pragma unroll 1
          for (int i = 8 * r0 + lane; i < 8 * PF_KEYS; i += 32) {
#pragma unroll
            for (int h = 0; h < C::HDV / 64; ++h)
              *reinterpret_cast<uint4*>(vs + h * C::HALF + 16 * i) = make_uint4(0, 0, 0, 0);
          }
          tc::fence_proxy_async_smem();
          __syncwarp();
        }
        ok = pf_wait(&bar.p_full[blk][buf], (j >> 1) & 1, abort_flag, lim);
        if (C::F32) ok = ok && (j == 0 || pf_wait(&bar.o_read, (j - 1) & 1, abort_flag, lim));
        ok = __all_sync(0xffffffffu, ok);
        if (!ok) break;
        ++j;
        tc::tc_fence_after();
        const uint32_t vd = pf_same(pf_desc(tc::smem_u32(sV) + (uint32_t)(st * C::VTILE), C::HALF));
        const uint32_t d = pf_same(tmem + C::o_col(blk));
        const bool first = !C::F32 && kb == it.kb0;
#pragma unroll
        for (int part = C::P_PARTS - 1; part >= 0; --part) {
          const uint32_t pa = pf_same(tmem + C::p_col(blk, part, buf));
#pragma unroll
          for (int kk = 0; kk < PF_KEYS / 16; ++kk)
            pf_mma_ts(leader, d, pa + 8u * kk, vd + (uint32_t)(2048 / 16 * kk), idesc,
                      part != C::P_PARTS - 1 || kk != 0 || (!C::F32 && !first));
        }
        if (C::BLOCKS == 1 || blk == 0 || a.p.a.fault != 2) pf_commit(leader, &bar.pv_done[blk][buf]);
        pf_commit(leader, &bar.v_empty[st]);
      }
    }
    pf_commit(leader, &bar.drain[2 + blk]);
    volatile int never = 0;
    pf_wait(&bar.drain[2 + blk], 0, &never, lim);
    __syncwarp();
  }

  __syncwarp();
  tc::tc_fence_before();
  __syncthreads();
  tc::tc_fence_after();
  // (behind the barrier: a wait may run out when the first warps have long left)
  if (*abort_flag && threadIdx.x == 0) record_status(a.p.a.status, QMOE_ERR_TIMEOUT);
  if (warp == PF_SWARP) tc::tmem_dealloc(tmem, 512);
}

// ---------------------------------------------------------------- parts of tiles
// A tile over several CTAs: its parts, in order of the CTAs, joined by their maxima. As many CTAs of this kernel as
// the tile has parts share its groups of 32 rows, each with a part of the columns; a lane has a row. Few parts: a warp
// takes them all for its group; many (few rows on a long axis): eight warps take the parts of a group
// in turn, and their sums meet in shared memory.
constexpr int PJ_THREADS = 256, PJ_WARPS = 8, PJ_C4 = 8;  // PJ_C4 float4s of a row in a CTA
constexpr int PF_MAX_CTAS = 256;  // the workspace does not depend on the device

struct PfJoin {
  PrefillView p;
  PfTiling w;
  int block_pos;  // positions of a block of 128 rows
  const float2* part_ml;
  float* part_o;
};

__device__ __forceinline__ bool pj_same(int4 a, int4 b) { return a.x == b.x && a.y == b.y && a.z == b.z; }

template <typename T, int HDP, int BLOCKS>
__global__ void __launch_bounds__(PJ_THREADS) prefill_join_kernel(const PfJoin j) {
  __shared__ int parts[PF_MAX_CTAS], n_parts, rank_here;
  __shared__ float4 sum[PJ_WARPS][PJ_C4][32];
  __shared__ float2 ml[PJ_WARPS][32];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hd = j.p.c.head_dim, c0 = blockIdx.y * PJ_C4;
#pragma unroll 1
  for (int slot = 0; slot < 2; ++slot) {
    // this CTA's part: of a tile that began in an earlier CTA, of one that begins here
    const int4 d = j.w.desc[2 * blockIdx.x + slot];
    if (d.x < 0) continue;
    __syncthreads();
    if (warp == 0) {
      int x0 = blockIdx.x;
      if (slot == 0) {  // back to the CTA that the tile begins in
        x0 = -1;
        for (int x = (int)blockIdx.x - 1; x0 < 0 && x >= 0; x -= 32) {
          const int4 e = x - lane >= 0 ? j.w.desc[2 * (x - lane) + 1] : make_int4(-1, 0, 0, 0);
          const unsigned begins = __ballot_sync(0xffffffffu, pj_same(e, d));
          if (begins) x0 = x - (__ffs(begins) - 1);
        }
      }
      int n = x0 >= 0 ? 1 : 0, rank = 0;  // (a CTA that gave up may have left no beginning)
      if (lane == 0) parts[0] = 2 * x0 + 1;
      bool open = x0 >= 0;
      for (int x = x0 + 1; open && x < j.w.ctas; x += 32) {
        const int4 e = x + lane < j.w.ctas ? j.w.desc[2 * (x + lane)] : make_int4(-1, 0, 0, 0);
        const bool mine = pj_same(e, d);
        unsigned have = __ballot_sync(0xffffffffu, mine);
        const unsigned last = __ballot_sync(0xffffffffu, mine && e.w);
        if (last) {
          have &= 0xffffffffu >> (32 - __ffs(last));
          open = false;
        }
        if ((have >> lane) & 1u) parts[n + __popc(have & ((1u << lane) - 1u))] = 2 * (x + lane);
        if (slot == 0 && (int)blockIdx.x >= x && (int)blockIdx.x < x + 32)
          rank = n + __popc(have & ((1u << (blockIdx.x - x)) - 1u));
        n += __popc(have);
      }
      if (lane == 0) {
        n_parts = n;
        rank_here = rank;
      }
    }
    __syncthreads();
    const int n = n_parts, rank = rank_here;
    if (n == 0) continue;
    const PfHeads hs = pf_heads(j.w, j.p.c.n_kv, j.p.group, d.z);
    const PrefillRows rr = prefill_rows(j.p, d.x);
    const bool many = n > PJ_WARPS;
    for (int group = many ? rank : rank + n * warp; group < 4 * BLOCKS; group += many ? n : n * PJ_WARPS) {
      const int in = 32 * (group & 3) + lane, blk = group >> 2, place = in / j.w.row_heads;
      const int pos = d.y * j.w.span + blk * j.block_pos + place, h = in - place * j.w.row_heads;
      const bool valid = place < j.block_pos && pos < rr.count && h < hs.n;
      if (!__any_sync(0xffffffffu, valid)) continue;  // (the same for all warps of a group)
      float top = -INFINITY, l = 0.f;
      float4 acc[PJ_C4];
#pragma unroll
      for (int e = 0; e < PJ_C4; ++e) acc[e] = make_float4(0.f, 0.f, 0.f, 0.f);
      constexpr int U = 2;
      const int step = many ? PJ_WARPS : 1;
      for (int i0 = many ? warp : 0; valid && i0 < n; i0 += U * step) {
        float2 x[U];
        float4 v[U][PJ_C4];
#pragma unroll
        for (int u = 0; u < U; ++u) {
          x[u] = make_float2(-INFINITY, 0.f);
          if (i0 + u * step >= n) continue;
          const int part = parts[i0 + u * step];
          x[u] = j.part_ml[((long long)part * BLOCKS + blk) * 128 + in];
          const float4* o = pf_part(j.part_o, part, blk, BLOCKS, HDP, c0, in);
#pragma unroll
          for (int e = 0; e < PJ_C4; ++e) v[u][e] = o[128 * e];
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
          if (x[u].x == -INFINITY) continue;
          const float m = fmaxf(top, x[u].x), old = exp2f(top - m), w = exp2f(x[u].x - m);
          top = m;
          l = l * old + x[u].y * w;
#pragma unroll
          for (int e = 0; e < PJ_C4; ++e) {
            acc[e].x = acc[e].x * old + v[u][e].x * w;
            acc[e].y = acc[e].y * old + v[u][e].y * w;
            acc[e].z = acc[e].z * old + v[u][e].z * w;
            acc[e].w = acc[e].w * old + v[u][e].w * w;
          }
        }
      }
      if (many) {
        ml[warp][lane] = make_float2(top, l);
#pragma unroll
        for (int e = 0; e < PJ_C4; ++e) sum[warp][e][lane] = acc[e];
        __syncthreads();
        // a warp finishes one float4
        float m = -INFINITY;
#pragma unroll
        for (int x = 0; x < PJ_WARPS; ++x) m = fmaxf(m, ml[x][lane].x);
        l = 0.f;
        acc[0] = make_float4(0.f, 0.f, 0.f, 0.f);
        if (warp < PJ_C4) {
#pragma unroll
          for (int x = 0; x < PJ_WARPS; ++x) {
            const float2 y = ml[x][lane];
            const float w = y.x == -INFINITY ? 0.f : exp2f(y.x - m);
            const float4 v = sum[x][warp][lane];
            l += y.y * w;
            acc[0].x += v.x * w;
            acc[0].y += v.y * w;
            acc[0].z += v.z * w;
            acc[0].w += v.w * w;
          }
        }
        __syncthreads();
      }
      const float il = l > 0.f ? 1.f / l : 0.f;
      T* out = static_cast<T*>(j.p.a.out) + ((long long)(rr.first + pos) * j.p.a.n_heads + hs.h0 + h) * hd + hs.dv;
      const int e0 = many ? warp : 0;
#pragma unroll
      for (int e = 0; e < PJ_C4; ++e) {
        const int col = 4 * (c0 + e0 + e);
        if (!valid || hs.dv + col >= hd || (many && (e > 0 || warp >= PJ_C4))) continue;
        *reinterpret_cast<typename Four<T>::raw*>(out + col) =
            Four<T>::narrow(make_float4(acc[e].x * il, acc[e].y * il, acc[e].z * il, acc[e].w * il));
      }
    }
  }
}

template <typename T, int HDP, int BLOCKS>
cudaError_t launch_join(const PfJoin& j, cudaStream_t st) {
  return launch_overlapped(prefill_join_kernel<T, HDP, BLOCKS>, dim3(j.w.ctas, HDP / (4 * PJ_C4)), PJ_THREADS, 0, 0, st, j);
}

// ---------------------------------------------------------------- host
struct PfPlan {
  int hdp, row_heads, row_tiles, v_parts, block_pos, blocks, span, ctas;
  bool cuts;        // tiles may be cut between CTAs
  size_t desc, ml, o, q, total;
};

size_t pf_up(size_t v) { return (v + 255) & ~size_t(255); }

PfPlan pf_plan(const PagedView& c, int n_rows, int n_heads, bool f32) {
  PfPlan p{};
  const int group = n_heads / c.n_kv;
  p.hdp = c.head_dim <= 64 ? 64 : c.head_dim <= 128 ? 128 : 256;
  p.blocks = f32 || p.hdp == 256 ? 1 : 2;
  const int block = f32 && p.hdp == 256 ? 64 : 128;  // query rows
  p.v_parts = 128 / block;
  p.row_tiles = (group + block - 1) / block;
  p.row_heads = (group + p.row_tiles - 1) / p.row_tiles;
  p.block_pos = block / p.row_heads;
  p.span = p.blocks * p.block_pos;
  const long long seqs = c.n_seqs < n_rows ? c.n_seqs : n_rows;
  const long long tiles = ((long long)n_rows / p.span + seqs) * c.n_kv * p.row_tiles * p.v_parts;
  const long long keys = (paged_slots(c) + PF_KEYS - 1) / PF_KEYS;
  p.cuts = keys >= 2 * PF_MIN_BLOCKS;
  const long long pieces = tiles * (p.cuts ? keys / PF_MIN_BLOCKS : 1);
  p.ctas = pieces < 1 ? 1 : pieces < PF_MAX_CTAS ? (int)pieces : PF_MAX_CTAS;
  size_t o = 0;
  p.desc = o; o += pf_up(sizeof(int4) * 2 * (size_t)p.ctas);
  p.ml = o;   o += p.cuts ? pf_up(sizeof(float2) * 512 * (size_t)p.ctas) : 0;
  p.o = o;    o += p.cuts ? pf_up(sizeof(float) * 512 * (size_t)p.hdp * p.ctas) : 0;
  // two tiles of fp32 rows with more than 128 head dims read the same queries: where out is q, they read a copy
  p.q = o;    o += p.v_parts == 2 ? pf_up(sizeof(float) * (size_t)n_rows * n_heads * c.head_dim) : 0;
  p.total = o;
  return p;
}

// A pool as a tensor map [head dim][slot of a page][KV head][page], boxes of 64 head
// dims (those from head_dim on read as zero) by ``box_rows`` slots, 128-byte swizzled.
bool pf_encode(CUtensorMap* m, const void* base, const PagedView& c, int box_rows) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t ss = (cuuint64_t)c.slot_stride * 2;
  // (a dimension of one element never steps: its stride may be anything that is valid)
  const cuuint64_t strides[3] = {ss, c.n_kv > 1 ? (cuuint64_t)c.head_stride * 2 : ss,
                                 c.n_pages > 1 ? (cuuint64_t)c.page_stride * 2 : ss};
  const cuuint64_t dims[4] = {(cuuint64_t)c.head_dim, (cuuint64_t)1 << c.page_log2, (cuuint64_t)c.n_kv,
                              (cuuint64_t)c.n_pages};
  const cuuint32_t box[4] = {64, (cuuint32_t)box_rows, 1, 1}, estr[4] = {1, 1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(base), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

// bf16 queries as a tensor map [head dim][head][row], boxes of a block's rows.
bool pf_encode_q(CUtensorMap* m, const PfArgs& x) {
  PFN_cuTensorMapEncodeTiled_v12000 fn = tensor_map_encoder();
  if (fn == nullptr) return false;
  const cuuint64_t hd = (cuuint64_t)x.p.c.head_dim, heads = (cuuint64_t)x.p.a.n_heads;
  const cuuint64_t dims[3] = {hd, heads, (cuuint64_t)x.p.a.n_rows}, strides[2] = {2 * hd, 2 * hd * heads};
  const cuuint32_t box[3] = {64, (cuuint32_t)x.w.row_heads, (cuuint32_t)x.block_pos}, estr[3] = {1, 1, 1};
  return fn(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p.a.q), dims, strides, box, estr,
            CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
            CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class C>
cudaError_t launch_tc(PfArgs& x, cudaStream_t st) {
  const PagedView& c = x.p.c;
  x.box_rows = 1 << c.page_log2 < PF_KEYS ? 1 << c.page_log2 : PF_KEYS;
  CUtensorMap km, vm, qm{};
  if (!pf_encode(&km, c.k, c, x.box_rows) || !pf_encode(&vm, c.v, c, x.box_rows) || (!C::F32 && !pf_encode_q(&qm, x)))
    return cudaErrorInvalidValue;
  cudaError_t e = ensure_kernel_smem(reinterpret_cast<const void*>(prefill_tc_kernel<C>), C::SMEM);
  if (e != cudaSuccess) return e;
  return launch_overlapped(prefill_tc_kernel<C>, dim3(x.w.ctas), C::THREADS, C::SMEM, 0, st, x, km, vm, qm);
}

}  // namespace

size_t paged_prefill_ws_bytes(const PagedView& c, int n_rows, int n_heads) {
  const size_t a = pf_plan(c, n_rows, n_heads, false).total, b = pf_plan(c, n_rows, n_heads, true).total;
  return a > b ? a : b;
}

int paged_prefill_launches(const PagedView& c, const PrefillArgs& a) {
  const PfPlan pl = pf_plan(c, a.n_rows, a.n_heads, a.f32);
  return pl.cuts ? 2 : 1;
}

cudaError_t launch_paged_prefill(const PagedView& c, const PrefillArgs& a, cudaStream_t st) {
  const PfPlan pl = pf_plan(c, a.n_rows, a.n_heads, a.f32);
  PrefillView p{c, a, a.scale * 1.4426950408889634f, a.n_heads / c.n_kv};
  if (pl.v_parts == 2 && a.out == a.q) {
    p.a.q = static_cast<char*>(a.ws) + pl.q;
    const size_t bytes = sizeof(float) * (size_t)a.n_rows * a.n_heads * c.head_dim;
    const cudaError_t e = cudaMemcpyAsync(const_cast<void*>(p.a.q), a.q, bytes, cudaMemcpyDeviceToDevice, st);
    if (e != cudaSuccess) return e;
  }
  char* ws = static_cast<char*>(a.ws);
  PfArgs x{};
  x.p = p;
  x.w.span = pl.span;
  x.w.head_rows = c.n_kv * pl.row_tiles * pl.v_parts;
  x.w.v_parts = pl.v_parts;
  x.w.row_heads = pl.row_heads;
  // in keys' worth of time: the change of tiles (bf16: 32 sequences of 1..1000 behind 0..3000 with 192 205 us, 256 201, 320 204,
  // 448 208, 8 of 300..2048 and 64 head dims 51.9, 52.0, 53.2, 56, 1 x 4096 and 256 head dims the same with all four within
  // its 4 % of spread; fp32 1 x 4096 with 256 175 us, 384 156, 512 157; of fp32 rows with 256 head dims not measured)
  x.w.tile_cost = a.f32 ? 384 : 256;
  x.w.ctas = device_sm_count() < pl.ctas ? device_sm_count() : pl.ctas;
  x.w.desc = reinterpret_cast<int4*>(ws + pl.desc);
  x.part_ml = reinterpret_cast<float2*>(ws + pl.ml);
  x.part_o = reinterpret_cast<float*>(ws + pl.o);
  x.block_pos = pl.block_pos;
  x.wide = reinterpret_cast<uintptr_t>(a.out) % 32 == 0 && c.head_dim * (a.f32 ? 4 : 2) % 32 == 0;
  x.scale = fminf(fmaxf(fabsf(p.scale_log2), FLT_MIN), FLT_MAX);
  x.flip = a.scale < 0.f ? 0x80000000u : 0u;
  cudaError_t e;
  if (a.f32)
    e = pl.hdp == 64    ? launch_tc<PfCfg<64, true>>(x, st)
        : pl.hdp == 128 ? launch_tc<PfCfg<128, true>>(x, st)
                        : launch_tc<PfCfg<256, true>>(x, st);
  else
    e = pl.hdp == 64    ? launch_tc<PfCfg<64, false>>(x, st)
        : pl.hdp == 128 ? launch_tc<PfCfg<128, false>>(x, st)
                        : launch_tc<PfCfg<256, false>>(x, st);
  if (e != cudaSuccess || !pl.cuts) return e;
  const PfJoin j{p, x.w, pl.block_pos, x.part_ml, x.part_o};
  if (a.f32) return pl.hdp == 64 ? launch_join<float, 64, 1>(j, st) : launch_join<float, 128, 1>(j, st);  // (of values)
  return pl.hdp == 64    ? launch_join<__nv_bfloat16, 64, 2>(j, st)
         : pl.hdp == 128 ? launch_join<__nv_bfloat16, 128, 2>(j, st)
                         : launch_join<__nv_bfloat16, 256, 1>(j, st);
}

}  // namespace qmoe
