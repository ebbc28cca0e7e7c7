// New rows into the pages of a key-value cache: rotary position embedding of
// the queries and keys, bf16 rounding, page lookup, and the bookkeeping of the
// written slots (position, accumulated weight, length).
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": the keys and values of 2 KV heads go to the cache; pages and a
// bound on the cache have no counterpart there.
#include <cmath>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

constexpr int AP_THREADS = 256, AP_MAX_THREADS = 512, AP_ROWS = 32, AP_CTAS_PER_SM = 4;

// theta^(-2i/hd) / (2 pi), the turns of one position, as a fraction of 2^64.
// Whole turns drop out of the product with a position modulo 2^64, so the
// angle of any position is reduced exactly in integers.
struct AppendFreq {
  uint64_t turns[128];
};

// Four elements in memory, as fp32, and back.
template <typename T>
struct Four;
template <>
struct Four<float> {
  using raw = float4;
  static __device__ __forceinline__ float4 wide(raw v) { return v; }
  static __device__ __forceinline__ raw narrow(float4 v) { return v; }
};
template <>
struct Four<__nv_bfloat16> {
  using raw = uint2;
  static __device__ __forceinline__ float4 wide(raw u) {
    return make_float4(__uint_as_float(u.x << 16), __uint_as_float(u.x & 0xFFFF0000u), __uint_as_float(u.y << 16),
                       __uint_as_float(u.y & 0xFFFF0000u));
  }
  static __device__ __forceinline__ raw narrow(float4 v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    return make_uint2(*reinterpret_cast<const uint32_t*>(&lo), *reinterpret_cast<const uint32_t*>(&hi));
  }
};

// A CTA takes ``rows`` rows. A unit is four elements of a head and the four
// half a head further on, which turn together: one thread reads a unit, turns it
// (queries and keys) and writes it to q_out or into the page; every byte is
// read and written once, 64 bytes of a thread at a time.
// One row takes 3.1 us (the launch, the page look-up, one read and one write); 16372
// bf16 rows of two KV heads of 128 6.5 us, 4.9 TB/s of reads and writes. Angles are
// exact to 2^-33 turns; a sine or cosine is single precision, off by 2^-21 at most.
template <typename T, bool ROT>
__global__ void __launch_bounds__(AP_MAX_THREADS, 2) append_kernel(const PagedView c, const AppendArgs a, int rows,
                                                            const __grid_constant__ AppendFreq fr) {
  __shared__ float2 turn[ROT ? AP_ROWS * 128 : 1];
  __shared__ long long off[AP_ROWS];
  __shared__ int2 at[AP_ROWS];  // (sequence, slot), slot -1: the row is not cached
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int n0 = blockIdx.x * rows, n = min(rows, a.n_rows - n0), tid = threadIdx.x, threads = blockDim.x, hd = c.head_dim, half = hd / 2;
  if (ROT) {
    for (int i = tid; i < n * half; i += threads) {
      const int r = i / half, d = i - r * half;
      const uint64_t frac = (uint64_t)(long long)a.pos[n0 + r] * fr.turns[d];
      // the upper 32 bits as a signed part of a turn: |error| <= 2^-33 turns, then one rounding to fp32
      const float x = (float)(int)((frac + 0x80000000ull) >> 32) * (6.283185307179586f / 4294967296.f);
      float s, k;
      sincosf(x, &s, &k);
      turn[i] = make_float2(k, s);
    }
  }
  if (tid < 32) {
    int seq = -1, slot = -1;
    long long o = -1;
    if (tid < n) {
      const int row = n0 + tid;
      seq = a.seq ? a.seq[row] : row;
      const bool known = seq >= 0 && seq < c.n_seqs;
      slot = a.slot ? a.slot[row] : known ? paged_len(c, seq) : 0;
      const bool padding = a.slot && slot < 0;
      if (known && slot >= 0 && slot < paged_slots(c)) o = paged_offset(c, seq, slot);
      if (o < 0 && !padding) record_status(a.status, QMOE_ERR_DEVICE_ARG);
      if (o < 0) seq = slot = -1;
      off[tid] = o;
      at[tid] = make_int2(seq, slot);
    }
    // the rows of one sequence raise its length together
    const unsigned peers = __match_any_sync(0xffffffffu, seq);
    const int top = __reduce_max_sync(peers, slot);
    if (seq >= 0 && (int)(threadIdx.x & 31) == __ffs(peers) - 1) atomicMax(c.lens + seq, top + 1);
  }
  using F = Four<T>;
  using B = Four<__nv_bfloat16>;
  using raw = typename F::raw;
  const int per_head = hd / 8, units = (a.n_heads + 2 * c.n_kv) * per_head;
  // a thread keeps its unit and walks rows; where a row has fewer units than the CTA threads, groups of threads take
  // rows side by side
  const int groups = units < threads ? threads / units : 1, group = units < threads ? tid / units : 0;
  constexpr int U = 64 / (int)sizeof(raw) / 2;  // 64 bytes of a thread in flight
  bool looked_up = false;
  for (int u0 = 0; u0 < units; u0 += threads) {
    const int u = u0 + tid - group * units;
    const bool mine = u < units && group < groups;
    const int h = u / per_head, d = 4 * (u - h * per_head), g = h - a.n_heads;
    const T* src = nullptr;
    long long step = 0;  // elements between a tensor's rows
    if (mine) {
      step = (long long)(g < 0 ? a.n_heads : c.n_kv) * hd;
      src = static_cast<const T*>(g < 0 ? a.q : g < c.n_kv ? a.k : a.v) + n0 * step +
            (g < 0 ? h : g < c.n_kv ? g : g - c.n_kv) * hd + d;
    }
    T* q_to = g < 0 ? static_cast<T*>(a.q_out) + n0 * step + h * hd + d : nullptr;
    __nv_bfloat16* kv_to = g < 0 ? nullptr : (g < c.n_kv ? c.k + g * c.head_stride : c.v + (g - c.n_kv) * c.head_stride) + d;
    for (int r0 = group; r0 - group < n; r0 += U * groups) {
      raw x[U], y[U];
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int r = r0 + k * groups;
        if (mine && r < n) {
          x[k] = *reinterpret_cast<const raw*>(src + r * step);
          y[k] = *reinterpret_cast<const raw*>(src + r * step + half);
        }
      }
      if (!looked_up) __syncthreads();  // the first reads go on while the pages are looked up
      looked_up = true;
#pragma unroll
      for (int k = 0; k < U; ++k) {
        const int r = r0 + k * groups;
        if (!mine || r >= n) continue;
        const long long o = off[r];
        if (g >= 0 && o < 0) continue;
        float4 p = F::wide(x[k]), q = F::wide(y[k]);
        if (ROT && g < c.n_kv) {
          const float2* t = turn + r * half + d;
          const float2 t0 = t[0], t1 = t[1], t2 = t[2], t3 = t[3];
          const float4 v = p, w = q;
          p = make_float4(v.x * t0.x - w.x * t0.y, v.y * t1.x - w.y * t1.y, v.z * t2.x - w.z * t2.y,
                          v.w * t3.x - w.w * t3.y);
          q = make_float4(w.x * t0.x + v.x * t0.y, w.y * t1.x + v.y * t1.y, w.z * t2.x + v.z * t2.y,
                          w.w * t3.x + v.w * t3.y);
        }
        if (g < 0) {
          *reinterpret_cast<raw*>(q_to + r * step) = F::narrow(p);
          *reinterpret_cast<raw*>(q_to + r * step + half) = F::narrow(q);
        } else {
          *reinterpret_cast<B::raw*>(kv_to + o) = B::narrow(p);
          *reinterpret_cast<B::raw*>(kv_to + o + half) = B::narrow(q);
        }
      }
    }
  }
  for (int i = tid; i < n * c.n_kv; i += threads) {
    const int r = i % n, g = i / n;
    if (at[r].y < 0) continue;
    const long long e = ((long long)at[r].x * c.n_kv + g) * paged_slots(c) + at[r].y;
    if (c.weight) c.weight[e] = 0.f;
    if (c.pos) c.pos[e] = a.pos[n0 + r];
  }
}

template <typename T>
cudaError_t append_rows(const PagedView& c, const AppendArgs& a, const AppendFreq& fr, cudaStream_t st) {
  // all CTAs at once on the SMs, as few rows in each as that allows
  const int fit = AP_CTAS_PER_SM * device_sm_count();
  int rows = (a.n_rows + fit - 1) / fit;
  if (rows > AP_ROWS) rows = AP_ROWS;
  // one row of many heads: a thread for each of its units
  const int units = (a.n_heads + 2 * c.n_kv) * (c.head_dim / 8);
  int threads = AP_THREADS;
  while (rows == 1 && threads < AP_MAX_THREADS && threads < units) threads += 32;
  const int ctas = (a.n_rows + rows - 1) / rows;
  if (a.rotate)
    return launch_overlapped(append_kernel<T, true>, dim3(ctas), threads, 0, 0, st, c, a, rows, fr);
  return launch_overlapped(append_kernel<T, false>, dim3(ctas), threads, 0, 0, st, c, a, rows, fr);
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& c, const AppendArgs& a, cudaStream_t st) {
  AppendFreq fr;
  if (a.rotate) {
    // powers of the ratio by squares and one product (an error of i half steps of a double at the i-th)
    double inv[128];
    const double ratio = std::pow(a.theta, -2.0 / (double)c.head_dim);
    inv[0] = 1.0;
    for (int i = 1; i < c.head_dim / 2; ++i) inv[i] = (i & 1) ? inv[i - 1] * ratio : inv[i / 2] * inv[i / 2];
    for (int i = 0; i < c.head_dim / 2; ++i) {
      const double t = inv[i] * 0.15915494309189535;
      fr.turns[i] = (uint64_t)((t - std::floor(t)) * 18446744073709551616.0);
    }
  }
  return a.f32 ? append_rows<float>(c, a, fr, st) : append_rows<__nv_bfloat16>(c, a, fr, st);
}

}  // namespace qmoe
