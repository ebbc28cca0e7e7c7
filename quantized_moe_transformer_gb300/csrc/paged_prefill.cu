// Causal attention of packed rows (prompts, parts of prompts, single tokens of
// many sequences) over a paged key-value cache. Defined in include/qmoe.h.
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": 16 query heads over 2 KV heads, causal. Pages and packed rows have
// no counterpart there.
#include <cmath>

#include "paged.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

constexpr int PP_THREADS = 128, PP_WARPS = 4;

struct PrefillView {
  PagedView c;
  PrefillArgs a;
  float scale_log2;
  int group;
};

// The rows of sequence b: (first row, rows, entries that its first row sees), no
// rows where they do not lie in the call's.
struct PrefillRows {
  int first, count, len;
  long long before;
};
__device__ __forceinline__ PrefillRows prefill_rows(const PrefillView& p, int b) {
  PrefillRows r{p.a.first[b], p.a.count[b], paged_len(p.c, b), 0};
  if (r.count < 0) r.count = 0;
  if (r.count > 0 && (r.first < 0 || (long long)r.first + r.count > p.a.n_rows)) {
    record_status(p.a.status, QMOE_ERR_DEVICE_ARG);
    r.count = 0;
  }
  r.before = (long long)r.len - r.count;
  return r;
}

// A warp has one row and head: a lane scores one key of 32 at a time, then all
// lanes add the 32 values, a part of the head dims each.
template <typename T>
__global__ void __launch_bounds__(PP_THREADS) prefill_rows_kernel(const PrefillView p) {
  __shared__ float sq[PP_WARPS][256];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, hd = p.c.head_dim;
  const PrefillRows r = prefill_rows(p, blockIdx.y);
  const int32_t* table = p.c.table + (long long)blockIdx.y * p.c.max_pages;
  const int items = p.a.n_heads * gridDim.x * PP_WARPS;
  (void)items;
  for (long long it = (long long)blockIdx.x * PP_WARPS + warp; it < (long long)r.count * p.a.n_heads;
       it += (long long)gridDim.x * PP_WARPS) {
    const int i = (int)(it / p.a.n_heads), h = (int)(it - (long long)i * p.a.n_heads), g = h / p.group;
    const long long at = ((long long)(r.first + i) * p.a.n_heads + h) * hd;
    const T* q = static_cast<const T*>(p.a.q) + at;
    __syncwarp();
    for (int d = lane; d < hd; d += 32) sq[warp][d] = (float)q[d];
    __syncwarp();
    const long long sees = r.before + i + 1;
    const int n = sees < 0 ? 0 : (int)sees;
    float m = -INFINITY, l = 0.f, o[8] = {0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f, 0.f};
    for (int j0 = 0; j0 < n; j0 += 32) {
      const int j = j0 + lane;
      long long off = -1;
      float s = -INFINITY;
      if (j < n) {
        const int page = table[j >> p.c.page_log2];
        if ((unsigned)page < (unsigned)p.c.n_pages)
          off = (long long)page * p.c.page_stride + (long long)(j & ((1 << p.c.page_log2) - 1)) * p.c.slot_stride +
                g * p.c.head_stride;
        else
          record_status(p.a.status, QMOE_ERR_DEVICE_ARG);
      }
      if (off >= 0) {
        s = 0.f;
        for (int d = 0; d < hd; d += 8) {
          const uint4 k = *reinterpret_cast<const uint4*>(p.c.k + off + d);
          const uint32_t w[4] = {k.x, k.y, k.z, k.w};
#pragma unroll
          for (int e = 0; e < 4; ++e) {
            s = fmaf(sq[warp][d + 2 * e], __uint_as_float(w[e] << 16), s);
            s = fmaf(sq[warp][d + 2 * e + 1], __uint_as_float(w[e] & 0xFFFF0000u), s);
          }
        }
        s *= p.scale_log2;
      }
      float top = s;
#pragma unroll
      for (int d = 16; d; d /= 2) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, d));
      if (top == -INFINITY) continue;
      const float m2 = fmaxf(m, top), alpha = exp2f(m - m2), w = s == -INFINITY ? 0.f : exp2f(s - m2);
      m = m2;
      l = l * alpha + w;
#pragma unroll
      for (int e = 0; e < 8; ++e) o[e] *= alpha;
      for (int k = 0; k < 32; ++k) {
        const float wk = __shfl_sync(0xffffffffu, w, k);
        const long long ok = __shfl_sync(0xffffffffu, off, k);
        if (ok < 0) continue;
#pragma unroll
        for (int e = 0; e < 8; ++e)
          if (lane + 32 * e < hd) o[e] = fmaf(wk, __bfloat162float(p.c.v[ok + lane + 32 * e]), o[e]);
      }
    }
#pragma unroll
    for (int d = 16; d; d /= 2) l += __shfl_xor_sync(0xffffffffu, l, d);
    T* out = static_cast<T*>(p.a.out) + at;
#pragma unroll
    for (int e = 0; e < 8; ++e)
      if (lane + 32 * e < hd) out[lane + 32 * e] = (T)(l > 0.f ? o[e] / l : 0.f);
  }
}

}  // namespace

size_t paged_prefill_ws_bytes(const PagedView&, int, int) { return 256; }

int paged_prefill_launches(const PagedView&, const PrefillArgs&) { return 1; }

cudaError_t launch_paged_prefill(const PagedView& c, const PrefillArgs& a, cudaStream_t st) {
  PrefillView p{c, a, a.scale * 1.4426950408889634f, a.n_heads / c.n_kv};
  long long ctas = ((long long)a.n_rows * a.n_heads + PP_WARPS - 1) / PP_WARPS;
  if (ctas > 16384) ctas = 16384;
  const dim3 grid((unsigned)ctas, (unsigned)c.n_seqs);
  return a.f32 ? launch_overlapped(prefill_rows_kernel<float>, grid, PP_THREADS, 0, 0, st, p)
               : launch_overlapped(prefill_rows_kernel<__nv_bfloat16>, grid, PP_THREADS, 0, 0, st, p);
}

}  // namespace qmoe
