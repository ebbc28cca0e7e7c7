// Attention of one new token for each sequence over a paged key-value cache.
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": 16 query heads over 2 KV heads, query head h reads KV head
// h / 8. "Distributed CPU: Zip Fusion Beyond Tensor Parallelism",
// "Two-Dimensional Attention at Long Context": the softmax over parts of the
// context carried by (max, normaliser, weighted output).
#include "paged.cuh"

namespace qmoe {

namespace {

constexpr int PA_CHUNK = 256;

__device__ __forceinline__ float block_reduce(float v, bool is_max, float* red) {
#pragma unroll
  for (int off = 16; off > 0; off >>= 1) {
    const float o = __shfl_xor_sync(0xffffffffu, v, off);
    v = is_max ? fmaxf(v, o) : v + o;
  }
  __syncthreads();
  if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
  __syncthreads();
  v = red[0];
  for (int w = 1; w < PA_CHUNK / 32; ++w) v = is_max ? fmaxf(v, red[w]) : v + red[w];
  return v;
}

// One CTA per (sequence, KV head), its query heads one after the other: scores
// of 256 slots at a time (a thread per slot), running maximum and sum, then a
// second walk adds the probabilities to the slots' weights.
template <typename T>
__global__ void __launch_bounds__(PA_CHUNK) paged_attention_simple_kernel(const PagedView c, const PagedAttnArgs a) {
  __shared__ float qs[256], ps[PA_CHUNK], red[PA_CHUNK / 32];
  __shared__ long long offs[PA_CHUNK];
  const int b = blockIdx.x, g = blockIdx.y, tid = threadIdx.x, hd = c.head_dim;
  const int group = a.n_heads / c.n_kv, n = paged_len(c, b);
  float* stat = static_cast<float*>(a.ws);  // (maximum, sum) of every query head
  for (int h = g * group; h < (g + 1) * group; ++h) {
    const long long qoff = ((long long)b * a.n_heads + h) * hd;
    __syncthreads();
    if (tid < hd)
      qs[tid] = a.f32 ? static_cast<const float*>(a.q)[qoff + tid]
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[qoff + tid]);
    float m = -INFINITY, l = 0.f, o = 0.f;
    for (int j0 = 0; j0 < n; j0 += PA_CHUNK) {
      const int j = j0 + tid;
      float s = -INFINITY;
      __syncthreads();
      offs[tid] = j < n ? paged_offset(c, b, j) : -1;
      if (j < n && offs[tid] < 0) record_status(a.status, QMOE_ERR_DEVICE_ARG);
      __syncthreads();
      if (offs[tid] >= 0) {
        const __nv_bfloat16* kr = c.k + offs[tid] + (long long)g * c.head_stride;
        s = 0.f;
        for (int i = 0; i < hd; ++i) s = fmaf(qs[i], __bfloat162float(kr[i]), s);
        s *= a.scale;
      }
      const float mn = fmaxf(m, block_reduce(s, true, red));
      const float p = s > -INFINITY ? __expf(s - mn) : 0.f;
      const float alpha = m > -INFINITY ? __expf(m - mn) : 0.f;
      ps[tid] = p;
      l = l * alpha + block_reduce(p, false, red);
      m = mn;
      if (tid < hd) {
        o *= alpha;
        for (int i = 0; i < min(PA_CHUNK, n - j0); ++i)
          if (offs[i] >= 0) o = fmaf(ps[i], __bfloat162float(c.v[offs[i] + (long long)g * c.head_stride + tid]), o);
      }
    }
    if (tid == 0) {
      stat[2 * ((long long)b * a.n_heads + h)] = m;
      stat[2 * ((long long)b * a.n_heads + h) + 1] = l;
    }
    if (tid < hd) {
      const float r = l > 0.f ? o / l : 0.f;
      if (a.f32)
        static_cast<float*>(a.out)[qoff + tid] = r;
      else
        static_cast<__nv_bfloat16*>(a.out)[qoff + tid] = __float2bfloat16_rn(r);
    }
  }
  if (!a.accumulate) return;
  __syncthreads();
  for (int j = tid; j < n; j += PA_CHUNK) {
    const long long off = paged_offset(c, b, j);
    if (off < 0) continue;
    const __nv_bfloat16* kr = c.k + off + (long long)g * c.head_stride;
    float w = 0.f;
    for (int h = g * group; h < (g + 1) * group; ++h) {
      const long long at = (long long)b * a.n_heads + h;
      float s = 0.f;
      for (int i = 0; i < hd; ++i)
        s = fmaf(a.f32 ? static_cast<const float*>(a.q)[at * hd + i]
                       : __bfloat162float(static_cast<const __nv_bfloat16*>(a.q)[at * hd + i]),
                 __bfloat162float(kr[i]), s);
      w += __expf(s * a.scale - stat[2 * at]) / stat[2 * at + 1];
    }
    c.weight[((long long)b * c.n_kv + g) * paged_slots(c) + j] += w;
  }
}

}  // namespace

size_t paged_attention_ws_bytes(const PagedView& c, int n_heads, bool) { return 8 * (size_t)c.n_seqs * n_heads; }
int paged_attention_launches(const PagedView&, int, bool) { return 1; }

cudaError_t launch_paged_attention(const PagedView& c, const PagedAttnArgs& a, cudaStream_t st) {
  paged_attention_simple_kernel<float><<<dim3(c.n_seqs, c.n_kv), PA_CHUNK, 0, st>>>(c, a);
  return cudaGetLastError();
}

}  // namespace qmoe
