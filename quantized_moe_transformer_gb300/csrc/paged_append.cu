// New rows into the pages of a key-value cache: rotary position embedding of
// the queries and keys, bf16 rounding, page lookup, and the bookkeeping of the
// written slots (position, accumulated weight, length).
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": the keys and values of 2 KV heads go to the cache; pages and a
// bound on the cache have no counterpart there.
#include <cmath>

#include "paged.cuh"

namespace qmoe {

namespace {

// Inverse frequencies theta^(-2i/hd), computed on the host in double.
struct AppendFreq {
  double inv[128];
};

__device__ __forceinline__ float load1(const float* p) { return *p; }
__device__ __forceinline__ float load1(const __nv_bfloat16* p) { return __bfloat162float(*p); }
__device__ __forceinline__ void store1(float* p, float v) { *p = v; }
__device__ __forceinline__ void store1(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }

// One CTA per row: pairs (i, i + hd/2) of every query and key head are turned
// by pos * theta^(-2i/hd). The angle is formed in double and reduced to
// [-pi, pi] by n turns, 2 pi as the double nearest to it and the remainder
// (positions reach millions of radians), then sine and cosine are taken in
// single precision, as the block's own rotation does.
template <typename T>
__global__ void __launch_bounds__(256) append_kernel(const PagedView c, const AppendArgs a,
                                                     const __grid_constant__ AppendFreq fr) {
  __shared__ float cs[128], sn[128];
  const int n = blockIdx.x, tid = threadIdx.x, hd = c.head_dim, half = hd / 2;
  if (a.rotate) {
    const int pos = a.pos[n];
    for (int i = tid; i < half; i += 256) {
      const double ang = (double)pos * fr.inv[i];
      const double turns = rint(ang * 0.15915494309189535);
      const double r = fma(-turns, 2.4492935982947064e-16, fma(-turns, 6.283185307179586, ang));
      sincosf((float)r, &sn[i], &cs[i]);
    }
  }
  const int seq = a.seq ? a.seq[n] : n;
  const bool seq_ok = seq >= 0 && seq < c.n_seqs;
  const int slot = a.slot ? a.slot[n] : seq_ok ? c.lens[seq] : -1;
  __syncthreads();
  if (a.q != nullptr) {
    const T* q = static_cast<const T*>(a.q) + (long long)n * a.n_heads * hd;
    T* qo = static_cast<T*>(a.q_out) + (long long)n * a.n_heads * hd;
    for (int idx = tid; idx < a.n_heads * half; idx += 256) {
      const int h = idx / half, i = idx % half;
      const float x = load1(q + h * hd + i), y = load1(q + h * hd + i + half);
      const float co = a.rotate ? cs[i] : 1.f, si = a.rotate ? sn[i] : 0.f;
      store1(qo + h * hd + i, x * co - y * si);
      store1(qo + h * hd + i + half, y * co + x * si);
    }
  }
  if (a.slot && slot < 0) return;  // a padding row
  long long off = -1;
  if (seq_ok && slot >= 0 && slot < paged_slots(c)) off = paged_offset(c, seq, slot);
  if (off < 0) {
    if (tid == 0) record_status(a.status, QMOE_ERR_DEVICE_ARG);
    return;
  }
  const T* k = static_cast<const T*>(a.k) + (long long)n * c.n_kv * hd;
  const T* v = static_cast<const T*>(a.v) + (long long)n * c.n_kv * hd;
  for (int idx = tid; idx < c.n_kv * half; idx += 256) {
    const int g = idx / half, i = idx % half;
    const float x = load1(k + g * hd + i), y = load1(k + g * hd + i + half);
    const float co = a.rotate ? cs[i] : 1.f, si = a.rotate ? sn[i] : 0.f;
    __nv_bfloat16* dst = c.k + off + (long long)g * c.head_stride;
    dst[i] = __float2bfloat16_rn(x * co - y * si);
    dst[i + half] = __float2bfloat16_rn(y * co + x * si);
  }
  for (int idx = tid; idx < c.n_kv * hd; idx += 256) {
    const int g = idx / hd, i = idx % hd;
    c.v[off + (long long)g * c.head_stride + i] = __float2bfloat16_rn(load1(v + idx));
  }
  for (int g = tid; g < c.n_kv; g += 256) {
    const long long at = ((long long)seq * c.n_kv + g) * paged_slots(c) + slot;
    if (c.weight) c.weight[at] = 0.f;
    if (c.pos) c.pos[at] = a.pos[n];
  }
  if (tid == 0) atomicMax(c.lens + seq, slot + 1);
}

}  // namespace

cudaError_t launch_paged_append(const PagedView& c, const AppendArgs& a, cudaStream_t st) {
  AppendFreq fr{};
  if (a.rotate)
    for (int i = 0; i < c.head_dim / 2; ++i) fr.inv[i] = std::pow(a.theta, -2.0 * (double)i / (double)c.head_dim);
  if (a.f32)
    append_kernel<float><<<a.n_rows, 256, 0, st>>>(c, a, fr);
  else
    append_kernel<__nv_bfloat16><<<a.n_rows, 256, 0, st>>>(c, a, fr);
  return cudaGetLastError();
}

}  // namespace qmoe
