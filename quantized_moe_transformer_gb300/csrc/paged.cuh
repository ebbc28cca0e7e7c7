// Kernels of the paged key-value cache (host-side launchers): paged_append.cu,
// paged_attention.cu, paged_evict.cu. The operations and the cache's layout
// are defined in include/qmoe.h.
#pragma once

#include "kernels.cuh"

namespace qmoe {

// The cache as the kernels take it. Strides are in elements of 2 bytes.
struct PagedView {
  __nv_bfloat16 *k, *v;
  const int32_t* table;
  int32_t* lens;
  float* weight;
  int32_t* pos;
  long long page_stride, slot_stride, head_stride;
  int n_seqs, n_kv, head_dim, page_log2, n_pages, max_pages;
};

__host__ __device__ __forceinline__ long long paged_slots(const PagedView& c) {
  return (long long)c.max_pages << c.page_log2;
}

// Element offset of (sequence, slot, KV head 0), -1 if the table has no valid
// page there. ``slot`` is below the table's capacity.
__device__ __forceinline__ long long paged_offset(const PagedView& c, int seq, int slot) {
  const int page = __ldg(c.table + (long long)seq * c.max_pages + (slot >> c.page_log2));
  if ((unsigned)page >= (unsigned)c.n_pages) return -1;
  return (long long)page * c.page_stride + (long long)(slot & ((1 << c.page_log2) - 1)) * c.slot_stride;
}

// Entries of sequence ``b``: its length, at most what its table can hold.
__device__ __forceinline__ int paged_len(const PagedView& c, int b) {
  const long long cap = paged_slots(c);
  const int n = c.lens[b];
  return n < 0 ? 0 : n > cap ? (int)cap : n;
}

// Launches ``k`` so that it may start while the kernel ahead of it on the stream
// ends: every kernel launched so waits on the device (griddepcontrol.wait) before
// it touches memory, and allows the next one to start when it starts itself.
template <class... Params, class... Args>
cudaError_t launch_overlapped(void (*k)(Params...), dim3 grid, int threads, size_t smem, int cluster, cudaStream_t st,
                              Args&&... args) {
  cudaLaunchConfig_t cfg{};
  cfg.gridDim = grid;
  cfg.blockDim = dim3((unsigned)threads);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = st;
  cudaLaunchAttribute attr[2]{};
  attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  attr[0].val.programmaticStreamSerializationAllowed = 1;
  attr[1].id = cudaLaunchAttributeClusterDimension;
  attr[1].val.clusterDim.x = (unsigned)cluster;
  attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
  cfg.attrs = attr;
  cfg.numAttrs = cluster > 0 ? 2 : 1;
  return cudaLaunchKernelEx(&cfg, k, static_cast<Params>(args)...);
}

struct AppendArgs {
  const void *q, *k, *v;
  void* q_out;
  const int32_t *seq, *slot, *pos;
  int n_rows, n_heads;
  bool f32, rotate;
  double theta;
  int* status;
};
cudaError_t launch_paged_append(const PagedView& c, const AppendArgs& a, cudaStream_t st);

struct PagedAttnArgs {
  const void* q;
  void* out;
  int n_heads;
  bool f32, accumulate;
  float scale;
  int* status;
  unsigned long long wait_ns;  // bound on a device wait
  bool fault;                  // test-only: the first CTA's first warp never copies its first tile
  void* ws;
};
size_t paged_attention_ws_bytes(const PagedView& c, int n_heads, bool accumulate);
int paged_attention_launches(const PagedView& c, int n_heads, bool accumulate);
cudaError_t launch_paged_attention(const PagedView& c, const PagedAttnArgs& a, cudaStream_t st);

struct EvictArgs {
  const int32_t* next_pos;
  int budget, recent;
  int32_t* lens_out;
  float* weight_out;
  int32_t* pos_out;
  int* status;
  void* ws;
};
size_t cache_evict_ws_bytes(const PagedView& c);
int cache_evict_launches(const PagedView& c, const EvictArgs& a);
cudaError_t launch_cache_evict(const PagedView& c, const EvictArgs& a, cudaStream_t st);

}  // namespace qmoe
