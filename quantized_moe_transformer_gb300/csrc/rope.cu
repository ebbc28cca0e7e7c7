// Rotary positions of rows of queries and keys, and the transpose (the gradient).
//
// "CKE Zip: From Splitting Tokens To Splitting Qwen3.5 Weights", "What PR #382
// Now Splits": the block's queries and keys carry their positions; layouts,
// parts of a head and scaled frequencies have no counterpart there.
#include "paged.cuh"
#include "rope.cuh"
#include "tc.cuh"

namespace qmoe {

namespace {

constexpr int RO_THREADS = 256, RO_ROWS = 32, RO_CTAS_PER_SM = 4;

// A CTA takes ``rows`` rows: first the (cos, sin) of each row's angles into shared
// memory, once for all its heads, then every unit of eight elements is read,
// turned and written by one thread. Each byte is read and written once.
template <typename T>
__global__ void __launch_bounds__(RO_THREADS, 4)
    rope_kernel(const RopeArgs a, int rows, const __grid_constant__ qmoe_rope_desc r) {
  __shared__ float2 turn[RO_ROWS * 128];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int n0 = blockIdx.x * rows, n = min(rows, a.n_rows - n0), tid = threadIdx.x, half = r.dims / 2;
  for (int i = tid; i < n * half; i += RO_THREADS) {
    const int row = i / half, d = i - row * half;
    float2 t = rope_turn(a.pos[n0 + row], r.turns[d], r.scale);
    t.y *= a.sign;
    turn[row * half + d] = t;
  }
  __syncthreads();
  using F = Four<T>;
  using raw = typename F::raw;
  const bool inter = r.layout == QMOE_ROPE_INTERLEAVED;
  const int per_head = a.head_dim / 8, units = (a.q.heads + a.k.heads) * per_head;
  for (int i = tid; i < n * units; i += RO_THREADS) {
    const int row = i / units, hu = i - row * units, h = hu / per_head;
    const RopeUnit u = rope_unit(hu - h * per_head, r.dims, inter);
    const bool is_q = h < a.q.heads;
    const RopeRows& t = is_q ? a.q : a.k;
    const int g = is_q ? h : h - a.q.heads;
    const T* x = static_cast<const T*>(t.x) + (n0 + row) * t.x_row + g * t.x_head;
    T* y = static_cast<T*>(t.y) + (n0 + row) * t.y_row + g * t.y_head;
    float4 p = F::wide(*reinterpret_cast<const raw*>(x + u.a)), q = F::wide(*reinterpret_cast<const raw*>(x + u.b));
    if (u.turned) rope_apply(p, q, turn + row * half + 4 * (hu - h * per_head), inter);
    *reinterpret_cast<raw*>(y + u.a) = F::narrow(p);
    *reinterpret_cast<raw*>(y + u.b) = F::narrow(q);
  }
}

}  // namespace

cudaError_t launch_rope(const qmoe_rope_desc& r, const RopeArgs& a, cudaStream_t st) {
  const int fit = RO_CTAS_PER_SM * device_sm_count();
  int rows = (a.n_rows + fit - 1) / fit;
  if (rows > RO_ROWS) rows = RO_ROWS;
  const dim3 grid((a.n_rows + rows - 1) / rows);
  return a.f32 ? launch_overlapped(rope_kernel<float>, grid, RO_THREADS, 0, 0, st, a, rows, r)
               : launch_overlapped(rope_kernel<__nv_bfloat16>, grid, RO_THREADS, 0, 0, st, a, rows, r);
}

}  // namespace qmoe
