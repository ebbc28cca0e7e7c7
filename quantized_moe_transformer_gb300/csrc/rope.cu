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

constexpr int RO_THREADS = 256, RO_TURNS = 4096, RO_CTAS_PER_SM = 3, RO_WAVES = 6;

// A piece of a head: 16 bytes of it, or 8 of bf16 rows whose turned part is no multiple of 16.
template <typename T, int N>
struct Piece;
template <>
struct Piece<float, 4> {
  using raw = float4;
  static __device__ __forceinline__ void wide(raw v, float* f) {
    f[0] = v.x; f[1] = v.y; f[2] = v.z; f[3] = v.w;
  }
  static __device__ __forceinline__ raw narrow(const float* f) { return make_float4(f[0], f[1], f[2], f[3]); }
};
template <int N>
struct Piece<__nv_bfloat16, N> {
  struct __align__(2 * N) raw {
    uint32_t w[N / 2];
  };
  static __device__ __forceinline__ void wide(const raw& v, float* f) {
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
      f[2 * i] = __uint_as_float(v.w[i] << 16);
      f[2 * i + 1] = __uint_as_float(v.w[i] & 0xFFFF0000u);
    }
  }
  static __device__ __forceinline__ raw narrow(const float* f) {
    raw v;
#pragma unroll
    for (int i = 0; i < N / 2; ++i) v.w[i] = tc::pack_bf16x2(f[2 * i], f[2 * i + 1]);
    return v;
  }
};

// A CTA takes ``rows`` rows: first the (cos, sin) of each row's angles into shared
// memory, once for all its heads, while the first elements are on their way; then every unit, two pieces of N
// elements that turn together, is read, turned and written by one thread, U units of a thread in flight. Each
// byte is read and written once. 16384 bf16 rows of 16 + 2 heads of 128 out of a joint projection, 151 MB: 27.1 us, 5.6
// TB/s, 0.82 of the copy rate; issue slots are half used (angles, places, conversions); one row 2.2 us, the launch.
template <typename T, int N, bool INTER>
__global__ void __launch_bounds__(RO_THREADS, RO_CTAS_PER_SM)
    rope_kernel(const RopeArgs a, int rows, const __grid_constant__ qmoe_rope_desc r) {
  constexpr int U = 4;
  using P = Piece<T, N>;
  using raw = typename P::raw;
  __shared__ float2 turn[RO_TURNS];
  tc::grid_dep_launch();
  tc::grid_dep_wait();
  const int n0 = blockIdx.x * rows, n = min(rows, a.n_rows - n0), tid = threadIdx.x, half = r.dims / 2;
  const int per_head = a.head_dim / (2 * N), units = (a.q.heads + a.k.heads) * per_head, all = n * units;
  bool turned_up = false;
  for (int i0 = tid; i0 - tid < all; i0 += U * RO_THREADS) {
    raw x[U], y[U];
    T* to[U];
    int at[U], apart[U];  // the unit's first angle in ``turn`` (-1: it does not turn), and its second piece
#pragma unroll
    for (int k = 0; k < U; ++k) {
      const int i = i0 + k * RO_THREADS;
      if (i >= all) break;
      const int row = i / units, hu = i - row * units, h = hu / per_head, u = hu - h * per_head;
      const bool turns = 2 * N * u < r.dims, apart_half = turns && !INTER, is_q = h < a.q.heads;
      const RopeRows& t = is_q ? a.q : a.k;
      const int g = is_q ? h : h - a.q.heads, first = apart_half ? N * u : 2 * N * u;
      apart[k] = apart_half ? half : N;
      at[k] = turns ? row * half + u : -1;
      const T* from = static_cast<const T*>(t.x) + (n0 + row) * t.x_row + g * t.x_head + first;
      to[k] = static_cast<T*>(t.y) + (n0 + row) * t.y_row + g * t.y_head + first;
      x[k] = *reinterpret_cast<const raw*>(from);
      y[k] = *reinterpret_cast<const raw*>(from + apart[k]);
    }
    if (!turned_up) {
      for (int i = tid; i < n * half; i += RO_THREADS) {
        // (the units' e-th angles side by side)
        const int row = i / half, d = i - row * half;
        float2 t = rope_turn(a.pos[n0 + row], r.turns[d], r.scale);
        t.y *= a.sign;
        turn[row * half + (d % N) * (half / N) + d / N] = t;
      }
      __syncthreads();
      turned_up = true;
    }
#pragma unroll
    for (int k = 0; k < U; ++k) {
      if (i0 + k * RO_THREADS >= all) break;
      float p[2 * N];
      P::wide(x[k], p);
      P::wide(y[k], p + N);
      if (at[k] >= 0) {
        const float2* t = turn + at[k];
#pragma unroll
        for (int e = 0; e < N; ++e) {
          rope_pair(p[INTER ? 2 * e : e], p[INTER ? 2 * e + 1 : N + e], t[e * (half / N)]);
        }
      }
      *reinterpret_cast<raw*>(to[k]) = P::narrow(p);
      *reinterpret_cast<raw*>(to[k] + apart[k]) = P::narrow(p + N);
    }
  }
}

template <typename T, int N>
cudaError_t rope_rows(const qmoe_rope_desc& r, const RopeArgs& a, cudaStream_t st) {
  // several CTAs after one another on an SM, so that some form their angles while others move rows (16384 rows in one wave
  // 30.3 us, in 3 28.1, in 6 27.1)
  const int fit = RO_WAVES * RO_CTAS_PER_SM * device_sm_count();
  int rows = (int)(((long long)a.n_rows + fit - 1) / fit);
  if (rows > 2 * RO_TURNS / r.dims) rows = 2 * RO_TURNS / r.dims;
  const dim3 grid((unsigned)(((long long)a.n_rows + rows - 1) / rows));
  return r.layout == QMOE_ROPE_INTERLEAVED
             ? launch_overlapped(rope_kernel<T, N, true>, grid, RO_THREADS, 0, 0, st, a, rows, r)
             : launch_overlapped(rope_kernel<T, N, false>, grid, RO_THREADS, 0, 0, st, a, rows, r);
}

}  // namespace

cudaError_t launch_rope(const qmoe_rope_desc& r, const RopeArgs& a, cudaStream_t st) {
  if (a.f32) return rope_rows<float, 4>(r, a, st);
  return r.dims % 16 == 0 && a.head_dim % 16 == 0 ? rope_rows<__nv_bfloat16, 8>(r, a, st)
                                                  : rope_rows<__nv_bfloat16, 4>(r, a, st);
}

}  // namespace qmoe
