// Rotary positions: the angle of a position and the turning of eight elements,
// shared by the calls that turn rows (rope.cu) and that append them
// (paged_append.cu). The operation is defined in include/qmoe.h.
#pragma once

#include "kernels.cuh"

namespace qmoe {

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

// (cos, sin) of ``pos`` times the angle whose turns are ``turns`` / 2^64, times
// ``scale``. Whole turns drop out of the product modulo 2^64, and quarter turns are
// taken off in integers too: what is left is at most an eighth of a turn and is
// rounded to fp32 relative to itself, so that both results are off by about 2^-23
// of ``scale`` at any position (sincospif, at most 2 units in the last place).
__device__ __forceinline__ float2 rope_turn(int pos, uint64_t turns, float scale) {
  const uint64_t frac = (uint64_t)(long long)pos * turns;
  const uint64_t quarter = (frac + (1ull << 61)) >> 62;
  const long long rest = (long long)(frac - (quarter << 62));
  float s, k;
  sincospif((float)rest * 1.0842021724855044e-19f, &s, &k);  // 2^-63: half turns
  if (quarter & 1) {
    const float t = s;
    s = k;
    k = -t;
  }
  const float f = (quarter & 2) ? -scale : scale;
  return make_float2(k * f, s * f);
}

// Places of a head's u-th unit: four elements from ``a`` on and four from ``b``
// on, turned by the angles 4 u' .. 4 u' + 3 where ``turned``.
struct RopeUnit {
  int a, b;
  bool turned;
};

__device__ __forceinline__ RopeUnit rope_unit(int u, int dims, bool interleaved) {
  const bool turned = 8 * u < dims;
  if (turned && !interleaved) return RopeUnit{4 * u, 4 * u + dims / 2, true};
  return RopeUnit{8 * u, 8 * u + 4, turned};
}

// The pair (v, w) turned by (cos, sin): the same roundings wherever it is called.
__device__ __forceinline__ void rope_pair(float& v, float& w, float2 t) {
  const float a = v, b = w;
  v = __fmaf_rn(a, t.x, -__fmul_rn(b, t.y));
  w = __fmaf_rn(b, t.x, __fmul_rn(a, t.y));
}

// The unit's elements p (from a) and q (from b) turned by the four (cos, sin) t0 .. t3.
__device__ __forceinline__ void rope_apply(float4& p, float4& q, float2 t0, float2 t1, float2 t2, float2 t3,
                                           bool interleaved) {
  if (interleaved) {
    rope_pair(p.x, p.y, t0);
    rope_pair(p.z, p.w, t1);
    rope_pair(q.x, q.y, t2);
    rope_pair(q.z, q.w, t3);
  } else {
    rope_pair(p.x, q.x, t0);
    rope_pair(p.y, q.y, t1);
    rope_pair(p.z, q.z, t2);
    rope_pair(p.w, q.w, t3);
  }
}

struct RopeRows {
  const void* x;
  void* y;
  int heads;
  long long x_row, x_head, y_row, y_head;
};

struct RopeArgs {
  RopeRows q, k;  // k.heads 0: none
  const int32_t* pos;
  int n_rows, head_dim;
  bool f32;
  float sign;  // -1: the transpose
};
cudaError_t launch_rope(const qmoe_rope_desc& r, const RopeArgs& a, cudaStream_t st);

}  // namespace qmoe
