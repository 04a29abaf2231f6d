// dit_heads.cuh -- device helpers shared by the operators around attention.
#pragma once

#include <algorithm>

#include "dit_attend.h"
#include "dit_device.cuh"
#include "dit_unit.cuh"

namespace dit {

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

// The sum over the N lanes of an aligned group, in every one of them.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// The largest magnitude of N lanes' v (not negative), NaN if any is.
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// r of a head's norm from its sum of squares: each step correctly rounded.
__device__ __forceinline__ float inverse_rms(float sum, int D, float eps) {
  return __frcp_rn(__fsqrt_rn(__fadd_rn(__fdiv_rn(sum, (float)D), eps)));
}

// The pair (a, b) turned: products and sums rounded one by one.
__device__ __forceinline__ float2 turned(float a, float b, float cos, float sin) {
  return make_float2(__fadd_rn(__fmul_rn(a, cos), -__fmul_rn(b, sin)),
                     __fadd_rn(__fmul_rn(b, cos), __fmul_rn(a, sin)));
}

// Head number i of all tokens' heads (the queries' before the keys').
struct HeadRow {
  int tensor, head;
  int64_t batch, place, table;  // table: its row of cos and sin
  __device__ __forceinline__ HeadRow(const RopeArgs& a, int64_t i, int heads) {
    const int64_t token = i / heads;
    head = (int)(i - token * heads);
    tensor = head >= a.t[0].H;
    if (tensor) head -= a.t[0].H;
    batch = token / a.L;
    place = token - batch * a.L;
    table = a.table_rows == a.L ? place : token;
  }
  __device__ __forceinline__ int64_t at(const dit_heads& t) const {
    return batch * t.batch + place * t.token + head * t.head;
  }
};

// scale and factors to codes of a row whose largest magnitude is m: codes of x are
// e4m3(fl(x (mul + low))), 448 / m as two fp32 numbers.  Rows so small that
// 448 / m would overflow are scaled up first (small).  m not finite: all NaN.
struct RowQuant {
  float mul, low, small, scale;
};
__device__ __forceinline__ RowQuant row_quant(float m) {
  constexpr float most = 448.0f;
  RowQuant q;
  q.small = m < 0x1p-60f ? 0x1p64f : 1.0f;
  const float v = __fmul_rn(m, q.small);
  const bool zero = m == 0.0f;
  q.mul = zero ? 0.0f : __fdiv_rn(most, v);
  q.low = zero ? 0.0f : __fdiv_rn(__fmaf_rn(-q.mul, v, most), v);
  q.scale = __fdiv_rn(m, most);
  if (!isfinite(m)) q.mul = q.low = q.scale = __int_as_float(0x7FC00000);
  return q;
}
__device__ __forceinline__ float code_value(float x, const RowQuant& q) {
  const float v = __fmul_rn(x, q.small);
  return __fmaf_rn(v, q.mul, __fmul_rn(v, q.low));
}

// E4M3 code -> fp32
__device__ __forceinline__ float2 from_e4m3x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float from_e4m3(uint8_t code) { return from_e4m3x2(code).x; }

// Entry i of an int32 or int64 array.
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i, bool wide) {
  return wide ? ((const int64_t*)ids)[i] : ((const int32_t*)ids)[i];
}

}  // namespace dit
