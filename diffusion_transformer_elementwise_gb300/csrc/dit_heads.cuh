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

// r of a head's norm from its sum of squares (inv_d: fl(1 / D)).
__device__ __forceinline__ float inverse_rms(float sum, float inv_d, float eps) {
  return rsqrtf(__fmaf_rn(sum, inv_d, eps));
}

// The pair (a, b) turned: one product rounded, the other one with the sum.
__device__ __forceinline__ float2 turned(float a, float b, float cos, float sin) {
  return make_float2(__fmaf_rn(a, cos, __fmul_rn(b, -sin)), __fmaf_rn(b, cos, __fmul_rn(a, sin)));
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

// ---------------------------------------------------------------------------
// heads in 16-byte granules
//
// A team of TEAM lanes (a power of two) has a head; a lane has two granules of
// it: those whose columns are turned together (j and j + R), two neighbouring pairs' ones
// where the pairs are adjacent columns, or two that are not turned.  So the partners of every
// rotation are in one lane, and a team's accesses are contiguous.  A warp takes a token, its
// teams the token's heads one beside the other, so that the angles (and the weights) are
// loaded once for all of a token's heads.
// ---------------------------------------------------------------------------

// units of a head: lanes that its granules take
inline int head_units(const RopeArgs& a, int per) {
  const int n = a.D / per, turned = a.interleaved ? 0 : a.R / per;
  return turned + (n - 2 * turned + 1) / 2;
}
// whether heads of T can be cut so: whole granules, each turned wholly or not at all
template <class T>
bool head_granules(const RopeArgs& a) {
  constexpr int per = 16 / (int)sizeof(T);
  return a.granules && (a.interleaved ? 2 * a.R : a.R) % per == 0 && head_units(a, per) <= 32 && a.D > 0;
}

template <class T>
struct HeadLane {
  static constexpr int PER = 16 / (int)sizeof(T);  // columns of a granule
  static constexpr int P = PER / 2;                // pairs of fp32
  int column[2];
  bool on[2], turn[2];
  __device__ __forceinline__ HeadLane(const RopeArgs& a, int unit) {
    const int n = a.D / PER;
    if (a.interleaved) {
      const int half = (n + 1) / 2;
      column[0] = unit * PER;
      column[1] = (unit + half) * PER;
      on[0] = unit < half;
      on[1] = unit + half < n && on[0];
      turn[0] = column[0] < 2 * a.R;
      turn[1] = column[1] < 2 * a.R;
    } else {
      const int t = a.R / PER;
      const bool pair = unit < t;
      column[0] = (pair ? unit : 2 * unit) * PER;  // (2 t + 2 (unit - t))
      column[1] = pair ? (unit + t) * PER : column[0] + PER;
      on[0] = column[0] < a.D;
      on[1] = column[1] < a.D;
      turn[0] = turn[1] = pair;
    }
  }
};

// The angles of a lane's columns.  INTER: cosines twice, sines with their signs, for each granule; else cosines,
// and sines with either sign, for both granules.
template <class T, bool INTER>
struct LaneAngles {
  static constexpr int P = HeadLane<T>::P;
  F2 c[INTER ? 2 : 1][P], s[2][P];
  __device__ __forceinline__ void load(const RopeArgs& a, const HeadLane<T>& h, int64_t row) {
    const float* cs = a.cos + row * a.R;
    const float* sn = a.sin + row * a.R;
    const float sign = a.inverse ? -1.0f : 1.0f;
    if constexpr (INTER) {
#pragma unroll
      for (int k = 0; k < 2; ++k)
#pragma unroll
        for (int i = 0; i < P; ++i) c[k][i] = f2(1.0f, 1.0f), s[k][i] = f2(0.0f, 0.0f);
#pragma unroll
      for (int k = 0; k < 2; ++k) {
        if (!h.on[k] || !h.turn[k]) continue;
        const Raw<P * 4> x = ld_bcast<P * 4>(cs + h.column[k] / 2), y = ld_bcast<P * 4>(sn + h.column[k] / 2);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float u = __uint_as_float(x.w[i]), v = __fmul_rn(sign, __uint_as_float(y.w[i]));
          c[k][i] = f2(u, u);
          s[k][i] = f2(-v, v);
        }
      }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) c[0][i] = f2(1.0f, 1.0f), s[0][i] = s[1][i] = f2(0.0f, 0.0f);
      if (!h.on[0] || !h.turn[0]) return;
#pragma unroll
      for (int i = 0; i < P; i += 2) {
        const Raw<16> x = ld_bcast<16>(cs + h.column[0] + 2 * i), y = ld_bcast<16>(sn + h.column[0] + 2 * i);
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          c[0][i + k] = f2(__uint_as_float(x.w[2 * k]), __uint_as_float(x.w[2 * k + 1]));
          const F2 v = f2(__uint_as_float(y.w[2 * k]), __uint_as_float(y.w[2 * k + 1]));
          s[1][i + k] = f2_mul(v, f2(sign, sign));
          s[0][i + k] = f2_mul(v, f2(-sign, -sign));
        }
      }
    }
  }
  // ALL: every column of a head is turned
  template <bool ALL>
  __device__ __forceinline__ void turn(F2 (&x)[2][P], const HeadLane<T>& h) const {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F2 a = x[0][i], b = x[1][i];
      F2 u, v;
      if constexpr (INTER) {
        u = f2_fma(a, c[0][i], f2_mul(f2(a.y, a.x), s[0][i]));
        v = f2_fma(b, c[1][i], f2_mul(f2(b.y, b.x), s[1][i]));
      } else {
        u = f2_fma(a, c[0][i], f2_mul(b, s[0][i]));
        v = f2_fma(b, c[0][i], f2_mul(a, s[1][i]));
      }
      x[0][i] = ALL || h.turn[0] ? u : a;
      x[1][i] = ALL || h.turn[1] ? v : b;
    }
  }
};

template <class T>
__device__ __forceinline__ void head_load(Raw<16> (&r)[2], const HeadLane<T>& h, const void* p, int64_t at, bool on) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    r[k] = Raw<16>{};
    if (on && h.on[k]) r[k] = ld_stream<16>((const T*)p + at + h.column[k]);
  }
}
template <class T>
__device__ __forceinline__ void head_weight(F2 (&w)[2][HeadLane<T>::P], const HeadLane<T>& h, const void* p, float offset) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    Raw<16> r = {};
    if (h.on[k]) r = ld_bcast<16>((const T*)p + h.column[k]);
    Granule<T>::widen(r, w[k]);
#pragma unroll
    for (int i = 0; i < HeadLane<T>::P; ++i) w[k][i] = f2_add(f2(offset, offset), w[k][i]);
  }
}

// How the heads of a call are given to warps: CTA (x, y) has tokens x WARPS + warp, and so on with a stride of
// gridDim.x WARPS, and block y of the heads: blocks [0, blocks[0]) of `heads` queries, then the keys'.
struct HeadBlocks {
  int heads, blocks[2];
};
// teams: heads that a warp has at once, `ahead` of them a lane
inline HeadBlocks head_blocks(const DeviceInfo& dev, const RopeArgs& a, int teams, int ahead) {
  // all heads of a token, unless that leaves less than 32 warps an SM
  const int64_t most = std::max(a.t[0].H, a.t[1].H), want = (int64_t)dev.sm_count * 32;
  const int64_t split = std::max<int64_t>(1, want / std::max<int64_t>(1, a.tokens));
  int64_t heads = std::max<int64_t>(teams, (most + split - 1) / split);
  heads = (heads + teams - 1) / teams * teams;
  if (heads > (int64_t)teams * ahead) heads = (heads + teams * ahead - 1) / (teams * ahead) * (teams * ahead);
  HeadBlocks b;
  b.heads = (int)heads;
  for (int i = 0; i < 2; ++i) b.blocks[i] = (int)((a.t[i].H + heads - 1) / heads);
  return b;
}

// A token's batch, place and row of angles (tokens < 2^31).
struct TokenAt {
  int64_t batch, place, table;
  __device__ __forceinline__ TokenAt(const RopeArgs& a, uint32_t token) {
    if (a.tokens == a.L) {
      batch = 0;
      place = token;
    } else {
      const uint32_t b = token / (uint32_t)a.L;
      batch = b;
      place = token - b * (uint32_t)a.L;
    }
    table = a.table_rows == a.L ? place : token;
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
