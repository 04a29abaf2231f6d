// k_norm.cu -- weighted RMSNorm with the residual's addition, and an E4M3
// output with dynamic scales.
//
//   s = rnd(hidden + update)                  (stored; or s = x alone)
//   r = 1 / sqrt(mean(s^2) + eps)             (the fast statistic)
//   y = fl(fl(s r) fl(offset + w))
//   out = rnd(y), or E4M3:  scale = max|y| / 448,  code = e4m3(y / scale)
//
// with the maximum over the row or over each 128 columns of it.
//
// The codes need no r: with t = fl(s fl(offset + w)), y / max|y| = t / max|t|,
// so code = e4m3(fl(t m')) with m' = 448 / max|t| as a sum of two fp32 numbers
// (a hardware reciprocal y, 448 y, and the rest of it: about 2^-44 of m' is
// lost) and scale = fl(fl(max|t| r) fl(1 / 448)).  The maximum is taken in the same
// reduction as the sum of squares, and beside t's own roundings a code has the one of
// its product, so few codes round otherwise than those of exact arithmetic.
// Rows whose sum of squares or maximum leaves [2^-100, 2^100] (overflow, infinities, NaN, all
// zero) take y itself: the maximum again, of y, and code = e4m3(y 448 /
// max|y|).  An all-zero row or group has scale 0 and codes 0; a NaN or an
// infinity makes its maximum NaN, so its scale and codes are NaN.
//
// A team of warps holds a row in registers, up to four units of 512 bytes a
// warp, so that each input is read once; longer rows are read twice by one CTA
// each.  What bounds it: memory for the norm in the tensors' type (add, [32640,
// 4096] bf16: 156 us, 6.87 TB/s; odd widths, [8193, 4099]: 45 us); the
// instructions for E4M3 (162 of a warp per unit: [8192, 4096] bf16 in groups of
// 128, 26.6 us, 3.8 TB/s; [4097, 3077] fp16, 24.2 us) and for the plain norm of odd
// widths without an update (131: [8193, 4099] 24.4 us, 5.5 TB/s); the launch for
// few rows (1.75 us).  Some E4M3 entries of 16-bit types spill (4 to 200 bytes).
// Shared by both: fp32 weights in shared memory, so that a row spends no
// instructions on widening them (they took E4M3 groups, [8192, 4096], from 39.5
// to 30.7 us when it was added), and consecutive units per warp, one base address
// each (then to 25.9).
#include <algorithm>

#include "dit_stat.cuh"
#include "dit_token.h"
#include "dit_unit.cuh"

namespace dit {
namespace {

constexpr float kE4M3Max = 448.0f;

__device__ __forceinline__ bool usable(float m) { return m >= 0x1p-100f && m <= 0x1p100f; }

// The factor from values to codes, and the scale, of one row or group.
struct Quant {
  float mul, low, scale;  // codes of t: t (mul + low)
};
// from the maximum of |t| (usable, or zero with a usable sum)
__device__ __forceinline__ Quant quant_of_t(float m, float r) {
  Quant q;
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(m == 0.0f ? 1.0f : m));
  q.mul = m == 0.0f ? 0.0f : __fmul_rn(kE4M3Max, y);
  q.low = m == 0.0f ? 0.0f : __fmul_rn(__fmaf_rn(-q.mul, m, kE4M3Max), y);
  q.scale = __fmul_rn(__fmul_rn(m, r), 1.0f / kE4M3Max);
  return q;
}
// from the maximum of |y|, whatever it is, for values that small_factor
// scaled up where they are so small that 448 / m would overflow
__device__ __forceinline__ float small_factor(float m) { return m < 0x1p-60f ? 0x1p64f : 1.0f; }
__device__ __forceinline__ Quant quant_of_y(float m) {
  Quant q;
  q.mul = m == 0.0f ? 0.0f : __fdiv_rn(kE4M3Max, __fmul_rn(m, small_factor(m)));
  q.low = 0.0f;
  q.scale = __fdiv_rn(m, kE4M3Max);
  return q;
}

template <class T, int LAYOUT>
struct NormRow {
  using U = Unit<T, LAYOUT>;
  static constexpr int P = U::P;
  // 128-column groups of a unit whose maxima a lane helps to find, and the
  // lanes that share one
  static constexpr int NG = LAYOUT == NARROW && sizeof(T) == 2 ? 2 : 1;
  static constexpr int LANES = LAYOUT != NARROW && sizeof(T) == 2 ? 16 : 32;
  static constexpr int BLOCKS = 32 / LANES * NG;  // groups of a unit
  static_assert(LANES * BLOCKS == 32 * NG, "every lane helps with NG groups");

  // hidden + update, rounded (the first value alone without an update)
  __device__ __forceinline__ static Raw<16> add(const Raw<16>& h, const Raw<16>& u) {
    F2 a[P], b[P];
    Granule<T>::widen(h, a);
    Granule<T>::widen(u, b);
#pragma unroll
    for (int i = 0; i < P; ++i) a[i] = f2_add(a[i], b[i]);
    return Granule<T>::narrow(a);
  }
  __device__ __forceinline__ static void weight(const Raw<16>& w, float offset, F2 (&f)[P]) {
    Granule<T>::widen(w, f);
#pragma unroll
    for (int i = 0; i < P; ++i) f[i] = f2_add(f2(offset, offset), f[i]);
  }
  __device__ __forceinline__ static void normed(const Raw<16>& x, const F2 (&w)[P], float r,
                                                F2 (&y)[P]) {
    Granule<T>::widen(x, y);
#pragma unroll
    for (int i = 0; i < P; ++i) y[i] = f2_mul(f2_mul(y[i], f2(r, r)), w[i]);
  }
  // s times the weight, without r
  __device__ __forceinline__ static void weighted(const Raw<16>& x, const F2 (&w)[P], F2 (&t)[P]) {
    Granule<T>::widen(x, t);
#pragma unroll
    for (int i = 0; i < P; ++i) t[i] = f2_mul(t[i], w[i]);
  }
  // columns outside the row hold zero; where r is not finite they became NaN
  __device__ __forceinline__ static void mask(F2 (&y)[P], const U& unit, int j) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = unit.col(j, 2 * i), d = unit.col(j, 2 * i + 1);
      if (c < 0 || c >= unit.D) y[i].x = 0.0f;
      if (d < 0 || d >= unit.D) y[i].y = 0.0f;
    }
  }
  __device__ __forceinline__ static void scale_by(F2 (&v)[P], float f) {
#pragma unroll
    for (int i = 0; i < P; ++i) v[i] = f2_mul(v[i], f2(f, f));
  }
  __device__ __forceinline__ static float max_of(const F2 (&v)[P]) {
    float m = 0.0f;
#pragma unroll
    for (int i = 0; i < P; ++i) m = max_abs3(m, f2_lo(v[i]), f2_hi(v[i]));
    return m;
  }
  __device__ __forceinline__ static Raw<U::EPL> codes(const F2 (&v)[P], const Quant (&q)[NG]) {
    Raw<U::EPL> r;
#pragma unroll
    for (int i = 0; i < P / 2; ++i) {
      const Quant& k = q[NG == 2 ? i : 0];
      const F2 m = f2(k.mul, k.mul), l = f2(k.low, k.low);
      r.w[i] = e4m3x2(f2_fma(v[2 * i], m, f2_mul(v[2 * i], l))) |
               e4m3x2(f2_fma(v[2 * i + 1], m, f2_mul(v[2 * i + 1], l))) << 16;
    }
    return r;
  }
  // the maxima of the lane's groups of a unit
  __device__ __forceinline__ static void group_max(const F2 (&v)[P], float (&m)[NG]) {
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      m[g] = 0.0f;
#pragma unroll
      for (int i = g * P / NG; i < (g + 1) * P / NG; ++i)
        m[g] = max_abs3(m[g], f2_lo(v[i]), f2_hi(v[i]));
#pragma unroll
      for (int o = LANES / 2; o > 0; o >>= 1)
        m[g] = max_nan(m[g], __shfl_xor_sync(0xFFFFFFFFu, m[g], o));
    }
  }

  // unit j of the output, one scale per 128 columns (the whole warp calls;
  // k: the group of this lane's first column; its groups lie inside the unit)
  __device__ __forceinline__ static void emit_groups(const NormArgs& a, U& unit, int64_t row,
                                                     int64_t e, int j, int k, const Raw<16>& x,
                                                     const F2 (&w)[P], float S, float r) {
    F2 v[P];
    weighted(x, w, v);
    float m[NG];
    group_max(v, m);
    Quant q[NG];
    bool slow = !usable(S);
#pragma unroll
    for (int g = 0; g < NG; ++g) {
      q[g] = quant_of_t(m[g], r);
      slow = slow || (m[g] != 0.0f && !usable(m[g]));
    }
    if (__any_sync(0xFFFFFFFFu, slow)) {  // rare
      F2 y[P];
      normed(x, w, r, y);
      mask(y, unit, j);
      group_max(y, m);
      if (slow) {
#pragma unroll
        for (int g = 0; g < NG; ++g) q[g] = quant_of_y(m[g]);
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float f = small_factor(m[NG == 2 ? i / 2 : 0]);
          v[i] = f2_mul(y[i], f2(f, f));
        }
      }
    }
    unit.store8(a.out, e, j, codes(v, q));
    if (unit.lane % LANES == 0) {
#pragma unroll
      for (int g = 0; g < NG; ++g)
        if (k + g < a.groups) a.scales[row * a.groups + k + g] = q[g].scale;
    }
  }
};

// r of a row from its fp32 sum of squares S; a sum outside the usable range
// is taken again, scaled, by `again(scale)` (uniform over the row's threads).
template <class Again>
__device__ __forceinline__ float inverse_rms(float S, const NormArgs& a, Again again) {
  if (fast_sum_in_range(S)) return fast_inverse_rms(S, a.d_f, a.inv_d, a.eps);
  const float sc = fast_rescale(S);
  return fast_inverse_rms_scaled(again(sc), sc, a.d_f, a.inv_d, a.eps);
}

// One row held by a team: its statistic, then its output.  e: unit.at(row);
// x: the lane's granules; weights(j, wf): unit j's weights, offset added;
// after_read(): called once the sums have been formed (the caller's next
// copies).
template <class T, int LAYOUT, int NU, int Q8, class Weights, class AfterRead>
__device__ __forceinline__ void finish_row(const NormArgs& a, Unit<T, LAYOUT>& unit, Team& t,
                                           int64_t row, int64_t e, const Raw<16> (&x)[NU],
                                           Weights weights, AfterRead after_read) {
  using R = NormRow<T, LAYOUT>;
  using U = Unit<T, LAYOUT>;
  constexpr int P = U::P;
  static_assert(!(LAYOUT == PHASED && Q8 == 2), "groups of columns: SHIFTED");
  const int m = t.m, lane = t.lane;

  F2 acc[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
  float big = 0.0f;
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    F2 f[P];
    Granule<T>::widen(x[j], f);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[i & 1] = f2_fma(f[i], f[i], acc[i & 1]);
    if constexpr (Q8 == 1) {
      F2 wf[P], v[P];
      weights(j, wf);
      R::weighted(x[j], wf, v);
      big = max_nan(big, R::max_of(v));
    }
  }
  after_read();
  acc[0] = f2_add(acc[0], acc[1]);
  float2 red = make_float2(warp_sum(__fadd_rn(acc[0].x, acc[0].y)), 0.0f);
  if constexpr (Q8 == 1) red.y = warp_max(big);
  red = t.combine<Q8 == 1>(red);
  const float r = inverse_rms(red.x, a, [&](float sc) {
    float s2 = 0.0f;
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      F2 f[P];
      Granule<T>::widen(x[j], f);
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const float u0 = __fmul_rn(f2_lo(f[i]), sc), u1 = __fmul_rn(f2_hi(f[i]), sc);
        s2 = __fmaf_rn(u1, u1, __fmaf_rn(u0, u0, s2));
      }
    }
    return t.combine<false>(make_float2(warp_sum(s2), 0.0f)).x;
  });

  if constexpr (Q8 == 0) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      F2 wf[P], y[P];
      weights(j, wf);
      R::normed(x[j], wf, r, y);
      unit.store(a.out, e, j, Granule<T>::narrow(y));
    }
  } else if constexpr (Q8 == 2) {
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      F2 wf[P];
      weights(j, wf);
      const int k = (m * NU + j) * R::BLOCKS + lane / R::LANES;  // this lane's group
      R::emit_groups(a, unit, row, e, j, k, x[j], wf, red.x, r);
    }
  } else {
    // one scale per row
    auto emit = [&](Quant q, auto values) {
      Quant all[R::NG];
#pragma unroll
      for (int g = 0; g < R::NG; ++g) all[g] = q;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        F2 wf[P], v[P];
        weights(j, wf);
        values(x[j], wf, v);
        unit.store8(a.out, e, j, R::codes(v, all));
      }
      if (m == 0 && lane == 0) a.scales[row] = q.scale;
    };
    if (usable(red.x) && (red.y == 0.0f || usable(red.y))) {
      emit(quant_of_t(red.y, r),
           [&](const Raw<16>& x, const F2(&wf)[P], F2(&v)[P]) { R::weighted(x, wf, v); });
    } else {  // rare, uniform over the row's threads: the maximum of y
      float my = 0.0f;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        F2 wf[P], y[P];
        weights(j, wf);
        R::normed(x[j], wf, r, y);
        R::mask(y, unit, j);
        my = max_nan(my, R::max_of(y));
      }
      my = t.combine<true>(make_float2(0.0f, warp_max(my))).y;
      const float f = small_factor(my);
      emit(quant_of_y(my), [&](const Raw<16>& x, const F2(&wf)[P], F2(&v)[P]) {
        R::normed(x, wf, r, v);
        R::scale_by(v, f);
      });
    }
  }
}

// A row or a few per team, straight from global memory (WIDE, NARROW): other
// CTAs' loads fill the memory's pipe.
template <class T, int LAYOUT, int NU, bool ADD, int Q8>
__global__ void __launch_bounds__(kTeamThreads, 2) norm_direct_kernel(NormArgs a) {
  using R = NormRow<T, LAYOUT>;
  using U = typename R::U;
  __shared__ float2 slots[2 * kTeamWarps];
  Team t(slots);
  U unit(a.D, t.lane, t.m * NU, NU, 0);
  for (int64_t row = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; row < a.rows;
       row += (int64_t)gridDim.x * blockDim.y) {
    const int64_t e = unit.at(row);
    Raw<16> x[NU], u[NU], w[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      x[j] = unit.load(a.x, e, j);
      if constexpr (ADD) u[j] = unit.load(a.u, e, j);
    }
#pragma unroll
    for (int j = 0; j < NU; ++j) w[j] = unit.load_weight(a.w, j);
    if constexpr (ADD) {
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        x[j] = R::add(x[j], u[j]);
        unit.store(a.res, e, j, x[j]);
      }
    }
    finish_row<T, LAYOUT, NU, Q8>(
        a, unit, t, row, e, x, [&](int j, F2(&wf)[U::P]) { R::weight(w[j], a.offset, wf); }, [] {});
  }
}

// One wave of CTAs over many rows (not NARROW).  The weights lie in shared
// memory as fp32, and each lane copies the granules of its team's next row into its
// own slots of shared memory (cp.async) as soon as it has read the current one out of
// them: the copies need no barrier (SHIFTED: a warp's), and are in flight while
// the team reduces and writes.  A CTA's rows are a multiple of gridDim.x apart, which for
// rows at an offset is a multiple of 8: all at one offset from a granule.
template <class T, int LAYOUT, int NU, bool ADD, int Q8>
__global__ void __launch_bounds__(kTeamThreads, 2) norm_staged_kernel(NormArgs a) {
  using R = NormRow<T, LAYOUT>;
  using U = typename R::U;
  constexpr int NS = ADD ? 2 : 1;  // streams
  // a warp's units of one stream (SHIFTED: and one granule)
  constexpr uint32_t kSlots = NU * 32 * 16 + (LAYOUT == SHIFTED ? 16 : 0);
  static_assert(LAYOUT != NARROW, "cp.async moves granules");
  __shared__ float2 slots[2 * kTeamWarps];
  extern __shared__ float4 shared[];  // weights, then [warps][streams][kSlots bytes]
  Team t(slots);
  const int W = t.warps, m = t.m;
  U unit(a.D, t.lane, m * NU, NU, blockIdx.x);
  const int ngr = W * NU * 32;  // granules of a row, padded
  const int64_t step = (int64_t)gridDim.x * blockDim.y;
  int64_t row = blockIdx.x + (int64_t)gridDim.x * threadIdx.y;
  const uint32_t stage = smem_addr(shared + ngr * (U::P / 2)) +
                         (threadIdx.y * W + m) * (NS * kSlots) + t.lane * 16;
  auto prefetch = [&](int64_t r) {
    if (r < a.rows) {
      const int64_t e = unit.at(r);
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        unit.copy(stage + j * 512, a.x, e, j);
        if constexpr (ADD) unit.copy(stage + kSlots + j * 512, a.u, e, j);
      }
      if (LAYOUT == SHIFTED && t.lane == 0) {
        unit.copy(stage + NU * 512, a.x, e, NU);
        if constexpr (ADD) unit.copy(stage + kSlots + NU * 512, a.u, e, NU);
      }
    }
    cp_async_commit();
  };
  prefetch(row);
  // (SHIFTED: the weights of the columns themselves, as row 0's)
  stage_weight<T, LAYOUT>(shared, ngr, a.D, LAYOUT == SHIFTED ? 0 : blockIdx.x, a.w, a.offset);
  __syncthreads();
  for (; row < a.rows; row += step) {
    const int64_t e = unit.at(row);
    cp_async_wait<0>();  // this lane's copies of the row
    if (LAYOUT == SHIFTED) __syncwarp();  // ... and the other lanes'
    Raw<16> x[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      x[j] = unit.copied(stage + j * 512, j);
      if constexpr (ADD) {
        x[j] = R::add(x[j], unit.copied(stage + kSlots + j * 512, j));
        unit.store(a.res, e, j, x[j]);
      }
    }
    finish_row<T, LAYOUT, NU, Q8>(
        a, unit, t, row, e, x,
        [&](int j, F2(&wf)[U::P]) {
          staged_weight<T>(shared, ngr, (m * NU + j) * 32 + t.lane, wf);
        },
        [&] {
          if (LAYOUT == SHIFTED) __syncwarp();  // every lane has read the slots
          prefetch(row + step);
        });
  }
}

// Rows longer than a CTA's registers: one CTA per row, the row read again for
// the output (with an update, each thread its own stores of the residual).
// A thread's units, thousands of them, are added in levels (LongSum).
template <class T, int LAYOUT, bool ADD, int Q8>
__global__ void __launch_bounds__(kTeamThreads) norm_long_kernel(NormArgs a) {
  using R = NormRow<T, LAYOUT>;
  using U = typename R::U;
  constexpr int P = U::P;
  __shared__ float2 slots[2 * kTeamWarps];
  Team t(slots);
  const int lane = t.lane, warp = t.m, W = t.warps;
  U unit(a.D, lane, warp, 1, 0);  // units warp, warp + W, ...
  const int units = (a.D + U::COLS - 1) / U::COLS - warp;  // from this warp's first

  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x) {
    const void* src = ADD ? a.res : a.x;
    const int64_t e = unit.at(row);
    LongSum sum;
    float big = 0.0f;
    for (int j = 0; j < units; j += W) {
      Raw<16> x = unit.load(a.x, e, j);
      if constexpr (ADD) {
        x = R::add(x, unit.load(a.u, e, j));
        unit.store(a.res, e, j, x);
      }
      F2 f[P];
      Granule<T>::widen(x, f);
      F2 acc = f2_mul(f[0], f[0]);
#pragma unroll
      for (int i = 1; i < P; ++i) acc = f2_fma(f[i], f[i], acc);
      sum.add(__fadd_rn(acc.x, acc.y));
      if constexpr (Q8 == 1) {
        F2 wf[P], v[P];
        R::weight(unit.load_weight(a.w, j), a.offset, wf);
        R::weighted(x, wf, v);
        big = max_nan(big, R::max_of(v));
      }
    }
    float2 red = make_float2(warp_sum(sum.total()), 0.0f);
    if constexpr (Q8 == 1) red.y = warp_max(big);
    red = t.combine<Q8 == 1>(red);
    const float S = red.x;
    big = red.y;
    const float r = inverse_rms(S, a, [&](float sc) {
      LongSum again;
      for (int j = 0; j < units; j += W) {
        F2 f[P];
        Granule<T>::widen(unit.load(src, e, j), f);
        float s2 = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const float u0 = __fmul_rn(f2_lo(f[i]), sc), u1 = __fmul_rn(f2_hi(f[i]), sc);
          s2 = __fmaf_rn(u1, u1, __fmaf_rn(u0, u0, s2));
        }
        again.add(s2);
      }
      return t.combine<false>(make_float2(warp_sum(again.total()), 0.0f)).x;
    });

    bool slow = false;
    float small = 1.0f;
    Quant q[R::NG] = {};
    if constexpr (Q8 == 1) {
      slow = !usable(S) || (big != 0.0f && !usable(big));
      if (slow) {
        float my = 0.0f;
        for (int j = 0; j < units; j += W) {
          F2 wf[P], y[P];
          R::weight(unit.load_weight(a.w, j), a.offset, wf);
          R::normed(unit.load(src, e, j), wf, r, y);
          R::mask(y, unit, j);
          my = max_nan(my, R::max_of(y));
        }
        my = t.combine<true>(make_float2(0.0f, warp_max(my))).y;
        q[0] = quant_of_y(my);
        small = small_factor(my);
      } else {
        q[0] = quant_of_t(big, r);
      }
#pragma unroll
      for (int g = 1; g < R::NG; ++g) q[g] = q[0];
      if (threadIdx.x == 0) a.scales[row] = q[0].scale;
    }
    for (int j = 0; j < units; j += W) {
      const Raw<16> x = unit.load(src, e, j);
      F2 wf[P], v[P];
      R::weight(unit.load_weight(a.w, j), a.offset, wf);
      if constexpr (Q8 == 2) {
        R::emit_groups(a, unit, row, e, j, (warp + j) * R::BLOCKS + lane / R::LANES, x, wf, S, r);
      } else {
        if (Q8 == 0 || slow)
          R::normed(x, wf, r, v);
        else
          R::weighted(x, wf, v);
        if (slow) R::scale_by(v, small);
        if constexpr (Q8 == 0)
          unit.store(a.out, e, j, Granule<T>::narrow(v));
        else
          unit.store8(a.out, e, j, R::codes(v, q));
      }
    }
  }
}

template <class T, int LAYOUT, int NU, bool ADD, int Q8>
cudaError_t launch_direct(const NormArgs& a, int64_t units, cudaStream_t s) {
  const int warps = (int)((units + NU - 1) / NU), teams = warps >= 8 ? 1 : 8 / warps;
  const int64_t grid = std::min<int64_t>((a.rows + teams - 1) / teams, int64_t(1) << 30);
  norm_direct_kernel<T, LAYOUT, NU, ADD, Q8><<<(unsigned)grid, dim3(warps * 32, teams), 0, s>>>(a);
  return cudaGetLastError();
}

template <class T, int LAYOUT, int NU, bool ADD, int Q8>
cudaError_t launch_staged(const DeviceInfo& dev, const NormArgs& a, int64_t units, cudaStream_t s) {
  const auto kern = norm_staged_kernel<T, LAYOUT, NU, ADD, Q8>;
  const int warps = (int)((units + NU - 1) / NU);
  // few rows: a CTA for each before a second team in any
  const int teams = (int)std::max<int64_t>(
      1, std::min<int64_t>(kTeamWarps / warps, (a.rows + dev.sm_count - 1) / dev.sm_count));
  const size_t smem = (size_t)warps * NU * 512 * (sizeof(T) == 2 ? 2 : 1) +
                      (size_t)warps * teams * (NU * 512 + (LAYOUT == SHIFTED ? 16 : 0)) * (ADD ? 2 : 1);
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  const int64_t wave =
      (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, warps * teams * 32, smem);
  int64_t grid = std::min<int64_t>(wave, (a.rows + teams - 1) / teams);
  if (LAYOUT != WIDE) grid = (grid + 7) / 8 * 8;
  kern<<<(unsigned)grid, dim3(warps * 32, teams), smem, s>>>(a);
  return cudaGetLastError();
}

template <class T, int LAYOUT, bool ADD, int Q8>
cudaError_t launch(const DeviceInfo& dev, const NormArgs& a, cudaStream_t s) {
  const int64_t units = row_units<T, LAYOUT>(a.D);
  if constexpr (LAYOUT != NARROW) {
    // PHASED rows; WIDE ones beyond 64 units per SM (bf16, L2-resident below:
    // [1216,2048] 3.6 us direct, 3.3 staged; [608,2048] 2.4 and 2.6;
    // [32768,1024] 37.9 and 19.6), but not the plain output with an update on rows of
    // more than 4 KB ([8192,4096] 41.2 us direct, 45.8 staged; [16384,2048]
    // 51.1 and 44.9); rows that direct CTAs do not hold
    const bool many = a.rows * units > 64 * (int64_t)dev.sm_count;
    const bool staged = LAYOUT == PHASED || units > 2 * kTeamWarps ||
                        (many && !(ADD && Q8 == 0 && units > 8));
    if (staged && units <= 4 * kTeamWarps) {
      // (groups of 128 columns of rows at an offset)
      constexpr int L = LAYOUT == PHASED && Q8 == 2 ? SHIFTED : LAYOUT;
      if (units == 1) return launch_staged<T, L, 1, ADD, Q8>(dev, a, units, s);
      // With an update, two units a warp and twice the warps, which hide more
      // of the memory's latency (E4M3 in groups, [8192,4096]: 39.7 us, with
      // four units 43.7; odd rows [8193,4099]: 44.0 and 48.5; [1,4099]: 3.0 and
      // 4.0), but not for so few units ([30000,768] E4M3: 29.9 and 29.2) nor
      // for E4M3 of odd rows, which gain 2 % ([8192,3001]: 59.7 and 60.8) and
      // keep the bits of the two calls that the fused one stands for.  Without, the instructions bound it, and those of a row's reduction are
      // fewer with four (E4M3, odd [8192,4099]: 29.7 us, with two 32.3).
      if (units == 2 || (ADD && (L == WIDE || Q8 == 0) && units > 4 && units <= 2 * kTeamWarps))
        return launch_staged<T, L, 2, ADD, Q8>(dev, a, units, s);
      return launch_staged<T, L, 4, ADD, Q8>(dev, a, units, s);
    }
  }
  if constexpr (LAYOUT != PHASED) {
    if (units <= 8) return launch_direct<T, LAYOUT, 1, ADD, Q8>(a, units, s);
    if (units <= 2 * kTeamWarps) return launch_direct<T, LAYOUT, 2, ADD, Q8>(a, units, s);
    const int64_t grid = std::min<int64_t>((int64_t)dev.sm_count * 4, a.rows);
    norm_long_kernel<T, LAYOUT, ADD, Q8><<<(unsigned)grid, kTeamThreads, 0, s>>>(a);
    return cudaGetLastError();
  } else {
    return launch<T, NARROW, ADD, Q8>(dev, a, s);
  }
}

template <class T, int LAYOUT>
cudaError_t launch_form(const DeviceInfo& dev, int q8, const NormArgs& a, cudaStream_t s) {
  if (a.u)
    return q8 == 0   ? launch<T, LAYOUT, true, 0>(dev, a, s)
           : q8 == 1 ? launch<T, LAYOUT, true, 1>(dev, a, s)
                     : launch<T, LAYOUT, true, 2>(dev, a, s);
  return q8 == 0   ? launch<T, LAYOUT, false, 0>(dev, a, s)
         : q8 == 1 ? launch<T, LAYOUT, false, 1>(dev, a, s)
                   : launch<T, LAYOUT, false, 2>(dev, a, s);
}

template <class T>
cudaError_t launch_layout(const DeviceInfo& dev, int layout, int q8, const NormArgs& a,
                          cudaStream_t s) {
  return layout == WIDE     ? launch_form<T, WIDE>(dev, q8, a, s)
         : layout == PHASED ? launch_form<T, PHASED>(dev, q8, a, s)
                            : launch_form<T, NARROW>(dev, q8, a, s);
}

}  // namespace

cudaError_t launch_norm(const DeviceInfo& dev, int dtype, int layout, int q8, const NormArgs& a,
                        cudaStream_t s) {
  return dtype == 0   ? launch_layout<__nv_bfloat16>(dev, layout, q8, a, s)
         : dtype == 1 ? launch_layout<__half>(dev, layout, q8, a, s)
                      : launch_layout<float>(dev, layout, q8, a, s);
}

}  // namespace dit
