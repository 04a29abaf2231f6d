// k_norm_grad.cu -- the gradient of the weighted RMSNorm.
//
// With n = x r, r = 1 / sqrt(mean(x^2) + eps), y = n (offset + w) and the
// gradient g of y,
//   t  = g (offset + w)
//   gx = r (t - n k) [+ the gradient arriving on the skip path],
//        k = mean(t n) = r sum(t x) / D
//   gw = sum over the rows of g n.
// Both sums of a row, x^2 and t x, are one reduction over the row held in
// registers, and r is formed again from x rather than read.
//
// A CTA takes rows c, c + G, c + 2G, ... and adds its part of gw in
// registers: each thread owns the same columns of every row.  Each CTA writes one
// row of `partial`, and a second kernel adds the rows in order: no atomics, so
// the same call gives the same bits.
#include <algorithm>

#include "dit_stat.cuh"
#include "dit_token.h"
#include "dit_unit.cuh"

namespace dit {
namespace {

// Rows whose sum of squares is outside the usable range are summed again from
// x scaled by sc; k then needs r / sc.
struct RowStat {
  float r, k;
};
template <class Again>
__device__ __forceinline__ RowStat row_stat(float2 sums, const NormGradArgs& a, Again again) {
  RowStat o;
  if (fast_sum_in_range(sums.x)) {
    o.r = fast_inverse_rms(sums.x, a.d_f, a.inv_d, a.eps);
    o.k = __fmul_rn(__fmul_rn(sums.y, a.inv_d), o.r);
  } else {
    const float sc = fast_rescale(sums.x);
    const float2 s2 = again(sc);
    o.r = fast_inverse_rms_scaled(s2.x, sc, a.d_f, a.inv_d, a.eps);
    o.k = __fmul_rn(__fmul_rn(s2.y, a.inv_d), __fmul_rn(o.r, sc < 1.0f ? 0x1p64f : 0x1p-64f));
  }
  return o;
}

template <class T, bool WIDE>
struct GradRow {
  using U = Unit<T, WIDE>;
  static constexpr int P = U::P;
  // sums of x^2 and of g (offset + w) x over a lane's elements of one unit,
  // x scaled by sc
  __device__ __forceinline__ static void sums(const Raw<16>& xr, const Raw<16>& gr,
                                              const Raw<16>& wr, float offset, float sc, F2& s,
                                              F2& q) {
    F2 x[P], g[P], w[P];
    Granule<T>::widen(xr, x);
    Granule<T>::widen(gr, g);
    Granule<T>::widen(wr, w);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = f2_mul(x[i], f2(sc, sc));
      const F2 t = f2_mul(g[i], f2_add(f2(offset, offset), w[i]));
      s = f2_fma(x[i], x[i], s);
      q = f2_fma(t, x[i], q);
    }
  }
  // gx of one unit, and g n added to acc
  __device__ __forceinline__ static Raw<16> grad(const Raw<16>& xr, const Raw<16>& gr,
                                                 const Raw<16>& wr, const Raw<16>& skip,
                                                 bool has_skip, float offset, RowStat st,
                                                 F2 (&acc)[P]) {
    F2 x[P], g[P], w[P], o[P];
    Granule<T>::widen(xr, x);
    Granule<T>::widen(gr, g);
    Granule<T>::widen(wr, w);
    const F2 r = f2(st.r, st.r), nk = f2(-st.k, -st.k);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F2 n = f2_mul(x[i], r);
      const F2 t = f2_mul(g[i], f2_add(f2(offset, offset), w[i]));
      acc[i] = f2_fma(g[i], n, acc[i]);
      o[i] = f2_mul(f2_fma(n, nk, t), r);
    }
    if (has_skip) {
      F2 k[P];
      Granule<T>::widen(skip, k);
#pragma unroll
      for (int i = 0; i < P; ++i) o[i] = f2_add(o[i], k[i]);
    }
    return Granule<T>::narrow(o);
  }
  // a lane's elements of one unit of fp32 columns (partial sums)
  __device__ __forceinline__ static void put(float* row, int c0, int D, int lane, const F2 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = U::col(c0, lane, 2 * i), d = U::col(c0, lane, 2 * i + 1);
      if (c < D) row[c] = v[i].x;
      if (d < D) row[d] = v[i].y;
    }
  }
};

template <class T, bool WIDE, int NU>
__global__ void __launch_bounds__(kTeamThreads) grad_team_kernel(NormGradArgs a) {
  using R = GradRow<T, WIDE>;
  using U = typename R::U;
  constexpr int P = U::P;
  __shared__ float2 slots[2 * kTeamWarps];
  extern __shared__ float merged[];  // [teams][warps * NU * U::COLS], more than one team
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int W = a.warps, teams = (blockDim.x >> 5) / W;
  const int team = warp / W, m = warp - team * W;
  Team t{slots + team * 2 * W, W, m, 1 + team, 0};
  const int64_t pitch = (int64_t)a.D * (int)sizeof(T);

  Raw<16> w[NU];
  F2 acc[NU][P];
#pragma unroll
  for (int j = 0; j < NU; ++j) {
    w[j] = U::load_weight(a.w, (m + j * W) * U::COLS, a.D, lane);
#pragma unroll
    for (int i = 0; i < P; ++i) acc[j][i] = f2(0.0f, 0.0f);
  }
  for (int64_t row = (int64_t)blockIdx.x * teams + team; row < a.rows;
       row += (int64_t)gridDim.x * teams) {
    Raw<16> x[NU], g[NU], k[NU];
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const int c0 = (m + j * W) * U::COLS;
      x[j] = U::load((const char*)a.x + row * pitch, c0, a.D, lane);
      g[j] = U::load((const char*)a.g + row * pitch, c0, a.D, lane);
      k[j] = Raw<16>{};
      if (a.gres) k[j] = U::load((const char*)a.gres + row * pitch, c0, a.D, lane);
    }
    auto sums = [&](float sc) {
      F2 s = f2(0.0f, 0.0f), q = s;
#pragma unroll
      for (int j = 0; j < NU; ++j) R::sums(x[j], g[j], w[j], a.offset, sc, s, q);
      return t.combine<false>(
          make_float2(warp_sum(__fadd_rn(s.x, s.y)), warp_sum(__fadd_rn(q.x, q.y))));
    };
    const RowStat st = row_stat(sums(1.0f), a, sums);
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      const Raw<16> o = R::grad(x[j], g[j], w[j], k[j], a.gres != nullptr, a.offset, st, acc[j]);
      U::store((char*)a.gx + row * pitch, (m + j * W) * U::COLS, a.D, lane, o);
    }
  }
  if (!a.partial) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.D;
  if (teams == 1) {
#pragma unroll
    for (int j = 0; j < NU; ++j) R::put(out, (m + j * W) * U::COLS, a.D, lane, acc[j]);
  } else {
    const int cols = W * NU * U::COLS;
#pragma unroll
    for (int j = 0; j < NU; ++j) R::put(merged + team * cols, (m + j * W) * U::COLS, a.D, lane, acc[j]);
    __syncthreads();
    for (int c = threadIdx.x; c < a.D; c += blockDim.x) {
      float v = merged[c];
      for (int q = 1; q < teams; ++q) v = __fadd_rn(v, merged[q * cols + c]);
      out[c] = v;
    }
  }
}

// Rows longer than a CTA's registers: read twice, gw added in the CTA's row
// of `partial` itself (each column by one thread).
template <class T, bool WIDE>
__global__ void __launch_bounds__(1024) grad_long_kernel(NormGradArgs a) {
  using R = GradRow<T, WIDE>;
  using U = typename R::U;
  constexpr int P = U::P;
  __shared__ double2 part[32];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, W = blockDim.x >> 5;
  const int64_t pitch = (int64_t)a.D * (int)sizeof(T);
  float* out = a.partial ? a.partial + (int64_t)blockIdx.x * a.D : nullptr;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false) {
    const char* xp = (const char*)a.x + row * pitch;
    const char* gp = (const char*)a.g + row * pitch;
    auto sums = [&](float sc) {
      double2 v = make_double2(0.0, 0.0);
      for (int c0 = warp * U::COLS; c0 < a.D; c0 += W * U::COLS) {
        F2 s = f2(0.0f, 0.0f), q = s;
        R::sums(U::load(xp, c0, a.D, lane), U::load(gp, c0, a.D, lane),
                U::load_weight(a.w, c0, a.D, lane), a.offset, sc, s, q);
        v.x += (double)__fadd_rn(s.x, s.y);
        v.y += (double)__fadd_rn(q.x, q.y);
      }
#pragma unroll
      for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xFFFFFFFFu, v.x, o);
        v.y += __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
      }
      __syncthreads();  // the previous sums have been read
      if (lane == 0) part[warp] = v;
      __syncthreads();
      v = make_double2(0.0, 0.0);
      for (int k = 0; k < W; ++k) {
        v.x += part[k].x;
        v.y += part[k].y;
      }
      return make_float2((float)v.x, (float)v.y);
    };
    const RowStat st = row_stat(sums(1.0f), a, sums);
    for (int c0 = warp * U::COLS; c0 < a.D; c0 += W * U::COLS) {
      F2 acc[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = U::col(c0, lane, 2 * i), d = U::col(c0, lane, 2 * i + 1);
        acc[i] = f2(!first && out && c < a.D ? out[c] : 0.0f, !first && out && d < a.D ? out[d] : 0.0f);
      }
      const Raw<16> k = a.gres ? U::load((const char*)a.gres + row * pitch, c0, a.D, lane) : Raw<16>{};
      const Raw<16> o = R::grad(U::load(xp, c0, a.D, lane), U::load(gp, c0, a.D, lane),
                                U::load_weight(a.w, c0, a.D, lane), k, a.gres != nullptr, a.offset,
                                st, acc);
      U::store((char*)a.gx + row * pitch, c0, a.D, lane, o);
      if (out) R::put(out, c0, a.D, lane, acc);
    }
  }
}

// gw[c] = the sum of `partial`'s column c over its `n` rows: a CTA takes 32
// columns, its 32 warps the rows w, w + 32, ..., then their sums in order.
template <class T>
__global__ void __launch_bounds__(1024) grad_weight_kernel(const float* partial, int n, int D, void* gw) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  if (c < D)
    for (int i = warp; i < n; i += 32) v = __fadd_rn(v, partial[(int64_t)i * D + c]);
  part[warp][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][warp]);  // warp w now holds column w
  const int k = blockIdx.x * 32 + warp;
  if (lane == 0 && k < D) {
    float f[1] = {v};
    st_stream<sizeof(T)>((char*)gw + (int64_t)k * sizeof(T), Vec<T, (int)sizeof(T)>::narrow(f));
  }
}

template <class T, bool WIDE>
cudaError_t launch(const DeviceInfo& dev, NormGradArgs a, void* gw, cudaStream_t s) {
  using U = Unit<T, WIDE>;
  const int64_t units = (a.D + U::COLS - 1) / U::COLS;
  int64_t grid = 0;
  auto team = [&](auto nu) {
    constexpr int NU = decltype(nu)::value;
    const TeamShape t = team_shape(units, NU);
    a.warps = t.warps;
    const int block = t.warps * t.teams * 32;
    const size_t smem = t.teams > 1 ? (size_t)t.teams * t.warps * NU * U::COLS * 4 : 0;
    const void* fn = (const void*)grad_team_kernel<T, WIDE, NU>;
    grid = (int64_t)dev.sm_count * resident_ctas(dev, fn, block, smem);
    grid = std::min(grid, std::min(kNormGradMaxCtas, (a.rows + t.teams - 1) / t.teams));
    grad_team_kernel<T, WIDE, NU><<<(unsigned)grid, block, smem, s>>>(a);
  };
  if (units <= 8) {
    team(std::integral_constant<int, 1>{});
  } else if (units <= 2 * kTeamWarps) {
    team(std::integral_constant<int, 2>{});
  } else if (units <= 4 * kTeamWarps) {
    team(std::integral_constant<int, 4>{});
  } else {
    grid = std::min(std::min<int64_t>(dev.sm_count, a.rows), kNormGradMaxCtas);
    grad_long_kernel<T, WIDE><<<(unsigned)grid, 1024, 0, s>>>(a);
  }
  const cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || !gw) return e;
  grad_weight_kernel<T><<<(unsigned)((a.D + 31) / 32), 1024, 0, s>>>(a.partial, (int)grid, a.D, gw);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_norm_grad(const DeviceInfo& dev, int dtype, bool wide, const NormGradArgs& a,
                             void* gw, cudaStream_t s) {
  switch (dtype) {
    case 0:
      return wide ? launch<__nv_bfloat16, true>(dev, a, gw, s) : launch<__nv_bfloat16, false>(dev, a, gw, s);
    case 1:
      return wide ? launch<__half, true>(dev, a, gw, s) : launch<__half, false>(dev, a, gw, s);
    default:
      return wide ? launch<float, true>(dev, a, gw, s) : launch<float, false>(dev, a, gw, s);
  }
}

}  // namespace dit
