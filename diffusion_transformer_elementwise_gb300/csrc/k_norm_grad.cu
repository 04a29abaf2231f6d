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
// One CTA per SM, of as many teams as its registers hold.  A team takes rows
// a grid's teams apart and adds its part of gw in registers: each thread owns
// the same columns of every row.  The CTA adds its teams' parts and writes one
// row of `partial`, and a second kernel adds the rows in order: no atomics, so
// the same call gives the same bits.
//
// Few rows (few_rows, with its measurements) take one launch and, up to
// kFewRowsD columns, no workspace: the CTAs are one cluster, and each adds a
// slice of gw's columns out of the others' shared memory.  That saves the host a
// launch and a workspace, and costs the GPU up to 4 us (2^18 elements), which a graph
// of such calls would rather not pay.
//
// Each lane copies the granules it will read itself into its own slots of
// shared memory (cp.async), a row or two ahead, so the copies need no barrier
// and a warp's loads are in flight while it reduces and writes.  Memory bounds
// it: [8160, 4096] bf16 with the skip path, 45 us and 2.5 us for the second kernel, 5.7
// TB/s over both (two units a warp; four took 54.8 us in all).
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

template <class T, int LAYOUT>
struct GradRow {
  using U = Unit<T, LAYOUT>;
  static constexpr int P = U::P;
  // a unit's weights from global memory, offset added
  __device__ __forceinline__ static void weight(const U& unit, const NormGradArgs& a, int j,
                                                F2 (&w)[P]) {
    Granule<T>::widen(unit.load_weight(a.w, j), w);
#pragma unroll
    for (int i = 0; i < P; ++i) w[i] = f2_add(f2(a.offset, a.offset), w[i]);
  }
  // sums of x^2 and of g w x over a lane's elements of one unit (w: offset +
  // weight), x scaled by sc
  __device__ __forceinline__ static void sums(const Raw<16>& xr, const Raw<16>& gr,
                                              const F2 (&w)[P], float sc, F2& s, F2& q) {
    F2 x[P], g[P];
    Granule<T>::widen(xr, x);
    Granule<T>::widen(gr, g);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      x[i] = f2_mul(x[i], f2(sc, sc));
      const F2 t = f2_mul(g[i], w[i]);
      s = f2_fma(x[i], x[i], s);
      q = f2_fma(t, x[i], q);
    }
  }
  // gx of one unit, and g n added to acc
  __device__ __forceinline__ static Raw<16> grad(const Raw<16>& xr, const Raw<16>& gr,
                                                 const F2 (&w)[P], const Raw<16>& skip,
                                                 bool has_skip, RowStat st, F2 (&acc)[P]) {
    F2 x[P], g[P], o[P];
    Granule<T>::widen(xr, x);
    Granule<T>::widen(gr, g);
    const F2 r = f2(st.r, st.r), nk = f2(-st.k, -st.k);
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const F2 n = f2_mul(x[i], r);
      const F2 t = f2_mul(g[i], w[i]);
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
  __device__ __forceinline__ static void put(float* row, const U& unit, int j, const F2 (&v)[P]) {
#pragma unroll
    for (int i = 0; i < P; ++i) {
      const int c = unit.col(j, 2 * i), d = unit.col(j, 2 * i + 1);
      if (c >= 0 && c < unit.D) row[c] = v[i].x;
      if (d >= 0 && d < unit.D) row[d] = v[i].y;
    }
  }
};

// rows staged ahead (shared memory holds one of the widest rows)
template <int NU>
constexpr int kStagesOf = NU == 4 ? 1 : 2;
// most warps of a CTA, which set the registers of a thread: 80 for one unit a
// warp, 96 for two, 128 for four
template <int NU>
constexpr int kGradWarps = NU == 1 ? 24 : NU == 2 ? 20 : 16;

// SKIP: the gradient of the skip path is added.  a.gw (few rows): the grid is
// one cluster, and gw is written here.
template <class T, int LAYOUT, int NU, bool SKIP>
__global__ void __launch_bounds__(kGradWarps<NU> * 32) grad_team_kernel(NormGradArgs a) {
  using R = GradRow<T, LAYOUT>;
  using U = typename R::U;
  constexpr int P = U::P;
  constexpr int NS = SKIP ? 3 : 2;              // streams
  constexpr int kStages = kStagesOf<NU>;
  constexpr bool kStaged = LAYOUT != NARROW;
  constexpr uint32_t kSlot = 32 * 16;           // a unit of one stream
  constexpr uint32_t kStage = NS * NU * kSlot;  // a warp's part of a row
  __shared__ float2 slots[2 * kGradWarps<NU>];
  // weights (not NARROW), [warps][stages][streams][NU][32]; in the end the
  // teams' parts of gw
  extern __shared__ float4 shared[];
  let_next();
  if (blockIdx.x >= a.rows && !a.gw) return;  // (the grid is rounded up for PHASED rows)
  Team t(slots);
  const int lane = t.lane, W = t.warps, m = t.m, team = threadIdx.y, teams = blockDim.y;
  const int ngr = W * NU * 32;  // granules of a row, padded
  const int64_t step = (int64_t)gridDim.x * teams;
  const uint32_t stage0 =
      smem_addr(shared + ngr * (P / 2)) + (team * W + m) * (kStages * kStage) + lane * 16;

  int64_t row = blockIdx.x + (int64_t)gridDim.x * team;
  U unit(a.D, lane, m * NU, NU, blockIdx.x);
  // this warp's part of row r, into stage s (an empty group past the end)
  auto prefetch = [&](int64_t r, int s) {
    if constexpr (kStaged) {
      if (r < a.rows) {
        const int64_t e = unit.at(r);
#pragma unroll
        for (int j = 0; j < NU; ++j) {
          const uint32_t dst = stage0 + s * kStage + j * kSlot;
          unit.copy(dst, a.x, e, j);
          unit.copy(dst + NU * kSlot, a.g, e, j);
          if constexpr (SKIP) unit.copy(dst + 2 * NU * kSlot, a.gres, e, j);
        }
      }
      cp_async_commit();
    }
  };
#pragma unroll
  for (int s = 0; s < kStages; ++s) prefetch(row + s * step, s);

  auto weights = [&](int j, F2(&w)[P]) {
    if constexpr (kStaged)
      staged_weight<T>(shared, ngr, (m * NU + j) * 32 + lane, w);
    else
      R::weight(unit, a, j, w);
  };
  F2 acc[NU][P];
#pragma unroll
  for (int j = 0; j < NU; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) acc[j][i] = f2(0.0f, 0.0f);
  if constexpr (kStaged) {
    stage_weight<T, LAYOUT>(shared, ngr, a.D, blockIdx.x, a.w, a.offset);
    __syncthreads();
  }
  int s = 0;
  for (; row < a.rows; row += step) {
    const int64_t e = unit.at(row);
    Raw<16> x[NU], g[NU], k[NU];
    if constexpr (kStaged) cp_async_wait<kStages - 1>();  // this lane's copies of the row
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      if constexpr (kStaged) {
        const uint32_t at = stage0 + s * kStage + j * kSlot;
        x[j] = unit.copied(at, j);
        g[j] = unit.copied(at + NU * kSlot, j);
        if constexpr (SKIP) k[j] = unit.copied(at + 2 * NU * kSlot, j);
      } else {
        x[j] = unit.load(a.x, e, j);
        g[j] = unit.load(a.g, e, j);
        if constexpr (SKIP) k[j] = unit.load(a.gres, e, j);
      }
    }
    auto row_sums = [&](float sc) {
      F2 s = f2(0.0f, 0.0f), q = s;
#pragma unroll
      for (int j = 0; j < NU; ++j) {
        F2 w[P];
        weights(j, w);
        R::sums(x[j], g[j], w, sc, s, q);
      }
      return make_float2(__fadd_rn(s.x, s.y), __fadd_rn(q.x, q.y));
    };
    const float2 mine = row_sums(1.0f);
    // the stage has been read
    prefetch(row + kStages * step, s);
    s = s + 1 == kStages ? 0 : s + 1;
    auto over_team = [&](float2 v) {
      return t.combine<false>(make_float2(warp_sum(v.x), warp_sum(v.y)));
    };
    const RowStat st = row_stat(over_team(mine), a, [&](float sc) { return over_team(row_sums(sc)); });
#pragma unroll
    for (int j = 0; j < NU; ++j) {
      F2 w[P];
      weights(j, w);
      const Raw<16> o = R::grad(x[j], g[j], w, k[j], SKIP, st, acc[j]);
      unit.store(a.gx, e, j, o);
    }
  }
  if (!a.partial && !a.gw) return;
  float* out = a.partial + (int64_t)blockIdx.x * a.D;
  if (teams == 1 && !a.gw) {
#pragma unroll
    for (int j = 0; j < NU; ++j) R::put(out, unit, j, acc[j]);
    return;
  }
  if constexpr (kStaged) cp_async_wait<0>();
  __syncthreads();  // the stages are no longer read or written
  float* merged = (float*)shared;  // [teams][D]
#pragma unroll
  for (int j = 0; j < NU; ++j) R::put(merged + team * a.D, unit, j, acc[j]);
  __syncthreads();
  const int tid = team * blockDim.x + threadIdx.x, nthr = blockDim.x * teams;
  for (int c = tid; c < a.D; c += nthr) {
    float v = merged[c];
    for (int q = 1; q < teams; ++q) v = __fadd_rn(v, merged[q * a.D + c]);
    if (a.gw)
      merged[c] = v;
    else
      out[c] = v;
  }
  if (!a.gw) return;
  cluster_barrier();
  // columns rank, rank + ctas, ... in runs of 32
  for (int c0 = (tid / 32 * gridDim.x + blockIdx.x) * 32; c0 < a.D; c0 += nthr * gridDim.x) {
    const int c = c0 + lane;
    if (c >= a.D) continue;
    float v[1] = {0.0f};
    for (unsigned r = 0; r < gridDim.x; ++r)
      v[0] = __fadd_rn(v[0], __uint_as_float(ld_cluster(smem_addr(merged + c), r)));
    st_stream<sizeof(T)>((char*)a.gw + (int64_t)c * sizeof(T), Vec<T, (int)sizeof(T)>::narrow(v));
  }
  cluster_barrier();  // the others have read this CTA's part
}

// Rows longer than a CTA's registers: read twice, gw added in the CTA's row
// of `partial` itself (each column by one thread).
template <class T, int LAYOUT>
__global__ void __launch_bounds__(kTeamThreads) grad_long_kernel(NormGradArgs a) {
  using R = GradRow<T, LAYOUT>;
  using U = typename R::U;
  constexpr int P = U::P;
  __shared__ float2 slots[2 * kTeamWarps];
  Team t(slots);
  const int lane = t.lane, warp = t.m, W = t.warps;
  U unit(a.D, lane, warp, 1, 0);  // units warp, warp + W, ...
  const int units = (a.D + U::COLS - 1) / U::COLS - warp;  // from this warp's first
  float* out = a.partial ? a.partial + (int64_t)blockIdx.x * a.D : nullptr;
  bool first = true;
  for (int64_t row = blockIdx.x; row < a.rows; row += gridDim.x, first = false) {
    const int64_t e = unit.at(row);
    auto sums = [&](float sc) {
      LongSum xx, tx;
      for (int j = 0; j < units; j += W) {
        F2 s = f2(0.0f, 0.0f), q = s;
        F2 w[P];
        R::weight(unit, a, j, w);
        R::sums(unit.load(a.x, e, j), unit.load(a.g, e, j), w, sc, s, q);
        xx.add(__fadd_rn(s.x, s.y));
        tx.add(__fadd_rn(q.x, q.y));
      }
      return t.combine<false>(make_float2(warp_sum(xx.total()), warp_sum(tx.total())));
    };
    const RowStat st = row_stat(sums(1.0f), a, sums);
    for (int j = 0; j < units; j += W) {
      F2 acc[P];
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const int c = unit.col(j, 2 * i), d = unit.col(j, 2 * i + 1);
        acc[i] = f2(!first && out && c < a.D ? out[c] : 0.0f, !first && out && d < a.D ? out[d] : 0.0f);
      }
      const Raw<16> k = a.gres ? unit.load(a.gres, e, j) : Raw<16>{};
      F2 w[P];
      R::weight(unit, a, j, w);
      const Raw<16> o = R::grad(unit.load(a.x, e, j), unit.load(a.g, e, j), w, k, a.gres != nullptr, st, acc);
      unit.store(a.gx, e, j, o);
      if (out) R::put(out, unit, j, acc);
    }
  }
}

// gw[c] = the sum of `partial`'s column c over its `n` rows: a CTA takes 32
// columns, its 32 warps the rows w, w + 32, ..., then their sums in order.
struct GradWeight {
  const float* partial;
  int n, D;
  void* gw;
};
template <class T>
__global__ void __launch_bounds__(1024) grad_weight_kernel(GradWeight a) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  after_previous();
  if (c < a.D) {
#pragma unroll 4
    for (int i = warp; i < a.n; i += 32) v = __fadd_rn(v, a.partial[(int64_t)i * a.D + c]);
  }
  part[warp][lane] = v;
  __syncthreads();
  v = warp_sum(part[lane][warp]);  // warp w now holds column w
  const int k = blockIdx.x * 32 + warp;
  if (lane == 0 && k < a.D) {
    float f[1] = {v};
    st_stream<sizeof(T)>((char*)a.gw + (int64_t)k * sizeof(T), Vec<T, (int)sizeof(T)>::narrow(f));
  }
}

// *ctas: the rows of a.partial written; 0 where gw is written already
template <class T, int LAYOUT, bool SKIP>
cudaError_t launch_rows(const DeviceInfo& dev, NormGradArgs a, int64_t* ctas, cudaStream_t s) {
  using U = Unit<T, LAYOUT>;
  const int64_t units = row_units<T, LAYOUT>(a.D);
  auto team = [&](auto nu) -> cudaError_t {
    constexpr int NU = decltype(nu)::value;
    const auto kern = grad_team_kernel<T, LAYOUT, NU, SKIP>;
    const int64_t warps = (units + NU - 1) / NU;
    // few rows: a CTA for each before a second team in any
    int64_t teams = std::max<int64_t>(
        1, std::min<int64_t>(kGradWarps<NU> / warps, (a.rows + dev.sm_count - 1) / dev.sm_count));
    int64_t grid = std::min(std::min<int64_t>(dev.sm_count, kNormGradMaxCtas - 8),
                            (a.rows + teams - 1) / teams);
    if (a.gw) {
      // one cluster: 8 CTAs, 16 for more rows than those hold at once
      teams = kGradWarps<NU> / warps;
      grid = a.rows <= 8 * teams ? 8 : 16;
    }
    // PHASED: a CTA's rows have one offset when they are a multiple of 8 apart
    if (LAYOUT == PHASED) grid = (grid + 7) / 8 * 8;
    size_t smem = 0;
    if (LAYOUT != NARROW)
      smem = (size_t)warps * NU * 512 * (sizeof(T) == 2 ? 2 : 1) +
             (size_t)warps * teams * NU * 512 * kStagesOf<NU> * (SKIP ? 3 : 2);
    if (teams > 1 || a.gw) smem = std::max(smem, (size_t)teams * a.D * 4);
    static std::atomic<int> opted[kOptinDevices];
    cudaError_t e = allow_shared((const void*)kern, dev, opted);
    if (e != cudaSuccess) return e;
    const dim3 block((unsigned)warps * 32, (unsigned)teams);
    if (a.gw) return launch_cluster(kern, (unsigned)grid, block, smem, s, a);
    kern<<<(unsigned)grid, block, smem, s>>>(a);
    *ctas = std::min(grid, a.rows);
    return cudaGetLastError();
  };
  if (units == 1) return team(std::integral_constant<int, 1>{});
  if (units <= 2 * kTeamWarps) return team(std::integral_constant<int, 2>{});
  if (units <= 4 * kTeamWarps) return team(std::integral_constant<int, 4>{});
  if constexpr (LAYOUT == PHASED) {
    return launch_rows<T, NARROW, SKIP>(dev, a, ctas, s);
  } else {
    a.gw = nullptr;
    *ctas = std::min(std::min<int64_t>(2 * dev.sm_count, a.rows), kNormGradMaxCtas);
    grad_long_kernel<T, LAYOUT><<<(unsigned)*ctas, kTeamThreads, 0, s>>>(a);
    return cudaGetLastError();
  }
}

template <class T>
cudaError_t launch(const DeviceInfo& dev, int layout, NormGradArgs a, void* gw, cudaStream_t s) {
  int64_t ctas = 0;
  a.gw = few_rows(a.rows, a.D) ? gw : nullptr;
  const bool skip = a.gres != nullptr;
  const cudaError_t e =
      layout == WIDE     ? (skip ? launch_rows<T, WIDE, true>(dev, a, &ctas, s)
                                 : launch_rows<T, WIDE, false>(dev, a, &ctas, s))
      : layout == PHASED ? (skip ? launch_rows<T, PHASED, true>(dev, a, &ctas, s)
                                 : launch_rows<T, PHASED, false>(dev, a, &ctas, s))
                         : (skip ? launch_rows<T, NARROW, true>(dev, a, &ctas, s)
                                 : launch_rows<T, NARROW, false>(dev, a, &ctas, s));
  if (e != cudaSuccess || !gw || ctas == 0) return e;
  return launch_after(grad_weight_kernel<T>, (unsigned)((a.D + 31) / 32), 1024, 0, s,
                      GradWeight{a.partial, (int)ctas, a.D, gw});
}

}  // namespace

cudaError_t launch_norm_grad(const DeviceInfo& dev, int dtype, int layout, const NormGradArgs& a,
                             void* gw, cudaStream_t s) {
  return dtype == 0   ? launch<__nv_bfloat16>(dev, layout, a, gw, s)
         : dtype == 1 ? launch<__half>(dev, layout, a, gw, s)
                      : launch<float>(dev, layout, a, gw, s);
}

}  // namespace dit
