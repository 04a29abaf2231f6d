// k_rope.cu -- rotary angles, and the rotation of queries and keys with or
// without the norm of each head (sm_103a).
//
//   angle[t, j] = position * freq,   cos and sin in fp32
//   y = x r (offset + w),  r = 1 / sqrt(mean(x^2) + eps)      (norm)
//   a' = a cos - b sin,  b' = b cos + a sin                     per pair (a, b)
//
// Both are bound by memory: a rotation reads and writes each element once, and the
// angles once for all of a token's heads.  Times are GPU times of a call in a
// replayed graph.
#include <math_constants.h>

#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {
namespace {

// ---------------------------------------------------------------------------
// the table
// ---------------------------------------------------------------------------

constexpr int kTableThreads = 512, kTablePairs = 512;

// The frequencies in turns per unit: for integer positions |f| modulo one turn as a 64-bit fraction (a position
// times it, modulo 2^64, is the angle whatever the position), for fp32 ones as the sum of three fp32 numbers.
// Made once a CTA: fp64 comes at two operations a clock and SM.
template <class P>
struct Turns;
template <>
struct Turns<int64_t> {
  uint64_t fraction;
  uint32_t flags;  // 1: negative, 2: not finite
  __device__ __forceinline__ explicit Turns(double freq) {
    const double f = freq * 0.15915494309189535, m = fabs(f);  // 1 / (2 pi)
    fraction = isfinite(freq) ? __double2ull_rn((m - floor(m)) * 18446744073709551616.0) : 0;
    flags = (f < 0.0 ? 1 : 0) | (isfinite(freq) ? 0 : 2);
  }
  Turns() = default;
};
template <>
struct Turns<float> {
  float part[3];
  uint32_t flags;
  __device__ __forceinline__ explicit Turns(double freq) {
    double f = freq * 0.15915494309189535;
    flags = 0;
    if (!isfinite(freq)) f = CUDART_NAN;
#pragma unroll
    for (int i = 0; i < 3; ++i) {
      part[i] = (float)f;
      f -= (double)part[i];
    }
  }
  Turns() = default;
};
// An angle as a quarter of a turn, modulo four, and the turns from it, at most 1/8.
struct Angle {
  int quarter;  // its last two bits
  float rest;
};
__device__ __forceinline__ Angle angle_of(const Turns<int64_t>& f, int64_t position) {
  const uint64_t x = (uint64_t)position * f.fraction;
  const uint64_t quarter = (x + (uint64_t(1) << 61)) >> 62;
  const int64_t rest = (int64_t)(x - (quarter << 62));
  // (both halves to fp32: small angles keep their digits)
  return Angle{(int)quarter, __fmaf_rn((float)(uint32_t)rest, 0x1p-64f, __fmul_rn((float)(int32_t)(rest >> 32), 0x1p-32f))};
}
__device__ __forceinline__ Angle angle_of(const Turns<float>& f, float p) {
  // the products' high parts and errors
  const float h0 = __fmul_rn(p, f.part[0]), l0 = __fmaf_rn(p, f.part[0], -h0);
  const float h1 = __fmul_rn(p, f.part[1]), l1 = __fmaf_rn(p, f.part[1], -h1);
  const float rest = __fmaf_rn(p, f.part[2], l1);
  constexpr float shift = 12582912.0f;  // 1.5 2^23: a sum with it ends in whole numbers
  float sum;
  if (fabsf(h0) < 0x1p22f) {  // then the other parts are below 1/2, and shift rounds
    sum = __fadd_rn(__fadd_rn(h0, -__fadd_rn(__fadd_rn(h0, shift), -shift)), __fadd_rn(l0, __fadd_rn(h1, rest)));
  } else {  // each without its whole turns; NaN where h0 is not finite
    auto fraction = [](float v) { return __fadd_rn(v, -rintf(v)); };
    sum = __fadd_rn(fraction(h0), __fadd_rn(fraction(l0), __fadd_rn(fraction(h1), fraction(rest))));
  }
  const float quarter = __fmaf_rn(sum, 4.0f, shift);
  return Angle{__float_as_int(quarter), __fmaf_rn(__fadd_rn(quarter, -shift), -0.25f, sum)};
}
// Its cosine and sine: Taylor's series of the rest, which is at most pi / 4 (the first terms left out: x^10 / 10! and
// x^11 / 11!, below 2^-25), and a quarter turn's exchange and signs.
__device__ __forceinline__ float2 cos_sin(const Angle& a) {
  constexpr float high = 6.2831855f, low = -1.7484556e-7f;  // 2 pi in two parts
  const float x = __fmaf_rn(a.rest, high, __fmul_rn(a.rest, low)), y = __fmul_rn(x, x);
  float s = __fmaf_rn(y, 1.0f / 362880, -1.0f / 5040), c = __fmaf_rn(y, 1.0f / 40320, -1.0f / 720);
  s = __fmaf_rn(s, y, 1.0f / 120);
  c = __fmaf_rn(c, y, 1.0f / 24);
  s = __fmaf_rn(s, y, -1.0f / 6);
  c = __fmaf_rn(c, y, -0.5f);
  s = __fmaf_rn(__fmul_rn(s, y), x, x);
  c = __fmaf_rn(c, y, 1.0f);
  const bool odd = a.quarter & 1;
  const float u = odd ? s : c, v = odd ? c : s;
  return make_float2((a.quarter + 1) & 2 ? -u : u, a.quarter & 2 ? -v : v);
}

// A thread has a column and every so many tokens.  32640 tokens of three axes and 64 columns: 6.8 us for 17 MB
// written, of which 2 are the launch; bound by instructions (87 an angle) and the latency of positions and
// frequencies.  With CUDA's sincospif, 64-bit counters and every CTA's fp64 behind the loads it was 10.3.
template <class P>
__global__ void __launch_bounds__(kTableThreads) table_kernel(const __grid_constant__ TableArgs a) {
  using F = Turns<typename std::conditional<std::is_same<P, float>::value, float, int64_t>::type>;
  __shared__ F turns[kTablePairs];
  after_previous();
  let_next();
  const int rows = kTableThreads / a.R, row = threadIdx.x / a.R, j = threadIdx.x - row * a.R;
  int axis = 0;
  while (axis < a.axes - 1 && j >= a.end[axis]) ++axis;
  const P* positions = (const P*)a.positions + (int64_t)axis * a.tokens;
  const uint32_t step = gridDim.x * rows, first = blockIdx.x * rows + row;
  // tokens of this thread; the next AHEAD positions are on their way, the first ones while the frequencies are made
  const int count = row < rows && first < a.tokens ? (int)(((uint32_t)a.tokens - first + step - 1) / step) : 0;
  constexpr int AHEAD = 4;
  P p[AHEAD];
  positions += first;
  auto load = [&](int i) {
#pragma unroll
    for (int k = 0; k < AHEAD; ++k)
      if (i + k < count) p[k] = positions[(int64_t)k * step];
    positions += (int64_t)AHEAD * step;
  };
  load(0);
  if ((int)threadIdx.x < a.R) turns[threadIdx.x] = F(a.freqs[threadIdx.x]);
  __syncthreads();
  if (count == 0) return;
  const F f = turns[j];
  const bool finite = !(f.flags & 2), negative = f.flags & 1;
  int64_t at = (int64_t)first * a.R + j;
  const int64_t skip = (int64_t)step * a.R;
  for (int i = 0; i < count; i += AHEAD) {
    P now[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) now[k] = p[k];
    load(i + AHEAD);
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      float2 y = cos_sin(angle_of(f, now[k]));
      if constexpr (!std::is_same<P, float>::value) {  // (of fp32 positions the products tell)
        if (!finite) y = make_float2(CUDART_NAN_F, CUDART_NAN_F);
        if (negative) y.y = -y.y;
      }
      if (i + k < count) {
        a.cos[at] = y.x;
        a.sin[at] = y.y;
      }
      at += skip;
    }
  }
}

// ---------------------------------------------------------------------------
// the rotation
// ---------------------------------------------------------------------------

constexpr int kRowThreads = 256;

// Any view, and any head: a warp has a head, an element per access.
template <class T, bool NORM>
__global__ void __launch_bounds__(kRowThreads) rope_kernel(const __grid_constant__ RopeArgs a) {
  const int lane = threadIdx.x & 31;
  const int heads = a.t[0].H + a.t[1].H;
  const int64_t rows = a.tokens * heads;
  const int64_t stride = (int64_t)gridDim.x * (kRowThreads / 32);
  after_previous();
  let_next();
  for (int64_t i = (int64_t)blockIdx.x * (kRowThreads / 32) + (threadIdx.x >> 5); i < rows; i += stride) {
    const HeadRow row(a, i, heads);
    const RopeTensor& t = a.t[row.tensor];
    const T* x = (const T*)t.x.p + row.at(t.x);
    T* out = (T*)t.out.p + row.at(t.out);
    float r = 1.0f;
    if constexpr (NORM) {
      float sum = 0.0f;
      for (int c = lane; c < a.D; c += 32) {
        const float v = to_float(x[c]);
        sum = __fmaf_rn(v, v, sum);
      }
      r = inverse_rms(lanes_sum<32>(sum), a.inv_d, a.eps);
    }
    auto value = [&](int c) {
      const float v = to_float(x[c]);
      if constexpr (!NORM) return v;
      return __fmul_rn(__fmul_rn(v, r), __fadd_rn(a.offset, to_float(((const T*)t.w)[c])));
    };
    const float* cs = a.cos + row.table * a.R;
    const float* sn = a.sin + row.table * a.R;
    for (int j = lane; j < a.R; j += 32) {
      const int c = a.interleaved ? 2 * j : j, d = a.interleaved ? c + 1 : c + a.R;
      const float2 y = turned(value(c), value(d), cs[j], a.inverse ? -sn[j] : sn[j]);
      out[c] = from_float<T>(y.x);
      out[d] = from_float<T>(y.y);
    }
    for (int c = 2 * a.R + lane; c < a.D; c += 32) {
      if constexpr (NORM)
        out[c] = from_float<T>(value(c));
      else
        out[c] = x[c];
    }
  }
}

// Heads in granules: a warp's items one after the other, the next kStages - 1 on their way.  An item is two heads of
// each team: 2.5 KB that wait in shared memory and not in registers, so that two CTAs of 8 warps share an SM.
// 32640 tokens x 64 heads of 128, bf16, norm, adjacent pairs: 164 us, 6.6 TB/s, 98 % of the time of a copy of the
// bytes.  Items of four heads 180, or 187 with three stages; two heads with three or four stages and more CTAs 191 to
// 205; loads to registers without stages 208 (at 16 warps) to 308 (at 8).
constexpr int kStages = 2;

struct RopeHeads {
  RopeArgs a;
  HeadGrid g;
};
template <class T, int TEAM, bool NORM, bool INTER, bool ALL>
__global__ void __launch_bounds__(kRowThreads, 2) rope_heads_kernel(const __grid_constant__ RopeHeads args) {
  using Stage = HeadStage<T, TEAM, INTER, 1>;
  constexpr int P = HeadLane<T>::P, TEAMS = Stage::TEAMS, HEADS = Stage::HEADS, WARPS = kRowThreads / 32;
  extern __shared__ __align__(16) unsigned char space[];
  const RopeArgs& a = args.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = lane / TEAM;
  const int which = (int)blockIdx.x >= args.g.ctas[0], cta = which ? blockIdx.x - args.g.ctas[0] : blockIdx.x;
  const RopeTensor& t = a.t[which];
  const HeadLane<T> h(a, lane % TEAM);
  const uint32_t stages = smem_addr(space) + warp * kStages * Stage::BYTES;
  after_previous();
  let_next();
  const HeadWalk start(args.g, which, (int64_t)cta * WARPS + warp, (int64_t)args.g.ctas[which] * WARPS);
  HeadWalk ahead = start;
  auto issue = [&](int s) {
    if (ahead.token < a.tokens) {
      const TokenAt at(a, (uint32_t)ahead.token);
      const uint32_t stage = stages + s * Stage::BYTES;
      Stage::copy_heads(stage, lane, h, 0, t.x.p, at.batch * t.x.batch + at.place * t.x.token, t.x.head,
                        ahead.part * HEADS * TEAMS + team, t.H);
      Stage::copy_angles(stage, lane, h, a, at.table);
      ahead.next();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  F2 w[2][P];
  if constexpr (NORM) head_weight<T>(w, h, t.w, a.offset);
  int s = 0;
  for (HeadWalk i = start; i.token < a.tokens; i.next()) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // every lane's copies are there, and every lane is done with the stage before
    issue(s == 0 ? kStages - 1 : s - 1);
    const uint32_t stage = stages + s * Stage::BYTES;
    const TokenAt at(a, (uint32_t)i.token);
    const int first = i.part * HEADS * TEAMS + team;
    T* out = (T*)t.out.p + at.batch * t.out.batch + at.place * t.out.token + first * t.out.head;
    Raw<16> raw[HEADS][2];
#pragma unroll
    for (int k = 0; k < HEADS; ++k)
#pragma unroll
      for (int j = 0; j < 2; ++j) raw[k][j] = lds16(Stage::granule(stage, lane, 0, k, j));
    LaneAngles<T, TEAM, INTER, 1> angles;
    if (a.R > 0) angles.load(stage, lane, a.inverse);
    float r[HEADS];
    if constexpr (NORM) {
      // the sums of all heads first; each lane then finds the r of one of them
      float mine = 0.0f;
#pragma unroll
      for (int k = 0; k < HEADS; ++k) {
        F2 sum = f2(0.0f, 0.0f);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          F2 x[P];
          Granule<T>::widen(raw[k][j], x);
#pragma unroll
          for (int n = 0; n < P; ++n) sum = f2_fma(x[n], x[n], sum);
        }
        const float total = lanes_sum<TEAM>(__fadd_rn(sum.x, sum.y));
        if (lane % HEADS == k) mine = total;
      }
      mine = inverse_rms(mine, a.inv_d, a.eps);
#pragma unroll
      for (int k = 0; k < HEADS; ++k) r[k] = __shfl_sync(0xFFFFFFFFu, mine, lane / HEADS * HEADS + k);
    }
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      F2 x[2][P];
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Granule<T>::widen(raw[k][j], x[j]);
        if constexpr (NORM) {
#pragma unroll
          for (int n = 0; n < P; ++n) x[j][n] = f2_mul(f2_mul(x[j][n], f2(r[k], r[k])), w[j][n]);
        }
      }
      if (a.R > 0) angles.template turn<ALL>(x, h);
      if (first + k * TEAMS < t.H) {
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (h.on[j]) st_stream<16>(out + h.column[j], Granule<T>::narrow(x[j]));
      }
      out += TEAMS * t.out.head;
    }
    s = s + 1 == kStages ? 0 : s + 1;
  }
  cp_async_wait<0>();  // no copy may outlive the CTA's shared memory
}

// Any view of up to 32 NC columns: a warp has a token's heads, kColumnHeads of them an item, kColumnAhead loaded before
// the first is computed.  For rows that granules do not fit, 64 or 128 bytes an access (8160 tokens x 64 heads of 80
// with 10 pairs, bf16: 87 us, where a copy's rate gives 25; with a head after the other, by its number: 215).
constexpr int kColumnHeads = 8, kColumnAhead = 4;

template <class T, int NC, bool NORM>
__global__ void __launch_bounds__(kRowThreads) rope_columns_kernel(const __grid_constant__ RopeHeads args) {
  constexpr int WARPS = kRowThreads / 32;
  __shared__ float rows[WARPS][kColumnAhead][32 * NC];
  const RopeArgs& a = args.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = (int)blockIdx.x >= args.g.ctas[0], cta = which ? blockIdx.x - args.g.ctas[0] : blockIdx.x;
  const RopeTensor& t = a.t[which];
  const LaneColumns<NC> columns(a, lane);
  after_previous();
  let_next();
  float w[NC];
  if constexpr (NORM) {
#pragma unroll
    for (int i = 0; i < NC; ++i)
      w[i] = lane + 32 * i < a.D ? __fadd_rn(a.offset, to_float(((const T*)t.w)[lane + 32 * i])) : 0.0f;
  }
  HeadWalk walk(args.g, which, (int64_t)cta * WARPS + warp, (int64_t)args.g.ctas[which] * WARPS);
  for (; walk.token < a.tokens; walk.next()) {
    const TokenAt at(a, (uint32_t)walk.token);
    float cs[NC], sn[NC];
    if (a.R > 0) columns.load(a, at.table, a.inverse, cs, sn);
    const int first = walk.part * args.g.together, last = min(first + args.g.together, t.H);
    const T* x = (const T*)t.x.p + at.batch * t.x.batch + at.place * t.x.token + first * t.x.head + lane;
    T* out = (T*)t.out.p + at.batch * t.out.batch + at.place * t.out.token + first * t.out.head + lane;
    for (int head = first; head < last; head += kColumnAhead) {
      T raw[kColumnAhead][NC];
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          raw[k][i] = from_float<T>(0.0f);
          if (head + k < last && lane + 32 * i < a.D) raw[k][i] = x[k * t.x.head + 32 * i];
        }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k) {
        float y[NC], r = 1.0f;
        if constexpr (NORM) {
          float sum = 0.0f;
#pragma unroll
          for (int i = 0; i < NC; ++i) sum = __fmaf_rn(to_float(raw[k][i]), to_float(raw[k][i]), sum);
          r = inverse_rms(lanes_sum<32>(sum), a.inv_d, a.eps);
        }
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          y[i] = to_float(raw[k][i]);
          if constexpr (NORM) y[i] = __fmul_rn(__fmul_rn(y[i], r), w[i]);
          rows[warp][k][lane + 32 * i] = y[i];
        }
        __syncwarp();
        if (head + k < last) {
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            if (lane + 32 * i >= a.D) continue;
            if (columns.angle[i] >= 0) y[i] = __fmaf_rn(y[i], cs[i], __fmul_rn(rows[warp][k][columns.partner[i]], sn[i]));
            out[k * t.out.head + 32 * i] = NORM || columns.angle[i] >= 0 ? from_float<T>(y[i]) : raw[k][i];
          }
        }
      }
      x += kColumnAhead * t.x.head;
      out += kColumnAhead * t.out.head;
    }
  }
}

template <class T, int TEAM, bool NORM, bool INTER>
cudaError_t launch_heads(const DeviceInfo& dev, const RopeArgs& a, cudaStream_t s) {
  using Stage = HeadStage<T, TEAM, INTER, 1>;
  const bool all = 2 * a.R == a.D;
  const auto kern = all ? rope_heads_kernel<T, TEAM, NORM, INTER, true> : rope_heads_kernel<T, TEAM, NORM, INTER, false>;
  static std::atomic<int> opted[2][kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted[all]);
  if (e != cudaSuccess) return e;
  constexpr int warps = kRowThreads / 32;
  const size_t smem = (size_t)warps * kStages * Stage::BYTES;
  const int64_t most = (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kRowThreads, smem);
  const RopeHeads h{a, head_grid(a, Stage::HEADS * Stage::TEAMS, warps, most)};
  return launch_after(kern, (unsigned)(h.g.ctas[0] + h.g.ctas[1]), kRowThreads, smem, s, h);
}
template <class T, int TEAM>
cudaError_t launch_heads(const DeviceInfo& dev, const RopeArgs& a, cudaStream_t s) {
  const bool norm = a.t[0].w || a.t[1].w;
  return a.interleaved ? (norm ? launch_heads<T, TEAM, true, true>(dev, a, s) : launch_heads<T, TEAM, false, true>(dev, a, s))
                       : (norm ? launch_heads<T, TEAM, true, false>(dev, a, s) : launch_heads<T, TEAM, false, false>(dev, a, s));
}

template <class T>
cudaError_t launch(const DeviceInfo& dev, const RopeArgs& a, cudaStream_t s) {
  if (head_granules<T>(a)) {
    const int units = head_units(a, HeadLane<T>::PER);
    return units <= 4    ? launch_heads<T, 4>(dev, a, s)
           : units <= 8  ? launch_heads<T, 8>(dev, a, s)
           : units <= 16 ? launch_heads<T, 16>(dev, a, s)
                         : launch_heads<T, 32>(dev, a, s);
  }
  const bool norm = a.t[0].w || a.t[1].w;
  if (a.D <= 256) {
    const auto columns = a.D <= 64    ? (norm ? rope_columns_kernel<T, 2, true> : rope_columns_kernel<T, 2, false>)
                         : a.D <= 128 ? (norm ? rope_columns_kernel<T, 4, true> : rope_columns_kernel<T, 4, false>)
                                      : (norm ? rope_columns_kernel<T, 8, true> : rope_columns_kernel<T, 8, false>);
    const int64_t most = (int64_t)dev.sm_count * resident_ctas(dev, (const void*)columns, kRowThreads);
    const int together = column_heads(dev, a, kColumnHeads, kColumnAhead);
    const RopeHeads h{a, head_grid(a, together, kRowThreads / 32, most)};
    return launch_after(columns, (unsigned)(h.g.ctas[0] + h.g.ctas[1]), kRowThreads, 0, s, h);
  }
  const int64_t rows = a.tokens * (a.t[0].H + a.t[1].H);
  const auto kern = norm ? rope_kernel<T, true> : rope_kernel<T, false>;
  const int64_t warps = kRowThreads / 32;
  const int64_t most = (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kRowThreads) * 8;
  return launch_after(kern, (unsigned)std::min(most, (rows + warps - 1) / warps), kRowThreads, 0, s, a);
}

}  // namespace

cudaError_t launch_table(const DeviceInfo& dev, int position_type, const TableArgs& a,
                         cudaStream_t s) {
  static_assert(kTablePairs <= kTableThreads, "a frequency a thread");
  const int64_t rows = kTableThreads / a.R;
  // (no more CTAs than are resident at once: each makes the frequencies anew)
  const unsigned grid = (unsigned)std::min((int64_t)dev.sm_count * 2, (a.tokens + rows - 1) / rows);
  return position_type == DIT_POS_INT32   ? launch_after(table_kernel<int32_t>, grid, kTableThreads, 0, s, a)
         : position_type == DIT_POS_INT64 ? launch_after(table_kernel<int64_t>, grid, kTableThreads, 0, s, a)
                                          : launch_after(table_kernel<float>, grid, kTableThreads, 0, s, a);
}

cudaError_t launch_rope(const DeviceInfo& dev, int dtype, const RopeArgs& a, cudaStream_t s) {
  return dtype == 0   ? launch<__nv_bfloat16>(dev, a, s)
         : dtype == 1 ? launch<__half>(dev, a, s)
                      : launch<float>(dev, a, s);
}

}  // namespace dit
