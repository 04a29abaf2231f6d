// k_rope_grad.cu -- the gradient of a head's norm and rotation (sm_103a).
//
//   u = the gradient of the output turned back,  n = x r,  t = u (offset + w)
//   grad_x = r (t - n mean(t n)),   grad_w = sum over tokens and heads of u n
#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// Any view, and any head: a warp has a head, an element per access; blockIdx.y tells queries from keys.  Each warp
// adds up its weight's gradient in shared memory (its own row of it), the CTA its warps'.
template <class T>
__global__ void __launch_bounds__(kRowThreads) rope_grad_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float sums[];  // [warps][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* mine = sums + (size_t)warp * a.D;
  if (a.partial) {
    for (int c = lane; c < a.D; c += 32) mine[c] = 0.0f;
    __syncwarp();
  }
  const RopeTensor& t = a.t[blockIdx.y > 0 || a.t[0].H == 0];
  const int64_t rows = a.tokens * t.H;
  const int64_t stride = (int64_t)gridDim.x * kRowWarps;
  after_previous();
  let_next();
  for (int64_t i = (int64_t)blockIdx.x * kRowWarps + warp; i < rows; i += stride) {
    const int64_t token = i / t.H, head = i - token * t.H;
    const TokenAt place(a, (uint32_t)token);
    auto at = [&](const dit_heads& v) { return place.batch * v.batch + place.place * v.token + head * v.head; };
    const T* x = (const T*)t.x.p + at(t.x);
    const T* g = (const T*)t.g.p + at(t.g);
    T* out = (T*)t.out.p + at(t.out);
    const T* w = (const T*)t.w;
    const float* cs = a.cos + place.table * a.R;
    const float* sn = a.sin + place.table * a.R;
    // columns come in pairs (c, d); those that are not turned come alone
    auto columns = [&](auto&& body) {
      for (int j = lane; j < a.R; j += 32) {
        const int c = a.interleaved ? 2 * j : j, d = a.interleaved ? c + 1 : c + a.R;
        const float2 u = turned(to_float(g[c]), to_float(g[d]), cs[j], -sn[j]);
        body(c, u.x, d, u.y);
      }
      for (int c = 2 * a.R + lane; c < a.D; c += 32) body(c, to_float(g[c]), -1, 0.0f);
    };
    auto weighted = [&](int c, float u) { return __fmul_rn(u, __fadd_rn(a.offset, to_float(w[c]))); };
    float sum = 0.0f, dot = 0.0f;
    columns([&](int c, float u, int d, float v) {
      const float p = to_float(x[c]);
      sum = __fmaf_rn(p, p, sum);
      dot = __fmaf_rn(weighted(c, u), p, dot);
      if (d < 0) return;
      const float q = to_float(x[d]);
      sum = __fmaf_rn(q, q, sum);
      dot = __fmaf_rn(weighted(d, v), q, dot);
    });
    const float r = inverse_rms(lanes_sum<32>(sum), a.inv_d, a.eps);
    // mean(t n), n = x r
    const float mean = __fmul_rn(__fmul_rn(lanes_sum<32>(dot), r), a.inv_d);
    columns([&](int c, float u, int d, float v) {
      auto one = [&](int k, float grad) {
        const float n = __fmul_rn(to_float(x[k]), r);
        const float y = __fmul_rn(r, __fadd_rn(weighted(k, grad), -__fmul_rn(n, mean)));
        if (a.partial) mine[k] = __fmaf_rn(grad, n, mine[k]);
        return from_float<T>(y);
      };
      const T first = one(c, u);
      if (d >= 0) {
        const T second = one(d, v);
        out[d] = second;
      }
      out[c] = first;
    });
  }
  if (!a.partial) return;
  __syncthreads();
  float* partial = a.partial + ((int64_t)blockIdx.y * gridDim.x + blockIdx.x) * a.D;
  for (int c = threadIdx.x; c < a.D; c += kRowThreads) {
    float v = 0.0f;
    for (int k = 0; k < kRowWarps; ++k) v = __fadd_rn(v, sums[(size_t)k * a.D + c]);
    partial[c] = v;
  }
}

// Heads in granules: a warp's items one after the other, the next kStages - 1 on their way.  A CTA has heads of the
// queries or of the keys alone, so that a lane adds up its columns' part of one weight's gradient in registers.
// Bound by memory: each gradient and input read once, each result written once, and a row of D sums a CTA.  8160
// tokens x 40 heads of 128, bf16: 42 us with the join, 6.0 TB/s, 88 % of a copy's rate (three stages 42.6; angles
// copied by every team 52; loads to registers without stages 72.6).
constexpr int kStages = 2;

struct GradHeads {
  RopeArgs a;
  HeadGrid g;
};
template <class T, int TEAM, bool INTER, bool ALL>
__global__ void __launch_bounds__(kRowThreads, 2) rope_grad_heads_kernel(const __grid_constant__ GradHeads args) {
  using Stage = HeadStage<T, TEAM, INTER, 2>;
  constexpr int P = HeadLane<T>::P, TEAMS = Stage::TEAMS, HEADS = Stage::HEADS;
  extern __shared__ __align__(16) unsigned char space[];
  const RopeArgs& a = args.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, team = lane / TEAM;
  const int which = (int)blockIdx.x >= args.g.ctas[0], cta = which ? blockIdx.x - args.g.ctas[0] : blockIdx.x;
  const RopeTensor& t = a.t[which];
  const HeadLane<T> h(a, lane % TEAM);
  const uint32_t stages = smem_addr(space) + warp * kStages * Stage::BYTES;
  after_previous();
  let_next();
  const HeadWalk start(args.g, which, (int64_t)cta * kRowWarps + warp, (int64_t)args.g.ctas[which] * kRowWarps);
  HeadWalk ahead = start;
  auto issue = [&](int s) {
    if (ahead.token < a.tokens) {
      const TokenAt at(a, (uint32_t)ahead.token);
      const uint32_t stage = stages + s * Stage::BYTES;
      const int first = ahead.part * HEADS * TEAMS + team;
      Stage::copy_heads(stage, lane, h, 0, t.x.p, at.batch * t.x.batch + at.place * t.x.token, t.x.head, first, t.H);
      Stage::copy_heads(stage, lane, h, 1, t.g.p, at.batch * t.g.batch + at.place * t.g.token, t.g.head, first, t.H);
      Stage::copy_angles(stage, lane, h, a, at.table);
      ahead.next();
    }
    cp_async_commit();
  };
#pragma unroll
  for (int s = 0; s < kStages - 1; ++s) issue(s);
  F2 w[2][P], acc[2][P];
  head_weight<T>(w, h, t.w, a.offset);
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) acc[j][i] = f2(0.0f, 0.0f);
  int s = 0;
  for (HeadWalk i = start; i.token < a.tokens; i.next()) {
    cp_async_wait<kStages - 2>();
    __syncwarp();  // every lane's copies are there, and every lane is done with the stage before
    issue(s == 0 ? kStages - 1 : s - 1);
    const uint32_t stage = stages + s * Stage::BYTES;
    const TokenAt at(a, (uint32_t)i.token);
    const int first = i.part * HEADS * TEAMS + team;
    T* out = (T*)t.out.p + at.batch * t.out.batch + at.place * t.out.token + first * t.out.head;
    LaneAngles<T, TEAM, INTER, 2> angles;
    if (a.R > 0) angles.load(stage, lane, true);  // the gradient is turned back
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      // (a head that is not there holds zeros, and adds none)
      F2 x[2][P], u[2][P];
      F2 square = f2(0.0f, 0.0f), dot = f2(0.0f, 0.0f);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Granule<T>::widen(lds16(Stage::granule(stage, lane, 0, k, j)), x[j]);
        Granule<T>::widen(lds16(Stage::granule(stage, lane, 1, k, j)), u[j]);
      }
      if (a.R > 0) angles.template turn<ALL>(u, h);
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int n = 0; n < P; ++n) {
          square = f2_fma(x[j][n], x[j][n], square);
          dot = f2_fma(f2_mul(u[j][n], w[j][n]), x[j][n], dot);
        }
      const float r = inverse_rms(lanes_sum<TEAM>(__fadd_rn(square.x, square.y)), a.inv_d, a.eps);
      const float mean = __fmul_rn(__fmul_rn(lanes_sum<TEAM>(__fadd_rn(dot.x, dot.y)), r), a.inv_d);
      const bool on = first + k * TEAMS < t.H;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        F2 y[P];
#pragma unroll
        for (int n = 0; n < P; ++n) {
          const F2 v = f2_mul(x[j][n], f2(r, r));
          if (on) acc[j][n] = f2_fma(u[j][n], v, acc[j][n]);
          y[n] = f2_mul(f2_fma(v, f2(-mean, -mean), f2_mul(u[j][n], w[j][n])), f2(r, r));
        }
        if (on && h.on[j]) st_stream<16>(out + h.column[j], Granule<T>::narrow(y));
      }
      out += TEAMS * t.out.head;
    }
    s = s + 1 == kStages ? 0 : s + 1;
  }
  cp_async_wait<0>();
  if (!a.partial) return;
  __syncthreads();  // the stages become the warps' sums, [warps][D]
  float* sums = (float*)space;
  // the warp's teams, then the CTA's warps, in order
#pragma unroll
  for (int j = 0; j < 2; ++j)
#pragma unroll
    for (int i = 0; i < P; ++i) {
#pragma unroll
      for (int o = TEAM; o < 32; o <<= 1) {
        acc[j][i].x = __fadd_rn(acc[j][i].x, __shfl_xor_sync(0xFFFFFFFFu, acc[j][i].x, o));
        acc[j][i].y = __fadd_rn(acc[j][i].y, __shfl_xor_sync(0xFFFFFFFFu, acc[j][i].y, o));
      }
      if (team == 0 && h.on[j]) *(float2*)(sums + warp * a.D + h.column[j] + 2 * i) = acc[j][i];
    }
  __syncthreads();
  float* out = a.partial + (int64_t)blockIdx.x * a.D;
  for (int c = threadIdx.x; c < a.D; c += kRowThreads) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) v = __fadd_rn(v, sums[k * a.D + c]);
    out[c] = v;
  }
}

// Any view of up to 32 NC columns: a warp has a token's heads, kColumnHeads of them an item, two loaded before the first
// is computed; a lane adds up its columns' part of one weight's gradient (8160 tokens x 40 heads of 99, bf16: 114
// us, where a copy's rate gives 29; with a head after the other, by its number: 283).
constexpr int kColumnHeads = 8, kColumnAhead = 2;

template <class T, int NC>
__global__ void __launch_bounds__(kRowThreads) rope_grad_columns_kernel(const __grid_constant__ GradHeads args) {
  __shared__ float rows[kRowWarps][kColumnAhead][32 * NC];
  const RopeArgs& a = args.a;
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int which = (int)blockIdx.x >= args.g.ctas[0], cta = which ? blockIdx.x - args.g.ctas[0] : blockIdx.x;
  const RopeTensor& t = a.t[which];
  const LaneColumns<NC> columns(a, lane);
  after_previous();
  let_next();
  float w[NC], acc[NC];
#pragma unroll
  for (int i = 0; i < NC; ++i) {
    w[i] = lane + 32 * i < a.D ? __fadd_rn(a.offset, to_float(((const T*)t.w)[lane + 32 * i])) : 0.0f;
    acc[i] = 0.0f;
  }
  HeadWalk walk(args.g, which, (int64_t)cta * kRowWarps + warp, (int64_t)args.g.ctas[which] * kRowWarps);
  for (; walk.token < a.tokens; walk.next()) {
    const TokenAt at(a, (uint32_t)walk.token);
    float cs[NC], sn[NC];
    if (a.R > 0) columns.load(a, at.table, true, cs, sn);  // the gradient is turned back
    const int first = walk.part * args.g.together, last = min(first + args.g.together, t.H);
    const T* x = (const T*)t.x.p + at.batch * t.x.batch + at.place * t.x.token + first * t.x.head + lane;
    const T* g = (const T*)t.g.p + at.batch * t.g.batch + at.place * t.g.token + first * t.g.head + lane;
    T* out = (T*)t.out.p + at.batch * t.out.batch + at.place * t.out.token + first * t.out.head + lane;
    for (int head = first; head < last; head += kColumnAhead) {
      T rx[kColumnAhead][NC], rg[kColumnAhead][NC];
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k)
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          rx[k][i] = rg[k][i] = from_float<T>(0.0f);
          if (head + k >= last || lane + 32 * i >= a.D) continue;
          rx[k][i] = x[k * t.x.head + 32 * i];
          rg[k][i] = g[k * t.g.head + 32 * i];
        }
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k)
#pragma unroll
        for (int i = 0; i < NC; ++i) rows[warp][k][lane + 32 * i] = to_float(rg[k][i]);
      __syncwarp();
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k) {
        float u[NC], square = 0.0f, dot = 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          u[i] = to_float(rg[k][i]);
          if (columns.angle[i] >= 0) u[i] = __fmaf_rn(u[i], cs[i], __fmul_rn(rows[warp][k][columns.partner[i]], sn[i]));
          const float v = to_float(rx[k][i]);
          square = __fmaf_rn(v, v, square);
          dot = __fmaf_rn(__fmul_rn(u[i], w[i]), v, dot);
        }
        const float r = inverse_rms(lanes_sum<32>(square), a.inv_d, a.eps);
        const float mean = __fmul_rn(__fmul_rn(lanes_sum<32>(dot), r), a.inv_d);
        if (head + k >= last) continue;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          if (lane + 32 * i >= a.D) continue;
          const float n = __fmul_rn(to_float(rx[k][i]), r);
          acc[i] = __fmaf_rn(u[i], n, acc[i]);
          out[k * t.out.head + 32 * i] = from_float<T>(__fmul_rn(r, __fmaf_rn(n, -mean, __fmul_rn(u[i], w[i]))));
        }
      }
      x += kColumnAhead * t.x.head;
      g += kColumnAhead * t.g.head;
      out += kColumnAhead * t.out.head;
    }
  }
  if (!a.partial) return;
  __syncthreads();
  float* sums = &rows[0][0][0];  // [warps][32 NC]
#pragma unroll
  for (int i = 0; i < NC; ++i) sums[warp * 32 * NC + lane + 32 * i] = acc[i];
  __syncthreads();
  float* partial = a.partial + (int64_t)blockIdx.x * a.D;
  for (int c = threadIdx.x; c < a.D; c += kRowThreads) {
    float v = 0.0f;
#pragma unroll
    for (int k = 0; k < kRowWarps; ++k) v = __fadd_rn(v, sums[k * 32 * NC + c]);
    partial[c] = v;
  }
}

// gw[which][c] = the sum over the partial rows [0, split) (queries) or [split, rows) (keys): 32 columns
// a CTA, its 32 warps every 32nd row, then their sums in order.
struct JoinArgs {
  const float* partial;
  int split, rows, D;
  void* gw[2];
};
template <class T>
__global__ void __launch_bounds__(1024) join_kernel(const __grid_constant__ JoinArgs a) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, which = blockIdx.y;
  T* gw = (T*)a.gw[which];
  after_previous();
  let_next();
  if (!gw) return;
  const int c = blockIdx.x * 32 + lane;
  const int end = which ? a.rows : a.split;
  float v = 0.0f;
  if (c < a.D) {
#pragma unroll 8
    for (int i = (which ? a.split : 0) + warp; i < end; i += 32) v = __fadd_rn(v, a.partial[(int64_t)i * a.D + c]);
  }
  part[warp][lane] = v;
  __syncthreads();
  v = lanes_sum<32>(part[lane][warp]);
  const int k = blockIdx.x * 32 + warp;
  if (lane == 0 && k < a.D) gw[k] = from_float<T>(v);
}

// split, rows: the partial rows written
template <class T, int TEAM, bool INTER>
cudaError_t launch_heads(const DeviceInfo& dev, const RopeArgs& a, int* split, int* rows, cudaStream_t s) {
  using Stage = HeadStage<T, TEAM, INTER, 2>;
  const bool all = 2 * a.R == a.D;
  const auto kern = all ? rope_grad_heads_kernel<T, TEAM, INTER, true> : rope_grad_heads_kernel<T, TEAM, INTER, false>;
  static std::atomic<int> opted[2][kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted[all]);
  if (e != cudaSuccess) return e;
  static_assert(Stage::BYTES * kStages >= 32 / Stage::TEAMS * 2 * 16 / (int)sizeof(T) * 4, "room for a warp's sums");
  const size_t smem = (size_t)kRowWarps * kStages * Stage::BYTES;
  const int64_t most = std::min(2 * kRopeGradMaxCtas, (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kRowThreads, smem));
  const GradHeads g{a, head_grid(a, Stage::HEADS * Stage::TEAMS, kRowWarps, most)};
  *split = g.g.ctas[0];
  *rows = g.g.ctas[0] + g.g.ctas[1];
  return launch_after(kern, (unsigned)*rows, kRowThreads, smem, s, g);
}
template <class T, int TEAM>
cudaError_t launch_heads(const DeviceInfo& dev, const RopeArgs& a, int* split, int* rows, cudaStream_t s) {
  return a.interleaved ? launch_heads<T, TEAM, true>(dev, a, split, rows, s)
                       : launch_heads<T, TEAM, false>(dev, a, split, rows, s);
}

template <class T>
cudaError_t launch(const DeviceInfo& dev, const RopeArgs& a, void* gwq, void* gwk, cudaStream_t s) {
  int split = 0, rows = 0;
  cudaError_t e;
  if (head_granules<T>(a)) {
    const int units = head_units(a, HeadLane<T>::PER);
    e = units <= 4    ? launch_heads<T, 4>(dev, a, &split, &rows, s)
        : units <= 8  ? launch_heads<T, 8>(dev, a, &split, &rows, s)
        : units <= 16 ? launch_heads<T, 16>(dev, a, &split, &rows, s)
                      : launch_heads<T, 32>(dev, a, &split, &rows, s);
  } else if (a.D <= 256) {
    const auto columns = a.D <= 64 ? rope_grad_columns_kernel<T, 2> : a.D <= 128 ? rope_grad_columns_kernel<T, 4> : rope_grad_columns_kernel<T, 8>;
    const int64_t most = std::min(2 * kRopeGradMaxCtas, (int64_t)dev.sm_count * resident_ctas(dev, (const void*)columns, kRowThreads));
    const int together = column_heads(dev, a, kColumnHeads, kColumnAhead);
    const GradHeads g{a, head_grid(a, together, kRowWarps, most)};
    split = g.g.ctas[0];
    rows = g.g.ctas[0] + g.g.ctas[1];
    e = launch_after(columns, (unsigned)rows, kRowThreads, 0, s, g);
  } else {
    const auto kern = rope_grad_kernel<T>;
    const size_t smem = a.partial ? (size_t)kRowWarps * a.D * 4 : 0;
    const int64_t most = std::min(kRopeGradMaxCtas, (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kRowThreads, smem));
    const int64_t heads = std::max(a.t[0].H, a.t[1].H);
    const unsigned grid = (unsigned)std::min(most, (a.tokens * heads + kRowWarps - 1) / kRowWarps);
    split = a.t[0].H ? (int)grid : 0;
    rows = split + (a.t[1].H ? (int)grid : 0);
    e = launch_after(kern, dim3(grid, (a.t[0].H > 0) + (a.t[1].H > 0)), kRowThreads, smem, s, a);
  }
  if (e != cudaSuccess || !a.partial) return e;
  return launch_after(join_kernel<T>, dim3((unsigned)((a.D + 31) / 32), 2), 1024, 0, s,
                      JoinArgs{a.partial, split, rows, a.D, {gwq, gwk}});
}

}  // namespace

cudaError_t launch_rope_grad(const DeviceInfo& dev, int dtype, const RopeArgs& a, void* gwq,
                             void* gwk, cudaStream_t s) {
  return dtype == 0   ? launch<__nv_bfloat16>(dev, a, gwq, gwk, s)
         : dtype == 1 ? launch<__half>(dev, a, gwq, gwk, s)
                      : launch<float>(dev, a, gwq, gwk, s);
}

}  // namespace dit
