// k_attend.cu -- attention of one new token per sequence over a paged cache
// (sm_103a): any head size, alignment and type, in fp32.
//
//   s = scale q.k,  m = max s,  l = sum 2^(s - m),  o = sum 2^(s - m) v
// in one pass over the tokens, with s in powers of two (scale times log2 e).  For rows
// that are not made of 16-byte granules, or of more than 256 columns: bound by the shuffles
// of its dot products (one sequence of 131072 tokens x 8 heads of 128, bf16: 3.1 ms).
#include "dit_attend.cuh"

namespace dit {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 64;  // at a time
constexpr int kMaxD = 512;
constexpr int kExtra = 4, kLeast = 8;  // units of a segment beside its tiles; the smallest part

template <class K>
__device__ __forceinline__ float cached(const void* p, int64_t i) {
  if constexpr (sizeof(K) == 1)
    return from_e4m3(((const uint8_t*)p)[i]);
  else
    return to_float(((const K*)p)[i]);
}

// K: the cache's type (uint8_t: E4M3), T: the queries'.
template <class T, class K>
__global__ void __launch_bounds__(kThreads) attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr bool FP8 = sizeof(K) == 1;
  __shared__ Plan<kThreads> plan;
  __shared__ int64_t place[kTokens];
  __shared__ float kscale[kTokens], vscale[kTokens];
  __shared__ float weight[kAttendRows][kTokens];
  __shared__ float m[kAttendRows], l[kAttendRows], factor[kAttendRows];
  extern __shared__ float space[];
  const int D = (int)a.c.D;
  float* q = space;                    // [rows][D]
  float* o = space + kAttendRows * D;  // [rows][D]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int blocks = (a.group + kAttendRows - 1) / kAttendRows;
  const Line line{(int)a.c.heads * blocks, kExtra};
  after_previous();
  const int64_t total = line.total(a, plan);
  const int64_t per = max((int64_t)kLeast, (total + gridDim.x - 1) / gridDim.x);
  const int64_t begin = min(blockIdx.x * per, total), end = min(begin + per, total);
  if (tid < 2) a.owner[2 * blockIdx.x + tid] = -1;
  let_next();
  if (begin >= end) return;
  const int slot_rows = min(a.group, kAttendRows);
  Walk walk(a, line, begin, end, line.find(a, begin, plan));
  Segment g;
  while (walk.next(a, line, g)) {
    const int head = g.s / blocks, row0 = (g.s - head * blocks) * kAttendRows;
    const int rows = min(kAttendRows, a.group - row0);
    const int h0 = head * a.group + row0;
    __syncthreads();
    for (int i = tid; i < rows * D; i += kThreads) {
      const int r = i / D, c = i - r * D;
      q[i] = __fmul_rn(to_float(((const T*)a.q.p)[g.b * a.q.token + (h0 + r) * a.q.head + c]),
                       a.scale);
      o[i] = 0.0f;
    }
    if (tid < kAttendRows) m[tid] = -INFINITY, l[tid] = 0.0f;
    for (int t0 = g.first * kTile; t0 < g.last * kTile; t0 += kTokens) {
      const int n = min(kTokens, g.last * kTile - t0);
      __syncthreads();
      if (tid < kTokens) {
        const Place p = tid < n ? place_of(a, g.b, head, t0 + tid, g.lo, g.hi) : Place{-1, -1};
        place[tid] = p.element;
        if constexpr (FP8) {
          kscale[tid] = p.element >= 0 ? a.c.k_scales[p.scale] : 0.0f;
          vscale[tid] = p.element >= 0 ? a.c.v_scales[p.scale] : 0.0f;
        }
      }
      __syncthreads();
      for (int t = warp; t < kTokens; t += kWarps) {
        if (place[t] < 0) {
          if (lane < rows) weight[lane][t] = -INFINITY;
          continue;
        }
        float k[kMaxD / 32];
#pragma unroll
        for (int i = 0; i < kMaxD / 32; ++i)
          if (lane + 32 * i < D) k[i] = cached<K>(a.c.k, place[t] + lane + 32 * i);
        for (int r = 0; r < rows; ++r) {
          float s = 0.0f;
#pragma unroll
          for (int i = 0; i < kMaxD / 32; ++i)
            if (lane + 32 * i < D) s = __fmaf_rn(q[r * D + lane + 32 * i], k[i], s);
          s = lanes_sum<32>(s);
          if constexpr (FP8) s = __fmul_rn(s, kscale[t]);
          if (lane == 0) weight[r][t] = __fmul_rn(s, 1.4426950408889634f);
        }
      }
      __syncthreads();
      for (int r = warp; r < rows; r += kWarps) {
        const float s0 = weight[r][lane], s1 = weight[r][lane + 32];
        float most = fmaxf(s0, s1);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, k));
        const float was = m[r], now = fmaxf(was, most);
        const float base = now == -INFINITY ? 0.0f : now;
        const float p0 = exp2f(__fadd_rn(s0, -base)), p1 = exp2f(__fadd_rn(s1, -base));
        const float f = exp2f(__fadd_rn(was, -base));
        const float sum = lanes_sum<32>(__fadd_rn(p0, p1));
        weight[r][lane] = p0;
        weight[r][lane + 32] = p1;
        __syncwarp();
        if (lane == 0) {
          m[r] = now;
          factor[r] = f;
          l[r] = __fmaf_rn(l[r], f, sum);
        }
      }
      __syncthreads();
      for (int c = tid; c < D; c += kThreads) {
        float acc[kAttendRows];
#pragma unroll
        for (int r = 0; r < kAttendRows; ++r) acc[r] = r < rows ? __fmul_rn(o[r * D + c], factor[r]) : 0.0f;
        for (int t = 0; t < n; ++t) {
          if (place[t] < 0) continue;
          float v = cached<K>(a.c.v, place[t] + c);
          if constexpr (FP8) v = __fmul_rn(v, vscale[t]);
#pragma unroll
          for (int r = 0; r < kAttendRows; ++r)
            if (r < rows) acc[r] = __fmaf_rn(weight[r][t], v, acc[r]);
        }
#pragma unroll
        for (int r = 0; r < kAttendRows; ++r)
          if (r < rows) o[r * D + c] = acc[r];
      }
    }
    __syncthreads();
    if (g.head || g.tail) {
      const int slot = g.head ? 0 : 1;
      float* out = a.partial + ((int64_t)blockIdx.x * 2 + slot) * slot_rows * (D + 2);
      if (tid == 0) a.owner[2 * blockIdx.x + slot] = segment_id(g.b, g.s);
      for (int i = tid; i < rows * D; i += kThreads) out[2 * slot_rows + i] = o[i];
      if (tid < rows) {
        out[tid] = m[tid];
        out[slot_rows + tid] = l[tid];
      }
    } else {
      for (int i = tid; i < rows * D; i += kThreads) {
        const int r = i / D, c = i - r * D;
        const float total = l[r];
        ((T*)a.out.p)[g.b * a.out.token + (h0 + r) * a.out.head + c] =
            from_float<T>(total == 0.0f ? 0.0f : __fdiv_rn(o[i], total));
      }
      if (a.lse && tid < rows) a.lse[(int64_t)g.b * a.Hq + h0 + tid] = lse_of(m[tid], l[tid]);
    }
  }
}

// The join of the segments that begin in CTA blockIdx.x and end in a later one: row blockIdx.y of it.  A warp has
// every kJoinWarps-th of the parts, columns lane, lane + 32, ..., each part scaled to the largest maximum so far.  What
// a part holds is loaded beside its owner's name, before that is known to be this segment's.
constexpr int kJoinWarps = 8;
struct JoinArgs {
  AttendArgs a;
  int ctas;
};
template <class T, int DP>
__global__ void __launch_bounds__(32 * kJoinWarps) join_kernel(const __grid_constant__ JoinArgs j) {
  constexpr int N = DP / 32;
  __shared__ float most[kJoinWarps], sums[kJoinWarps], columns[kJoinWarps][DP];
  const AttendArgs& a = j.a;
  const int D = (int)a.c.D, lane = threadIdx.x & 31, warp = threadIdx.x >> 5, r = blockIdx.y, cta = blockIdx.x;
  const int slot_rows = min(a.group, a.rows);
  const int64_t size = (int64_t)slot_rows * (D + 2);
  after_previous();
  let_next();
  const int64_t id = a.owner[2 * cta + 1];
  if (id < 0) return;
  const int blocks = (a.group + a.rows - 1) / a.rows;
  const int b = (int)(id >> 32), s = (int)(uint32_t)id;
  const int head = s / blocks, row0 = (s - head * blocks) * a.rows;
  if (r >= min(a.rows, a.group - row0)) return;
  float m = -INFINITY, l = 0.0f, o[N] = {};
  // (the parts of a segment are those of CTAs one after the other: the first is the second part of its CTA)
#pragma unroll 2
  for (int k = warp;; k += kJoinWarps) {
    const int at = min(cta + k, j.ctas - 1);
    const float* p = a.partial + (2 * (int64_t)at + (k == 0)) * size;
    const int64_t owner = a.owner[2 * at + (k == 0)];
    const float pm = p[r], pl = p[slot_rows + r];
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = 32 * i + lane < D ? p[2 * slot_rows + r * D + 32 * i + lane] : 0.0f;
    if (cta + k >= j.ctas || owner != id) break;
    const float now = fmaxf(m, pm), base = now == -INFINITY ? 0.0f : now;
    const float f = exp2f(__fadd_rn(m, -base)), g = exp2f(__fadd_rn(pm, -base));
    m = now;
    l = __fmaf_rn(l, f, __fmul_rn(pl, g));
#pragma unroll
    for (int i = 0; i < N; ++i) o[i] = __fmaf_rn(o[i], f, __fmul_rn(v[i], g));
  }
  if (lane == 0) most[warp] = m, sums[warp] = l;
#pragma unroll
  for (int i = 0; i < N; ++i) columns[warp][32 * i + lane] = o[i];
  __syncthreads();
  float top = -INFINITY, by[kJoinWarps], total = 0.0f;
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) top = fmaxf(top, most[w]);
#pragma unroll
  for (int w = 0; w < kJoinWarps; ++w) {
    by[w] = exp2f(__fadd_rn(most[w], -(top == -INFINITY ? 0.0f : top)));
    total = __fmaf_rn(sums[w], by[w], total);
  }
  const int h = head * a.group + row0 + r;
  for (int c = threadIdx.x; c < D; c += 32 * kJoinWarps) {
    float y = 0.0f;
#pragma unroll
    for (int w = 0; w < kJoinWarps; ++w) y = __fmaf_rn(columns[w][c], by[w], y);
    ((T*)a.out.p)[b * a.out.token + h * a.out.head + c] = from_float<T>(total == 0.0f ? 0.0f : __fdiv_rn(y, total));
  }
  if (threadIdx.x == 0 && a.lse) a.lse[(int64_t)b * a.Hq + h] = lse_of(top, total);
}

template <class T, class K>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  const auto kern = attend_kernel<T, K>;
  const size_t smem = (size_t)2 * kAttendRows * a.c.D * 4;
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  *ctas = std::min(kAttendMaxCtas,
                   (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kThreads, smem));
  return launch_after(kern, (unsigned)*ctas, kThreads, smem, s, a);
}

template <class T>
cudaError_t launch(const DeviceInfo& dev, int dtype, bool mma, AttendArgs a, cudaStream_t s) {
  int64_t ctas = 0;
  a.rows = kAttendRows;
  const cudaError_t e = mma                        ? launch_attend_mma(dev, dtype, a, &ctas, s)
                        : a.c.format == DIT_E4M3 ? launch<T, uint8_t>(dev, a, &ctas, s)
                                                 : launch<T, T>(dev, a, &ctas, s);
  if (e != cudaSuccess) return e;
  const JoinArgs j{a, (int)ctas};
  const auto join = a.c.D <= 128 ? join_kernel<T, 128> : a.c.D <= 256 ? join_kernel<T, 256> : join_kernel<T, kMaxD>;
  return launch_after(join, dim3((unsigned)ctas, (unsigned)std::min(a.group, a.rows)), 32 * kJoinWarps, 0, s, j);
}

}  // namespace

cudaError_t launch_attend(const DeviceInfo& dev, int dtype, bool granules, const AttendArgs& a,
                          cudaStream_t s) {
  const bool mma = attend_mma_takes(granules, a);
  return dtype == 0   ? launch<__nv_bfloat16>(dev, dtype, mma, a, s)
         : dtype == 1 ? launch<__half>(dev, dtype, mma, a, s)
                      : launch<float>(dev, dtype, mma, a, s);
}

}  // namespace dit
