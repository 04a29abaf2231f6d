// k_attend.cu -- attention of one new token per sequence over a paged cache
// (sm_103a): any head size, alignment and type, in fp32.
//
//   s = scale q.k,  m = max s,  l = sum 2^(s - m),  o = sum 2^(s - m) v
// in one pass over the tokens, with s in powers of two (scale times log2 e).  For rows
// that are not made of 16-byte granules (E4M3: of columns by sixteens), or of more than 256 columns, or whose pages are
// no whole number of rows apart (attend_mma_takes).  A CTA has 64 tokens at a time: a warp its
// keys, columns over the lanes; then a thread a column of the values and a share of the tokens.  Bound by
// instructions (264 of a warp a token and key head of 99, two bytes a load; 68 % of the issue slots) and, for
// longer heads, the latency of one stage after the other:
// 131072 tokens x 8 heads, bf16, heads of 99 316 us, of 320 1.07 ms, five times their bytes at the copy rate.  A load is
// converted only when all of its batch are under way: one that waits for its own takes 607 us, and 3.35 ms.
#include "dit_attend.cuh"

namespace dit {
namespace {

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kTokens = 64;  // at a time
constexpr int kMaxD = 512;
constexpr int kExtra = 4, kLeast = 2;  // units of a segment beside its tiles; the smallest part

// Threads of a column of values, each with its share of the tokens and its own sum.
__host__ __device__ inline int column_threads(int D) {
  const int threads = kThreads / ((D + 31) / 32 * 32);
  return threads > 1 ? threads : 1;
}

template <class K>
__device__ __forceinline__ float cached(K x) {
  if constexpr (sizeof(K) == 1)
    return from_e4m3(x);
  else
    return to_float(x);
}

// K: the cache's type (uint8_t: E4M3), T: the queries'.
// N: columns of a lane, at most; R: rows (query heads) at most.
template <class T, class K, int N, int R>
__global__ void __launch_bounds__(kThreads, N == 4 && R == 4 ? 4 : 2) attend_kernel(const __grid_constant__ AttendArgs a) {
  constexpr bool FP8 = sizeof(K) == 1;
  constexpr int kAhead = N == 4 ? 4 : 2, kValues = 8;  // keys of a warp, and values of a thread, in flight
  __shared__ Plan<kThreads> plan;
  __shared__ int64_t place[kTokens];
  __shared__ float kscale[kTokens], vscale[kTokens];
  __shared__ __align__(16) float weight[kTokens][R + 4];  // (4: banks, and 16-byte reads)
  __shared__ float m[R], l[R], factor[R];
  extern __shared__ float space[];
  const int D = (int)a.c.D;
  float* q = space;                    // [rows][D]
  float* o = space + R * D;            // [threads of a column][rows][D]
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int shares = column_threads(D), share = shares > 1 ? tid / ((D + 31) / 32 * 32) : 0;
  const int column = share < shares ? tid - share * ((D + 31) / 32 * 32) : D;
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
    }
    for (int i = tid; i < shares * rows * D; i += kThreads) o[i] = 0.0f;
    for (int i = tid; i < kTokens * (R + 4); i += kThreads) weight[0][i] = 0.0f;  // (rows beyond the last)
    if (tid < R) m[tid] = -INFINITY, l[tid] = 0.0f;
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
      for (int t0 = warp * kAhead; t0 < kTokens; t0 += kWarps * kAhead) {
        // (all loads before the first conversion, which would wait for its own)
        K raw[kAhead][N] = {};
#pragma unroll
        for (int j = 0; j < kAhead; ++j) {
          const K* row = (const K*)a.c.k + place[t0 + j] + lane;
          const int size = place[t0 + j] >= 0 ? D - lane : 0;
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (32 * i < size) raw[j][i] = row[32 * i];
        }
        float k[kAhead][N];
#pragma unroll
        for (int j = 0; j < kAhead; ++j)
#pragma unroll
          for (int i = 0; i < N; ++i) k[j][i] = cached(raw[j][i]);
        for (int r = 0; r < rows; ++r) {
          float s[kAhead] = {};
#pragma unroll
          for (int i = 0; i < N; ++i)
            if (lane + 32 * i < D) {
              const float x = q[r * D + lane + 32 * i];
#pragma unroll
              for (int j = 0; j < kAhead; ++j) s[j] = __fmaf_rn(x, k[j][i], s[j]);
            }
#pragma unroll
          for (int j = 0; j < kAhead; ++j) s[j] = lanes_sum<32>(s[j]);
          float mine = s[0];
#pragma unroll
          for (int j = 1; j < kAhead; ++j) mine = lane == j ? s[j] : mine;
          if (lane < kAhead) {
            if constexpr (FP8) mine = __fmul_rn(mine, kscale[t0 + lane]);
            weight[t0 + lane][r] = place[t0 + lane] >= 0 ? __fmul_rn(mine, 1.4426950408889634f) : -INFINITY;
          }
        }
      }
      __syncthreads();
      for (int r = warp; r < rows; r += kWarps) {
        const float s0 = weight[lane][r], s1 = weight[lane + 32][r];
        float most = fmaxf(s0, s1);
#pragma unroll
        for (int k = 16; k > 0; k >>= 1) most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, k));
        const float was = m[r], now = fmaxf(was, most);
        const float base = now == -INFINITY ? 0.0f : now;
        const float p0 = exp2f(__fadd_rn(s0, -base)), p1 = exp2f(__fadd_rn(s1, -base));
        const float f = exp2f(__fadd_rn(was, -base));
        const float sum = lanes_sum<32>(__fadd_rn(p0, p1));
        weight[lane][r] = p0;
        weight[lane + 32][r] = p1;
        __syncwarp();
        if (lane == 0) {
          m[r] = now;
          factor[r] = f;
          l[r] = __fmaf_rn(l[r], f, sum);
        }
      }
      __syncthreads();
      for (int c = column; c < D; c += kThreads) {
        float* sum = o + share * rows * D + c;
        float acc[R];
#pragma unroll
        for (int r = 0; r < R; ++r) acc[r] = r < rows ? __fmul_rn(sum[r * D], factor[r]) : 0.0f;
        for (int t = share * kValues; t < n; t += shares * kValues) {
          K raw[kValues] = {};
#pragma unroll
          for (int j = 0; j < kValues; ++j)
            if (place[t + j] >= 0) raw[j] = ((const K*)a.c.v)[place[t + j] + c];
#pragma unroll
          for (int j = 0; j < kValues; ++j) {
            float v = cached(raw[j]);
            if constexpr (FP8) v = __fmul_rn(v, vscale[t + j]);
#pragma unroll
            for (int r = 0; r < R; r += 4) {
              const float4 p = *(const float4*)&weight[t + j][r];
              acc[r] = __fmaf_rn(p.x, v, acc[r]);
              acc[r + 1] = __fmaf_rn(p.y, v, acc[r + 1]);
              acc[r + 2] = __fmaf_rn(p.z, v, acc[r + 2]);
              acc[r + 3] = __fmaf_rn(p.w, v, acc[r + 3]);
            }
          }
        }
#pragma unroll
        for (int r = 0; r < R; ++r)
          if (r < rows) sum[r * D] = acc[r];
      }
    }
    __syncthreads();
    const auto value = [&](int i) {
      float y = o[i];
      for (int k = 1; k < shares; ++k) y = __fadd_rn(y, o[k * rows * D + i]);
      return y;
    };
    if (g.head || g.tail) {
      const int slot = g.head ? 0 : 1;
      float* out = a.partial + ((int64_t)blockIdx.x * 2 + slot) * slot_rows * (D + 2);
      if (tid == 0) a.owner[2 * blockIdx.x + slot] = segment_id(g.b, g.s);
      for (int i = tid; i < rows * D; i += kThreads) out[2 * slot_rows + i] = value(i);
      if (tid < rows) {
        out[tid] = m[tid];
        out[slot_rows + tid] = l[tid];
      }
    } else {
      for (int i = tid; i < rows * D; i += kThreads) {
        const int r = i / D, c = i - r * D;
        const float total = l[r];
        ((T*)a.out.p)[g.b * a.out.token + (h0 + r) * a.out.head + c] =
            from_float<T>(total == 0.0f ? 0.0f : __fdiv_rn(value(i), total));
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

template <class T, class K, int N, int R>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  const auto kern = attend_kernel<T, K, N, R>;
  const size_t smem = (size_t)(1 + column_threads((int)a.c.D)) * R * a.c.D * 4;
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  *ctas = std::min(kAttendMaxCtas,
                   (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kThreads, smem));
  return launch_after(kern, (unsigned)*ctas, kThreads, smem, s, a);
}
template <class T, class K>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.c.D <= 128 ? (a.group <= 4 ? launch<T, K, 4, 4>(dev, a, ctas, s) : launch<T, K, 4, kAttendRows>(dev, a, ctas, s))
                      : (a.group <= 4 ? launch<T, K, kMaxD / 32, 4>(dev, a, ctas, s)
                                      : launch<T, K, kMaxD / 32, kAttendRows>(dev, a, ctas, s));
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
