// k_clip.cu -- the global 2-norm of many tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = rnd(g * c),  c = fl32(min(1, max_norm / (norm + eps)))
//
// One launch covers up to kClipBatch tensors: their descriptions travel in the
// kernel's parameters, so nothing is copied to the device and a captured
// graph carries them.  A tensor is cut into chunks of 16 or 32 KB
// (the smaller for few bytes in all, so that every SM has some), and CTA c of G
// takes chunks c, c + G, ... over all tensors; each thread sums its elements of a
// chunk in fp32 (two packed accumulators) and the chunks as (high, low) pairs
// of fp32 (dit_stat.cuh), which cost a tenth of this GPU's fp64.  A chunk's
// sum that leaves [2^-100, 2^100] (a square that overflowed or went below
// fp32's normal range) is taken again by its thread in fp64 and kept apart.
// Each CTA writes one fp64 partial sum, and every CTA of the second kernel
// adds them in the same order: the same call gives the same bits.  The second
// kernel takes the chunks from the last, which the L2 may still hold, to the
// first.
//
// Memory bounds large calls: 400 M bf16 elements in 291 tensors take 128 us for
// the norm (6.3 TB/s) and 255 us for the clipping (6.3 TB/s read and written);
// the norm has to be known before the first output, so the gradients are read
// twice.  60 fp32 tensors of 2 M elements take 7.4 us, two launches; with sums in
// fp64 they took 13.4.
#include <math.h>

#include <algorithm>

#include "dit_stat.cuh"
#include "dit_token.h"
#include "dit_unit.cuh"

namespace dit {
namespace {

constexpr int kMaxChunk = 32 << 10, kMinChunk = 16 << 10;
constexpr int kThreads = 512;
constexpr int kAhead = 4;  // granules of a thread in flight

template <int K>
struct Batch {
  const void* g[K];
  void* out[K];
  int64_t n[K];
  int32_t first[K + 1];  // the tensors' first chunks
  uint8_t dtype[K];
  int count, chunk;  // tensors; bytes of a chunk
};

template <int K>
struct NormSum {
  Batch<K> b;
  double* partial;  // one per CTA
};
template <int K>
struct Clip {
  Batch<K> b;
  const double* partial;
  int64_t npartial;
  float max_norm, eps;
  float* norm;  // written by CTA 0 (NULL: not by this launch)
};

// the tensor of chunk c
template <int K>
__device__ __forceinline__ int tensor_of(const Batch<K>& b, int c) {
  int lo = 0, hi = b.count - 1;
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (b.first[mid] <= c)
      lo = mid;
    else
      hi = mid - 1;
  }
  return lo;
}

// One chunk: scalar elements up to the first 16-byte boundary, granules, the
// elements after the last one.
struct Span16 {
  int head, body, tail;  // elements, granules, elements
};
template <class T>
__device__ __forceinline__ Span16 cut(const void* p, int n) {
  constexpr int ES = (int)sizeof(T), EPG = 16 / ES;
  Span16 s;
  s.head = (int)(((16u - ((uintptr_t)p & 15u)) & 15u) / ES);
  if (s.head > n) s.head = n;
  s.body = (n - s.head) / EPG;
  s.tail = n - s.head - s.body * EPG;
  return s;
}

template <class T>
__device__ __forceinline__ float element(const void* p, int i) {
  float f[1];
  Vec<T, (int)sizeof(T)>::widen(ld_stream<sizeof(T)>((const char*)p + (int64_t)i * (int)sizeof(T)), f);
  return f[0];
}

// this thread's sum of the squares of a chunk, added to `sum`, or to `far`
// when it is out of fp32's range
template <class T>
__device__ __forceinline__ void chunk_sum(const char* p, int n, SumPair& sum, double& far) {
  constexpr int ES = (int)sizeof(T), EPG = 16 / ES, P = Granule<T>::P;
  const Span16 s = cut<T>(p, n);
  const char* body = p + s.head * ES;
  const int tid = threadIdx.x;
  F2 acc[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
  uint32_t any = 0;  // a bit of any element but its sign
  for (int i0 = tid; i0 < s.body; i0 += kAhead * kThreads) {
    Raw<16> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      r[j] = Raw<16>{};
      if (i0 + j * kThreads < s.body) r[j] = ld_stream<16>(body + (int64_t)(i0 + j * kThreads) * 16);
    }
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      F2 f[P];
      Granule<T>::widen(r[j], f);
      any |= r[j].w[0] | r[j].w[1] | r[j].w[2] | r[j].w[3];
#pragma unroll
      for (int i = 0; i < P; ++i) acc[i & 1] = f2_fma(f[i], f[i], acc[i & 1]);
    }
  }
  // the edges: one element for each of the first threads
  float e = 0.0f;
  if (tid < s.head + s.tail)
    e = element<T>(p, tid < s.head ? tid : s.head + s.body * EPG + tid - s.head);
  acc[0] = f2_add(acc[0], acc[1]);
  const float S = __fmaf_rn(e, e, __fadd_rn(acc[0].x, acc[0].y));
  constexpr uint32_t kBits = ES == 4 ? 0x7FFFFFFFu : 0x7FFF7FFFu;
  if ((S >= 0x1p-100f && S <= 0x1p100f) || (S == 0.0f && (any & kBits) == 0 && e == 0.0f)) {
    sum = merge(sum, SumPair{S, 0.0f});
    return;
  }
  double d = (double)e * (double)e;
  for (int i = tid; i < s.body; i += kThreads) {
    F2 f[P];
    Granule<T>::widen(ld_stream<16>(body + (int64_t)i * 16), f);
#pragma unroll
    for (int k = 0; k < P; ++k)
      d += (double)f[k].x * (double)f[k].x + (double)f[k].y * (double)f[k].y;
  }
  far += d;
}

template <class F>
__device__ __forceinline__ void with_type(int dtype, F&& f) {
  if (dtype == 0)
    f(TypeTag<__nv_bfloat16>{});
  else if (dtype == 1)
    f(TypeTag<__half>{});
  else
    f(TypeTag<float>{});
}

__device__ __forceinline__ double warp_sum(double v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  return v;
}

template <int K>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ NormSum<K> a) {
  let_next();
  __shared__ SumPair pairs[32];
  __shared__ double fars[kThreads / 32];
  SumPair sum{0.0f, 0.0f};
  double far = 0.0;
  const int chunks = a.b.first[a.b.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a.b, c);
    with_type(a.b.dtype[t], [&](auto tag) {
      using T = typename decltype(tag)::type;
      const int most = a.b.chunk / (int)sizeof(T);
      const int64_t at = (int64_t)(c - a.b.first[t]) * most;
      const int n = (int)min((int64_t)most, a.b.n[t] - at);
      chunk_sum<T>((const char*)a.b.g[t] + at * (int)sizeof(T), n, sum, far);
    });
  }
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  sum = warp_merge(sum);
  if (threadIdx.x < 32) pairs[lane] = SumPair{0.0f, 0.0f};
  const bool any_far = __syncthreads_or(far != 0.0) != 0;  // (NaN != 0)
  if (lane == 0) pairs[warp] = sum;
  if (any_far) {
    far = warp_sum(far);
    if (lane == 0) fars[warp] = far;
  }
  __syncthreads();
  if (warp > 0) return;
  sum = warp_merge(pairs[lane]);
  if (lane == 0) {
    double total = (double)sum.h + (double)sum.l;
    if (any_far)
      for (int w = 0; w < kThreads / 32; ++w) total += fars[w];
    a.partial[blockIdx.x] = total;
  }
}

// The sum of the partial sums, in one order: by one warp.
__device__ __forceinline__ double total_of(const double* partial, int64_t n) {
  double v = 0.0;
#pragma unroll 8
  for (int64_t i = threadIdx.x & 31; i < n; i += 32) v += partial[i];
  return warp_sum(v);
}
__device__ __forceinline__ float norm_of(double total) {
  return total >= 0x1p-100 && total <= 0x1p100 ? __fsqrt_rn((float)total) : (float)sqrt(total);
}

struct Norm {
  const double* partial;
  int64_t npartial;
  float* norm;
};
__global__ void __launch_bounds__(32) norm_kernel(Norm a) {
  after_previous();
  const float n = norm_of(total_of(a.partial, a.npartial));
  if (threadIdx.x == 0) *a.norm = n;
}

// granules when g and out are alike modulo 16 bytes, else single elements
template <class T>
__device__ __forceinline__ void scale_chunk(const char* g, char* out, int n, float c) {
  constexpr int ES = (int)sizeof(T), EPG = 16 / ES, P = Granule<T>::P;
  const int tid = threadIdx.x;
  auto one = [&](int i) {
    float f[1] = {__fmul_rn(element<T>(g, i), c)};
    st_stream<ES>(out + (int64_t)i * ES, Vec<T, ES>::narrow(f));
  };
  if ((((uintptr_t)g ^ (uintptr_t)out) & 15u) != 0) {
    for (int i = tid; i < n; i += kThreads) one(i);
    return;
  }
  const Span16 s = cut<T>(g, n);
  const char* gb = g + s.head * ES;
  char* ob = out + s.head * ES;
  for (int i0 = tid; i0 < s.body; i0 += kAhead * kThreads) {
    Raw<16> r[kAhead];
#pragma unroll
    for (int j = 0; j < kAhead; ++j)
      if (i0 + j * kThreads < s.body) r[j] = ld_stream<16>(gb + (int64_t)(i0 + j * kThreads) * 16);
#pragma unroll
    for (int j = 0; j < kAhead; ++j) {
      if (i0 + j * kThreads >= s.body) continue;
      F2 f[P];
      Granule<T>::widen(r[j], f);
#pragma unroll
      for (int k = 0; k < P; ++k) f[k] = f2_mul(f[k], f2(c, c));
      st_stream<16>(ob + (int64_t)(i0 + j * kThreads) * 16, Granule<T>::narrow(f));
    }
  }
  if (tid < s.head + s.tail) one(tid < s.head ? tid : s.head + s.body * EPG + tid - s.head);
}

template <int K>
__global__ void __launch_bounds__(kThreads) clip_kernel(const __grid_constant__ Clip<K> a) {
  __shared__ float factor;
  after_previous();
  if (threadIdx.x < 32) {
    const float norm = norm_of(total_of(a.partial, a.npartial));
    const float q = __fdiv_rn(a.max_norm, __fadd_rn(norm, a.eps));
    if (threadIdx.x == 0) {
      factor = q > 1.0f ? 1.0f : q;  // NaN stays NaN
      if (a.norm && blockIdx.x == 0) *a.norm = norm;
    }
  }
  __syncthreads();
  const float c = factor;
  const int chunks = a.b.first[a.b.count];
  for (int i = chunks - 1 - (int)blockIdx.x; i >= 0; i -= gridDim.x) {
    const int t = tensor_of(a.b, i);
    with_type(a.b.dtype[t], [&](auto tag) {
      using T = typename decltype(tag)::type;
      const int most = a.b.chunk / (int)sizeof(T);
      const int64_t at = (int64_t)(i - a.b.first[t]) * most;
      const int n = (int)min((int64_t)most, a.b.n[t] - at);
      scale_chunk<T>((const char*)a.b.g[t] + at * (int)sizeof(T),
                     (char*)a.b.out[t] + at * (int)sizeof(T), n, c);
    });
  }
}

// the descriptions of tensors [at, at + K) in chunks of `chunk` bytes; -1 when there
// are too many chunks
template <int K>
int fill(Batch<K>& b, const ClipTensor* t, int64_t count, int chunk) {
  int64_t chunks = 0;
  b.count = (int)std::min<int64_t>(K, count);
  b.chunk = chunk;
  for (int i = 0; i < b.count; ++i) {
    b.g[i] = t[i].g;
    b.out[i] = t[i].out;
    b.n[i] = t[i].n;
    b.dtype[i] = (uint8_t)t[i].dtype;
    b.first[i] = (int32_t)chunks;
    const int most = chunk / (t[i].dtype == 2 ? 4 : 2);
    chunks += (t[i].n + most - 1) / most;
    if (chunks > 0x7FFFFFFF - kClipMaxCtas) return -1;
  }
  b.first[b.count] = (int32_t)chunks;
  return (int)chunks;
}

template <int K>
cudaError_t launch(const DeviceInfo& dev, const ClipTensor* t, int64_t count, bool clip,
                   float max_norm, float eps, double* partial, float* norm, cudaStream_t s) {
  // the smallest chunk that leaves at most 2 chunks per SM
  double bytes = 0.0;
  for (int64_t i = 0; i < count; ++i) bytes += (double)t[i].n * (t[i].dtype == 2 ? 4 : 2);
  int chunk = kMinChunk;
  while (chunk < kMaxChunk && bytes > 2.0 * dev.sm_count * chunk) chunk *= 2;
  int64_t npartial = 0;
  auto ctas = [&](const void* fn, int chunks) {
    const int64_t wave = (int64_t)dev.sm_count * resident_ctas(dev, fn, kThreads);
    return (unsigned)std::min<int64_t>({(int64_t)chunks, kClipMaxCtas, wave});
  };
  for (int64_t at = 0; at < count; at += K) {
    NormSum<K> a;
    const int chunks = fill(a.b, t + at, count - at, chunk);
    if (chunks < 0) return cudaErrorInvalidValue;
    if (chunks == 0) continue;
    a.partial = partial + npartial;
    const unsigned grid = ctas((const void*)sum_kernel<K>, chunks);
    sum_kernel<K><<<grid, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    npartial += grid;
  }
  if (!clip || npartial == 0) return launch_after(norm_kernel, 1, 32, 0, s, Norm{partial, npartial, norm});
  bool first = true;
  for (int64_t at = 0; at < count; at += K) {
    Clip<K> a;
    const int chunks = fill(a.b, t + at, count - at, chunk);
    if (chunks <= 0) continue;
    a.partial = partial;
    a.npartial = npartial;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = first ? norm : nullptr;
    const unsigned grid = ctas((const void*)clip_kernel<K>, chunks);
    cudaError_t e;
    if (first) {
      e = launch_after(clip_kernel<K>, grid, kThreads, 0, s, a);
    } else {
      clip_kernel<K><<<grid, kThreads, 0, s>>>(a);
      e = cudaGetLastError();
    }
    if (e != cudaSuccess) return e;
    first = false;
  }
  return cudaSuccess;
}

}  // namespace

// Few tensors take a launch with small parameters (1.9 KB, the others 28 KB).
// Host us a call with its workspace, small tensors: 60 in the small form 10.4, in the
// large one 12.3; 65 in batches of the small form 16.0, in the large one 12.3; 300
// 37.5 and 18.6.
cudaError_t launch_clip(const DeviceInfo& dev, const ClipTensor* t, int64_t count, bool clip,
                        float max_norm, float eps, double* partial, float* norm, cudaStream_t s) {
  return count <= 64 ? launch<64>(dev, t, count, clip, max_norm, eps, partial, norm, s)
                     : launch<kClipBatch>(dev, t, count, clip, max_norm, eps, partial, norm, s);
}

}  // namespace dit
