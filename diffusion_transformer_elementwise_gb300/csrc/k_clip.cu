// k_clip.cu -- the global 2-norm of many tensors, and clipping by it.
//
//   norm = sqrt(sum over all tensors and elements of g^2)
//   out  = rnd(g * c),  c = fl32(min(1, max_norm / (norm + eps)))
//
// One launch covers up to kClipBatch tensors: their descriptions travel in the
// kernel's parameters, so nothing is copied to the device and a captured
// graph carries them.  A tensor is cut into chunks of 16384 elements, and CTA c of
// G takes chunks c, c + G, ... over all tensors; each thread sums its elements of a
// chunk in fp32 (two packed accumulators) and the chunks in fp64.  A chunk's sum that
// leaves [2^-100, 2^100] (a square that overflowed or went below fp32's
// normal range) is taken again by its thread in fp64.  Each CTA writes one fp64 partial sum, and every
// CTA of the second kernel adds them in the same order: the same call gives the same
// bits.
#include <math.h>

#include <algorithm>

#include "dit_stat.cuh"
#include "dit_token.h"
#include "dit_unit.cuh"

namespace dit {
namespace {

constexpr int kChunk = 16384;
constexpr int kThreads = 256;

template <int K>
struct Batch {
  const void* g[K];
  void* out[K];
  int64_t n[K];
  int32_t first[K + 1];  // the tensors' first chunks
  uint8_t dtype[K];
  int count;
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

// this thread's sum of the squares of a chunk
template <class T>
__device__ __forceinline__ double chunk_sum(const char* p, int n) {
  constexpr int ES = (int)sizeof(T), EPG = 16 / ES, P = Granule<T>::P;
  const Span16 s = cut<T>(p, n);
  const char* body = p + s.head * ES;
  const int tid = threadIdx.x;
  F2 acc[2] = {f2(0.0f, 0.0f), f2(0.0f, 0.0f)};
  uint32_t any = 0;  // a bit of any element but its sign
  for (int i0 = tid; i0 < s.body; i0 += 4 * kThreads) {
    Raw<16> r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      r[j] = Raw<16>{};
      if (i0 + j * kThreads < s.body) r[j] = ld_stream<16>(body + (int64_t)(i0 + j * kThreads) * 16);
    }
#pragma unroll
    for (int j = 0; j < 4; ++j) {
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
  if (fast_sum_in_range(S) || (S == 0.0f && (any & kBits) == 0 && e == 0.0f)) return (double)S;
  double d = (double)e * (double)e;
  for (int i = tid; i < s.body; i += kThreads) {
    F2 f[P];
    Granule<T>::widen(ld_stream<16>(body + (int64_t)i * 16), f);
#pragma unroll
    for (int k = 0; k < P; ++k)
      d += (double)f[k].x * (double)f[k].x + (double)f[k].y * (double)f[k].y;
  }
  return d;
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

// a value of every thread summed over the CTA, in one order
__device__ __forceinline__ double cta_sum(double v) {
  __shared__ double part[kThreads / 32];
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = v;
  __syncthreads();
  double t = 0.0;
#pragma unroll
  for (int w = 0; w < kThreads / 32; ++w) t += part[w];
  return t;
}

template <int K>
__global__ void __launch_bounds__(kThreads) sum_kernel(const __grid_constant__ NormSum<K> a) {
  double total = 0.0;
  const int chunks = a.b.first[a.b.count];
  for (int c = blockIdx.x; c < chunks; c += gridDim.x) {
    const int t = tensor_of(a.b, c);
    const int64_t at = (int64_t)(c - a.b.first[t]) * kChunk;
    const int n = (int)min((int64_t)kChunk, a.b.n[t] - at);
    with_type(a.b.dtype[t], [&](auto tag) {
      using T = typename decltype(tag)::type;
      total += chunk_sum<T>((const char*)a.b.g[t] + at * (int)sizeof(T), n);
    });
  }
  total = cta_sum(total);
  if (threadIdx.x == 0) a.partial[blockIdx.x] = total;
}

__device__ __forceinline__ double total_of(const double* partial, int64_t n) {
  double v = 0.0;
  for (int64_t i = threadIdx.x; i < n; i += kThreads) v += partial[i];
  return cta_sum(v);
}

__global__ void __launch_bounds__(kThreads) norm_kernel(const double* partial, int64_t n, float* norm) {
  const double t = total_of(partial, n);
  if (threadIdx.x == 0) *norm = (float)sqrt(t);
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
  for (int i0 = tid; i0 < s.body; i0 += 4 * kThreads) {
    Raw<16> r[4];
#pragma unroll
    for (int j = 0; j < 4; ++j)
      if (i0 + j * kThreads < s.body) r[j] = ld_stream<16>(gb + (int64_t)(i0 + j * kThreads) * 16);
#pragma unroll
    for (int j = 0; j < 4; ++j) {
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
  const double norm = sqrt(total_of(a.partial, a.npartial));
  const double q = (double)a.max_norm / (norm + (double)a.eps);
  const float c = q > 1.0 ? 1.0f : (float)q;  // NaN stays NaN
  if (a.norm && blockIdx.x == 0 && threadIdx.x == 0) *a.norm = (float)norm;
  const int chunks = a.b.first[a.b.count];
  for (int i = blockIdx.x; i < chunks; i += gridDim.x) {
    const int t = tensor_of(a.b, i);
    const int64_t at = (int64_t)(i - a.b.first[t]) * kChunk;
    const int n = (int)min((int64_t)kChunk, a.b.n[t] - at);
    with_type(a.b.dtype[t], [&](auto tag) {
      using T = typename decltype(tag)::type;
      scale_chunk<T>((const char*)a.b.g[t] + at * (int)sizeof(T),
                     (char*)a.b.out[t] + at * (int)sizeof(T), n, c);
    });
  }
}

// the descriptions of tensors [at, at + K); false when the chunks overflow
template <int K>
int fill(Batch<K>& b, const ClipTensor* t, int64_t count) {
  int64_t chunks = 0;
  b.count = (int)std::min<int64_t>(K, count);
  for (int i = 0; i < b.count; ++i) {
    b.g[i] = t[i].g;
    b.out[i] = t[i].out;
    b.n[i] = t[i].n;
    b.dtype[i] = (uint8_t)t[i].dtype;
    b.first[i] = (int32_t)chunks;
    chunks += (t[i].n + kChunk - 1) / kChunk;
    if (chunks > 0x7FFFFFFF - kClipMaxCtas) return -1;
  }
  b.first[b.count] = (int32_t)chunks;
  return (int)chunks;
}

template <int K>
cudaError_t launch(const DeviceInfo& dev, const ClipTensor* t, int64_t count, bool clip,
                   float max_norm, float eps, double* partial, float* norm, cudaStream_t s) {
  int64_t npartial = 0;
  auto ctas = [&](int chunks) {
    return (int)std::min<int64_t>({(int64_t)chunks, kClipMaxCtas, (int64_t)dev.sm_count * 8});
  };
  for (int64_t at = 0; at < count; at += K) {
    NormSum<K> a;
    const int chunks = fill(a.b, t + at, count - at);
    if (chunks < 0) return cudaErrorInvalidValue;
    if (chunks == 0) continue;
    a.partial = partial + npartial;
    const int grid = ctas(chunks);
    sum_kernel<K><<<grid, kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
    npartial += grid;
  }
  if (!clip || npartial == 0) {
    norm_kernel<<<1, kThreads, 0, s>>>(partial, npartial, norm);
    return cudaGetLastError();
  }
  bool first = true;
  for (int64_t at = 0; at < count; at += K) {
    Clip<K> a;
    const int chunks = fill(a.b, t + at, count - at);
    if (chunks <= 0) continue;
    a.partial = partial;
    a.npartial = npartial;
    a.max_norm = max_norm;
    a.eps = eps;
    a.norm = first ? norm : nullptr;
    first = false;
    clip_kernel<K><<<ctas(chunks), kThreads, 0, s>>>(a);
    const cudaError_t e = cudaGetLastError();
    if (e != cudaSuccess) return e;
  }
  return cudaSuccess;
}

}  // namespace

// Few tensors take a launch with small parameters.
cudaError_t launch_clip(const DeviceInfo& dev, const ClipTensor* t, int64_t count, bool clip,
                        float max_norm, float eps, double* partial, float* norm, cudaStream_t s) {
  return count <= 64 ? launch<64>(dev, t, count, clip, max_norm, eps, partial, norm, s)
                     : launch<kClipBatch>(dev, t, count, clip, max_norm, eps, partial, norm, s);
}

}  // namespace dit
