// k_cache.cu -- rows of keys and values into and out of a paged cache (sm_103a).
//
// A row is one head of one token, D columns.  In E4M3 it is written as
//   m = max|x|,  scale = m / 448,  code = e4m3(x 448 / m)
// with the quotient in two fp32 numbers, so that a code is the nearest to the exact
// quotient but where that lies within 2^-24 of itself from the middle of two codes.
#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {
namespace {

constexpr int kThreads = 256;

struct CacheRow {
  int which, head;  // 0: keys, 1: values
  int64_t token, page, place;
  bool inside;
  __device__ __forceinline__ CacheRow(const CacheArgs& a, int64_t i) {
    const int rows = 2 * (int)a.c.heads;
    token = i / rows;
    head = (int)(i - token * rows);
    which = head >= (int)a.c.heads;
    if (which) head -= (int)a.c.heads;
    const int64_t slot = id_at(a.slots, token, a.ids64);
    inside = slot >= 0 && slot < a.c.pages * a.c.page_size;
    page = inside ? slot / a.c.page_size : 0;
    place = inside ? slot - page * a.c.page_size : 0;
  }
  // element and scale number in the cache
  __device__ __forceinline__ int64_t at(const dit_cache& c) const {
    return page * c.page_stride + ((int64_t)head * c.page_size + place) * c.D;
  }
  __device__ __forceinline__ int64_t scale_at(const dit_cache& c) const {
    return page * c.scale_stride + (int64_t)head * c.page_size + place;
  }
  __device__ __forceinline__ int64_t at(const dit_heads& t) const {
    return token * t.token + head * t.head;
  }
};

// Any view: a warp has a row, an element per access.
template <class T, bool FP8>
__global__ void __launch_bounds__(kThreads) write_kernel(const __grid_constant__ CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.tokens * 2 * a.c.heads;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  const int D = (int)a.c.D;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < rows; i += stride) {
    const CacheRow row(a, i);
    if (!row.inside) continue;
    const dit_heads& from = row.which ? a.v : a.k;
    const T* x = (const T*)from.p + row.at(from);
    if constexpr (FP8) {
      float m = 0.0f;
      for (int c = lane; c < D; c += 32) m = max_nan(m, fabsf(to_float(x[c])));
      const RowQuant q = row_quant(lanes_max<32>(m));
      uint8_t* out = (uint8_t*)(row.which ? a.c.v : a.c.k) + row.at(a.c);
      for (int c = lane; c < D; c += 32)
        out[c] = (uint8_t)e4m3x2(f2(code_value(to_float(x[c]), q), 0.0f));
      if (lane == 0) (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)] = q.scale;
    } else {
      T* out = (T*)(row.which ? a.c.v : a.c.k) + row.at(a.c);
      for (int c = lane; c < D; c += 32) out[c] = x[c];
    }
  }
}

template <class T, bool FP8>
__global__ void __launch_bounds__(kThreads) read_kernel(const __grid_constant__ CacheArgs a) {
  const int lane = threadIdx.x & 31;
  const int64_t rows = a.tokens * 2 * a.c.heads;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  const int D = (int)a.c.D;
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < rows; i += stride) {
    const CacheRow row(a, i);
    const dit_heads& to = row.which ? a.v : a.k;
    T* out = (T*)to.p + row.at(to);
    if (!row.inside) {
      for (int c = lane; c < D; c += 32) out[c] = from_float<T>(0.0f);
    } else if constexpr (FP8) {
      const uint8_t* x = (const uint8_t*)(row.which ? a.c.v : a.c.k) + row.at(a.c);
      const float scale = (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)];
      for (int c = lane; c < D; c += 32) out[c] = from_float<T>(__fmul_rn(from_e4m3(x[c]), scale));
    } else {
      const T* x = (const T*)(row.which ? a.c.v : a.c.k) + row.at(a.c);
      for (int c = lane; c < D; c += 32) out[c] = x[c];
    }
  }
}

cudaError_t launch(const DeviceInfo& dev, void (*kern)(CacheArgs), const CacheArgs& a, cudaStream_t s) {
  const int64_t warps = kThreads / 32, rows = a.tokens * 2 * a.c.heads;
  const int64_t most = (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kThreads) * 8;
  kern<<<(unsigned)std::min(most, (rows + warps - 1) / warps), kThreads, 0, s>>>(a);
  return cudaGetLastError();
}

}  // namespace

cudaError_t launch_cache_write(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s) {
  const bool fp8 = a.c.format == DIT_E4M3;
  return dtype == 0   ? launch(dev, fp8 ? write_kernel<__nv_bfloat16, true> : write_kernel<__nv_bfloat16, false>, a, s)
         : dtype == 1 ? launch(dev, fp8 ? write_kernel<__half, true> : write_kernel<__half, false>, a, s)
                      : launch(dev, fp8 ? write_kernel<float, true> : write_kernel<float, false>, a, s);
}

cudaError_t launch_cache_read(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s) {
  const bool fp8 = a.c.format == DIT_E4M3;
  return dtype == 0   ? launch(dev, fp8 ? read_kernel<__nv_bfloat16, true> : read_kernel<__nv_bfloat16, false>, a, s)
         : dtype == 1 ? launch(dev, fp8 ? read_kernel<__half, true> : read_kernel<__half, false>, a, s)
                      : launch(dev, fp8 ? read_kernel<float, true> : read_kernel<float, false>, a, s);
}

}  // namespace dit
