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
  after_previous();
  let_next();
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
  after_previous();
  let_next();
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

// Rows in 16-byte granules: a team of TEAM lanes has a row, a lane granules l and l + TEAM of it; a warp
// takes kAhead rows of each team at once, which are consecutive: a token's keys, its values, the next token's keys.
constexpr int kAhead = 4;

struct CacheRows {
  CacheArgs a;
  Divisor rows, page;  // 2 heads, page_size
  int64_t items;
};
// The row `local` rows behind row `part` of token `token`.
struct RowAt {
  int which, head;
  int64_t token, page, place;
  bool on, inside;
  __device__ __forceinline__ RowAt(const CacheRows& c, int64_t token0, int part, int local) {
    const uint32_t r = part + local, q = quotient(r, c.rows);
    token = token0 + q;
    head = (int)(r - q * c.rows.d);
    which = head >= (int)c.a.c.heads;
    if (which) head -= (int)c.a.c.heads;
    on = token < c.a.tokens;
    const int64_t slot = on ? id_at(c.a.slots, token, c.a.ids64) : -1;
    inside = slot >= 0 && slot < c.a.c.pages * c.a.c.page_size;
    page = inside ? quotient((uint32_t)slot, c.page) : 0;
    place = inside ? slot - page * c.page.d : 0;
  }
  // granule 0 of the row in the cache (ES bytes an element), its scale, and its granule 0 among the tokens'
  template <int ES>
  __device__ __forceinline__ char* cached(const dit_cache& c) const {
    return (char*)(which ? c.v : c.k) + (page * c.page_stride + ((int64_t)head * c.page_size + place) * c.D) * ES;
  }
  __device__ __forceinline__ float* scale(const dit_cache& c) const {
    return (which ? c.v_scales : c.k_scales) + page * c.scale_stride + (int64_t)head * c.page_size + place;
  }
  template <int ES>
  __device__ __forceinline__ char* row(const CacheArgs& a) const {
    const dit_heads& t = which ? a.v : a.k;
    return (char*)t.p + (token * t.token + head * t.head) * ES;
  }
};

template <class T, int TEAM, bool FP8>
__global__ void __launch_bounds__(kThreads) write_rows_kernel(const __grid_constant__ CacheRows args) {
  constexpr int ES = (int)sizeof(T), PER = 16 / ES, P = PER / 2, TEAMS = 32 / TEAM;
  const CacheArgs& a = args.a;
  const int lane = threadIdx.x & 31, team = lane / TEAM, l = lane % TEAM, n = (int)a.c.D / PER;
  after_previous();
  let_next();
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < args.items; i += stride) {
    const int64_t token0 = i * (kAhead * TEAMS) / args.rows.d;
    const int part = (int)(i * (kAhead * TEAMS) - token0 * args.rows.d);
    Raw<16> raw[kAhead][2];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const RowAt row(args, token0, part, k * TEAMS + team);
      const char* x = row.row<ES>(a);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        raw[k][j] = Raw<16>{};
        if (row.inside && l + j * TEAM < n) raw[k][j] = ld_stream<16>(x + (l + j * TEAM) * 16);
      }
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const RowAt row(args, token0, part, k * TEAMS + team);
      if constexpr (FP8) {
        F2 x[2][P];
        float m = 0.0f;
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          Granule<T>::widen(raw[k][j], x[j]);
#pragma unroll
          for (int e = 0; e < P; ++e) m = max_abs3(m, x[j][e].x, x[j][e].y);
        }
        const RowQuant q = row_quant(lanes_max<TEAM>(m));
        if (!row.inside) continue;
        char* out = row.cached<1>(a.c);
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          Raw<PER> codes;
#pragma unroll
          for (int e = 0; e < P / 2; ++e) {
            F2 v[2];
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const F2 y = f2_mul(x[j][2 * e + h], f2(q.small, q.small));
              v[h] = f2_fma(y, f2(q.mul, q.mul), f2_mul(y, f2(q.low, q.low)));
            }
            codes.w[e] = e4m3x2(v[0]) | e4m3x2(v[1]) << 16;
          }
          if (l + j * TEAM < n) st_stream<PER>(out + (l + j * TEAM) * PER, codes);
        }
        if (l == 0) *row.scale(a.c) = q.scale;
      } else {
        if (!row.inside) continue;
        char* out = row.cached<ES>(a.c);
#pragma unroll
        for (int j = 0; j < 2; ++j)
          if (l + j * TEAM < n) st_stream<16>(out + (l + j * TEAM) * 16, raw[k][j]);
      }
    }
  }
}

template <class T, int TEAM, bool FP8>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ CacheRows args) {
  constexpr int ES = (int)sizeof(T), PER = 16 / ES, P = PER / 2, TEAMS = 32 / TEAM;
  constexpr int CB = FP8 ? PER : 16;  // bytes of a granule's columns in the cache
  const CacheArgs& a = args.a;
  const int lane = threadIdx.x & 31, team = lane / TEAM, l = lane % TEAM, n = (int)a.c.D / PER;
  after_previous();
  let_next();
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < args.items; i += stride) {
    const int64_t token0 = i * (kAhead * TEAMS) / args.rows.d;
    const int part = (int)(i * (kAhead * TEAMS) - token0 * args.rows.d);
    Raw<CB> raw[kAhead][2];
    float scale[kAhead];
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const RowAt row(args, token0, part, k * TEAMS + team);
      const char* x = row.cached<FP8 ? 1 : ES>(a.c);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        raw[k][j] = Raw<CB>{};
        if (row.inside && l + j * TEAM < n) raw[k][j] = ld_stream<CB>(x + (l + j * TEAM) * CB);
      }
      if constexpr (FP8) scale[k] = row.inside ? *row.scale(a.c) : 0.0f;
    }
#pragma unroll
    for (int k = 0; k < kAhead; ++k) {
      const RowAt row(args, token0, part, k * TEAMS + team);
      if (!row.on) continue;
      char* out = row.row<ES>(a);
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        Raw<16> y;
        if constexpr (FP8) {
          F2 x[P];
#pragma unroll
          for (int e = 0; e < P; ++e) {
            const float2 v = from_e4m3x2((uint16_t)(raw[k][j].w[e / 2] >> (16 * (e & 1))));
            x[e] = f2_mul(v, f2(scale[k], scale[k]));
          }
          y = Granule<T>::narrow(x);
        } else {
          y = raw[k][j];
        }
        if (l + j * TEAM < n) st_stream<16>(out + (l + j * TEAM) * 16, y);
      }
    }
  }
}

template <class Args>
cudaError_t launch(const DeviceInfo& dev, void (*kern)(Args), int64_t warps, const Args& a, cudaStream_t s) {
  const int64_t most = (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kThreads) * 8;
  return launch_after(kern, (unsigned)std::min(most, (warps + kThreads / 32 - 1) / (kThreads / 32)), kThreads, 0, s, a);
}

template <class T, bool FP8>
cudaError_t launch(const DeviceInfo& dev, bool write, const CacheArgs& a, cudaStream_t s) {
  const int64_t rows = a.tokens * 2 * a.c.heads, half = (a.c.D * (int)sizeof(T) / 16 + 1) / 2;
  if (!a.granules || half > 32) return launch(dev, write ? write_kernel<T, FP8> : read_kernel<T, FP8>, rows, a, s);
  CacheRows c{a, divisor((uint32_t)(2 * a.c.heads)), divisor((uint32_t)a.c.page_size), 0};
  auto team = [&](auto lanes) {
    constexpr int TEAM = decltype(lanes)::value;
    c.items = (rows + kAhead * 32 / TEAM - 1) / (kAhead * 32 / TEAM);
    return launch(dev, write ? write_rows_kernel<T, TEAM, FP8> : read_rows_kernel<T, TEAM, FP8>, c.items, c, s);
  };
  return half <= 4    ? team(std::integral_constant<int, 4>{})
         : half <= 8  ? team(std::integral_constant<int, 8>{})
         : half <= 16 ? team(std::integral_constant<int, 16>{})
                      : team(std::integral_constant<int, 32>{});
}
cudaError_t launch(const DeviceInfo& dev, int dtype, bool write, const CacheArgs& a, cudaStream_t s) {
  const bool fp8 = a.c.format == DIT_E4M3;
  return dtype == 0   ? (fp8 ? launch<__nv_bfloat16, true>(dev, write, a, s) : launch<__nv_bfloat16, false>(dev, write, a, s))
         : dtype == 1 ? (fp8 ? launch<__half, true>(dev, write, a, s) : launch<__half, false>(dev, write, a, s))
                      : (fp8 ? launch<float, true>(dev, write, a, s) : launch<float, false>(dev, write, a, s));
}

}  // namespace

cudaError_t launch_cache_write(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s) {
  return launch(dev, dtype, true, a, s);
}
cudaError_t launch_cache_read(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s) {
  return launch(dev, dtype, false, a, s);
}

}  // namespace dit
