// k_cache.cu -- rows of keys and values into and out of a paged cache (sm_103a).
//
// A row is one head of one token, D columns.  In E4M3 it is written as
//   m = max|x|,  scale = m / 448,  code = e4m3(x 448 / m)
// with the quotient in two fp32 numbers, so that a code is the nearest to the exact
// quotient but where that lies within 2^-24 of itself from the middle of two codes.
// Both ways are bound by memory; the way in is held up by its instructions too (760 of a warp for a token's 16 rows,
// 53 % of the issue slots).  32640 tokens x 8 heads of 128, 1/20 of them padding, bf16: into E4M3 39 us, 4.9 TB/s, 72 %
// of a copy's rate; back 32 us, 6.2 TB/s, 92 %; in bf16 40 us in and 41 back, 6.3 and 6.4 TB/s.  By rows of any kind one
// after the other, each with its own places, E4M3 took 48 and 34 us; an element per access 168 and 112.
#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {
namespace {

constexpr int kThreads = 256;

// Any view: a warp has rows of a token one after the other, keys and then values of each head, an element per access;
// AHEAD rows of up to 32 NC columns are loaded before the first is computed (NC = 0: any row, read as often as it
// takes).  32640 tokens x 8 heads of 99, bf16, into E4M3 80 us, where a copy's rate gives
// 22, back 59; one row after the other 168 and 112 (of 128 columns).
constexpr int kColumnAhead = 4;

struct CacheRow {
  int which, head;  // 0: keys, 1: values
  int64_t page, place;
  bool inside;
  __device__ __forceinline__ void find(const CacheArgs& a, int64_t token) {
    const int64_t slot = id_at(a.slots, token, a.ids64);
    inside = slot >= 0 && slot < a.c.pages * a.c.page_size;
    page = inside ? (int64_t)((uint32_t)slot / (uint32_t)a.c.page_size) : 0;
    place = inside ? slot - page * a.c.page_size : 0;
  }
  __device__ __forceinline__ void row(int n) { which = n & 1, head = n >> 1; }
  // element and scale number in the cache
  __device__ __forceinline__ int64_t at(const dit_cache& c) const {
    return page * c.page_stride + ((int64_t)head * c.page_size + place) * c.D;
  }
  __device__ __forceinline__ int64_t scale_at(const dit_cache& c) const {
    return page * c.scale_stride + (int64_t)head * c.page_size + place;
  }
};

template <class T, int NC, bool FP8, bool WRITE>
__global__ void __launch_bounds__(kThreads) columns_kernel(const __grid_constant__ CacheArgs a) {
  using K = typename std::conditional<FP8, uint8_t, T>::type;
  const int lane = threadIdx.x & 31;
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  const int D = (int)a.c.D, rows = 2 * (int)a.c.heads;
  // a token's rows in parts: as many warps as it takes to have kColumnAhead rows each
  const int parts = (rows + kColumnAhead - 1) / kColumnAhead;
  const int64_t items = a.tokens * parts;
  after_previous();
  let_next();
  for (int64_t item = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); item < items; item += stride) {
    const int64_t token = items >> 32 ? item / parts : (uint32_t)item / (uint32_t)parts;
    const int first = (int)(item - token * parts) * kColumnAhead;
    CacheRow row;
    row.find(a, token);
    if (WRITE && !row.inside) continue;
    auto tokens = [&]() {
      const dit_heads& v = row.which ? a.v : a.k;
      return (T*)v.p + token * v.token + row.head * v.head;
    };
    auto cached = [&]() { return (K*)(row.which ? a.c.v : a.c.k) + row.at(a.c); };
    auto value = [&](K x) {
      if constexpr (FP8)
        return from_e4m3(x);
      else
        return to_float(x);
    };
    if constexpr (NC > 0) {
      using From = typename std::conditional<WRITE, T, K>::type;
      From raw[kColumnAhead][NC];
      float scale[kColumnAhead];
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k) {
        row.row(first + k);
        const From* x;
        if constexpr (WRITE)
          x = tokens();
        else
          x = cached();
        const bool on = first + k < rows && row.inside;
        if constexpr (FP8 && !WRITE) scale[k] = on ? (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)] : 0.0f;
#pragma unroll
        for (int i = 0; i < NC; ++i) {
          raw[k][i] = From();
          if (on && lane + 32 * i < D) raw[k][i] = x[lane + 32 * i];
        }
      }
#pragma unroll
      for (int k = 0; k < kColumnAhead; ++k) {
        row.row(first + k);
        if (first + k >= rows) break;
        if constexpr (WRITE) {
          K* out = cached();
          RowQuant q;
          if constexpr (FP8) {
            float m = 0.0f;
#pragma unroll
            for (int i = 0; i < NC; ++i) m = max_nan(m, fabsf(to_float(raw[k][i])));
            q = row_quant(lanes_max<32>(m));
            if (lane == 0) (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)] = q.scale;
          }
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            if (lane + 32 * i >= D) continue;
            if constexpr (FP8)
              out[lane + 32 * i] = (uint8_t)e4m3x2(f2(code_value(to_float(raw[k][i]), q), 0.0f));
            else
              out[lane + 32 * i] = raw[k][i];
          }
        } else {
          T* out = tokens();
#pragma unroll
          for (int i = 0; i < NC; ++i) {
            if (lane + 32 * i >= D) continue;
            if constexpr (FP8)
              out[lane + 32 * i] = from_float<T>(__fmul_rn(value(raw[k][i]), scale[k]));
            else
              out[lane + 32 * i] = row.inside ? raw[k][i] : from_float<T>(0.0f);
          }
        }
      }
    } else {
      for (int k = 0; k < kColumnAhead && first + k < rows; ++k) {
        row.row(first + k);
        T* x = tokens();
        K* kept = cached();
        if constexpr (WRITE && FP8) {
          float m = 0.0f;
          for (int c = lane; c < D; c += 32) m = max_nan(m, fabsf(to_float(x[c])));
          const RowQuant q = row_quant(lanes_max<32>(m));
          for (int c = lane; c < D; c += 32) kept[c] = (uint8_t)e4m3x2(f2(code_value(to_float(x[c]), q), 0.0f));
          if (lane == 0) (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)] = q.scale;
        } else if constexpr (WRITE) {
          for (int c = lane; c < D; c += 32) kept[c] = x[c];
        } else {
          const float scale = FP8 && row.inside ? (row.which ? a.c.v_scales : a.c.k_scales)[row.scale_at(a.c)] : 1.0f;
          for (int c = lane; c < D; c += 32)
            x[c] = row.inside ? from_float<T>(FP8 ? __fmul_rn(value(kept[c]), scale) : value(kept[c])) : from_float<T>(0.0f);
        }
      }
    }
  }
}

// Rows in 16-byte granules.  A team of TEAM lanes has a row, a lane granules l and l + TEAM of it.  `abreast` of a
// warp's teams (a power of two, at most the heads) have the heads of one token, the others the next tokens'; so a
// team finds its token's places once, and goes on from head to head, keys and values both (BOTH; else one of them,
// for few tokens: twice the warps).
struct CacheRows {
  CacheArgs a;
  Divisor page;        // page_size
  int abreast;
  int64_t items;       // of 32 / TEAM / abreast tokens
};
// A team's token: its rows of keys [0] and values [1] and their places in the cache (ES bytes an element there).
template <class T, int ES>
struct CacheToken {
  const char* row[2];
  char* cached[2];
  int64_t scale;
  bool on, inside;
  __device__ __forceinline__ CacheToken(const CacheRows& c, int64_t token, int head) {
    const CacheArgs& a = c.a;
    on = token < a.tokens;
    if (!on) token = 0;
    const int64_t slot = on ? id_at(a.slots, token, a.ids64) : -1;
    inside = slot >= 0 && slot < a.c.pages * a.c.page_size;
    const uint32_t page = inside ? quotient((uint32_t)slot, c.page) : 0;
    const uint32_t place = inside ? (uint32_t)slot - page * c.page.d : 0;
    const int64_t in_page = (int64_t)head * a.c.page_size + place;
    scale = page * a.c.scale_stride + in_page;
    const int64_t at = (page * a.c.page_stride + in_page * a.c.D) * ES;
    cached[0] = (char*)a.c.k + at;
    cached[1] = (char*)a.c.v + at;
    row[0] = (const char*)a.k.p + (token * a.k.token + head * a.k.head) * (int)sizeof(T);
    row[1] = (const char*)a.v.p + (token * a.v.token + head * a.v.head) * (int)sizeof(T);
  }
};
constexpr int kHeads = 2;  // heads of a lane at once, beside keys and values

template <class T, int TEAM, bool FP8, bool BOTH>
__global__ void __launch_bounds__(kThreads) write_rows_kernel(const __grid_constant__ CacheRows args) {
  constexpr int ES = (int)sizeof(T), PER = 16 / ES, P = PER / 2, TEAMS = 32 / TEAM;
  constexpr int CES = FP8 ? 1 : ES, N = BOTH ? 2 : 1;
  const CacheArgs& a = args.a;
  const int lane = threadIdx.x & 31, team = lane / TEAM, l = lane % TEAM, n = (int)a.c.D / PER;
  const int heads = (int)a.c.heads, abreast = args.abreast;
  const int64_t head_bytes = a.c.page_size * a.c.D * CES * abreast;
  const int64_t step[2] = {a.k.head * ES * abreast, a.v.head * ES * abreast};
  after_previous();
  let_next();
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < args.items; i += stride) {
    const int64_t group = BOTH ? i : i >> 1;
    const int only = BOTH ? 0 : (int)(i & 1);
    int head = team & (abreast - 1);
    CacheToken<T, CES> t(args, group * (TEAMS / abreast) + team / abreast, head);
    for (int h0 = 0; h0 < heads; h0 += kHeads * abreast) {
      Raw<16> raw[kHeads][N][2];
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int w = 0; w < N; ++w) {
          const int which = BOTH ? w : only;
          const char* x = (which ? t.row[1] : t.row[0]) + h * step[which];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            raw[h][w][j] = Raw<16>{};
            if (t.inside && head + h * abreast < heads && l + j * TEAM < n) raw[h][w][j] = ld_stream<16>(x + (l + j * TEAM) * 16);
          }
        }
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int w = 0; w < N; ++w) {
          const int which = BOTH ? w : only;
          char* out = (which ? t.cached[1] : t.cached[0]) + h * head_bytes;
          const bool on = t.inside && head + h * abreast < heads;
          if constexpr (FP8) {
            F2 x[2][P];
            float m = 0.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              Granule<T>::widen(raw[h][w][j], x[j]);
#pragma unroll
              for (int e = 0; e < P; ++e) m = max_abs3(m, x[j][e].x, x[j][e].y);
            }
            const RowQuant q = row_quant(lanes_max<TEAM>(m));
            if (!on) continue;
            const bool plain = q.by == 1.0f;
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              Raw<PER> codes;
#pragma unroll
              for (int e = 0; e < P / 2; ++e) {
                F2 v[2];
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                  F2 y = x[j][2 * e + k];
                  if (!plain) y = f2_mul(y, f2(q.by, q.by));
                  v[k] = f2_fma(y, f2(q.mul, q.mul), f2_mul(y, f2(q.low, q.low)));
                }
                codes.w[e] = e4m3x2(v[0]) | e4m3x2(v[1]) << 16;
              }
              if (l + j * TEAM < n) st_stream<PER>(out + (l + j * TEAM) * PER, codes);
            }
            if (l == 0) (which ? a.c.v_scales : a.c.k_scales)[t.scale + (int64_t)h * a.c.page_size * abreast] = q.scale;
          } else if (on) {
#pragma unroll
            for (int j = 0; j < 2; ++j)
              if (l + j * TEAM < n) st_stream<16>(out + (l + j * TEAM) * 16, raw[h][w][j]);
          }
        }
      head += kHeads * abreast;
      t.scale += kHeads * a.c.page_size * abreast;
#pragma unroll
      for (int w = 0; w < 2; ++w) t.row[w] += kHeads * step[w], t.cached[w] += kHeads * head_bytes;
    }
  }
}

template <class T, int TEAM, bool FP8, bool BOTH>
__global__ void __launch_bounds__(kThreads) read_rows_kernel(const __grid_constant__ CacheRows args) {
  constexpr int ES = (int)sizeof(T), PER = 16 / ES, P = PER / 2, TEAMS = 32 / TEAM;
  constexpr int CES = FP8 ? 1 : ES, CB = FP8 ? PER : 16, N = BOTH ? 2 : 1;  // CB: bytes of a granule's columns in the cache
  const CacheArgs& a = args.a;
  const int lane = threadIdx.x & 31, team = lane / TEAM, l = lane % TEAM, n = (int)a.c.D / PER;
  const int heads = (int)a.c.heads, abreast = args.abreast;
  const int64_t head_bytes = a.c.page_size * a.c.D * CES * abreast;
  const int64_t step[2] = {a.k.head * ES * abreast, a.v.head * ES * abreast};
  after_previous();
  let_next();
  const int64_t stride = (int64_t)gridDim.x * (kThreads / 32);
  for (int64_t i = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); i < args.items; i += stride) {
    const int64_t group = BOTH ? i : i >> 1;
    const int only = BOTH ? 0 : (int)(i & 1);
    int head = team & (abreast - 1);
    CacheToken<T, CES> t(args, group * (TEAMS / abreast) + team / abreast, head);
    for (int h0 = 0; h0 < heads; h0 += kHeads * abreast) {
      Raw<CB> raw[kHeads][N][2];
      float scale[kHeads][N];
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int w = 0; w < N; ++w) {
          const int which = BOTH ? w : only;
          const char* x = (which ? t.cached[1] : t.cached[0]) + h * head_bytes;
          const bool on = t.inside && head + h * abreast < heads;
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            raw[h][w][j] = Raw<CB>{};
            if (on && l + j * TEAM < n) raw[h][w][j] = ld_stream<CB>(x + (l + j * TEAM) * CB);
          }
          if constexpr (FP8)
            scale[h][w] = on ? (which ? a.c.v_scales : a.c.k_scales)[t.scale + (int64_t)h * a.c.page_size * abreast] : 0.0f;
        }
#pragma unroll
      for (int h = 0; h < kHeads; ++h)
#pragma unroll
        for (int w = 0; w < N; ++w) {
          const int which = BOTH ? w : only;
          if (!t.on || head + h * abreast >= heads) continue;
          char* out = (char*)(which ? t.row[1] : t.row[0]) + h * step[which];
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            Raw<16> y;
            if constexpr (FP8) {
              F2 x[P];
#pragma unroll
              for (int e = 0; e < P; ++e) {
                const float2 v = from_e4m3x2((uint16_t)(raw[h][w][j].w[e / 2] >> (16 * (e & 1))));
                x[e] = f2_mul(v, f2(scale[h][w], scale[h][w]));
              }
              y = Granule<T>::narrow(x);
            } else {
              y = raw[h][w][j];
            }
            if (l + j * TEAM < n) st_stream<16>(out + (l + j * TEAM) * 16, y);
          }
        }
      head += kHeads * abreast;
      t.scale += kHeads * a.c.page_size * abreast;
#pragma unroll
      for (int w = 0; w < 2; ++w) t.row[w] += kHeads * step[w], t.cached[w] += kHeads * head_bytes;
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
  const int64_t half = (a.c.D * (int)sizeof(T) / 16 + 1) / 2;  // granules of a lane's pair
  if (!a.granules || half > 32) {
    const auto columns = a.c.D <= 64    ? (write ? columns_kernel<T, 2, FP8, true> : columns_kernel<T, 2, FP8, false>)
                         : a.c.D <= 128 ? (write ? columns_kernel<T, 4, FP8, true> : columns_kernel<T, 4, FP8, false>)
                         : a.c.D <= 256 ? (write ? columns_kernel<T, 8, FP8, true> : columns_kernel<T, 8, FP8, false>)
                                        : (write ? columns_kernel<T, 0, FP8, true> : columns_kernel<T, 0, FP8, false>);
    return launch(dev, columns, a.tokens * ((2 * a.c.heads + kColumnAhead - 1) / kColumnAhead), a, s);
  }
  CacheRows c{a, divisor((uint32_t)a.c.page_size), 1, 0};
  auto team = [&](auto lanes) {
    constexpr int TEAM = decltype(lanes)::value, TEAMS = 32 / TEAM;
    while (c.abreast * 2 <= std::min<int64_t>(TEAMS, a.c.heads)) c.abreast *= 2;
    const int64_t tokens = TEAMS / c.abreast;
    c.items = (a.tokens + tokens - 1) / tokens;
    const bool both = c.items >= (int64_t)dev.sm_count * 16;
    if (!both) c.items *= 2;
    const auto kern = write ? (both ? write_rows_kernel<T, TEAM, FP8, true> : write_rows_kernel<T, TEAM, FP8, false>)
                            : (both ? read_rows_kernel<T, TEAM, FP8, true> : read_rows_kernel<T, TEAM, FP8, false>);
    return launch(dev, kern, c.items, c, s);
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
