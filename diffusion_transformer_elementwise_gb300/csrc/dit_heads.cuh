// dit_heads.cuh -- device helpers shared by the operators around attention.
#pragma once

#include <algorithm>

#include "dit_attend.h"
#include "dit_device.cuh"
#include "dit_unit.cuh"

namespace dit {

__device__ __forceinline__ void cp_async8_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ Raw<8> lds8(uint32_t at) {
  Raw<8> r;
  asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(r.w[0]), "=r"(r.w[1]) : "r"(at));
  return r;
}

__device__ __forceinline__ float to_float(__nv_bfloat16 v) { return __bfloat162float(v); }
__device__ __forceinline__ float to_float(__half v) { return __half2float(v); }
__device__ __forceinline__ float to_float(float v) { return v; }
template <class T>
__device__ __forceinline__ T from_float(float v);
template <>
__device__ __forceinline__ __nv_bfloat16 from_float(float v) { return __float2bfloat16_rn(v); }
template <>
__device__ __forceinline__ __half from_float(float v) { return __float2half_rn(v); }
template <>
__device__ __forceinline__ float from_float(float v) { return v; }

// q = t / d for 0 <= t < 2^31: t m / 2^(31 + s) with 2^(s - 1) < d <= 2^s, m = ceil(2^(31 + s) / d): m d exceeds
// 2^(31 + s) by less than 2^s, which moves the quotient by less than 1 / d.
struct Divisor {
  uint32_t d, m, s;
};
__device__ __forceinline__ uint32_t quotient(uint32_t t, const Divisor& v) {
  return (uint32_t)(((uint64_t)t * v.m) >> (31 + v.s));
}
inline Divisor divisor(uint32_t d) {
  Divisor v{d, 0, 0};
  while ((uint64_t(1) << v.s) < d) ++v.s;
  v.m = (uint32_t)(((uint64_t(1) << (31 + v.s)) + d - 1) / d);
  return v;
}

// The sum over the N lanes of an aligned group, in every one of them.
template <int N>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
// The largest magnitude of N lanes' v (not negative), NaN if any is.
template <int N>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
  for (int o = N / 2; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// r of a head's norm from its sum of squares (inv_d: fl(1 / D)).  The root halves the two roundings before it (2 u, u =
// 2^-24), and rsqrtf's own error was at most 2.1 u over all numbers of two binades: 3.1 u together.  A Newton step
// would leave 2.5 u; it costs the kernels for any alignment 3 to 4 % (8160 x 64 heads of 99: 95.6 us with the root alone, 99.6).
__device__ __forceinline__ float inverse_rms(float sum, float inv_d, float eps) {
  return rsqrtf(__fmaf_rn(sum, inv_d, eps));
}

// The pair (a, b) turned: one product rounded, the other one with the sum.
__device__ __forceinline__ float2 turned(float a, float b, float cos, float sin) {
  return make_float2(__fmaf_rn(a, cos, __fmul_rn(b, -sin)), __fmaf_rn(b, cos, __fmul_rn(a, sin)));
}

// Head number i of all tokens' heads (the queries' before the keys').
struct HeadRow {
  int tensor, head;
  int64_t batch, place, table;  // table: its row of cos and sin
  __device__ __forceinline__ HeadRow(const RopeArgs& a, int64_t i, int heads) {
    const int64_t token = i / heads;
    head = (int)(i - token * heads);
    tensor = head >= a.t[0].H;
    if (tensor) head -= a.t[0].H;
    batch = token / a.L;
    place = token - batch * a.L;
    table = a.table_rows == a.L ? place : token;
  }
  __device__ __forceinline__ int64_t at(const dit_heads& t) const {
    return batch * t.batch + place * t.token + head * t.head;
  }
};

// ---------------------------------------------------------------------------
// heads in 16-byte granules
//
// A team of TEAM lanes (a power of two) has a head; a lane has two granules of
// it: those whose columns are turned together (j and j + R), two neighbouring pairs' ones
// where the pairs are adjacent columns, or two that are not turned.  So the partners of every
// rotation are in one lane, and a team's accesses are contiguous.  A warp takes a token, its
// teams the token's heads one beside the other, so that the angles (and the weights) are
// loaded once for several heads.
// ---------------------------------------------------------------------------

// units of a head: lanes that its granules take
inline int head_units(const RopeArgs& a, int per) {
  const int n = a.D / per, turned = a.interleaved ? 0 : a.R / per;
  return turned + (n - 2 * turned + 1) / 2;
}
// whether heads of T can be cut so: whole granules, each turned wholly or not at all
template <class T>
bool head_granules(const RopeArgs& a) {
  constexpr int per = 16 / (int)sizeof(T);
  return a.granules && (a.interleaved ? 2 * a.R : a.R) % per == 0 && head_units(a, per) <= 32 && a.D > 0;
}

template <class T>
struct HeadLane {
  static constexpr int PER = 16 / (int)sizeof(T);  // columns of a granule
  static constexpr int P = PER / 2;                // pairs of fp32
  int column[2];
  bool on[2], turn[2];
  __device__ __forceinline__ HeadLane(const RopeArgs& a, int unit) {
    const int n = a.D / PER;
    if (a.interleaved) {
      const int half = (n + 1) / 2;
      column[0] = unit * PER;
      column[1] = (unit + half) * PER;
      on[0] = unit < half;
      on[1] = unit + half < n && on[0];
      turn[0] = column[0] < 2 * a.R;
      turn[1] = column[1] < 2 * a.R;
    } else {
      const int t = a.R / PER;
      const bool pair = unit < t;
      column[0] = (pair ? unit : 2 * unit) * PER;  // (2 t + 2 (unit - t))
      column[1] = pair ? (unit + t) * PER : column[0] + PER;
      on[0] = column[0] < a.D;
      on[1] = column[1] < a.D;
      turn[0] = turn[1] = pair;
    }
  }
};

// The copies of one item of work, a token's next HEADS heads of each team: for each lane its granules of NT tensors,
// each to a place of its own in shared memory that no other lane reads, and the angles, which the teams
// copy a share of each.
template <class T, int TEAM, bool INTER, int NT>
struct HeadStage {
  using Lane = HeadLane<T>;
  static constexpr int TEAMS = 32 / TEAM;
  static constexpr int HEADS = 2;
  static constexpr int GRANULES = HEADS * NT * 2;
  // angles: cosines and sines of PER columns (both granules'), or of PER / 2 pairs for each granule
  static constexpr int AB = INTER && sizeof(T) == 4 ? 8 : 16;  // bytes of a piece
  static constexpr int AN = INTER ? 2 : Lane::PER * 4 / 16;    // pieces of cosines
  static constexpr int BYTES = 32 * GRANULES * 16 + TEAM * 2 * AN * AB;

  __device__ __forceinline__ static uint32_t granule(uint32_t stage, int lane, int tensor, int head, int j) {
    return stage + (((tensor * HEADS + head) * 2 + j) * 32 + lane) * 16;
  }
  __device__ __forceinline__ static uint32_t angle(uint32_t stage, int lane, int i) {
    return stage + GRANULES * 512 + (i * TEAM + lane % TEAM) * AB;
  }
  // tensor[at + head k stride]: heads [first, last)
  __device__ __forceinline__ static void copy_heads(uint32_t stage, int lane, const Lane& h, int tensor, const void* p,
                                                    int64_t at, int64_t stride, int first, int last) {
    const T* src = (const T*)p + at + first * stride;
#pragma unroll
    for (int k = 0; k < HEADS; ++k) {
      const bool on = first + k * TEAMS < last;
#pragma unroll
      for (int j = 0; j < 2; ++j) {
        const bool any = on && h.on[j];
        cp_async16_part(granule(stage, lane, tensor, k, j), any ? src + h.column[j] : (const T*)p, any ? 16 : 0);
      }
      src += TEAMS * stride;
    }
  }
  __device__ __forceinline__ static void copy_angles(uint32_t stage, int lane, const Lane& h, const RopeArgs& a,
                                                     int64_t row) {
    if (a.R == 0) return;
#pragma unroll
    for (int n = 0; n < 2 * AN; n += TEAMS) {
      const int i = n + lane / TEAM;  // the team's piece
      if (TEAMS > 2 * AN && i >= 2 * AN) break;
      const int k = INTER ? i % AN : 0;
      const bool any = k ? h.on[1] && h.turn[1] : h.on[0] && h.turn[0];
      const int column = k ? h.column[1] : h.column[0];
      const float* from = (i < AN ? a.cos : a.sin) + (any ? row * a.R + (INTER ? column / 2 : column + i % AN * 4) : 0);
      if constexpr (AB == 16)
        cp_async16_part(angle(stage, lane, i), from, any ? 16 : 0);
      else
        cp_async8_part(angle(stage, lane, i), from, any ? 8 : 0);
    }
  }
};

// The angles of a lane's columns: cosines and sines of PER columns, or of the pairs of both granules.
template <class T, int TEAM, bool INTER, int NT>
struct LaneAngles {
  using Stage = HeadStage<T, TEAM, INTER, NT>;
  static constexpr int P = HeadLane<T>::P, N = 2 * P;
  float c[N], s[N];
  __device__ __forceinline__ void load(uint32_t stage, int lane, bool inverse) {
    constexpr int F = Stage::AB / 4;
#pragma unroll
    for (int i = 0; i < Stage::AN; ++i) {
      if constexpr (F == 4) {
        const Raw<16> x = lds16(Stage::angle(stage, lane, i)), y = lds16(Stage::angle(stage, lane, Stage::AN + i));
#pragma unroll
        for (int k = 0; k < 4; ++k) c[4 * i + k] = __uint_as_float(x.w[k]), s[4 * i + k] = __uint_as_float(y.w[k]);
      } else {
        const Raw<8> x = lds8(Stage::angle(stage, lane, i)), y = lds8(Stage::angle(stage, lane, Stage::AN + i));
#pragma unroll
        for (int k = 0; k < 2; ++k) c[2 * i + k] = __uint_as_float(x.w[k]), s[2 * i + k] = __uint_as_float(y.w[k]);
      }
    }
    if (inverse) {
#pragma unroll
      for (int i = 0; i < N; ++i) s[i] = -s[i];
    }
  }
  // ALL: every column of a head is turned
  template <bool ALL>
  __device__ __forceinline__ void turn(F2 (&x)[2][P], const HeadLane<T>& h) const {
    if constexpr (INTER) {
#pragma unroll
      for (int j = 0; j < 2; ++j)
#pragma unroll
        for (int i = 0; i < P; ++i) {
          const F2 y = turned(x[j][i].x, x[j][i].y, c[j * P + i], s[j * P + i]);
          if (ALL || h.turn[j]) x[j][i] = y;
        }
    } else {
#pragma unroll
      for (int i = 0; i < P; ++i) {
        const F2 y = turned(x[0][i].x, x[1][i].x, c[2 * i], s[2 * i]), z = turned(x[0][i].y, x[1][i].y, c[2 * i + 1], s[2 * i + 1]);
        if (ALL || h.turn[0]) x[0][i] = f2(y.x, z.x), x[1][i] = f2(y.y, z.y);
      }
    }
  }
};

template <class T>
__device__ __forceinline__ void head_weight(F2 (&w)[2][HeadLane<T>::P], const HeadLane<T>& h, const void* p, float offset) {
#pragma unroll
  for (int k = 0; k < 2; ++k) {
    Raw<16> r = {};
    // (not by the read-only path: the call before, which may have written them, can have run beside this kernel)
    if (h.on[k]) r = ld_stream<16>((const T*)p + h.column[k]);
    Granule<T>::widen(r, w[k]);
#pragma unroll
    for (int i = 0; i < HeadLane<T>::P; ++i) w[k][i] = f2_add(f2(offset, offset), w[k][i]);
  }
}

// How the items of a call are given to warps: CTAs [0, ctas[0]) have the queries', the others the keys'; a
// tensor's warps take its items in turn.  A token has per[i] items.
struct HeadGrid {
  int ctas[2], per[2], together;  // together: heads of an item
};
// most: CTAs
inline HeadGrid head_grid(const RopeArgs& a, int together, int warps, int64_t most) {
  HeadGrid g = {};
  g.together = together;
  double items[2];
  for (int i = 0; i < 2; ++i) {
    g.per[i] = (a.t[i].H + together - 1) / together;
    items[i] = (double)g.per[i] * (double)a.tokens;
  }
  for (int i = 0; i < 2; ++i) {
    if (items[i] == 0) continue;
    const double share = items[1 - i] == 0 ? (double)most : std::max(1.0, (double)(most - 1) * items[i] / (items[0] + items[1]));
    g.ctas[i] = (int)std::min(share, (items[i] + warps - 1) / warps);
  }
  return g;
}

// Heads of an item of the kernels for any alignment: `many`, which share a token's angles, unless that leaves
// less than eight warps an SM (126 tokens x 8 heads of 80, gradient: 6.5 us with eight, 4.7 with two).
inline int column_heads(const DeviceInfo& dev, const RopeArgs& a, int many, int few) {
  const int64_t items = a.tokens * ((a.t[0].H + many - 1) / many + (a.t[1].H + many - 1) / many);
  return items >= (int64_t)dev.sm_count * 8 ? many : few;
}

// A warp's walk over its items.
struct HeadWalk {
  int64_t token, step;
  int part, per, rest;
  __device__ __forceinline__ HeadWalk(const HeadGrid& g, int which, int64_t warp, int64_t warps)
      : per(g.per[which]) {
    token = warp / per;
    part = (int)(warp - token * per);
    step = warps / per;
    rest = (int)(warps - step * per);
  }
  __device__ __forceinline__ void next() {
    token += step;
    part += rest;
    if (part >= per) part -= per, ++token;
  }
};

// ---------------------------------------------------------------------------
// heads of any alignment
//
// A warp has a head, a lane its columns lane + 32 i.  What a column is turned with lies in another lane: the
// warp passes the head's columns through its row in shared memory.
// ---------------------------------------------------------------------------
template <int NC>
struct LaneColumns {
  int partner[NC], angle[NC];  // the column turned with this one, and the angle's number (-1: not turned)
  bool second[NC];             // the pair's second column
  __device__ __forceinline__ LaneColumns(const RopeArgs& a, int lane) {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      const int c = lane + 32 * i;
      const bool turn = c < 2 * a.R;
      second[i] = a.interleaved ? c & 1 : c >= a.R;
      partner[i] = !turn ? c : a.interleaved ? c ^ 1 : second[i] ? c - a.R : c + a.R;
      angle[i] = !turn ? -1 : a.interleaved ? c >> 1 : second[i] ? c - a.R : c;
    }
  }
  // cosines, and sines with the partner's sign
  __device__ __forceinline__ void load(const RopeArgs& a, int64_t row, bool inverse, float (&c)[NC], float (&s)[NC]) const {
#pragma unroll
    for (int i = 0; i < NC; ++i) {
      c[i] = 1.0f, s[i] = 0.0f;
      if (angle[i] < 0) continue;
      c[i] = a.cos[row * a.R + angle[i]];
      s[i] = a.sin[row * a.R + angle[i]];
      if (second[i] == inverse) s[i] = -s[i];
    }
  }
};

// A token's batch, place and row of angles (tokens < 2^31).
struct TokenAt {
  int64_t batch, place, table;
  __device__ __forceinline__ TokenAt(const RopeArgs& a, uint32_t token) {
    if (a.tokens == a.L) {
      batch = 0;
      place = token;
    } else {
      const uint32_t b = token / (uint32_t)a.L;
      batch = b;
      place = token - b * (uint32_t)a.L;
    }
    table = a.table_rows == a.L ? place : token;
  }
};

// Scale and factors to codes of a row whose largest magnitude is m: scale = fl(m / 448), and codes of x are
// e4m3(fl(x (mul + low))), 448 / m as two fp32 numbers: an approximate reciprocal and what it leaves of 448.  Rows
// so small or large that such steps would leave fp32 are scaled first (by `by`).  m not finite: all NaN.
struct RowQuant {
  float mul, low, by, scale;
};
__device__ __forceinline__ RowQuant row_quant(float m) {
  constexpr float most = 448.0f;
  RowQuant q;
  const bool usable = m >= 0x1p-100f && m <= 0x1p100f;
  q.by = usable ? 1.0f : m < 1.0f ? 0x1p64f : 0x1p-64f;
  const float v = __fmul_rn(m, q.by);
  float y;
  asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(m == 0.0f ? 1.0f : v));
  q.mul = m == 0.0f ? 0.0f : __fmul_rn(most, y);
  q.low = m == 0.0f ? 0.0f : __fmul_rn(__fmaf_rn(-q.mul, v, most), y);
  if (usable) {  // the quotient by a rounded reciprocal, corrected by its remainder
    const float part = __fmul_rn(m, 1.0f / most);
    q.scale = __fmaf_rn(__fmaf_rn(-part, most, m), 1.0f / most, part);
  } else {
    q.scale = __fdiv_rn(m, most);
  }
  if (!isfinite(m)) q.mul = q.low = q.scale = __int_as_float(0x7FC00000);
  return q;
}
__device__ __forceinline__ float code_value(float x, const RowQuant& q) {
  const float v = __fmul_rn(x, q.by);
  return __fmaf_rn(v, q.mul, __fmul_rn(v, q.low));
}

// E4M3 code -> fp32
__device__ __forceinline__ float2 from_e4m3x2(uint16_t codes) {
  uint32_t h;
  asm("cvt.rn.f16x2.e4m3x2 %0, %1;" : "=r"(h) : "h"(codes));
  return __half22float2(*reinterpret_cast<const __half2*>(&h));
}
__device__ __forceinline__ float from_e4m3(uint8_t code) { return from_e4m3x2(code).x; }

// Entry i of an int32 or int64 array.
__device__ __forceinline__ int64_t id_at(const void* ids, int64_t i, bool wide) {
  return wide ? ((const int64_t*)ids)[i] : ((const int32_t*)ids)[i];
}

}  // namespace dit
