// dit_unit.cuh -- rows cut into units of one warp (sm_103a): the loads,
// stores and reductions shared by the weighted-norm kernels.
//
// A unit is 512 bytes of a row: 256 columns of a 16-bit type or 128 of fp32,
// 16 bytes per lane.  In a wide unit lane l holds the 16-byte granule l, so an
// access of the warp is 512 contiguous bytes.  Rows that are not made of
// 16-byte granules (an odd width, or a tensor that starts off a 16-byte
// boundary) take narrow units: lane l's element i is column 32 i + l, one
// element per access, 64 or 128 contiguous bytes of the warp.  Both keep a
// lane's elements packed in a Raw<16>, so the arithmetic does not see the
// difference.  Columns past the row read as zero and are not stored.
#pragma once

#include "dit_device.cuh"
#include "dit_internal.h"
#include "dit_pipe.cuh"

namespace dit {

// the larger of two values, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

template <class T, bool WIDE>
struct Unit {
  static constexpr int ES = (int)sizeof(T);
  static constexpr int EPL = 16 / ES;       // elements per lane
  static constexpr int COLS = 32 * EPL;     // columns of a unit
  static constexpr int P = Granule<T>::P;   // fp32 pairs per lane

  // the column of a lane's element i in the unit that starts at column c0
  __device__ __forceinline__ static int col(int c0, int lane, int i) {
    return WIDE ? c0 + lane * EPL + i : c0 + i * 32 + lane;
  }
  template <bool STREAM>
  __device__ __forceinline__ static Raw<16> load_as(const void* row, int c0, int D, int lane) {
    Raw<16> r = {};
    if constexpr (WIDE) {
      if (col(c0, lane, 0) < D) {
        const char* p = (const char*)row + (int64_t)col(c0, lane, 0) * ES;
        r = STREAM ? ld_stream<16>(p) : ld_bcast<16>(p);
      }
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int c = col(c0, lane, i);
        if (c >= D) continue;
        const char* p = (const char*)row + (int64_t)c * ES;
        const Raw<ES> e = STREAM ? ld_stream<ES>(p) : ld_bcast<ES>(p);
        if constexpr (ES == 4)
          r.w[i] = e.w[0];
        else
          r.w[i >> 1] |= (uint32_t)e.h << (16 * (i & 1));
      }
    }
    return r;
  }
  // activations, read once
  __device__ __forceinline__ static Raw<16> load(const void* row, int c0, int D, int lane) {
    return load_as<true>(row, c0, D, lane);
  }
  // weights, re-read by every row
  __device__ __forceinline__ static Raw<16> load_weight(const void* w, int c0, int D, int lane) {
    return load_as<false>(w, c0, D, lane);
  }
  __device__ __forceinline__ static void store(void* row, int c0, int D, int lane, const Raw<16>& r) {
    if constexpr (WIDE) {
      if (col(c0, lane, 0) < D) st_stream<16>((char*)row + (int64_t)col(c0, lane, 0) * ES, r);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int c = col(c0, lane, i);
        if (c >= D) continue;
        Raw<ES> e;
        if constexpr (ES == 4)
          e.w[0] = r.w[i];
        else
          e.h = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
        st_stream<ES>((char*)row + (int64_t)c * ES, e);
      }
    }
  }
  // one byte per element, element i in byte i of q
  __device__ __forceinline__ static void store8(void* row, int c0, int D, int lane,
                                                const Raw<EPL>& q) {
    if constexpr (WIDE) {
      if (col(c0, lane, 0) < D) st_stream<EPL>((char*)row + col(c0, lane, 0), q);
    } else {
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int c = col(c0, lane, i);
        if (c < D) ((uint8_t*)row)[c] = (uint8_t)(q.w[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
};

// ---------------------------------------------------------------------------
// the warps of one row
// ---------------------------------------------------------------------------

// A team of `warps` warps holds a row; a CTA holds blockDim.x / 32 / warps
// teams.  sum2 and max1 combine a value of every warp over the team: through
// shared memory and one barrier of the team's threads (a named barrier; none
// for a team of one warp).  The slots alternate, so a slot is rewritten only
// behind the next call's barrier, which the team's other warps reach after
// reading it.
struct Team {
  float2* slots;  // this team's [2][warps]
  int warps, m, id;
  int par;
  __device__ __forceinline__ void barrier() const {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
  }
  // both members of v over the team, in the warps' order: sums (MAX: .y the
  // maximum)
  template <bool MAX>
  __device__ __forceinline__ float2 combine(float2 v) {
    if (warps == 1) return v;
    float2* s = slots + par * warps;
    par ^= 1;
    if ((threadIdx.x & 31) == 0) s[m] = v;
    barrier();
    float2 t = s[0];
    for (int w = 1; w < warps; ++w) {
      const float2 o = s[w];
      t.x = __fadd_rn(t.x, o.x);
      t.y = MAX ? max_nan(t.y, o.y) : __fadd_rn(t.y, o.y);
    }
    return t;
  }
};

// The most warps of a team's CTA: a row of up to 4 units a warp (64 units,
// 32 KB) stays in registers at up to 128 of them a thread.
constexpr int kTeamWarps = 16;
constexpr int kTeamThreads = 32 * kTeamWarps;

// Shape of the teams for rows of `units` units with up to `nu` units a warp:
// warps per row, and teams per CTA of at least eight warps.
struct TeamShape {
  int warps, teams;
};
inline TeamShape team_shape(int64_t units, int nu) {
  TeamShape t;
  t.warps = (int)((units + nu - 1) / nu);
  t.teams = t.warps >= 8 ? 1 : 8 / t.warps;
  return t;
}

}  // namespace dit
