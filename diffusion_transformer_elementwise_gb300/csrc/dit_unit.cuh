// dit_unit.cuh -- rows cut into units of one warp (sm_103a): the loads,
// stores and reductions shared by the weighted-norm kernels.
//
// A unit is 512 bytes of a row: 256 columns of a 16-bit type or 128 of fp32,
// 16 bytes per lane, kept packed in a Raw<16>.  Three layouts:
//   WIDE     the rows are made of 16-byte granules.  Lane l holds granule l of
//            the unit; a warp's access is 512 contiguous bytes.
//   PHASED   the tensors start on 16-byte boundaries but the rows do not (an odd
//            width).  Lanes hold the granules of the tensor, not of the row: row
//            r starts `off` elements into its first granule, so that
//            granule's first elements, and its last granule's last ones,
//            belong to the neighbours: they read as zero and are not stored.
//            Rows whose numbers differ by a multiple of EPL (elements per
//            granule) have the same `off`, so a team that takes such rows loads
//            its weights, at that offset, once.
//   NARROW   a tensor that starts off a 16-byte boundary.  Lane l's element i is
//            column 32 i + l, one element per access.
// The arithmetic is the same for all three.  Columns past the row read as
// zero and are not stored.
#pragma once

#include <atomic>

#include "dit_device.cuh"
#include "dit_internal.h"
#include "dit_pipe.cuh"
#include "dit_token.h"

namespace dit {

// the larger of two values, NaN if either is
__device__ __forceinline__ float max_nan(float a, float b) {
  float r;
  asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
  return r;
}
// the larger magnitude of a, b and c (NaN if any is)
__device__ __forceinline__ float max_abs3(float a, float b, float c) {
  float r;
  asm("max.NaN.abs.f32 %0, %1, %2, %3;" : "=f"(r) : "f"(a), "f"(b), "f"(c));
  return r;
}
__device__ __forceinline__ float warp_max(float v) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v = max_nan(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

template <class T, int LAYOUT>
struct Unit {
  static constexpr int ES = (int)sizeof(T);
  static constexpr int EPL = 16 / ES;       // elements per lane
  static constexpr int COLS = 32 * EPL;     // columns of a unit
  static constexpr int P = Granule<T>::P;   // fp32 pairs per lane

  int D, lane;
  int off;    // PHASED: the row's offset from a granule's start, elements
  bool last;  // PHASED: the tensors' last row: nothing past its end is read

  __device__ __forceinline__ Unit(int D, int lane) : D(D), lane(lane), off(0), last(false) {}
  __device__ __forceinline__ void at_row(int64_t row, int64_t rows) {
    if constexpr (LAYOUT == PHASED) {
      off = (int)(((uint64_t)row * (uint64_t)(D % EPL)) % EPL);
      last = row == rows - 1;
    }
  }
  // the column of this lane's element i in the unit that starts at column c0
  // (PHASED: negative in a first granule shared with the row before)
  __device__ __forceinline__ int col(int c0, int i) const {
    return LAYOUT == NARROW ? c0 + i * 32 + lane : c0 + lane * EPL + i - off;
  }
  // whether all of a lane's columns are the row's
  __device__ __forceinline__ bool whole(int c) const { return c >= 0 && c + EPL <= D; }
  __device__ __forceinline__ static void put(Raw<16>& r, int i, const Raw<ES>& e) {
    if constexpr (ES == 4)
      r.w[i] = e.w[0];
    else
      r.w[i >> 1] |= (uint32_t)e.h << (16 * (i & 1));
  }
  __device__ __forceinline__ static Raw<ES> get(const Raw<16>& r, int i) {
    Raw<ES> e;
    if constexpr (ES == 4)
      e.w[0] = r.w[i];
    else
      e.h = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
    return e;
  }
  template <bool STREAM>
  __device__ __forceinline__ Raw<16> elements(const void* row, int c0) const {
    Raw<16> r = {};
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      const int c = col(c0, i);
      if (c < 0 || c >= D) continue;
      const char* p = (const char*)row + (int64_t)c * ES;
      put(r, i, STREAM ? ld_stream<ES>(p) : ld_bcast<ES>(p));
    }
    return r;
  }
  // copy this lane's granule of row `row` of a tensor to its slot at shared
  // address dst (cp.async; not NARROW)
  __device__ __forceinline__ void copy(uint32_t dst, const void* tensor, int64_t row, int64_t rows,
                                       int c0) const {
    const int c = col(c0, 0);
    if (c >= D) return;
    const int64_t pitch = (int64_t)D * ES, at = row * pitch + (int64_t)c * ES;
    // PHASED: the tensor's last granule may run past its end
    if (LAYOUT == PHASED && row == rows - 1 && c + EPL > D)
      cp_async16_part(dst, (const char*)tensor + at, (uint32_t)((D - c) * ES));
    else
      cp_async16(dst, (const char*)tensor + at);
  }
  // what copy() left in the slot
  __device__ __forceinline__ Raw<16> copied(uint32_t src, int c0) const {
    Raw<16> r = {};
    const int c = col(c0, 0);
    if (c < D) {
      r = lds16(src);
      if (LAYOUT == PHASED && !whole(c)) mask(r, c);
    }
    return r;
  }
  // PHASED: zero the neighbours' elements of a granule that starts at column c
  __device__ __forceinline__ void mask(Raw<16>& r, int c) const {
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (c + i >= 0 && c + i < D) continue;
      if constexpr (ES == 4)
        r.w[i] = 0;
      else
        r.w[i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
    }
  }
  // activations, read once
  __device__ __forceinline__ Raw<16> load(const void* row, int c0) const {
    if constexpr (LAYOUT == NARROW) {
      return elements<true>(row, c0);
    } else {
      Raw<16> r = {};
      const int c = col(c0, 0);
      if (c < D) {
        const char* p = (const char*)row + (int64_t)c * ES;
        if (LAYOUT == WIDE || whole(c)) {
          r = ld_stream<16>(p);
        } else if (last && c + EPL > D) {
          r = elements<true>(row, c0);
        } else {
          r = ld_stream<16>(p);
          mask(r, c);
        }
      }
      return r;
    }
  }
  // weights, read by every row
  __device__ __forceinline__ Raw<16> load_weight(const void* w, int c0) const {
    if constexpr (LAYOUT != WIDE) {
      return elements<false>(w, c0);
    } else {
      Raw<16> r = {};
      if (col(c0, 0) < D) r = ld_bcast<16>((const char*)w + (int64_t)col(c0, 0) * ES);
      return r;
    }
  }
  __device__ __forceinline__ void store(void* row, int c0, const Raw<16>& r) const {
    const int c = col(c0, 0);
    if constexpr (LAYOUT == WIDE) {
      if (c < D) st_stream<16>((char*)row + (int64_t)c * ES, r);
    } else {
      if (LAYOUT == PHASED && whole(c)) {
        st_stream<16>((char*)row + (int64_t)c * ES, r);
        return;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int k = col(c0, i);
        if (k >= 0 && k < D) st_stream<ES>((char*)row + (int64_t)k * ES, get(r, i));
      }
    }
  }
  // one byte per element, element i in byte i of q
  __device__ __forceinline__ void store8(void* row, int c0, const Raw<EPL>& q) const {
    const int c = col(c0, 0);
    if constexpr (LAYOUT == WIDE) {
      if (c < D) st_stream<EPL>((char*)row + c, q);
    } else {
      if (LAYOUT == PHASED && whole(c)) {
        st_stream<EPL>((char*)row + c, q);
        return;
      }
#pragma unroll
      for (int i = 0; i < EPL; ++i) {
        const int k = col(c0, i);
        if (k >= 0 && k < D) ((uint8_t*)row)[k] = (uint8_t)(q.w[i >> 2] >> (8 * (i & 3)));
      }
    }
  }
};

// ---------------------------------------------------------------------------
// the warps of one row
// ---------------------------------------------------------------------------

// A team of `warps` warps (at most 16) holds a row; a CTA is blockDim.y teams
// of blockDim.x threads.  combine adds (MAX: .y takes the larger of) a value of every warp
// over the team: through shared memory, one barrier of the team's threads (a
// named barrier; none for a team of one warp) and a butterfly.  The slots
// alternate, so a slot is rewritten only behind the next call's barrier,
// which the team's other warps reach after reading it.
struct Team {
  float2* slots;  // this team's [2][warps]
  int warps, m, lane, id;
  int par;
  // slots: [2][the CTA's warps]
  __device__ __forceinline__ explicit Team(float2* slots)
      : slots(slots + threadIdx.y * 2 * (blockDim.x >> 5)),
        warps(blockDim.x >> 5),
        m(threadIdx.x >> 5),
        lane(threadIdx.x & 31),
        id(1 + threadIdx.y),
        par(0) {}
  template <bool MAX>
  __device__ __forceinline__ float2 combine(float2 v) {
    if (warps == 1) return v;
    float2* s = slots + par * warps;
    par ^= 1;
    if (lane == 0) s[m] = v;
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(warps * 32) : "memory");
    auto join = [&](int o) {
      const float x = __shfl_xor_sync(0xFFFFFFFFu, v.x, o), y = __shfl_xor_sync(0xFFFFFFFFu, v.y, o);
      v.x = __fadd_rn(v.x, x);
      v.y = MAX ? max_nan(v.y, y) : __fadd_rn(v.y, y);
    };
    const int k = lane & (warps <= 4 ? 3 : warps <= 8 ? 7 : 15);
    v = make_float2(0.0f, 0.0f);
    if (k < warps) v = s[k];
    join(1);
    join(2);
    if (warps > 4) join(4);
    if (warps > 8) join(8);
    return v;
  }
};

// The most warps of a team's CTA: a row of up to 4 units a warp (64 units,
// 32 KB) stays in registers at up to 128 of them a thread.
constexpr int kTeamWarps = 16;
constexpr int kTeamThreads = 32 * kTeamWarps;

// Lets kernel `fn` take all the shared memory its static arrays leave, once per
// (kernel, device).  `opted`: the kernel's flags.
inline cudaError_t allow_shared(const void* fn, const DeviceInfo& dev, std::atomic<int>* opted) {
  const bool cached = dev.device >= 0 && dev.device < kOptinDevices;
  if (cached && opted[dev.device].load(std::memory_order_acquire)) return cudaSuccess;
  cudaFuncAttributes at;
  cudaError_t e = cudaFuncGetAttributes(&at, fn);
  if (e == cudaSuccess)
    e = cudaFuncSetAttribute(fn, cudaFuncAttributeMaxDynamicSharedMemorySize,
                             dev.smem_optin - (int)at.sharedSizeBytes);
  if (e != cudaSuccess) {
    (void)cudaGetLastError();  // do not leave it for the next call to report
    return e;
  }
  if (cached) opted[dev.device].store(1, std::memory_order_release);
  return cudaSuccess;
}

// Units of a row of D columns (PHASED: at most, over the rows' offsets).
template <class T, int LAYOUT>
int64_t row_units(int64_t D) {
  using U = Unit<T, LAYOUT>;
  return (D + (LAYOUT == PHASED ? U::EPL - 1 : 0) + U::COLS - 1) / U::COLS;
}

// The weight, offset added, in shared memory as fp32 for rows at `unit`'s
// offset: plane q of granule g (of ngr) holds columns 4q .. 4q + 3 of it, so a
// warp reads 512 contiguous bytes of a plane.  Columns outside the row are zero.
template <class T, int LAYOUT>
__device__ __forceinline__ void stage_weight(float4* planes, int ngr, Unit<T, LAYOUT> unit,
                                             const void* weight, float offset) {
  using U = Unit<T, LAYOUT>;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  for (int g = tid; g < ngr; g += blockDim.x * blockDim.y) {
    // granule g of the row: lane 0's of a unit that starts there
    unit.lane = 0;
    const int c0 = g * U::EPL;
    F2 f[U::P];
    Granule<T>::widen(unit.load_weight(weight, c0), f);
#pragma unroll
    for (int i = 0; i < U::P; ++i) {
      f[i] = f2_add(f2(offset, offset), f[i]);
      const int c = unit.col(c0, 2 * i), d = unit.col(c0, 2 * i + 1);
      if (c < 0 || c >= unit.D) f[i].x = 0.0f;
      if (d < 0 || d >= unit.D) f[i].y = 0.0f;
    }
#pragma unroll
    for (int q = 0; q < U::P / 2; ++q)
      planes[q * ngr + g] = make_float4(f[2 * q].x, f[2 * q].y, f[2 * q + 1].x, f[2 * q + 1].y);
  }
}
// granule g's weights
template <class T>
__device__ __forceinline__ void staged_weight(const float4* planes, int ngr, int g,
                                              F2 (&w)[Granule<T>::P]) {
#pragma unroll
  for (int q = 0; q < Granule<T>::P / 2; ++q) {
    const float4 v = planes[q * ngr + g];
    w[2 * q] = f2(v.x, v.y);
    w[2 * q + 1] = f2(v.z, v.w);
  }
}

}  // namespace dit
