// dit_unit.cuh -- rows cut into units of one warp (sm_103a): the loads,
// stores and reductions shared by the weighted-norm kernels.
//
// A unit is 512 bytes of a row: 256 columns of a 16-bit type or 128 of fp32,
// 16 bytes per lane, kept packed in a Raw<16>.  A warp holds consecutive units
// of a row.  Four layouts:
//   WIDE     the rows are made of 16-byte granules.  Lane l holds granule l of
//            the unit; a warp's access is 512 contiguous bytes.
//   PHASED   the tensors start on 16-byte boundaries but the rows do not (an odd
//            width).  Lanes hold the granules of the tensor, not of the row: row
//            r starts `off` elements into its first granule, so that
//            granule's first elements, and its last granule's last ones,
//            belong to the neighbours: they read as zero and are not stored.
//            Rows whose numbers differ by a multiple of EPL (elements per
//            granule) have the same `off`.
//   SHIFTED  the same rows, for work on fixed blocks of columns: the granules
//            are copied as they lie (and one more for the warp), and each lane takes its
//            16 bytes from column c0 + EPL l on out of two of them; stores
//            pass the elements on to the lane that has the rest of a granule.
//   NARROW   a tensor that starts off a 16-byte boundary.  Lane l's element i is
//            column 32 i + l, one element per access.
// The arithmetic is the same for all.  Columns past the row read as
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

// The 16 bytes that start s elements (0 < s < 16 / ES) into the 32 bytes lo,
// hi.  s is the same for the whole warp.
template <int ES>
__device__ __forceinline__ Raw<16> shifted(const Raw<16>& lo, const Raw<16>& hi, int s) {
  const int q = s * ES / 4;  // whole words
  uint32_t a[6], b[5];
#pragma unroll
  for (int i = 0; i < 6; ++i) {
    const uint32_t x = i < 4 ? lo.w[i] : hi.w[i - 4];
    const uint32_t y = i + 2 < 4 ? lo.w[i + 2] : hi.w[i - 2];
    a[i] = q & 2 ? y : x;
  }
#pragma unroll
  for (int i = 0; i < 5; ++i) b[i] = q & 1 ? a[i + 1] : a[i];
  const uint32_t bits = ES == 2 && (s & 1) ? 16u : 0u;
  Raw<16> r;
#pragma unroll
  for (int i = 0; i < 4; ++i) r.w[i] = __funnelshift_r(b[i], b[i + 1], bits);
  return r;
}

// The units of one warp: `units` of them from unit `first` of the row.  j
// counts them; e is the tensor's element index of the lane's first column
// (at()), so that an access is one base address and a constant offset.
template <class T, int LAYOUT>
struct Unit {
  static constexpr int ES = (int)sizeof(T);
  static constexpr int EPL = 16 / ES;       // elements per lane
  static constexpr int COLS = 32 * EPL;     // columns of a unit
  static constexpr int P = Granule<T>::P;   // fp32 pairs per lane

  static constexpr bool OFFSET = LAYOUT == PHASED || LAYOUT == SHIFTED;
  int D, lane, units;
  int off;     // OFFSET: the row's offset from a granule's start, elements
  int c;       // the lane's first column (PHASED: negative in a granule shared with the row before)
  bool edges;  // PHASED: the warp holds a granule shared with a neighbouring row
  // SHIFTED: what lane 31 held of the unit before
  Raw<16> last;
  uint64_t last8;

  // rows row, row + 8 k, ...
  __device__ __forceinline__ Unit(int D, int lane, int first, int units, int64_t row)
      : D(D), lane(lane), units(units), off(0), edges(false), last{}, last8(0) {
    if constexpr (OFFSET) off = (int)(((uint64_t)row * (uint64_t)(D % EPL)) % EPL);
    c = first * COLS + (LAYOUT == NARROW ? lane : LAYOUT == PHASED ? lane * EPL - off : lane * EPL);
    if constexpr (LAYOUT == PHASED) {
      bool mine = false;
      for (int j = 0; j < units; ++j) mine = mine || (valid(j) && !whole(j));
      edges = __any_sync(0xFFFFFFFFu, mine);
    }
  }
  __device__ __forceinline__ int64_t at(int64_t row) const { return row * D + c; }
  // the column of element i of unit j
  __device__ __forceinline__ int col(int j, int i) const {
    return c + j * COLS + (LAYOUT == NARROW ? i * 32 : i);
  }
  __device__ __forceinline__ bool valid(int j) const { return col(j, 0) < D; }
  __device__ __forceinline__ bool whole(int j) const {
    return LAYOUT == WIDE ? valid(j) : col(j, 0) >= 0 && col(j, 0) + EPL <= D;
  }
  __device__ __forceinline__ static const char* ptr(const void* tensor, int64_t e, int j) {
    return (const char*)tensor + e * ES + j * (COLS * ES);
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
  __device__ __forceinline__ Raw<16> elements(const char* p, int j) const {
    constexpr int S = LAYOUT == NARROW ? 32 * ES : ES;
    Raw<16> r = {};
#pragma unroll
    for (int i = 0; i < EPL; ++i) {
      if (col(j, i) < 0 || col(j, i) >= D) continue;
      const Raw<ES> e = STREAM ? ld_stream<ES>(p + i * S) : ld_bcast<ES>(p + i * S);
      if constexpr (ES == 4)
        r.w[i] = e.w[0];
      else
        r.w[i >> 1] |= (uint32_t)e.h << (16 * (i & 1));
    }
    return r;
  }
  // activations, read once (WIDE, NARROW)
  __device__ __forceinline__ Raw<16> load(const void* tensor, int64_t e, int j) const {
    static_assert(!OFFSET, "rows at an offset are copied");
    if constexpr (LAYOUT == NARROW) {
      return elements<true>(ptr(tensor, e, j), j);
    } else {
      Raw<16> r = {};
      if (valid(j)) r = ld_stream<16>(ptr(tensor, e, j));
      return r;
    }
  }
  // weights, read by every row
  __device__ __forceinline__ Raw<16> load_weight(const void* w, int j) const {
    if constexpr (LAYOUT != WIDE) {  // (any alignment)
      return elements<false>(ptr(w, c, j), j);
    } else {
      Raw<16> r = {};
      if (valid(j)) r = ld_bcast<16>(ptr(w, c, j));
      return r;
    }
  }
  // Copy the lane's granule of unit j to its slot at shared address dst
  // (cp.async; not NARROW): the row's bytes from the granule's start on, zeros after
  // them, nothing past the row's end is read.
  __device__ __forceinline__ void copy(uint32_t dst, const void* tensor, int64_t e, int j) const {
    const int back = LAYOUT == SHIFTED ? off : 0;
    const int left = (D - col(j, 0) + back) * ES;
    cp_async16_part(dst, ptr(tensor, e - back, j), (uint32_t)(left < 0 ? 0 : left > 16 ? 16 : left));
  }
  // what copy() left in the slot, without the row before (SHIFTED: the lane's
  // elements of it and the next slot, after a __syncwarp)
  __device__ __forceinline__ Raw<16> copied(uint32_t src, int j) const {
    Raw<16> r = lds16(src);
    if constexpr (LAYOUT == SHIFTED) {
      if (off) r = shifted<ES>(r, lds16(src + 16), off);
    }
    if (LAYOUT == PHASED && j == 0 && c < 0) {
#pragma unroll
      for (int i = 0; i < EPL - 1; ++i) {
        if (i >= off) continue;
        if constexpr (ES == 4)
          r.w[i] = 0;
        else
          r.w[i >> 1] &= i & 1 ? 0x0000FFFFu : 0xFFFF0000u;
      }
    }
    return r;
  }
  // SHIFTED: the granule of unit j that starts `off` elements before the
  // lane's first; elements [from, ...) of it are the warp's
  __device__ __forceinline__ int from(int j) const { return lane == 0 && j == 0 ? off : 0; }
  // (SHIFTED: the whole warp, units in order)
  __device__ __forceinline__ void store(void* tensor, int64_t e, int j, const Raw<16>& r) {
    char* p = (char*)ptr(tensor, e, j);
    if constexpr (LAYOUT == SHIFTED) {
      Raw<16> g = r;
      if (off) {
        Raw<16> before;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          before.w[i] = __shfl_up_sync(0xFFFFFFFFu, r.w[i], 1);
          if (lane == 0) before.w[i] = last.w[i];
          last.w[i] = __shfl_sync(0xFFFFFFFFu, r.w[i], 31);
        }
        g = shifted<ES>(before, r, EPL - off);
      }
      const int c0 = col(j, 0) - off, lo = from(j);
      if (lo == 0 && c0 + EPL <= D) {
        st_stream<16>(p - off * ES, g);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i >= lo && c0 + i < D) st_stream<ES>(p + (i - off) * ES, get(g, i));
      }
      if (j == units - 1 && lane == 31) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i >= EPL - off && col(j, i) < D) st_stream<ES>(p + i * ES, get(r, i));
      }
    } else {
      if constexpr (LAYOUT != NARROW) {
        if (whole(j)) st_stream<16>(p, r);
        if (LAYOUT == WIDE || !edges) return;
      }
      if (LAYOUT == PHASED && (whole(j) || !valid(j))) return;
      constexpr int S = LAYOUT == NARROW ? 32 * ES : ES;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (col(j, i) >= 0 && col(j, i) < D) st_stream<ES>(p + i * S, get(r, i));
    }
  }
  // one byte per element, element i in byte i of q (SHIFTED: the whole warp,
  // units in order)
  __device__ __forceinline__ void store8(void* tensor, int64_t e, int j, const Raw<EPL>& q) {
    char* p = (char*)tensor + e + j * COLS;
    if constexpr (LAYOUT == SHIFTED) {
      uint64_t own = q.w[0];
      if constexpr (EPL == 8) own |= (uint64_t)q.w[EPL / 4 - 1] << 32;
      uint64_t g = own;
      if (off) {
        uint64_t before = __shfl_up_sync(0xFFFFFFFFu, own, 1);
        if (lane == 0) before = last8;
        last8 = __shfl_sync(0xFFFFFFFFu, own, 31);
        g = (before >> (8 * (EPL - off))) | (own << (8 * off));
      }
      const int c0 = col(j, 0) - off, lo = from(j);
      if (lo == 0 && c0 + EPL <= D) {
        Raw<EPL> v;
        v.w[0] = (uint32_t)g;
        if constexpr (EPL == 8) v.w[EPL / 4 - 1] = (uint32_t)(g >> 32);
        st_stream<EPL>(p - off, v);
      } else {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i >= lo && c0 + i < D) p[i - off] = (char)(g >> (8 * i));
      }
      if (j == units - 1 && lane == 31) {
#pragma unroll
        for (int i = 0; i < EPL; ++i)
          if (i >= EPL - off && col(j, i) < D) p[i] = (char)(own >> (8 * i));
      }
    } else {
      if constexpr (LAYOUT != NARROW) {
        if (whole(j)) st_stream<EPL>(p, q);
        if (LAYOUT == WIDE || !edges) return;
      }
      if (LAYOUT == PHASED && (whole(j) || !valid(j))) return;
      constexpr int S = LAYOUT == NARROW ? 32 : 1;
#pragma unroll
      for (int i = 0; i < EPL; ++i)
        if (col(j, i) >= 0 && col(j, i) < D) p[i * S] = (char)(q.w[i >> 2] >> (8 * (i & 3)));
    }
  }
};

// ---------------------------------------------------------------------------
// the warps of one row
// ---------------------------------------------------------------------------

// A team of `warps` warps (at most 16) holds a row; a CTA is blockDim.y teams
// of blockDim.x threads.  combine adds (MAX: .y takes the larger of) a value of
// every warp over the team: through shared memory, one barrier of the team's
// threads (a named barrier; none for a team of one warp) and a butterfly.  The
// slots alternate, so a slot is rewritten only behind the next call's barrier,
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

// A thread's sum of up to some thousand fp32 terms in three levels, 16 and
// 256 at a time: at most 16 + 16 + n / 256 roundings on a term's way.
// Infinities and NaN pass through.
struct LongSum {
  float a = 0.0f, b = 0.0f, c = 0.0f;
  int k = 0;
  __device__ __forceinline__ void add(float v) {
    a = __fadd_rn(a, v);
    if ((++k & 15) == 0) {
      b = __fadd_rn(b, a);
      a = 0.0f;
      if ((k & 255) == 0) {
        c = __fadd_rn(c, b);
        b = 0.0f;
      }
    }
  }
  __device__ __forceinline__ float total() const { return __fadd_rn(__fadd_rn(a, b), c); }
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

// A barrier of the cluster's CTAs (a hardware wait), which orders their shared
// and global accesses; a word of the shared memory of its CTA `rank`.
__device__ __forceinline__ void cluster_barrier() {
  __syncwarp();  // (.aligned: the whole warp at once)
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

// The launch of launch_after and launch_cluster.  An error is returned and not
// left for the next launch's cudaGetLastError, which would report it again.
template <class Args>
cudaError_t launch_config(const cudaLaunchConfig_t& cfg, void (*kern)(Args), const Args& args) {
  const cudaError_t e = cudaLaunchKernelEx(&cfg, kern, args);
  if (e != cudaSuccess) (void)cudaGetLastError();
  return e;
}

// A kernel launched by launch_after starts while the one before it in the
// stream ends: it waits for that one's results (after_previous, before it
// touches memory), which says early that the next may come (let_next).
// griddepcontrol waits in hardware.
__device__ __forceinline__ void after_previous() { asm volatile("griddepcontrol.wait;" ::: "memory"); }
__device__ __forceinline__ void let_next() {
  asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
}
template <class Args>
cudaError_t launch_after(void (*kern)(Args), dim3 grid, dim3 block, size_t smem, cudaStream_t s,
                         const Args& args) {
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = grid;
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
  at[0].val.programmaticStreamSerializationAllowed = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch_config(cfg, kern, args);
}

// A launch of one cluster of `grid` CTAs (16: the size that a kernel opts in to).
template <class Args>
cudaError_t launch_cluster(void (*kern)(Args), unsigned grid, dim3 block, size_t smem, cudaStream_t s,
                           const Args& args) {
  if (grid > 8) {
    const cudaError_t e =
        cudaFuncSetAttribute((const void*)kern, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return e;
    }
  }
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(grid);
  cfg.blockDim = block;
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = grid;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return launch_config(cfg, kern, args);
}

// Units of a row of D columns (PHASED: at most, over the rows' offsets).
template <class T, int LAYOUT>
int64_t row_units(int64_t D) {
  using U = Unit<T, LAYOUT>;
  return (D + (LAYOUT == PHASED ? U::EPL - 1 : 0) + U::COLS - 1) / U::COLS;
}

// The weight, offset added, in shared memory as fp32 for rows at offset `off`
// from a granule: plane q of granule g (of ngr) holds columns 4q .. 4q + 3 of
// it, so a warp reads 512 contiguous bytes of a plane.  Columns outside the
// row are zero.
template <class T, int LAYOUT>
__device__ __forceinline__ void stage_weight(float4* planes, int ngr, int D, int64_t row,
                                             const void* weight, float offset) {
  using U = Unit<T, LAYOUT>;
  const int tid = threadIdx.y * blockDim.x + threadIdx.x;
  const U start(D, 0, 0, 0, row);
  for (int g = tid; g < ngr; g += blockDim.x * blockDim.y) {
    U unit = start;
    unit.c += g * U::EPL;
    F2 f[U::P];
    Granule<T>::widen(unit.load_weight(weight, 0), f);
#pragma unroll
    for (int i = 0; i < U::P; ++i) {
      f[i] = f2_add(f2(offset, offset), f[i]);
      const int c = unit.col(0, 2 * i), d = unit.col(0, 2 * i + 1);
      if (c < 0 || c >= D) f[i].x = 0.0f;
      if (d < 0 || d >= D) f[i].y = 0.0f;
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
