// k_embedding.cu -- embedding lookup with a scale, and its gradient.
//
//   out[t] = rnd(table[id_t] * scale)
//   gt[v]  = rnd(scale * sum over {t : id_t = v} of g[t])
//
// An id outside [0, V) (a padded place) gives a row of zeros and takes no
// gradient.
//
// The gradient sorts the tokens first: a stable radix sort of (id, position),
// so the rows of one id stand together in the order of their positions, and
// every sum has one order -- no atomics, the same bits from every call.  The
// sorted tokens are cut into segments of 32, one team of threads each,
// whatever the ids' distribution.  A run of one id inside a segment is summed
// and written once.  A run that crosses segments leaves one fp32 row per
// segment in the workspace, and a last kernel adds those in order.  The rows
// of the table that no token names are found in the sorted ids and filled
// with zeros by further CTAs of the same launch, so each row of the gradient
// is written once.
#include <algorithm>

#include "dit_stat.cuh"
#include "dit_token.h"
#include "dit_unit.cuh"

namespace dit {
namespace {

// the id at position t as a key in [0, V], V for an id outside [0, V)
__device__ __forceinline__ uint32_t key_at(const void* ids, bool ids64, int64_t t, int64_t V) {
  const int64_t id = ids64 ? ((const int64_t*)ids)[t] : (int64_t)((const int32_t*)ids)[t];
  return id >= 0 && id < V ? (uint32_t)id : (uint32_t)V;
}

// VB bytes of T times a scale, rounded once
template <class T, int VB>
__device__ __forceinline__ Raw<VB> scaled(const Raw<VB>& r, float scale) {
  using V = Vec<T, VB>;
  float f[V::N];
  V::widen(r, f);
#pragma unroll
  for (int i = 0; i < V::N; ++i) f[i] = __fmul_rn(f[i], scale);
  return V::narrow(f);
}

// threads of a CTA over the vectors of a row (a power of two, at most 256)
int row_threads(int64_t nvec) {
  int t = 1;
  while (t < 256 && t < nvec) t *= 2;
  return t;
}

// blockDim = (threads of a row, tokens of a CTA)
template <class T, int VB>
__global__ void __launch_bounds__(256) embedding_kernel(EmbedArgs a) {
  constexpr int ES = (int)sizeof(T);
  const int64_t pitch = (int64_t)a.D * ES;
  const int nvec = (int)(pitch / VB);
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.tokens;
       t += (int64_t)gridDim.x * blockDim.y) {
    const uint32_t key = key_at(a.ids, a.ids64, t, a.V);
    const char* src = (const char*)a.table + (int64_t)key * pitch;
    char* dst = (char*)a.out + t * pitch;
    const bool seen = key < a.V;
    for (int v = threadIdx.x; v < nvec; v += blockDim.x) {
      Raw<VB> r = {};
      if (seen) r = scaled<T, VB>(ld_stream<VB>(src + (int64_t)v * VB), a.scale);
      st_stream<VB>(dst + (int64_t)v * VB, r);
    }
  }
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------

__device__ __forceinline__ void cluster_barrier() {
  asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::
                   : "memory");
}
__device__ __forceinline__ uint32_t ld_cluster(uint32_t addr, uint32_t rank) {
  uint32_t remote, v;
  asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(remote) : "r"(addr), "r"(rank));
  asm volatile("ld.shared::cluster.u32 %0, [%1];" : "=r"(v) : "r"(remote) : "memory");
  return v;
}

constexpr int kSortWarps = 32;
constexpr int kSortBits = 9;  // at most, per pass: 32 counters per digit in shared memory
constexpr int kSortCluster = 8;

struct SortArgs {
  const void* ids;
  uint2* pairs[2];
  int64_t tokens, V;
  int64_t per_warp;  // consecutive tokens of a warp, a multiple of 32
  int ctas;          // CTAs of the cluster
  int passes, bits;  // digits, and bits of each
  bool ids64;
};

// Stable least-significant-digit radix sort by one cluster.  Warp w of CTA c
// owns the tokens [(32 c + w) per_warp, ...) of every pass, and counts them
// per digit; a digit's place is the count of smaller digits, then of earlier
// CTAs, then of earlier warps, then of earlier tokens of the warp.  Pass p
// writes pairs[p & 1].
__global__ void __launch_bounds__(kSortWarps * 32) sort_kernel(SortArgs a) {
  extern __shared__ uint32_t count[];  // [warps][digits]
  __shared__ uint32_t total[1 << kSortBits];
  __shared__ uint32_t scan[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << a.bits;
  const uint32_t cta = a.ctas > 1 ? blockIdx.x : 0;
  const int64_t first = ((int64_t)cta * kSortWarps + warp) * a.per_warp;
  const int64_t last = first + a.per_warp < a.tokens ? first + a.per_warp : a.tokens;
  uint32_t* mine = count + warp * digits;

  for (int p = 0; p < a.passes; ++p) {
    const uint2* src = a.pairs[(p & 1) ^ 1];
    auto load = [&](int64_t i) {
      return p == 0 ? make_uint2(key_at(a.ids, a.ids64, i, a.V), (uint32_t)i) : __ldcg(src + i);
    };
    auto digit = [&](uint32_t key) { return (int)((key >> (p * a.bits)) & (uint32_t)(digits - 1)); };
    for (int i = lane; i < digits; i += 32) mine[i] = 0;
    __syncwarp();
    for (int64_t i = first + lane; i < last; i += 32) atomicAdd(&mine[digit(load(i).x)], 1u);
    __syncthreads();
    // counters of a digit -> counts of earlier warps; the CTA's total
    uint32_t sum = 0;
    if ((int)threadIdx.x < digits) {
      for (int w = 0; w < kSortWarps; ++w) {
        const uint32_t n = count[w * digits + threadIdx.x];
        count[w * digits + threadIdx.x] = sum;
        sum += n;
      }
      total[threadIdx.x] = sum;
    }
    // counts of earlier CTAs, and of the whole cluster
    uint32_t before = 0, all = sum;
    if (a.ctas > 1) {
      cluster_barrier();
      if ((int)threadIdx.x < digits) {
        all = 0;
        const uint32_t addr = smem_addr(&total[threadIdx.x]);
        for (int c = 0; c < a.ctas; ++c) {
          const uint32_t n = ld_cluster(addr, c);
          before += (uint32_t)c < cta ? n : 0u;
          all += n;
        }
      }
      cluster_barrier();  // every total has been read
    }
    // the digits' first places: an exclusive sum over the digits
    uint32_t inc = (int)threadIdx.x < digits ? all : 0u;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const uint32_t n = __shfl_up_sync(0xFFFFFFFFu, inc, o);
      if (lane >= o) inc += n;
    }
    __syncthreads();  // (a CTA alone: total and scan of the previous pass have been read)
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    uint32_t place = before + inc - all;
    for (int w = 0; w < warp; ++w) place += scan[w];
    if ((int)threadIdx.x < digits)
      for (int w = 0; w < kSortWarps; ++w) count[w * digits + threadIdx.x] += place;
    __syncthreads();
    // place the warp's tokens, 32 at a time in their order
    uint2* dst = a.pairs[p & 1];
    for (int64_t i0 = first; i0 < last; i0 += 32) {
      const bool has = i0 + lane < last;
      const uint2 v = has ? load(i0 + lane) : make_uint2(0u, 0u);
      const int d = digit(v.x);
      uint32_t same = __ballot_sync(0xFFFFFFFFu, has);
      for (int b = 0; b < a.bits; ++b) {
        const uint32_t set = __ballot_sync(0xFFFFFFFFu, (d >> b) & 1);
        same &= (d >> b) & 1 ? set : ~set;
      }
      const uint32_t base = has ? mine[d] : 0u;
      __syncwarp();
      if (has) {
        dst[base + __popc(same & ((1u << lane) - 1u))] = v;
        if (lane == __ffs(same) - 1) mine[d] = base + __popc(same);
      }
      __syncwarp();
    }
    if (a.ctas > 1)
      cluster_barrier();  // the next pass reads what the other CTAs placed
    else
      __syncthreads();
  }
}

// ---------------------------------------------------------------------------
// the sums
// ---------------------------------------------------------------------------

struct SumArgs {
  void* gt;
  const void* g;
  const uint2* sorted;
  float* partial;
  int64_t tokens, V;
  int64_t segments;
  int64_t seg_ctas;   // CTAs of the segments; the others fill rows with zeros
  int D;
  int zero_rows;      // rows of the table per CTA that fills zeros
  float scale;
};

constexpr int kMaxZeroRows = 256;

// the first index of sorted whose key is at least `key` (a whole warp)
__device__ __forceinline__ int64_t lower_bound(const uint2* sorted, int64_t n, uint32_t key,
                                               int lane) {
  int64_t lo = 0, hi = n;  // the answer is in [lo, hi]
  while (hi > lo) {
    const int64_t step = (hi - lo + 31) / 32;
    const int64_t at = lo + step * lane + step - 1;  // the last of this lane's part
    const bool below = at < hi && __ldg(&sorted[at].x) < key;
    const int parts = __popc(__ballot_sync(0xFFFFFFFFu, below));
    lo += step * parts;
    if (lo > hi) lo = hi;
    if (lo + step - 1 < hi) hi = lo + step - 1;
  }
  return lo;
}

// Zeros over `bytes` bytes at p (element-aligned), by the warp: 16-byte stores
// between the first and last 16-byte boundary.
template <int ES>
__device__ __forceinline__ void fill_zero(char* p, int64_t bytes, int lane) {
  int64_t head = (int64_t)((16u - ((uintptr_t)p & 15u)) & 15u);
  if (head > bytes) head = bytes;
  for (int64_t i = lane * ES; i < head; i += 32 * ES) st_stream<ES>(p + i, Raw<ES>{});
  const int64_t body = (bytes - head) / 16;
  for (int64_t i = lane; i < body; i += 32) st_stream<16>(p + head + i * 16, Raw<16>{});
  for (int64_t i = head + body * 16 + lane * ES; i < bytes; i += 32 * ES) st_stream<ES>(p + i, Raw<ES>{});
}

// blockDim = (threads of a row, segments of a CTA); gridDim.y column tiles of
// blockDim.x * 16 bytes (elements, for rows that are not made of granules).
template <class T, int VB>
__global__ void __launch_bounds__(256) embedding_sum_kernel(SumArgs a) {
  using V = Vec<T, VB>;
  constexpr int N = V::N, ES = (int)sizeof(T);
  const int64_t pitch = (int64_t)a.D * ES;
  if ((int64_t)blockIdx.x >= a.seg_ctas) {
    if (blockIdx.y > 0) return;
    // rows that no token names
    __shared__ uint32_t named[kMaxZeroRows / 32];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int nthr = blockDim.x * blockDim.y;
    const int64_t v0 = ((int64_t)blockIdx.x - a.seg_ctas) * a.zero_rows;
    const int64_t v1 = v0 + a.zero_rows < a.V ? v0 + a.zero_rows : a.V;
    if (tid < kMaxZeroRows / 32) named[tid] = 0;
    __syncthreads();
    const int64_t lo = lower_bound(a.sorted, a.tokens, (uint32_t)v0, tid & 31);
    const int64_t hi = lo + lower_bound(a.sorted + lo, a.tokens - lo, (uint32_t)v1, tid & 31);
    for (int64_t i = lo + tid; i < hi; i += nthr) {
      const int k = (int)((int64_t)a.sorted[i].x - v0);
      atomicOr(&named[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    for (int64_t v = v0 + (tid >> 5); v < v1; v += nthr >> 5) {
      const int k = (int)(v - v0);
      if (!((named[k >> 5] >> (k & 31)) & 1u)) 
        fill_zero<ES>((char*)a.gt + v * pitch, pitch, tid & 31);
    }
    return;
  }
  const int64_t seg = (int64_t)blockIdx.x * blockDim.y + threadIdx.y;
  const int vec = blockIdx.y * blockDim.x + threadIdx.x;
  if (seg >= a.segments || vec >= (int)(pitch / VB)) return;
  const int64_t i0 = seg * kEmbedSegment;
  const int64_t i1 = i0 + kEmbedSegment < a.tokens ? i0 + kEmbedSegment : a.tokens;
  const char* src = (const char*)a.g + (int64_t)vec * VB;
  uint32_t key = __ldg(&a.sorted[i0].x);
  bool head = i0 > 0 && __ldg(&a.sorted[i0 - 1].x) == key;
  const uint32_t after = i1 < a.tokens ? __ldg(&a.sorted[i1].x) : (uint32_t)a.V;
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  // the run of `key` ends here (open: it goes on in the next segment)
  auto flush = [&](bool open) {
    if (key < a.V) {
      if (head || open) {
        float* p = a.partial + (seg * 2 + (head ? 0 : 1)) * a.D + (int64_t)vec * N;
#pragma unroll
        for (int e = 0; e < N; ++e) p[e] = acc[e];
      } else {
        float f[N];
#pragma unroll
        for (int e = 0; e < N; ++e) f[e] = __fmul_rn(acc[e], a.scale);
        st_stream<VB>((char*)a.gt + (int64_t)key * pitch + (int64_t)vec * VB, V::narrow(f));
      }
    }
#pragma unroll
    for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  };
  constexpr int AHEAD = 8;  // rows in flight
  for (int64_t i = i0; i < i1; i += AHEAD) {
    Raw<VB> r[AHEAD];
    uint32_t k[AHEAD];
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      k[j] = (uint32_t)a.V;
      if (i + j < i1) {
        const uint2 s = __ldg(a.sorted + i + j);
        k[j] = s.x;
        if (s.x < a.V) r[j] = ld_stream<VB>(src + (int64_t)s.y * pitch);
      }
    }
#pragma unroll
    for (int j = 0; j < AHEAD; ++j) {
      if (i + j >= i1) break;
      if (k[j] != key) {
        flush(false);
        key = k[j];
        head = false;
      }
      if (key < a.V) {
        float f[N];
        V::widen(r[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
      }
    }
  }
  flush(after == key);
}

// A run that starts in segment s and goes on: its parts added in order.
template <class T>
__global__ void __launch_bounds__(256) embedding_join_kernel(SumArgs a) {
  const int64_t seg = (int64_t)blockIdx.x;
  const int64_t i1 = (seg + 1) * kEmbedSegment;
  if (i1 >= a.tokens) return;
  const uint32_t key = __ldg(&a.sorted[i1 - 1].x);
  if (key >= a.V || __ldg(&a.sorted[i1].x) != key) return;  // ends here
  const int64_t i0 = seg * kEmbedSegment;
  if (i0 > 0 && __ldg(&a.sorted[i0].x) == key && __ldg(&a.sorted[i0 - 1].x) == key) return;  // began before
  int64_t n = 1;  // further segments of the run
  while (i1 + n * kEmbedSegment < a.tokens && __ldg(&a.sorted[i1 + n * kEmbedSegment].x) == key) ++n;
  const float* p = a.partial + (seg * 2 + 1) * a.D;
  for (int c = blockIdx.y * blockDim.x + threadIdx.x; c < a.D; c += gridDim.y * blockDim.x) {
    float v = p[c];
    for (int64_t j = 0; j < n; ++j) v = __fadd_rn(v, p[(1 + 2 * j) * a.D + c]);
    float f[1] = {__fmul_rn(v, a.scale)};
    st_stream<sizeof(T)>((char*)a.gt + ((int64_t)key * a.D + c) * (int)sizeof(T),
                         Vec<T, (int)sizeof(T)>::narrow(f));
  }
}

template <class T, int VB>
cudaError_t launch_sums(SumArgs a, cudaStream_t s) {
  const int64_t nvec = (int64_t)a.D * (int)sizeof(T) / VB;
  const int tx = row_threads(nvec), ty = 256 / tx;
  a.seg_ctas = (a.segments + ty - 1) / ty;
  // about 128 KB of zeros per CTA
  a.zero_rows = (int)std::min<int64_t>(kMaxZeroRows, std::max<int64_t>(1, (128 << 10) / ((int64_t)a.D * (int)sizeof(T))));
  const int64_t zero_ctas = (a.V + a.zero_rows - 1) / a.zero_rows;
  const int64_t tiles = (nvec + tx - 1) / tx;
  if (a.seg_ctas + zero_ctas > 0x7FFFFFFF || tiles > 65535) return cudaErrorInvalidConfiguration;
  embedding_sum_kernel<T, VB><<<dim3((unsigned)(a.seg_ctas + zero_ctas), (unsigned)tiles),
                                dim3(tx, ty), 0, s>>>(a);
  cudaError_t e = cudaGetLastError();
  if (e != cudaSuccess || a.segments < 2) return e;
  const unsigned cols = (unsigned)std::min<int64_t>(64, ((int64_t)a.D + 255) / 256);
  embedding_join_kernel<T><<<dim3((unsigned)(a.segments - 1), cols), 256, 0, s>>>(a);
  return cudaGetLastError();
}

cudaError_t launch_sort(const DeviceInfo& dev, SortArgs a, cudaStream_t s) {
  a.ctas = a.tokens > 4096 ? kSortCluster : 1;
  const int64_t warps = (int64_t)a.ctas * kSortWarps;
  a.per_warp = ((a.tokens + warps - 1) / warps + 31) / 32 * 32;
  const size_t smem = (size_t)kSortWarps * (1 << a.bits) * 4;
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)sort_kernel, dev, opted);
  if (e != cudaSuccess) return e;
  cudaLaunchConfig_t cfg = {};
  cfg.gridDim = dim3(a.ctas);
  cfg.blockDim = dim3(kSortWarps * 32);
  cfg.dynamicSmemBytes = smem;
  cfg.stream = s;
  cudaLaunchAttribute at[1];
  at[0].id = cudaLaunchAttributeClusterDimension;
  at[0].val.clusterDim.x = a.ctas;
  at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
  cfg.attrs = at;
  cfg.numAttrs = 1;
  return cudaLaunchKernelEx(&cfg, sort_kernel, a);
}

}  // namespace

cudaError_t launch_embedding(int dtype, bool wide, const EmbedArgs& a, cudaStream_t s) {
  const int es = dtype == 2 ? 4 : 2;
  return dispatch_dtype_width(dtype, wide ? 16 : es, [&](auto tt, auto w) -> cudaError_t {
    using T = typename decltype(tt)::type;
    constexpr int VB = decltype(w)::value;
    if constexpr (VB == 16 || VB == (int)sizeof(T)) {
      const int tx = row_threads((int64_t)a.D * es / VB), ty = 256 / tx;
      const int64_t grid = std::min<int64_t>((a.tokens + ty - 1) / ty, int64_t(1) << 30);
      embedding_kernel<T, VB><<<(unsigned)grid, dim3(tx, ty), 0, s>>>(a);
      return cudaGetLastError();
    } else {
      return cudaErrorInvalidValue;
    }
  });
}

cudaError_t launch_embedding_grad(const DeviceInfo& dev, int dtype, bool wide,
                                  const EmbedGradArgs& a, cudaStream_t s) {
  SortArgs q = {};
  q.ids = a.ids;
  q.ids64 = a.ids64;
  q.tokens = a.tokens;
  q.V = a.V;
  q.pairs[0] = a.pairs[0];
  q.pairs[1] = a.pairs[1];
  int bits = 1;  // of the keys 0 .. V
  while (bits < 32 && (a.V >> bits) != 0) ++bits;
  q.passes = (bits + kSortBits - 1) / kSortBits;
  q.bits = (bits + q.passes - 1) / q.passes;
  if (a.tokens > 0) {
    const cudaError_t e = launch_sort(dev, q, s);
    if (e != cudaSuccess) return e;
  }
  SumArgs m = {};
  m.gt = a.gt;
  m.g = a.g;
  m.sorted = a.pairs[(q.passes - 1) & 1];
  m.partial = a.partial;
  m.tokens = a.tokens;
  m.V = a.V;
  m.segments = embed_segments(a.tokens);
  m.D = a.D;
  m.scale = a.scale;
  const int es = dtype == 2 ? 4 : 2;
  return dispatch_dtype_width(dtype, wide ? 16 : es, [&](auto tt, auto w) -> cudaError_t {
    using T = typename decltype(tt)::type;
    constexpr int VB = decltype(w)::value;
    if constexpr (VB == 16 || VB == (int)sizeof(T))
      return launch_sums<T, VB>(m, s);
    else
      return cudaErrorInvalidValue;
  });
}

}  // namespace dit
