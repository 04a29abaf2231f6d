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
// every sum has one order -- no atomics on values, the same bits from every
// call.  The sorted tokens are cut into segments of 32, one team of threads
// each, whatever the ids' distribution.  A run of one id inside a segment is
// summed and written once; one that ends in the next segment too, by its first
// segment's team, each segment's part for itself.  A longer run leaves one fp32
// row per segment in the workspace, and a last kernel adds those.  The rows of
// the table that no token names are found in the sorted ids and filled with
// zeros by further CTAs of the same launch, so each row of the gradient is
// written once.  Up to kFewTokens tokens need no sort: every CTA reads all ids, the
// first token of each id adds its rows, and one launch does it all.
//
// Lookup of 32640 bf16 rows of 4096: 77 us, 6.9 TB/s, bound by memory (odd
// width, 16000 of 3077: 45 us).  Gradient of 32640 tokens for [128000, 2048]
// bf16: 119 us, of which the sort 17 (one cluster: bound by latency) and the
// join 8 to 13; the sums and the zeros are bound by memory, for odd widths by
// the instructions that shift and store them (16000 x 3077: 84 us).  126
// tokens for [32000, 2048] fp32: 40 us, 6.6 TB/s, nearly all of it zeros.
#include <algorithm>
#include <type_traits>

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

// The 16 bytes that start at element e (>= 0) of a tensor of `total` elements
// whose first byte is 16-byte aligned: two granules and a shift, which is the
// same for every lane (their e are alike modulo a granule).  Elements past
// the tensor's end read as zero.
template <class T>
__device__ __forceinline__ Raw<16> load_shifted(const void* tensor, int64_t e, int64_t total) {
  constexpr int ES = (int)sizeof(T), EPG = 16 / ES;
  const int s = (int)(e & (EPG - 1));
  const int64_t g = e - s;
  if (g + (s ? 2 : 1) * EPG <= total) {
    const Raw<16> lo = ld_stream<16>((const char*)tensor + g * ES);
    if (s == 0) return lo;
    return shifted<ES>(lo, ld_stream<16>((const char*)tensor + (g + EPG) * ES), s);
  }
  Raw<16> r = {};
#pragma unroll
  for (int i = 0; i < EPG; ++i) {
    if (e + i >= total) continue;
    const Raw<ES> v = ld_stream<ES>((const char*)tensor + (e + i) * ES);
    if constexpr (ES == 4)
      r.w[i] = v.w[0];
    else
      r.w[i >> 1] |= (uint32_t)v.h << (16 * (i & 1));
  }
  return r;
}

// Rows cut into tiles, a few columns per thread.  WIDE: a granule of rows that
// are made of 16-byte granules.  PHASED: the same columns of rows that are
// not, in tensors that start on 16-byte boundaries (load_shifted).  NARROW: four
// single elements blockDim.x columns apart.
template <class T, int LAYOUT>
struct Tile {
  static constexpr int ES = (int)sizeof(T);
  static constexpr int N = LAYOUT == NARROW ? 4 : 16 / ES;
  static constexpr int VB = N * ES;
  using R = Raw<VB>;
  int D, c;  // c: the thread's first column
  __device__ __forceinline__ Tile(int D, int tile)
      : D(D), c(tile * (int)blockDim.x * N + (LAYOUT == NARROW ? threadIdx.x : threadIdx.x * N)) {}
  __device__ __forceinline__ int col(int i) const {
    return LAYOUT == NARROW ? c + i * (int)blockDim.x : c + i;
  }
  __device__ __forceinline__ bool valid() const { return c < D; }
  __device__ __forceinline__ static void put(R& r, int i, const void* p) {
    const Raw<ES> e = ld_stream<ES>(p);
    if constexpr (ES == 4)
      r.w[i] = e.w[0];
    else
      r.w[i >> 1] |= (uint32_t)e.h << (16 * (i & 1));
  }
  // the thread's columns of row `row` of `rows` (PHASED: past the row's end,
  // what follows it)
  __device__ __forceinline__ R load(const void* tensor, int64_t row, int64_t rows) const {
    const int64_t e = row * D + c;
    if constexpr (LAYOUT == WIDE) {
      return ld_stream<16>((const char*)tensor + e * ES);
    } else {
      if (LAYOUT == PHASED && c >= 0) {
        if constexpr (LAYOUT == PHASED) return load_shifted<T>(tensor, e, rows * D);
      }
      R r = {};
      constexpr int S = LAYOUT == NARROW ? 0 : 1;
#pragma unroll
      for (int i = 0; i < N; ++i)
        if (col(i) >= 0 && col(i) < D)
          put(r, i, (const char*)tensor + (e + (S ? i : i * (int)blockDim.x)) * ES);
      return r;
    }
  }
  __device__ __forceinline__ static void widen(const R& r, float (&f)[N]) {
    Vec<T, VB>::widen(r, f);
  }
  // elements [lo, hi) of r, whose first is element e of the tensor
  __device__ __forceinline__ static void scatter(void* tensor, int64_t e, const R& r, int lo, int hi) {
#pragma unroll
    for (int i = 0; i < N; ++i) {
      if (i < lo || i >= hi) continue;
      Raw<ES> v;
      if constexpr (ES == 4)
        v.w[0] = r.w[i];
      else
        v.h = (uint16_t)(r.w[i >> 1] >> (16 * (i & 1)));
      st_stream<ES>((char*)tensor + (e + i * (LAYOUT == NARROW ? (int)blockDim.x : 1)) * ES, v);
    }
  }
  // f * scale, rounded once, to row `row`.  granules: element c of the row is
  // the first of a granule; PHASED rows without are stored by the whole warp.
  __device__ __forceinline__ void store(void* tensor, int64_t row, const float (&f)[N], float scale,
                                        bool granules = false) const {
    float v[N];
#pragma unroll
    for (int i = 0; i < N; ++i) v[i] = __fmul_rn(f[i], scale);
    const R r = Vec<T, VB>::narrow(v);
    const int64_t e = row * D + c;
    if constexpr (LAYOUT == WIDE) {
      if (valid()) st_stream<16>((char*)tensor + e * ES, r);
    } else if constexpr (LAYOUT == NARROW) {
      // columns c, c + blockDim.x, ... below D
      const int left = D - c, w = (int)blockDim.x;
      scatter(tensor, e, r, 0, left <= 0 ? 0 : (left + w - 1) / w);
    } else {
      const int s = granules ? 0 : (int)(e & (N - 1)), lane = threadIdx.x & 31;
      if (s == 0) {
        if (c >= 0 && c + N <= D)
          st_stream<16>((char*)tensor + e * ES, r);
        else
          scatter(tensor, e, r, -c, D - c);
        return;
      }
      // the granule that starts s elements before column c: the previous
      // lane's last s elements and this lane's first ones
      R before;
#pragma unroll
      for (int i = 0; i < 4; ++i) before.w[i] = __shfl_up_sync(0xFFFFFFFFu, r.w[i], 1);
      const R g = shifted<ES>(before, r, N - s);
      const int first = lane ? 0 : s;  // (lane 0 has no previous lane)
      if (first == 0 && c - s + N <= D)
        st_stream<16>((char*)tensor + (e - s) * ES, g);
      else
        scatter(tensor, e - s, g, first, D - (c - s));
      if (lane == 31) scatter(tensor, e, r, N - s, D - c);
    }
  }
};

// columns a thread takes, threads of a CTA over a row (a power of two, 32 to
// 256), and the row's tiles
int tile_columns(int es, int layout) { return layout == NARROW ? 4 : 16 / es; }
int row_threads(int64_t D, int n) {
  int t = 32;
  while (t < 256 && (int64_t)t * n < D) t *= 2;
  return t;
}
int64_t row_tiles(int64_t D, int n) {
  const int64_t tile = (int64_t)n * row_threads(D, n);
  return (D + tile - 1) / tile;
}

// blockDim = (threads of a row, tokens of a CTA).  PHASED: the threads' columns
// are the output's granules, so only the loads are shifted.
template <class T, int LAYOUT>
__global__ void __launch_bounds__(256) embedding_kernel(EmbedArgs a, int tiles) {
  using L = Tile<T, LAYOUT>;
  for (int64_t t = (int64_t)blockIdx.x * blockDim.y + threadIdx.y; t < a.tokens;
       t += (int64_t)gridDim.x * blockDim.y) {
    const uint32_t key = key_at(a.ids, a.ids64, t, a.V);
    const bool seen = key < a.V;
    const int off = LAYOUT == PHASED ? (int)((t * (a.D % L::N)) % L::N) : 0;
    constexpr int AHEAD = LAYOUT == NARROW ? 4 : 2;  // tiles in flight
    for (int k = 0; k < tiles; k += AHEAD) {
      typename L::R r[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        L tile(a.D, k + j);
        tile.c -= off;
        r[j] = typename L::R{};
        if (seen && tile.valid()) r[j] = tile.load(a.table, key, a.V);
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        L tile(a.D, k + j);
        tile.c -= off;
        float f[L::N];
        L::widen(r[j], f);
        if (tile.valid()) tile.store(a.out, t, f, seen ? a.scale : 0.0f, true);
      }
    }
  }
}

// ---------------------------------------------------------------------------
// the sort
// ---------------------------------------------------------------------------

constexpr int kSortWarps = 32;
constexpr int kSortBits = 9;  // at most, per pass: 32 counters per digit in shared memory
constexpr int kSortCluster = 16;  // (the opt-in size; 60000 tokens: 8 took 20.8 us, 16 take 16.7)

struct SortArgs {
  const void* ids;
  uint2* pairs[2];
  uint32_t* runs;    // the count of runs that cross segments: set to zero here
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
// writes pairs[p & 1].  Tokens are read 32 * kRounds at a time, once a pass
// where a warp has no more than that.
__global__ void __launch_bounds__(kSortWarps * 32) sort_kernel(SortArgs a) {
  constexpr int kRounds = 8;
  extern __shared__ uint32_t count[];  // [warps][digits]
  __shared__ uint32_t total[1 << kSortBits];
  __shared__ uint32_t start[1 << kSortBits];
  __shared__ uint32_t scan[kSortWarps];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int digits = 1 << a.bits;
  const uint32_t cta = a.ctas > 1 ? blockIdx.x : 0;
  const int64_t first = ((int64_t)cta * kSortWarps + warp) * a.per_warp;
  const int64_t last = first + a.per_warp < a.tokens ? first + a.per_warp : a.tokens;
  const bool once = a.per_warp <= 32 * kRounds;
  uint32_t* mine = count + warp * digits;
  if (blockIdx.x == 0 && threadIdx.x == 0) *a.runs = 0;
  let_next();

  for (int p = 0; p < a.passes; ++p) {
    const uint2* src = a.pairs[(p & 1) ^ 1];
    uint2 v[kRounds];
    auto load = [&](int64_t i0) {
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        const int64_t i = i0 + 32 * k + lane;
        v[k] = make_uint2(0u, 0u);
        if (i < last)
          v[k] = p == 0 ? make_uint2(key_at(a.ids, a.ids64, i, a.V), (uint32_t)i) : __ldcg(src + i);
      }
    };
    auto digit = [&](uint32_t key) { return (int)((key >> (p * a.bits)) & (uint32_t)(digits - 1)); };
    for (int i = lane; i < digits; i += 32) mine[i] = 0;
    __syncwarp();
    for (int64_t i0 = first; i0 < last; i0 += 32 * kRounds) {
      load(i0);
#pragma unroll
      for (int k = 0; k < kRounds; ++k)
        if (i0 + 32 * k + lane < last) atomicAdd(&mine[digit(v[k].x)], 1u);
    }
    __syncthreads();
    // counters of a digit -> counts of earlier warps; the CTA's total
    uint32_t sum = 0;
    if ((int)threadIdx.x < digits) {
      uint32_t n[kSortWarps];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) n[w] = count[w * digits + threadIdx.x];
#pragma unroll
      for (int w = 0; w < kSortWarps; ++w) {
        count[w * digits + threadIdx.x] = sum;
        sum += n[w];
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
#pragma unroll
        for (int c = 0; c < kSortCluster; ++c) {
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
    if (lane == 31) scan[warp] = inc;
    __syncthreads();
    const uint32_t part = lane < warp ? scan[lane] : 0u;  // the warps before this one
    uint32_t place = before + inc - all + __reduce_add_sync(0xFFFFFFFFu, part);
    if ((int)threadIdx.x < digits) start[threadIdx.x] = place;
    __syncthreads();
    // place the warp's tokens, 32 at a time in their order
    uint2* dst = a.pairs[p & 1];
    for (int64_t i0 = first; i0 < last; i0 += 32 * kRounds) {
      if (!once) load(i0);
#pragma unroll
      for (int k = 0; k < kRounds; ++k) {
        if (i0 + 32 * k >= last) break;  // the whole warp
        const bool has = i0 + 32 * k + lane < last;
        const int d = digit(v[k].x);
        uint32_t same = __ballot_sync(0xFFFFFFFFu, has);
        for (int b = 0; b < a.bits; ++b) {
          const uint32_t set = __ballot_sync(0xFFFFFFFFu, (d >> b) & 1);
          same &= (d >> b) & 1 ? set : ~set;
        }
        const uint32_t base = has ? mine[d] : 0u;
        __syncwarp();
        if (has) {
          dst[start[d] + base + __popc(same & ((1u << lane) - 1u))] = v[k];
          if (lane == __ffs(same) - 1) mine[d] = base + __popc(same);
        }
        __syncwarp();
      }
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
  const void* ids;      // few tokens: unsorted
  const uint2* sorted;
  float* partial;
  uint32_t* runs;       // [0] the count of, [1...] the first segments of runs that cross segments
  int64_t tokens, V;
  int64_t segments;
  int64_t seg_ctas;     // the first CTAs, of the segments (or tokens); the others fill rows with zeros
  int D, tiles;
  int zero_rows;        // rows of the table per CTA that fills zeros
  bool ids64;
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
    const bool below = at < hi && sorted[at].x < key;
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

// Rows [v0, v1) of the table that `named` (a bit each, shared) does not mark,
// filled with zeros by the CTA's warps.
template <int ES>
__device__ __forceinline__ void fill_rows(const SumArgs& a, const uint32_t* named, int64_t v0,
                                          int64_t v1, int tid, int nthr) {
  const int64_t pitch = (int64_t)a.D * ES;
  for (int64_t v = v0 + (tid >> 5); v < v1; v += nthr >> 5) {
    const int k = (int)(v - v0);
    if (!((named[k >> 5] >> (k & 31)) & 1u)) fill_zero<ES>((char*)a.gt + v * pitch, pitch, tid & 31);
  }
}

// blockDim = (threads of a row, segments of a CTA); segment CTAs come in
// groups of `tiles`, one column tile each.  The rows of a segment come through
// a ring in shared memory (cp.async), eight in flight for every thread: loaded
// into registers, eight at a time, they left room for three CTAs an SM and waited
// on memory for most of the time (60000 tokens of 1024 for 1000 ids: 65 us,
// the ring 51).
constexpr int kSumAhead = 8;  // rows in flight (a power of two)

template <class T, int LAYOUT>
__global__ void __launch_bounds__(256, LAYOUT == NARROW ? 3 : 4) embedding_sum_kernel(SumArgs a) {
  let_next();
  after_previous();
  using L = Tile<T, LAYOUT>;
  constexpr int N = L::N;
  const int64_t role = (int64_t)blockIdx.x;
  if (role >= a.seg_ctas) {
    __shared__ uint32_t named[kMaxZeroRows / 32];
    const int tid = threadIdx.y * blockDim.x + threadIdx.x;
    const int nthr = blockDim.x * blockDim.y;
    const int64_t v0 = (role - a.seg_ctas) * a.zero_rows;
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
    fill_rows<L::ES>(a, named, v0, v1, tid, nthr);
    return;
  }
  const int tile = (int)(role % a.tiles);
  const int64_t seg = role / a.tiles * blockDim.y + threadIdx.y;
  const L t(a.D, tile);
  if (seg >= a.segments) return;  // the whole team
  // warps without columns
  if (t.c - (int)(threadIdx.x & 31) * (LAYOUT == NARROW ? 1 : N) >= a.D) return;
  const int64_t i0 = seg * kEmbedSegment;
  // the segment's ids and the next one's, one per lane of each warp
  const int lane = threadIdx.x & 31;
  const uint32_t none = (uint32_t)a.V;
  const uint2* sorted = a.sorted + i0;
  auto key_of = [&](int i) { return i0 + i >= 0 && i0 + i < a.tokens ? sorted[i].x : none; };
  const uint32_t mine = key_of(lane), next = key_of(kEmbedSegment + lane);
  const uint32_t before = key_of(-1), start = key_of(-1 - kEmbedSegment);
  const uint32_t end = key_of(2 * kEmbedSegment);
  const uint32_t after = __shfl_sync(0xFFFFFFFFu, next, 0);
  uint32_t key = __shfl_sync(0xFFFFFFFFu, mine, 0);
  bool head = i0 > 0 && before == key;
  // tokens [i, m) are this team's: those with an id in the table, without the
  // end of a run of two segments (which the first segment's team adds), and with
  // that of the last run here if it is one
  int i = 0, m = __popc(__ballot_sync(0xFFFFFFFFu, mine < none));
  if (head && start != key && after != key) {
    i = __popc(__ballot_sync(0xFFFFFFFFu, mine == key));
    key = __shfl_sync(0xFFFFFFFFu, mine, i & 31);
    head = false;
  }
  if (i >= m) return;
  const uint32_t last = __shfl_sync(0xFFFFFFFFu, mine, m - 1);
  const bool open = after == last && (end == last || (head && last == key));
  // bit k: a sum ends before token k (at a new run, the next segment, the end)
  const uint32_t previous = __shfl_up_sync(0xFFFFFFFFu, mine, 1);
  uint64_t ends = __ballot_sync(0xFFFFFFFFu, mine != previous);
  if (after == last && !open) {
    m += __popc(__ballot_sync(0xFFFFFFFFu, next == last));
    ends |= uint64_t(1) << kEmbedSegment;
  }
  auto end_of = [&](int k) {  // of the sum that token k is in
    const uint64_t e = ends >> k >> 1;
    return e ? min(m, k + __ffsll((long long)e)) : m;
  };
  F2 acc[N / 2], first[N / 2];
#pragma unroll
  for (int e = 0; e < N / 2; ++e) acc[e] = first[e] = f2(0.0f, 0.0f);
  // the run of `key` ends here (goes_on: but not in the tokens)
  auto flush = [&](bool goes_on) {
    float f[N];
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = e & 1 ? f2_hi(acc[e / 2]) : f2_lo(acc[e / 2]);
    if (head || goes_on) {
      float* p = a.partial + (seg * 2 + (head ? 0 : 1)) * a.D;
      if constexpr (LAYOUT == WIDE) {
        if (t.valid()) {
#pragma unroll
          for (int e = 0; e < N; e += 4)
            *(float4*)(p + t.c + e) = make_float4(f[e], f[e + 1], f[e + 2], f[e + 3]);
        }
      } else {
#pragma unroll
        for (int e = 0; e < N; ++e)
          if (t.col(e) < a.D) p[t.col(e)] = f[e];
      }
      if (!head && tile == 0 && threadIdx.x == 0) a.runs[1 + atomicAdd(a.runs, 1u)] = (uint32_t)seg;
    } else {
      t.store(a.gt, key, f, a.scale);
    }
#pragma unroll
    for (int e = 0; e < N / 2; ++e) acc[e] = f2(0.0f, 0.0f);
  };
  auto add = [&](const typename L::R& r) {
    float f[N];
    L::widen(r, f);
#pragma unroll
    for (int e = 0; e < N / 2; ++e) acc[e] = f2_add(acc[e], f2(f[2 * e], f[2 * e + 1]));
  };
  // before token k, which is not the team's first
  auto turn = [&](int k) {
    if (k == kEmbedSegment) {  // the next segment's part, added on its own
#pragma unroll
      for (int e = 0; e < N / 2; ++e) {
        first[e] = acc[e];
        acc[e] = f2(0.0f, 0.0f);
      }
    } else {
      flush(false);
      key = sorted[k].x;
      head = false;
    }
  };
  if constexpr (LAYOUT == NARROW) {
    constexpr int AHEAD = 8;  // rows in flight
    int stop = end_of(i);
    for (; i < m; i += AHEAD) {
      typename L::R r[AHEAD];
#pragma unroll
      for (int j = 0; j < AHEAD; ++j)
        if (i + j < m && t.valid()) r[j] = t.load(a.g, sorted[i + j].y, a.tokens);
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (i + j >= m) break;
        if (i + j == stop) {
          turn(stop);
          stop = end_of(stop);
        }
        add(r[j]);
      }
    }
  } else {
    // a ring of rows in shared memory, each warp's own columns: 32 granules,
    // and for rows at an offset the one behind them
    __shared__ __align__(16) char ring[kSumAhead][8][33 * 16];
    const int warp = threadIdx.y * (blockDim.x >> 5) + (threadIdx.x >> 5);
    const uint32_t base = smem_addr(&ring[0][warp][0]) + lane * 16;
    auto slot = [&](int k) { return base + ((uint32_t)k % kSumAhead) * (uint32_t)sizeof(ring[0]); };
    const char* column = (const char*)a.g + (int64_t)t.c * L::ES;
    const uint32_t pitch = (uint32_t)a.D * L::ES;
    // elements of row y before its first granule's end (PHASED)
    auto offset = [&](uint32_t y) { return (int)((y & (N - 1)) * (a.D & (N - 1)) & (N - 1)); };
    auto fetch = [&](int k) {
      if (k < m) {
        const uint32_t y = sorted[k].y;
        const char* p = column + (uint64_t)y * pitch;
        if constexpr (LAYOUT == WIDE) {
          if (t.valid()) cp_async16(slot(k), p);
        } else {
          // granules that hold columns of the row (nothing past the tensor)
          const int s = offset(y);
          auto copy = [&](int g) {
            const int c = t.c - s + g * N;
            const int64_t left = (a.tokens - 1 - (int64_t)y) * a.D + (a.D - c);
            if (c < a.D)
              cp_async16_part(slot(k) + g * 16, p + (g * N - s) * L::ES,
                              (uint32_t)(left < N ? left : N) * L::ES);
          };
          copy(0);
          if (s && lane == 31) copy(1);
        }
      }
      cp_async_commit();
    };
    for (int k = 0; k < kSumAhead - 1; ++k) fetch(i + k);
    for (;;) {
      const int stop = end_of(i);
      for (; i < stop; ++i) {
        cp_async_wait<kSumAhead - 2>();
        __syncwarp();  // the warp's copies of row i are there, row i - 1 has been read
        fetch(i + kSumAhead - 1);
        typename L::R r = lds16(slot(i));
        if constexpr (LAYOUT == PHASED) {
          const int s = offset(sorted[i].y);
          if (s) r = shifted<L::ES>(r, lds16(slot(i) + 16), s);
        }
        add(r);
      }
      if (i >= m) break;
      turn(i);
    }
    cp_async_wait<0>();
  }
#pragma unroll
  for (int e = 0; e < N / 2; ++e) acc[e] = f2_add(first[e], acc[e]);
  flush(open);
}

// The parts of each run that crosses segments, added: 128 columns by 8 groups
// of parts per CTA, group q taking parts q, q + 8, ... (the run's first
// segment is part 0), then the groups in order.  A lane takes columns 32 apart.
template <class T>
__global__ void __launch_bounds__(256) embedding_join_kernel(SumArgs a) {
  constexpr int N = 4;
  __shared__ float part[8][N][33];
  after_previous();
  const int lane = threadIdx.x, q = threadIdx.y;
  const int64_t tiles = (a.D + 32 * N - 1) / (32 * N), items = (int64_t)a.runs[0] * tiles;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t seg = a.runs[1 + it / tiles];
    const int c = (int)(it % tiles) * (32 * N) + lane;
    const int64_t i1 = (seg + 1) * kEmbedSegment;
    const uint32_t key = a.sorted[i1 - 1].x;
    // the parts behind the first: segments that start with the key, 256 at a
    // time (they are the first ones, so a count is enough)
    int64_t n = 0;
    for (int more = 256; more == 256; n += more) {
      const int64_t i = i1 + (n + q * 32 + lane) * kEmbedSegment;
      more = __syncthreads_count(i < a.tokens && a.sorted[i].x == key);
    }
    const float* p = a.partial + (seg * 2 + 1) * a.D + c;
    float v[N];
#pragma unroll
    for (int k = 0; k < N; ++k) v[k] = 0.0f;
#pragma unroll 4
    for (int64_t j = q; j <= n; j += 8) {
      const float* at = p + (j ? 2 * j - 1 : 0) * a.D;
#pragma unroll
      for (int k = 0; k < N; ++k)
        if (c + 32 * k < a.D) v[k] = __fadd_rn(v[k], at[32 * k]);
    }
#pragma unroll
    for (int k = 0; k < N; ++k) part[q][k][lane] = v[k];
    __syncthreads();
    // group q < N finishes the lanes' column q
    if (q < N && c + 32 * q < a.D) {
      float f[1] = {part[0][q][lane]};
#pragma unroll
      for (int k = 1; k < 8; ++k) f[0] = __fadd_rn(f[0], part[k][q][lane]);
      f[0] = __fmul_rn(f[0], a.scale);
      st_stream<sizeof(T)>((char*)a.gt + ((int64_t)key * a.D + c + 32 * q) * (int)sizeof(T),
                           Vec<T, (int)sizeof(T)>::narrow(f));
    }
    __syncthreads();  // read before the next item's
  }
}

// Few tokens, unsorted, in one launch: CTA (token, tile) adds the rows of its
// token's id if no earlier token has it; the others fill rows with zeros.
template <class T, int LAYOUT>
__global__ void __launch_bounds__(256) embedding_few_kernel(SumArgs a) {
  using L = Tile<T, LAYOUT>;
  constexpr int N = L::N;
  __shared__ uint32_t named[kMaxZeroRows / 32];  // (zero rows) a bit per row of the table
  __shared__ uint32_t match[kFewTokens / 32];    // (tokens) a bit per token with this id
  const int tid = threadIdx.y * blockDim.x + threadIdx.x, nthr = blockDim.x * blockDim.y;
  const int n = (int)a.tokens;
  const int64_t role = (int64_t)blockIdx.x;
  if (role >= a.seg_ctas) {
    const int64_t v0 = (role - a.seg_ctas) * a.zero_rows;
    const int64_t v1 = v0 + a.zero_rows < a.V ? v0 + a.zero_rows : a.V;
    if (tid < kMaxZeroRows / 32) named[tid] = 0;
    __syncthreads();
    for (int i = tid; i < n; i += nthr) {
      const int64_t k = (int64_t)key_at(a.ids, a.ids64, i, a.V) - v0;
      if (k >= 0 && k < v1 - v0) atomicOr(&named[k >> 5], 1u << (k & 31));
    }
    __syncthreads();
    fill_rows<L::ES>(a, named, v0, v1, tid, nthr);
    return;
  }
  const int me = (int)(role / a.tiles);
  const uint32_t key = key_at(a.ids, a.ids64, me, a.V);
  if (key >= a.V) return;
  for (int i0 = tid & ~31; i0 < kFewTokens; i0 += nthr) {
    const int i = i0 + (tid & 31);
    const uint32_t m = __ballot_sync(0xFFFFFFFFu, i < n && key_at(a.ids, a.ids64, i, a.V) == key);
    if ((tid & 31) == 0) match[i0 >> 5] = m;
  }
  __syncthreads();
  for (int w = 0; w <= me >> 5; ++w) {
    const uint32_t earlier = w < me >> 5 ? 0xFFFFFFFFu : (1u << (me & 31)) - 1u;
    if (match[w] & earlier) return;  // an earlier token adds them
  }
  const L t(a.D, (int)(role % a.tiles));
  if (threadIdx.y > 0) return;  // whole warps
  float acc[N];
#pragma unroll
  for (int e = 0; e < N; ++e) acc[e] = 0.0f;
  for (int w = me >> 5; w < kFewTokens / 32; ++w) {
    uint32_t m = match[w];
    while (m) {
      constexpr int AHEAD = 4;  // rows in flight
      typename L::R r[AHEAD];
      int got = 0;
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (!m) continue;
        const int i = w * 32 + __ffs(m) - 1;
        m &= m - 1;
        if (t.valid()) r[j] = t.load(a.g, i, a.tokens);
        got = j + 1;
      }
#pragma unroll
      for (int j = 0; j < AHEAD; ++j) {
        if (j >= got || !t.valid()) continue;
        float f[N];
        L::widen(r[j], f);
#pragma unroll
        for (int e = 0; e < N; ++e) acc[e] = __fadd_rn(acc[e], f[e]);
      }
    }
  }
  t.store(a.gt, key, acc, a.scale);
}

template <class T, int LAYOUT>
cudaError_t launch_sums(const DeviceInfo& dev, SumArgs a, cudaStream_t s) {
  const int64_t row_bytes = (int64_t)a.D * (int)sizeof(T);
  const int n = tile_columns((int)sizeof(T), LAYOUT);
  const int tx = row_threads(a.D, n), ty = 256 / tx;
  a.tiles = (int)row_tiles(a.D, n);
  // about 128 KB of zeros per CTA
  a.zero_rows = (int)std::min<int64_t>(kMaxZeroRows, std::max<int64_t>(1, (128 << 10) / row_bytes));
  const int64_t zero_ctas = (a.V + a.zero_rows - 1) / a.zero_rows;
  const bool few = a.tokens <= kFewTokens;
  a.seg_ctas = (few ? a.tokens : (a.segments + ty - 1) / ty) * a.tiles;
  if (a.seg_ctas + zero_ctas > 0x7FFFFFFF) return cudaErrorInvalidConfiguration;
  const unsigned grid = (unsigned)(a.seg_ctas + zero_ctas);
  if (few) {
    embedding_few_kernel<T, LAYOUT><<<grid, dim3(tx, ty), 0, s>>>(a);
    return cudaGetLastError();
  }
  const cudaError_t e = launch_after(embedding_sum_kernel<T, LAYOUT>, grid, dim3(tx, ty), 0, s, a);
  if (e != cudaSuccess) return e;
  const int64_t most = (a.segments - 1) * ((a.D + 127) / 128);
  return launch_after(embedding_join_kernel<T>, (unsigned)std::min<int64_t>(most, 8 * dev.sm_count),
                      dim3(32, 8), 0, s, a);
}

cudaError_t launch_sort(const DeviceInfo& dev, SortArgs a, cudaStream_t s) {
  a.ctas = a.tokens > 4096 ? kSortCluster : 1;
  const int64_t warps = (int64_t)a.ctas * kSortWarps;
  a.per_warp = ((a.tokens + warps - 1) / warps + 31) / 32 * 32;
  const size_t smem = (size_t)kSortWarps * (1 << a.bits) * 4;
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)sort_kernel, dev, opted);
  if (e != cudaSuccess) return e;
  return launch_cluster(sort_kernel, (unsigned)a.ctas, kSortWarps * 32, smem, s, a);
}

template <class T, class Fn>
cudaError_t with_layout(int layout, Fn&& fn) {
  return layout == WIDE     ? fn(TypeTag<T>{}, std::integral_constant<int, WIDE>{})
         : layout == PHASED ? fn(TypeTag<T>{}, std::integral_constant<int, PHASED>{})
                            : fn(TypeTag<T>{}, std::integral_constant<int, NARROW>{});
}
template <class Fn>
cudaError_t with_tile(int dtype, int layout, Fn&& fn) {
  return dtype == 0   ? with_layout<__nv_bfloat16>(layout, fn)
         : dtype == 1 ? with_layout<__half>(layout, fn)
                      : with_layout<float>(layout, fn);
}

}  // namespace

cudaError_t launch_embedding(int dtype, int layout, const EmbedArgs& a, cudaStream_t s) {
  return with_tile(dtype, layout, [&](auto tt, auto w) -> cudaError_t {
    using T = typename decltype(tt)::type;
    constexpr int LAYOUT = decltype(w)::value;
    const int n = tile_columns((int)sizeof(T), LAYOUT);
    const int tx = row_threads(a.D, n), ty = 256 / tx;
    const int64_t grid = std::min<int64_t>((a.tokens + ty - 1) / ty, int64_t(1) << 30);
    // PHASED: a row reaches into one granule more
    const int tiles = (int)((a.D + (LAYOUT == PHASED ? n - 1 : 0) + tx * n - 1) / (tx * n));
    embedding_kernel<T, LAYOUT><<<(unsigned)grid, dim3(tx, ty), 0, s>>>(a, tiles);
    return cudaGetLastError();
  });
}

cudaError_t launch_embedding_grad(const DeviceInfo& dev, int dtype, int layout,
                                  const EmbedGradArgs& a, cudaStream_t s) {
  SumArgs m = {};
  m.gt = a.gt;
  m.g = a.g;
  m.ids = a.ids;
  m.ids64 = a.ids64;
  m.partial = a.partial;
  m.runs = a.runs;
  m.tokens = a.tokens;
  m.V = a.V;
  m.segments = embed_segments(a.tokens);
  m.D = a.D;
  m.scale = a.scale;
  if (a.tokens > kFewTokens) {
    SortArgs q = {};
    q.ids = a.ids;
    q.ids64 = a.ids64;
    q.tokens = a.tokens;
    q.V = a.V;
    q.pairs[0] = a.pairs[0];
    q.pairs[1] = a.pairs[1];
    q.runs = a.runs;
    int bits = 1;  // of the keys 0 .. V
    while (bits < 32 && (a.V >> bits) != 0) ++bits;
    q.passes = (bits + kSortBits - 1) / kSortBits;
    q.bits = (bits + q.passes - 1) / q.passes;
    const cudaError_t e = launch_sort(dev, q, s);
    if (e != cudaSuccess) return e;
    m.sorted = a.pairs[(q.passes - 1) & 1];
  }
  return with_tile(dtype, layout, [&](auto tt, auto w) -> cudaError_t {
    return launch_sums<typename decltype(tt)::type, decltype(w)::value>(dev, m, s);
  });
}

}  // namespace dit
