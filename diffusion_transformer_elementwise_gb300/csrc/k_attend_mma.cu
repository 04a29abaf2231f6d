// k_attend_mma.cu -- attention of one new token per sequence over a paged
// cache of 16-bit or E4M3 rows, on the tensor cores (sm_103a).
//
//   s = scale q.k,  m = max s,  l = sum 2^(s - m),  o = sum 2^(s - m) v
// in one pass over the tokens, with s in powers of two (scale times log2 e).
//
// What bounds it is memory: each key and value is read once for all query heads
// of its key head.  A warp takes tiles of 32 tokens, each two products of 16 x 8 x 16
// steps (mma.sync): S (tokens x heads) = K Q^T, then O (columns x heads) += V^T P,
// so that up to eight heads of a key head fill a product, and sixteen two.  The
// 5th generation's instructions want 64 or 128 rows and their operands in shared
// memory in a layout of their own; here the tensor cores are busy 8 to 22 % of the time,
// so that what they could do beyond does not count.
// Measured (GPU time with the join): one sequence of 131072 tokens x 8 heads of 128, bf16, 88.6 us for 537 MB, 6.1
// TB/s or 89 % of a copy's rate: 6.9 TB/s while it lasts and some 9 us for lengths, pages, first rows and joins one
// after the other.  128 sequences of 8 to 8192 tokens in E4M3 80 us for 422 MB (5.3 TB/s; with the conversion of codes
// some 730 instructions a tile and head, 45 % of the issue slots).  64 x 2048 tokens fp32 189 us, 5.7 TB/s.
//
// The contraction index of a product may be permuted if both operands agree, and so may
// the rows of O.  So every lane's operands are 16 contiguous bytes of a row: of keys,
// lane (g, c) = (lane / 4, lane % 4) has bytes 16 c of each 64 of tokens g and g + 8; of
// values, bytes 16 g of each 128 of the tokens 2c, 2c + 1, 2c + 8, 2c + 9 (or others in
// their place).  They come through the warp's own stages in shared memory (cp.async): no bank
// conflicts, no barriers but the warp's, no transposition but of P (two movmatrix).
//
// Every warp has a part of the line of tiles (dit_attend.cuh) and finishes its
// segments alone; what it shares with others it leaves in the workspace, where the CTA's warps
// join what the CTA holds all of, and the second kernel the rest.
#include "dit_attend.cuh"

namespace dit {
namespace {

__device__ __forceinline__ void cp_async4_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

struct Tf32 {};

// d += a b: a 16 x 16, b 16 x 8, of M (Tf32: 16 x 8 and 8 x 8).
template <class M>
__device__ __forceinline__ void mma(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1) {
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else if constexpr (std::is_same<M, Tf32>::value)
    asm("mma.sync.aligned.m16n8k8.row.col.f32.tf32.tf32.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}
template <int N>
__device__ __forceinline__ void add(float (&d)[N], const float (&x)[N]) {
#pragma unroll
  for (int i = 0; i < N; ++i) d[i] = __fadd_rn(d[i], x[i]);
}
// fp32 as the nearest tf32 and the rest, of which the tensor cores read the first 11 bits
struct Split {
  uint32_t high, low;
  __device__ __forceinline__ explicit Split(uint32_t x) {
    asm("cvt.rna.tf32.f32 %0, %1;" : "=r"(high) : "f"(__uint_as_float(x)));
    low = __float_as_uint(__fadd_rn(__uint_as_float(x), -__uint_as_float(high)));
  }
};
// an 8 x 8 matrix of 16-bit numbers, a row's pairs over four lanes, transposed
__device__ __forceinline__ uint32_t transposed(uint32_t x) {
  uint32_t y;
  asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(y) : "r"(x));
  return y;
}
// the larger of both upper and of both lower halves
__device__ __forceinline__ uint32_t max_halves(uint32_t x, uint32_t y) {
  uint32_t z;
  asm("max.u16x2 %0, %1, %2;" : "=r"(z) : "r"(x), "r"(y));
  return z;
}
__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {  // the low two codes
  uint32_t h;
  asm("{ .reg .b16 c, d; mov.b32 {c, d}, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(h) : "r"(codes));
  return h;
}
// the sum or maximum over the lanes of one c
__device__ __forceinline__ float column_sum(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = __fadd_rn(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}
__device__ __forceinline__ float column_max(float v) {
#pragma unroll
  for (int o = 4; o < 32; o <<= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
  return v;
}

// Where chunk c (16 bytes) of row t is in a tile of keys or values: the rows lie one after the other, and each
// 128 bytes of them have their chunks exchanged so that the eight lanes of a quarter of a warp
// find theirs in eight different places, as the copies that write them do.  (Copies that spread a
// line over the tile instead, to the order of the reading lanes, left the memory at 4.0 of 7.0 TB/s.)
// Keys are read as chunks 0 to 3 or 4 to 7 of two rows by such eight lanes, values as two
// chunks of four rows; with rows 0 5 2 7 4 1 6 3 in the place of 0 to 7 (chunk numbers change by the row's),
// both do.  Rows of 64 bytes: two of them share 128.
template <int ROW, bool VALUE>
__device__ __forceinline__ uint32_t chunk_xor(int t) {
  return (ROW >= 128 ? t & 7 : VALUE ? t / 2 * 2 & 7 : t / 2 & 3) * 16;
}
template <int ROW, bool VALUE>
__device__ __forceinline__ uint32_t chunk_at(int t, int c) {
  return (t * ROW + c * 16) ^ chunk_xor<ROW, VALUE>(t);
}
// chunk 4 p + c of the row whose chunk c is at `key`
template <int ROW>
__device__ __forceinline__ uint32_t key_at(uint32_t key, int p) {
  return (key ^ (p & 1) * 64) + p / 2 * 128;
}

// T: the queries' type; FP8: an E4M3 cache; DP: columns, D rounded up (the rest is zero); NB: blocks of
// eight heads.  With fp32 queries every product is one of two parts each (SPLIT): keys and values of fp32 as two
// tf32 numbers, queries and weights too, or, over an E4M3 cache, as two fp16 numbers; what is left out is 2^-22 of
// a product.  The tensor cores cut their sums off where fp32 rounds them: such sums are kept short (a product of the
// high parts, or a tile) and added up outside (lse over 128 columns is 8e-8 off so, in long sums 6.5e-7).
template <class T, bool FP8_, int DP_, int NB_>
struct Shape {
  static constexpr bool FP8 = FP8_, SPLIT = sizeof(T) == 4, TF32 = SPLIT && !FP8;
  static constexpr int DP = DP_, NB = NB_;
  using M = typename std::conditional<FP8, __half, typename std::conditional<TF32, Tf32, T>::type>::type;  // of the products
  static constexpr bool HALF = std::is_same<M, __half>::value;  // weights in fp16
  static constexpr int ES = FP8 ? 1 : (int)sizeof(T);
  static constexpr int ROW = DP * ES;                 // bytes
  static constexpr int KP = ROW / 64;                 // 16-byte pieces of a key that a lane has
  static constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16;  // bytes of a piece of a value
  static constexpr int VP = ROW / 8 / VB;             // pieces of a value that a lane has
  static constexpr int CE = VB / ES;                  // columns of such a piece
  static constexpr int PER = 16 / ES;                 // columns of a key's piece
  static constexpr int KN = FP8 ? 4 : 2;              // products of a key's piece
  static constexpr int LOAD = 16 / (int)sizeof(T);    // queries' columns of 16 bytes
  static constexpr int MB = ROW >= 512 || (NB == 2 && ROW >= 256) ? 1 : 2;  // blocks of 16 tokens of a stage
  static constexpr int TOKENS = 16 * MB, PARTS = kTile / TOKENS;  // stages of a tile
  static constexpr int STAGE = 2 * TOKENS * ROW;      // bytes of a warp's stage: keys and values
  // behind them: their scales (E4M3), and which tokens count
  static constexpr int EXTRA = FP8 ? 8 * TOKENS + 128 : 128;
  // As many warps as registers and two stages of each in 220 KB let in.  Long sequences are as fast with fewer and more
  // stages (bf16, D = 128: six warps of two, four of three), E4M3 wants the warps (12: 96.7 us for 553 MB, 8: 100.9).
  static constexpr int WARPS = ROW <= 64 && NB == 1 && !SPLIT ? 16
                               : ROW <= 128                   ? (NB == 1 && !SPLIT ? 12 : 8)
                               : ROW <= 256                   ? (NB == 1 ? 6 : 8)
                               : ROW <= 512                   ? 6
                                                              : 3;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int FIT = (220 * 1024) / (WARPS * (STAGE + EXTRA));
  static constexpr int STAGES = FIT > 6 ? 6 : FIT;
  static constexpr int SMEM = STAGES * WARPS * (STAGE + EXTRA);
  static_assert(STAGES >= 2, "a stage in flight and one in use");
  static_assert(WARPS <= attend_warps(DP), "the workspace has room for their parts");
};

// The units of fp16 weights.  fp16 holds eleven digits down to 2^-14 and fewer below, so weights are brought near its
// top: of an fp16 cache 2^14 of them (the largest is one).  Over an E4M3 cache a weight is a token's share times its
// value's scale, and what counts is the largest of those: a large scale with next to no share must not push the others
// down, so each head has a bound of its own on them, which falls as the maximum of the logits rises and its older tokens'
// shares fall.  It is held as the upper half of an fp32 number (rounded up), two heads a word; the unit is 2^-14 of the
// power of two above it.  (With one bound on the scales alone, a row of values 2^40 times the others' left nothing of
// them, whatever its own share, and a first token of e^16 times the others' share and 2^-10 of their values left
// the output 4 % off.)  64 x 4096 tokens in E4M3: 97.6 us as with the one bound; sixteen query heads a key head 55.7
// where that took 55.0, fp32 queries 105.5 where 102.4.
struct Unit {
  static constexpr uint32_t kLeast = 0x0700, kMost = 0x7EFF;  // so that what follows are normal numbers
  // 2^14 over the power of two above bound j of a word, and its reciprocal
  __device__ __forceinline__ static float factor(uint32_t bounds, int j) {
    return __uint_as_float(0x85800000u - ((j ? bounds : bounds << 16) & 0x7F800000u));
  }
  __device__ __forceinline__ static float value(uint32_t bounds, int j) {
    return __uint_as_float(((j ? bounds : bounds << 16) & 0x7F800000u) - 0x06800000u);
  }
  // Bound j of the next word, from a word, the factor that the logits' maximum leaves of older shares, and the largest
  // of this tile's; f becomes the factor from old units to new ones.
  __device__ __forceinline__ static uint32_t moved(uint32_t bounds, uint32_t most, int j, float& f) {
    const uint32_t was = j ? bounds >> 16 : bounds & 0xFFFFu, tile = j ? most >> 16 : most & 0xFFFFu;
    uint32_t now = (__float_as_uint(__fmul_rn(__uint_as_float(was << 16), f)) + 0xFFFFu) >> 16;
    if (tile > now) now = tile | 0x7Fu;  // (all below the next power of two: seldom raised)
    now = max(min(now, kMost), kLeast);
    const int up = (int)(was >> 7) - (int)(now >> 7) + 127;
    f = __fmul_rn(f, __uint_as_float((uint32_t)max(min(up, 253), 1) << 23));
    return now << (16 * j);
  }
};

// Units of a segment beside its tiles (128 sequences of 8 to 8192 tokens, E4M3: 1 80.0 us, 2 78.8, 4 78.1), and the
// smallest part of a warp.
constexpr int kExtra = 4;
constexpr int kLeast = 1;

struct MmaArgs {
  AttendArgs a;
  Divisor page;         // page_size
  int page_rows;        // rows of D from page to page
  bool whole;           // no page ends within half a tile
  float* warp_partial;  // [ctas][warps][2][rows][D]: the unscaled outputs of segments that warps share
};

// a part of a segment in the workspace: maxima, sums, and the unscaled output
struct Piece {
  float *m, *l, *o;
  __device__ __forceinline__ Piece(float* base, int64_t i, int rows, int D)
      : m(base + i * rows * (D + 2)), l(m + rows), o(l + rows) {}
};

template <class T, class S>
__global__ void __launch_bounds__(S::THREADS, 1) attend_mma_kernel(const __grid_constant__ MmaArgs args) {
  using M = typename S::M;
  constexpr bool FP8 = S::FP8;
  constexpr int NB = S::NB, NCE = S::CE / 2, MB = S::MB, TOKENS = S::TOKENS;
  constexpr bool SPLIT = S::SPLIT, TF32 = S::TF32, HALF = S::HALF;
  // Parts of a weight.  Over E4M3 one fp16 number leaves an output that is itself rounded to fp16 1.4 times
  // as far off as it need be (3.1e-4 of 2.1e-4), so fp16 queries have two there as well as fp32 ones: 64 x 4096 tokens
  // 98.6 us where one takes 97.6.  bf16's own rounding hides it (1 %), as the types' own do over their caches (1 to 7 %), where
  // a second part would also make NaN of an infinite value, as infinity times 0 or less.
  constexpr int WN = FP8 && !std::is_same<T, __nv_bfloat16>::value ? 2 : 1;
  __shared__ Plan<S::THREADS> plan;
  // the segments that warps share: which (or -1), their maxima and sums, and whether the first goes on in
  // the next warp's part
  __shared__ int64_t owner[S::WARPS][2];
  __shared__ float piece_m[S::WARPS][2][8 * NB], piece_l[S::WARPS][2][8 * NB];
  __shared__ bool open[S::WARPS];
  __shared__ float factors[S::WARPS][S::WARPS + 1];  // of the pieces that a warp joins
  extern __shared__ __align__(1024) unsigned char space[];
  const AttendArgs& a = args.a;
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gl = lane >> 2, cl = lane & 3;
  const int D = (int)a.c.D;
  const int blocks = (a.group + 8 * NB - 1) / (8 * NB);
  const Line line{(int)a.c.heads * blocks, kExtra};
  const int slot_rows = min(a.group, 8 * NB);
  unsigned char* stages = space + warp * S::STAGES * (S::STAGE + S::EXTRA);
  const uint32_t stages_at = smem_addr(stages);
  // Rows of a product of tokens are not tokens g but tg, and g + 8 but tg + 8: see chunk_at.
  const int tg = gl ^ ((gl & 1) << 2);

  after_previous();
  const int64_t total = line.total(a, plan);
  const int64_t warps = (int64_t)gridDim.x * S::WARPS;
  const int64_t per = max((int64_t)kLeast, divided(total + warps - 1, warps));
  const int64_t begin = min((blockIdx.x * (int64_t)S::WARPS + warp) * per, total), end = min(begin + per, total);
  const int64_t cta_begin = min(blockIdx.x * (int64_t)S::WARPS * per, total);
  if (tid < 2) a.owner[2 * blockIdx.x + tid] = -1;
  let_next();
  if (cta_begin >= total) return;
  const Mark mark = a.B <= S::THREADS ? Mark{0, 0} : line.find(a, cta_begin, plan);
  const int64_t slot = (blockIdx.x * (int64_t)S::WARPS + warp) * 2;
  if (lane < 2) owner[warp][lane] = -1;

  if (begin < end) {
    const Mark mine = a.B <= S::THREADS ? line.find(a, begin, plan) : line.find_from(a, begin, mark);

    // ----- copies, some tiles ahead -----
    Walk ahead(a, line, begin, end, mine);
    Segment ag = {};
    bool more = ahead.next(a, line, ag);
    int tile = ag.first * S::PARTS, head = more ? ag.s / blocks : 0;  // (tile: of TOKENS)
    int page = -1, place = 0;  // of token lane % TOKENS of that tile
    auto look = [&]() {
      if (more && tile >= ag.last * S::PARTS) {
        more = ahead.next(a, line, ag);
        tile = ag.first * S::PARTS;
        head = ag.s / blocks;
      }
      page = -1;
      if (more) {
        const int t = tile * TOKENS + lane % TOKENS;
        if (t >= ag.lo && t < ag.hi) {
          const int n = (int)quotient(t, args.page);
          place = t - n * (int)args.page.d;
          page = a.pages[ag.b * a.pages_stride + n];
        }
      }
    };
    // A copy takes 512 bytes as they lie in memory: lane l has chunk l % LPR of row l / LPR of RPC, or of
    // rows of more than 512 bytes chunk l of one of CPR parts.
    constexpr int LPR = S::ROW < 512 ? S::ROW / 16 : 32, RPC = 32 / LPR, CPR = S::ROW > 512 ? S::ROW / 512 : 1;
    constexpr int COPIES = TOKENS / RPC * CPR;
    const int row_bytes = D * S::ES;
    const int my_row = lane / LPR, my_chunk = lane % LPR;
    const uint32_t k_to = chunk_at<S::ROW, false>(my_row, my_chunk), v_to = chunk_at<S::ROW, true>(my_row, my_chunk);
    auto issue = [&](int stage) {
      if (more) {
        const uint32_t to = stages_at + stage * (S::STAGE + S::EXTRA);
        asm volatile("" : "+r"(page));  // (not waited for before it is needed)
        const bool there = page >= 0 && page < a.c.pages;
        const int in_page = head * (int)args.page.d + place;
        // (of a token that does not count nothing is read, and zeros are written)
        const int row = there ? page * args.page_rows + in_page : -1;
        const uint32_t count = __ballot_sync(0xFFFFFFFFu, there);
        // copy n: of the row that starts at element offset `at` in bytes, or of none
        auto copy = [&](int n, int64_t at, bool on) {
          const int chunk = (n % CPR * 32 + my_chunk) * 16;
          const bool any = on && chunk < row_bytes;
          at = any ? at + chunk : 0;
          // chunk_at of the copy's row: its part in n moves by constants
          const int t = n / CPR * RPC;
          const uint32_t k = (to + k_to) ^ chunk_xor<S::ROW, false>(t), v = (to + v_to) ^ chunk_xor<S::ROW, true>(t);
          cp_async16_part(k + n * 512, (const char*)a.c.k + at, any ? 16 : 0);
          cp_async16_part(v + S::STAGE / 2 + n * 512, (const char*)a.c.v + at, any ? 16 : 0);
        };
        if (count == 0xFFFFFFFFu && args.whole) {  // 16 rows each that lie side by side
#pragma unroll
          for (int h = 0; h < MB; ++h) {
            int64_t at = (int64_t)(__shfl_sync(0xFFFFFFFFu, row, 16 * h) + my_row) * row_bytes;
#pragma unroll
            for (int n = 0; n < COPIES / MB; ++n) {
              copy(h * (COPIES / MB) + n, at, true);
              if (n % CPR == CPR - 1) at += RPC * row_bytes;
            }
          }
        } else {
#pragma unroll
          for (int n = 0; n < COPIES; ++n) {
            const int r = __shfl_sync(0xFFFFFFFFu, row, n / CPR * RPC + my_row);
            copy(n, (int64_t)r * row_bytes, r >= 0);
          }
        }
        if constexpr (FP8) {
          const int64_t at = there ? page * a.c.scale_stride + in_page : 0;
          const uint32_t dst = to + S::STAGE + lane * 4;  // MB = 1: the upper lanes have the same tokens' values
          cp_async4_part(dst, (MB == 1 && lane >= 16 ? a.c.v_scales : a.c.k_scales) + at, there ? 4 : 0);
          if constexpr (MB == 2) cp_async4_part(dst + 4 * TOKENS, a.c.v_scales + at, there ? 4 : 0);
        }
        if (lane == 0)
          *(uint32_t*)(stages + stage * (S::STAGE + S::EXTRA) + S::STAGE + S::EXTRA - 16) = count;
        ++tile;
        look();
      }
      cp_async_commit();
    };
    look();
#pragma unroll
    for (int s = 0; s < S::STAGES - 1; ++s) issue(s);

    // ----- products -----
    // where the lane's first key is, and its values of tokens 2c and 2c + 1 (as rows of a product)
    const uint32_t key = chunk_at<S::ROW, false>(tg, cl);
    uint32_t value[2];
#pragma unroll
    for (int i = 0; i < 2; ++i) {
      // (TF32: of tokens c and c + 4)
      const int t = TF32 ? cl ^ (cl & 1) << 2 ^ i << 2 : (2 * cl + i) ^ (i << 2);
      value[i] = S::VB == 16 ? chunk_at<S::ROW, true>(t, gl) : chunk_at<S::ROW, true>(t, gl >> 1) + (gl & 1) * 8;
    }
    int stage = 0;
    Walk walk(a, line, begin, end, mine);
    Segment g;
    while (walk.next(a, line, g)) {
      const int key_head = g.s / blocks, row0 = (g.s - key_head * blocks) * 8 * NB;
      const int rows = min(8 * NB, a.group - row0);
      const int h0 = key_head * a.group + row0;

      // queries of head 8 nb + g, in the order of the keys' bytes, and what the products of heads 8 nb + 2c and
      // the next are multiplied by
      // (over an E4M3 cache as fp16, by a power of two that brings the head's largest below 2^14; SPLIT: the rest too)
      constexpr int LOADS = S::KP * S::PER / S::LOAD, SUB = S::PER / S::LOAD, QN = SPLIT && FP8 ? 2 : 1;
      uint32_t q[QN][NB][S::KP * S::KN][2];
      float factor[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) {
        const bool real = gl + 8 * nb < rows;
        const T* from = (const T*)a.q.p + g.b * a.q.token + (int64_t)(h0 + gl + 8 * nb) * a.q.head;
        float by = __fmul_rn(a.scale, 1.4426950408889634f);
        Raw<16> raw[LOADS];
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          const int c = (i / SUB * 4 + cl) * S::PER + i % SUB * S::LOAD;
          raw[i] = Raw<16>{};
          // (not by the read-only path: the kernel before, which wrote them, may have run beside this one)
          if (real && c < D) raw[i] = ld_stream<16>(from + c);
        }
        float up = 1.0f;
        if constexpr (FP8 && !std::is_same<T, __half>::value) {
          float most = 0.0f;
#pragma unroll
          for (int i = 0; i < LOADS; ++i) {
            float f[S::LOAD];
            Vec<T, 16>::widen(raw[i], f);
#pragma unroll
            for (int k = 0; k < S::LOAD; ++k) most = max_nan(most, fabsf(f[k]));
          }
          most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
          most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
          int e = (int)(__float_as_uint(most) >> 23) - 127;
          e = most == 0.0f || !isfinite(most) ? 13 : max(e, -100);
          up = __uint_as_float((uint32_t)(13 - e + 127) << 23);
          by = __fmul_rn(by, __uint_as_float((uint32_t)(e - 13 + 127) << 23));
        }
#pragma unroll
        for (int j = 0; j < 2; ++j) factor[nb][j] = __shfl_sync(0xFFFFFFFFu, by, 4 * (2 * cl + j));
#pragma unroll
        for (int i = 0; i < LOADS; ++i) {
          if constexpr (FP8) {
            float f[S::LOAD];
            Vec<T, 16>::widen(raw[i], f);
#pragma unroll
            for (int k = 0; k < S::LOAD / 2; ++k) {
              const float x = __fmul_rn(f[2 * k], up), y = __fmul_rn(f[2 * k + 1], up);
              const __half2 h = __floats2half2_rn(x, y);
              uint32_t(&to)[2] = q[0][nb][(i * S::LOAD + 2 * k) / 4];
              to[k & 1] = *(const uint32_t*)&h;
              if constexpr (SPLIT) {
                const float2 back = __half22float2(h);
                q[QN - 1][nb][(i * S::LOAD + 2 * k) / 4][k & 1] =
                    Pair<__half>::narrow(f2(__fadd_rn(x, -back.x), __fadd_rn(y, -back.y)));
              }
            }
          } else {
#pragma unroll
            for (int k = 0; k < 4; ++k) q[0][nb][2 * i + k / 2][k & 1] = raw[i].w[k];
          }
        }
      }

      // o[nb][p][i]: columns (8 p + g) CE + 2 i (twice) and the next, heads 8 nb + 2c and the next
      float o[NB][S::VP][NCE][4] = {};
      float m[NB][2], l[NB][2];
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) m[nb][j] = -INFINITY, l[nb][j] = 0.0f;
      uint32_t bound[NB];  // E4M3: see Unit; o is in these units
#pragma unroll
      for (int nb = 0; nb < NB; ++nb) bound[nb] = Unit::kLeast * 0x10001u;

      for (int n = (g.last - g.first) * S::PARTS; n > 0; --n) {
        cp_async_wait<S::STAGES - 2>();
        __syncwarp();
        const uint32_t from = stages_at + stage * (S::STAGE + S::EXTRA);
        const unsigned char* extra = stages + stage * (S::STAGE + S::EXTRA) + S::STAGE;
        // bits 0, 8, 16 and 24: the lane's tokens tg, tg + 8 of both halves of the tile
        const uint32_t count = *(const uint32_t*)(extra + S::EXTRA - 16) >> tg;
        const float* scales = (const float*)extra;

        // pieces of keys, KG at a time, in registers before the products that wait for each other
        constexpr int KG = S::KP < 4 ? S::KP : 4;
        float s[NB][MB][4] = {}, rest[TF32 ? NB : 1][TF32 ? MB : 1][4] = {};
#pragma unroll
        for (int p0 = 0; p0 < S::KP; p0 += KG) {
          Raw<16> x[MB][KG], y[MB][KG];
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int p = 0; p < KG; ++p) {
              const uint32_t at = from + key_at<S::ROW>(key, p0 + p) + 16 * b * S::ROW;
              x[b][p] = lds16(at);
              y[b][p] = lds16(at + 8 * S::ROW);
            }
          if (p0 == 0) issue(stage == 0 ? S::STAGES - 1 : stage - 1);
#pragma unroll
          for (int p = 0; p < KG; ++p) {
#pragma unroll
            for (int i = 0; i < S::KN; ++i)
#pragma unroll
              for (int b = 0; b < MB; ++b) {
                const Raw<16>&u = x[b][p], &v = y[b][p];
                const int step = (p0 + p) * S::KN + i;
                if constexpr (TF32) {
                  const Split a0(u.w[2 * i]), a1(v.w[2 * i]), a2(u.w[2 * i + 1]), a3(v.w[2 * i + 1]);
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    const Split b0(q[0][nb][step][0]), b1(q[0][nb][step][1]);
                    mma<M>(rest[nb][b], a0.low, a1.low, a2.low, a3.low, b0.high, b1.high);
                    mma<M>(rest[nb][b], a0.high, a1.high, a2.high, a3.high, b0.low, b1.low);
                    float sum[4] = {};
                    mma<M>(sum, a0.high, a1.high, a2.high, a3.high, b0.high, b1.high);
                    add(s[nb][b], sum);
                  }
                } else {
                  const uint32_t a0 = FP8 ? e4m3x2_to_half2(u.w[i]) : u.w[2 * i];
                  const uint32_t a1 = FP8 ? e4m3x2_to_half2(v.w[i]) : v.w[2 * i];
                  const uint32_t a2 = FP8 ? e4m3x2_to_half2(u.w[i] >> 16) : u.w[2 * i + 1];
                  const uint32_t a3 = FP8 ? e4m3x2_to_half2(v.w[i] >> 16) : v.w[2 * i + 1];
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (SPLIT) {
                      float sum[4] = {};
                      mma<M>(sum, a0, a1, a2, a3, q[QN - 1][nb][step][0], q[QN - 1][nb][step][1]);
                      mma<M>(sum, a0, a1, a2, a3, q[0][nb][step][0], q[0][nb][step][1]);
                      add(s[nb][b], sum);
                    } else {
                      mma<M>(s[nb][b], a0, a1, a2, a3, q[0][nb][step][0], q[0][nb][step][1]);
                    }
                  }
                }
              }
          }
        }
        if constexpr (TF32) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int b = 0; b < MB; ++b) add(s[nb][b], rest[nb][b]);
        }
        // the first pieces of the values, on their way meanwhile
        const uint32_t values = from + S::STAGE / 2;
        auto load = [&](int b, int i, int p) {
          const uint32_t at = values + value[i & 1] + (16 * b + (i >> 1) * 8) * S::ROW + p * 128;
          if constexpr (S::VB == 16)
            return lds16(at);
          else
            return lds8(at);
        };
        // (pieces in the order p, b)
        constexpr int VN = S::VP * MB, VG = VN < 2 ? VN : 2;
        Raw<S::VB> v[VG][4];
#pragma unroll
        for (int n = 0; n < VG; ++n)
#pragma unroll
          for (int i = 0; i < 4; ++i) v[n][i] = load(n % MB, i, n / MB);
        float ks[2 * MB], vs[2 * MB];  // scales of the lane's tokens
        if constexpr (FP8) {
#pragma unroll
          for (int t = 0; t < 2 * MB; ++t) ks[t] = scales[tg + 8 * t], vs[t] = scales[TOKENS + tg + 8 * t];
        }
        float f[NB][2];
        bool moved = false;
#pragma unroll
        for (int nb = 0; nb < NB; ++nb) {
#pragma unroll
          for (int j = 0; j < 2; ++j) {
            float most = m[nb][j];
#pragma unroll
            for (int t = 0; t < 2 * MB; ++t) {
              float& x = s[nb][t / 2][2 * (t & 1) + j];
              if constexpr (FP8) x = __fmul_rn(x, ks[t]);
              x = count >> (8 * t) & 1 ? __fmul_rn(x, factor[nb][j]) : -INFINITY;
              most = fmaxf(most, x);
            }
            most = column_max(most);
            const float base = most == -INFINITY ? 0.0f : most;
            f[nb][j] = exp2_fast(__fadd_rn(m[nb][j], -base));
            moved = moved || most != m[nb][j];
            m[nb][j] = most;
            float sum = 0.0f;
#pragma unroll
            for (int t = 0; t < 2 * MB; ++t) {
              float& x = s[nb][t / 2][2 * (t & 1) + j];
              x = exp2_fast(__fadd_rn(x, -base));
              sum = __fadd_rn(sum, x);
            }
            l[nb][j] = __fmaf_rn(l[nb][j], f[nb][j], sum);
          }
        }
        uint32_t top[NB];  // E4M3: the upper halves of the largest magnitudes
        if constexpr (FP8) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb) {
            top[nb] = 0;
#pragma unroll
            for (int t = 0; t < 2 * MB; ++t) {
              float &x = s[nb][t / 2][2 * (t & 1)], &y = s[nb][t / 2][2 * (t & 1) + 1];
              x = __fmul_rn(x, vs[t]);
              y = __fmul_rn(y, vs[t]);
              top[nb] = max_halves(top[nb], __byte_perm(__float_as_uint(x), __float_as_uint(y), 0x7632) & 0x7FFF7FFFu);
            }
#pragma unroll
            for (int i = 4; i < 32; i <<= 1) top[nb] = max_halves(top[nb], __shfl_xor_sync(0xFFFFFFFFu, top[nb], i));
            moved = moved || max_halves(top[nb], bound[nb]) != bound[nb];
          }
        }
        if (__any_sync(0xFFFFFFFFu, moved)) {
          if constexpr (FP8) {
#pragma unroll
            for (int nb = 0; nb < NB; ++nb)
              bound[nb] = Unit::moved(bound[nb], top[nb], 0, f[nb][0]) | Unit::moved(bound[nb], top[nb], 1, f[nb][1]);
          }
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int p = 0; p < S::VP; ++p)
#pragma unroll
              for (int i = 0; i < NCE; ++i)
#pragma unroll
                for (int k = 0; k < 4; ++k) o[nb][p][i][k] = __fmul_rn(o[nb][p][i][k], f[nb][k & 1]);
        }
        if constexpr (HALF) {
#pragma unroll
          for (int nb = 0; nb < NB; ++nb)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const float by = FP8 ? Unit::factor(bound[nb], j) : 0x1p14f;
#pragma unroll
              for (int t = 0; t < 2 * MB; ++t) s[nb][t / 2][2 * (t & 1) + j] = __fmul_rn(s[nb][t / 2][2 * (t & 1) + j], by);
            }
        }
        // weights of head g: of tokens 2c, 2c + 1 and 8 more (TF32: c, c + 4, and 8 more)
        uint32_t w[WN][NB][MB][TF32 ? 4 : 2];
#pragma unroll
        for (int nb = 0; nb < NB; ++nb)
#pragma unroll
          for (int b = 0; b < MB; ++b)
#pragma unroll
            for (int k = 0; k < 2; ++k) {
              const float x = s[nb][b][2 * k], y = s[nb][b][2 * k + 1];
              if constexpr (TF32) {
#pragma unroll
                for (int i = 0; i < 2; ++i) {
                  const int src = (cl + 4 * i) * 4 + gl / 2;
                  const float u = __shfl_sync(0xFFFFFFFFu, x, src), v = __shfl_sync(0xFFFFFFFFu, y, src);
                  w[0][nb][b][(2 * k + i) % (TF32 ? 4 : 2)] = __float_as_uint(gl & 1 ? v : u);
                }
              } else {
                const uint32_t h = Pair<typename std::conditional<TF32, __half, M>::type>::narrow(f2(x, y));
                w[0][nb][b][k] = transposed(h);
                if constexpr (WN == 2) {
                  // (what is left is at most 16; -64 in the place of infinity less infinity changes no infinite product)
                  const F2 back = Pair<__half>::widen(h);
                  const float u = fmaxf(__fadd_rn(x, -back.x), -64.0f), v = fmaxf(__fadd_rn(y, -back.y), -64.0f);
                  w[1][nb][b][k] = transposed(Pair<__half>::narrow(f2(u, v)));
                }
              }
            }
#pragma unroll
        for (int n = 0; n < VN; ++n) {
          const int p = n / MB, b = n % MB;
          Raw<S::VB>(&u)[4] = v[n % VG];
          if constexpr (TF32) {
#pragma unroll
            for (int e = 0; e < 2; ++e) {  // two columns
              float sum[NB][4] = {};
#pragma unroll
              for (int k = 0; k < 2; ++k) {  // eight tokens
                const Split a0(u[2 * k].w[2 * e]), a1(u[2 * k].w[2 * e + 1]), a2(u[2 * k + 1].w[2 * e]), a3(u[2 * k + 1].w[2 * e + 1]);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) {
                  const Split b0(w[0][nb][b][(2 * k) % (TF32 ? 4 : 2)]), b1(w[0][nb][b][(2 * k + 1) % (TF32 ? 4 : 2)]);
                  float(&d)[4] = sum[nb];
                  mma<M>(d, a0.low, a1.low, a2.low, a3.low, b0.high, b1.high);
                  mma<M>(d, a0.high, a1.high, a2.high, a3.high, b0.low, b1.low);
                  mma<M>(d, a0.high, a1.high, a2.high, a3.high, b0.high, b1.high);
                }
              }
#pragma unroll
              for (int nb = 0; nb < NB; ++nb) add(o[nb][p][e], sum[nb]);
            }
          } else {
#pragma unroll
            for (int k = 0; k < S::VB / 4; ++k) {
              if constexpr (FP8) {
                // the codes of two tokens side by side, column by column
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                  const uint32_t sel = h ? 0x7362 : 0x5140;
                  const uint32_t x = __byte_perm(u[0].w[k], u[1].w[k], sel), y = __byte_perm(u[2].w[k], u[3].w[k], sel);
                  const uint32_t a0 = e4m3x2_to_half2(x), a1 = e4m3x2_to_half2(x >> 16);
                  const uint32_t a2 = e4m3x2_to_half2(y), a3 = e4m3x2_to_half2(y >> 16);
#pragma unroll
                  for (int nb = 0; nb < NB; ++nb) {
                    if constexpr (SPLIT) {
                      float sum[4] = {};
                      mma<M>(sum, a0, a1, a2, a3, w[WN - 1][nb][b][0], w[WN - 1][nb][b][1]);
                      mma<M>(sum, a0, a1, a2, a3, w[0][nb][b][0], w[0][nb][b][1]);
                      add(o[nb][p][2 * k + h], sum);
                    } else {
                      if constexpr (WN == 2) mma<M>(o[nb][p][2 * k + h], a0, a1, a2, a3, w[WN - 1][nb][b][0], w[WN - 1][nb][b][1]);
                      mma<M>(o[nb][p][2 * k + h], a0, a1, a2, a3, w[0][nb][b][0], w[0][nb][b][1]);
                    }
                  }
                }
              } else {
                const uint32_t a0 = __byte_perm(u[0].w[k], u[1].w[k], 0x5410);
                const uint32_t a1 = __byte_perm(u[0].w[k], u[1].w[k], 0x7632);
                const uint32_t a2 = __byte_perm(u[2].w[k], u[3].w[k], 0x5410);
                const uint32_t a3 = __byte_perm(u[2].w[k], u[3].w[k], 0x7632);
#pragma unroll
                for (int nb = 0; nb < NB; ++nb) mma<M>(o[nb][p][k], a0, a1, a2, a3, w[0][nb][b][0], w[0][nb][b][1]);
              }
            }
          }
          if (n + VG < VN) {
#pragma unroll
            for (int i = 0; i < 4; ++i) u[i] = load((n + VG) % MB, i, (n + VG) / MB);
          }
        }
        stage = stage + 1 == S::STAGES ? 0 : stage + 1;
      }

      // ----- the segment's result, or its piece -----
      const bool piece = g.head || g.tail;
      float* to = args.warp_partial + (slot + (g.head ? 0 : 1)) * slot_rows * D;
      if (piece && lane == 0) {
        owner[warp][g.head ? 0 : 1] = segment_id(g.b, g.s);
        if (g.head) open[warp] = g.open;
      }
#pragma unroll
      for (int nb = 0; nb < NB; ++nb)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
          const float sum = column_sum(l[nb][j]);
          const int r = 8 * nb + 2 * cl + j;
          if (r >= rows) continue;
          const float by = piece ? 1.0f : sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
          const float unit = FP8 ? Unit::value(bound[nb], j) : 0x1p-14f;
#pragma unroll
          for (int p = 0; p < S::VP; ++p) {
            float out[S::CE];
#pragma unroll
            for (int i = 0; i < NCE; ++i) {
              out[2 * i] = __fmul_rn(o[nb][p][i][j], by);
              out[2 * i + 1] = __fmul_rn(o[nb][p][i][2 + j], by);
              if constexpr (HALF) out[2 * i] = __fmul_rn(out[2 * i], unit), out[2 * i + 1] = __fmul_rn(out[2 * i + 1], unit);
            }
            const int c = (8 * p + gl) * S::CE;
#pragma unroll
            for (int i = 0; i < S::CE; i += S::LOAD) {
              if (c + i >= D) continue;
              const float(&x)[S::LOAD] = *(const float(*)[S::LOAD])(out + i);
              if (piece) {
                float2* dst = (float2*)(to + r * D + c + i);
#pragma unroll
                for (int k = 0; k < S::LOAD / 2; ++k) dst[k] = make_float2(x[2 * k], x[2 * k + 1]);
              } else {
                st_stream<16>((T*)a.out.p + g.b * a.out.token + (int64_t)(h0 + r) * a.out.head + c + i,
                              Vec<T, 16>::narrow(x));
              }
            }
          }
          if (gl != 0) continue;
          if (piece) {
            piece_m[warp][g.head ? 0 : 1][r] = m[nb][j];
            piece_l[warp][g.head ? 0 : 1][r] = sum;
          } else if (a.lse) {
            a.lse[(int64_t)g.b * a.Hq + h0 + r] = lse_of(m[nb][j], sum);
          }
        }
    }
    cp_async_wait<0>();  // no copy may outlive the CTA's shared memory
  }

  // ----- pieces of the same segment in this CTA, together: a warp takes a head of one -----
  // (short code: what runs once is bound by fetching its instructions)
  __syncthreads();
  static_assert(S::WARPS < 32, "a piece a lane");
#pragma unroll 1
  for (int task = warp; task < (S::WARPS + 1) * slot_rows; task += S::WARPS) {
    // chain 0 begins before this CTA, chain i + 1 with the second piece of warp i
    const int chain = task / slot_rows, r = task - chain * slot_rows;
    const bool begun = chain > 0;
    const int64_t id = begun ? owner[chain - 1][1] : owner[0][0];
    if (id < 0) continue;
    const int b = (int)(id >> 32), s = (int)(uint32_t)id;
    const int key_head = s / blocks, row0 = (s - key_head * blocks) * 8 * NB;
    if (r >= min(8 * NB, a.group - row0)) continue;
    // the warps [chain, last) go on with it
    const int last = __ffs(~__ballot_sync(0xFFFFFFFFu, lane >= chain && lane < S::WARPS && owner[min(lane, S::WARPS - 1)][0] == id) >> chain) - 1 + chain;
    const bool done = begun && last > chain && !open[last - 1];
    const int pieces = last - chain + begun;
    // lane k has piece k's maximum and sum
    auto from = [&](int k) { return begun ? 2 * (chain - 1 + k) + (k == 0) : 2 * k; };
    const bool on = lane < pieces;
    const float m = on ? (&piece_m[0][0][0])[from(lane) * 8 * NB + r] : -INFINITY;
    float top = m;
#pragma unroll
    for (int i = 16; i > 0; i >>= 1) top = fmaxf(top, __shfl_xor_sync(0xFFFFFFFFu, top, i));
    const float f = exp2_fast(__fadd_rn(m, -(top == -INFINITY ? 0.0f : top)));
    const float sum = lanes_sum<32>(on ? __fmul_rn((&piece_l[0][0][0])[from(lane) * 8 * NB + r], f) : 0.0f);
    if (on) factors[warp][lane] = f;
    __syncwarp();
    const float* base = args.warp_partial + (blockIdx.x * (int64_t)S::WARPS * 2 * slot_rows + r) * D;
    const float by = !done ? 1.0f : sum == 0.0f ? 0.0f : __fdiv_rn(1.0f, sum);
    const int h = key_head * a.group + row0 + r;
    const Piece p(a.partial, 2 * blockIdx.x + begun, slot_rows, D);
#pragma unroll 1
    for (int c = 2 * lane; c < D; c += 64) {
      float2 o = {};
#pragma unroll 4
      for (int k = 0; k < pieces; ++k) {
        const float2 v = *(const float2*)(base + from(k) * slot_rows * D + c);
        const float fk = factors[warp][k];
        o = make_float2(__fmaf_rn(v.x, fk, o.x), __fmaf_rn(v.y, fk, o.y));
      }
      o = make_float2(__fmul_rn(o.x, by), __fmul_rn(o.y, by));
      T* out = (T*)a.out.p + b * a.out.token + h * a.out.head + c;
      if (!done)
        *(float2*)(p.o + r * D + c) = o;
      else if constexpr (sizeof(T) == 4)
        *(float2*)out = o;
      else
        *(uint32_t*)out = Pair<T>::narrow(o);
    }
    __syncwarp();
    if (lane != 0) continue;
    if (!done) {
      p.m[r] = top;
      p.l[r] = sum;
      a.owner[2 * blockIdx.x + begun] = id;
    } else if (a.lse) {
      a.lse[(int64_t)b * a.Hq + h] = lse_of(top, sum);
    }
  }
}

template <class T, bool FP8, int DP, int NB>
cudaError_t launch(const DeviceInfo& dev, AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  using S = Shape<T, FP8, DP, NB>;
  const auto kern = attend_mma_kernel<T, S>;
  static std::atomic<int> opted[kOptinDevices];
  const cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  *ctas = std::min(kAttendMmaCtas, (int64_t)dev.sm_count);
  a.rows = 8 * NB;
  MmaArgs m;
  m.a = a;
  m.page = divisor((uint32_t)a.c.page_size);
  m.whole = a.c.page_size % 16 == 0;
  m.page_rows = (int)(a.c.page_stride / a.c.D);
  m.warp_partial = a.partial + *ctas * 2 * std::min(a.group, a.rows) * (a.c.D + 2);
  return launch_after(kern, (unsigned)*ctas, S::THREADS, S::SMEM, s, m);
}

// (fp32 queries: eight heads at a time, for registers)
template <class T, bool FP8, int DP>
cudaError_t launch(const DeviceInfo& dev, AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  if constexpr (sizeof(T) == 2) {
    if (a.group > 8) return launch<T, FP8, DP, 2>(dev, a, ctas, s);
  }
  return launch<T, FP8, DP, 1>(dev, a, ctas, s);
}
template <class T, bool FP8>
cudaError_t launch(const DeviceInfo& dev, AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.c.D <= 64    ? launch<T, FP8, 64>(dev, a, ctas, s)
         : a.c.D <= 128 ? launch<T, FP8, 128>(dev, a, ctas, s)
                        : launch<T, FP8, 256>(dev, a, ctas, s);
}

}  // namespace

// (two compilations: 16-bit types in one, fp32 in the other)
#ifdef DIT_ATTEND_FP32
cudaError_t launch_attend_mma_fp32(const DeviceInfo& dev, AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.c.format == DIT_E4M3 ? launch<float, true>(dev, a, ctas, s) : launch<float, false>(dev, a, ctas, s);
}
#else
bool attend_mma_takes(bool granules, const AttendArgs& a) {
  return granules && a.c.D <= 256 && a.capacity > 0 && a.c.page_stride % a.c.D == 0 &&
         a.c.pages * (a.c.page_stride / a.c.D) <= 0x7FFFFFFF;
}
cudaError_t launch_attend_mma(const DeviceInfo& dev, int dtype, AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  const bool fp8 = a.c.format == DIT_E4M3;
  return dtype == 2   ? launch_attend_mma_fp32(dev, a, ctas, s)
         : dtype == 1 ? (fp8 ? launch<__half, true>(dev, a, ctas, s) : launch<__half, false>(dev, a, ctas, s))
                      : (fp8 ? launch<__nv_bfloat16, true>(dev, a, ctas, s) : launch<__nv_bfloat16, false>(dev, a, ctas, s));
}
#endif

}  // namespace dit
