// k_attend_mma.cu -- attention of one new token per sequence over a paged
// cache of 16-bit or E4M3 rows, on the tensor cores (sm_103a).
//
//   s = scale q.k,  m = max s,  l = sum 2^(s - m),  o = sum 2^(s - m) v
// in one pass over the tokens, with s in powers of two (scale times log2 e).
//
// What bounds it is memory: each key and value is read once for all query heads
// of its key head, 16 bit for 4 * group operations.  A warp takes tiles of 16 tokens.  Both
// products are mma.sync of 16 x 8 x 16: S (heads x tokens) = Q K^T, then O
// (heads x columns) += P V, P in the registers that S came in.  The tensor cores' 5th
// generation instructions want 64 or 128 rows, of which a group of heads fills
// 1 to 16; these here take 2 of 22 cycles that an SM needs to load a token's head at
// the memory's rate (D = 128, bf16).
//
// The contraction index of a product may be permuted if both operands agree, and so may
// the columns of O.  So every lane's operands are 16 contiguous bytes of a row: of keys,
// lane (g, c) = (lane / 4, lane % 4) has bytes 16 c of each 64 of tokens g and g + 8; of
// values, bytes 16 g of each 128 of the tokens 2c, 2c + 1, 2c + 8, 2c + 9.  Each lane
// copies the bytes that it will read itself to its own places in shared memory
// (cp.async), S stages ahead: no bank conflicts, no barriers between warps,
// and no shuffles.
#include "dit_attend.cuh"

namespace dit {
namespace {

template <int N>
struct Words {
  uint32_t w[N];
};

__device__ __forceinline__ void cp_async8_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 8, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ void cp_async4_part(uint32_t dst, const void* src, uint32_t bytes) {
  asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(bytes) : "memory");
}
__device__ __forceinline__ float exp2_fast(float x) {  // within 2^-22
  float y;
  asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
  return y;
}

// d += a b: a 16 x 16 (rows of heads), b 16 x 8, of M.  HALF: rows 8 to 15 are zero, and their sums are not kept.
template <class M, bool HALF>
__device__ __forceinline__ void mma(float (&d)[HALF ? 2 : 4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                    uint32_t b0, uint32_t b1) {
  float e2 = 0.0f, e3 = 0.0f;
  float& d2 = *(HALF ? &e2 : &d[HALF ? 0 : 2]);
  float& d3 = *(HALF ? &e3 : &d[HALF ? 1 : 3]);
  if constexpr (std::is_same<M, __nv_bfloat16>::value)
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d2), "+f"(d3)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
  else
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d2), "+f"(d3)
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t e4m3x2_to_half2(uint32_t codes) {  // the low two codes
  uint32_t h;
  asm("{ .reg .b16 c, d; mov.b32 {c, d}, %1; cvt.rn.f16x2.e4m3x2 %0, c; }" : "=r"(h) : "r"(codes));
  return h;
}

// T: the queries' type; FP8: an E4M3 cache; DP: columns, D rounded up (the rest is zero); HALF: at most 8 heads a
// key head.
template <class T, bool FP8_, int DP_, bool HALF_>
struct Shape {
  static constexpr bool FP8 = FP8_, HALF = HALF_;
  static constexpr int DP = DP_;
  using M = typename std::conditional<FP8, __half, T>::type;  // of the products
  static constexpr int ES = FP8 ? 1 : 2;
  static constexpr int ROW = DP * ES;                 // bytes
  static constexpr int WARPS = ROW <= 256 ? 8 : 4;
  static constexpr int THREADS = 32 * WARPS;
  static constexpr int KP = ROW / 64;                 // 16-byte pieces of a key that a lane has
  static constexpr int VB = ROW / 8 < 16 ? ROW / 8 : 16;  // bytes of a piece of a value
  static constexpr int VP = ROW / 8 / VB;             // pieces of a value that a lane has
  static constexpr int CE = VB / ES;                  // columns of such a piece
  static constexpr int STEPS = DP / 16;               // products of 16 columns
  static constexpr int QW = HALF ? 2 : 4;             // words of a lane's queries for each
  static constexpr int NC = HALF ? 2 : 4;             // sums of a lane for each 8 columns
  static constexpr int STAGE = 32 * ROW;              // bytes of a warp's stage: 16 keys and values
  // behind them: the scales of 16 keys and values (E4M3), and which tokens count
  static constexpr int EXTRA = FP8 ? 144 : 16;
  static constexpr int ROWS = HALF ? 8 : 16;
  static constexpr int PAD = DP + 4;                  // floats of a row of sums in shared memory
  static constexpr int SLOTS = WARPS / 2;
  static constexpr int JOIN = SLOTS * ROWS * PAD * 4 + 2 * WARPS * ROWS * 4;
  static constexpr int ROOM = 227 * 1024 - 1024 - JOIN;
  static constexpr int FIT = ROOM / (WARPS * (STAGE + EXTRA));
  static constexpr int STAGES = FIT > 8 ? 8 : FIT;
  static constexpr int SMEM = STAGES * WARPS * (STAGE + EXTRA) + JOIN;
  static_assert(STAGES >= 2, "a stage in flight and one in use");
};

// A warp's walk over its tiles.
struct Cursor {
  Part part;
  Segment g;
  int tile;
  bool live;
};

template <class T, class S>
__global__ void __launch_bounds__(S::THREADS, 1) attend_mma_kernel(const __grid_constant__ AttendArgs a) {
  using M = typename S::M;
  constexpr bool FP8 = S::FP8, HALF = S::HALF;
  constexpr int NC = S::NC;
  __shared__ int64_t numbers[S::WARPS + 2];
  extern __shared__ __align__(128) unsigned char space[];
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  const int gl = lane >> 2, cl = lane & 3;
  const int D = (int)a.c.D;
  const int blocks = (a.group + S::ROWS - 1) / S::ROWS;
  const int segments = (int)a.c.heads * blocks;
  const int slot_rows = min(a.group, kAttendRows);

  float* joined = (float*)space;                              // [SLOTS][ROWS][PAD]
  float* warp_m = joined + S::SLOTS * S::ROWS * S::PAD;       // [WARPS][ROWS]
  float* warp_l = warp_m + S::WARPS * S::ROWS;                // [WARPS][ROWS]
  unsigned char* stages = space + S::JOIN + warp * S::STAGES * (S::STAGE + S::EXTRA);
  const uint32_t stages_at = smem_addr(stages);

  Part part = part_of<S::THREADS>(a, segments, S::WARPS, numbers);
  if (tid < 2) a.owner[2 * blockIdx.x + tid] = -1;
  let_next();
  if (part.begin >= part.end) return;

  // ----- copies -----
  // (of a token that does not count nothing is read, from any address, and zeros are written)
  const char* zeros = (const char*)a.q.p;
  Cursor ahead;
  ahead.part = part;
  ahead.live = next_segment(a, ahead.part, segments, ahead.g);
  ahead.tile = ahead.g.first + warp;
  int page = -1;  // of token lane % 16 of the tile ahead
  auto find = [&]() {
    while (ahead.live && ahead.tile >= ahead.g.last) {
      ahead.live = next_segment(a, ahead.part, segments, ahead.g);
      if (ahead.live) ahead.tile = ahead.g.first + warp;
    }
    page = -1;
    if (ahead.live) {
      const int t = ahead.tile * kTile + (lane & 15);
      if (t >= ahead.g.lo && t < ahead.g.hi)
        page = __ldg(a.pages + (int64_t)ahead.g.b * a.pages_stride + t / (int)a.c.page_size);
    }
  };
  auto issue = [&](int stage) {
    if (ahead.live) {
      const uint32_t to = stages_at + stage * (S::STAGE + S::EXTRA);
      const int head = ahead.g.s / blocks;
      const int t = ahead.tile * kTile + (lane & 15);
      const bool there = page >= 0 && page < a.c.pages;
      const int64_t row = (int64_t)head * a.c.page_size + t % (int)a.c.page_size;
      const int64_t at = there ? (page * a.c.page_stride + row * D) * S::ES : -1;
      const uint32_t count = __ballot_sync(0xFFFFFFFFu, there);
      const int bytes = D * S::ES;
#pragma unroll
      for (int b = 0; b < 2; ++b) {
        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, gl + 8 * b);
#pragma unroll
        for (int p = 0; p < S::KP; ++p) {
          const int c = (p * 4 + cl) * 16;
          const bool any = from >= 0 && c < bytes;
          cp_async16_part(to + ((b * S::KP + p) * 32 + lane) * 16, any ? (const char*)a.c.k + from + c : zeros,
                          any ? 16 : 0);
        }
      }
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        const int64_t from = __shfl_sync(0xFFFFFFFFu, at, 2 * cl + (i & 1) + 8 * (i >> 1));
#pragma unroll
        for (int p = 0; p < S::VP; ++p) {
          const int c = (p * 8 + gl) * S::VB;
          const bool any = from >= 0 && c < bytes;
          const uint32_t dst = to + S::STAGE / 2 + ((i * S::VP + p) * 32 + lane) * S::VB;
          const char* src = any ? (const char*)a.c.v + from + c : zeros;
          if constexpr (S::VB == 16)
            cp_async16_part(dst, src, any ? 16 : 0);
          else
            cp_async8_part(dst, src, any ? 8 : 0);
        }
      }
      if constexpr (FP8) {
        const float* scales = lane < 16 ? a.c.k_scales : a.c.v_scales;
        cp_async4_part(to + S::STAGE + lane * 4,
                       there ? (const void*)(scales + page * a.c.scale_stride + row) : zeros, there ? 4 : 0);
      }
      if (lane == 0) *(uint32_t*)(stages + stage * (S::STAGE + S::EXTRA) + S::STAGE + S::EXTRA - 16) = count & 0xFFFFu;
      ahead.tile += S::WARPS;
      find();
    }
    cp_async_commit();
  };
  find();
#pragma unroll
  for (int s = 0; s < S::STAGES - 1; ++s) issue(s);

  // ----- products -----
  int stage = 0;
  Segment g;
  while (next_segment(a, part, segments, g)) {
    const int head = g.s / blocks, row0 = (g.s - head * blocks) * S::ROWS;
    const int rows = min(S::ROWS, a.group - row0);
    const int h0 = head * a.group + row0;

    // queries, in the order of the keys' bytes, and what a product of theirs is multiplied by
    uint32_t q[S::STEPS][S::QW];
    float factor[HALF ? 1 : 2];
#pragma unroll
    for (int r = 0; r < (HALF ? 1 : 2); ++r) {
      const bool real = gl + 8 * r < rows;
      const T* from = (const T*)a.q.p + g.b * a.q.token + (int64_t)(h0 + gl + 8 * r) * a.q.head;
      constexpr int PER = 16 / S::ES;  // columns of a key's piece
      factor[r] = __fmul_rn(a.scale, 1.4426950408889634f);
      Raw<16> raw[S::KP * PER / 8];
#pragma unroll
      for (int i = 0; i < S::KP * PER / 8; ++i) {
        const int p = i / (PER / 8), c = (p * 4 + cl) * PER + (i % (PER / 8)) * 8;
        raw[i] = Raw<16>{};
        if (real && c < D) raw[i] = ld_bcast<16>(from + c);
      }
      if constexpr (FP8 && std::is_same<T, __nv_bfloat16>::value) {
        // to fp16 by a power of two that brings the largest below 2^14
        float most = 0.0f;
#pragma unroll
        for (int i = 0; i < S::KP * PER / 8; ++i) {
          float f[8];
          Vec<T, 16>::widen(raw[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) most = max_nan(most, fabsf(f[k]));
        }
        most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = max_nan(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        int e = (int)(__float_as_uint(most) >> 23) - 127;  // its exponent
        e = most == 0.0f || !isfinite(most) ? 0 : max(e, -100);
        const float up = __uint_as_float((uint32_t)(min(13 - e, 127) + 127) << 23);
        factor[r] = __fmul_rn(factor[r], __uint_as_float((uint32_t)(max(e - 13, -126) + 127) << 23));
#pragma unroll
        for (int i = 0; i < S::KP * PER / 8; ++i) {
          float f[8];
          Vec<T, 16>::widen(raw[i], f);
#pragma unroll
          for (int k = 0; k < 8; ++k) f[k] = __fmul_rn(f[k], up);
          raw[i] = Vec<__half, 16>::narrow(f);
        }
      }
#pragma unroll
      for (int i = 0; i < S::KP * PER / 8; ++i) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
          q[2 * i + k][HALF ? 0 : r] = raw[i].w[2 * k];
          q[2 * i + k][HALF ? 1 : 2 + r] = raw[i].w[2 * k + 1];
        }
      }
    }

    float o[S::VP][S::CE][NC] = {};
    float m[HALF ? 1 : 2], l[HALF ? 1 : 2];
#pragma unroll
    for (int r = 0; r < (HALF ? 1 : 2); ++r) m[r] = -INFINITY, l[r] = 0.0f;
    float vref = 0x1p-126f;  // E4M3: o is in units of this power of two

    for (int tile = g.first + warp; tile < g.last; tile += S::WARPS) {
      cp_async_wait<S::STAGES - 2>();
      __syncwarp();
      issue(stage == 0 ? S::STAGES - 1 : stage - 1);
      const uint32_t from = stages_at + stage * (S::STAGE + S::EXTRA);
      const unsigned char* extra = stages + stage * (S::STAGE + S::EXTRA) + S::STAGE;
      const uint32_t count = *(const uint32_t*)(extra + S::EXTRA - 16);

      float s[2][NC] = {};
#pragma unroll
      for (int p = 0; p < S::KP; ++p) {
#pragma unroll
        for (int b = 0; b < 2; ++b) {
          const Raw<16> k = lds16(from + ((b * S::KP + p) * 32 + lane) * 16);
          constexpr int N = FP8 ? 4 : 2;  // products of a piece
#pragma unroll
          for (int i = 0; i < N; ++i) {
            const uint32_t b0 = FP8 ? e4m3x2_to_half2(k.w[i]) : k.w[2 * i];
            const uint32_t b1 = FP8 ? e4m3x2_to_half2(k.w[i] >> 16) : k.w[2 * i + 1];
            const uint32_t(&w)[S::QW] = q[p * N + i];
            mma<M, HALF>(s[b], w[0], HALF ? 0 : w[1], w[HALF ? 1 : 2], HALF ? 0 : w[HALF ? 1 : 3], b0, b1);
          }
        }
      }
      float ks[2][2], vs[2][2];
      if constexpr (FP8) {
        const float* scales = (const float*)extra;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            ks[b][i] = scales[8 * b + 2 * cl + i];
            vs[b][i] = scales[16 + 8 * b + 2 * cl + i];
          }
      }
      float f[HALF ? 1 : 2];
      bool moved = false;
#pragma unroll
      for (int r = 0; r < (HALF ? 1 : 2); ++r) {
        float most = m[r];
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& x = s[b][2 * r + i];
            x = __fmul_rn(x, FP8 ? __fmul_rn(factor[r], ks[b][i]) : factor[r]);
            if (!(count >> (8 * b + 2 * cl + i) & 1)) x = -INFINITY;
            most = fmaxf(most, x);
          }
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 1));
        most = fmaxf(most, __shfl_xor_sync(0xFFFFFFFFu, most, 2));
        const float base = most == -INFINITY ? 0.0f : most;
        f[r] = exp2_fast(__fadd_rn(m[r], -base));
        moved = moved || most != m[r];
        m[r] = most;
        float sum = 0.0f;
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            float& x = s[b][2 * r + i];
            x = exp2_fast(__fadd_rn(x, -base));
            sum = __fadd_rn(sum, x);
          }
        l[r] = __fmaf_rn(l[r], f[r], sum);
      }
      float of[HALF ? 1 : 2];
#pragma unroll
      for (int r = 0; r < (HALF ? 1 : 2); ++r) of[r] = f[r];
      if constexpr (FP8) {
        // weights times the values' scales, in units of a power of two above all of them so far, fit fp16
        const uint32_t mine = __float_as_uint(((const float*)extra)[16 + (lane & 15)]);
        const uint32_t most = __reduce_max_sync(0xFFFFFFFFu, mine);
        if (most >= __float_as_uint(vref)) {
          const uint32_t e = min((most >> 23) + 1, 254u);
          const float now = most > 0x7F800000u ? __uint_as_float(0x7FC00000u) : __uint_as_float(e << 23);
          const float down = __fdiv_rn(vref, now);
          vref = now;
          moved = true;
#pragma unroll
          for (int r = 0; r < (HALF ? 1 : 2); ++r) of[r] = __fmul_rn(of[r], down);
        }
        const float unit = __fdiv_rn(1.0f, vref);
#pragma unroll
        for (int b = 0; b < 2; ++b)
#pragma unroll
          for (int i = 0; i < 2; ++i) {
            const float w = __fmul_rn(vs[b][i], unit);
#pragma unroll
            for (int r = 0; r < (HALF ? 1 : 2); ++r) s[b][2 * r + i] = __fmul_rn(s[b][2 * r + i], w);
          }
      }
      if (__any_sync(0xFFFFFFFFu, moved)) {
#pragma unroll
        for (int p = 0; p < S::VP; ++p)
#pragma unroll
          for (int i = 0; i < S::CE; ++i)
#pragma unroll
            for (int k = 0; k < NC; ++k) o[p][i][k] = __fmul_rn(o[p][i][k], of[k >> 1]);
      }
      uint32_t w[2][HALF ? 1 : 2];
#pragma unroll
      for (int b = 0; b < 2; ++b)
#pragma unroll
        for (int r = 0; r < (HALF ? 1 : 2); ++r) w[b][r] = Pair<M>::narrow(f2(s[b][2 * r], s[b][2 * r + 1]));
      const uint32_t values = from + S::STAGE / 2;
#pragma unroll
      for (int p = 0; p < S::VP; ++p) {
        constexpr int N = S::VB / 4;
        Words<N> v[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
          const uint32_t at = values + ((i * S::VP + p) * 32 + lane) * S::VB;
          if constexpr (N == 4) {
            const Raw<16> x = lds16(at);
#pragma unroll
            for (int k = 0; k < 4; ++k) v[i].w[k] = x.w[k];
          } else {
            asm volatile("ld.shared.v2.b32 {%0,%1}, [%2];" : "=r"(v[i].w[0]), "=r"(v[i].w[1]) : "r"(at));
          }
        }
#pragma unroll
        for (int k = 0; k < N; ++k) {
          if constexpr (FP8) {
            // the codes of two tokens side by side, column by column
#pragma unroll
            for (int h = 0; h < 2; ++h) {
              const uint32_t sel = h ? 0x7362 : 0x5140;
              const uint32_t x = __byte_perm(v[0].w[k], v[1].w[k], sel), y = __byte_perm(v[2].w[k], v[3].w[k], sel);
#pragma unroll
              for (int j = 0; j < 2; ++j)
                mma<M, HALF>(o[p][4 * k + 2 * h + j], w[0][0], HALF ? 0 : w[0][HALF ? 0 : 1], w[1][0],
                             HALF ? 0 : w[1][HALF ? 0 : 1], e4m3x2_to_half2(j ? x >> 16 : x),
                             e4m3x2_to_half2(j ? y >> 16 : y));
            }
          } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
              const uint32_t sel = j ? 0x7632 : 0x5410;
              mma<M, HALF>(o[p][2 * k + j], w[0][0], HALF ? 0 : w[0][HALF ? 0 : 1], w[1][0],
                           HALF ? 0 : w[1][HALF ? 0 : 1], __byte_perm(v[0].w[k], v[1].w[k], sel),
                           __byte_perm(v[2].w[k], v[3].w[k], sel));
            }
          }
        }
      }
      stage = stage + 1 == S::STAGES ? 0 : stage + 1;
    }

    // ----- the warps' parts together -----
#pragma unroll
    for (int r = 0; r < (HALF ? 1 : 2); ++r) {
      l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xFFFFFFFFu, l[r], 1));
      l[r] = __fadd_rn(l[r], __shfl_xor_sync(0xFFFFFFFFu, l[r], 2));
      if (cl == 0) {
        warp_m[warp * S::ROWS + gl + 8 * r] = m[r];
        warp_l[warp * S::ROWS + gl + 8 * r] = l[r];
      }
    }
    __syncthreads();
    float top[HALF ? 1 : 2];
#pragma unroll
    for (int r = 0; r < (HALF ? 1 : 2); ++r) {
      top[r] = -INFINITY;
#pragma unroll
      for (int k = 0; k < S::WARPS; ++k) top[r] = fmaxf(top[r], warp_m[k * S::ROWS + gl + 8 * r]);
      float by = exp2_fast(__fadd_rn(m[r], -(top[r] == -INFINITY ? 0.0f : top[r])));
      if constexpr (FP8) by = __fmul_rn(by, vref);
#pragma unroll
      for (int p = 0; p < S::VP; ++p)
#pragma unroll
        for (int i = 0; i < S::CE; ++i)
#pragma unroll
          for (int k = 0; k < 2; ++k) o[p][i][2 * r + k] = __fmul_rn(o[p][i][2 * r + k], by);
    }
    // the column of o[p][i][2 r + k]
    auto column = [&](int p, int i, int k) { return (p * 8 + 2 * cl + k) * S::CE + i; };
    auto each = [&](int slot, auto&& body) {
      float* base = joined + slot * S::ROWS * S::PAD;
#pragma unroll
      for (int p = 0; p < S::VP; ++p)
#pragma unroll
        for (int k = 0; k < NC; ++k)
#pragma unroll
          for (int i = 0; i < S::CE; i += 4)
            body(*(float4*)(base + (gl + 8 * (k >> 1)) * S::PAD + column(p, i, k & 1)), o[p][i][k], o[p][i + 1][k],
                 o[p][i + 2][k], o[p][i + 3][k]);
    };
    if (warp >= S::SLOTS)
      each(warp - S::SLOTS, [](float4& x, float& p, float& q, float& r, float& s) { x = make_float4(p, q, r, s); });
    __syncthreads();
    if (warp < S::SLOTS)
      each(warp, [](float4& x, float& p, float& q, float& r, float& s) {
        x = make_float4(__fadd_rn(p, x.x), __fadd_rn(q, x.y), __fadd_rn(r, x.z), __fadd_rn(s, x.w));
      });
    __syncthreads();
    const bool shared_out = g.head || g.tail;
    const int place = g.head ? 0 : 1;
    float* parts = a.partial + ((int64_t)blockIdx.x * 2 + place) * slot_rows * (D + 2);
    if (shared_out && tid == 0) a.owner[2 * blockIdx.x + place] = g.id;
    for (int i = tid; i < rows * (S::DP / 8); i += S::THREADS) {
      const int r = i / (S::DP / 8), c = (i - r * (S::DP / 8)) * 8;
      if (c >= D) continue;
      float most = -INFINITY, total = 0.0f;
#pragma unroll
      for (int k = 0; k < S::WARPS; ++k) most = fmaxf(most, warp_m[k * S::ROWS + r]);
#pragma unroll
      for (int k = 0; k < S::WARPS; ++k)
        total = __fmaf_rn(warp_l[k * S::ROWS + r],
                          exp2_fast(__fadd_rn(warp_m[k * S::ROWS + r], -(most == -INFINITY ? 0.0f : most))), total);
      float sum[8] = {};
#pragma unroll
      for (int k = 0; k < S::SLOTS; ++k) {
        const float* x = joined + (k * S::ROWS + r) * S::PAD + c;
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = __fadd_rn(sum[j], x[j]);
      }
      if (shared_out) {
#pragma unroll
        for (int j = 0; j < 8; ++j) parts[2 * slot_rows + r * D + c + j] = sum[j];
        if (c == 0) {
          parts[r] = most;
          parts[slot_rows + r] = total;
        }
      } else {
        const float by = total == 0.0f ? 0.0f : __fdiv_rn(1.0f, total);
#pragma unroll
        for (int j = 0; j < 8; ++j) sum[j] = total == 0.0f ? 0.0f : __fmul_rn(sum[j], by);
        st_stream<16>((T*)a.out.p + g.b * a.out.token + (int64_t)(h0 + r) * a.out.head + c, Vec<T, 16>::narrow(sum));
        if (a.lse && c == 0) a.lse[(int64_t)g.b * a.Hq + h0 + r] = lse_of(most, total);
      }
    }
    __syncthreads();
  }
  cp_async_wait<0>();  // no copy may outlive the CTA's shared memory
}

template <class T, bool FP8, int DP, bool HALF>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  using S = Shape<T, FP8, DP, HALF>;
  const auto kern = attend_mma_kernel<T, S>;
  static std::atomic<int> opted[kOptinDevices];
  cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  *ctas = std::min(kAttendMaxCtas, (int64_t)dev.sm_count);
  kern<<<(unsigned)*ctas, S::THREADS, S::SMEM, s>>>(a);
  return cudaGetLastError();
}

template <class T, bool FP8, int DP>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.group <= 8 ? launch<T, FP8, DP, true>(dev, a, ctas, s)
                      : launch<T, FP8, DP, false>(dev, a, ctas, s);
}
template <class T, bool FP8>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.c.D <= 64    ? launch<T, FP8, 64>(dev, a, ctas, s)
         : a.c.D <= 128 ? launch<T, FP8, 128>(dev, a, ctas, s)
                        : launch<T, FP8, 256>(dev, a, ctas, s);
}
template <class T>
cudaError_t launch(const DeviceInfo& dev, const AttendArgs& a, int64_t* ctas, cudaStream_t s) {
  return a.c.format == DIT_E4M3 ? launch<T, true>(dev, a, ctas, s) : launch<T, false>(dev, a, ctas, s);
}

}  // namespace

cudaError_t launch_attend_mma(const DeviceInfo& dev, bool half, const AttendArgs& a, int64_t* ctas,
                              cudaStream_t s) {
  return half ? launch<__half>(dev, a, ctas, s) : launch<__nv_bfloat16>(dev, a, ctas, s);
}

}  // namespace dit
