// dit_attend.cuh -- how the attention of one token per sequence is divided
// over the GPU (sm_103a).
//
// A segment is one sequence's tokens for up to kAttendRows query heads of one
// key head; its tokens come in tiles of 16.  The tiles of all segments form one
// line, which the CTAs cut into equal parts, so that sequences of any lengths
// keep every SM equally busy: a CTA's part may hold many short segments or a piece of a
// long one.  A segment within one CTA is finished there; of one that several
// CTAs share, each writes its maximum, sum and unscaled output, which a second
// kernel joins in the order of the CTAs.  Only the first and the last
// segment of a CTA can be shared, so there are two such places per CTA.
#pragma once

#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {

constexpr int kTile = 16;

// A sequence's tokens: [lo, hi), in tiles [first, last).
struct Sequence {
  int lo, hi, first, tiles;
  __device__ __forceinline__ Sequence(const AttendArgs& a, int b) {
    const int64_t n = id_at(a.lengths, b, a.ids64);
    hi = (int)min(max(n, (int64_t)0), a.capacity);
    lo = a.window > 0 && a.window < hi ? hi - (int)a.window : 0;
    first = lo / kTile;
    // a sequence without tokens has one empty tile, which writes its output
    tiles = max(1, (hi + kTile - 1) / kTile - first);
  }
};

// A CTA's part of the line, and a walk over its segments.
struct Part {
  int64_t begin, end;   // tiles of the line
  int64_t at;           // where the walk is
  int b;                // its sequence
  int64_t start;        // where that sequence starts on the line
};

template <int THREADS>
__device__ __forceinline__ int64_t cta_sum(int64_t v, int64_t* shared) {
#pragma unroll
  for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
  if ((threadIdx.x & 31) == 0) shared[threadIdx.x >> 5] = v;
  __syncthreads();
  v = 0;
#pragma unroll
  for (int w = 0; w < THREADS / 32; ++w) v += shared[w];
  __syncthreads();
  return v;
}

// segments: of a sequence.  least: tiles that a CTA takes at least.
// shared: THREADS / 32 + 2 numbers.
template <int THREADS>
__device__ __forceinline__ Part part_of(const AttendArgs& a, int segments, int least, int64_t* shared) {
  const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
  int64_t mine = 0;
  for (int b = tid; b < a.B; b += THREADS) mine += Sequence(a, b).tiles;
  const int64_t total = cta_sum<THREADS>(mine, shared) * segments;
  const int64_t per = max((int64_t)least, (total + gridDim.x - 1) / gridDim.x);
  Part p;
  p.begin = min((int64_t)blockIdx.x * per, total);
  p.end = min(p.begin + per, total);
  p.at = p.begin;
  p.b = 0;
  p.start = 0;
  if (p.begin >= p.end) return p;
  // the sequence that holds `begin`
  int64_t before = 0;
  for (int b0 = 0; b0 < a.B; b0 += THREADS) {
    const int b = b0 + tid;
    const int64_t n = b < a.B ? (int64_t)Sequence(a, b).tiles * segments : 0;
    int64_t sum = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t v = __shfl_up_sync(0xFFFFFFFFu, sum, o);
      if (lane >= o) sum += v;
    }
    if (lane == 31) shared[warp] = sum;
    __syncthreads();
    int64_t upto = before + sum;
    int64_t all = 0;
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w) {
      if (w < warp) upto += shared[w];
      all += shared[w];
    }
    if (p.begin < upto && p.begin >= upto - n) {
      shared[THREADS / 32] = b;
      shared[THREADS / 32 + 1] = upto - n;
    }
    __syncthreads();
    before += all;
    if (p.begin < before) break;
  }
  p.b = (int)shared[THREADS / 32];
  p.start = shared[THREADS / 32 + 1];
  return p;
}

// The next segment of a part: which, its tiles within the part, and where
// its result goes.
struct Segment {
  int b, s;             // sequence, and number within it
  int64_t id;           // b * segments + s
  int lo, hi;           // tokens of the sequence
  int first, last;      // tiles here, of the sequence's
  bool head, tail;      // shared with the CTAs before, or only with those after
};
__device__ __forceinline__ bool next_segment(const AttendArgs& a, Part& p, int segments, Segment& g) {
  if (p.at >= p.end) return false;
  Sequence q(a, p.b);
  if (p.at >= p.start + (int64_t)q.tiles * segments) {
    p.start += (int64_t)q.tiles * segments;
    q = Sequence(a, ++p.b);
  }
  g.b = p.b;
  g.s = (int)((p.at - p.start) / q.tiles);
  g.id = (int64_t)p.b * segments + g.s;
  const int64_t start = p.start + (int64_t)g.s * q.tiles, end = start + q.tiles;
  g.lo = q.lo;
  g.hi = q.hi;
  g.first = q.first + (int)(p.at - start);
  g.last = q.first + (int)(min(end, p.end) - start);
  g.head = start < p.begin;
  g.tail = !g.head && end > p.end;
  p.at = min(end, p.end);
  return true;
}

// Where token t's rows lie: its row's element and scale number, or -1.
struct Place {
  int64_t element, scale;
};
__device__ __forceinline__ Place place_of(const AttendArgs& a, int b, int head, int t, int lo, int hi) {
  Place p{-1, -1};
  if (t < lo || t >= hi) return p;
  const int slot = t / (int)a.c.page_size, at = t - slot * (int)a.c.page_size;
  const int page = a.pages[(int64_t)b * a.pages_stride + slot];
  if (page < 0 || page >= a.c.pages) return p;
  const int64_t row = (int64_t)head * a.c.page_size + at;
  p.element = page * a.c.page_stride + row * a.c.D;
  p.scale = page * a.c.scale_stride + row;
  return p;
}

// A row's result from its maximum m (of logits in powers of two), sum l and
// unscaled output; log 2 turns m into powers of e.
__device__ __forceinline__ float lse_of(float m, float l) {
  return l > 0.0f || isnan(l) ? __fmaf_rn(m, 0.6931471805599453f, logf(l)) : -INFINITY;
}

}  // namespace dit
