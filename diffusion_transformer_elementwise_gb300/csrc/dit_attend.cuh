// dit_attend.cuh -- how the attention of one token per sequence is divided
// over the GPU (sm_103a).
//
// A segment is one sequence's tokens for up to kAttendRows query heads of one
// key head; its tokens come in tiles of 32.  The tiles of all segments form one
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

constexpr int kTile = 32;

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

// Shared memory of a CTA that finds its place on the line.
template <int THREADS>
struct Plan {
  int64_t start[THREADS];
  int64_t sum[THREADS / 32];
  // the sum of v over this thread and those before it
  __device__ __forceinline__ int64_t upto(int64_t v) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
      const int64_t w = __shfl_up_sync(0xFFFFFFFFu, v, o);
      if (lane >= o) v += w;
    }
    if (lane == 31) sum[warp] = v;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < THREADS / 32; ++w)
      if (w < warp) v += sum[w];
    __syncthreads();
    return v;
  }
};

// a / b of positive numbers, in 32 bits where they fit
__device__ __forceinline__ int64_t divided(int64_t a, int64_t b) {
  return ((a | b) >> 32) == 0 ? (int64_t)((uint32_t)a / (uint32_t)b) : a / b;
}
// A segment's name.
__device__ __forceinline__ int64_t segment_id(int b, int s) { return (int64_t)b << 32 | (uint32_t)s; }

// A place of the line: a sequence, and where on the line it starts.
struct Mark {
  int b;
  int64_t start;
};

// The line: each of a sequence's `segments` segments takes its tiles and `extra` units more, which stand for
// the time that a segment takes whatever its length.
struct Line {
  int segments, extra;
  __device__ __forceinline__ int64_t length(const Sequence& q) const {
    return (int64_t)(q.tiles + extra) * segments;
  }
  // The line's length, for the whole CTA; `plan` keeps where up to THREADS sequences start.
  template <int THREADS>
  __device__ __forceinline__ int64_t total(const AttendArgs& a, Plan<THREADS>& plan) const {
    int64_t mine = 0;
    if (a.B <= THREADS) {
      if (threadIdx.x < a.B) mine = length(Sequence(a, threadIdx.x));
      const int64_t upto = plan.upto(mine);
      plan.start[threadIdx.x] = upto - mine;
      if (threadIdx.x == THREADS - 1) plan.sum[0] = upto;
      __syncthreads();
      return plan.sum[0];
    }
    for (int b = threadIdx.x; b < a.B; b += THREADS) mine += length(Sequence(a, b));
    mine = plan.upto(mine);
    if (threadIdx.x == THREADS - 1) plan.start[0] = mine;
    __syncthreads();
    mine = plan.start[0];
    __syncthreads();
    return mine;
  }
  // the sequence that holds unit `at` of the line, for the whole CTA
  template <int THREADS>
  __device__ __forceinline__ Mark find(const AttendArgs& a, int64_t at, Plan<THREADS>& plan) const {
    if (a.B <= THREADS) {
      int lo = 0, hi = a.B;  // start[lo] <= at < start[hi]
      while (hi - lo > 1) {
        const int mid = (lo + hi) / 2;
        if (plan.start[mid] <= at)
          lo = mid;
        else
          hi = mid;
      }
      return Mark{lo, plan.start[lo]};
    }
    int64_t before = 0;
    for (int b0 = 0; b0 < a.B; b0 += THREADS) {
      const int b = b0 + threadIdx.x;
      const int64_t n = b < a.B ? length(Sequence(a, b)) : 0;
      const int64_t upto = before + plan.upto(n);
      if (at < upto && at >= upto - n) {
        plan.start[0] = b;
        plan.start[1] = upto - n;
      }
      if (threadIdx.x == THREADS - 1) plan.start[2] = upto;
      __syncthreads();
      before = plan.start[2];
      if (at < before) break;
      __syncthreads();
    }
    const Mark m{(int)plan.start[0], plan.start[1]};
    __syncthreads();
    return m;
  }
  // the same for one warp, from a mark at or before it
  __device__ __forceinline__ Mark find_from(const AttendArgs& a, int64_t at, Mark m) const {
    const int lane = threadIdx.x & 31;
    for (;;) {
      const int b = m.b + lane;
      const int64_t n = b < a.B ? length(Sequence(a, b)) : 0;
      int64_t upto = n;
#pragma unroll
      for (int o = 1; o < 32; o <<= 1) {
        const int64_t v = __shfl_up_sync(0xFFFFFFFFu, upto, o);
        if (lane >= o) upto += v;
      }
      upto += m.start;
      const uint32_t past = __ballot_sync(0xFFFFFFFFu, at < upto);
      if (past) {
        const int first = __ffs(past) - 1;
        return Mark{m.b + first, __shfl_sync(0xFFFFFFFFu, upto - n, first)};
      }
      m.start = __shfl_sync(0xFFFFFFFFu, upto, 31);
      m.b += 32;
    }
  }
};

// A segment's tiles within a part of the line.
struct Segment {
  int b, s;             // sequence, and number within it
  int lo, hi;           // tokens of the sequence
  int first, last;      // tiles here, of the sequence's
  bool open, head, tail;  // goes on in the next part; begun in an earlier one; begun here and open
};

// A walk over the segments of the part [at, end) of the line.
struct Walk {
  int64_t at, end, start;  // start: of the segment at hand
  int b, s;
  Sequence q;
  // mark: the sequence that holds `at`, if the part is not empty
  __device__ __forceinline__ Walk(const AttendArgs& a, const Line& line, int64_t at, int64_t end, Mark mark)
      : at(at), end(end), start(mark.start), b(mark.b), s(0), q(a, mark.b) {
    if (at >= end) return;
    const int64_t n = q.tiles + line.extra;
    s = (int)divided(at - start, n);
    start += s * n;
  }
  __device__ __forceinline__ bool next(const AttendArgs& a, const Line& line, Segment& g) {
    while (at < end) {
      const int64_t n = q.tiles + line.extra, stop = min(end - start, n);
      const int first = max(0, (int)(at - start) - line.extra), last = max(0, (int)stop - line.extra);
      g.b = b;
      g.s = s;
      g.lo = q.lo;
      g.hi = q.hi;
      g.first = q.first + first;
      g.last = q.first + last;
      g.head = first > 0;
      g.open = last < q.tiles;
      g.tail = g.open && !g.head;
      at = start + stop;
      if (stop == n) {
        start = at;
        if (++s == line.segments) {
          s = 0;
          if (++b < a.B) q = Sequence(a, b);
        }
      }
      if (last > first) return true;  // (no tile where the part ends within `extra`)
    }
    return false;
  }
};

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
