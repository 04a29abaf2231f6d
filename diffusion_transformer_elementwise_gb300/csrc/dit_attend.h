// dit_attend.h -- host-side interface between the C entry points of the
// operators around attention (dit_attend_api.cu) and their kernels.
#pragma once

#include "dit_elementwise.h"
#include "dit_internal.h"

namespace dit {

// cos and sin of rotary angles (k_rope.cu)
struct TableArgs {
  float *cos, *sin;
  const void* positions;  // [axes, tokens]
  const double* freqs;    // [R]
  int64_t tokens;
  int R, axes;
  int end[DIT_MAX_AXES];  // the first column behind each axis
};
cudaError_t launch_table(const DeviceInfo& dev, int position_type, const TableArgs& a,
                         cudaStream_t s);

// Rotation of heads, with or without a norm (k_rope.cu), and the gradient
// (k_rope_grad.cu).  Tensor 0 holds the queries, 1 the keys (H = 0: none).
struct RopeTensor {
  dit_heads x, out, g;  // g: the gradient of out (gradient only, where out is x's)
  const void* w;        // weight [D], or NULL (no norm)
  int H;
};
struct RopeArgs {
  RopeTensor t[2];
  const float *cos, *sin;
  int64_t tokens, L;      // B * L, L
  int64_t table_rows;     // of cos and sin
  int D, R;
  float eps, offset, inv_d;  // inv_d: fl(1 / D)
  bool interleaved, inverse;
  bool granules;          // every tensor lies on 16-byte boundaries, row by row
  float* partial;         // gradient: rows of D, the CTAs' sums of a weight's gradient
};
cudaError_t launch_rope(const DeviceInfo& dev, int dtype, const RopeArgs& a, cudaStream_t s);
// half of the most rows of `partial`
constexpr int64_t kRopeGradMaxCtas = 608;
cudaError_t launch_rope_grad(const DeviceInfo& dev, int dtype, const RopeArgs& a, void* gwq,
                             void* gwk, cudaStream_t s);

// Rows into and out of a paged cache (k_cache.cu)
struct CacheArgs {
  dit_cache c;
  dit_heads k, v;
  int64_t tokens;
  const void* slots;
  bool ids64;
  bool granules;  // every row lies on 16-byte boundaries
};
cudaError_t launch_cache_write(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s);
cudaError_t launch_cache_read(const DeviceInfo& dev, int dtype, const CacheArgs& a, cudaStream_t s);

// Attention of one token per sequence (k_attend.cu)
struct AttendArgs {
  dit_cache c;
  dit_heads q, out;
  float* lse;
  const int32_t* pages;
  int64_t pages_stride;
  int64_t capacity;     // width * page_size
  const void* lengths;
  bool ids64;
  int B, Hq, group;     // group: query heads of a key head
  int rows;             // of them in a segment: kAttendRows, or 8
  float scale;
  int64_t window;
  float* partial;       // [ctas][2][rows][D + 2]: the parts of split segments
  int64_t* owner;       // [ctas][2]: their segments, or -1
};
// query heads that share a pass over the keys, and the most CTAs
constexpr int kAttendRows = 16;
constexpr int64_t kAttendMaxCtas = 608;
cudaError_t launch_attend(const DeviceInfo& dev, int dtype, bool granules, const AttendArgs& a,
                          cudaStream_t s);

// The tensor cores' form of its first kernel (k_attend_mma.cu): at most 256
// columns in 16-byte granules.  Sets a.rows.  Its CTAs and their warps have parts of their own behind
// `partial`: [ctas][warps][2][rows][D + 2].
constexpr int64_t kAttendMmaCtas = 160;
// the most warps of a CTA, of any type, for heads of D columns (0: it does not take them)
constexpr int attend_warps(int64_t D) { return D <= 64 ? 16 : D <= 128 ? 12 : D <= 256 ? 8 : 0; }
bool attend_mma_takes(bool granules, const AttendArgs& a);
cudaError_t launch_attend_mma(const DeviceInfo& dev, int dtype, AttendArgs& a, int64_t* ctas, cudaStream_t s);
cudaError_t launch_attend_mma_fp32(const DeviceInfo& dev, AttendArgs& a, int64_t* ctas, cudaStream_t s);

}  // namespace dit
