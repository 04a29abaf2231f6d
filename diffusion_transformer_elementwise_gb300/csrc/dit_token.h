// dit_token.h -- host-side interface between the C entry points of the
// token-transformer operators (dit_token_api.cu) and their kernels.
#pragma once

#include "dit_internal.h"

namespace dit {

// How the rows of a call's tensors are accessed (Unit of dit_unit.cuh, Tile of
// k_embedding.cu).
enum Layout { WIDE, PHASED, NARROW, SHIFTED };

// Weighted RMSNorm over `rows` rows of D elements (k_norm.cu).
struct NormArgs {
  void* res;        // hidden + update (NULL: no update)
  void* out;        // the normed row: the tensors' type, or E4M3
  float* scales;    // E4M3: [rows, groups]
  const void* x;    // hidden
  const void* u;    // update, or NULL
  const void* w;    // weight [D]
  int64_t rows;
  int D;
  float eps, offset;
  float d_f, inv_d;
  int groups;       // E4M3: scales per row
};
// layout: a Layout of dit_unit.cuh that the tensors allow (the E4M3 output,
// a byte an element, needs 8-byte rows beside 16-byte granules of a 16-bit
// type, 4-byte ones beside fp32).  q8: 0 none, 1 one scale per row, 2 one per
// 128 columns.
cudaError_t launch_norm(const DeviceInfo& dev, int dtype, int layout, int q8, const NormArgs& a,
                        cudaStream_t s);

// Its gradient (k_norm_grad.cu).
struct NormGradArgs {
  void* gx;
  void* gw;         // the weight's gradient, where the launcher has it written at once
  float* partial;   // [ctas, D] sums of the weight's gradient, or NULL
  const void* g;    // gradient of the normed output
  const void* gres; // gradient arriving on the skip path, or NULL
  const void* x;    // the norm's input
  const void* w;
  int64_t rows;
  int D;
  float eps, offset;
  float d_f, inv_d;
};
// the most CTAs (rows of `partial`) a call takes
constexpr int64_t kNormGradMaxCtas = 304;
// Up to this many rows that stay in registers take one launch of one cluster;
// up to this width they do in every type and layout, and the call needs no
// workspace.  Wider ones (16-bit types) bring a workspace, whose size is not
// told the type, and take the cluster only up to this many elements.
// Measured, one cluster against two launches over all SMs, with the skip path:
// GPU us, and in brackets us a call among calls (host time included).
//   fp32 128 x 64     3.3  (7.9) |  3.2 (10.6)   bf16 16 x 8184    8.1 (10.4) |  9.2 (11.8)
//   fp32 128 x 2048   8.2 (10.4) |  3.8 (10.9)   bf16  1 x 16384  11.0 (13.5) | 14.7 (16.6)
//   fp32  64 x 4096   8.6 (10.7) |  5.0 (10.8)   bf16 16 x 16384  11.8 (14.5) | 15.2 (17.8)
//   fp32 128 x 4096  12.7 (14.8) |  5.1 (11.0)   bf16 64 x 16384  20.4 (22.7) | 16.5 (18.6)
//   fp32 128 x 8184  20.9 (22.9) |  7.9 (10.7)   bf16 128 x 16384 31.6 (34.1) | 17.2 (19.7)
// A call is the shorter in one cluster up to 2^18 elements; more of at most
// kFewRowsD columns stay there because callers bring no workspace for them.
constexpr int64_t kFewRows = 128, kFewRowsD = 8189, kFewElements = int64_t(1) << 18;
inline bool few_rows(int64_t rows, int64_t D) {
  return rows <= kFewRows && (D <= kFewRowsD || rows * D <= kFewElements);
}
// gw: the weight's gradient, or NULL
cudaError_t launch_norm_grad(const DeviceInfo& dev, int dtype, int layout, const NormGradArgs& a,
                             void* gw, cudaStream_t s);

// Embedding lookup and its gradient (k_embedding.cu).  ids: int32 or int64
// (ids64); ids outside [0, V) give zero rows and take no gradient.
struct EmbedArgs {
  void* out;
  const void* ids;
  const void* table;
  int64_t tokens, V;
  int D;
  bool ids64;
  float scale;
};
cudaError_t launch_embedding(int dtype, int layout, const EmbedArgs& a, cudaStream_t s);

struct EmbedGradArgs {
  void* gt;          // gradient of the table [V, D]
  const void* g;     // gradient of the rows [tokens, D]
  const void* ids;
  int64_t tokens, V;
  int D;
  bool ids64;
  float scale;
  // workspace (more than kFewTokens tokens): two buffers of (key, position)
  // pairs, the list of runs that cross segments, and the partial rows
  uint2* pairs[2];
  uint32_t* runs;    // a count, then at most `segments` entries
  float* partial;    // [segments][2][D]
};
// up to this many tokens the gradient takes one launch and no workspace
constexpr int kFewTokens = 256;
// sorted tokens per segment, and segments of a call
constexpr int kEmbedSegment = 32;
inline int64_t embed_segments(int64_t tokens) { return (tokens + kEmbedSegment - 1) / kEmbedSegment; }
cudaError_t launch_embedding_grad(const DeviceInfo& dev, int dtype, int layout,
                                  const EmbedGradArgs& a, cudaStream_t s);

// The global norm of many tensors, and their clipping (k_clip.cu).
struct ClipTensor {
  const void* g;
  void* out;  // NULL: the norm alone
  int64_t n;
  int dtype;
};
// the most tensors of one launch, and partial sums it writes
constexpr int kClipBatch = 960;
constexpr int64_t kClipMaxCtas = 1216;
// partial: kClipMaxCtas doubles per kClipBatch tensors.  norm: the norm.
// clip: also out = g * min(1, max_norm / (norm + eps)).
cudaError_t launch_clip(const DeviceInfo& dev, const ClipTensor* t, int64_t count, bool clip,
                        float max_norm, float eps, double* partial, float* norm, cudaStream_t s);

}  // namespace dit
