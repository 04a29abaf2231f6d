// dit_token_api.cu -- the C entry points of the token-transformer operators
// (include/dit_elementwise.h): argument validation, aliasing rules and the
// division of the workspaces.  Nothing is allocated on the device.
#include <math.h>

#include <algorithm>
#include <new>

#include "dit_checks.h"
#include "dit_elementwise.h"
#include "dit_token.h"

using dit::DeviceInfo;
using dit::Span;
using dit::elem_size;
using dit::element_count;
using dit::launch_status;
using dit::misaligned;
using dit::overlaps;
using dit::span;
using dit::valid_dtype;

namespace {

constexpr int64_t kMaxRow = int64_t(1) << 24;
constexpr int64_t kMaxCount = 0x7FFFFFFF;
constexpr int64_t kAlign = 256;

bool finite(float v) { return !isnan(v) && !isinf(v); }
int64_t round_up(int64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

// sizes of a [rows, D] tensor: the element count, or false
bool row_shape(int64_t rows, int64_t D, int es, int64_t* n) {
  return rows <= kMaxCount && D <= kMaxRow && element_count(rows, D, 1, es, n);
}

// whether tensors that start at the addresses in `bits` (ORed) with rows of
// row_bytes are made of 16-byte granules
bool wide_rows(uint64_t bits, int64_t row_bytes) { return ((bits | (uint64_t)row_bytes) & 15u) == 0; }

// streamed: the addresses (ORed) of the tensors read or written row by row
dit::Layout layout_of(uint64_t streamed, const void* weight, int64_t row_bytes) {
  if (wide_rows(streamed | (uintptr_t)weight, row_bytes)) return dit::WIDE;
  return (streamed & 15u) == 0 ? dit::PHASED : dit::NARROW;
}

dit_status workspace_status(const void* w, int64_t have, int64_t need) {
  if (!w || ((uintptr_t)w & (uintptr_t)(kAlign - 1)) != 0 || have < need) return DIT_ERR_WORKSPACE;
  return DIT_OK;
}

// q8: 0 none, 1 a scale per row, 2 one per 128 columns
dit_status norm_impl(bool add, int q8, void* res, void* out, float* scales, const void* x,
                     const void* u, const void* w, int64_t rows, int64_t D, float eps,
                     float offset, dit_dtype dtype, dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  const int es = elem_size(dtype);
  int64_t n;
  if (!row_shape(rows, D, es, &n)) return DIT_ERR_BAD_SHAPE;
  if (!(eps >= 0.0f) || isinf(eps)) return DIT_ERR_BAD_EPS;
  if (!finite(offset)) return DIT_ERR_BAD_SCALAR;
  if (n == 0 && (q8 != 1 || rows == 0 || !scales)) return DIT_OK;
  if (n == 0) {  // rows of no columns: their scales are zero
    if (misaligned(scales, 4)) return DIT_ERR_MISALIGNED;
    DeviceInfo dev;
    if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
    const cudaError_t e = cudaMemsetAsync(scales, 0, (size_t)rows * 4, (cudaStream_t)stream);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return launch_status(e);
  }
  if (!out || !x || !w || (add && (!res || !u)) || (q8 && !scales)) return DIT_ERR_NULL_PTR;
  if (misaligned(x, es) || misaligned(w, es) || (!q8 && misaligned(out, es)) ||
      (add && (misaligned(res, es) || misaligned(u, es))) || (q8 && misaligned(scales, 4)))
    return DIT_ERR_MISALIGNED;
  const int64_t groups = q8 == 2 ? (D + 127) / 128 : 1;
  const int64_t bytes = n * es;
  const Span ins[3] = {span(x, bytes), span(w, D * es), span(u, bytes)};
  const int nins = add ? 3 : 2;
  Span outs[3];
  int nouts = 0;
  outs[nouts++] = span(out, q8 ? n : bytes);
  if (q8) outs[nouts++] = span(scales, rows * groups * 4);
  const int ires = nouts;
  if (add) outs[nouts++] = span(res, bytes);
  for (int i = 0; i < nouts; ++i) {
    for (int j = i + 1; j < nouts; ++j)
      if (overlaps(outs[i], outs[j])) return DIT_ERR_ALIAS;
    for (int j = 0; j < nins; ++j) {
      if (i == ires && j == 0 && res == x) continue;  // the residual in place
      if (overlaps(outs[i], ins[j])) return DIT_ERR_ALIAS;
    }
  }
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  dit::NormArgs a = {};
  a.res = add ? res : nullptr;
  a.out = out;
  a.scales = scales;
  a.x = x;
  a.u = add ? u : nullptr;
  a.w = w;
  a.rows = rows;
  a.D = (int)D;
  a.eps = eps;
  a.offset = offset;
  a.d_f = (float)D;
  a.inv_d = 1.0f / (float)D;
  a.groups = (int)groups;
  uint64_t bits = (uintptr_t)x;
  if (add) bits |= (uintptr_t)u | (uintptr_t)res;
  // an E4M3 row has 8 (fp32: 4) bytes for each granule of the input's
  bits |= q8 ? (uint64_t)((uintptr_t)out & (uintptr_t)(16 / es - 1)) : (uint64_t)(uintptr_t)out;
  return launch_status(dit::launch_norm(dev, dtype, layout_of(bits, w, D * es), q8, a,
                                        (cudaStream_t)stream));
}

bool valid_group(int64_t group) { return group == 0 || group == 128; }

}  // namespace

extern "C" {

dit_status dit_rmsnorm(void* out, const void* x, const void* weight, int64_t rows, int64_t D,
                       float eps, float weight_offset, dit_dtype dtype, dit_stream_t stream) {
  return norm_impl(false, 0, nullptr, out, nullptr, x, nullptr, weight, rows, D, eps,
                   weight_offset, dtype, stream);
}

dit_status dit_add_rmsnorm(void* residual_out, void* out, const void* hidden, const void* update,
                           const void* weight, int64_t rows, int64_t D, float eps,
                           float weight_offset, dit_dtype dtype, dit_stream_t stream) {
  return norm_impl(true, 0, residual_out, out, nullptr, hidden, update, weight, rows, D, eps,
                   weight_offset, dtype, stream);
}

dit_status dit_rmsnorm_fp8(void* out, float* scales, const void* x, const void* weight,
                           int64_t rows, int64_t D, int64_t group, float eps, float weight_offset,
                           dit_dtype dtype, dit_stream_t stream) {
  if (!valid_group(group)) return DIT_ERR_BAD_FORMAT;
  return norm_impl(false, group ? 2 : 1, nullptr, out, scales, x, nullptr, weight, rows, D, eps,
                   weight_offset, dtype, stream);
}

dit_status dit_add_rmsnorm_fp8(void* residual_out, void* out, float* scales, const void* hidden,
                               const void* update, const void* weight, int64_t rows, int64_t D,
                               int64_t group, float eps, float weight_offset, dit_dtype dtype,
                               dit_stream_t stream) {
  if (!valid_group(group)) return DIT_ERR_BAD_FORMAT;
  return norm_impl(true, group ? 2 : 1, residual_out, out, scales, hidden, update, weight, rows, D,
                   eps, weight_offset, dtype, stream);
}

int64_t dit_rmsnorm_backward_workspace_bytes(int64_t rows, int64_t D) {
  int64_t n;
  if (!row_shape(rows, D, 4, &n)) return -1;
  if (rows <= dit::kFewRows && D <= dit::kFewRowsD) return 0;
  return round_up(std::min(rows, dit::kNormGradMaxCtas) * D * 4);
}

dit_status dit_rmsnorm_backward(void* grad_x, void* grad_weight, const void* grad_out,
                                const void* grad_residual, const void* x, const void* weight,
                                int64_t rows, int64_t D, float eps, float weight_offset,
                                dit_dtype dtype, void* workspace, int64_t workspace_bytes,
                                dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  const int es = elem_size(dtype);
  int64_t n;
  if (!row_shape(rows, D, es, &n)) return DIT_ERR_BAD_SHAPE;
  if (!(eps >= 0.0f) || isinf(eps)) return DIT_ERR_BAD_EPS;
  if (!finite(weight_offset)) return DIT_ERR_BAD_SCALAR;
  if (D == 0 || (n == 0 && !grad_weight)) return DIT_OK;
  if (n > 0 && (!grad_x || !grad_out || !x || !weight)) return DIT_ERR_NULL_PTR;
  if (misaligned(grad_x, es) || misaligned(grad_weight, es) || misaligned(grad_out, es) ||
      misaligned(grad_residual, es) || misaligned(x, es) || misaligned(weight, es))
    return DIT_ERR_MISALIGNED;
  const int64_t need = dit_rmsnorm_backward_workspace_bytes(rows, D);
  const bool use_ws = grad_weight && n > 0 && need > 0;
  if (use_ws) {
    const dit_status st = workspace_status(workspace, workspace_bytes, need);
    if (st != DIT_OK) return st;
  }
  const int64_t bytes = n * es, wbytes = D * es;
  const Span ins[4] = {span(grad_out, bytes), span(grad_residual, grad_residual ? bytes : 0),
                       span(x, bytes), span(weight, wbytes)};
  const Span sx = span(grad_x, bytes), sw = span(grad_weight, grad_weight ? wbytes : 0);
  const Span ws = span(workspace, use_ws ? need : 0);
  if (overlaps(sx, sw) || overlaps(sx, ws) || overlaps(sw, ws)) return DIT_ERR_ALIAS;
  for (int i = 0; i < 4; ++i) {
    if (overlaps(sw, ins[i]) || overlaps(ws, ins[i])) return DIT_ERR_ALIAS;
    if ((i == 0 && grad_x == grad_out) || (i == 1 && grad_x == grad_residual)) continue;
    if (overlaps(sx, ins[i])) return DIT_ERR_ALIAS;
  }
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  if (n == 0) {  // no rows: the weight's gradient is zero
    const cudaError_t e = cudaMemsetAsync(grad_weight, 0, (size_t)wbytes, (cudaStream_t)stream);
    if (e != cudaSuccess) (void)cudaGetLastError();
    return launch_status(e);
  }
  dit::NormGradArgs a = {};
  a.gx = grad_x;
  a.partial = use_ws ? (float*)workspace : nullptr;
  a.g = grad_out;
  a.gres = grad_residual;
  a.x = x;
  a.w = weight;
  a.rows = rows;
  a.D = (int)D;
  a.eps = eps;
  a.offset = weight_offset;
  a.d_f = (float)D;
  a.inv_d = 1.0f / (float)D;
  const uint64_t bits =
      (uintptr_t)grad_x | (uintptr_t)grad_out | (uintptr_t)grad_residual | (uintptr_t)x;
  return launch_status(dit::launch_norm_grad(dev, dtype, layout_of(bits, weight, D * es), a,
                                             grad_weight, (cudaStream_t)stream));
}

dit_status dit_embedding(void* out, const void* ids, const void* table, int64_t tokens, int64_t V,
                         int64_t D, float scale, dit_dtype dtype, dit_id_type id_type,
                         dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  if (id_type != DIT_INT32 && id_type != DIT_INT64) return DIT_ERR_BAD_FORMAT;
  const int es = elem_size(dtype), is = id_type == DIT_INT64 ? 8 : 4;
  int64_t n, nt;
  if (!row_shape(tokens, D, es, &n) || !row_shape(V, D, es, &nt)) return DIT_ERR_BAD_SHAPE;
  if (!finite(scale)) return DIT_ERR_BAD_SCALAR;
  if (n == 0) return DIT_OK;
  if (!out || !ids || (nt > 0 && !table)) return DIT_ERR_NULL_PTR;
  if (misaligned(out, es) || misaligned(ids, is) || misaligned(table, es)) return DIT_ERR_MISALIGNED;
  const Span so = span(out, n * es);
  if (overlaps(so, span(ids, tokens * is)) || overlaps(so, span(table, nt * es)))
    return DIT_ERR_ALIAS;
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  dit::EmbedArgs a = {};
  a.out = out;
  a.ids = ids;
  a.table = table;
  a.tokens = tokens;
  a.V = V;
  a.D = (int)D;
  a.ids64 = id_type == DIT_INT64;
  a.scale = scale;
  const dit::Layout layout = layout_of((uintptr_t)out | (uintptr_t)table, nullptr, D * es);
  return launch_status(dit::launch_embedding(dtype, layout, a, (cudaStream_t)stream));
}

int64_t dit_embedding_backward_workspace_bytes(int64_t tokens, int64_t D) {
  int64_t n, m;
  if (!row_shape(tokens, D, 4, &n)) return -1;
  if (tokens <= dit::kFewTokens) return 0;
  // two buffers of (key, position) pairs, the list of runs that cross
  // segments, two partial rows per segment
  const int64_t segments = dit::embed_segments(tokens);
  if (__builtin_mul_overflow(segments * 2, D * 4, &m)) return -1;
  return 2 * round_up(tokens * 8) + round_up((segments + 1) * 4) + round_up(m);
}

dit_status dit_embedding_backward(void* grad_table, const void* grad_out, const void* ids,
                                  int64_t tokens, int64_t V, int64_t D, float scale,
                                  dit_dtype dtype, dit_id_type id_type, void* workspace,
                                  int64_t workspace_bytes, dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  if (id_type != DIT_INT32 && id_type != DIT_INT64) return DIT_ERR_BAD_FORMAT;
  const int es = elem_size(dtype), is = id_type == DIT_INT64 ? 8 : 4;
  int64_t n, nt;
  if (!row_shape(tokens, D, es, &n) || !row_shape(V, D, es, &nt)) return DIT_ERR_BAD_SHAPE;
  if (!finite(scale)) return DIT_ERR_BAD_SCALAR;
  if (nt == 0) return DIT_OK;
  if (!grad_table || (tokens > 0 && (!grad_out || !ids))) return DIT_ERR_NULL_PTR;
  if (misaligned(grad_table, es) || misaligned(grad_out, es) || misaligned(ids, is))
    return DIT_ERR_MISALIGNED;
  const int64_t need = dit_embedding_backward_workspace_bytes(tokens, D);
  if (need < 0) return DIT_ERR_BAD_SHAPE;
  if (need > 0) {
    const dit_status st = workspace_status(workspace, workspace_bytes, need);
    if (st != DIT_OK) return st;
  }
  const Span so = span(grad_table, nt * es), ws = span(workspace, need);
  const Span sg = span(grad_out, n * es), si = span(ids, tokens * is);
  if (overlaps(so, ws) || overlaps(so, sg) || overlaps(so, si) || overlaps(ws, sg) ||
      overlaps(ws, si))
    return DIT_ERR_ALIAS;
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  dit::EmbedGradArgs a = {};
  a.gt = grad_table;
  a.g = grad_out;
  a.ids = ids;
  a.tokens = tokens;
  a.V = V;
  a.D = (int)D;
  a.ids64 = id_type == DIT_INT64;
  a.scale = scale;
  if (need > 0) {
    char* w = (char*)workspace;
    a.pairs[0] = (uint2*)w;
    a.pairs[1] = (uint2*)(w += round_up(tokens * 8));
    a.runs = (uint32_t*)(w += round_up(tokens * 8));
    a.partial = (float*)(w + round_up((dit::embed_segments(tokens) + 1) * 4));
  }
  const dit::Layout layout =
      layout_of((uintptr_t)grad_table | (uintptr_t)grad_out, nullptr, D * es);
  return launch_status(dit::launch_embedding_grad(dev, dtype, layout, a, (cudaStream_t)stream));
}

}  // extern "C"

namespace {

// An input or output span of a clipping call; an in-place tensor is one
// output.
struct Region {
  Span s;
  bool out;
};

// Checks the descriptions and their overlaps (clip: with the outputs), and
// fills `t` (count entries) and `r` (2 * count).
dit_status prepare_clip(bool clip, const dit_tensor* q, int64_t count, Span norm, Span ws,
                        dit::ClipTensor* t, Region* r) {
  int64_t nr = 0;
  for (int64_t i = 0; i < count; ++i) {
    if (q[i].dtype < 0 || q[i].dtype > 2) return DIT_ERR_BAD_DTYPE;
    const int es = elem_size((dit_dtype)q[i].dtype);
    if (q[i].n < 0 || q[i].n > (int64_t(1) << 44)) return DIT_ERR_BAD_SHAPE;
    if (q[i].n > 0) {
      if (!q[i].g || (clip && !q[i].out)) return DIT_ERR_NULL_PTR;
      if (misaligned(q[i].g, es) || (clip && misaligned(q[i].out, es))) return DIT_ERR_MISALIGNED;
      const Span g = span(q[i].g, q[i].n * es);
      if (overlaps(g, norm) || overlaps(g, ws)) return DIT_ERR_ALIAS;
      if (clip) {
        const Span o = span(q[i].out, q[i].n * es);
        if (overlaps(o, norm) || overlaps(o, ws)) return DIT_ERR_ALIAS;
        r[nr++] = Region{o, true};
        if (q[i].out != q[i].g) r[nr++] = Region{g, false};
      }
    }
    t[i] = dit::ClipTensor{q[i].g, clip ? q[i].out : nullptr, q[i].n, (int)q[i].dtype};
  }
  // sorted by address: an output overlaps an earlier region if it starts
  // before the furthest end of them all, an input if before that of the outputs
  std::sort(r, r + nr, [](const Region& a, const Region& b) { return a.s.lo < b.s.lo; });
  uintptr_t end_all = 0, end_out = 0;
  for (int64_t i = 0; i < nr; ++i) {
    if (r[i].s.lo < (r[i].out ? end_all : end_out)) return DIT_ERR_ALIAS;
    end_all = std::max(end_all, r[i].s.hi);
    if (r[i].out) end_out = std::max(end_out, r[i].s.hi);
  }
  return DIT_OK;
}

dit_status clip_impl(bool clip, float* norm, const dit_tensor* tensors, int64_t count,
                     float max_norm, float eps, void* workspace, int64_t workspace_bytes,
                     dit_stream_t stream) {
  if (count < 0 || count > kMaxCount) return DIT_ERR_BAD_SHAPE;
  if (clip && (!finite(max_norm) || max_norm < 0.0f)) return DIT_ERR_BAD_SCALAR;
  if (clip && (!(eps >= 0.0f) || isinf(eps))) return DIT_ERR_BAD_EPS;
  if (!norm || (count > 0 && !tensors)) return DIT_ERR_NULL_PTR;
  if (misaligned(norm, 4)) return DIT_ERR_MISALIGNED;
  const int64_t need = dit_grad_norm_workspace_bytes(count);
  const dit_status wst = workspace_status(workspace, workspace_bytes, need);
  if (wst != DIT_OK) return wst;
  const Span sn = span(norm, 4), ws = span(workspace, need);
  if (overlaps(sn, ws)) return DIT_ERR_ALIAS;
  dit::ClipTensor* t = new (std::nothrow) dit::ClipTensor[count > 0 ? count : 1];
  Region* r = new (std::nothrow) Region[count > 0 ? 2 * count : 1];
  dit_status st = t && r ? prepare_clip(clip, tensors, count, sn, ws, t, r) : DIT_ERR_NO_MEMORY;
  DeviceInfo dev;
  if (st == DIT_OK && dit::current_device(&dev) != cudaSuccess) st = DIT_ERR_NO_DEVICE;
  if (st == DIT_OK)
    st = launch_status(dit::launch_clip(dev, t, count, clip, max_norm, eps, (double*)workspace,
                                        norm, (cudaStream_t)stream));
  delete[] t;
  delete[] r;
  return st;
}

}  // namespace

extern "C" {

int64_t dit_grad_norm_workspace_bytes(int64_t count) {
  if (count < 0 || count > kMaxCount) return -1;
  // launches of up to 64 or kClipBatch tensors, each with its partial sums
  const int64_t batches = (count + dit::kClipBatch - 1) / dit::kClipBatch;
  return round_up(std::max<int64_t>(1, batches) * dit::kClipMaxCtas * 8);
}

dit_status dit_grad_norm(float* norm, const dit_tensor* tensors, int64_t count, void* workspace,
                         int64_t workspace_bytes, dit_stream_t stream) {
  return clip_impl(false, norm, tensors, count, 0.0f, 0.0f, workspace, workspace_bytes, stream);
}

dit_status dit_clip_grads(float* norm, const dit_tensor* tensors, int64_t count, float max_norm,
                          float eps, void* workspace, int64_t workspace_bytes,
                          dit_stream_t stream) {
  return clip_impl(true, norm, tensors, count, max_norm, eps, workspace, workspace_bytes, stream);
}

}  // extern "C"
