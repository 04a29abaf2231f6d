// dit_attend_api.cu -- the C entry points of the operators around attention
// (include/dit_elementwise.h): argument validation, aliasing rules and the
// division of the workspaces.  Nothing is allocated on the device.
#include <math.h>

#include <algorithm>

#include "dit_attend.h"
#include "dit_checks.h"

using dit::DeviceInfo;
using dit::Span;
using dit::elem_size;
using dit::launch_status;
using dit::misaligned;
using dit::overlaps;
using dit::span;
using dit::valid_dtype;

namespace {

constexpr int64_t kMaxCount = 0x7FFFFFFF;
constexpr int64_t kMaxStride = int64_t(1) << 40;
constexpr int64_t kMaxHeadDim = 1024, kMaxAttendDim = 512;
constexpr int64_t kMaxHeads = 65535;
constexpr int64_t kMaxPairs = 512;
constexpr int64_t kMaxTokens = 0x7FFFF000;  // of a sequence: token numbers past its end fit an int
constexpr int64_t kAlign = 256;

bool finite(float v) { return !isnan(v) && !isinf(v); }
int64_t round_up(int64_t n) { return (n + kAlign - 1) / kAlign * kAlign; }

dit_status workspace_status(const void* w, int64_t have, int64_t need) {
  if (!w || ((uintptr_t)w & (uintptr_t)(kAlign - 1)) != 0 || have < need) return DIT_ERR_WORKSPACE;
  return DIT_OK;
}

// A view in bytes: four sizes (the last contiguous) and their strides.
struct View {
  uintptr_t p;
  int64_t size[3], stride[3];
  int64_t row;  // bytes of a row
};
// false for a stride that is negative or too large.  (Strides below 2^40 and counts below 2^31
// keep every sum below in 64 bits only if checked: overflow is a refusal.)
bool view(const dit_heads& t, int64_t B, int64_t L, int64_t H, int64_t D, int es, View* v) {
  const int64_t size[3] = {B, L, H}, stride[3] = {t.batch, t.token, t.head};
  int64_t end = D * es;
  for (int i = 0; i < 3; ++i) {
    const int64_t s = size[i] > 1 ? stride[i] : 0;
    int64_t far;
    if (s < 0 || s > kMaxStride || __builtin_mul_overflow(s * es, size[i] > 1 ? size[i] - 1 : 0, &far) ||
        __builtin_add_overflow(end, far, &end))
      return false;
    v->size[i] = size[i];
    v->stride[i] = s * es;
  }
  if (end > (int64_t(1) << 46)) return false;
  v->p = (uintptr_t)t.p;
  v->row = D * es;
  return true;
}
Span span_of(const View& v) {
  int64_t n = v.row;
  for (int i = 0; i < 3; ++i) n += v.size[i] > 1 ? (v.size[i] - 1) * v.stride[i] : 0;
  return Span{v.p, v.p + (uintptr_t)n};
}
bool same(const View& a, const View& b) {
  if (a.p != b.p) return false;
  for (int i = 0; i < 3; ++i)
    if (a.size[i] != b.size[i] || (a.size[i] > 1 && a.stride[i] != b.stride[i])) return false;
  return a.row == b.row;
}
// whether no two elements of the view are the same
bool apart(const View& v) {
  int order[3] = {0, 1, 2};
  std::sort(order, order + 3, [&](int a, int b) { return v.stride[a] < v.stride[b]; });
  int64_t end = v.row;
  for (int i : order) {
    if (v.size[i] <= 1) continue;
    if (v.stride[i] < end) return false;
    end += (v.size[i] - 1) * v.stride[i];
  }
  return true;
}
// Bytes that a view covers modulo m: the strides that are multiples of m stay in place.
int64_t within(const View& v, int64_t m) {
  int64_t n = v.row;
  for (int i = 0; i < 3; ++i)
    if (v.size[i] > 1 && v.stride[i] % m != 0) n += (v.size[i] - 1) * v.stride[i];
  return n;
}
// Whether two views touch: not if their spans do not, nor if they lie in different
// parts of a common period (a token of a packed projection, say).
bool touch(const View& a, const View& b) {
  if (!overlaps(span_of(a), span_of(b))) return false;
  for (const View* v : {&a, &b}) {
    for (int i = 0; i < 3; ++i) {
      const int64_t m = v->size[i] > 1 ? v->stride[i] : 0;
      if (m <= 0) continue;
      const int64_t ea = within(a, m), eb = within(b, m);
      int64_t at = (int64_t)(b.p - a.p) % m;
      if (at < 0) at += m;
      if (at >= ea && at + eb <= m) return false;
    }
  }
  return true;
}
bool touch(const View& a, Span s) { return overlaps(span_of(a), s); }

// every row of the view starts on a 16-byte boundary and is made of granules
bool granules(const View& v) {
  uint64_t bits = (uint64_t)v.p | (uint64_t)v.row;
  for (int i = 0; i < 3; ++i)
    if (v.size[i] > 1) bits |= (uint64_t)v.stride[i];
  return (bits & 15u) == 0;
}

struct RopeCall {
  const dit_heads *out[2], *g[2], *x[2];
  const void* w[2];
  const float *cos, *sin;
  int64_t B, L, H[2], D, R, table_rows;
  float eps, offset;
  int interleaved, inverse;
  dit_dtype dtype;
  bool norm, grad;
};

// The checks of the rotating calls; `go` tells whether there is anything to launch.
dit_status rope_checks(const RopeCall& c, dit::RopeArgs* a, View (*views)[3], bool* go) {
  *go = false;
  if (!valid_dtype(c.dtype)) return DIT_ERR_BAD_DTYPE;
  if ((c.interleaved != 0 && c.interleaved != 1) || (c.inverse != 0 && c.inverse != 1))
    return DIT_ERR_BAD_LAYOUT;
  const int es = elem_size(c.dtype);
  int64_t tokens;
  if (c.B < 0 || c.L < 0 || __builtin_mul_overflow(c.B, c.L, &tokens) || tokens > kMaxCount ||
      c.H[0] < 0 || c.H[0] > kMaxHeads || c.H[1] < 0 || c.H[1] > kMaxHeads || c.D < 0 ||
      c.D > kMaxHeadDim || c.R < 0 || 2 * c.R > c.D ||
      (c.table_rows != c.L && c.table_rows != tokens))
    return DIT_ERR_BAD_SHAPE;
  if (c.norm && (!(c.eps >= 0.0f) || isinf(c.eps))) return DIT_ERR_BAD_EPS;
  if (c.norm && !finite(c.offset)) return DIT_ERR_BAD_SCALAR;
  *a = dit::RopeArgs{};
  a->granules = true;
  const bool any = tokens > 0 && c.D > 0 && c.H[0] + c.H[1] > 0;
  const int64_t table = any ? c.table_rows * c.R * 4 : 0;
  if (table > 0 && (!c.cos || !c.sin)) return DIT_ERR_NULL_PTR;
  if (misaligned(c.cos, 4) || misaligned(c.sin, 4)) return DIT_ERR_MISALIGNED;
  for (int i = 0; i < 2; ++i) {
    if (!any || c.H[i] == 0) continue;
    const dit_heads* t[3] = {c.out[i], c.x[i], c.g[i]};
    for (int j = 0; j < 3; ++j) {
      if (j == 2 && !c.grad) continue;
      if (!t[j] || !t[j]->p) return DIT_ERR_NULL_PTR;
      if (misaligned(t[j]->p, es)) return DIT_ERR_MISALIGNED;
      if (!view(*t[j], c.B, c.L, c.H[i], c.D, es, &views[i][j])) return DIT_ERR_BAD_SHAPE;
      a->granules = a->granules && granules(views[i][j]);
    }
    if (c.norm && !c.w[i]) return DIT_ERR_NULL_PTR;
    if (c.norm && misaligned(c.w[i], es)) return DIT_ERR_MISALIGNED;
    a->granules = a->granules && !misaligned(c.w[i], 16);
    a->t[i].out = *c.out[i];
    a->t[i].x = *c.x[i];
    if (c.grad) a->t[i].g = *c.g[i];
    a->t[i].w = c.w[i];
    a->t[i].H = (int)c.H[i];
  }
  a->granules = a->granules && !misaligned(c.cos, 16) && !misaligned(c.sin, 16);
  for (int i = 0; i < 2; ++i) {
    if (a->t[i].H == 0) continue;
    const View& out = views[i][0];
    if (!apart(out)) return DIT_ERR_ALIAS;
    if (touch(out, span(c.cos, table)) || touch(out, span(c.sin, table))) return DIT_ERR_ALIAS;
    for (int k = 0; k < 2; ++k) {
      if (a->t[k].H == 0) continue;
      if (k > i && touch(out, views[k][0])) return DIT_ERR_ALIAS;
      if (c.norm && touch(out, span(c.w[k], c.D * es))) return DIT_ERR_ALIAS;
      for (int j = 1; j < (c.grad ? 3 : 2); ++j) {
        // in place: the input of the same tensor, or the gradient it arrives as
        if (k == i && j == (c.grad ? 2 : 1) && same(out, views[k][j])) continue;
        if (touch(out, views[k][j])) return DIT_ERR_ALIAS;
      }
    }
  }
  a->cos = c.cos;
  a->sin = c.sin;
  a->tokens = tokens;
  a->L = c.L;
  a->table_rows = c.table_rows;
  a->D = (int)c.D;
  a->R = (int)c.R;
  a->eps = c.eps;
  a->offset = c.offset;
  a->inv_d = c.D > 0 ? 1.0f / (float)c.D : 0.0f;
  a->interleaved = c.interleaved != 0;
  a->inverse = c.inverse != 0;
  *go = any;
  return DIT_OK;
}

dit_status rope_impl(const RopeCall& c, dit_stream_t stream) {
  dit::RopeArgs a;
  View views[2][3];
  bool go;
  const dit_status st = rope_checks(c, &a, views, &go);
  if (st != DIT_OK || !go) return st;
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  return launch_status(dit::launch_rope(dev, c.dtype, a, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

dit_status dit_rotary_table(float* cos, float* sin, const void* positions, const double* freqs,
                            int64_t tokens, const int64_t* sections, int64_t axes,
                            dit_position_type position_type, dit_stream_t stream) {
  if (position_type != DIT_POS_INT32 && position_type != DIT_POS_INT64 &&
      position_type != DIT_POS_FP32)
    return DIT_ERR_BAD_FORMAT;
  if (tokens < 0 || tokens > kMaxCount || axes < 1 || axes > DIT_MAX_AXES) return DIT_ERR_BAD_SHAPE;
  if (!sections) return DIT_ERR_NULL_PTR;
  dit::TableArgs a = {};
  int64_t R = 0;
  for (int64_t i = 0; i < axes; ++i) {
    if (sections[i] < 0 || sections[i] > kMaxPairs) return DIT_ERR_BAD_SHAPE;
    R += sections[i];
    a.end[i] = (int)R;
  }
  if (R > kMaxPairs) return DIT_ERR_BAD_SHAPE;
  if (tokens == 0 || R == 0) return DIT_OK;
  if (!cos || !sin || !positions || !freqs) return DIT_ERR_NULL_PTR;
  const int ps = position_type == DIT_POS_INT64 ? 8 : 4;
  if (misaligned(cos, 4) || misaligned(sin, 4) || misaligned(positions, ps) || misaligned(freqs, 8))
    return DIT_ERR_MISALIGNED;
  const Span outs[2] = {span(cos, tokens * R * 4), span(sin, tokens * R * 4)};
  const Span ins[2] = {span(positions, axes * tokens * ps), span(freqs, R * 8)};
  if (overlaps(outs[0], outs[1])) return DIT_ERR_ALIAS;
  for (const Span& o : outs)
    for (const Span& i : ins)
      if (overlaps(o, i)) return DIT_ERR_ALIAS;
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  a.cos = cos;
  a.sin = sin;
  a.positions = positions;
  a.freqs = freqs;
  a.tokens = tokens;
  a.R = (int)R;
  a.axes = (int)axes;
  return launch_status(dit::launch_table(dev, position_type, a, (cudaStream_t)stream));
}

dit_status dit_rope(const dit_heads* q_out, const dit_heads* k_out, const dit_heads* q,
                    const dit_heads* k, const float* cos, const float* sin, int64_t B, int64_t L,
                    int64_t Hq, int64_t Hk, int64_t D, int64_t R, int64_t table_rows,
                    int interleaved, int inverse, dit_dtype dtype, dit_stream_t stream) {
  return rope_impl(RopeCall{{q_out, k_out}, {}, {q, k}, {}, cos, sin, B, L, {Hq, Hk}, D, R, table_rows,
                            0.0f, 0.0f, interleaved, inverse, dtype, false, false},
                   stream);
}

dit_status dit_rmsnorm_rope(const dit_heads* q_out, const dit_heads* k_out, const dit_heads* q,
                            const dit_heads* k, const void* weight_q, const void* weight_k,
                            const float* cos, const float* sin, int64_t B, int64_t L, int64_t Hq,
                            int64_t Hk, int64_t D, int64_t R, int64_t table_rows, float eps,
                            float weight_offset, int interleaved, dit_dtype dtype,
                            dit_stream_t stream) {
  return rope_impl(RopeCall{{q_out, k_out}, {}, {q, k}, {weight_q, weight_k}, cos, sin, B, L, {Hq, Hk}, D,
                            R, table_rows, eps, weight_offset, interleaved, 0, dtype, true, false},
                   stream);
}

int64_t dit_rmsnorm_rope_backward_workspace_bytes(int64_t D) {
  if (D < 0 || D > kMaxHeadDim) return -1;
  return round_up(dit::kRopeGradMaxCtas * 2 * D * 4);
}

dit_status dit_rmsnorm_rope_backward(const dit_heads* q_grad, const dit_heads* k_grad,
                                     void* grad_weight_q, void* grad_weight_k,
                                     const dit_heads* q_out_grad, const dit_heads* k_out_grad,
                                     const dit_heads* q, const dit_heads* k, const void* weight_q,
                                     const void* weight_k, const float* cos, const float* sin,
                                     int64_t B, int64_t L, int64_t Hq, int64_t Hk, int64_t D,
                                     int64_t R, int64_t table_rows, float eps, float weight_offset,
                                     int interleaved, dit_dtype dtype, void* workspace,
                                     int64_t workspace_bytes, dit_stream_t stream) {
  const RopeCall c{{q_grad, k_grad}, {q_out_grad, k_out_grad}, {q, k}, {weight_q, weight_k}, cos, sin, B, L,
                   {Hq, Hk}, D, R, table_rows, eps, weight_offset, interleaved, 0, dtype, true, true};
  dit::RopeArgs a;
  View views[2][3];
  bool go;
  dit_status st = rope_checks(c, &a, views, &go);
  if (st != DIT_OK) return st;
  const int es = elem_size(dtype);
  void* gw[2] = {grad_weight_q, grad_weight_k};
  if (D == 0 || (!go && !gw[0] && !gw[1])) return DIT_OK;
  if (misaligned(gw[0], es) || misaligned(gw[1], es)) return DIT_ERR_MISALIGNED;
  const bool use_ws = go && (gw[0] || gw[1]);
  const int64_t need = dit_rmsnorm_rope_backward_workspace_bytes(D);
  if (use_ws) {
    st = workspace_status(workspace, workspace_bytes, need);
    if (st != DIT_OK) return st;
  }
  // what the call writes beside the heads: against everything else
  const Span own[3] = {span(gw[0], gw[0] ? D * es : 0), span(gw[1], gw[1] ? D * es : 0),
                       span(workspace, use_ws ? need : 0)};
  const int64_t table = go ? table_rows * R * 4 : 0;
  for (int i = 0; i < 3; ++i) {
    if (own[i].lo == own[i].hi) continue;
    for (int j = i + 1; j < 3; ++j)
      if (overlaps(own[i], own[j])) return DIT_ERR_ALIAS;
    if (overlaps(own[i], span(cos, table)) || overlaps(own[i], span(sin, table))) return DIT_ERR_ALIAS;
    for (int k = 0; k < 2; ++k) {
      if (a.t[k].H == 0) continue;
      if (overlaps(own[i], span(c.w[k], D * es))) return DIT_ERR_ALIAS;
      for (int j = 0; j < 3; ++j)
        if (touch(views[k][j], own[i])) return DIT_ERR_ALIAS;
    }
  }
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  const cudaStream_t s = (cudaStream_t)stream;
  for (int k = 0; k < 2; ++k) {  // no rows: the weight's gradient is zero
    if (!gw[k] || (go && a.t[k].H > 0)) continue;
    const cudaError_t e = cudaMemsetAsync(gw[k], 0, (size_t)(D * es), s);
    if (e != cudaSuccess) {
      (void)cudaGetLastError();
      return launch_status(e);
    }
    gw[k] = nullptr;
  }
  if (!go) return DIT_OK;
  a.partial = gw[0] || gw[1] ? (float*)workspace : nullptr;
  return launch_status(dit::launch_rope_grad(dev, dtype, a, gw[0], gw[1], s));
}

}  // extern "C"

namespace {

struct CacheViews {
  View k, v;      // [pages, heads, page_size, D]
  Span sk, sv;    // scales
  bool granules;  // every row on 16-byte boundaries
};

dit_status cache_checks(const dit_cache* c, CacheViews* o) {
  if (!c) return DIT_ERR_NULL_PTR;
  const bool fp8 = c->format == DIT_E4M3;
  if (!fp8 && (c->format < 0 || c->format > 2)) return DIT_ERR_BAD_FORMAT;
  const int es = fp8 ? 1 : elem_size((dit_dtype)c->format);
  int64_t slots, rows, n;
  // (page_size has a bound of its own: of no pages too, a launch divides by its low 32 bits)
  if (c->pages < 0 || c->heads < 0 || c->heads > kMaxHeads || c->page_size < 1 ||
      c->page_size > kMaxCount || c->D < 0 ||
      c->D > kMaxHeadDim || __builtin_mul_overflow(c->pages, c->page_size, &slots) ||
      slots > kMaxCount || __builtin_mul_overflow(c->heads, c->page_size, &rows) ||
      __builtin_mul_overflow(rows, c->D, &n) || n > kMaxStride || c->page_stride < n ||
      c->page_stride > kMaxStride || (fp8 && (c->scale_stride < rows || c->scale_stride > kMaxStride)))
    return DIT_ERR_BAD_SHAPE;
  const bool any = c->pages > 0 && n > 0;
  if (any && (!c->k || !c->v || (fp8 && (!c->k_scales || !c->v_scales)))) return DIT_ERR_NULL_PTR;
  if (misaligned(c->k, es) || misaligned(c->v, es) ||
      (fp8 && (misaligned(c->k_scales, 4) || misaligned(c->v_scales, 4))))
    return DIT_ERR_MISALIGNED;
  for (int i = 0; i < 2; ++i) {
    const dit_heads h{i ? c->v : c->k, c->page_stride, 0, 0};
    View* v = i ? &o->v : &o->k;
    if (!view(h, c->pages, 1, 1, any ? n : 0, es, v)) return DIT_ERR_BAD_SHAPE;
  }
  const int64_t sb = fp8 && any ? ((c->pages - 1) * c->scale_stride + rows) * 4 : 0;
  o->sk = span(c->k_scales, sb);
  o->sv = span(c->v_scales, sb);
  o->granules = ((((uint64_t)(uintptr_t)c->k | (uint64_t)(uintptr_t)c->v) |
                  (uint64_t)(c->page_stride * es) | (uint64_t)(c->D * es)) & 15u) == 0;
  return DIT_OK;
}
// the parts that a write changes, against each other and a view that it reads
bool cache_apart(const dit_cache* c, const CacheViews& o) {
  if (touch(o.k, o.v)) return false;
  if (c->format != DIT_E4M3) return true;
  View sk, sv;
  const int64_t rows = c->heads * c->page_size;
  if (!view(dit_heads{c->k_scales, c->scale_stride, 0, 0}, c->pages, 1, 1, rows, 4, &sk) ||
      !view(dit_heads{c->v_scales, c->scale_stride, 0, 0}, c->pages, 1, 1, rows, 4, &sv))
    return false;
  return !touch(sk, sv) && !touch(o.k, sk) && !touch(o.k, sv) && !touch(o.v, sk) && !touch(o.v, sv);
}
bool touches_cache(const View& x, const dit_cache* c, const CacheViews& o) {
  return touch(x, span_of(o.k)) || touch(x, span_of(o.v)) ||
         (c->format == DIT_E4M3 && (touch(x, o.sk) || touch(x, o.sv)));
}

dit_status cache_impl(bool write, const dit_cache* cache, const dit_heads* k, const dit_heads* v,
                      int64_t tokens, const void* slots, dit_id_type id_type, dit_dtype dtype,
                      dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  if (id_type != DIT_INT32 && id_type != DIT_INT64) return DIT_ERR_BAD_FORMAT;
  CacheViews o;
  const dit_status st = cache_checks(cache, &o);
  if (st != DIT_OK) return st;
  if (cache->format != DIT_E4M3 && cache->format != (int64_t)dtype) return DIT_ERR_BAD_DTYPE;
  if (tokens < 0 || tokens > kMaxCount) return DIT_ERR_BAD_SHAPE;
  if (tokens == 0 || cache->heads == 0 || cache->D == 0) return DIT_OK;
  if (write && cache->pages == 0) return DIT_OK;
  if (!k || !v || !k->p || !v->p || !slots) return DIT_ERR_NULL_PTR;
  const int es = elem_size(dtype), is = id_type == DIT_INT64 ? 8 : 4;
  if (misaligned(k->p, es) || misaligned(v->p, es) || misaligned(slots, is)) return DIT_ERR_MISALIGNED;
  View vk, vv;
  if (!view(*k, 1, tokens, cache->heads, cache->D, es, &vk) ||
      !view(*v, 1, tokens, cache->heads, cache->D, es, &vv))
    return DIT_ERR_BAD_SHAPE;
  const Span si = span(slots, tokens * is);
  if (touches_cache(vk, cache, o) || touches_cache(vv, cache, o)) return DIT_ERR_ALIAS;
  if (write) {
    if (!cache_apart(cache, o)) return DIT_ERR_ALIAS;
    if (touch(o.k, si) || touch(o.v, si) ||
        (cache->format == DIT_E4M3 && (overlaps(o.sk, si) || overlaps(o.sv, si))))
      return DIT_ERR_ALIAS;
  } else {
    if (!apart(vk) || !apart(vv) || touch(vk, vv) || touch(vk, si) || touch(vv, si)) return DIT_ERR_ALIAS;
  }
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  dit::CacheArgs a = {};
  a.c = *cache;
  a.k = *k;
  a.v = *v;
  a.tokens = tokens;
  a.slots = slots;
  a.ids64 = id_type == DIT_INT64;
  a.granules = granules(vk) && granules(vv) && o.granules;
  return launch_status(write ? dit::launch_cache_write(dev, dtype, a, (cudaStream_t)stream)
                             : dit::launch_cache_read(dev, dtype, a, (cudaStream_t)stream));
}

}  // namespace

extern "C" {

dit_status dit_cache_write(const dit_cache* cache, const dit_heads* k, const dit_heads* v,
                           int64_t tokens, const void* slots, dit_id_type id_type,
                           dit_dtype dtype, dit_stream_t stream) {
  return cache_impl(true, cache, k, v, tokens, slots, id_type, dtype, stream);
}

dit_status dit_cache_read(const dit_cache* cache, const dit_heads* k, const dit_heads* v,
                          int64_t tokens, const void* slots, dit_id_type id_type, dit_dtype dtype,
                          dit_stream_t stream) {
  return cache_impl(false, cache, k, v, tokens, slots, id_type, dtype, stream);
}

int64_t dit_paged_attention_workspace_bytes(int64_t Hq, int64_t heads, int64_t D) {
  if (heads < 1 || heads > kMaxHeads || Hq < heads || Hq > kMaxHeads || Hq % heads != 0 || D < 1 ||
      D > kMaxAttendDim)
    return -1;
  const int64_t rows = std::min<int64_t>(Hq / heads, dit::kAttendRows);
  const int64_t parts = std::max(dit::kAttendMaxCtas, dit::kAttendMmaCtas * (1 + dit::attend_warps(D)));
  return round_up(dit::kAttendMaxCtas * 2 * 8) + round_up(parts * 2 * rows * (D + 2) * 4);
}

dit_status dit_paged_attention(const dit_heads* out, float* lse, const dit_heads* q,
                               const dit_cache* cache, const int32_t* pages, int64_t pages_stride,
                               int64_t width, const void* lengths, int64_t B, int64_t Hq,
                               float scale, int64_t window, dit_id_type id_type, dit_dtype dtype,
                               void* workspace, int64_t workspace_bytes, dit_stream_t stream) {
  if (!valid_dtype(dtype)) return DIT_ERR_BAD_DTYPE;
  if (id_type != DIT_INT32 && id_type != DIT_INT64) return DIT_ERR_BAD_FORMAT;
  CacheViews o;
  dit_status st = cache_checks(cache, &o);
  if (st != DIT_OK) return st;
  if (cache->format != DIT_E4M3 && cache->format != (int64_t)dtype) return DIT_ERR_BAD_DTYPE;
  int64_t capacity, segments;
  // (the page table is only read: a stride of 0 repeats its row, as of the views)
  if (B < 0 || B > kMaxCount || width < 0 || pages_stride < (B > 1 && pages_stride != 0 ? width : 0) ||
      pages_stride > kMaxStride || __builtin_mul_overflow(width, cache->page_size, &capacity) ||
      capacity > kMaxTokens || window < 0 || __builtin_mul_overflow(B, Hq, &segments) ||
      segments > kMaxCount)
    return DIT_ERR_BAD_SHAPE;
  const int64_t need = dit_paged_attention_workspace_bytes(Hq, cache->heads, cache->D);
  if (need < 0) return DIT_ERR_BAD_SHAPE;
  if (!finite(scale)) return DIT_ERR_BAD_SCALAR;
  if (B == 0) return DIT_OK;
  if (!out || !q || !out->p || !q->p || !lengths || (capacity > 0 && !pages)) return DIT_ERR_NULL_PTR;
  const int es = elem_size(dtype), is = id_type == DIT_INT64 ? 8 : 4;
  if (misaligned(out->p, es) || misaligned(q->p, es) || misaligned(lse, 4) || misaligned(pages, 4) ||
      misaligned(lengths, is))
    return DIT_ERR_MISALIGNED;
  st = workspace_status(workspace, workspace_bytes, need);
  if (st != DIT_OK) return st;
  View vq, vo;
  if (!view(*q, 1, B, Hq, cache->D, es, &vq) || !view(*out, 1, B, Hq, cache->D, es, &vo))
    return DIT_ERR_BAD_SHAPE;
  const Span table = span(pages, capacity > 0 ? ((B - 1) * pages_stride + width) * 4 : 0);
  const Span len = span(lengths, B * is), ws = span(workspace, need);
  const Span sl = span(lse, lse ? B * Hq * 4 : 0);
  if (!apart(vo) || touch(vo, vq) || touch(vo, table) || touch(vo, len) || touch(vo, ws) ||
      touch(vo, sl) || touches_cache(vo, cache, o))
    return DIT_ERR_ALIAS;
  for (const Span& s : {sl, ws}) {
    if (s.lo == s.hi) continue;
    if (touch(vq, s) || overlaps(s, table) || overlaps(s, len) || touch(o.k, s) || touch(o.v, s) ||
        (cache->format == DIT_E4M3 && (overlaps(o.sk, s) || overlaps(o.sv, s))))
      return DIT_ERR_ALIAS;
  }
  if (overlaps(sl, ws)) return DIT_ERR_ALIAS;
  DeviceInfo dev;
  if (dit::current_device(&dev) != cudaSuccess) return DIT_ERR_NO_DEVICE;
  dit::AttendArgs a = {};
  a.c = *cache;
  a.q = *q;
  a.out = *out;
  a.lse = lse;
  a.pages = pages;
  a.pages_stride = pages_stride;
  a.capacity = cache->pages > 0 ? capacity : 0;
  a.lengths = lengths;
  a.ids64 = id_type == DIT_INT64;
  a.B = (int)B;
  a.Hq = (int)Hq;
  a.group = (int)(Hq / cache->heads);
  a.scale = scale;
  a.window = window;
  a.owner = (int64_t*)workspace;
  a.partial = (float*)((char*)workspace + round_up(dit::kAttendMaxCtas * 2 * 8));
  return launch_status(dit::launch_attend(dev, dtype, granules(vq) && granules(vo) && o.granules, a,
                                          (cudaStream_t)stream));
}

}  // extern "C"
