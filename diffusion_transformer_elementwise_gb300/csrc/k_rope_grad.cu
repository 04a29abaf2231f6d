// k_rope_grad.cu -- the gradient of a head's norm and rotation (sm_103a).
//
//   u = the gradient of the output turned back,  n = x r,  t = u (offset + w)
//   grad_x = r (t - n mean(t n)),   grad_w = sum over tokens and heads of u n
#include "dit_attend.h"
#include "dit_heads.cuh"

namespace dit {
namespace {

constexpr int kRowThreads = 256;
constexpr int kRowWarps = kRowThreads / 32;

// Any view: a warp has a head, an element per access.  Each warp adds up its
// weights' gradients in shared memory (its own row of it), the CTA its warps'.
template <class T>
__global__ void __launch_bounds__(kRowThreads) rope_grad_kernel(const __grid_constant__ RopeArgs a) {
  extern __shared__ float sums[];  // [warps][2][D]
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  float* mine = sums + (size_t)warp * 2 * a.D;
  if (a.partial) {
    for (int c = lane; c < 2 * a.D; c += 32) mine[c] = 0.0f;
    __syncwarp();
  }
  const int heads = a.t[0].H + a.t[1].H;
  const int64_t rows = a.tokens * heads;
  const int64_t stride = (int64_t)gridDim.x * kRowWarps;
  for (int64_t i = (int64_t)blockIdx.x * kRowWarps + warp; i < rows; i += stride) {
    const HeadRow row(a, i, heads);
    const RopeTensor& t = a.t[row.tensor];
    const T* x = (const T*)t.x.p + row.at(t.x);
    const T* g = (const T*)t.g.p + row.at(t.g);
    T* out = (T*)t.out.p + row.at(t.out);
    const T* w = (const T*)t.w;
    const float* cs = a.cos + row.table * a.R;
    const float* sn = a.sin + row.table * a.R;
    // columns come in pairs (c, d); those that are not turned come alone
    auto columns = [&](auto&& body) {
      for (int j = lane; j < a.R; j += 32) {
        const int c = a.interleaved ? 2 * j : j, d = a.interleaved ? c + 1 : c + a.R;
        const float2 u = turned(to_float(g[c]), to_float(g[d]), cs[j], -sn[j]);
        body(c, u.x, d, u.y);
      }
      for (int c = 2 * a.R + lane; c < a.D; c += 32) body(c, to_float(g[c]), -1, 0.0f);
    };
    auto weighted = [&](int c, float u) { return __fmul_rn(u, __fadd_rn(a.offset, to_float(w[c]))); };
    float sum = 0.0f, dot = 0.0f;
    columns([&](int c, float u, int d, float v) {
      const float p = to_float(x[c]);
      sum = __fmaf_rn(p, p, sum);
      dot = __fmaf_rn(weighted(c, u), p, dot);
      if (d < 0) return;
      const float q = to_float(x[d]);
      sum = __fmaf_rn(q, q, sum);
      dot = __fmaf_rn(weighted(d, v), q, dot);
    });
    const float r = inverse_rms(lanes_sum<32>(sum), a.D, a.eps);
    // mean(t n), n = x r
    const float mean = __fdiv_rn(__fmul_rn(lanes_sum<32>(dot), r), (float)a.D);
    columns([&](int c, float u, int d, float v) {
      auto one = [&](int k, float grad) {
        const float n = __fmul_rn(to_float(x[k]), r);
        const float y = __fmul_rn(r, __fadd_rn(weighted(k, grad), -__fmul_rn(n, mean)));
        if (a.partial) mine[row.tensor * a.D + k] = __fmaf_rn(grad, n, mine[row.tensor * a.D + k]);
        return from_float<T>(y);
      };
      const T first = one(c, u);
      if (d >= 0) {
        const T second = one(d, v);
        out[d] = second;
      }
      out[c] = first;
    });
  }
  if (!a.partial) return;
  __syncthreads();
  for (int c = threadIdx.x; c < 2 * a.D; c += kRowThreads) {
    float v = 0.0f;
    for (int k = 0; k < kRowWarps; ++k) v = __fadd_rn(v, sums[(size_t)k * 2 * a.D + c]);
    a.partial[(int64_t)blockIdx.x * 2 * a.D + c] = v;
  }
}

// gw[k][c] = the sum over the CTAs' partial sums: 32 columns a CTA, its 32
// warps the rows w, w + 32, ..., then their sums in order.
struct JoinArgs {
  const float* partial;
  int ctas, D;
  void* gw[2];
};
template <class T>
__global__ void __launch_bounds__(1024) join_kernel(JoinArgs a) {
  __shared__ float part[32][33];
  const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
  const int c = blockIdx.x * 32 + lane;
  float v = 0.0f;
  after_previous();
  if (c < 2 * a.D)
    for (int i = warp; i < a.ctas; i += 32) v = __fadd_rn(v, a.partial[(int64_t)i * 2 * a.D + c]);
  part[warp][lane] = v;
  __syncthreads();
  v = lanes_sum<32>(part[lane][warp]);
  const int k = blockIdx.x * 32 + warp;
  if (lane == 0 && k < 2 * a.D) {
    T* gw = (T*)a.gw[k >= a.D];
    if (gw) gw[k >= a.D ? k - a.D : k] = from_float<T>(v);
  }
}

template <class T>
cudaError_t launch(const DeviceInfo& dev, const RopeArgs& a, void* gwq, void* gwk, cudaStream_t s) {
  const int64_t rows = a.tokens * (a.t[0].H + a.t[1].H);
  const auto kern = rope_grad_kernel<T>;
  const size_t smem = a.partial ? (size_t)kRowWarps * 2 * a.D * 4 : 0;
  static std::atomic<int> opted[kOptinDevices];
  cudaError_t e = allow_shared((const void*)kern, dev, opted);
  if (e != cudaSuccess) return e;
  const int64_t most = std::min(kRopeGradMaxCtas, (int64_t)dev.sm_count * resident_ctas(dev, (const void*)kern, kRowThreads, smem));
  const unsigned grid = (unsigned)std::min(most, (rows + kRowWarps - 1) / kRowWarps);
  kern<<<grid, kRowThreads, smem, s>>>(a);
  e = cudaGetLastError();
  if (e != cudaSuccess || !a.partial) return e;
  return launch_after(join_kernel<T>, (unsigned)((2 * a.D + 31) / 32), 1024, 0, s,
                      JoinArgs{a.partial, (int)grid, a.D, {gwq, gwk}});
}

}  // namespace

cudaError_t launch_rope_grad(const DeviceInfo& dev, int dtype, const RopeArgs& a, void* gwq,
                             void* gwk, cudaStream_t s) {
  return dtype == 0   ? launch<__nv_bfloat16>(dev, a, gwq, gwk, s)
         : dtype == 1 ? launch<__half>(dev, a, gwq, gwk, s)
                      : launch<float>(dev, a, gwq, gwk, s);
}

}  // namespace dit
