// kda_glr.hip -- gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel (gfx950).
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

struct Span { int64_t b, e; };

// tokens of sequence n among the packed ones, kept inside [0, tokens]
__device__ __forceinline__ Span glr_span(const GlrParams& p, int n) {
  if (!p.cu) return {(int64_t)n * p.T, (int64_t)(n + 1) * p.T};
  int64_t a = p.cu[n], b = p.cu[n + 1];
  a = a < 0 ? 0 : (a > p.T ? p.T : a);
  b = b < a ? a : (b > p.T ? p.T : b);
  return {a, b};
}

// One lane per channel, token by token.
template <int DT>
__global__ __launch_bounds__(64) void kda_glr_fwd_kernel(GlrParams p) {
  const int n = blockIdx.y, d = blockIdx.x * 64 + threadIdx.x;
  if (d >= p.D) return;
  const Span s = glr_span(p, n);
  float h = 0.0f;
  const int64_t in_row = p.in_slots ? p.in_slots[n] : n;
  if (!p.in_slots || (in_row >= 0 && in_row < p.n_slots)) load_state<1>(p.init, p.init_dtype, (size_t)in_row * p.D + d, &h);
  for (int64_t t = s.b; t < s.e; ++t) {
    float g, x;
    load_f32<DT, 1>(p.g, (size_t)t * p.D + d, &g);
    load_f32<DT, 1>(p.x, (size_t)t * p.D + d, &x);
    if (p.carry && t % GLR_TILE == 0) p.carry[(size_t)(t / GLR_TILE) * p.D + d] = h;
    h = fmaf(expf(g), h, x);
    store_f32<DT, 1>(p.y, (size_t)t * p.D + d, &h);
  }
  const int64_t out_row = p.out_slots ? p.out_slots[n] : n;
  if (!p.out_slots || (out_row >= 0 && out_row < p.n_slots)) store_state<1>(p.fin, p.fin_dtype, (size_t)out_row * p.D + d, &h);
}

// One lane per channel: per tile of GLR_TILE tokens the states before each token are
// computed again from the saved one into shared memory, then the tokens are taken backwards.
template <int DT>
__global__ __launch_bounds__(64) void kda_glr_bwd_kernel(GlrParams p) {
  __shared__ float hs[GLR_TILE][64];
  const int n = blockIdx.y, lane = threadIdx.x, d = blockIdx.x * 64 + lane;
  if (d >= p.D) return;
  const Span s = glr_span(p, n);
  float e = 0.0f, h0 = 0.0f;
  load_state<1>(p.dfin, p.dfin_dtype, (size_t)n * p.D + d, &e);
  load_state<1>(p.init, p.init_dtype, (size_t)n * p.D + d, &h0);
  for (int64_t hi = s.e; hi > s.b;) {
    const int64_t c = (hi - 1) / GLR_TILE, lo = c * GLR_TILE > s.b ? c * GLR_TILE : s.b;
    float h = lo == s.b ? h0 : p.carry[(size_t)c * p.D + d];
    for (int64_t t = lo; t < hi; ++t) {
      float g, x;
      load_f32<DT, 1>(p.g, (size_t)t * p.D + d, &g);
      load_f32<DT, 1>(p.x, (size_t)t * p.D + d, &x);
      hs[t - lo][lane] = h;
      h = fmaf(expf(g), h, x);
    }
    for (int64_t t = hi - 1; t >= lo; --t) {
      float g, dy;
      load_f32<DT, 1>(p.g, (size_t)t * p.D + d, &g);
      load_f32<DT, 1>(p.dy, (size_t)t * p.D + d, &dy);
      const float G = dy + e;
      e = expf(g) * G;
      const float dg = e * hs[t - lo][lane];
      store_f32<DT, 1>(p.dx, (size_t)t * p.D + d, &G);
      store_f32<DT, 1>(p.dg, (size_t)t * p.D + d, &dg);
    }
    hi = lo;
  }
  store_state<1>(p.fin, p.fin_dtype, (size_t)n * p.D + d, &e);
}

template <typename F>
hipError_t by_dtype(int dt, F f) {
  if (dt == BF16) f(std::integral_constant<int, BF16>{});
  else if (dt == FP32) f(std::integral_constant<int, FP32>{});
  else f(std::integral_constant<int, FP16>{});
  return hipGetLastError();
}

}  // namespace

hipError_t launch_glr_fwd(const GlrParams& p, hipStream_t stream) {
  if (p.nseq <= 0) return hipSuccess;
  return by_dtype(p.dtype, [&](auto dt) {
    hipLaunchKernelGGL(kda_glr_fwd_kernel<dt.value>, dim3((p.D + 63) / 64, p.nseq), dim3(64), 0, stream, p);
  });
}

hipError_t launch_glr_bwd(const GlrParams& p, hipStream_t stream) {
  if (p.nseq <= 0) return hipSuccess;
  return by_dtype(p.dtype, [&](auto dt) {
    hipLaunchKernelGGL(kda_glr_bwd_kernel<dt.value>, dim3((p.D + 63) / 64, p.nseq), dim3(64), 0, stream, p);
  });
}

}  // namespace kda
