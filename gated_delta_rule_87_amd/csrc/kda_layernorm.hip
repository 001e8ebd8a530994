// kda_layernorm.hip -- layer norm of rows, forward and backward (gfx950).
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

__device__ __forceinline__ float block_sum(float v, float* buf) {   // 256 threads
#pragma unroll
  for (int o = 32; o >= 1; o >>= 1) v += __shfl_xor(v, o, 64);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return buf[0] + buf[1] + buf[2] + buf[3];
}

// One workgroup per row, the row read three times.
template <int DT>
__global__ __launch_bounds__(256) void kda_layernorm_fwd_kernel(NormParams p) {
  __shared__ float buf[4];
  const int tid = threadIdx.x;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = (size_t)m * p.D;
    float s = 0.0f, q = 0.0f, v;
    for (int d = tid; d < p.D; d += 256) {
      load_f32<DT, 1>(p.x, row + d, &v);
      s += v;
    }
    const float mean = block_sum(s, buf) / p.D;
    for (int d = tid; d < p.D; d += 256) {
      load_f32<DT, 1>(p.x, row + d, &v);
      q += (v - mean) * (v - mean);
    }
    const float rstd = 1.0f / sqrtf(block_sum(q, buf) / p.D + p.eps);
    if (tid == 0) {
      if (p.mean) p.mean[m] = mean;
      if (p.rstd) p.rstd[m] = rstd;
    }
    for (int d = tid; d < p.D; d += 256) {
      load_f32<DT, 1>(p.x, row + d, &v);
      const float y = fmaf((v - mean) * rstd, p.weight ? p.weight[d] : 1.0f, p.bias ? p.bias[d] : 0.0f);
      store_f32<DT, 1>(p.out, row + d, &y);
    }
  }
}

// One workgroup per run of rows; each thread keeps the sums of its columns in its part of
// the workspace.
template <int DT>
__global__ __launch_bounds__(256) void kda_layernorm_bwd_kernel(NormParams p, int parts) {
  __shared__ float buf[4];
  const int tid = threadIdx.x;
  float* pw = p.partial + (size_t)blockIdx.x * p.D;
  float* pb = p.partial + ((size_t)parts + blockIdx.x) * p.D;
  if (p.partial)
    for (int d = tid; d < p.D; d += 256) pw[d] = pb[d] = 0.0f;
  for (int64_t m = blockIdx.x; m < p.M; m += parts) {
    const size_t row = (size_t)m * p.D;
    const float mean = p.mean[m], rstd = p.rstd[m];
    float s1 = 0.0f, s2 = 0.0f, x, dy;
    for (int d = tid; d < p.D; d += 256) {
      load_f32<DT, 1>(p.x, row + d, &x);
      load_f32<DT, 1>(p.dy, row + d, &dy);
      const float a = dy * (p.weight ? p.weight[d] : 1.0f);
      s1 += a;
      s2 += a * (x - mean) * rstd;
    }
    const float c1 = block_sum(s1, buf) / p.D;
    const float c2 = block_sum(s2, buf) / p.D;
    for (int d = tid; d < p.D; d += 256) {
      load_f32<DT, 1>(p.x, row + d, &x);
      load_f32<DT, 1>(p.dy, row + d, &dy);
      const float xh = (x - mean) * rstd, a = dy * (p.weight ? p.weight[d] : 1.0f);
      if (p.partial) {
        pw[d] += dy * xh;
        pb[d] += dy;
      }
      const float dx = rstd * (a - c1 - xh * c2);
      if (p.out) store_f32<DT, 1>(p.out, row + d, &dx);
    }
  }
}

__global__ __launch_bounds__(256) void kda_layernorm_sum_kernel(NormParams p, int parts) {
  const int d = blockIdx.x * 256 + threadIdx.x;
  if (d >= p.D) return;
  float w = 0.0f, b = 0.0f;
  for (int i = 0; i < parts; ++i) {
    w += p.partial[(size_t)i * p.D + d];
    b += p.partial[((size_t)parts + i) * p.D + d];
  }
  if (p.dw) p.dw[d] = w;
  if (p.db) p.db[d] = b;
}

template <typename F>
hipError_t by_dtype(int dt, F f) {
  if (dt == BF16) f(std::integral_constant<int, BF16>{});
  else if (dt == FP32) f(std::integral_constant<int, FP32>{});
  else f(std::integral_constant<int, FP16>{});
  return hipGetLastError();
}

}  // namespace

size_t layernorm_parts(int64_t M, int64_t D) {
  (void)D;
  return (size_t)(M < 512 ? M : 512);
}

hipError_t launch_layernorm_fwd(const NormParams& p, hipStream_t stream) {
  if (p.M == 0) return hipSuccess;
  const unsigned blocks = (unsigned)(p.M < 65536 ? p.M : 65536);
  return by_dtype(p.dtype, [&](auto dt) {
    hipLaunchKernelGGL(kda_layernorm_fwd_kernel<dt.value>, dim3(blocks), dim3(256), 0, stream, p);
  });
}

hipError_t launch_layernorm_bwd(const NormParams& p, hipStream_t stream) {
  const int parts = (int)layernorm_parts(p.M, p.D);
  hipError_t e = hipSuccess;
  if (p.M > 0)
    e = by_dtype(p.dtype, [&](auto dt) {
      hipLaunchKernelGGL(kda_layernorm_bwd_kernel<dt.value>, dim3(parts), dim3(256), 0, stream, p, parts);
    });
  if (e == hipSuccess && (p.dw || p.db)) {
    hipLaunchKernelGGL(kda_layernorm_sum_kernel, dim3((p.D + 255) / 256), dim3(256), 0, stream, p, parts);
    e = hipGetLastError();
  }
  return e;
}

}  // namespace kda
