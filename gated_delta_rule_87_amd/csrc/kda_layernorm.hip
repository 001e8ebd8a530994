// kda_layernorm.hip -- layer norm of rows, forward and backward (gfx950).
//
// Both directions are bound by memory: the forward pass reads x and writes y (524288 rows of
// 128 bf16: 48 us, 5.7 TB/s), the backward pass reads dy and x and writes dx (there 78 us, 5.2
// TB/s; 8192 rows of 8192: 87 us, 4.8 TB/s with its sums; both and 5 us for adding them). A row
// is loaded once into the registers of LANES lanes (8 of a wave for the shortest rows, a
// workgroup of 1024 for the widest), 16 bytes a lane and vector; statistics are two sums over
// those registers: the mean, then the squares of the differences from it. That mean is off by
// the sum's roundings, some u = 2^-24 of |x|, which is nothing beside a deviation of |mean| and
// more, and too much in a row far from zero (one of 12345.678 throughout came out as -0.3 and
// not 0). Such rows take a third sum, of the differences, which are exact there: its mean is
// what the first one is off by. Workgroups take rows in strides and keep the weight, and in the backward pass
// the sums of dy xhat and dy of their columns, in registers from row to row; each writes its
// sums once to the workspace, and a second kernel adds those in a fixed order.
//
// Rows need not be whole numbers of vectors nor aligned to them: vectors are loaded at any
// address (the hardware splits what crosses a line), a row's last elements in smaller pieces.
// Rows of more than 16384 elements do not fit the registers of a workgroup and are read three
// times.
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}
__device__ __forceinline__ float swap16_add(float x) {
  const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
__device__ __forceinline__ float swap32_add(float x) {
  const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
  return __uint_as_float(a[0]) + __uint_as_float(a[1]);
}
// Sum over groups of 8, 16 or 64 lanes, the same bits in every lane.
template <int LANES>
__device__ __forceinline__ float lanes_sum(float x) {
  x = dpp_add<0xB1>(x);    // lane ^ 1
  x = dpp_add<0x1B>(x);    // lane ^ 3
  x = dpp_add<0x141>(x);   // lane ^ 7
  if constexpr (LANES >= 16) x = dpp_add<0x140>(x);   // lane ^ 15
  if constexpr (LANES >= 64) x = swap32_add(swap16_add(x));
  return x;
}

// Sums of K values over LANES lanes. Rows of several waves go through buf, one barrier a call:
// consecutive calls take different parts of it.
template <int LANES, int K>
__device__ __forceinline__ void row_sums(float* v, float (*buf)[K], int part) {
#pragma unroll
  for (int k = 0; k < K; ++k) v[k] = lanes_sum<(LANES > 64 ? 64 : LANES)>(v[k]);
  if constexpr (LANES > 64) {
    constexpr int W = LANES / 64;
    float (*b)[K] = buf + part * W;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int k = 0; k < K; ++k) b[threadIdx.x >> 6][k] = v[k];
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {   // a wave's sum in every lane, added up over 4, 8 or 16 lanes
      float s = b[threadIdx.x % W][k];
      s = dpp_add<0x1B>(dpp_add<0xB1>(s));
      if constexpr (W >= 8) s = dpp_add<0x141>(s);
      if constexpr (W == 16) s = dpp_add<0x140>(s);
      v[k] = s;
    }
  }
}

// c fp32 parameters of columns i on (i a multiple of VEC), or a constant
template <int VEC>
__device__ __forceinline__ void load_param(const float* p, int i, int c, float none, float* f) {
  if (p && c >= VEC) {
    load_f32<FP32, VEC>(p, i, f);
    return;
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) f[e] = e < c ? (p ? p[i + e] : none) : 0.0f;
}

template <int DT>
constexpr int vec_of() { return 16 / elem_size(DT); }
constexpr int wg_of(int lanes) { return lanes > 256 ? lanes : 256; }

// ---- forward ----------------------------------------------------------------------

// A row whose mean is more than its deviation (squares: the mean of the squared differences
// from it): only there can the roundings of the mean be more than those of what follows.
__device__ __forceinline__ bool is_far(float mean, float squares) { return mean * mean > squares; }
// The variance, from that and what the mean was off by, which is roundings only: nothing
// cancels, but a row of one value may come out below zero.
__device__ __forceinline__ float about_mean(float squares, float off) {
  const float var = fmaf(-off, off, squares);
  return var < 0.0f ? 0.0f : var;
}

// A lane holds NV vectors of a row, U rows at a time.
template <int DT, bool EXACT, int LANES, int NV, int U>
__global__ __launch_bounds__(wg_of(LANES)) void kda_layernorm_fwd_kernel(NormParams p) {
  constexpr int VEC = vec_of<DT>(), G = wg_of(LANES) / LANES;
  __shared__ float buf[LANES > 64 ? 3 * LANES / 64 : 1][U];
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const float inv = 1.0f / p.D;
  float w[NV][VEC], b[NV][VEC];
  int c[NV];   // elements of this lane's vectors
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * LANES + lane) * VEC;
    c[i] = p.D - col < 0 ? 0 : p.D - col > VEC ? VEC : p.D - col;
    load_param<VEC>(p.weight, col, c[i], 1.0f, w[i]);
    load_param<VEC>(p.bias, col, c[i], 0.0f, b[i]);
  }
  for (int64_t m0 = (int64_t)blockIdx.x * G * U; m0 < p.M; m0 += (int64_t)gridDim.x * G * U) {
    Pack<DT, VEC> x[U][NV];
    float s[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[u][i].clear();
        if (m < p.M && c[i] > 0) load_part<EXACT>(x[u][i], p.x, (size_t)m * p.D + (i * LANES + lane) * VEC, c[i]);
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[VEC];
        x[u][i].unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) s[u] += f[e];
      }
    }
    row_sums<LANES, U>(s, buf, 0);
#pragma unroll
    for (int u = 0; u < U; ++u) {
      s[u] /= p.D;
      q[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[VEC];
        x[u][i].unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float d = (EXACT ? c[i] > 0 : e < c[i]) ? f[e] - s[u] : 0.0f;
          q[u] = fmaf(d, d, q[u]);
        }
      }
    }
    row_sums<LANES, U>(q, buf, 1);
    bool far = false;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u] *= inv;
      far = far || is_far(s[u], q[u]);
    }
    auto outputs = [&](auto corrected, const float* off) {
      constexpr bool CORRECTED = decltype(corrected)::value;
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * G + grp;
        const float mean = s[u], rstd = 1.0f / sqrtf(q[u] + p.eps);
        if (m >= p.M) continue;
        if (lane == 0) {
          if (p.mean) p.mean[m] = CORRECTED ? mean + off[u] : mean;
          if (p.rstd) p.rstd[m] = rstd;
        }
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[VEC];
          if (CORRECTED) x[u][i].opaque();
          x[u][i].unpack(f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) {
            const float d = CORRECTED ? (f[e] - mean) - off[u] : f[e] - mean;
            f[e] = fmaf(d * rstd, w[i][e], b[i][e]);
          }
          Pack<DT, VEC> y;
          y.pack(f);
          if (c[i] > 0) store_part<EXACT>(y, p.out, (size_t)m * p.D + (i * LANES + lane) * VEC, c[i]);
        }
      }
    };
    // Outputs of their own where no row is far: the differences from the mean are kept from the
    // sum of their squares (3001 bf16: 48.1 us, 50.9 with one form for both; fp32 rows of whole
    // vectors take a subtraction more and 20 registers fewer: 8192 wide 41.3 us, 43.4 with two).
    constexpr bool TWO = DT != FP32 || !EXACT;
    const bool any_far = __any(far);   // (of a row over several waves: the same in all of them)
    if (TWO && !any_far) {
      outputs(std::false_type{}, nullptr);
      continue;
    }
    float off[U] = {};
    if (any_far) {
#pragma unroll
      for (int u = 0; u < U; ++u) {
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          float f[VEC];
          x[u][i].opaque();   // its elements are not kept for here (up to 30 registers)
          x[u][i].unpack(f);
#pragma unroll
          for (int e = 0; e < VEC; ++e) off[u] += (EXACT ? c[i] > 0 : e < c[i]) ? f[e] - s[u] : 0.0f;
        }
      }
      row_sums<LANES, U>(off, buf, 2);
#pragma unroll
      for (int u = 0; u < U; ++u) {   // no row's result depends on the rows beside it
        off[u] = is_far(s[u], q[u]) ? off[u] / p.D : 0.0f;
        q[u] = about_mean(q[u], off[u]);
      }
    }
    outputs(std::true_type{}, off);
  }
}

// Rows of more than 16384 elements: a workgroup reads a row three times, four where it is far
// from zero.
template <int DT>
__global__ __launch_bounds__(1024) void kda_layernorm_fwd_long_kernel(NormParams p) {
  constexpr int VEC = vec_of<DT>();
  __shared__ float buf[3 * 16][1];
  const float inv = 1.0f / p.D;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = (size_t)m * p.D;
    float s = 0.0f, q = 0.0f, off = 0.0f;
    auto each = [&](auto f) {
      for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.D; col += 1024 * VEC) {
        const int c = p.D - col < VEC ? (int)(p.D - col) : VEC;
        Pack<DT, VEC> x;
        load_part<false>(x, p.x, row + col, c);
        float v[VEC];
        x.unpack(v);
        f((int)col, c, v);
      }
    };
    each([&](int, int, const float* v) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) s += v[e];
    });
    row_sums<1024, 1>(&s, buf, 0);
    const float mean = s / p.D;
    each([&](int, int c, const float* v) {
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < c) q = fmaf(v[e] - mean, v[e] - mean, q);
    });
    row_sums<1024, 1>(&q, buf, 1);
    q *= inv;
    if (is_far(mean, q)) {
      each([&](int, int c, const float* v) {
#pragma unroll
        for (int e = 0; e < VEC; ++e)
          if (e < c) off += v[e] - mean;
      });
      row_sums<1024, 1>(&off, buf, 2);
      off /= p.D;
      q = about_mean(q, off);
    }
    const float rstd = 1.0f / sqrtf(q + p.eps);
    if (threadIdx.x == 0) {
      if (p.mean) p.mean[m] = mean + off;
      if (p.rstd) p.rstd[m] = rstd;
    }
    each([&](int col, int c, const float* v) {
      float w[VEC], b[VEC];
      load_param<VEC>(p.weight, col, c, 1.0f, w);
      load_param<VEC>(p.bias, col, c, 0.0f, b);
#pragma unroll
      for (int e = 0; e < VEC; ++e) w[e] = fmaf(((v[e] - mean) - off) * rstd, w[e], b[e]);
      Pack<DT, VEC> y;
      y.pack(w);
      store_part<false>(y, p.out, row + col, c);
    });
  }
}

// ---- backward ---------------------------------------------------------------------

// Sum over the row groups of a workgroup: the groups of a wave by lane swaps, the waves'
// through shared memory; lanes 0 .. LANES - 1 of the workgroup end with the total.
template <int LANES>
__device__ __forceinline__ float groups_sum(float v, float* buf) {
  if constexpr (LANES == 8) v = v + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(v), 0x128, 0xf, 0xf, false));   // row_ror 8
  if constexpr (LANES <= 16) v = swap32_add(swap16_add(v));
  if constexpr (LANES <= 64) {
    const int lane = threadIdx.x & 63, wave = threadIdx.x >> 6;
    __syncthreads();
    if (lane < LANES) buf[wave * LANES + lane] = v;
    __syncthreads();
    v = 0.0f;
    if (threadIdx.x < LANES) v = (buf[lane] + buf[LANES + lane]) + (buf[2 * LANES + lane] + buf[3 * LANES + lane]);
  }
  return v;
}

template <int DT, bool EXACT, int LANES, int NV, int U>
__global__ __launch_bounds__(wg_of(LANES)) void kda_layernorm_bwd_kernel(NormParams p, int parts) {
  constexpr int VEC = vec_of<DT>(), G = wg_of(LANES) / LANES;
  __shared__ float buf[LANES > 64 ? 2 * LANES / 64 : 1][2 * U];
  __shared__ float gbuf[LANES <= 64 ? 4 * LANES : 1];
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const float inv = 1.0f / p.D;
  float w[NV][VEC], aw[NV][VEC], ab[NV][VEC];
  int c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * LANES + lane) * VEC;
    c[i] = p.D - col < 0 ? 0 : p.D - col > VEC ? VEC : p.D - col;
    load_param<VEC>(p.weight, col, c[i], 1.0f, w[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) aw[i][e] = ab[i][e] = 0.0f;
  }
  int half = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * G * U; m0 < p.M; m0 += (int64_t)gridDim.x * G * U) {
    Pack<DT, VEC> x[U][NV], dy[U][NV];
    float mean[U], rstd[U], s[2 * U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      mean[u] = rstd[u] = 0.0f;
      if (m < p.M) {
        mean[u] = p.mean[m];
        rstd[u] = p.rstd[m];
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        x[u][i].clear();
        dy[u][i].clear();
        if (m < p.M && c[i] > 0) {
          const size_t at = (size_t)m * p.D + (i * LANES + lane) * VEC;
          load_part<EXACT>(x[u][i], p.x, at, c[i]);
          load_part<EXACT>(dy[u][i], p.dy, at, c[i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      float s1 = 0.0f, s2 = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[VEC], df[VEC];
        x[u][i].unpack(xf);
        dy[u][i].unpack(df);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {   // dy and the weight are zero behind a row's end
          const float xh = (xf[e] - mean[u]) * rstd[u], a = df[e] * w[i][e];
          s1 += a;
          s2 = fmaf(a, xh, s2);
          aw[i][e] = fmaf(df[e], xh, aw[i][e]);
          ab[i][e] += df[e];
        }
      }
      s[2 * u] = s1;
      s[2 * u + 1] = s2;
    }
    if (!p.out) continue;
    row_sums<LANES, 2 * U>(s, buf, half);
    half ^= 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      if (m >= p.M) continue;
      const float c1 = s[2 * u] * inv, c2 = s[2 * u + 1] * inv;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float xf[VEC], df[VEC];
        x[u][i].unpack(xf);
        dy[u][i].unpack(df);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = (xf[e] - mean[u]) * rstd[u];
          df[e] = rstd[u] * (fmaf(df[e], w[i][e], -c1) - xh * c2);
        }
        Pack<DT, VEC> dx;
        dx.pack(df);
        if (c[i] > 0) store_part<EXACT>(dx, p.out, (size_t)m * p.D + (i * LANES + lane) * VEC, c[i]);
      }
    }
  }
  if (!p.partial) return;
  float* pw = p.partial + (size_t)blockIdx.x * p.D;
  float* pb = p.partial + ((size_t)parts + blockIdx.x) * p.D;
#pragma unroll
  for (int i = 0; i < NV; ++i) {
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      const float sw = groups_sum<LANES>(aw[i][e], gbuf), sb = groups_sum<LANES>(ab[i][e], gbuf);
      if (grp == 0 && e < c[i]) {
        const int col = (i * LANES + lane) * VEC + e;
        pw[col] = sw;
        pb[col] = sb;
      }
    }
  }
}

// Rows of more than 16384 elements: dx from a row read twice by a workgroup ...
template <int DT>
__global__ __launch_bounds__(1024) void kda_layernorm_bwd_long_kernel(NormParams p) {
  constexpr int VEC = vec_of<DT>();
  __shared__ float buf[2 * 16][2];
  const float inv = 1.0f / p.D;
  int half = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = (size_t)m * p.D;
    const float mean = p.mean[m], rstd = p.rstd[m];
    float s[2] = {0.0f, 0.0f};
    auto each = [&](auto f) {
      for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.D; col += 1024 * VEC) {
        const int c = p.D - col < VEC ? (int)(p.D - col) : VEC;
        Pack<DT, VEC> x, dy;
        load_part<false>(x, p.x, row + col, c);
        load_part<false>(dy, p.dy, row + col, c);
        float xf[VEC], df[VEC], w[VEC];
        x.unpack(xf);
        dy.unpack(df);
        load_param<VEC>(p.weight, (int)col, c, 1.0f, w);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          xf[e] = (xf[e] - mean) * rstd;
          df[e] *= w[e];
        }
        f(col, c, xf, df);
      }
    };
    each([&](int64_t, int, const float* xh, const float* a) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) {
        s[0] += a[e];
        s[1] = fmaf(a[e], xh[e], s[1]);
      }
    });
    row_sums<1024, 2>(s, buf, half);
    half ^= 1;
    const float c1 = s[0] * inv, c2 = s[1] * inv;
    each([&](int64_t col, int c, const float* xh, float* a) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) a[e] = rstd * (a[e] - c1 - xh[e] * c2);
      Pack<DT, VEC> dx;
      dx.pack(a);
      store_part<false>(dx, p.out, row + col, c);
    });
  }
}

// ... and before it (dx may be written over dy or x) the columns' sums: a lane per VEC columns,
// part i the rows i, i + parts, ...
template <int DT>
__global__ __launch_bounds__(64) void kda_layernorm_cols_kernel(NormParams p, int parts) {
  constexpr int VEC = vec_of<DT>();
  const int part = blockIdx.x % parts;
  const int64_t col = ((int64_t)(blockIdx.x / parts) * 64 + threadIdx.x) * VEC;
  if (col >= p.D) return;
  const int c = p.D - col < VEC ? (int)(p.D - col) : VEC;
  float aw[VEC] = {}, ab[VEC] = {};
  for (int64_t m = part; m < p.M; m += parts) {
    const float mean = p.mean[m], rstd = p.rstd[m];
    Pack<DT, VEC> x, dy;
    load_part<false>(x, p.x, (size_t)m * p.D + col, c);
    load_part<false>(dy, p.dy, (size_t)m * p.D + col, c);
    float xf[VEC], df[VEC];
    x.unpack(xf);
    dy.unpack(df);
#pragma unroll
    for (int e = 0; e < VEC; ++e) {
      aw[e] = fmaf(df[e], (xf[e] - mean) * rstd, aw[e]);
      ab[e] += df[e];
    }
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e) {
    if (e < c) {
      p.partial[(size_t)part * p.D + col + e] = aw[e];
      p.partial[((size_t)parts + part) * p.D + col + e] = ab[e];
    }
  }
}

// The parts' sums: COLS columns of dw (blockIdx.y 0) or db by 1024 / COLS runs of parts a
// workgroup: many runs where there are few columns, whole lines where there are many (8192
// columns, 256 parts: 8 us with 16 columns).
template <int COLS>
__global__ __launch_bounds__(1024) void kda_layernorm_sum_kernel(NormParams p, int parts) {
  constexpr int RUNS = 1024 / COLS;
  __shared__ float buf[RUNS][COLS + 1];
  float* out = blockIdx.y ? p.db : p.dw;
  if (!out) return;
  const float* in = p.partial + (blockIdx.y ? (size_t)parts * p.D : 0);
  const int j = threadIdx.x % COLS, run = threadIdx.x / COLS, col = blockIdx.x * COLS + j;
  float s = 0.0f;
  if (col < p.D) {
#pragma unroll 8
    for (int i = run; i < parts; i += RUNS) s += in[(size_t)i * p.D + col];
  }
  buf[run][j] = s;
  __syncthreads();
#pragma unroll
  for (int o = RUNS / 2; o >= 1; o >>= 1) {
    if (run < o) buf[run][j] += buf[run + o][j];
    __syncthreads();
  }
  if (run == 0 && col < p.D) out[col] = buf[0][j];
}

using std::integral_constant;
template <bool E, int L, int V, int U>
struct Shape {
  static constexpr bool exact = E;
  static constexpr int lanes = L, nv = V, rows = U;
};

// f(shape) for the fewest lanes, and vectors of a lane, that hold a row; false: none does. Few
// vectors leave registers for more rows at once (8192 bf16 backward: 108 us with 256 lanes of
// 4 vectors, a row at a time; 93 with 1024 lanes, 4 rows). Rows that are not whole vectors take
// more registers, so fewer at once.
template <int DT, bool BWD, bool E, typename F>
bool by_width_of(int32_t D, F f) {
  constexpr bool FULL = BWD && !E && DT != FP32;   // 175 registers with two vectors (3001 bf16: 120 against 112 us)
  constexpr int V = vec_of<DT>(), MANY = E || !BWD || V == 4 ? 4 : 2;
  if (D <= 8 * V) f(Shape<E, 8, 1, MANY>{});
  else if (D <= 16 * V) f(Shape<E, 16, 1, MANY>{});
  else if (D <= 32 * V) f(Shape<E, 16, 2, 2>{});
  else if (D <= 64 * V) f(Shape<E, 64, 1, MANY>{});
  else if (D <= 128 * V) f(Shape<E, 64, 2, 2>{});
  else if (D <= 256 * V) f(Shape<E, 256, 1, MANY>{});
  else if (D <= 512 * V) f(Shape<E, FULL ? 512 : 256, FULL ? 1 : 2, 2>{});
  else if (D <= 1024 * V) f(Shape<E, BWD ? 1024 : 512, BWD ? 1 : 2, BWD ? MANY : 2>{});
  else if (D <= 2048 * V) f(Shape<E, 1024, 2, BWD ? 1 : 2>{});
  else if constexpr (V == 4) {
    if (D <= 4096 * V) f(Shape<E, 1024, 4, 1>{});
    else return false;
  } else {
    return false;
  }
  return true;
}
template <int DT, bool BWD, typename F>
bool by_width(int32_t D, F f) {
  return D % vec_of<DT>() == 0 ? by_width_of<DT, BWD, true>(D, f) : by_width_of<DT, BWD, false>(D, f);
}

template <typename F>
void by_dtype(int dt, F f) {
  if (dt == BF16) f(integral_constant<int, BF16>{});
  else if (dt == FP32) f(integral_constant<int, FP32>{});
  else f(integral_constant<int, FP16>{});
}

unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

}  // namespace

// Workgroups of a backward pass, at most: their sums take two rows of D each in the workspace,
// so wide rows get one workgroup per compute unit and short ones enough to fill the GPU. Rows of
// more than 16384 elements: as many parts as fill it beside their columns' lanes.
size_t layernorm_parts(int64_t M, int64_t D) {
  const int64_t most = D <= 1024 ? 1024 : D <= 2048 ? 768 : D <= 4096 ? 512 : D <= 16384 ? 256 : 1 + (8192 * 512) / D;
  return (size_t)(M < most ? M : most);
}

hipError_t launch_layernorm_fwd(const NormParams& p, hipStream_t stream) {
  if (p.M == 0) return hipSuccess;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    const bool done = by_width<DT, false>(p.D, [&](auto shape) {
      using S = decltype(shape);
      constexpr int wg = wg_of(S::lanes), step = wg / S::lanes * S::rows;
      hipLaunchKernelGGL((kda_layernorm_fwd_kernel<DT, S::exact, S::lanes, S::nv, S::rows>),
                         dim3(at_most((p.M + step - 1) / step, 2048 * 256 / wg)), dim3(wg), 0, stream, p);
    });
    if (!done)
      hipLaunchKernelGGL(kda_layernorm_fwd_long_kernel<DT>, dim3(at_most(p.M, 4096)), dim3(1024), 0, stream, p);
  });
  return hipGetLastError();
}

hipError_t launch_layernorm_bwd(const NormParams& p, hipStream_t stream) {
  int parts = (int)layernorm_parts(p.M, p.D);
  if (p.M > 0) {
    by_dtype(p.dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      const bool done = by_width<DT, true>(p.D, [&](auto shape) {
        using S = decltype(shape);
        constexpr int wg = wg_of(S::lanes), step = wg / S::lanes * S::rows;
        parts = (int)at_most((p.M + step - 1) / step, parts < 256 * 1024 / wg ? parts : 256 * 1024 / wg);
        hipLaunchKernelGGL((kda_layernorm_bwd_kernel<DT, S::exact, S::lanes, S::nv, S::rows>), dim3(parts), dim3(wg), 0, stream, p, parts);
      });
      if (!done) {
        if (p.partial) {
          const int64_t cols = ((int64_t)p.D + 64 * vec_of<DT>() - 1) / (64 * vec_of<DT>());
          hipLaunchKernelGGL(kda_layernorm_cols_kernel<DT>, dim3((unsigned)cols * parts), dim3(64), 0, stream, p, parts);
        }
        if (p.out)
          hipLaunchKernelGGL(kda_layernorm_bwd_long_kernel<DT>, dim3(at_most(p.M, 4096)), dim3(1024), 0, stream, p);
      }
    });
    const hipError_t e = hipGetLastError();
    if (e != hipSuccess) return e;
  }
  if (p.dw || p.db) {
    if (p.D <= 2048)
      hipLaunchKernelGGL(kda_layernorm_sum_kernel<16>, dim3((p.D + 15) / 16, 2), dim3(1024), 0, stream, p, parts);
    else
      hipLaunchKernelGGL(kda_layernorm_sum_kernel<64>, dim3((p.D + 63) / 64, 2), dim3(1024), 0, stream, p, parts);
    return hipGetLastError();
  }
  return hipSuccess;
}

}  // namespace kda
