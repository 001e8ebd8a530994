// kda_rmsnorm.hip -- root-mean-square norm of rows with the residual's addition, forward (into
// the inputs' type or 8 bits with scales) and backward (gfx950).
//
//     s = x + residual,  r = 1 / sqrt(mean(s^2) + eps),  y = s r weight
//     dx = r (a - s r^2 mean(a s)) + d_residual,  a = dy weight;   d_weight = sum dy s r
//
// Bound by memory (8192 x 8192 bf16: with residual into 8 bits 83 us, 5.7 TB/s; backward 97 us, 5.5
// TB/s, and 5 for adding the sums). A row is loaded once into the registers of LANES lanes (16 of a wave for the
// shortest rows, a workgroup of 1024 for the widest), 16 bytes a lane, vector and tensor; one sum
// over them gives r. The sum s is kept in fp32 and rounded only where it is stored. A scale
// belongs to 128 neighbouring elements, which 16 neighbouring lanes hold (fp32: 32), or to the
// row. Backward, workgroups take rows in strides and keep the sums of dy s r of their columns in
// registers from row to row; each writes its sums once to the workspace, and a second kernel adds
// those in a fixed order.
//
// Rows need not be whole numbers of vectors nor aligned to them: vectors are loaded at any
// address (the hardware splits what crosses a line), a row's last elements in smaller pieces.
// Rows of more than 16384 elements are read from memory once for the sum and again for what
// follows from it.
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

using std::integral_constant;

constexpr float E4M3_MAX = 448.0f;
constexpr int BLOCK = 128;   // elements of a scale that is not the row's

template <int CTRL>
__device__ __forceinline__ float dpp(float x) {
  return __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}
struct Add {
  __device__ __forceinline__ float operator()(float a, float b) const { return a + b; }
};
// of magnitudes as bits: NaN above infinity above all numbers
struct Most {
  __device__ __forceinline__ float operator()(float a, float b) const {
    const uint32_t x = __float_as_uint(a), y = __float_as_uint(b);
    return __uint_as_float(x > y ? x : y);
  }
};
// Over groups of 16, 32 or 64 lanes, the same bits in every lane.
template <int LANES, typename OP>
__device__ __forceinline__ float over_lanes(float x, OP op) {
  x = op(x, dpp<0xB1>(x));    // lane ^ 1
  x = op(x, dpp<0x1B>(x));    // lane ^ 3
  x = op(x, dpp<0x141>(x));   // lane ^ 7
  x = op(x, dpp<0x140>(x));   // lane ^ 15
  if constexpr (LANES >= 32) {
    const auto a = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  if constexpr (LANES >= 64) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
  }
  return x;
}
// Over the LANES lanes of a row, U rows at once. Rows of several waves go through buf, one barrier
// a call: consecutive calls take different parts of it.
template <int LANES, int U, typename OP>
__device__ __forceinline__ void over_row(float* v, float (*buf)[U], int part, OP op) {
#pragma unroll
  for (int u = 0; u < U; ++u) v[u] = over_lanes<(LANES > 64 ? 64 : LANES)>(v[u], op);
  if constexpr (LANES > 64) {
    constexpr int WAVES = LANES / 64;
    float (*b)[U] = buf + part * WAVES;
    if ((threadIdx.x & 63) == 0) {
#pragma unroll
      for (int u = 0; u < U; ++u) b[threadIdx.x >> 6][u] = v[u];
    }
    __syncthreads();
#pragma unroll
    for (int u = 0; u < U; ++u) {   // a wave's result in every lane, over 4, 8 or 16 lanes
      float s = b[threadIdx.x % WAVES][u];
      s = op(s, dpp<0xB1>(s));
      s = op(s, dpp<0x1B>(s));
      if constexpr (WAVES >= 8) s = op(s, dpp<0x141>(s));
      if constexpr (WAVES == 16) s = op(s, dpp<0x140>(s));
      v[u] = s;
    }
  }
}

template <int DT>
constexpr int vec_of() { return 16 / elem_size(DT); }
constexpr int wg_of(int lanes) { return lanes > 256 ? lanes : 256; }

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

// ---- 8-bit outputs ------------------------------------------------------------------

// A group's scale, and what its values are multiplied by, first with `up`: values whose scale is
// tiny (and its reciprocal infinite) are brought nearer to 1 before. A scale below the normal numbers
// is rounded to whole steps of 2^-149, at the worst to two thirds of what it should be: the quotients
// then pass 448 by up to half, and are held there.
struct Scale {
  float value, up, inv;
  bool coarse;
  __device__ __forceinline__ explicit Scale(float most) {
    value = most / E4M3_MAX;
    if (value == 0.0f) value = 1.0f;
    up = most < 0x1p-100f ? 0x1p96f : 1.0f;
    inv = 1.0f / (value * up);
    if (up != 1.0f && value == 1.0f) up = inv = 1.0f;
    coarse = value < 0x1p-126f;
  }
  template <int V>
  __device__ __forceinline__ void divide(float* f) const {
#pragma unroll
    for (int e = 0; e < V; ++e) f[e] = f[e] * up * inv;
    if (coarse) {
#pragma unroll
      for (int e = 0; e < V; ++e) f[e] = f[e] > E4M3_MAX ? E4M3_MAX : f[e] < -E4M3_MAX ? -E4M3_MAX : f[e];   // (NaN stays)
    }
  }
};
// rounded to nearest; finite values of a group over its scale are within what the format holds
template <int V>
__device__ __forceinline__ void store_e4m3(const float* f, void* p, size_t i, int c, bool whole) {
  uint8_t* a = static_cast<uint8_t*>(p) + i;
  uint32_t w[V / 4];
#pragma unroll
  for (int e = 0; e < V; e += 4) {
    int q = __builtin_amdgcn_cvt_pk_fp8_f32(f[e], f[e + 1], 0, false);
    w[e / 4] = (uint32_t)__builtin_amdgcn_cvt_pk_fp8_f32(f[e + 2], f[e + 3], q, true);
  }
  if (whole && c >= V) {
    if constexpr (V == 8) __builtin_nontemporal_store(u32x2{w[0], w[1]}, reinterpret_cast<u32x2*>(a));
    else __builtin_nontemporal_store(w[0], reinterpret_cast<uint32_t*>(a));
    return;
  }
#pragma unroll
  for (int e = 0; e < V; ++e)
    if (e < c) a[e] = (uint8_t)(w[e / 4] >> (8 * (e % 4)));
}

// ---- forward ----------------------------------------------------------------------

// A lane holds NV vectors of a row, U rows at a time. GROUP: 0 an output of x's type, 1 a scale
// for each 128 elements, 2 one for the row.
template <int DT, bool EXACT, int LANES, int NV, int U, int GROUP>
__global__ __launch_bounds__(wg_of(LANES)) void kda_rmsnorm_fwd_kernel(RmsParams p) {
  constexpr int VEC = vec_of<DT>(), G = wg_of(LANES) / LANES;
  __shared__ float buf[LANES > 64 ? 2 * LANES / 64 : 1][U];
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  const int blocks = (p.D + BLOCK - 1) / BLOCK;
  float w[NV][VEC];
  int c[NV];   // elements of this lane's vectors
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * LANES + lane) * VEC;
    c[i] = p.D - col < 0 ? 0 : p.D - col > VEC ? VEC : p.D - col;
    load_param<VEC>(p.weight, col, c[i], 1.0f, w[i]);
  }
  int half = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * G * U; m0 < p.M; m0 += (int64_t)gridDim.x * G * U) {
    float s[U][NV][VEC], q[U];
    {
      Pack<DT, VEC> x[U][NV], r[U][NV];
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * G + grp;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          const size_t at = (size_t)m * p.D + (i * LANES + lane) * VEC;
          x[u][i].clear();
          r[u][i].clear();
          if (m < p.M && c[i] > 0) {
            load_part<EXACT>(x[u][i], p.x, at, c[i]);
            if (p.res) load_part<EXACT>(r[u][i], p.res, at, c[i]);
          }
        }
      }
#pragma unroll
      for (int u = 0; u < U; ++u) {
        const int64_t m = m0 + u * G + grp;
        q[u] = 0.0f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
          x[u][i].unpack(s[u][i]);
          if (p.res) {
            float f[VEC];
            r[u][i].unpack(f);
#pragma unroll
            for (int e = 0; e < VEC; ++e) s[u][i][e] += f[e];
          }
#pragma unroll
          for (int e = 0; e < VEC; ++e) q[u] = fmaf(s[u][i][e], s[u][i][e], q[u]);
          if (p.res_out && m < p.M && c[i] > 0) {
            Pack<DT, VEC> o;
            o.pack(s[u][i]);
            store_part<EXACT>(o, p.res_out, (size_t)m * p.D + (i * LANES + lane) * VEC, c[i]);
          }
        }
      }
    }
    over_row<LANES, U>(q, buf, half, Add{});
    half ^= 1;
    float most[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      const float rstd = 1.0f / sqrtf(q[u] / p.D + p.eps);
      if (p.rstd && lane == 0 && m < p.M) p.rstd[m] = rstd;
      most[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          s[u][i][e] = s[u][i][e] * rstd * w[i][e];
          if (GROUP == 2) most[u] = Most{}(most[u], fabsf(s[u][i][e]));
        }
    }
    if (GROUP == 2) {
      over_row<LANES, U>(most, buf, half, Most{});
      half ^= 1;
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      if (GROUP == 2) {
        const Scale sc(most[u]);
        if (m < p.M && lane == 0) p.scales[m] = sc.value;
#pragma unroll
        for (int i = 0; i < NV; ++i) sc.divide<VEC>(s[u][i]);
      }
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const int col = (i * LANES + lane) * VEC;
        if (GROUP == 1) {
          float a = 0.0f;
#pragma unroll
          for (int e = 0; e < VEC; ++e) a = Most{}(a, fabsf(s[u][i][e]));
          const Scale sc(over_lanes<BLOCK / VEC>(a, Most{}));
          if (m < p.M && col % BLOCK == 0 && c[i] > 0) p.scales[m * blocks + col / BLOCK] = sc.value;
          sc.divide<VEC>(s[u][i]);
        }
        if (m >= p.M || c[i] <= 0) continue;
        const size_t at = (size_t)m * p.D + col;
        if (GROUP == 0) {
          Pack<DT, VEC> y;
          y.pack(s[u][i]);
          store_part<EXACT>(y, p.out, at, c[i]);
        } else {
          store_e4m3<VEC>(s[u][i], p.out, at, c[i], EXACT);
        }
      }
    }
  }
}

// Rows of more than 16384 elements, a workgroup each
template <int DT, int GROUP>
__global__ __launch_bounds__(1024) void kda_rmsnorm_fwd_long_kernel(RmsParams p) {
  constexpr int VEC = vec_of<DT>();
  __shared__ float buf[2 * 16][1];
  const int64_t blocks = (p.D + BLOCK - 1) / BLOCK;
  int half = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = (size_t)m * p.D;
    // f(column, elements, their sums): all lanes of a wave go through each round together
    auto each = [&](auto f) {
      for (int64_t c0 = 0; c0 < p.D; c0 += 1024 * VEC) {
        const int64_t col = c0 + (int64_t)threadIdx.x * VEC;
        const int c = p.D - col < 0 ? 0 : p.D - col < VEC ? (int)(p.D - col) : VEC;
        Pack<DT, VEC> x, r;
        x.clear();
        r.clear();
        if (c > 0) {
          load_part<false>(x, p.x, row + col, c);
          if (p.res) load_part<false>(r, p.res, row + col, c);
        }
        float s[VEC], g[VEC];
        x.unpack(s);
        r.unpack(g);
        if (p.res) {
#pragma unroll
          for (int e = 0; e < VEC; ++e) s[e] += g[e];
        }
        f((int)col, c, s);
      }
    };
    float q = 0.0f, most = 0.0f;
    each([&](int, int, const float* s) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) q = fmaf(s[e], s[e], q);
    });
    over_row<1024, 1>(&q, buf, half, Add{});
    half ^= 1;
    const float rstd = 1.0f / sqrtf(q / p.D + p.eps);
    if (p.rstd && threadIdx.x == 0) p.rstd[m] = rstd;
    auto norm = [&](int col, int c, float* s) {
      float w[VEC];
      load_param<VEC>(p.weight, col, c, 1.0f, w);
#pragma unroll
      for (int e = 0; e < VEC; ++e) s[e] = s[e] * rstd * w[e];
    };
    if (GROUP == 2) {
      each([&](int col, int c, float* s) {
        norm(col, c, s);
#pragma unroll
        for (int e = 0; e < VEC; ++e) most = Most{}(most, fabsf(s[e]));
      });
      over_row<1024, 1>(&most, buf, half, Most{});
      half ^= 1;
      if (threadIdx.x == 0) p.scales[m] = Scale(most).value;
    }
    each([&](int col, int c, float* s) {
      if (p.res_out && c > 0) {
        Pack<DT, VEC> o;
        o.pack(s);
        store_part<false>(o, p.res_out, row + col, c);
      }
      norm(col, c, s);
      if (GROUP == 1) {
        most = 0.0f;
#pragma unroll
        for (int e = 0; e < VEC; ++e) most = Most{}(most, fabsf(s[e]));
        most = over_lanes<BLOCK / VEC>(most, Most{});
      }
      if (GROUP != 0) {
        const Scale sc(most);
        if (GROUP == 1 && col % BLOCK == 0 && c > 0) p.scales[m * blocks + col / BLOCK] = sc.value;
        sc.divide<VEC>(s);
      }
      if (c <= 0) return;
      if (GROUP == 0) {
        Pack<DT, VEC> y;
        y.pack(s);
        store_part<false>(y, p.out, row + col, c);
      } else {
        store_e4m3<VEC>(s, p.out, row + col, c, p.D % VEC == 0);
      }
    });
  }
}

// ---- backward ---------------------------------------------------------------------

// Sum over the row groups of a workgroup; lanes 0 .. LANES - 1 of the workgroup end with the total.
template <int LANES>
__device__ __forceinline__ float groups_sum(float v, float* buf) {
  if constexpr (LANES <= 64) {
    constexpr int G = 256 / LANES;
    __syncthreads();
    buf[threadIdx.x] = v;
    __syncthreads();
    v = 0.0f;
    if (threadIdx.x < LANES) {
#pragma unroll
      for (int g = 0; g < G; ++g) v += buf[g * LANES + threadIdx.x];
    }
  }
  return v;
}

template <int DT, bool EXACT, int LANES, int NV, int U>
__global__ __launch_bounds__(wg_of(LANES)) void kda_rmsnorm_bwd_kernel(RmsParams p) {
  constexpr int VEC = vec_of<DT>(), G = wg_of(LANES) / LANES;
  __shared__ float buf[LANES > 64 ? 2 * LANES / 64 : 1][U];
  __shared__ float gbuf[LANES <= 64 ? 256 : 1];
  const int lane = threadIdx.x % LANES, grp = threadIdx.x / LANES;
  float w[NV][VEC], aw[NV][VEC];
  int c[NV];
#pragma unroll
  for (int i = 0; i < NV; ++i) {
    const int col = (i * LANES + lane) * VEC;
    c[i] = p.D - col < 0 ? 0 : p.D - col > VEC ? VEC : p.D - col;
    load_param<VEC>(p.weight, col, c[i], 1.0f, w[i]);
#pragma unroll
    for (int e = 0; e < VEC; ++e) aw[i][e] = 0.0f;
  }
  int half = 0;
  for (int64_t m0 = (int64_t)blockIdx.x * G * U; m0 < p.M; m0 += (int64_t)gridDim.x * G * U) {
    Pack<DT, VEC> x[U][NV], dy[U][NV], dr[U][NV];
    float rstd[U], q[U];
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      rstd[u] = m < p.M ? p.rstd[m] : 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        const size_t at = (size_t)m * p.D + (i * LANES + lane) * VEC;
        x[u][i].clear();
        dy[u][i].clear();
        dr[u][i].clear();
        if (m < p.M && c[i] > 0) {
          load_part<EXACT>(x[u][i], p.x, at, c[i]);
          load_part<EXACT>(dy[u][i], p.dy, at, c[i]);
          if (p.res && p.out) load_part<EXACT>(dr[u][i], p.res, at, c[i]);
        }
      }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
      q[u] = 0.0f;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float f[VEC], g[VEC];
        x[u][i].unpack(f);
        dy[u][i].unpack(g);
#pragma unroll
        for (int e = 0; e < VEC; ++e) {
          const float xh = f[e] * rstd[u];
          aw[i][e] = fmaf(g[e], xh, aw[i][e]);
          q[u] = fmaf(g[e] * w[i][e], xh, q[u]);
        }
      }
    }
    if (!p.out) continue;
    over_row<LANES, U>(q, buf, half, Add{});
    half ^= 1;
#pragma unroll
    for (int u = 0; u < U; ++u) {
      const int64_t m = m0 + u * G + grp;
      if (m >= p.M) continue;
      const float mean = q[u] / p.D;
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        if (c[i] <= 0) continue;
        float f[VEC], g[VEC], d[VEC];
        x[u][i].unpack(f);
        dy[u][i].unpack(g);
        dr[u][i].unpack(d);
#pragma unroll
        for (int e = 0; e < VEC; ++e) d[e] = fmaf(rstd[u], fmaf(-f[e] * rstd[u], mean, g[e] * w[i][e]), d[e]);
        Pack<DT, VEC> o;
        o.pack(d);
        store_part<EXACT>(o, p.out, (size_t)m * p.D + (i * LANES + lane) * VEC, c[i]);
      }
    }
  }
  if (!p.partial) return;
#pragma unroll
  for (int i = 0; i < NV; ++i)
#pragma unroll
    for (int e = 0; e < VEC; ++e) aw[i][e] = groups_sum<LANES>(aw[i][e], gbuf);
  if (threadIdx.x < LANES) {
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      float* to = p.partial + (size_t)blockIdx.x * p.D + (i * LANES + lane) * VEC;
#pragma unroll
      for (int e = 0; e < VEC; ++e)
        if (e < c[i]) to[e] = aw[i][e];
    }
  }
}

// Rows of more than 16384 elements: dx, a workgroup each; the weight's sums by columns
template <int DT>
__global__ __launch_bounds__(1024) void kda_rmsnorm_bwd_long_kernel(RmsParams p) {
  constexpr int VEC = vec_of<DT>();
  __shared__ float buf[2 * 16][1];
  int half = 0;
  for (int64_t m = blockIdx.x; m < p.M; m += gridDim.x) {
    const size_t row = (size_t)m * p.D;
    const float rstd = p.rstd[m];
    auto each = [&](auto f) {
      for (int64_t col = (int64_t)threadIdx.x * VEC; col < p.D; col += 1024 * VEC) {
        const int c = p.D - col < VEC ? (int)(p.D - col) : VEC;
        Pack<DT, VEC> x, dy;
        load_part<false>(x, p.x, row + col, c);
        load_part<false>(dy, p.dy, row + col, c);
        float s[VEC], g[VEC], w[VEC];
        x.unpack(s);
        dy.unpack(g);
        load_param<VEC>(p.weight, (int)col, c, 1.0f, w);
        f((int)col, c, s, g, w);
      }
    };
    float q = 0.0f;
    each([&](int, int, const float* s, const float* g, const float* w) {
#pragma unroll
      for (int e = 0; e < VEC; ++e) q = fmaf(g[e] * w[e], s[e] * rstd, q);
    });
    over_row<1024, 1>(&q, buf, half, Add{});
    half ^= 1;
    const float mean = q / p.D;
    each([&](int col, int c, const float* s, const float* g, const float* w) {
      Pack<DT, VEC> dr;
      dr.clear();
      if (p.res) load_part<false>(dr, p.res, row + col, c);
      float d[VEC];
      dr.unpack(d);
#pragma unroll
      for (int e = 0; e < VEC; ++e) d[e] = fmaf(rstd, fmaf(-s[e] * rstd, mean, g[e] * w[e]), d[e]);
      Pack<DT, VEC> o;
      o.pack(d);
      store_part<false>(o, p.out, row + col, c);
    });
  }
}
template <int DT>
__global__ __launch_bounds__(64) void kda_rmsnorm_cols_kernel(RmsParams p, int parts) {
  constexpr int VEC = vec_of<DT>();
  const int64_t cols = ((int64_t)p.D + 64 * VEC - 1) / (64 * VEC);
  const int64_t part = blockIdx.x / cols, col = ((blockIdx.x % cols) * 64 + threadIdx.x) * VEC;
  if (col >= p.D) return;
  const int c = p.D - col < VEC ? (int)(p.D - col) : VEC;
  float s[VEC] = {};
  for (int64_t m = part; m < p.M; m += parts) {
    Pack<DT, VEC> x, dy;
    load_part<false>(x, p.x, (size_t)m * p.D + col, c);
    load_part<false>(dy, p.dy, (size_t)m * p.D + col, c);
    float f[VEC], g[VEC];
    x.unpack(f);
    dy.unpack(g);
#pragma unroll
    for (int e = 0; e < VEC; ++e) s[e] = fmaf(g[e], f[e] * p.rstd[m], s[e]);
  }
#pragma unroll
  for (int e = 0; e < VEC; ++e)
    if (e < c) p.partial[(size_t)part * p.D + col + e] = s[e];
}

// d_weight: the sum of the parts, 64 columns by 16 runs of parts
__global__ __launch_bounds__(1024) void kda_rmsnorm_sum_kernel(RmsParams p, int parts) {
  __shared__ float buf[16][64];
  const int j = threadIdx.x & 63, run = threadIdx.x >> 6;
  const int64_t col = (int64_t)blockIdx.x * 64 + j;
  float s = 0.0f;
  if (col < p.D) {
#pragma unroll 8
    for (int i = run; i < parts; i += 16) s += p.partial[(size_t)i * p.D + col];
  }
  buf[run][j] = s;
  __syncthreads();
#pragma unroll
  for (int o = 8; o >= 1; o >>= 1) {
    if (run < o) buf[run][j] += buf[run + o][j];
    __syncthreads();
  }
  if (run == 0 && col < p.D) p.dw[col] = buf[0][j];
}

// ---- launches ---------------------------------------------------------------------

template <bool E, int L, int V, int U>
struct Shape {
  static constexpr bool exact = E;
  static constexpr int lanes = L, nv = V, rows = U;
};

// f(shape) for the fewest lanes, and vectors of a lane, that hold a row; false: none does. Few
// vectors leave registers for more rows at once.
template <int DT, bool E, typename F>
bool by_width_of(int32_t D, F f) {
  constexpr int V = vec_of<DT>(), LEAST = BLOCK / V;   // lanes that hold what has one scale
  if (D <= LEAST * V) f(Shape<E, LEAST, 1, 2>{});
  else if (D <= 64 * V) f(Shape<E, 64, 1, 2>{});
  else if (D <= 128 * V) f(Shape<E, 64, 2, 2>{});
  else if (D <= 256 * V) f(Shape<E, 256, 1, 2>{});
  else if (D <= 512 * V) f(Shape<E, 512, 1, 2>{});
  else if (D <= 1024 * V) f(Shape<E, 1024, 1, 2>{});
  else if (D <= 2048 * V) f(Shape<E, 1024, 2, 1>{});
  else if constexpr (V == 4) {
    if (D <= 4096 * V) f(Shape<E, 1024, 4, 1>{});
    else return false;
  } else {
    return false;
  }
  return true;
}
template <int DT, typename F>
bool by_width(int32_t D, F f) {
  return D % vec_of<DT>() == 0 ? by_width_of<DT, true>(D, f) : by_width_of<DT, false>(D, f);
}
template <typename F>
void by_dtype(int dt, F f) {
  if (dt == BF16) f(integral_constant<int, BF16>{});
  else if (dt == FP32) f(integral_constant<int, FP32>{});
  else f(integral_constant<int, FP16>{});
}
unsigned at_most(int64_t n, int64_t most) { return (unsigned)(n < most ? n : most); }

template <int DT, int GROUP>
void forward(const RmsParams& p, hipStream_t stream) {
  const bool done = by_width<DT>(p.D, [&](auto shape) {
    using S = decltype(shape);
    constexpr int wg = wg_of(S::lanes), step = wg / S::lanes * S::rows;
    hipLaunchKernelGGL((kda_rmsnorm_fwd_kernel<DT, S::exact, S::lanes, S::nv, S::rows, GROUP>),
                       dim3(at_most((p.M + step - 1) / step, 2048 * 256 / wg)), dim3(wg), 0, stream, p);
  });
  if (!done) hipLaunchKernelGGL((kda_rmsnorm_fwd_long_kernel<DT, GROUP>), dim3(at_most(p.M, 4096)), dim3(1024), 0, stream, p);
}

}  // namespace

// Workgroups of a backward pass, at most: their sums take a row of D each in the workspace
size_t rmsnorm_parts(int64_t M, int64_t D) {
  const int64_t most = D <= 1024 ? 1024 : D <= 2048 ? 768 : D <= 4096 ? 512 : D <= 16384 ? 256 : 1 + (8192 * 512) / D;
  return (size_t)(M < most ? M : most);
}

hipError_t launch_rmsnorm_fwd(const RmsParams& p, hipStream_t stream) {
  if (p.M == 0) return hipSuccess;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    // (rows of at most 128 elements have one scale either way)
    if (p.group == 0) forward<DT, 0>(p, stream);
    else if (p.group == BLOCK) forward<DT, 1>(p, stream);
    else forward<DT, 2>(p, stream);
  });
  return hipGetLastError();
}

hipError_t launch_rmsnorm_bwd(const RmsParams& p, hipStream_t stream) {
  int parts = (int)rmsnorm_parts(p.M, p.D);
  if (p.M > 0) {
    by_dtype(p.dtype, [&](auto dt) {
      constexpr int DT = decltype(dt)::value;
      const bool done = by_width<DT>(p.D, [&](auto shape) {
        using S = decltype(shape);
        constexpr int wg = wg_of(S::lanes), step = wg / S::lanes * S::rows;
        parts = (int)at_most((p.M + step - 1) / step, parts < 256 * 1024 / wg ? parts : 256 * 1024 / wg);
        hipLaunchKernelGGL((kda_rmsnorm_bwd_kernel<DT, S::exact, S::lanes, S::nv, S::rows>), dim3(parts), dim3(wg), 0, stream, p);
      });
      if (!done) {
        if (p.partial) {
          const int64_t cols = ((int64_t)p.D + 64 * vec_of<DT>() - 1) / (64 * vec_of<DT>());
          hipLaunchKernelGGL(kda_rmsnorm_cols_kernel<DT>, dim3((unsigned)cols * parts), dim3(64), 0, stream, p, parts);
        }
        if (p.out) hipLaunchKernelGGL(kda_rmsnorm_bwd_long_kernel<DT>, dim3(at_most(p.M, 4096)), dim3(1024), 0, stream, p);
      }
    });
  }
  if (p.dw) hipLaunchKernelGGL(kda_rmsnorm_sum_kernel, dim3((p.D + 63) / 64), dim3(1024), 0, stream, p, parts);
  return hipGetLastError();
}

}  // namespace kda
