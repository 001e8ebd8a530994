// kda_ssm.hip -- selective state space scan, forward, backward and single tokens (gfx950).
//
//     h_t[e] = exp(s_t A[e]) h_{t-1}[e] + s_t x_t B_t[e]
//     y_t = (sum_e C_t[e] h_t[e] + skip x_t) SiLU(z_t)
//
// per channel, s_t = softplus(dt_t + bias). Bound by the vector units: each of the T D E updates
// takes an exponential (16 cycles of a wave) and four operations (16). The states of a channel
// are four to a lane (LPC lanes a channel, E rounded up to LPC 4), so that the sum over e stays
// in a few neighbouring lanes; everything that is the same for a channel's states (s_t, s_t x_t,
// SiLU(z_t)) is computed once, by the lanes that load it, 16 tokens at a time, and handed over
// in shared memory together with B and C.
//
// A sequence's tokens follow each other; where channels and states alone do not fill the GPU the
// packed tokens are cut into chunks. A chunk acts on the state entering it as h -> P h + R with
// P = exp(A sum s_t): one launch computes R and the sum of s of all chunks but the last, a second
// one runs through the chunks for the state that enters each, the third computes the outputs. A
// sequence's first token puts its initial state in the place of h; a chunk with one passes no state
// on (reset), whatever is before it.
//
// Backward, with g = dy SiLU(z): G_t = C_t g_t + exp(s_{t+1} A) G_{t+1} runs from the last token to
// the first, by chunks in the same manner. The states h are recomputed from those that the forward
// pass has saved every 64 tokens, 16 tokens at a time in registers. The sums over channels (dB,
// dC) are halved from lane to lane with two values at once, added up over a workgroup, and over
// workgroups by a kernel after it, as the sums over chunks (dA, d_skip, d_bias) are.
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"
#include "kda_seq.h"

namespace kda {
namespace {

using std::integral_constant;

constexpr int SUB = 16;     // tokens that a workgroup stages at once
constexpr int BLK = SSM_BLOCK;
static_assert(BLK == 4 * SUB, "");

__device__ __forceinline__ Seqs seqs_of(const SsmParams& p) { return {p.cu, p.nseq, p.T, p.tokens}; }

template <int CTRL>
__device__ __forceinline__ float dpp_add(float x) {
  return x + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(x), CTRL, 0xf, 0xf, false));
}
// Sum over groups of N neighbouring lanes (2, 4, 8 or 16), the same bits in every lane
template <int N>
__device__ __forceinline__ float part_sum(float x) {
  if constexpr (N >= 2) x = dpp_add<0xB1>(x);    // lane ^ 1
  if constexpr (N >= 4) x = dpp_add<0x4E>(x);    // lane ^ 2
  if constexpr (N >= 8) x = dpp_add<0x141>(x);   // lane ^ 7
  if constexpr (N >= 16) x = dpp_add<0x140>(x);  // lane ^ 15
  return x;
}
// a summed over lanes l, l ^ 32 in the lower half of the wave, b in the upper one
__device__ __forceinline__ float halves32(float a, float b) {
  const auto r = __builtin_amdgcn_permlane32_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
// likewise over l, l ^ 16: a in lanes without bit 4, b in those with it
__device__ __forceinline__ float halves16(float a, float b) {
  const auto r = __builtin_amdgcn_permlane16_swap(__float_as_uint(a), __float_as_uint(b), false, false);
  return __uint_as_float(r[0]) + __uint_as_float(r[1]);
}
__device__ __forceinline__ float xor4_add(float x) {
  int o = __builtin_amdgcn_update_dpp(0, __float_as_int(x), 0x104, 0xf, 0x5, false);   // row_shl 4: lanes without bit 2
  o = __builtin_amdgcn_update_dpp(o, __float_as_int(x), 0x114, 0xf, 0xa, false);       // row_shr 4: lanes with it
  return x + __int_as_float(o);
}

// e = exp(-|u|) gives log(1 + exp(u)) and its derivative. log(1 + e) as 2 atanh(e / (2 + e)), a
// series in powers of at most 1/9: the hardware's logarithm of 1 + e would lose a small e's digits.
__device__ __forceinline__ float softplus(float u) {
  const float e = fast_exp2(-fabsf(u) * LOG2E);
  const float r = e * fast_rcp(2.0f + e), q = r * r;
  float s = 1.0f / 13.0f;
  s = fmaf(s, q, 1.0f / 11.0f);
  s = fmaf(s, q, 1.0f / 9.0f);
  s = fmaf(s, q, 1.0f / 7.0f);
  s = fmaf(s, q, 1.0f / 5.0f);
  s = fmaf(s, q, 1.0f / 3.0f);
  s = fmaf(s, q, 1.0f);
  return fmaf(2.0f * r, s, u > 0.0f ? u : u != u ? u : 0.0f);
}
__device__ __forceinline__ float sigmoid(float u) {
  const float e = fast_exp2(-fabsf(u) * LOG2E), r = fast_rcp(1.0f + e);
  return u < 0.0f ? e * r : r;
}

// N elements of a token tensor from element i on, the first c of them; `vec`: all, aligned
template <int DT, int N>
__device__ __forceinline__ void load_some(const void* p, size_t i, int c, bool vec, float* f) {
  if (vec) {
    if (c >= N) {
      load_f32<DT, N>(p, i, f);
      return;
    }
#pragma unroll
    for (int e = 0; e < N; ++e) f[e] = 0.0f;
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e) {
    f[e] = 0.0f;
    if (e < c) load_f32<DT, 1>(p, i + e, f + e);
  }
}
template <int DT, int N>
__device__ __forceinline__ void store_some(void* p, size_t i, int c, bool vec, const float* f) {
  if (vec) {
    if (c >= N) store_f32<DT, N>(p, i, f);
    return;
  }
#pragma unroll
  for (int e = 0; e < N; ++e)
    if (e < c) store_f32<DT, 1>(p, i + e, f + e);
}
template <int N>
__device__ __forceinline__ void load_vec(const float* p, size_t i, int c, float none, float* f) {
#pragma unroll
  for (int e = 0; e < N; ++e) f[e] = p && e < c ? p[i + e] : none;
}

// ---- a workgroup's part of the channels, and its lanes' ------------------------------

template <int LPC>
struct Tile {
  static constexpr int CW = 256 / LPC;     // channels of a workgroup, all of one group
  static constexpr int EPT = 16 / LPC;     // channels of a lane that loads: 16 lanes a token
  static constexpr int EW = 4 * LPC;       // states of a channel, with those that are none
  int g, d0, dn;                           // group, first channel, channels
  int ch, part, d, e0, ec;                 // a lane's channel and its states e0 .. e0 + ec - 1
  int row, c0, cn;                         // as one that loads: token, first channel (of CW), channels

  __device__ __forceinline__ Tile(const SsmParams& p, int tile, int per_group) {
    const int Dg = p.D / p.G;
    g = tile / per_group;
    const int at = (tile - g * per_group) * CW;
    d0 = g * Dg + at;
    dn = Dg - at < CW ? Dg - at : CW;
    ch = threadIdx.x / LPC;
    part = threadIdx.x % LPC;
    d = d0 + ch;
    e0 = 4 * part;
    ec = ch < dn ? (p.E - e0 < 0 ? 0 : p.E - e0 < 4 ? p.E - e0 : 4) : 0;
    row = threadIdx.x >> 4;
    c0 = (threadIdx.x & 15) * EPT;
    cn = dn - c0 < 0 ? 0 : dn - c0 < EPT ? dn - c0 : EPT;
  }
  // fp32 [rows, D, E] arrays of the library
  __device__ __forceinline__ size_t at(const SsmParams& p, size_t row_) const { return (row_ * p.D + d) * p.E + e0; }
  __device__ __forceinline__ void load4(const SsmParams& p, const float* a, size_t row_, float* h) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = 0.0f;
    if (ec == 4 && p.E % 4 == 0) load_f32<FP32, 4>(a, at(p, row_), h);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ec) h[j] = a[at(p, row_) + j];
    }
  }
  __device__ __forceinline__ void store4(const SsmParams& p, float* a, size_t row_, const float* h) const {
    if (ec == 4 && p.E % 4 == 0) store_f32<FP32, 4>(a, at(p, row_), h);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ec) a[at(p, row_) + j] = h[j];
    }
  }
  __device__ __forceinline__ void load_state4(const SsmParams& p, const void* a, int dtype, size_t row_, float* h) const {
#pragma unroll
    for (int j = 0; j < 4; ++j) h[j] = 0.0f;
    if (ec == 4 && p.E % 4 == 0) load_state<4>(a, dtype, at(p, row_), h);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ec) load_state<1>(a, dtype, at(p, row_) + j, h + j);
    }
  }
  __device__ __forceinline__ void store_state4(const SsmParams& p, void* a, int dtype, size_t row_, const float* h) const {
    if (ec == 4 && p.E % 4 == 0) store_state<4>(a, dtype, at(p, row_), h);
    else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < ec) store_state<1>(a, dtype, at(p, row_) + j, h + j);
    }
  }
};

// B and C of SUB tokens as they lie in shared memory
template <int LPC>
struct alignas(16) Shared2 {
  float b[SUB][4 * LPC], c[SUB][4 * LPC];
};
template <int DT, int LPC, bool WITH_B, bool WITH_C>
struct StageBC {
  static constexpr int N = SUB * 4 * LPC, K = (N + 255) / 256;   // values of a lane, of B and of C
  float b[K], c[K];
  __device__ __forceinline__ void load(const SsmParams& p, int g, int32_t t, int32_t lo, int32_t hi) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = threadIdx.x + 256 * k, r = i / (4 * LPC), e = i % (4 * LPC);
      b[k] = c[k] = 0.0f;
      if (i < N && e < p.E && t + r >= lo && t + r < hi) {
        const size_t at = ((size_t)(t + r) * p.G + g) * p.E + e;
        if (WITH_B) load_f32<DT, 1>(p.Bm, at, b + k);
        if (WITH_C) load_f32<DT, 1>(p.Cm, at, c + k);
      }
    }
  }
  __device__ __forceinline__ void store(float* sb, float* sc) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = threadIdx.x + 256 * k;
      if (i < N) {
        if (WITH_B) sb[i] = b[k];
        if (WITH_C) sc[i] = c[k];
      }
    }
  }
};

// ---- forward ----------------------------------------------------------------------

// FINAL: the outputs; else the chunk's map.
template <int DT, int LPC, bool FINAL>
__global__ __launch_bounds__(256) void kda_ssm_fwd_kernel(SsmParams p, SsmWs w) {
  using TileT = Tile<LPC>;
  constexpr int CW = TileT::CW, EPT = TileT::EPT;
  __shared__ f32x2 s_d[2][SUB][CW];   // s, s x
  __shared__ Shared2<LPC> s_bc[2];
  __shared__ float s_y[FINAL ? 2 : 1][FINAL ? SUB : 1][CW];
  const Seqs seqs = seqs_of(p);
  const int tile = blockIdx.x % w.tiles, chunk = blockIdx.x / w.tiles;
  const TileT T(p, tile, w.per_group);
  const bool vec = (p.D / p.G) % EPT == 0 && p.D % EPT == 0;
  const int32_t t_lo = chunk * w.len, t_hi = p.tokens - t_lo < w.len ? p.tokens : t_lo + w.len;
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n) < t_hi ? seqs.begin(seqs.n) : t_hi;
  float A[4], h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
  T.load4(p, p.A, 0, A);
#pragma unroll
  for (int j = 0; j < 4; ++j) A[j] *= LOG2E;
  float bias[EPT], skip[EPT];
  load_vec<EPT>(p.dt_bias, T.d0 + T.c0, T.cn, 0.0f, bias);
  if (FINAL) load_vec<EPT>(p.skip, T.d0 + T.c0, T.cn, 0.0f, skip);
  if (FINAL && chunk > 0) T.load4(p, w.maps, chunk - 1, h);
  bool reset = false;

  float x[EPT], dt[EPT], z[EPT], ox[EPT], oz[EPT];
  StageBC<DT, LPC, true, FINAL> bc;
  auto load = [&](int32_t t) {
    const int32_t tt = t + T.row;
    const int c = tt >= lo && tt < hi ? T.cn : 0;
    const size_t i = (size_t)tt * p.D + T.d0 + T.c0;
    load_some<DT, EPT>(p.x, i, c, vec, x);
    load_some<DT, EPT>(p.dt, i, c, vec, dt);
    if (FINAL && p.z) load_some<DT, EPT>(p.z, i, c, vec, z);
    bc.load(p, T.g, t, lo, hi);
  };
  auto stage = [&](int32_t t, int buf) {
    const bool in = t + T.row >= lo && t + T.row < hi;   // others leave the state as it is: s = 0
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float u = dt[i] + bias[i];
      const float s = in && i < T.cn ? (p.softplus ? softplus(u) : u) : 0.0f;
      s_d[buf][T.row][T.c0 + i] = f32x2{s, in && i < T.cn ? s * x[i] : 0.0f};
      ox[i] = x[i];
      oz[i] = z[i];
    }
    bc.store(&s_bc[buf].b[0][0], &s_bc[buf].c[0][0]);
  };
  auto step = [&](int buf, int r) {   // one token; the lane's part of its y
    const f32x2 d = s_d[buf][r][T.ch];
    const f32x4 b = *reinterpret_cast<const f32x4*>(&s_bc[buf].b[r][T.e0]);
    f32x4 c = {};
    if (FINAL) c = *reinterpret_cast<const f32x4*>(&s_bc[buf].c[r][T.e0]);
    float y = 0.0f;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = fmaf(fast_exp2(d.x * A[j]), h[j], d.y * b[j]);
      if (FINAL) y = fmaf(c[j], h[j], y);
    }
    if (!FINAL) sum += d.x;
    return y;
  };
  SeqWalk q;
  q.start(seqs, t_lo);
  if (t_lo < t_hi) {
    load(t_lo);
    stage(t_lo, 0);
  }
  __syncthreads();
  int buf = 0;
  for (int32_t t = t_lo; t < t_hi; t += SUB, buf ^= 1) {
    float px[EPT], pz[EPT];
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      px[i] = ox[i];
      pz[i] = oz[i];
    }
    if (t + SUB < t_hi) load(t + SUB);
    if (FINAL && p.carry && t % BLK == 0) T.store4(p, p.carry, t / BLK, h);
    if (q.b < t && q.e > t + SUB) {   // no sequence begins or ends here
#pragma unroll
      for (int r = 0; r < SUB; r += 4) {
        float y[4];
#pragma unroll
        for (int u = 0; u < 4; ++u) y[u] = step(buf, r + u);
        if (FINAL) {
#pragma unroll
          for (int u = 0; u < 4; ++u) y[u] = part_sum<LPC>(y[u]);
          if constexpr (LPC >= 4) {
            if (T.part < 4) s_y[buf][r + T.part][T.ch] = T.part == 0 ? y[0] : T.part == 1 ? y[1] : T.part == 2 ? y[2] : y[3];
          } else {
            s_y[buf][r + T.part][T.ch] = T.part ? y[1] : y[0];
            s_y[buf][r + 2 + T.part][T.ch] = T.part ? y[3] : y[2];
          }
        }
      }
    } else {
#pragma unroll 1
      for (int r = 0; r < SUB && t + r < t_hi; ++r) {
        if (t + r >= q.e) q.forward(seqs, t + r);
        if (t + r == q.b && q.holds(t + r)) {
          // the last sequence that goes on after this chunk has its final state written elsewhere,
          // perhaps over its initial state: that is put aside
          const bool goes_on = w.stage && q.e > t_hi;
          if (FINAL && goes_on) T.load4(p, w.stage, chunk, h);
          else T.load_state4(p, p.init, p.init_dtype, q.i, h);
          if (!FINAL && goes_on) T.store4(p, w.stage, chunk, h);
          reset = true;
        }
        const float y = part_sum<LPC>(step(buf, r));
        if (FINAL && T.part == 0) s_y[buf][r][T.ch] = y;
        if (FINAL && p.fin && t + r == q.e - 1 && q.holds(t + r)) T.store_state4(p, p.fin, p.fin_dtype, q.i, h);
      }
    }
    if (t + SUB < t_hi) stage(t + SUB, buf ^ 1);
    __syncthreads();
    if (FINAL) {
      const int32_t tt = t + T.row;
      if (tt >= lo && tt < hi) {
        float y[EPT];
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          y[i] = fmaf(skip[i], px[i], s_y[buf][T.row][T.c0 + i]);
          if (p.z) y[i] *= pz[i] * sigmoid(pz[i]);
        }
        store_some<DT, EPT>(p.y, (size_t)tt * p.D + T.d0 + T.c0, T.cn, vec, y);
      }
    }
  }
  if (FINAL) {   // sequences without tokens
    if (p.fin)
      for (int n = chunk; n < p.nseq; n += w.chunks)
        if (seqs.begin(n) >= seqs.begin(n + 1)) {
          T.load_state4(p, p.init, p.init_dtype, n, h);
          T.store_state4(p, p.fin, p.fin_dtype, n, h);
        }
  } else {
    T.store4(p, w.maps, chunk, h);
    if (T.part == 0 && T.ch < T.dn) w.sums[(size_t)chunk * p.D + T.d] = sum;
    if (tile == 0 && threadIdx.x == 0) w.resets[chunk] = reset;
  }
}

// maps[c] becomes the state that leaves chunk c (BACK: the gradient that leaves chunk count - c
// towards its first token); one lane a channel's state
template <bool BACK>
__global__ __launch_bounds__(256) void kda_ssm_pass_kernel(SsmParams p, SsmWs w, int count) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)p.D * p.E;
  if (i >= n) return;
  const int64_t d = i / p.E;
  const float A = p.A[i] * LOG2E;
  float h = 0.0f;
  constexpr int AHEAD = 8;
  for (int c0 = 0; c0 < count; c0 += AHEAD) {
    float r[AHEAD], s[AHEAD];
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      const int c = BACK ? count - 1 - (c0 + k) : c0 + k;
      r[k] = s[k] = 0.0f;
      if (c0 + k < count) {
        r[k] = w.maps[c * n + i];
        s[k] = w.sums[(int64_t)c * p.D + d];
      }
    }
#pragma unroll
    for (int k = 0; k < AHEAD; ++k) {
      if (c0 + k >= count) break;
      const int c = BACK ? count - 1 - (c0 + k) : c0 + k;
      h = c0 + k == 0 || w.resets[c] ? r[k] : fmaf(fast_exp2(A * s[k]), h, r[k]);
      w.maps[c * n + i] = h;
    }
  }
}

// ---- single tokens ------------------------------------------------------------------

template <int DT, int LPC>
__global__ __launch_bounds__(256) void kda_ssm_step_kernel(SsmParams p, SsmWs w) {
  const Tile<LPC> T(p, blockIdx.x % w.tiles, w.per_group);
  if (T.ch >= T.dn) return;
  float A[4];
  T.load4(p, p.A, 0, A);
  const float bias = p.dt_bias ? p.dt_bias[T.d] : 0.0f, skip = p.skip ? p.skip[T.d] : 0.0f;
  for (int n = blockIdx.x / w.tiles; n < p.nseq; n += gridDim.x / w.tiles) {
    const int from = p.in_slots[n], to = p.out_slots[n];
    const size_t i = (size_t)n * p.D + T.d, bc = ((size_t)n * p.G + T.g) * p.E + T.e0;
    float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, x, dt, z = 0.0f, y = 0.0f;
    if (from >= 0 && from < p.n_slots) T.load_state4(p, p.init, p.init_dtype, from, h);
    load_f32<DT, 1>(p.x, i, &x);
    load_f32<DT, 1>(p.dt, i, &dt);
    if (p.z) load_f32<DT, 1>(p.z, i, &z);
    const float s = p.softplus ? softplus(dt + bias) : dt + bias;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      float b = 0.0f, c = 0.0f;
      if (j < T.ec) {
        load_f32<DT, 1>(p.Bm, bc + j, &b);
        load_f32<DT, 1>(p.Cm, bc + j, &c);
      }
      h[j] = fmaf(fast_exp2(s * A[j] * LOG2E), h[j], s * x * b);
      y = fmaf(c, h[j], y);
    }
    if (to >= 0 && to < p.n_slots) T.store_state4(p, p.fin, p.fin_dtype, to, h);
    y = fmaf(skip, x, part_sum<LPC>(y));
    if (p.z) y *= z * sigmoid(z);
    if (T.part == 0) store_f32<DT, 1>(p.y, i, &y);
  }
}

// ---- backward ---------------------------------------------------------------------

// g = dy SiLU(z)
__device__ __forceinline__ float gated(float dy, float z, bool has_z) { return has_z ? dy * (z * sigmoid(z)) : dy; }

// A chunk's map of the gradient that comes from the tokens after it
template <int DT, int LPC>
__global__ __launch_bounds__(256) void kda_ssm_bwd_map_kernel(SsmParams p, SsmWs w) {
  using TileT = Tile<LPC>;
  constexpr int CW = TileT::CW, EPT = TileT::EPT;
  __shared__ f32x2 s_d[2][SUB][CW];   // s, g
  __shared__ Shared2<LPC> s_bc[2];
  const Seqs seqs = seqs_of(p);
  const int tile = blockIdx.x % w.tiles, chunk = 1 + blockIdx.x / w.tiles;
  const TileT T(p, tile, w.per_group);
  const bool vec = (p.D / p.G) % EPT == 0 && p.D % EPT == 0;
  const int32_t t_lo = chunk * w.len, t_hi = p.tokens - t_lo < w.len ? p.tokens : t_lo + w.len;
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n) < t_hi ? seqs.begin(seqs.n) : t_hi;
  float A[4], G[4] = {0.0f, 0.0f, 0.0f, 0.0f}, sum = 0.0f;
  T.load4(p, p.A, 0, A);
#pragma unroll
  for (int j = 0; j < 4; ++j) A[j] *= LOG2E;
  float bias[EPT], dt[EPT], z[EPT], dy[EPT];
  load_vec<EPT>(p.dt_bias, T.d0 + T.c0, T.cn, 0.0f, bias);
  bool reset = false;
  StageBC<DT, LPC, false, true> bc;
  auto load = [&](int32_t t) {
    const int32_t tt = t + T.row;
    const int c = tt >= lo && tt < hi ? T.cn : 0;
    const size_t i = (size_t)tt * p.D + T.d0 + T.c0;
    load_some<DT, EPT>(p.dt, i, c, vec, dt);
    load_some<DT, EPT>(p.dy, i, c, vec, dy);
    if (p.z) load_some<DT, EPT>(p.z, i, c, vec, z);
    bc.load(p, T.g, t, lo, hi);
  };
  auto stage = [&](int32_t t, int buf) {
    const bool in = t + T.row >= lo && t + T.row < hi;
#pragma unroll
    for (int i = 0; i < EPT; ++i) {
      const float u = dt[i] + bias[i];
      const bool ok = in && i < T.cn;
      s_d[buf][T.row][T.c0 + i] = f32x2{ok ? (p.softplus ? softplus(u) : u) : 0.0f, ok ? gated(dy[i], z[i], p.z) : 0.0f};
    }
    bc.store(&s_bc[buf].b[0][0], &s_bc[buf].c[0][0]);
  };
  auto step = [&](int buf, int r) {
    const f32x2 d = s_d[buf][r][T.ch];
    const f32x4 c = *reinterpret_cast<const f32x4*>(&s_bc[buf].c[r][T.e0]);
#pragma unroll
    for (int j = 0; j < 4; ++j) G[j] = fast_exp2(d.x * A[j]) * fmaf(c[j], d.y, G[j]);
    sum += d.x;
  };
  SeqWalk q;
  q.start(seqs, t_hi - 1);
  const int32_t last = t_lo + (t_hi - t_lo - 1) / SUB * SUB;
  load(last);
  stage(last, 0);
  __syncthreads();
  int buf = 0;
  for (int32_t t = last; t >= t_lo; t -= SUB, buf ^= 1) {
    if (t > t_lo) load(t - SUB);
    if (q.b < t && q.e > t + SUB) {
#pragma unroll
      for (int r = SUB - 1; r >= 0; --r) step(buf, r);
    } else {
#pragma unroll 1
      for (int r = SUB - 1; r >= 0; --r) {
        if (t + r >= t_hi) continue;
        if (t + r < q.b) q.back(seqs, t + r);
        if (p.dfin && t + r == q.e - 1 && q.holds(t + r)) {
          float f[4];
          T.load_state4(p, p.dfin, p.dfin_dtype, q.i, f);
#pragma unroll
          for (int j = 0; j < 4; ++j) G[j] += f[j];
        }
        step(buf, r);
        if (t + r == q.b && q.holds(t + r)) {
#pragma unroll
          for (int j = 0; j < 4; ++j) G[j] = 0.0f;
          reset = true;
        }
      }
    }
    if (t > t_lo) stage(t - SUB, buf ^ 1);
    __syncthreads();
  }
  T.store4(p, w.maps, chunk - 1, G);
  if (T.part == 0 && T.ch < T.dn) w.sums[(size_t)(chunk - 1) * p.D + T.d] = sum;
  if (tile == 0 && threadIdx.x == 0) w.resets[chunk - 1] = reset;
}

template <int DT, int LPC>
__global__ __launch_bounds__(256, 2) void kda_ssm_bwd_kernel(SsmParams p, SsmWs w) {
  using TileT = Tile<LPC>;
  constexpr int CW = TileT::CW, EPT = TileT::EPT, EW = TileT::EW;
  __shared__ f32x2 s_d[BLK][CW];        // s, s x
  __shared__ float s_g[BLK][CW];
  __shared__ alignas(16) float s_b[BLK][EW], s_c[BLK][EW];
  __shared__ float s_o[3][SUB][CW];     // sums over e of B G, of A a h G, of C h
  __shared__ float s_r[4][SUB][2][EW];  // each wave's sums over channels of s x G and g h
  const Seqs seqs = seqs_of(p);
  const int tile = blockIdx.x % w.tiles, chunk = blockIdx.x / w.tiles;
  const TileT T(p, tile, w.per_group);
  const bool vec = (p.D / p.G) % EPT == 0 && p.D % EPT == 0;
  const int32_t t_lo = chunk * w.len, t_hi = p.tokens - t_lo < w.len ? p.tokens : t_lo + w.len;
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n) < t_hi ? seqs.begin(seqs.n) : t_hi;
  const int wave = threadIdx.x >> 6, lane = threadIdx.x & 63;
  float A[4], AL[4], G[4] = {0.0f, 0.0f, 0.0f, 0.0f}, dA[4] = {0.0f, 0.0f, 0.0f, 0.0f};
  T.load4(p, p.A, 0, A);
#pragma unroll
  for (int j = 0; j < 4; ++j) AL[j] = A[j] * LOG2E;
  if (chunk + 1 < w.chunks) T.load4(p, w.maps, chunk, G);
  float bias[EPT], skip[EPT], dskip[EPT], dbias[EPT];
  load_vec<EPT>(p.dt_bias, T.d0 + T.c0, T.cn, 0.0f, bias);
  load_vec<EPT>(p.skip, T.d0 + T.c0, T.cn, 0.0f, skip);
#pragma unroll
  for (int i = 0; i < EPT; ++i) dskip[i] = dbias[i] = 0.0f;
  SeqWalk q;
  for (int32_t t_blk = t_lo + (t_hi - t_lo - 1) / BLK * BLK; t_blk >= t_lo; t_blk -= BLK) {
    // everything of the block's tokens into shared memory
#pragma unroll 1
    for (int s = 0; s < BLK; s += SUB) {
      const int32_t tt = t_blk + s + T.row;
      const bool in = tt >= lo && tt < hi;
      const int c = in ? T.cn : 0;
      const size_t i0 = (size_t)tt * p.D + T.d0 + T.c0;
      float x[EPT], dt[EPT], z[EPT], dy[EPT];
      load_some<DT, EPT>(p.x, i0, c, vec, x);
      load_some<DT, EPT>(p.dt, i0, c, vec, dt);
      load_some<DT, EPT>(p.dy, i0, c, vec, dy);
      if (p.z) load_some<DT, EPT>(p.z, i0, c, vec, z);
      StageBC<DT, LPC, true, true> bc;
      bc.load(p, T.g, t_blk + s, lo, hi);
#pragma unroll
      for (int i = 0; i < EPT; ++i) {
        const float u = dt[i] + bias[i];
        const bool ok = in && i < T.cn;
        const float sp = ok ? (p.softplus ? softplus(u) : u) : 0.0f;
        s_d[s + T.row][T.c0 + i] = f32x2{sp, ok ? sp * x[i] : 0.0f};
        s_g[s + T.row][T.c0 + i] = ok ? gated(dy[i], z[i], p.z) : 0.0f;
      }
      bc.store(&s_b[s][0], &s_c[s][0]);
    }
    __syncthreads();
    // the state that enters each SUB tokens
    float h[4], in4[BLK / SUB][4];
    T.load4(p, p.carry, t_blk / BLK, h);
    q.start(seqs, t_blk);
    auto begins = [&](int32_t t) {   // token t, next in order, is a sequence's first
      if (t >= q.e) q.forward(seqs, t);
      if (t == q.b && q.holds(t)) T.load_state4(p, p.init, p.init_dtype, q.i, h);
    };
#pragma unroll 1
    for (int s = 0; s < BLK / SUB; ++s) {
      const int32_t t = t_blk + s * SUB;
#pragma unroll
      for (int k = 0; k < BLK / SUB; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) in4[k][j] = k == s || s == 0 ? h[j] : in4[k][j];
      if (s + 1 == BLK / SUB) break;
      auto sweep = [&](auto plain) {
#pragma unroll 4
        for (int r = 0; r < SUB; ++r) {
          if (!decltype(plain)::value) begins(t + r);
          const f32x2 d = s_d[s * SUB + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * SUB + r][T.e0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = fmaf(fast_exp2(d.x * AL[j]), h[j], d.y * b[j]);
        }
      };
      if (q.b < t && q.e >= t + SUB) sweep(std::true_type{});
      else sweep(std::false_type{});
    }
#pragma unroll 1
    for (int s = BLK / SUB - 1; s >= 0; --s) {
      const int32_t t = t_blk + s * SUB;
      if (t >= t_hi) continue;
      q.start(seqs, t);
      float hb[SUB][4], a[SUB][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) h[j] = s == 0 ? in4[0][j] : s == 1 ? in4[1][j] : s == 2 ? in4[2][j] : in4[3][j];
      auto sweep = [&](auto plain) {
        constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
        for (int r = 0; r < SUB; ++r) {
          if (!PLAIN) begins(t + r);
          const f32x2 d = s_d[s * SUB + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * SUB + r][T.e0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hb[r][j] = h[j];
            a[r][j] = fast_exp2(d.x * AL[j]);
            h[j] = fmaf(a[r][j], h[j], d.y * b[j]);
          }
        }
        if (!PLAIN) q.start(seqs, t + SUB - 1 < p.tokens ? t + SUB - 1 : p.tokens - 1);
#pragma unroll
        for (int r = SUB - 1; r >= 0; --r) {
          if (!PLAIN && t + r < t_hi) {
            if (t + r < q.b) q.back(seqs, t + r);
            if (p.dfin && t + r == q.e - 1 && q.holds(t + r)) {
              float f[4];
              T.load_state4(p, p.dfin, p.dfin_dtype, q.i, f);
#pragma unroll
              for (int j = 0; j < 4; ++j) G[j] += f[j];
            }
          }
          const f32x2 d = s_d[s * SUB + r][T.ch];
          const float g = s_g[s * SUB + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * SUB + r][T.e0]);
          const f32x4 c = *reinterpret_cast<const f32x4*>(&s_c[s * SUB + r][T.e0]);
          float bg = 0.0f, ahg = 0.0f, chs = 0.0f, v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            const float hj = fmaf(a[r][j], hb[r][j], d.y * b[j]);
            G[j] = fmaf(c[j], g, G[j]);
            bg = fmaf(b[j], G[j], bg);
            chs = fmaf(c[j], hj, chs);
            const float vb = d.y * G[j];
            G[j] *= a[r][j];
            const float ah = G[j] * hb[r][j];
            ahg = fmaf(A[j], ah, ahg);
            dA[j] = fmaf(d.x, ah, dA[j]);
            v[j] = halves32(vb, g * hj);
          }
          bg = part_sum<LPC>(bg);
          ahg = part_sum<LPC>(ahg);
          chs = part_sum<LPC>(chs);
          if (T.part < 3) s_o[T.part][r][T.ch] = T.part == 0 ? bg : T.part == 1 ? ahg : chs;
          // over channels: bit 5 of the lane B or C, bit 4 (and 3) the state, the rest of them summed
          const float u0 = halves16(v[0], v[1]), u1 = halves16(v[2], v[3]);
          if constexpr (LPC == 16) {
            float* to = &s_r[wave][r][lane >> 5][T.e0 + ((lane >> 4) & 1)];
            to[0] = u0;
            to[2] = u1;
          } else {
            const bool up = lane & 8;
            const float keep = up ? u1 : u0, give = up ? u0 : u1;
            float u = keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), 0x128, 0xf, 0xf, false));   // row_ror 8
            if constexpr (LPC == 4) u = xor4_add(u);
            if (LPC != 4 || !(lane & 4)) s_r[wave][r][lane >> 5][T.e0 + ((lane >> 4) & 1) + (up ? 2 : 0)] = u;
          }
          if (!PLAIN && t + r == q.b && q.holds(t + r)) {
            if (p.dinit && t + r < t_hi) T.store_state4(p, p.dinit, p.dinit_dtype, q.i, G);
#pragma unroll
            for (int j = 0; j < 4; ++j) G[j] = 0.0f;
          }
        }
      };
      if (q.b < t && q.e > t + SUB) sweep(std::true_type{});
      else sweep(std::false_type{});
      __syncthreads();
      // outputs of these tokens
      const int32_t tt = t + T.row;
      if (tt >= lo && tt < hi && T.cn > 0) {
        const size_t i0 = (size_t)tt * p.D + T.d0 + T.c0;
        float x[EPT], dt[EPT], z[EPT], dy[EPT], odx[EPT], odt[EPT], odz[EPT];
        load_some<DT, EPT>(p.x, i0, T.cn, vec, x);
        load_some<DT, EPT>(p.dt, i0, T.cn, vec, dt);
        if (p.dz) {
          load_some<DT, EPT>(p.z, i0, T.cn, vec, z);
          load_some<DT, EPT>(p.dy, i0, T.cn, vec, dy);
        }
#pragma unroll
        for (int i = 0; i < EPT; ++i) {
          const float g = s_g[s * SUB + T.row][T.c0 + i], sp = s_d[s * SUB + T.row][T.c0 + i].x;
          const float bg = s_o[0][T.row][T.c0 + i], ahg = s_o[1][T.row][T.c0 + i], ch = s_o[2][T.row][T.c0 + i];
          odx[i] = fmaf(skip[i], g, sp * bg);
          odt[i] = fmaf(x[i], bg, ahg);
          if (p.softplus) odt[i] *= sigmoid(dt[i] + bias[i]);
          if (p.dz) {
            const float sg = sigmoid(z[i]);
            odz[i] = dy[i] * fmaf(skip[i], x[i], ch) * (sg * fmaf(z[i], 1.0f - sg, 1.0f));
          }
          if (i < T.cn) {
            dskip[i] = fmaf(g, x[i], dskip[i]);
            dbias[i] += odt[i];
          }
        }
        store_some<DT, EPT>(p.dx, i0, T.cn, vec, odx);
        store_some<DT, EPT>(p.ddt, i0, T.cn, vec, odt);
        if (p.dz) store_some<DT, EPT>(p.dz, i0, T.cn, vec, odz);
      }
      for (int i = threadIdx.x; i < SUB * 2 * EW; i += 256) {
        const int r = i / (2 * EW), k = i % (2 * EW), e = k % EW;
        if (e < p.E && t + r < t_hi)
          w.bc[(((size_t)tile * p.tokens + t + r) * 2 + k / EW) * p.E + e] =
              (s_r[0][r][k / EW][e] + s_r[1][r][k / EW][e]) + (s_r[2][r][k / EW][e] + s_r[3][r][k / EW][e]);
      }
      __syncthreads();
    }
  }
  T.store4(p, w.dA, chunk, dA);
  // d_skip and d_bias over the 16 rows of lanes that load
#pragma unroll
  for (int i = 0; i < EPT; ++i) {
    s_o[0][T.row][T.c0 + i] = dskip[i];
    s_o[1][T.row][T.c0 + i] = dbias[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * CW; i += 256) {
    const int k = i / CW, c = i % CW;
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < SUB; ++r) v += s_o[k][r][c];
    if (c < T.dn) w.dvec[((size_t)chunk * 2 + k) * p.D + T.d0 + c] = v;
  }
}

// dB and dC: the sums over the workgroups of a group of channels
template <int DT>
__global__ __launch_bounds__(256) void kda_ssm_sum_bc_kernel(SsmParams p, SsmWs w) {
  const Seqs seqs = seqs_of(p);
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n);
  const int64_t row = 2 * (int64_t)p.E, n = (int64_t)p.tokens * row * p.G;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int g = (int)(i / (p.tokens * row));
    const int64_t j = i - g * (p.tokens * row), t = j / row, k = j - t * row;
    if (t < lo || t >= hi) continue;
    const float* in = w.bc + (size_t)g * w.per_group * p.tokens * row + j;
    float v = 0.0f;
#pragma unroll 8
    for (int c = 0; c < w.per_group; ++c) v += in[(size_t)c * p.tokens * row];
    const bool is_c = k >= p.E;
    store_f32<DT, 1>(is_c ? p.dC : p.dB, ((size_t)t * p.G + g) * p.E + (is_c ? k - p.E : k), &v);
  }
}

// dA, d_skip and d_bias: the sums over chunks
__global__ __launch_bounds__(256) void kda_ssm_sum_kernel(SsmParams p, SsmWs w, int chunks) {
  const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x, n = (int64_t)p.D * p.E;
  if (i >= n + 2 * (int64_t)p.D) return;
  const float* in = i < n ? w.dA + i : w.dvec + (i - n);
  const int64_t row = i < n ? n : 2 * (int64_t)p.D;
  float v = 0.0f;
#pragma unroll 8
  for (int c = 0; c < chunks; ++c) v += in[c * row];
  if (i < n) p.dA[i] = v;
  else if (i < n + p.D) {
    if (p.dskip) p.dskip[i - n] = v;
  } else if (p.dbias) {
    p.dbias[i - n - p.D] = v;
  }
}

// d_initial of sequences without tokens
__global__ __launch_bounds__(256) void kda_ssm_empty_kernel(SsmParams p) {
  const Seqs seqs = seqs_of(p);
  const int64_t n = (int64_t)p.D * p.E;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n * p.nseq; i += (int64_t)gridDim.x * 256) {
    const int s = (int)(i / n);
    if (seqs.begin(s) < seqs.begin(s + 1)) continue;
    float v;
    load_state<1>(p.dfin, p.dfin_dtype, i, &v);
    store_state<1>(p.dinit, p.dinit_dtype, i, &v);
  }
}

// ---- launches ---------------------------------------------------------------------

int lanes_of(int64_t E, bool backward) {
  return E <= 8 && !backward ? 2 : E <= 16 ? 4 : E <= 32 ? 8 : 16;
}

// Chunks of a multiple of BLK tokens: as many as give the GPU 4 workgroups a compute unit (waves
// hide each other's waits), 64 at most.
SsmWs shape_of(int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward) {
  SsmWs w{};
  const int64_t cw = 256 / lanes_of(E, backward), Dg = D / G;
  w.per_group = (int32_t)((Dg + cw - 1) / cw);
  w.tiles = (int32_t)(w.per_group * G);
  int64_t want = (1024 + w.tiles - 1) / w.tiles;
  if (want > 64) want = 64;
  const int64_t blocks = (tokens + BLK - 1) / BLK;
  int64_t len = (blocks + want - 1) / want;
  if (len < 1) len = 1;
  w.len = (int32_t)(len * BLK);
  w.chunks = (int32_t)((blocks + len - 1) / len);
  if (w.chunks < 1) w.chunks = 1;
  return w;
}

// The parts of a workspace, each aligned to 256 bytes; at: its start, or NULL for the size alone
size_t lay_out(SsmWs& w, uint8_t* at, int64_t tokens, int64_t D, int64_t E, bool backward) {
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = at ? at + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return r;
  };
  const size_t links = w.chunks - 1, states = (size_t)D * E * sizeof(float);
  w.maps = reinterpret_cast<float*>(take(links * states));
  w.sums = reinterpret_cast<float*>(take(links * D * sizeof(float)));
  w.resets = reinterpret_cast<int32_t*>(take(links * sizeof(int32_t)));
  if (!backward) {
    w.stage = reinterpret_cast<float*>(take(links * states));
  } else {
    w.dA = reinterpret_cast<float*>(take(w.chunks * states));
    w.dvec = reinterpret_cast<float*>(take((size_t)w.chunks * 2 * D * sizeof(float)));
    w.bc = reinterpret_cast<float*>(take((size_t)w.tiles * tokens * 2 * E * sizeof(float)));
  }
  return used;
}

template <int DT, typename F>
void by_lanes(int lpc, F f) {
  if (lpc == 2) f(integral_constant<int, 2>{});
  else if (lpc == 4) f(integral_constant<int, 4>{});
  else if (lpc == 8) f(integral_constant<int, 8>{});
  else f(integral_constant<int, 16>{});
}
template <typename F>
void by_dtype(int dt, F f) {
  if (dt == BF16) f(integral_constant<int, BF16>{});
  else if (dt == FP32) f(integral_constant<int, FP32>{});
  else f(integral_constant<int, FP16>{});
}
unsigned blocks_of(int64_t n, int64_t most) { return (unsigned)((n + 255) / 256 < most ? (n + 255) / 256 : most); }

}  // namespace

bool ssm_fits(int64_t tokens, int64_t D, int64_t E, int64_t G) {
  const SsmWs a = shape_of(tokens, D, E, G, false), b = shape_of(tokens, D, E, G, true);
  return (int64_t)a.tiles * a.chunks < INT32_MAX / 256 && (int64_t)b.tiles * b.chunks < INT32_MAX / 256;
}

size_t ssm_workspace(int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward) {
  SsmWs w = shape_of(tokens, D, E, G, backward);
  return lay_out(w, nullptr, tokens, D, E, backward);
}

hipError_t launch_ssm_fwd(const SsmParams& p, void* workspace, hipStream_t stream) {
  SsmWs w = shape_of(p.tokens, p.D, p.E, p.G, false);
  lay_out(w, static_cast<uint8_t*>(workspace), p.tokens, p.D, p.E, false);
  if (p.fin != p.init || !p.fin) w.stage = nullptr;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_lanes<DT>(lanes_of(p.E, false), [&](auto lpc) {
      constexpr int L = decltype(lpc)::value;
      if (w.chunks > 1) {
        hipLaunchKernelGGL((kda_ssm_fwd_kernel<DT, L, false>), dim3((unsigned)w.tiles * (w.chunks - 1)), dim3(256), 0, stream, p, w);
        hipLaunchKernelGGL(kda_ssm_pass_kernel<false>, dim3(blocks_of((int64_t)p.D * p.E, INT32_MAX)), dim3(256), 0, stream, p, w,
                           w.chunks - 1);
      }
      hipLaunchKernelGGL((kda_ssm_fwd_kernel<DT, L, true>), dim3((unsigned)w.tiles * w.chunks), dim3(256), 0, stream, p, w);
    });
  });
  return hipGetLastError();
}

hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream) {
  if (p.nseq == 0) return hipSuccess;
  const SsmWs w = shape_of(0, p.D, p.E, p.G, false);
  const int64_t rows = p.nseq < 65536 / w.tiles + 1 ? p.nseq : 65536 / w.tiles + 1;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_lanes<DT>(lanes_of(p.E, false), [&](auto lpc) {
      hipLaunchKernelGGL((kda_ssm_step_kernel<DT, decltype(lpc)::value>), dim3((unsigned)(rows * w.tiles)), dim3(256), 0, stream, p, w);
    });
  });
  return hipGetLastError();
}

hipError_t launch_ssm_bwd(const SsmParams& p, void* workspace, hipStream_t stream) {
  SsmWs w = shape_of(p.tokens, p.D, p.E, p.G, true);
  lay_out(w, static_cast<uint8_t*>(workspace), p.tokens, p.D, p.E, true);
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.tokens > 0) {
      auto go = [&](auto lpc) {
        constexpr int L = decltype(lpc)::value;
        if (w.chunks > 1) {
          hipLaunchKernelGGL((kda_ssm_bwd_map_kernel<DT, L>), dim3((unsigned)w.tiles * (w.chunks - 1)), dim3(256), 0, stream, p, w);
          hipLaunchKernelGGL(kda_ssm_pass_kernel<true>, dim3(blocks_of((int64_t)p.D * p.E, INT32_MAX)), dim3(256), 0, stream, p, w,
                             w.chunks - 1);
        }
        hipLaunchKernelGGL((kda_ssm_bwd_kernel<DT, L>), dim3((unsigned)w.tiles * w.chunks), dim3(256), 0, stream, p, w);
      };
      const int l = lanes_of(p.E, true);
      if (l == 4) go(integral_constant<int, 4>{});
      else if (l == 8) go(integral_constant<int, 8>{});
      else go(integral_constant<int, 16>{});
      hipLaunchKernelGGL(kda_ssm_sum_bc_kernel<DT>, dim3(blocks_of((int64_t)p.tokens * 2 * p.E * p.G, 16384)), dim3(256), 0, stream, p, w);
    }
  });
  hipLaunchKernelGGL(kda_ssm_sum_kernel, dim3(blocks_of((int64_t)p.D * (p.E + 2), INT32_MAX)), dim3(256), 0, stream, p, w,
                     p.tokens > 0 ? w.chunks : 0);
  if (p.dinit && (p.cu || p.T == 0))
    hipLaunchKernelGGL(kda_ssm_empty_kernel, dim3(blocks_of((int64_t)p.D * p.E * p.nseq, 16384)), dim3(256), 0, stream, p);
  return hipGetLastError();
}

}  // namespace kda
