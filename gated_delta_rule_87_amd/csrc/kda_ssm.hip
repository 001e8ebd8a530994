// kda_ssm.hip -- selective state space scan, forward, backward and single tokens (gfx950).
//
//     h_t[e] = exp(s_t A[e]) h_{t-1}[e] + s_t x_t B_t[e]
//     y_t = (sum_e C_t[e] h_t[e] + skip x_t) SiLU(z_t)
//
// per channel, s_t = softplus(dt_t + bias). Bound by the vector units: each of the T D E updates
// takes an exponential (8.4 cycles of a SIMD, measured) and four operations (2.6 to 3 each, with
// more than one wave; 4.4 where an operand is scalar or comes from another lane). At 8192 tokens x
// 8192 channels x 16 states, bf16, those alone are 140 us of the outputs' pass, where the memory
// traffic takes 105; it measures 320 us, and the pass before it 235.
//
// A sequence's tokens follow each other, so the packed tokens are cut into chunks until the GPU is
// filled. A chunk acts on the state entering it as h -> P h + R with P = exp(A sum s_t): one launch
// computes R and the sum of s of all chunks but the last, a second one passes the states from chunk
// to chunk, the third computes the outputs. (The exponentials are so taken twice; storing them
// would be 16 times the inputs.) A sequence's first token puts its initial state in the place of h;
// a chunk with one passes no state on (reset), whatever is before it.
//
// Backward, with g = dy SiLU(z): G_t = C_t g_t + exp(s_{t+1} A) G_{t+1} runs from the last token to
// the first, by chunks in the same manner. The states h are recomputed from those that the forward
// pass has saved every 64 tokens: once through the 64 for the state that enters every 8th, then 8
// tokens at a time, their states and decays in registers. The sums over channels (dB, dC) are
// halved from lane to lane with two values at once, added up over a workgroup, and over workgroups
// by a kernel after it, as the sums over chunks (dA, d_skip, d_bias) are. There the states of a
// channel are four to a lane, and what they share is computed by the lanes that load it and handed
// over in shared memory (8192 tokens x 4096 channels x 16 states 830 us, 35 operations an update).
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"
#include "kda_seq.h"

namespace kda {
namespace {

using std::integral_constant;

constexpr int SUB = 16;     // tokens that a workgroup stages at once
constexpr int RUN = 8;      // tokens whose states the backward pass holds in registers
constexpr int BLK = SSM_BLOCK;
static_assert(BLK == 8 * RUN && SUB == 2 * RUN, "");

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

// the same in every lane, and said so to the compiler
__device__ __forceinline__ size_t uniform(size_t v) {
  return (size_t)(uint32_t)__builtin_amdgcn_readfirstlane((int)(v >> 32)) << 32 |
         (uint32_t)__builtin_amdgcn_readfirstlane((int)v);
}

// v, of which the compiler does not know that it stays the same: an address formed of it is formed
// of a scalar base and 32 bits a lane, not kept in two registers a lane
__device__ __forceinline__ uint32_t hidden(uint32_t v) {
  asm volatile("" : "+v"(v));
  return v;
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

// ---- a workgroup's part of the channels, and its lanes' (single tokens, backward) -----
//
// LPC lanes a channel, four states each; E rounded up to 4 LPC.

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
  // past the caches (states of 256 sequences x 8192 channels x 16: a step 74 -> 70 us)
  __device__ __forceinline__ void store_past4(const SsmParams& p, void* a, int dtype, size_t row_, const float* h) const {
    if (ec != 4 || p.E % 4 != 0) {
      store_state4(p, a, dtype, row_, h);
    } else if (dtype == FP32) {
      __builtin_nontemporal_store(f32x4{h[0], h[1], h[2], h[3]}, reinterpret_cast<f32x4*>(static_cast<float*>(a) + at(p, row_)));
    } else {
      Pack<BF16, 4> q;
      q.pack(h);
      __builtin_nontemporal_store(q.r, reinterpret_cast<u32x2*>(static_cast<uint16_t*>(a) + at(p, row_)));
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

// ---- B and C in fp32 ----------------------------------------------------------------
//
// [G][tokens][2][EP]: B, then C, E rounded up to EP = 4 S with zeros, and zeros for tokens that no
// sequence covers (their values are not used, and may be NaN)
template <int DT>
__global__ __launch_bounds__(256) void kda_ssm_table_kernel(SsmParams p, float* table, int EP) {
  const Seqs seqs = seqs_of(p);
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n);
  const int64_t n = (int64_t)p.G * p.tokens * 2 * EP;
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < n; i += (int64_t)gridDim.x * 256) {
    const int e = (int)(i % EP);
    const int64_t r = i / EP;
    const bool is_c = r & 1;
    const int64_t gt = r >> 1, g = gt / p.tokens, t = gt - g * p.tokens;
    float v = 0.0f;
    if (e < p.E && t >= lo && t < hi) load_f32<DT, 1>(is_c ? p.Cm : p.Bm, ((size_t)t * p.G + g) * p.E + e, &v);
    table[i] = v;
  }
}

// ---- a wave's channels ----------------------------------------------------------------
//
// A wave takes 64 channels of one group, four to a quad of lanes. Lane p of a quad has the states
// S p .. S p + S - 1 of all four, and is besides the owner of channel p: it loads that channel's
// x, dt and z and computes what all its states share, which the other three take over by lane
// permutes. So B and C, the same for all channels, are read once for four channels' states. Lanes
// beyond the last channel work on that one too, so that nothing of the tokens needs a condition.
template <int S>
struct Quad {
  static constexpr int EP = 4 * S;
  int g, d0, dn;        // group, first channel, channels
  int lane, part, own;  // own: the lane's channel (the last one again beyond dn)
  int e0, ec;           // its states e0 .. e0 + ec - 1
  bool mine;            // owns a channel

  __device__ __forceinline__ Quad(const SsmParams& p, int tile, int per_group) {
    const int Dg = p.D / p.G;
    g = tile / per_group;
    const int at = (tile - g * per_group) * 64;
    d0 = g * Dg + at;
    dn = Dg - at < 64 ? Dg - at : 64;
    lane = threadIdx.x & 63;
    part = lane & 3;
    mine = lane < dn;
    own = d0 + (mine ? lane : dn - 1);
    e0 = S * part;
    ec = p.E - e0 < 0 ? 0 : p.E - e0 < S ? p.E - e0 : S;
  }
  __device__ __forceinline__ bool has(int c) const { return (lane & ~3) + c < dn; }
  __device__ __forceinline__ int channel(int c) const { return d0 + (has(c) ? (lane & ~3) + c : dn - 1); }
  // The lane's states of the quad's channels, of row `row` of [rows, D, E]: f(channel of the quad,
  // state, byte of the row, the lane's own offset) for V of them each
  template <int DT, bool ALL, typename F>
  __device__ __forceinline__ void each(const SsmParams& p, size_t row, F f) const {
    constexpr int V = S < 4 ? S : 4, SIZE = elem_size(DT);
    const bool whole = ec == S && p.E % 4 == 0;
    const size_t at = uniform(row * p.D * p.E * SIZE);
#pragma unroll
    for (int c = 0; c < 4; ++c) {
      if (!ALL && !has(c)) continue;
      const uint32_t off = hidden((uint32_t)(channel(c) * p.E + e0) * SIZE);
      if (whole) {
#pragma unroll
        for (int j = 0; j < S; j += V) f(integral_constant<int, V>{}, c, j, at + j * SIZE, off);
      } else {
#pragma unroll
        for (int j = 0; j < S; ++j)
          if (j < ec) f(integral_constant<int, 1>{}, c, j, at + j * SIZE, off);
      }
    }
  }
  template <int DT>
  __device__ __forceinline__ void load_as(const SsmParams& p, const void* a, size_t row, float (&h)[4][S]) const {
    each<DT, true>(p, row, [&](auto v, int c, int j, size_t at, uint32_t off) {
      Pack<DT, decltype(v)::value> q;
      q.load_at(a, at, off);
      q.unpack(&h[c][j]);
    });
  }
  template <int DT>
  __device__ __forceinline__ void store_as(const SsmParams& p, void* a, size_t row, const float (&h)[4][S]) const {
    each<DT, false>(p, row, [&](auto v, int c, int j, size_t at, uint32_t off) {
      Pack<DT, decltype(v)::value> q;
      q.pack(&h[c][j]);
      q.store_at(a, at, off);
    });
  }
  __device__ __forceinline__ void load(const SsmParams& p, const void* a, int dtype, size_t row, float (&h)[4][S]) const {
#pragma unroll
    for (int c = 0; c < 4; ++c)
#pragma unroll
      for (int j = 0; j < S; ++j) h[c][j] = 0.0f;
    if (dtype == FP32) load_as<FP32>(p, a, row, h);
    else if (dtype == BF16) load_as<BF16>(p, a, row, h);
  }
  __device__ __forceinline__ void store(const SsmParams& p, void* a, int dtype, size_t row, const float (&h)[4][S]) const {
    if (dtype == FP32) store_as<FP32>(p, a, row, h);
    else if (dtype == BF16) store_as<BF16>(p, a, row, h);
  }
};

// x of lane C of the quad
template <int C>
__device__ __forceinline__ float of_lane(float x) {
  int r = __builtin_amdgcn_mov_dpp(__float_as_int(x), C * 0x55, 0xf, 0xf, true);
  asm("" : "+v"(r));   // an instruction of its own: as an operand it halves the rate of each that uses it
  return __int_as_float(r);
}
template <int CTRL>
__device__ __forceinline__ float moved(float x) {
  return __int_as_float(__builtin_amdgcn_mov_dpp(__float_as_int(x), CTRL, 0xf, 0xf, true));
}
// v[p] summed over the quad, in lane p
__device__ __forceinline__ float quad_sums(const float (&v)[4], bool odd, bool high) {
  const float a = (odd ? v[1] : v[0]) + moved<0xB1>(odd ? v[0] : v[1]);
  const float b = (odd ? v[3] : v[2]) + moved<0xB1>(odd ? v[2] : v[3]);
  return (high ? b : a) + moved<0x4E>(high ? a : b);
}

// ROWS tokens' rows of the table in shared memory, two of them in turn; one wave, so no barriers
template <int S, int ROWS>
struct Rows {
  static constexpr int EP = 4 * S, N = ROWS * 2 * EP / 4, K = (N + 63) / 64;   // 16-byte pieces, of a lane
  f32x4 r[K];
  __device__ __forceinline__ void load(const float* table, int32_t t, int32_t end, int lane) {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = lane + 64 * k;
      r[k] = f32x4{0.0f, 0.0f, 0.0f, 0.0f};
      if (i < N && t + i * 4 / (2 * EP) < end) r[k] = *reinterpret_cast<const f32x4*>(table + (size_t)t * 2 * EP + i * 4);
    }
  }
  __device__ __forceinline__ void store(float* to, int lane) const {
#pragma unroll
    for (int k = 0; k < K; ++k) {
      const int i = lane + 64 * k;
      if (i < N) *reinterpret_cast<f32x4*>(to + i * 4) = r[k];
    }
  }
};
template <int S>
__device__ __forceinline__ void row_of(const float* s, float (&f)[S]) {
  if constexpr (S >= 4) {
#pragma unroll
    for (int j = 0; j < S; j += 4) {
      const f32x4 v = *reinterpret_cast<const f32x4*>(s + j);
#pragma unroll
      for (int k = 0; k < 4; ++k) f[j + k] = v[k];
    }
  } else if constexpr (S == 2) {
    const f32x2 v = *reinterpret_cast<const f32x2*>(s);
    f[0] = v[0];
    f[1] = v[1];
  } else {
    f[0] = *s;
  }
}

// ---- forward ----------------------------------------------------------------------

// h = exp(s A) h + w B for the channels of the quad; AL = A log2 e; y[c] += C . h where wanted
template <int S, bool Y>
__device__ __forceinline__ void advance(float (&h)[4][S], const float (&AL)[4][S], float s, float w, const float* b, const float* c,
                                        float (&y)[4]) {
  auto channel = [&](auto ch) {
    constexpr int N = decltype(ch)::value;
    const float sc = of_lane<N>(s), wc = of_lane<N>(w);
#pragma unroll
    for (int j = 0; j < S; ++j) {
      h[N][j] = fmaf(fast_exp2(sc * AL[N][j]), h[N][j], wc * b[j]);
      if (Y) y[N] = j == 0 ? c[0] * h[N][0] : fmaf(c[j], h[N][j], y[N]);
    }
  };
  channel(integral_constant<int, 0>{});
  channel(integral_constant<int, 1>{});
  channel(integral_constant<int, 2>{});
  channel(integral_constant<int, 3>{});
}

// Tokens loaded at once, and waves to a SIMD that the registers are to leave room for
constexpr int FSUB = 4;
constexpr int waves_of(int S) { return S >= 16 ? 1 : S >= 8 ? 2 : 4; }

// FINAL: the outputs; else the chunk's map. A workgroup is one wave.
template <int DT, int S, bool FINAL>
__global__ __launch_bounds__(64, waves_of(S)) void kda_ssm_fwd_kernel(SsmParams p, SsmWs w) {
  constexpr int EP = 4 * S;
  __shared__ alignas(16) float s_bc[2][FSUB][2][EP];
  __shared__ float s_own[3][FSUB][64];   // x, dt, z where tokens are taken one by one
  const Seqs seqs = seqs_of(p);
  const int tile = blockIdx.x % w.tiles, chunk = blockIdx.x / w.tiles;
  const Quad<S> T(p, tile, w.per_group);
  const int32_t t_lo = chunk * w.len, t_hi = p.tokens - t_lo < w.len ? p.tokens : t_lo + w.len;
  const int32_t lo = seqs.begin(0), hi = seqs.begin(seqs.n) < t_hi ? seqs.begin(seqs.n) : t_hi;
  const float* table = w.table + (size_t)T.g * p.tokens * 2 * EP;
  const bool odd = T.lane & 1, high = T.lane & 2;
  float AL[4][S], h[4][S], sum = 0.0f;
  T.load(p, p.A, FP32, 0, AL);
#pragma unroll
  for (int c = 0; c < 4; ++c)
#pragma unroll
    for (int j = 0; j < S; ++j) {
      AL[c][j] *= LOG2E;
      h[c][j] = 0.0f;
    }
  const float bias = p.dt_bias ? p.dt_bias[T.own] : 0.0f, skip = FINAL && p.skip ? p.skip[T.own] : 0.0f;
  if (FINAL && chunk > 0) T.load(p, w.maps, FP32, chunk - 1, h);
  bool reset = false;

  const uint32_t off = (uint32_t)T.own * elem_size(DT);
  const size_t line = (size_t)p.D * elem_size(DT);
  Pack<DT, 1> x[FSUB], d[FSUB], z[FSUB];   // of the next FSUB tokens: each is loaded as soon as the one before has been used
  Rows<S, FSUB> rows;
  auto load = [&](int r, int32_t t) {   // (tokens beyond the covered ones are read as the last of them and not used)
    const size_t at = uniform((t < lo ? lo : t < hi ? t : hi - 1) * line);
    const uint32_t o = hidden(off);
    x[r].load_at(p.x, at, o);
    d[r].load_at(p.dt, at, o);
    if (FINAL) z[r].load_at(p.z ? p.z : p.x, at, o);
  };
  SeqWalk q;
  q.start(seqs, t_lo);
  const bool any = t_lo < hi && t_hi > lo;   // tokens of a sequence
  if (any) {
#pragma unroll
    for (int r = 0; r < FSUB; ++r) load(r, t_lo + r);
    rows.load(table, t_lo, t_hi, T.lane);
    rows.store(&s_bc[0][0][0][0], T.lane);
  }
  int buf = 0;
  for (int32_t t = t_lo; any && t < t_hi; t += FSUB, buf ^= 1) {
    if (t + FSUB < t_hi) rows.load(table, t + FSUB, t_hi, T.lane);
    if (FINAL && p.carry && t % BLK == 0) T.store(p, p.carry, FP32, t / BLK, h);
    // one token; in: it belongs to a sequence (others leave the state as it is)
    auto step = [&](int r, bool in, float xv, float dv, float zv) {
      float b[S], c[S], y[4];
      row_of<S>(&s_bc[buf][r][0][T.e0], b);
      if (FINAL) row_of<S>(&s_bc[buf][r][1][T.e0], c);
      const float u = dv + bias;
      const float sp = softplus(u);   // (selects, no branches: they would cut up the code of a token)
      const float s = !in ? 0.0f : p.softplus ? sp : u, v = in ? s * xv : 0.0f;
      advance<S, FINAL>(h, AL, s, v, b, c, y);
      if (!FINAL) sum += s;
      if (FINAL) {
        float out = fmaf(skip, xv, quad_sums(y, odd, high));
        const float gate = zv * sigmoid(zv);
        out *= p.z ? gate : 1.0f;
        Pack<DT, 1> o;
        o.pack(&out);
        if (in) o.store_at(p.y, uniform((t + r) * line), hidden(off));
      }
    };
    if (q.b < t && q.e > t + FSUB) {   // no sequence begins or ends here
#pragma unroll
      for (int r = 0; r < FSUB; ++r) {
        float xv, dv, zv;
        x[r].unpack(&xv);
        d[r].unpack(&dv);
        z[r].unpack(&zv);
        load(r, t + FSUB + r);
        step(r, true, xv, dv, zv);
        __builtin_amdgcn_sched_barrier(0);   // (more tokens at once would only take registers)
      }
    } else {
#pragma unroll
      for (int r = 0; r < FSUB; ++r) {
        x[r].unpack(&s_own[0][r][T.lane]);
        d[r].unpack(&s_own[1][r][T.lane]);
        z[r].unpack(&s_own[2][r][T.lane]);
        load(r, t + FSUB + r);
      }
#pragma unroll 1
      for (int r = 0; r < FSUB && t + r < t_hi; ++r) {
        if (t + r >= q.e) q.forward(seqs, t + r);
        const bool in = q.holds(t + r);
        if (t + r == q.b && in) {
          // the last sequence that goes on after this chunk has its final state written elsewhere,
          // perhaps over its initial state: that is put aside
          const bool goes_on = w.stage && q.e > t_hi;
          if (FINAL && goes_on) T.load(p, w.stage, FP32, chunk, h);
          else T.load(p, p.init, p.init_dtype, q.i, h);
          if (!FINAL && goes_on) T.store(p, w.stage, FP32, chunk, h);
          reset = true;
        }
        step(r, in, s_own[0][r][T.lane], s_own[1][r][T.lane], s_own[2][r][T.lane]);
        if (FINAL && p.fin && t + r == q.e - 1 && in) T.store(p, p.fin, p.fin_dtype, q.i, h);
      }
    }
    if (t + FSUB < t_hi) rows.store(&s_bc[buf ^ 1][0][0][0], T.lane);
  }
  if (FINAL) {   // sequences without tokens
    if (p.fin)
      for (int n = chunk; n < p.nseq; n += w.chunks)
        if (seqs.begin(n) >= seqs.begin(n + 1)) {
          T.load(p, p.init, p.init_dtype, n, h);
          T.store(p, p.fin, p.fin_dtype, n, h);
        }
  } else {
    T.store(p, w.maps, FP32, chunk, h);
    if (T.mine) w.sums[(size_t)chunk * p.D + T.own] = sum;
    if (tile == 0 && threadIdx.x == 0) w.resets[chunk] = reset;
  }
}

// 2^e h + r. A chunk's decay can be beyond fp32 (A > 0, or s < 0) where its product with h is not, or
// where h is 0, as behind zeros of padding: then the exponent's whole part is applied to the product.
__device__ __forceinline__ float passed_on(float e, float h, float r) {
  if (e > 64.0f && e < INFINITY) {
    const float n = __builtin_rintf(e);
    return __builtin_ldexpf(fast_exp2(e - n) * h, n < 1024.0f ? (int)n : 1024) + r;
  }
  return fmaf(fast_exp2(e), h, r);
}

// maps[c] becomes the state that leaves chunk c (BACK: the gradient that leaves chunk c + 1 towards
// its first token). 32 states of channels to a workgroup, 8 lanes each: a lane joins the maps of an
// eighth of the chunks, takes the state that enters them from the lanes before it, and runs through
// its chunks again. (One lane for all of them: 19 us for 256 chunks of 16384 states.)
template <bool BACK>
__global__ __launch_bounds__(256) void kda_ssm_pass_kernel(SsmParams p, SsmWs w, int count) {
  __shared__ float s_r[8][32], s_s[8][32];
  __shared__ bool s_reset[8];
  const int j = threadIdx.x & 31, part = threadIdx.x >> 5;
  const int64_t n = (int64_t)p.D * p.E, at = (int64_t)blockIdx.x * 32 + j, i = at < n ? at : n - 1;
  const int64_t d = i / p.E;
  const float A = p.A[i] * LOG2E;
  const int each = (count + 7) / 8, c0 = part * each, c1 = count < c0 + each ? count : c0 + each;
  auto chunk = [&](int c) { return BACK ? count - 1 - c : c; };
  auto run = [&](float h, bool first, auto put) {   // first: nothing enters
    constexpr int AHEAD = 8;
    for (int c = c0; c < c1; c += AHEAD) {
      float r[AHEAD], s[AHEAD];
      int reset[AHEAD];
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        const int at_c = chunk(c + k < c1 ? c + k : c1 - 1);
        r[k] = w.maps[at_c * n + i];
        s[k] = w.sums[(int64_t)at_c * p.D + d];
        reset[k] = w.resets[at_c];
      }
#pragma unroll
      for (int k = 0; k < AHEAD; ++k) {
        if (c + k >= c1) break;
        h = first || reset[k] ? r[k] : passed_on(A * s[k], h, r[k]);
        first = false;
        put(c + k, h, s[k], reset[k] != 0);
      }
    }
    return h;
  };
  float sum = 0.0f;
  bool any = false;
  const float r = run(0.0f, true, [&](int, float, float s, bool reset) {
    sum += s;
    any = any || reset;
  });
  s_r[part][j] = r;
  s_s[part][j] = sum;
  if (j == 0) s_reset[part] = any;
  __syncthreads();
  float h = 0.0f;
  for (int k = 0; k < part; ++k)
    if (k * each < count) h = k == 0 || s_reset[k] ? s_r[k][j] : passed_on(A * s_s[k][j], h, s_r[k][j]);
  run(h, part == 0, [&](int c, float v, float, bool) {
    if (at < n) w.maps[chunk(c) * n + i] = v;
  });
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
    float h[4] = {0.0f, 0.0f, 0.0f, 0.0f}, b[4] = {}, c[4] = {}, x, dt, z = 0.0f, y = 0.0f;
    if (from >= 0 && from < p.n_slots) T.load_state4(p, p.init, p.init_dtype, from, h);
    load_f32<DT, 1>(p.x, i, &x);
    load_f32<DT, 1>(p.dt, i, &dt);
    if (p.z) load_f32<DT, 1>(p.z, i, &z);
    if (T.ec == 4 && p.E % 4 == 0) {
      load_f32<DT, 4>(p.Bm, bc, b);
      load_f32<DT, 4>(p.Cm, bc, c);
    } else {
#pragma unroll
      for (int j = 0; j < 4; ++j)
        if (j < T.ec) {
          load_f32<DT, 1>(p.Bm, bc + j, b + j);
          load_f32<DT, 1>(p.Cm, bc + j, c + j);
        }
    }
    const float s = p.softplus ? softplus(dt + bias) : dt + bias;
#pragma unroll
    for (int j = 0; j < 4; ++j) {
      h[j] = fmaf(fast_exp2(s * A[j] * LOG2E), h[j], s * x * b[j]);
      y = fmaf(c[j], h[j], y);
    }
    if (to >= 0 && to < p.n_slots) T.store_past4(p, p.fin, p.fin_dtype, to, h);
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
  __shared__ float s_o[3][SUB * CW + 16];   // sums over e of B G, of A a h G, of C h (16: other banks)
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
    // the state that enters each RUN tokens
    float h[4], in4[BLK / RUN][4];
    T.load4(p, p.carry, t_blk / BLK, h);
    q.start(seqs, t_blk);
    auto begins = [&](int32_t t) {   // before token t, next in order
      if (t >= q.e) q.forward(seqs, t);
      if (!q.holds(t)) h[0] = h[1] = h[2] = h[3] = 0.0f;   // (of no sequence: nothing was saved there)
      else if (t == q.b) T.load_state4(p, p.init, p.init_dtype, q.i, h);
    };
#pragma unroll 1
    for (int s = 0; s < BLK / RUN; ++s) {
      const int32_t t = t_blk + s * RUN;
#pragma unroll
      for (int k = 0; k < BLK / RUN; ++k)
#pragma unroll
        for (int j = 0; j < 4; ++j) in4[k][j] = k == s || s == 0 ? h[j] : in4[k][j];
      if (s + 1 == BLK / RUN) break;
      auto sweep = [&](auto plain) {
#pragma unroll 4
        for (int r = 0; r < RUN; ++r) {
          if (!decltype(plain)::value) begins(t + r);
          const f32x2 d = s_d[s * RUN + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * RUN + r][T.e0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) h[j] = fmaf(fast_exp2(d.x * AL[j]), h[j], d.y * b[j]);
        }
      };
      if (q.b < t && q.e >= t + RUN) sweep(std::true_type{});
      else sweep(std::false_type{});
    }
#pragma unroll 1
    for (int s = BLK / RUN - 1; s >= 0; --s) {
      const int32_t t = t_blk + s * RUN;
      if (t >= t_hi) continue;
      const int at0 = (s & 1) * RUN;   // two runs share what follows
      q.start(seqs, t);
      float hb[RUN][4], a[RUN][4];
#pragma unroll
      for (int j = 0; j < 4; ++j) {
        h[j] = in4[0][j];
#pragma unroll
        for (int k = 1; k < BLK / RUN; ++k) h[j] = s == k ? in4[k][j] : h[j];
      }
      auto sweep = [&](auto plain) {
        constexpr bool PLAIN = decltype(plain)::value;
#pragma unroll
        for (int r = 0; r < RUN; ++r) {
          if (!PLAIN) begins(t + r);
          const f32x2 d = s_d[s * RUN + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * RUN + r][T.e0]);
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            hb[r][j] = h[j];
            a[r][j] = fast_exp2(d.x * AL[j]);
            h[j] = fmaf(a[r][j], h[j], d.y * b[j]);
          }
        }
        if (!PLAIN) q.start(seqs, t + RUN - 1 < p.tokens ? t + RUN - 1 : p.tokens - 1);
#pragma unroll
        for (int r = RUN - 1; r >= 0; --r) {
          if (!PLAIN && t + r < t_hi) {
            if (t + r < q.b) q.back(seqs, t + r);
            if (p.dfin && t + r == q.e - 1 && q.holds(t + r)) {
              float f[4];
              T.load_state4(p, p.dfin, p.dfin_dtype, q.i, f);
#pragma unroll
              for (int j = 0; j < 4; ++j) G[j] += f[j];
            }
          }
          const f32x2 d = s_d[s * RUN + r][T.ch];
          const float g = s_g[s * RUN + r][T.ch];
          const f32x4 b = *reinterpret_cast<const f32x4*>(&s_b[s * RUN + r][T.e0]);
          const f32x4 c = *reinterpret_cast<const f32x4*>(&s_c[s * RUN + r][T.e0]);
          float bg = 0.0f, ahg = 0.0f, chs = 0.0f, v[4];
#pragma unroll
          for (int j = 0; j < 4; ++j) {
            // (where no sequence begins the state after a token is the one before the next)
            const float hj = !PLAIN ? fmaf(a[r][j], hb[r][j], d.y * b[j]) : r + 1 < RUN ? hb[r + 1 < RUN ? r + 1 : 0][j] : h[j];
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
          if (T.part < 3) s_o[T.part][(at0 + r) * CW + T.ch] = T.part == 0 ? bg : T.part == 1 ? ahg : chs;
          // over channels: bit 5 of the lane B or C, bit 4 (and 3) the state, the rest of them summed
          const float u0 = halves16(v[0], v[1]), u1 = halves16(v[2], v[3]);
          if constexpr (LPC == 16) {
            float* to = &s_r[wave][at0 + r][lane >> 5][T.e0 + ((lane >> 4) & 1)];
            to[0] = u0;
            to[2] = u1;
          } else {
            const bool up = lane & 8;
            const float keep = up ? u1 : u0, give = up ? u0 : u1;
            float u = keep + __int_as_float(__builtin_amdgcn_update_dpp(0, __float_as_int(give), 0x128, 0xf, 0xf, false));   // row_ror 8
            if constexpr (LPC == 4) u = xor4_add(u);
            if (LPC != 4 || !(lane & 4)) s_r[wave][at0 + r][lane >> 5][T.e0 + ((lane >> 4) & 1) + (up ? 2 : 0)] = u;
          }
          if (!PLAIN && t + r == q.b && q.holds(t + r)) {
            if (p.dinit && t + r < t_hi) T.store_state4(p, p.dinit, p.dinit_dtype, q.i, G);
#pragma unroll
            for (int j = 0; j < 4; ++j) G[j] = 0.0f;
          }
        }
      };
      if (q.b < t && q.e > t + RUN) sweep(std::true_type{});
      else sweep(std::false_type{});
      if (s & 1) continue;
      __syncthreads();
      // outputs of these SUB tokens
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
          const float g = s_g[s * RUN + T.row][T.c0 + i], sp = s_d[s * RUN + T.row][T.c0 + i].x;
          const float bg = s_o[0][T.row * CW + T.c0 + i], ahg = s_o[1][T.row * CW + T.c0 + i], ch = s_o[2][T.row * CW + T.c0 + i];
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
    s_o[0][T.row * CW + T.c0 + i] = dskip[i];
    s_o[1][T.row * CW + T.c0 + i] = dbias[i];
  }
  __syncthreads();
  for (int i = threadIdx.x; i < 2 * CW; i += 256) {
    const int k = i / CW, c = i % CW;
    float v = 0.0f;
#pragma unroll
    for (int r = 0; r < SUB; ++r) v += s_o[k][r * CW + c];
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
int states_of(int64_t E) { return E <= 4 ? 1 : E <= 8 ? 2 : E <= 16 ? 4 : E <= 32 ? 8 : 16; }

// Chunks of a multiple of BLK tokens: as many as give the GPU enough waves to hide each other's
// waits (forward four to a SIMD, backward workgroups of four of them, 8 to a compute unit).
SsmWs shape_of(int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward) {
  SsmWs w{};
  const int64_t cw = backward ? 256 / lanes_of(E, true) : 64, Dg = D / G;
  w.per_group = (int32_t)((Dg + cw - 1) / cw);
  w.tiles = (int32_t)(w.per_group * G);
  const int64_t fill = backward ? 2048 : 4096, most = backward ? 128 : 256;
  int64_t want = (fill + w.tiles - 1) / w.tiles;
  if (want > most) want = most;
  const int64_t blocks = (tokens + BLK - 1) / BLK;
  int64_t len = (blocks + want - 1) / want;
  if (len < 1) len = 1;
  w.len = (int32_t)(len * BLK);
  w.chunks = (int32_t)((blocks + len - 1) / len);
  if (w.chunks < 1) w.chunks = 1;
  w.most = (int32_t)(blocks < 1 ? 1 : blocks < want ? blocks : want);
  return w;
}

// The parts of a workspace, each aligned to 256 bytes; at: its start, or NULL for the size alone
size_t lay_out(SsmWs& w, uint8_t* at, int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward) {
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
    w.table = reinterpret_cast<float*>(take((size_t)G * tokens * 2 * 4 * states_of(E) * sizeof(float)));
  } else {
    w.dA = reinterpret_cast<float*>(take(w.chunks * states));
    w.dvec = reinterpret_cast<float*>(take((size_t)w.chunks * 2 * D * sizeof(float)));
    w.bc = reinterpret_cast<float*>(take((size_t)w.tiles * tokens * 2 * E * sizeof(float)));
  }
  return used;
}

template <typename F>
void by_states(int S, F f) {
  if (S == 1) f(integral_constant<int, 1>{});
  else if (S == 2) f(integral_constant<int, 2>{});
  else if (S == 4) f(integral_constant<int, 4>{});
  else if (S == 8) f(integral_constant<int, 8>{});
  else f(integral_constant<int, 16>{});
}
template <typename F>
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

// Room for what any call of at most so many tokens takes (chunks are whole blocks: fewer tokens can
// have more of them)
size_t ssm_workspace(int64_t tokens, int64_t D, int64_t E, int64_t G, bool backward) {
  SsmWs w = shape_of(tokens, D, E, G, backward);
  w.chunks = w.most;
  return lay_out(w, nullptr, tokens, D, E, G, backward);
}

hipError_t launch_ssm_fwd(const SsmParams& p, void* workspace, hipStream_t stream) {
  SsmWs w = shape_of(p.tokens, p.D, p.E, p.G, false);
  lay_out(w, static_cast<uint8_t*>(workspace), p.tokens, p.D, p.E, p.G, false);
  if (p.fin != p.init || !p.fin) w.stage = nullptr;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_states(states_of(p.E), [&](auto states) {
      constexpr int S = decltype(states)::value;
      if (p.tokens > 0)
        hipLaunchKernelGGL(kda_ssm_table_kernel<DT>, dim3(blocks_of((int64_t)p.G * p.tokens * 8 * S, 4096)), dim3(256), 0, stream, p,
                           w.table, 4 * S);
      if (w.chunks > 1) {
        hipLaunchKernelGGL((kda_ssm_fwd_kernel<DT, S, false>), dim3((unsigned)w.tiles * (w.chunks - 1)), dim3(64), 0, stream, p, w);
        hipLaunchKernelGGL(kda_ssm_pass_kernel<false>, dim3((unsigned)(((int64_t)p.D * p.E + 31) / 32)), dim3(256), 0, stream, p, w,
                           w.chunks - 1);
      }
      hipLaunchKernelGGL((kda_ssm_fwd_kernel<DT, S, true>), dim3((unsigned)w.tiles * w.chunks), dim3(64), 0, stream, p, w);
    });
  });
  return hipGetLastError();
}

hipError_t launch_ssm_step(const SsmParams& p, hipStream_t stream) {
  if (p.nseq == 0) return hipSuccess;
  SsmWs w{};
  const int cw = 256 / lanes_of(p.E, false);
  w.per_group = (p.D / p.G + cw - 1) / cw;
  w.tiles = w.per_group * p.G;
  // Sequences at once; the others in turn, so that A is loaded once for some (16384 workgroups 69 us
  // at 256 sequences of 8192 channels, 4096 71, one for each sequence 80).
  const int64_t most = 16384 / w.tiles + 1, rows = p.nseq < most ? p.nseq : most;
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    by_lanes(lanes_of(p.E, false), [&](auto lpc) {
      hipLaunchKernelGGL((kda_ssm_step_kernel<DT, decltype(lpc)::value>), dim3((unsigned)(rows * w.tiles)), dim3(256), 0, stream, p, w);
    });
  });
  return hipGetLastError();
}

hipError_t launch_ssm_bwd(const SsmParams& p, void* workspace, hipStream_t stream) {
  SsmWs w = shape_of(p.tokens, p.D, p.E, p.G, true);
  lay_out(w, static_cast<uint8_t*>(workspace), p.tokens, p.D, p.E, p.G, true);
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (p.tokens > 0) {
      auto go = [&](auto lpc) {
        constexpr int L = decltype(lpc)::value;
        if (w.chunks > 1) {
          hipLaunchKernelGGL((kda_ssm_bwd_map_kernel<DT, L>), dim3((unsigned)w.tiles * (w.chunks - 1)), dim3(256), 0, stream, p, w);
          hipLaunchKernelGGL(kda_ssm_pass_kernel<true>, dim3((unsigned)(((int64_t)p.D * p.E + 31) / 32)), dim3(256), 0, stream, p, w,
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
