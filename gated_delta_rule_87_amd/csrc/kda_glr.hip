// kda_glr.hip -- gated linear recurrence h_t = exp(g_t) h_{t-1} + x_t per channel, forward
// and backward (gfx950).
//
// The B * T packed tokens are cut into tiles of GLR_TILE tokens by 256 bytes of channels, one
// workgroup each. A tile acts on the state that enters it as an affine map h -> A h + L, with
// A = prod exp(g): the workgroup loads its tile once into registers, reduces it to (A, L) per
// channel, publishes that, obtains the state that enters it from the tiles before, and runs
// through its registers a second time for the outputs. So every element is read once and
// written once, also for few channels on long sequences, where one lane per channel would leave
// most of the GPU idle (8192 x 8192 bf16 so: 3.59 ms forward). Bound by memory: at that size
// forward 83 us (5.0 TB/s), backward 133 us (5.2 TB/s) after a forward pass.
//
// Inside a tile, 16 groups of 16 lanes hold R = 8 consecutive tokens each, 16 bytes a lane and
// token (rows that are no whole vectors: at any address, the last elements in smaller pieces);
// their maps are composed through shared memory. 8 tokens of three tensors are 96 registers a
// lane backward, as many as three workgroups a compute unit can hold. A sequence's first token
// sets the state instead of continuing it: A = RESET (-1; an exp is never negative) marks a map
// that does not depend on the state before, which is then not multiplied by zero but left out
// (it may be NaN).
//
// A decay of zero is such a start as well: zero times an infinite or NaN state would be NaN.
// (Gates below -87.4 have one: the instruction for 2^x gives zero below 2^-126.) Every other
// decay is above zero, and so has to be every product of them, or an infinite state would become
// NaN where tiles are joined: products are kept at FAINT, the smallest number, or above. Only
// waves that find a zero among their decays, or among the products over 8 tokens, take the
// paths that look at each decay.
//
// Between tiles: every tile publishes its map; the last of BLOCK tiles also their composition,
// the block's map, and the state that leaves the block. A tile takes the maps of the tiles
// before it in its block, and the state that enters the block: as published, or, looking back
// over up to WINDOW blocks, from an earlier block's state and the maps of the blocks between.
// (Passing a state from tile to tile over 7 of them at once, 32768 tokens of 256 channels took
// 47 us: many tiles in flight and little data.) A block's state is always its map applied to the
// state before it, and a tile's its block's map so far applied to that, whoever computes it, so
// the bits do not depend on how far a tile looked back. Each word is EMPTY (all ones) until it
// is published, as a single relaxed atomic of device scope: no fences, no flags beside the data;
// a NaN is stored as one whose bits are not EMPTY.
//
// Every wait ends: a workgroup takes its tile's number from a counter of its channels when it
// starts, so all tiles that it waits for belong to workgroups that have started before it and
// which themselves wait only for earlier ones; the first waits for none. Only another call in
// the same workspace could break that; so a wait also ends, with NaN, after a number of polls
// (seconds), and for all workgroups of its channels once it has ended so for one.
#include <cstdlib>
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

constexpr float RESET = -1.0f;
constexpr uint32_t EMPTY = 0xffffffffu;
constexpr int BLOCK = 8;    // tiles of a block
constexpr int WINDOW = 6;   // blocks looked back over at once
constexpr int TICK_STRIDE = 16;   // a counter per 64 bytes

constexpr int LR = 16;             // lanes across a row
constexpr int GRP = 256 / LR;      // groups of lanes along the tokens
constexpr int R = GLR_TILE / GRP;  // tokens of a lane
template <int DT>
struct Geom {
  static constexpr int VEC = 16 / elem_size(DT);   // elements of a lane
  static constexpr int CH = LR * VEC;              // channels of a tile
};

constexpr float FAINT = 0x1p-149f;

__device__ __forceinline__ float decay(float g) { return fast_exp2(g * LOG2E); }
// a h + x, for a decay of zero x alone
__device__ __forceinline__ float follow(float a, float h, float x) { return a == 0.0f ? x : fmaf(a, h, x); }
// the map (A, L) on a state
__device__ __forceinline__ float apply(float A, float L, float h) { return A < 0.0f ? L : fmaf(A, h, L); }
// the A of a map followed by the decay a >= 0, and by another map's (fmaxf drops a NaN, but then
// L is NaN)
__device__ __forceinline__ float lasting(float A, float a) {
  return A < 0.0f || a == 0.0f ? RESET : fmaxf(A * a, FAINT);
}
// (A, L) followed by (a, l)
__device__ __forceinline__ void compose(float& A, float& L, float a, float l) {
  L = apply(a, l, L);
  A = a < 0.0f || A < 0.0f ? RESET : fmaxf(A * a, FAINT);
}

__device__ __forceinline__ uint32_t word_of(float f) { return f != f ? 0x7fc00000u : __float_as_uint(f); }
template <typename T>
__device__ __forceinline__ void publish(T* p, T v) {
  __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ __forceinline__ T observe(const T* p) {
  return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

struct TileWs {
  uint64_t* maps;           // [tiles][D] (L, A) of each tile, by the order of processing
  uint64_t* block_maps;     // [blocks][D] of each whole block of BLOCK tiles
  uint32_t* block_states;   // [blocks][D] state entering each block
  uint32_t* ticks;          // [channel tiles * TICK_STRIDE] next tile of the channels, whether a wait was given up
  uint32_t polls;           // of a wait, at most
  float* stage;             // [nseq][D] initial states, where final_state overwrites them
  int32_t tiles, cols;
};

__device__ __forceinline__ float map_A(uint64_t m) { return __uint_as_float((uint32_t)m); }
__device__ __forceinline__ float map_L(uint64_t m) { return __uint_as_float((uint32_t)(m >> 32)); }
__device__ __forceinline__ uint64_t map_word(float A, float L) { return ((uint64_t)word_of(L) << 32) | __float_as_uint(A); }

// 32-bit words of all maps and states
__host__ __device__ inline int64_t glr_words(int64_t tiles, int64_t D) {
  return (2 * tiles + 3 * ((tiles + BLOCK - 1) / BLOCK)) * D;
}

// Publishes the tile's map, waits for the state that enters it, and, for the last tile of a
// block, publishes the block's map and the state that leaves it; k: the tile's place in the
// order of processing, c0 + ch: the lane's channel. Addresses are formed anew at every poll (t
// is opaque): kept over the loops they cost 30 registers.
__device__ __forceinline__ float pass_state(const TileWs& w, int k, int32_t D, int c0, uint32_t ch, uint32_t* stop, float A,
                                            float L) {
  auto row = [&](int i) { return (size_t)i * D + c0; };
  uint32_t left = w.polls;
  auto give_up = [&]() {   // after a poll that did not find everything
    if (left == 0 || (left % 1024 == 0 && observe(stop) != 0)) {
      publish(stop, 1u);
      return true;
    }
    --left;
    __builtin_amdgcn_s_sleep(1);
    return false;
  };
  const int b = k / BLOCK, j = k % BLOCK;
  const bool more = k + 1 < w.tiles, closes = more && j == BLOCK - 1;
  if (more && !closes) publish(w.maps + row(k) + ch, map_word(A, L));
  uint64_t m[BLOCK - 1];   // maps of the block's tiles before this one
#pragma unroll
  for (int i = 0; i < BLOCK - 1; ++i) m[i] = 0;
  for (bool whole = j == 0; !whole;) {
    int t = b * BLOCK;
    asm volatile("" : "+s"(t));
#pragma unroll
    for (int i = 0; i < BLOCK - 1; ++i)
      if (i < j) m[i] = observe(w.maps + row(t + i) + ch);
    whole = true;
#pragma unroll
    for (int i = 0; i < BLOCK - 1; ++i) whole = whole && m[i] != ~0ull;
    if (!whole && give_up()) break;   // (a map that is not there is NaN)
  }
  float BA = 1.0f, BL = 0.0f;   // the block's map up to this tile
#pragma unroll
  for (int i = 0; i < BLOCK - 1; ++i)
    if (i < j) compose(BA, BL, map_A(m[i]), map_L(m[i]));
  float CA = BA, CL = BL;       // and through it
  compose(CA, CL, A, L);
  if (closes) {
    publish(w.block_maps + row(b) + ch, map_word(CA, CL));
    if (CA < 0.0f || b == 0) publish(w.block_states + row(b + 1) + ch, word_of(apply(CA, CL, 0.0f)));
  }
  float S = 0.0f;   // the state that enters the block: not needed where a sequence begins in it before this tile
  for (bool found = b == 0 || BA < 0.0f; !found;) {
    int t = b;
    asm volatile("" : "+s"(t));
    uint32_t s[WINDOW];   // s[i]: the state that enters block b - i (zero for the first); n[i]: that block's map
    uint64_t n[WINDOW];
#pragma unroll
    for (int i = 0; i < WINDOW; ++i) {
      s[i] = t - i > 0 ? observe(w.block_states + row(t - i) + ch) : t == i ? 0u : EMPTY;
      n[i] = i > 0 && t - i >= 0 ? observe(w.block_maps + row(t - i) + ch) : ~0ull;
    }
    int at = -1;   // the nearest published state with all maps after it: i = at
    bool whole = true;
#pragma unroll
    for (int i = 0; i < WINDOW; ++i) {
      whole = whole && (i == 0 || n[i] != ~0ull);
      if (whole && at < 0 && s[i] != EMPTY) at = i;
    }
    if (at >= 0) {
#pragma unroll
      for (int i = WINDOW - 1; i >= 0; --i) {
        if (i == at) S = __uint_as_float(s[i]);
        if (i > 0 && i <= at) S = apply(map_A(n[i]), map_L(n[i]), S);
      }
      found = true;
    } else if (give_up()) {
      S = __uint_as_float(0x7fc00000u);
      found = true;
    }
  }
  if (closes && !(CA < 0.0f) && b > 0) publish(w.block_states + row(b + 1) + ch, word_of(apply(CA, CL, S)));
  return j == 0 ? S : apply(BA, BL, S);
}

// ---- which sequence a token belongs to -------------------------------------------

struct Place {
  int n;              // sequence, -1: none
  bool first, last;   // token of it
};

__device__ __forceinline__ int64_t bound_of(const int64_t* cu, int i, int T) {
  const int64_t v = cu[i];
  return v < 0 ? 0 : v > T ? T : v;
}

// largest n in [lo, hi] with cu[n] <= t, or lo
__device__ __forceinline__ int find_seq(const int64_t* cu, int lo, int hi, int t) {
  while (lo < hi) {
    const int mid = (lo + hi + 1) >> 1;
    if (cu[mid] <= t) lo = mid;
    else hi = mid - 1;
  }
  return lo;
}

__device__ __forceinline__ Place place_of(const GlrParams& p, const int64_t* cu, int lo, int hi, int t) {
  if (t >= p.tokens) return {-1, false, false};
  if (!cu) {
    const int n = (int)((uint32_t)t / (uint32_t)p.T), r = t - n * p.T;
    return {n, r == 0, r == p.T - 1};
  }
  const int n = find_seq(cu, lo, hi, t);
  const int64_t b = bound_of(cu, n, p.T), e = bound_of(cu, n + 1, p.T);
  if (t < b || t >= e) return {-1, false, false};
  return {n, t == b, t == e - 1};
}

// The lowest of a lane's gates as bits, which grow with a negative number's size: one maximum a
// word. is_low: -87 or less, so that its exp may be zero; is_nan: NaN of that sign.
template <int DT, int VEC>
using Bits = std::conditional_t<DT == FP32, uint32_t, uint16_t> __attribute__((ext_vector_type(VEC)));
template <int DT, int VEC>
__device__ __forceinline__ uint32_t lowest(const Pack<DT, VEC> (&g)[R]) {
  Bits<DT, VEC> m = __builtin_bit_cast(Bits<DT, VEC>, g[0].r);
#pragma unroll
  for (int r = 1; r < R; ++r) m = __builtin_elementwise_max(m, __builtin_bit_cast(Bits<DT, VEC>, g[r].r));
  return __builtin_reduce_max(m);
}
template <int DT>
__device__ __forceinline__ bool is_low(uint32_t bits) {
  return bits >= (DT == FP32 ? 0xc2ae0000u : DT == BF16 ? 0xc2aeu : 0xd570u);
}
template <int DT>
__device__ __forceinline__ bool is_nan(uint32_t bits) {
  return bits > (DT == FP32 ? 0xff800000u : DT == BF16 ? 0xff80u : 0xfc00u);
}
// Whether one of them is above zero (or a NaN of that sign)
template <int DT, int VEC>
__device__ __forceinline__ bool any_above(const Pack<DT, VEC> (&g)[R]) {
  using Int = std::conditional_t<DT == FP32, int32_t, int16_t> __attribute__((ext_vector_type(VEC)));
  Int m = __builtin_bit_cast(Int, g[0].r);
#pragma unroll
  for (int r = 1; r < R; ++r) m = __builtin_elementwise_max(m, __builtin_bit_cast(Int, g[r].r));
  return __builtin_reduce_max(m) > 0;
}
// Values that sums of a run's 8, each multiplied by at most 1, may not stay finite with: of 2^120
// and more, infinities and NaN
__device__ __forceinline__ bool is_large(float f) { return !(fabsf(f) < 0x1p120f); }
template <int DT, int VEC>
__device__ __forceinline__ bool any_large(const Pack<DT, VEC> (&q)[R]) {
  constexpr uint32_t SIZE = DT == FP32 ? 0x7fffffffu : 0x7fffu;
  Bits<DT, VEC> m = {};
#pragma unroll
  for (int r = 0; r < R; ++r) m = __builtin_elementwise_max(m, __builtin_bit_cast(Bits<DT, VEC>, q[r].r) & (Bits<DT, VEC>)SIZE);
  return __builtin_reduce_max(m) >= (DT == FP32 ? 0x7b800000u : DT == BF16 ? 0x7b80u : 0x7c00u);
}

// The sequences that a tile's tokens belong to, in shared memory: masks of tokens in a
// sequence, first of one and last of one; numbers of the sequences of all tokens.
struct TilePlaces {
  uint64_t in[GLR_TILE / 64], first[GLR_TILE / 64], last[GLR_TILE / 64];
  int n[GLR_TILE];
};

__device__ __forceinline__ void find_places(const GlrParams& p, const int64_t* cu, int t_base, TilePlaces& s) {
  const int tid = threadIdx.x;
  int lo = 0, hi = 0;
  if (cu) {   // the same search in every lane
    lo = find_seq(cu, 0, p.nseq - 1, t_base);
    hi = find_seq(cu, lo, p.nseq - 1, t_base + GLR_TILE - 1);
  }
  if (tid < GLR_TILE) {
    const Place q = place_of(p, cu, lo, hi, t_base + tid);
    s.n[tid] = q.n;
    const uint64_t in = __ballot(q.n >= 0), first = __ballot(q.first), last = __ballot(q.last);
    if ((tid & 63) == 0) {
      s.in[tid >> 6] = in;
      s.first[tid >> 6] = first;
      s.last[tid >> 6] = last;
    }
  }
}

// The channels of this workgroup. Workgroups go to the 8 XCDs in turn: neighbouring channels,
// which share lines where rows are not aligned, are put on one XCD and its L2 (8191 channels
// bf16 backward 214 -> 186 us; 8192: 141 -> 137).
__device__ __forceinline__ int tile_col(int cols) {
  const int b = blockIdx.x % cols, eighth = cols >> 3;
  return b < 8 * eighth ? (b & 7) * eighth + (b >> 3) : b;
}

// The next tile in the order of processing, from the counter of the channels (one lane asks)
__device__ __forceinline__ int take_tile(const TileWs& w, int col) {
  if (w.tiles == 1) return 0;
  return (int)__hip_atomic_fetch_add(w.ticks + col * TICK_STRIDE, 1u, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}

// ---- before the tiles: the words EMPTY, the counters zero; states of empty sequences ----
//
// A launch of its own (the words must be EMPTY before the first tile starts, and a workspace may
// hold anything): 5 us at 8192 x 8192, 5 MB, nearly all of it the launch; its grid makes no
// difference between 256 and 2048 workgroups.

__global__ __launch_bounds__(256) void kda_glr_prep_kernel(GlrParams p, TileWs w, const void* from, int from_dtype) {
  const int64_t i0 = (int64_t)blockIdx.x * 256 + threadIdx.x, step = (int64_t)gridDim.x * 256;
  const int64_t words = glr_words(w.tiles, p.D);   // maps and states lie one after the other
  const u32x4 ones = {EMPTY, EMPTY, EMPTY, EMPTY};
  for (int64_t i = i0; i < (words + 3) / 4; i += step) reinterpret_cast<u32x4*>(w.maps)[i] = ones;
  for (int64_t i = i0; i < (int64_t)w.cols * TICK_STRIDE; i += step) w.ticks[i] = 0;
  if (!w.stage && !p.cu && p.T > 0) return;
  for (int64_t i = i0; i < (int64_t)p.nseq * p.D; i += step) {
    const int n = (int)(i / p.D);
    const bool empty = p.cu ? bound_of(p.cu, n, p.T) >= bound_of(p.cu, n + 1, p.T) : p.T == 0;
    if (!w.stage && !empty) continue;
    float h;
    load_state<1>(from, from_dtype, i, &h);
    if (w.stage) w.stage[i] = h;
    if (empty) store_state<1>(p.fin, p.fin_dtype, i, &h);
  }
}

// ---- forward -----------------------------------------------------------------------

template <int DT, bool EXACT>
__global__ __launch_bounds__(256) void kda_glr_fwd_tile_kernel(GlrParams p, const int64_t* __restrict__ cu, TileWs w) {
  constexpr int VEC = Geom<DT>::VEC, CH = Geom<DT>::CH;
  __shared__ float sA[GRP][CH], sL[GRP][CH];
  __shared__ TilePlaces places;
  __shared__ int s_tile;
  const int tid = threadIdx.x, lr = tid % LR, grp = tid / LR;
  const int col = tile_col(w.cols);
  if (tid == 0) s_tile = take_tile(w, col);
  __syncthreads();
  const int tile = __builtin_amdgcn_readfirstlane(s_tile);
  if ((uint32_t)tile >= (uint32_t)w.tiles) return;   // (another call in the same workspace)
  const int t_base = tile * GLR_TILE, t0 = t_base + grp * R;
  const int d = col * CH + lr * VEC;
  const int c = p.D - d < 0 ? 0 : p.D - d > VEC ? VEC : p.D - d;   // elements of this lane (EXACT: VEC or none)

  // token r of a group: a uniform base and the lane's 32-bit offset (one register for all)
  const uint32_t off = ((uint32_t)(grp * R) * p.D + lr * VEC) * elem_size(DT);
  auto at = [&](int r) { return ((size_t)(t_base + r) * p.D + col * CH) * elem_size(DT); };
  Pack<DT, VEC> g[R], x[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    g[r].clear();
    x[r].clear();
    if (c > 0 && t0 + r < p.tokens) {
      load_part<EXACT>(g[r], static_cast<const uint8_t*>(p.g) + at(r) + off, c);
      load_part<EXACT>(x[r], static_cast<const uint8_t*>(p.x) + at(r) + off, c);
    }
  }
  find_places(p, cu, t_base, places);
  __syncthreads();
  const int word = grp * R / 64, bit = grp * R % 64;
  const uint32_t all = (uint32_t)((1ull << R) - 1);
  const uint32_t in = (uint32_t)(places.in[word] >> bit) & all, first = (uint32_t)(places.first[word] >> bit) & all,
                 last = (uint32_t)(places.last[word] >> bit) & all;
  // What a wave has to look out for: nothing (PLAIN), boundaries of sequences (ENDS), or those and
  // decays of zero, or products of them (CARE).
  enum { PLAIN, ENDS, CARE };
  int mode = __all(in == all && first == 0) ? PLAIN : __any(is_low<DT>(lowest(g))) ? CARE : ENDS;

  auto reduce = [&](auto mode_c, float* A, float* L) {   // returns whether decays of this lane multiply to zero, or are NaN
    constexpr int MODE = decltype(mode_c)::value;
#pragma unroll
    for (int v = 0; v < VEC; ++v) A[v] = 1.0f, L[v] = 0.0f;
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (MODE != PLAIN && !(in >> r & 1)) continue;
      float gf[VEC], xf[VEC];
      g[r].unpack(gf);
      x[r].unpack(xf);
      if (MODE != PLAIN && (first >> r & 1)) {
        float h0[VEC] = {};
        if (c > 0) load_state_part<EXACT, VEC>(p.init, p.init_dtype, (size_t)places.n[grp * R + r] * p.D + d, c, h0);
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          L[v] = follow(decay(gf[v]), h0[v], xf[v]);
          A[v] = RESET;
        }
      } else {
#pragma unroll
        for (int v = 0; v < VEC; ++v) {
          const float a = decay(gf[v]);
          L[v] = MODE == CARE ? follow(a, L[v], xf[v]) : fmaf(a, L[v], xf[v]);
          A[v] = MODE == CARE ? lasting(A[v], a) : MODE == ENDS && A[v] < 0.0f ? RESET : A[v] * a;
        }
      }
    }
    bool zero = false;
    if (MODE != CARE) {
#pragma unroll
      for (int v = 0; v < VEC; ++v) zero = zero || !(MODE == ENDS ? A[v] != 0.0f : A[v] > 0.0f);
    }
    return zero;
  };
  {
    float A[VEC], L[VEC];
    if (mode == PLAIN && __any(reduce(std::integral_constant<int, PLAIN>{}, A, L))) mode = CARE;
    else if (mode == ENDS && __any(reduce(std::integral_constant<int, ENDS>{}, A, L))) mode = CARE;
    if (mode == CARE) reduce(std::integral_constant<int, CARE>{}, A, L);
#pragma unroll
    for (int v = 0; v < VEC; ++v) {
      sA[grp][lr * VEC + v] = A[v];
      sL[grp][lr * VEC + v] = L[v];
    }
  }
  __syncthreads();
  if (tid < CH && col * CH + tid < p.D) {   // a lane per channel
    float TA = 1.0f, TL = 0.0f;
#pragma unroll 4
    for (int i = 0; i < GRP; ++i) compose(TA, TL, sA[i][tid], sL[i][tid]);
    float h = pass_state(w, tile, p.D, col * CH, tid, w.ticks + col * TICK_STRIDE + 1, TA, TL);
    if (p.carry) p.carry[(size_t)tile * p.D + col * CH + tid] = h;
#pragma unroll 4
    for (int i = 0; i < GRP; ++i) {   // the state that enters each group
      const float A = sA[i][tid], L = sL[i][tid];
      sL[i][tid] = h;
      h = apply(A, L, h);
    }
  }
  __syncthreads();
  if (c == 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {
    g[r].opaque();
    x[r].opaque();
  }
  auto outputs = [&](auto mode_c) {
    constexpr int MODE = decltype(mode_c)::value;
    float h[VEC];
#pragma unroll
    for (int v = 0; v < VEC; ++v) h[v] = sL[grp][lr * VEC + v];
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (MODE != PLAIN && !(in >> r & 1)) continue;
      float gf[VEC], xf[VEC];
      g[r].unpack(gf);
      x[r].unpack(xf);
      if (MODE != PLAIN && (first >> r & 1))
        load_state_part<EXACT, VEC>(p.init, p.init_dtype, (size_t)places.n[grp * R + r] * p.D + d, c, h);
#pragma unroll
      for (int v = 0; v < VEC; ++v)
        h[v] = MODE == PLAIN ? fmaf(decay(gf[v]), h[v], xf[v]) : follow(decay(gf[v]), h[v], xf[v]);
      Pack<DT, VEC> y;
      y.pack(h);
      store_part<EXACT>(y, static_cast<uint8_t*>(p.y) + at(r) + off, c);
      if (last >> r & 1) store_state_part<EXACT, VEC>(p.fin, p.fin_dtype, (size_t)places.n[grp * R + r] * p.D + d, c, h);
    }
  };
  if (mode == PLAIN) outputs(std::integral_constant<int, PLAIN>{});
  else outputs(std::integral_constant<int, CARE>{});
}

// ---- backward ------------------------------------------------------------------------
//
// E is the gradient that reaches the state behind a token from the tokens after it:
// G_t = dy_t + E, dx_t = G_t, then E = exp(g_t) G_t is passed to the token before, and
// dg_t = E h_{t-1}. E runs through the tiles from the last to the first as h does from the
// first to the last, with maps of the same A; the state that enters a tile was saved by the
// forward pass, so only E is passed between tiles here. Words of two channels (one in fp32)
// are worked on one after the other, their dx and dg written over x and g in the registers:
// of the states before each token only R times two are held at once (all channels' would take
// 64 more registers and a third of the waves).
template <int DT, bool EXACT>
__global__ __launch_bounds__(256) void kda_glr_bwd_tile_kernel(GlrParams p, const int64_t* __restrict__ cu, TileWs w) {
  constexpr int VEC = Geom<DT>::VEC, CH = Geom<DT>::CH;
  constexpr int NV = 4 / elem_size(DT);   // channels of a word
  __shared__ float sA[GRP][CH], sL[GRP][CH], sB[GRP][CH], sM[GRP][CH];
  __shared__ TilePlaces places;
  __shared__ int s_tile;
  const int tid = threadIdx.x, lr = tid % LR, grp = tid / LR;
  const int col = tile_col(w.cols);
  if (tid == 0) s_tile = take_tile(w, col);
  __syncthreads();
  const int k = __builtin_amdgcn_readfirstlane(s_tile), tile = w.tiles - 1 - k;
  if ((uint32_t)k >= (uint32_t)w.tiles) return;   // (another call in the same workspace)
  const int t_base = tile * GLR_TILE, t0 = t_base + grp * R;
  const int d = col * CH + lr * VEC;
  const int n_el = p.D - d < 0 ? 0 : p.D - d > VEC ? VEC : p.D - d;   // elements of this lane (EXACT: VEC or none)
  const uint32_t off = ((uint32_t)(grp * R) * p.D + lr * VEC) * elem_size(DT);
  auto at = [&](int r) { return ((size_t)(t_base + r) * p.D + col * CH) * elem_size(DT); };
  Pack<DT, VEC> g[R], x[R], dy[R];
#pragma unroll
  for (int r = 0; r < R; ++r) {
    g[r].clear();
    x[r].clear();
    dy[r].clear();
    if (n_el > 0 && t0 + r < p.tokens) {
      load_part<EXACT>(g[r], static_cast<const uint8_t*>(p.g) + at(r) + off, n_el);
      load_part<EXACT>(x[r], static_cast<const uint8_t*>(p.x) + at(r) + off, n_el);
      load_part<EXACT>(dy[r], static_cast<const uint8_t*>(p.dy) + at(r) + off, n_el);
    }
  }
  find_places(p, cu, t_base, places);
  __syncthreads();
  const int word = grp * R / 64, bit = grp * R % 64;
  const uint32_t all = (uint32_t)((1ull << R) - 1);
  const uint32_t in = (uint32_t)(places.in[word] >> bit) & all, first = (uint32_t)(places.first[word] >> bit) & all,
                 last = (uint32_t)(places.last[word] >> bit) & all;
  // What a wave has to look out for among its lanes' runs of tokens: nothing (PLAIN), at most
  // one first and one last token of a sequence in a run (chosen by selects) and decays of zero,
  // or products of them (ONE), or MANY, also where tokens lie before or behind all sequences.
  // (Rows behind the last token were not loaded: zeros, that is no decay, no input and no
  // gradient.) The outputs of ONE multiply by decays of zero, which gives the zero it has to be
  // as long as everything is finite: waves where it might not be (odd) become MANY.
  enum { PLAIN, ONE, MANY };
  const int left = p.tokens - t0;
  const bool whole = in == (left >= R ? all : left <= 0 ? 0u : all >> (R - left));
  int mode = !__all(whole && (first & (first - 1)) == 0 && (last & (last - 1)) == 0) ? MANY
             : __all(first == 0 && last == 0) ? PLAIN : ONE;
  bool low = false;   // ONE: whether there are decays of zero
  auto row = [&](int r) { return (size_t)places.n[grp * R + r] * p.D + d; };
  // a run's initial state and final gradient (ONE), elements c on
  auto ends = [&](int c, float* h0, float* e0) {
    int q = grp * R;
    asm volatile("" : "+v"(q));   // not kept from word to word
    if (first != 0 && n_el > c)
      load_state_part<EXACT, NV>(p.init, p.init_dtype, (size_t)places.n[q + __builtin_ctz(first)] * p.D + d + c, n_el - c, h0);
    if (last != 0 && n_el > c)
      load_state_part<EXACT, NV>(p.dfin, p.dfin_dtype, (size_t)places.n[q + __builtin_ctz(last)] * p.D + d + c, n_el - c, e0);
  };

  auto reduce = [&](auto mode_c) {   // returns PLAIN: whether decays of this lane multiply to zero, or are NaN; ONE: whether it is odd
    constexpr int MODE = decltype(mode_c)::value;
    bool found = false;
#pragma unroll
    for (int c = 0; c < VEC; c += NV) {
      __builtin_amdgcn_sched_barrier(0);   // one word after the other
      float a[R][NV], A[NV], L[NV], B[NV], M[NV], h0[NV], e0[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        A[v] = B[v] = 1.0f;
        L[v] = M[v] = h0[v] = e0[v] = 0.0f;
      }
      if (MODE == ONE) {
        ends(c, h0, e0);
#pragma unroll
        for (int v = 0; v < NV; ++v) found = found || is_large(h0[v]) || is_large(e0[v]);
      }
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float xf[NV];
        unpack_word<DT, VEC, NV>(g[r], c, a[r]);
        unpack_word<DT, VEC, NV>(x[r], c, xf);
        const bool start = MODE != PLAIN && (first >> r & 1), used = MODE != MANY || (in >> r & 1);
        if (MODE == MANY && start && n_el > c) load_state_part<EXACT, NV>(p.init, p.init_dtype, row(r) + c, n_el - c, h0);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float before = start ? h0[v] : L[v];
          if (MODE != PLAIN) {
            a[r][v] = used ? decay(a[r][v]) : 1.0f;   // a token of no sequence: no decay, no input, no gradient
            L[v] = follow(a[r][v], before, used ? xf[v] : 0.0f);
            A[v] = start ? RESET : lasting(A[v], a[r][v]);
          } else {
            a[r][v] = decay(a[r][v]);
            L[v] = fmaf(a[r][v], before, xf[v]);
            A[v] *= a[r][v];
          }
        }
      }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float df[NV];
        unpack_word<DT, VEC, NV>(dy[r], c, df);
        const bool end = MODE != PLAIN && (last >> r & 1), used = MODE != MANY || (in >> r & 1);
        if (MODE == MANY && end && n_el > c) load_state_part<EXACT, NV>(p.dfin, p.dfin_dtype, row(r) + c, n_el - c, e0);
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          const float G = (used ? df[v] : 0.0f) + (end ? e0[v] : M[v]);
          M[v] = MODE != PLAIN && a[r][v] == 0.0f ? 0.0f : a[r][v] * G;
          B[v] = MODE == PLAIN ? B[v] * a[r][v] : end ? RESET : lasting(B[v], a[r][v]);
        }
      }
      if (MODE == PLAIN) {
#pragma unroll
        for (int v = 0; v < NV; ++v) found = found || !(A[v] > 0.0f) || !(B[v] > 0.0f);
      }
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        const int ch = lr * VEC + c + v;
        sA[grp][ch] = A[v];
        sL[grp][ch] = L[v];
        sB[grp][ch] = B[v];
        sM[grp][ch] = M[v];
      }
    }
    return found;
  };
  if (mode == PLAIN && __any(reduce(std::integral_constant<int, PLAIN>{}))) mode = ONE;
  if (mode != PLAIN) {
    if (EXACT) {   // nothing is kept from the other form (56 registers; without whole vectors none)
#pragma unroll
      for (int r = 0; r < R; ++r) {
        g[r].opaque();
        x[r].opaque();
        dy[r].opaque();
      }
    }
    if (mode == MANY) {
      reduce(std::integral_constant<int, MANY>{});
    } else {
      const uint32_t lowest_gate = lowest(g);
      low = __any(is_low<DT>(lowest_gate));
      const bool odd = reduce(std::integral_constant<int, ONE>{});
      if (low && __any(odd || is_nan<DT>(lowest_gate) || any_above(g) || any_large(x) || any_large(dy))) mode = MANY;
    }
  }
  __syncthreads();
  if (tid < CH && col * CH + tid < p.D) {
    const size_t dc = (size_t)col * CH + tid;
    float TB = 1.0f, TM = 0.0f;
#pragma unroll 4
    for (int i = GRP - 1; i >= 0; --i) compose(TB, TM, sB[i][tid], sM[i][tid]);
    float h = p.carry[(size_t)tile * p.D + dc];
    float E = pass_state(w, k, p.D, col * CH, tid, w.ticks + col * TICK_STRIDE + 1, TB, TM);
#pragma unroll 4
    for (int i = 0; i < GRP; ++i) {
      const float A = sA[i][tid], L = sL[i][tid];
      sL[i][tid] = h;
      h = apply(A, L, h);
    }
#pragma unroll 4
    for (int i = GRP - 1; i >= 0; --i) {
      const float B = sB[i][tid], M = sM[i][tid];
      sM[i][tid] = E;
      E = apply(B, M, E);
    }
  }
  __syncthreads();
  if (n_el == 0) return;
#pragma unroll
  for (int r = 0; r < R; ++r) {   // the exps are computed again: kept, they would take R * VEC registers
    g[r].opaque();
    x[r].opaque();
    dy[r].opaque();
  }

  if (mode == ONE && low) {
    bool odd = false;
#pragma unroll
    for (int v = 0; v < VEC; ++v) odd = odd || is_large(sL[grp][lr * VEC + v]) || is_large(sM[grp][lr * VEC + v]);
    if (__any(odd)) mode = MANY;
  }
  if (mode != MANY) {
#pragma unroll
    for (int c = 0; c < VEC; c += NV) {
      __builtin_amdgcn_sched_barrier(0);
      float a[R][NV], before[R][NV], h[NV], E[NV], h0[NV], e0[NV];
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        h[v] = sL[grp][lr * VEC + c + v];
        E[v] = sM[grp][lr * VEC + c + v];
        h0[v] = e0[v] = 0.0f;
      }
      if (mode != PLAIN) ends(c, h0, e0);
#pragma unroll
      for (int r = 0; r < R; ++r) {
        float xf[NV];
        unpack_word<DT, VEC, NV>(g[r], c, a[r]);
        unpack_word<DT, VEC, NV>(x[r], c, xf);
        const bool start = first >> r & 1;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          a[r][v] = decay(a[r][v]);
          before[r][v] = start ? h0[v] : h[v];
          h[v] = fmaf(a[r][v], before[r][v], xf[v]);
        }
      }
#pragma unroll
      for (int r = R - 1; r >= 0; --r) {
        float df[NV], dg[NV];
        unpack_word<DT, VEC, NV>(dy[r], c, df);
        const bool end = last >> r & 1, start = first >> r & 1;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
          df[v] += end ? e0[v] : E[v];
          E[v] = a[r][v] * df[v];
          dg[v] = E[v] * before[r][v];
          if (start) h0[v] = E[v];   // the gradient of the initial state, from here on
        }
        pack_word<DT, VEC, NV>(x[r], c, df);
        pack_word<DT, VEC, NV>(g[r], c, dg);
      }
      if (first != 0 && n_el > c)
        store_state_part<EXACT, NV>(p.fin, p.fin_dtype, row(__builtin_ctz(first)) + c, n_el - c, h0);
#pragma unroll
      for (int r = 0; r < R; ++r) {   // each pack stays one run of registers: no copies of it
        g[r].opaque();
        x[r].opaque();
      }
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!(in >> r & 1)) continue;
      // (lines shared with the next tile's rows are completed in the cache: 8191 channels 207 -> 187 us;
      // forward, with half as many stores, streaming is faster there too: 111 -> 100 us)
      store_part<EXACT, EXACT>(x[r], static_cast<uint8_t*>(p.dx) + at(r) + off, n_el);
      store_part<EXACT, EXACT>(g[r], static_cast<uint8_t*>(p.dg) + at(r) + off, n_el);
    }
    return;
  }
  // MANY: the tokens are read again (they are in the caches), a word at a time: with the packs
  // and every case of every token in registers at once, the kernel would need 242 of them and
  // lose a third of its waves. A wave is here with all its 32 tokens if one of its runs of 8 has
  // two first or two last tokens, a token of no sequence, or both a decay of zero and a value
  // that is not finite.
  for (int c = 0; c < VEC && c < n_el; c += NV) {
    float a[R][NV], before[R][NV], h[NV], E[NV];
    int q = grp * R;
    uint32_t o = off + c * elem_size(DT);
    asm volatile("" : "+v"(q), "+v"(o));   // no address is kept from word to word
    auto row = [&](int r) { return (size_t)places.n[q + r] * p.D + d + c; };
    auto read = [&](const void* from, int r, float* f) {
#pragma unroll
      for (int v = 0; v < NV; ++v) f[v] = 0.0f;
      if (EXACT) {
        Pack<DT, NV> k;
        k.load_at(from, at(r), o);
        k.unpack(f);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (c + v < n_el) {
            Pack<DT, 1> k;
            k.load_at(from, at(r), o + v * elem_size(DT));
            k.unpack(f + v);
          }
      }
    };
    auto write = [&](void* to, int r, const float* f) {
      if (EXACT) {
        Pack<DT, NV> k;
        k.pack(f);
        k.store_at(to, at(r), o);
      } else {
#pragma unroll
        for (int v = 0; v < NV; ++v)
          if (c + v < n_el) {
            Pack<DT, 1> k;
            k.pack(f + v);
            k.store_at(to, at(r), o + v * elem_size(DT));
          }
      }
    };
#pragma unroll
    for (int v = 0; v < NV; ++v) {
      h[v] = sL[grp][lr * VEC + c + v];
      E[v] = sM[grp][lr * VEC + c + v];
    }
#pragma unroll
    for (int r = 0; r < R; ++r) {
      if (!(in >> r & 1)) continue;
      float xf[NV];
      read(p.g, r, a[r]);
      read(p.x, r, xf);
      if (first >> r & 1) load_state_part<EXACT, NV>(p.init, p.init_dtype, row(r), n_el - c, h);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        a[r][v] = decay(a[r][v]);
        before[r][v] = h[v];
        h[v] = follow(a[r][v], h[v], xf[v]);
      }
    }
#pragma unroll
    for (int r = R - 1; r >= 0; --r) {
      if (!(in >> r & 1)) continue;
      float df[NV], dg[NV];
      read(p.dy, r, df);
      if (last >> r & 1) load_state_part<EXACT, NV>(p.dfin, p.dfin_dtype, row(r), n_el - c, E);
#pragma unroll
      for (int v = 0; v < NV; ++v) {
        df[v] += E[v];
        E[v] = a[r][v] == 0.0f ? 0.0f : a[r][v] * df[v];
        dg[v] = a[r][v] == 0.0f ? 0.0f : E[v] * before[r][v];
      }
      write(p.dx, r, df);
      write(p.dg, r, dg);
      if (first >> r & 1) store_state_part<EXACT, NV>(p.fin, p.fin_dtype, row(r), n_el - c, E);
    }
  }
}

// ---- few tokens per sequence -----------------------------------------------------------

// One lane per VEC channels of a sequence, token by token, from and to rows of the states or
// slots of a cache (SLOTS: a single token). Otherwise 8 tokens are loaded at once (16 tokens of
// one row of 8192 channels: 6.0 -> 4.8 us).
template <int DT, int VEC, bool SLOTS>
__global__ __launch_bounds__(64) void kda_glr_tokens_kernel(GlrParams p, int cols) {
  constexpr int AHEAD = SLOTS ? 1 : 8;
  const int n = blockIdx.x / cols, d = ((blockIdx.x - n * cols) * 64 + threadIdx.x) * VEC;
  if (d >= p.D) return;
  int64_t b = (int64_t)n * p.T, e = b + p.T;
  if (p.cu) {
    b = bound_of(p.cu, n, p.T);
    e = bound_of(p.cu, n + 1, p.T);
  }
  int in_row = n, out_row = n, in_dtype = p.init_dtype, out_dtype = p.fin_dtype;
  if (SLOTS) {
    in_row = p.in_slots[n];
    out_row = p.out_slots[n];
    if (in_row < 0 || in_row >= p.n_slots) in_dtype = 0;
    if (out_row < 0 || out_row >= p.n_slots) out_dtype = 0;
  }
  float h[VEC];
  load_state<VEC>(p.init, in_dtype, (size_t)in_row * p.D + d, h);
  for (int64_t t0 = b; t0 < e; t0 += AHEAD) {
    Pack<DT, VEC> g[AHEAD], x[AHEAD];
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      if (t0 + r < e) {
        g[r].load(p.g, (size_t)(t0 + r) * p.D + d);
        x[r].load(p.x, (size_t)(t0 + r) * p.D + d);
      }
    }
#pragma unroll
    for (int r = 0; r < AHEAD; ++r) {
      const int64_t t = t0 + r;
      if (t >= e) break;
      float gf[VEC], xf[VEC];
      g[r].unpack(gf);
      x[r].unpack(xf);
      if (p.carry && t % GLR_TILE == 0) store_f32<FP32, VEC>(p.carry, (size_t)(t / GLR_TILE) * p.D + d, h);
#pragma unroll
      for (int v = 0; v < VEC; ++v) h[v] = follow(decay(gf[v]), h[v], xf[v]);
      Pack<DT, VEC> y;
      y.pack(h);
      y.store(p.y, (size_t)t * p.D + d);
    }
  }
  store_state<VEC>(p.fin, out_dtype, (size_t)out_row * p.D + d, h);
}

// f(element type, elements of a vector, whether rows are whole vectors)
template <typename F>
hipError_t by_type(int dt, int32_t D, F f) {
  const auto go = [&](auto type) {
    constexpr int VEC = 16 / elem_size(decltype(type)::value);
    if (D % VEC == 0) f(type, std::integral_constant<int, VEC>{}, std::true_type{});
    else f(type, std::integral_constant<int, 1>{}, std::false_type{});
  };
  if (dt == BF16) go(std::integral_constant<int, BF16>{});
  else if (dt == FP16) go(std::integral_constant<int, FP16>{});
  else go(std::integral_constant<int, FP32>{});
  return hipGetLastError();
}

int32_t tile_count(int64_t tokens) { return (int32_t)((tokens + GLR_TILE - 1) / GLR_TILE); }
int32_t tile_cols(int dt, int32_t D) {
  const int ch = LR * (16 / elem_size(dt));
  return (D + ch - 1) / ch;
}
size_t up256(size_t x) { return (x + 255) / 256 * 256; }

// Polls of a wait at most: a poll takes a microsecond. KDA_GLR_POLLS where it is a whole number
// (above 32 bits: the most there can be); any other text leaves it as it is.
uint32_t polls_of_a_wait() {
  constexpr uint32_t MOST = 1u << 24;
  const char* e = std::getenv("KDA_GLR_POLLS");
  if (!e || *e < '0' || *e > '9') return MOST;
  char* end = nullptr;
  const unsigned long long v = std::strtoull(e, &end, 10);
  if (*end != '\0') return MOST;
  return v < UINT32_MAX ? (uint32_t)v : UINT32_MAX;
}

TileWs tile_ws(const GlrParams& p, void* workspace, bool stage) {
  TileWs w{};
  uint8_t* b = static_cast<uint8_t*>(workspace);
  w.polls = polls_of_a_wait();
  w.tiles = tile_count(p.tokens);
  w.cols = tile_cols(p.dtype, p.D);
  const size_t words = (size_t)glr_words(w.tiles, p.D), blocks = (size_t)((w.tiles + BLOCK - 1) / BLOCK);
  w.maps = reinterpret_cast<uint64_t*>(b);
  w.block_maps = w.maps + (size_t)w.tiles * p.D;
  w.block_states = reinterpret_cast<uint32_t*>(w.block_maps + blocks * p.D);
  const size_t ticks = up256(words * 4 + 16);   // (the fill writes whole vectors)
  w.ticks = reinterpret_cast<uint32_t*>(b + ticks);
  if (stage) w.stage = reinterpret_cast<float*>(b + ticks + up256((size_t)((p.D + 63) / 64) * TICK_STRIDE * 4));
  return w;
}

hipError_t launch_prep(const GlrParams& p, const TileWs& w, const void* from, int from_dtype, hipStream_t stream) {
  const int64_t fill = (glr_words(w.tiles, p.D) + 3) / 4, rows = w.stage || p.cu || p.T == 0 ? (int64_t)p.nseq * p.D : 0;
  const int64_t blocks = ((fill > rows ? fill : rows) + 255) / 256;
  hipLaunchKernelGGL(kda_glr_prep_kernel, dim3((unsigned)(blocks < 2048 ? blocks : 2048)), dim3(256), 0, stream, p, w, from,
                     from_dtype);
  return hipGetLastError();
}

// Few tokens per sequence: rows of at most FEW tokens (8192 channels bf16: 16 tokens 4.8 us
// against 8.1 in tiles, 32 the same, 64 13.0 against 7.5), packed batches of at most 2 on average
// (1024 channels, 512 tokens of a sequence each 4.3 against 19.7 us). Their lengths stay on the
// device, and the tokens of a long sequence among them are walked one after the other, 0.21 us
// each, which tiles would not do: of 512 tokens half in one sequence 53 against 18 us, all 102
// against 13; of 8192 870 against 35 and 1727 against 30. So not beyond FEW_PACKED tokens, where
// what the even batch gains is about what the uneven one loses.
constexpr int32_t FEW = 32, FEW_PACKED = 512;
bool few_tokens(const GlrParams& p) {
  return p.cu ? p.T <= FEW_PACKED && p.T <= 2 * (int64_t)p.nseq : p.T <= FEW;
}
// One tile, and nothing to do before it: no counters, no words to fill.
bool lone_tile(const GlrParams& p, const TileWs& w) { return w.tiles == 1 && !p.cu && !w.stage; }

}  // namespace

size_t glr_workspace(int64_t tokens, int64_t D, int64_t nseq) {
  return up256((size_t)glr_words(tile_count(tokens), D) * 4 + 16) + up256((size_t)((D + 63) / 64) * TICK_STRIDE * 4) + up256((size_t)nseq * D * 4);
}

bool glr_fits(int64_t tokens, int64_t D, int64_t nseq) {
  const int64_t cols = (D + 63) / 64, most = (int64_t)1 << 24;   // workgroups of a launch
  return cols * ((tokens + GLR_TILE - 1) / GLR_TILE) < most && cols * nseq < most;
}

hipError_t launch_glr_fwd(const GlrParams& p, void* workspace, hipStream_t stream) {
  if (p.nseq <= 0) return hipSuccess;
  if (p.in_slots || few_tokens(p)) {
    return by_type(p.dtype, p.D, [&](auto dt, auto vec, auto) {
      const int cols = (p.D + 64 * vec.value - 1) / (64 * vec.value);
      const dim3 grid((unsigned)cols * (unsigned)p.nseq);
      if (p.in_slots)
        hipLaunchKernelGGL((kda_glr_tokens_kernel<dt.value, vec.value, true>), grid, dim3(64), 0, stream, p, cols);
      else
        hipLaunchKernelGGL((kda_glr_tokens_kernel<dt.value, vec.value, false>), grid, dim3(64), 0, stream, p, cols);
    });
  }
  // a sequence's final state may be written while another workgroup still reads its initial one
  const bool stage = p.init && p.init == p.fin;
  const TileWs w = tile_ws(p, workspace, stage);
  if (!lone_tile(p, w)) {
    const hipError_t e = launch_prep(p, w, p.init, p.init_dtype, stream);
    if (e != hipSuccess) return e;
  }
  GlrParams q = p;
  if (stage) {
    q.init = w.stage;
    q.init_dtype = FP32;
  }
  return by_type(p.dtype, p.D, [&](auto dt, auto, auto exact) {
    hipLaunchKernelGGL((kda_glr_fwd_tile_kernel<dt.value, exact.value>), dim3((unsigned)w.cols * (unsigned)w.tiles), dim3(256),
                       0, stream, q, q.cu, w);
  });
}

hipError_t launch_glr_bwd(const GlrParams& p, void* workspace, hipStream_t stream) {
  if (p.nseq <= 0) return hipSuccess;
  const TileWs w = tile_ws(p, workspace, false);
  if (!lone_tile(p, w)) {
    const hipError_t e = launch_prep(p, w, p.dfin, p.dfin_dtype, stream);
    if (e != hipSuccess) return e;
  }
  if (w.tiles == 0) return hipSuccess;
  return by_type(p.dtype, p.D, [&](auto dt, auto, auto exact) {
    hipLaunchKernelGGL((kda_glr_bwd_tile_kernel<dt.value, exact.value>), dim3((unsigned)w.cols * (unsigned)w.tiles), dim3(256),
                       0, stream, p, p.cu, w);
  });
}

}  // namespace kda
