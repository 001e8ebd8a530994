// kda_conv.hip -- short causal convolution per channel, forward, backward and single tokens
// (gfx950).
//
//     u_t = bias + sum_j w[j] x_{t-W+1+j},   y_t = u_t or u_t sigmoid(u_t)
//
// Bound by memory: x is read and y written once (8192 tokens x 8192 channels bf16: 70 us, 3.9 TB/s;
// backward, 26810 x 1024 with 32 sequences, 54 us). A lane takes 16 bytes of channels of a run of
// consecutive tokens and keeps the last W - 1 inputs in registers, so a run costs W - 1 tokens
// read twice (from the caches: its neighbours read them too). Forward, the next 8 tokens are loaded
// while 8 are computed, in runs of more than 8: a run is 32 tokens, or half and a quarter of that
// where longer ones would leave less than 1024 workgroups (8 at 26810 x 1024: 38 us). A sequence's
// first token puts the initial state, or zeros, into those registers.
//
// Backward, with du = dy SiLU'(u) recomputed from x: an input gets w[W-1-o] du_{t+o} from the
// output o tokens after it, so a lane also keeps W - 1 unfinished sums, and reads W - 1 tokens
// past its run; it loads 4 tokens, then computes them. The weight's sums stay in registers over all
// of a lane's runs, are added up over the workgroup, and a second kernel adds the workgroups' sums in
// a fixed order.
//
// States are written by workgroups of their own, a lane all of a sequence's state after it has read
// all of it; where final_state is initial_state, in a launch after the one that reads it.
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"
#include "kda_seq.h"

namespace kda {
namespace {

using std::integral_constant;

constexpr int BATCH = 8, BWD_BATCH = 4;   // tokens loaded at once

template <int DT>
constexpr int vec_of() { return 16 / elem_size(DT); }

// V neighbouring channels of a tensor, at any alignment (the hardware splits what crosses a line)
template <int DT, int V>
__device__ __forceinline__ void load_any(Pack<DT, V>& q, const void* p, size_t i) {
  __builtin_memcpy(&q.r, static_cast<const uint8_t*>(p) + i * elem_size(DT), V * elem_size(DT));
}
template <int DT, int V>
__device__ __forceinline__ void store_any(const Pack<DT, V>& q, void* p, size_t i) {
  if constexpr (V == 1) {
    q.store(p, i);
  } else {   // past the caches
    using Any = typename Pack<DT, V>::Raw __attribute__((aligned(2)));
    __builtin_nontemporal_store(q.r, reinterpret_cast<Any*>(static_cast<uint8_t*>(p) + i * elem_size(DT)));
  }
}
template <int DT, int V>
__device__ __forceinline__ void load_any_f32(const void* p, size_t i, float* f) {
  constexpr int M = V * elem_size(DT) > 16 ? 16 / elem_size(DT) : V;
#pragma unroll
  for (int j = 0; j < V; j += M) {
    Pack<DT, M> q;
    load_any(q, p, i + j);
    q.unpack(f + j);
  }
}
template <int V>
__device__ __forceinline__ void load_state_any(const void* p, int dtype, size_t i, float* f) {
  if (dtype == FP32) load_any_f32<FP32, V>(p, i, f);
  else if (dtype == BF16) load_any_f32<BF16, V>(p, i, f);
  else {
#pragma unroll
    for (int j = 0; j < V; ++j) f[j] = 0.0f;
  }
}

template <int DT, int V>
__device__ __forceinline__ void store_any_f32(void* p, size_t i, const float* f) {
  constexpr int M = V * elem_size(DT) > 16 ? 16 / elem_size(DT) : V;
#pragma unroll
  for (int j = 0; j < V; j += M) {
    Pack<DT, M> q;
    q.pack(f + j);
    __builtin_memcpy(static_cast<uint8_t*>(p) + (i + j) * elem_size(DT), &q.r, M * elem_size(DT));
  }
}
template <int V>
__device__ __forceinline__ void store_state_any(void* p, int dtype, size_t i, const float* f) {
  if (dtype == FP32) store_any_f32<FP32, V>(p, i, f);
  else if (dtype == BF16) store_any_f32<BF16, V>(p, i, f);
}

__device__ __forceinline__ Seqs seqs_of(const ConvParams& p) { return {p.cu, p.nseq, p.T, p.tokens}; }

template <int W, int V>
struct Taps {
  float w[W][V], b[V];

  __device__ __forceinline__ void load(const ConvParams& p, int d) {
#pragma unroll
    for (int e = 0; e < V; ++e) {
#pragma unroll
      for (int j = 0; j < W; ++j) w[j][e] = p.weight[(size_t)(d + e) * W + j];
      b[e] = p.bias ? p.bias[d + e] : 0.0f;
    }
  }
  // u of the inputs before (old[0] the oldest) and x
  __device__ __forceinline__ void apply(const float (&old)[W - 1][V], const float* x, float* u) const {
#pragma unroll
    for (int e = 0; e < V; ++e) {
      float s = b[e];
#pragma unroll
      for (int j = 0; j < W - 1; ++j) s = fmaf(w[j][e], old[j][e], s);
      u[e] = fmaf(w[W - 1][e], x[e], s);
    }
  }
};

template <int V, int N>
__device__ __forceinline__ void shift(float (&old)[N][V], const float* x) {
#pragma unroll
  for (int j = 0; j + 1 < N; ++j)
#pragma unroll
    for (int e = 0; e < V; ++e) old[j][e] = old[j + 1][e];
#pragma unroll
  for (int e = 0; e < V; ++e) old[N - 1][e] = x[e];
}

// The W - 1 inputs before token t of the sequence [b, e) with number n: of x, or of the state
template <int DT, int W, int V>
__device__ __forceinline__ void load_before(const ConvParams& p, int n, int32_t b, int32_t t, int d,
                                            float (&old)[W - 1][V]) {
#pragma unroll
  for (int j = 0; j < W - 1; ++j) {
    const int32_t at = t - (W - 1) + j;
    if (at >= b) {
      load_any_f32<DT, V>(p.x, (size_t)at * p.D + d, old[j]);
    } else {
      load_state_any<V>(p.init, p.init_dtype, ((size_t)n * (W - 1) + (at - b + W - 1)) * p.D + d, old[j]);
    }
  }
}

// A lane's channels d .. d + V - 1 and its place among the workgroup's runs: 2^lr_log lanes across
// the channels. The last channels of a width that is no multiple of V belong to two lanes, which
// both write the same.
struct Where {
  int grp, d;
  bool any;
  __device__ __forceinline__ Where(int lr_log, int col, int D, int V) {
    grp = threadIdx.x >> lr_log;
    const int64_t at = (((int64_t)col << lr_log) + (threadIdx.x & ((1 << lr_log) - 1))) * V;
    any = at < D;
    d = (int)(at + V <= D ? at : D - V);
  }
};

// ---- forward ----------------------------------------------------------------------

// The last W - 1 inputs of every sequence, the state before it included: the share of workgroup
// `block` of `blocks`. A lane: a sequence's V channels.
template <int DT, int W, int V>
__device__ __forceinline__ void final_states(const ConvParams& p, int block, int blocks) {
  const Seqs s = seqs_of(p);
  const int vecs = p.D / V;
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < (int64_t)p.nseq * vecs; i += (int64_t)blocks * 256) {
    const int n = (int)(i / vecs), d = (int)(i - (int64_t)n * vecs) * V;
    const int32_t b = s.begin(n), e = s.begin(n + 1);
    float old[W - 1][V];
    load_before<DT, W, V>(p, n, b, e > b ? e : b, d, old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) store_state<V>(p.fin, p.fin_dtype, ((size_t)n * (W - 1) + j) * p.D + d, old[j]);
  }
}
template <int DT, int W, int V>
__device__ __forceinline__ void any_final_states(const ConvParams& p, int block, int blocks) {
  if (p.D % V == 0) final_states<DT, W, V>(p, block, blocks);
  else final_states<DT, W, 1>(p, block, blocks);
}
template <int DT, int W, int V>
__global__ __launch_bounds__(256) void kda_conv_final_kernel(ConvParams p) {
  any_final_states<DT, W, V>(p, blockIdx.x, gridDim.x);
}

template <int DT, int W, int V>
__global__ __launch_bounds__(256) void kda_conv_fwd_kernel(ConvParams p, int lr_log, int cols, int run, int states) {
  if ((int)blockIdx.x < states) {
    any_final_states<DT, W, V>(p, blockIdx.x, states);
    return;
  }
  const int block = blockIdx.x - states;
  const Seqs s = seqs_of(p);
  const Where at(lr_log, block % cols, p.D, V);
  const int64_t first = ((int64_t)(block / cols) * (256 >> lr_log) + at.grp) * run;
  if (!at.any || first >= p.tokens) return;
  const int32_t t0 = (int32_t)first, t1 = p.tokens - t0 < run ? p.tokens : t0 + run;
  const int d = at.d;
  Pack<DT, V> next[BATCH];
  auto load = [&](int32_t t) {
#pragma unroll
    for (int r = 0; r < BATCH; ++r)
      if (t + r < t1) load_any(next[r], p.x, (size_t)(t + r) * p.D + d);
  };
  load(t0);
  Taps<W, V> taps;
  taps.load(p, d);
  SeqWalk q;
  q.start(s, t0);
  float old[W - 1][V];
  load_before<DT, W, V>(p, q.i, t0 > q.b && t0 < q.e ? q.b : t0, t0, d, old);   // (a first token loads its own below)
  for (int32_t t = t0; t < t1; t += BATCH) {
    Pack<DT, V> x[BATCH];
#pragma unroll
    for (int r = 0; r < BATCH; ++r) x[r] = next[r];
    load(t + BATCH);
#pragma unroll
    for (int r = 0; r < BATCH; ++r) {
      if (t + r >= t1) break;
      if (t + r >= q.e) q.forward(s, t + r);
      if (t + r == q.b) load_before<DT, W, V>(p, q.i, q.b, q.b, d, old);
      if (!q.holds(t + r)) continue;
      float f[V], u[V];
      x[r].unpack(f);
      taps.apply(old, f, u);
      shift<V, W - 1>(old, f);
      if (p.silu) {
#pragma unroll
        for (int e = 0; e < V; ++e) u[e] *= sigmoidf_fast(u[e]);
      }
      Pack<DT, V> y;
      y.pack(u);
      store_any(y, p.out, (size_t)(t + r) * p.D + d);
    }
  }
}

// One token for each sequence, states in slots
template <int DT, int W, int V>
__global__ __launch_bounds__(256) void kda_conv_step_kernel(ConvParams p, int vecs) {
  for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < (int64_t)p.nseq * vecs; i += (int64_t)gridDim.x * 256) {
    const int n = (int)(i / vecs), d = (int)(i - (int64_t)n * vecs) * V;
    const int from = p.in_slots[n], to = p.out_slots[n];
    Pack<DT, V> x;
    load_any(x, p.x, (size_t)n * p.D + d);
    float old[W - 1][V];
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const bool some = from >= 0 && from < p.n_slots;
      load_state_any<V>(p.init, some ? p.init_dtype : 0, ((size_t)(some ? from : 0) * (W - 1) + j) * p.D + d, old[j]);
    }
    Taps<W, V> taps;
    taps.load(p, d);
    float f[V], u[V];
    x.unpack(f);
    taps.apply(old, f, u);
    shift<V, W - 1>(old, f);
    if (p.silu) {
#pragma unroll
      for (int e = 0; e < V; ++e) u[e] *= sigmoidf_fast(u[e]);
    }
    Pack<DT, V> y;
    y.pack(u);
    y.store(p.out, (size_t)n * p.D + d);
    if (to >= 0 && to < p.n_slots) {
#pragma unroll
      for (int j = 0; j < W - 1; ++j)
        store_state<V>(p.fin, p.fin_dtype, ((size_t)to * (W - 1) + j) * p.D + d, old[j]);
    }
  }
}

// ---- backward ---------------------------------------------------------------------

// du of u and dy
__device__ __forceinline__ float grad_of(float u, float dy) {
  const float sg = sigmoidf_fast(u);
  return dy * (sg * fmaf(u, 1.0f - sg, 1.0f));
}

// Gradient of the initial states: from the first W - 1 tokens, and from the final state where a
// sequence is shorter than that
template <int DT, int W, int V>
__device__ __forceinline__ void initial_grads(const ConvParams& p, int block, int blocks) {
  const int vecs = p.D / V;
  const Seqs s = seqs_of(p);
  for (int64_t i = (int64_t)block * 256 + threadIdx.x; i < (int64_t)p.nseq * vecs; i += (int64_t)blocks * 256) {
    const int n = (int)(i / vecs), d = (int)(i - (int64_t)n * vecs) * V;
    const int32_t b = s.begin(n), len = s.begin(n + 1) - b;
    Taps<W, V> taps;
    taps.load(p, d);
    float old[W - 1][V], out[W - 1][V];
    load_before<DT, W, V>(p, n, b, b, d, old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j) {
      const int row = j - (len > 0 ? len : 0);   // of the final state
      load_state_any<V>(p.dfin, row >= 0 ? p.dfin_dtype : 0, ((size_t)n * (W - 1) + (row >= 0 ? row : 0)) * p.D + d, out[j]);
    }
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      if (r >= len) break;
      float f[V], g[V], u[V];
      load_any_f32<DT, V>(p.x, (size_t)(b + r) * p.D + d, f);
      load_any_f32<DT, V>(p.dy, (size_t)(b + r) * p.D + d, g);
      taps.apply(old, f, u);
      if (p.silu) {
#pragma unroll
        for (int e = 0; e < V; ++e) g[e] = grad_of(u[e], g[e]);
      }
      shift<V, W - 1>(old, f);
#pragma unroll
      for (int j = 0; j < W - 1; ++j)   // state row j is input r - (W - 1) + j - r of this output, tap j - r
        if (j >= r) {
#pragma unroll
          for (int e = 0; e < V; ++e) out[j][e] = fmaf(taps.w[j - r][e], g[e], out[j][e]);
        }
    }
#pragma unroll
    for (int j = 0; j < W - 1; ++j)   // (4 channels of rows that are no whole 16 bytes: states begin anywhere there)
      store_state_any<V>(p.dinit, p.dinit_dtype, ((size_t)n * (W - 1) + j) * p.D + d, out[j]);
  }
}

template <int DT, int W, int V>
__global__ __launch_bounds__(256) void kda_conv_bwd_kernel(ConvParams p, int lr_log, int cols, int run, int parts, int states) {
  constexpr int K = V * (W + 1);
  __shared__ float sums[256 * (K + 1)];
  if ((int)blockIdx.x < states) {
    if (p.D % V == 0) initial_grads<DT, W, V>(p, blockIdx.x, states);
    else initial_grads<DT, W, 1>(p, blockIdx.x, states);
    return;
  }
  const Seqs s = seqs_of(p);
  const int col = (blockIdx.x - states) % cols, part = (blockIdx.x - states) / cols, groups = 256 >> lr_log;
  const Where at(lr_log, col, p.D, V);
  const int d = at.d;
  const int32_t lo = s.begin(0), hi = s.begin(s.n);   // tokens of any sequence
  float dw[W][V], db[V];
#pragma unroll
  for (int e = 0; e < V; ++e) {
    db[e] = 0.0f;
#pragma unroll
    for (int j = 0; j < W; ++j) dw[j][e] = 0.0f;
  }
  Taps<W, V> taps;
  taps.load(p, d);
  const int64_t step = (int64_t)parts * groups * run;
  for (int64_t first = ((int64_t)part * groups + at.grp) * run; at.any && first < p.tokens; first += step) {
    const int32_t t0 = (int32_t)first, t1 = p.tokens - t0 < run ? p.tokens : t0 + run;
    SeqWalk q;
    q.start(s, t0);
    float old[W - 1][V], pend[W - 1][V];   // pend: dx of the W - 1 tokens before, without what comes after
    load_before<DT, W, V>(p, q.i, t0 > q.b && t0 < q.e ? q.b : t0, t0, d, old);
#pragma unroll
    for (int j = 0; j < W - 1; ++j)
#pragma unroll
      for (int e = 0; e < V; ++e) pend[j][e] = 0.0f;
    // adds du of token t to the sums, stores dx of the token W - 1 before and starts that of t
    auto add = [&](int32_t t, const float* du) {
      float last[V];
#pragma unroll
      for (int o = W - 1; o >= 1; --o)
        if (o <= t - q.b) {
#pragma unroll
          for (int e = 0; e < V; ++e) pend[W - 1 - o][e] = fmaf(taps.w[W - 1 - o][e], du[e], pend[W - 1 - o][e]);
        }
#pragma unroll
      for (int e = 0; e < V; ++e) last[e] = taps.w[W - 1][e] * du[e];
      const int32_t from_end = t - (q.e - (W - 1));   // its row of the final state
      if (p.dfin && from_end >= 0 && t < q.e) {
        float g[V];
        load_state_any<V>(p.dfin, p.dfin_dtype, ((size_t)q.i * (W - 1) + from_end) * p.D + d, g);
#pragma unroll
        for (int e = 0; e < V; ++e) last[e] += g[e];
      }
      const int32_t done = t - (W - 1);
      if (done >= t0 && done >= lo && done < hi) {
        Pack<DT, V> out;
        out.pack(pend[0]);
        store_any(out, p.out, (size_t)done * p.D + d);
      }
      shift<V, W - 1>(pend, last);
    };
    const float none[V] = {};
    Pack<DT, V> nx[BWD_BATCH], ny[BWD_BATCH];
    auto load = [&](int32_t t) {
#pragma unroll
      for (int r = 0; r < BWD_BATCH; ++r)
        if (t + r < t1) {
          load_any(nx[r], p.x, (size_t)(t + r) * p.D + d);
          load_any(ny[r], p.dy, (size_t)(t + r) * p.D + d);
        }
    };
    for (int32_t t = t0; t < t1; t += BWD_BATCH) {
      load(t);
#pragma unroll
      for (int r = 0; r < BWD_BATCH; ++r) {
        if (t + r >= t1) break;
        if (t + r >= q.e) q.forward(s, t + r);
        if (t + r == q.b) load_before<DT, W, V>(p, q.i, q.b, q.b, d, old);
        if (!q.holds(t + r)) {
          add(t + r, none);
          continue;
        }
        float f[V], u[V], g[V];
        nx[r].unpack(f);
        ny[r].unpack(g);
        taps.apply(old, f, u);
        if (p.silu) {
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] = grad_of(u[e], g[e]);
        }
#pragma unroll
        for (int e = 0; e < V; ++e) {
          db[e] += g[e];
#pragma unroll
          for (int j = 0; j < W - 1; ++j) dw[j][e] = fmaf(g[e], old[j][e], dw[j][e]);
          dw[W - 1][e] = fmaf(g[e], f[e], dw[W - 1][e]);
        }
        shift<V, W - 1>(old, f);
        add(t + r, g);
      }
    }
    // the W - 1 tokens after the run, as far as they belong to the sequence of its last token
#pragma unroll
    for (int r = 0; r < W - 1; ++r) {
      const int32_t t = t1 + r;
      float g[V];
#pragma unroll
      for (int e = 0; e < V; ++e) g[e] = 0.0f;
      if (q.holds(t)) {
        float f[V], u[V];
        load_any_f32<DT, V>(p.x, (size_t)t * p.D + d, f);
        load_any_f32<DT, V>(p.dy, (size_t)t * p.D + d, g);
        taps.apply(old, f, u);
        if (p.silu) {
#pragma unroll
          for (int e = 0; e < V; ++e) g[e] = grad_of(u[e], g[e]);
        }
        shift<V, W - 1>(old, f);
      }
      add(t, g);
    }
  }
  if (!p.partial) return;
  float* mine = sums + threadIdx.x * (K + 1);   // odd stride: no bank conflicts
#pragma unroll
  for (int e = 0; e < V; ++e) {
#pragma unroll
    for (int j = 0; j < W; ++j) mine[j * V + e] = dw[j][e];
    mine[W * V + e] = db[e];
  }
  __syncthreads();
  const int lr = 1 << lr_log;
  for (int i = threadIdx.x; i < lr * K; i += 256) {
    const int k = i / (lr * V), ch = i - k * (lr * V), lane = ch / V, e = ch - lane * V;   // channels side by side
    int64_t dd = (((int64_t)col << lr_log) + lane) * V;   // that lane's first channel
    if (dd >= p.D) continue;
    dd = (dd + V <= p.D ? dd : p.D - V) + e;
    float v = 0.0f;
    for (int g = 0; g < groups; ++g) v += sums[(g * lr + lane) * (K + 1) + k * V + e];
    p.partial[((size_t)part * (W + 1) + k) * p.D + dd] = v;
  }
}

// d_weight and d_bias from the parts: 64 columns of the [W + 1][D] sums, 16 runs of parts
template <int W>
__global__ __launch_bounds__(1024) void kda_conv_sum_kernel(ConvParams p, int parts) {
  __shared__ float buf[16][64];
  const int64_t col = (int64_t)blockIdx.x * 64 + (threadIdx.x & 63);
  const int run = threadIdx.x >> 6;
  const int64_t width = (int64_t)(W + 1) * p.D;
  float v = 0.0f;
  if (col < width) {
#pragma unroll 8
    for (int i = run; i < parts; i += 16) v += p.partial[(size_t)i * width + col];
  }
  buf[run][threadIdx.x & 63] = v;
  __syncthreads();
  if (run != 0 || col >= width) return;
#pragma unroll
  for (int i = 1; i < 16; ++i) v += buf[i][threadIdx.x];
  const int k = (int)(col / p.D);
  const int64_t d = col - (int64_t)k * p.D;
  if (k < W) {
    if (p.dw) p.dw[d * W + k] = v;
  } else if (p.db) {
    p.db[d] = v;
  }
}

// ---- launches ---------------------------------------------------------------------

// f(type, W)
template <typename F>
void dispatch(const ConvParams& p, F f) {
  auto with_type = [&](auto dt) {
    if (p.W == 2) f(dt, integral_constant<int, 2>{});
    else if (p.W == 3) f(dt, integral_constant<int, 3>{});
    else f(dt, integral_constant<int, 4>{});
  };
  if (p.dtype == BF16) with_type(integral_constant<int, BF16>{});
  else if (p.dtype == FP32) with_type(integral_constant<int, FP32>{});
  else with_type(integral_constant<int, FP16>{});
}

// Lanes across the channels (at most a wave), workgroups across them, tokens of a run, and, of
// the backward pass, workgroups along the tokens.
struct Grid {
  int lr_log, cols, run;
  int64_t blocks;   // along the tokens
};
Grid grid_of(int64_t tokens, int64_t D, int V, int most_run) {
  Grid g;
  const int64_t vecs = (D + V - 1) / V;
  g.lr_log = 3;
  while (g.lr_log < 6 && (1 << g.lr_log) < vecs) ++g.lr_log;
  g.cols = (int)((vecs + (1 << g.lr_log) - 1) >> g.lr_log);
  const int groups = 256 >> g.lr_log;
  g.run = most_run;
  auto count = [&]() { return (tokens + (int64_t)groups * g.run - 1) / ((int64_t)groups * g.run); };
  while (g.run > BATCH && count() * g.cols < 1024) g.run /= 2;
  g.blocks = count();
  return g;
}

constexpr int64_t FWD_RUN = 32, BWD_RUN = 32;
// Channels of a lane backward: with 8 of 16 bits each it takes 256 registers, one wave to a SIMD
constexpr int BWD_VEC = 4;

int64_t parts_of(int64_t tokens, int64_t D, int V) {
  const Grid g = grid_of(tokens, D, V, BWD_RUN);
  const int64_t most = (1024 + g.cols - 1) / g.cols;
  return g.blocks < most ? g.blocks : most;
}

unsigned state_blocks(int64_t n) { return (unsigned)((n + 255) / 256 < 16384 ? (n + 255) / 256 : 16384); }

}  // namespace

bool conv_fits(int64_t tokens, int64_t D) {
  const Grid g = grid_of(tokens, D, D < 8 ? 1 : 4, FWD_RUN);   // (the most workgroups of all types)
  return g.blocks < (1 << 24) && g.blocks * g.cols < (1 << 24) - 16384;   // (and 16384 for the states)
}

size_t conv_workspace(int64_t tokens, int64_t D, int64_t W) {
  if (tokens == 0) return 0;
  int64_t most = 0;   // whatever the type
  for (int V : {1, BWD_VEC}) {
    const int64_t n = parts_of(tokens, D, V);
    if ((V == 1 || D >= V) && n > most) most = n;
  }
  return (size_t)most * (size_t)(W + 1) * (size_t)D * sizeof(float);
}

// Token tensors are taken in vectors of 16 bytes at any alignment, rows of fewer channels one by
// one. States in vectors only where they are whole ones: what overlaps would be read by one lane
// after another has written it. The first workgroups write the states beside the others (a launch
// of their own took 5 us, 7 backward), except where final states overwrite the initial ones that
// the others read.
hipError_t launch_conv_fwd(const ConvParams& p, hipStream_t stream) {
  dispatch(p, [&](auto dt, auto w) {
    constexpr int DT = decltype(dt)::value, W = decltype(w)::value, V = vec_of<DT>();
    auto go = [&](auto v) {
      constexpr int N = decltype(v)::value;
      const unsigned states = p.fin ? state_blocks((int64_t)p.nseq * p.D / (p.D % N == 0 ? N : 1)) : 0;
      const bool apart = p.fin == p.init || p.tokens == 0;
      if (p.tokens > 0) {
        const Grid g = grid_of(p.tokens, p.D, N, FWD_RUN);
        const unsigned beside = apart ? 0 : states;
        hipLaunchKernelGGL((kda_conv_fwd_kernel<DT, W, N>), dim3((unsigned)(g.blocks * g.cols) + beside), dim3(256), 0, stream, p,
                           g.lr_log, g.cols, g.run, (int)beside);
      }
      if (apart && states > 0) hipLaunchKernelGGL((kda_conv_final_kernel<DT, W, N>), dim3(states), dim3(256), 0, stream, p);
    };
    if (p.D >= V) go(integral_constant<int, V>{});
    else go(integral_constant<int, 1>{});
  });
  return hipGetLastError();
}

hipError_t launch_conv_bwd(const ConvParams& p, hipStream_t stream) {
  dispatch(p, [&](auto dt, auto w) {
    constexpr int DT = decltype(dt)::value, W = decltype(w)::value;
    int parts = 0;
    auto go = [&](auto v) {
      constexpr int N = decltype(v)::value;
      const unsigned states = p.dinit ? state_blocks((int64_t)p.nseq * p.D / (p.D % N == 0 ? N : 1)) : 0;
      const Grid g = grid_of(p.tokens, p.D, N, BWD_RUN);
      if (p.tokens > 0) parts = (int)parts_of(p.tokens, p.D, N);
      const unsigned blocks = (unsigned)parts * g.cols + states;
      if (blocks > 0)
        hipLaunchKernelGGL((kda_conv_bwd_kernel<DT, W, N>), dim3(blocks), dim3(256), 0, stream, p, g.lr_log, g.cols, g.run, parts,
                           (int)states);
    };
    if (p.D >= BWD_VEC) go(integral_constant<int, BWD_VEC>{});
    else go(integral_constant<int, 1>{});
    if (p.dw || p.db)
      hipLaunchKernelGGL((kda_conv_sum_kernel<W>), dim3((unsigned)(((int64_t)(W + 1) * p.D + 63) / 64)), dim3(1024), 0, stream, p, parts);
  });
  return hipGetLastError();
}

hipError_t launch_conv_step(const ConvParams& p, hipStream_t stream) {
  if (p.nseq == 0) return hipSuccess;
  dispatch(p, [&](auto dt, auto w) {
    constexpr int DT = decltype(dt)::value, W = decltype(w)::value, V = vec_of<DT>();
    auto go = [&](auto v) {
      constexpr int N = decltype(v)::value;
      hipLaunchKernelGGL((kda_conv_step_kernel<DT, W, N>), dim3(state_blocks((int64_t)p.nseq * p.D / N)), dim3(256), 0, stream, p,
                         p.D / N);
    };
    if (p.D % V == 0) go(integral_constant<int, V>{});
    else go(integral_constant<int, 1>{});
  });
  return hipGetLastError();
}

}  // namespace kda
