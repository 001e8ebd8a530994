// kda_beam.hip -- beam search: the best continuations of every sequence's beams (gfx950).
//
//     score(b, v) = scores[b] + logits[b][v] - log sum_v' exp(logits[b][v'])
//
// A beam's logits are cut into pieces, one workgroup each, which holds its piece in registers: it
// is read once for the largest value, the sum of exponentials and the best k values. A second
// kernel, one workgroup a sequence, joins the beams' sums and picks the best k of all pieces'.
// Their time goes to the exponentials and to the steps that a workgroup takes one after the other
// (256 beams of 131072 bf16 logits: 54 us, of which reading is 13). Scores of different beams lie
// close together and their order is the result, so sums and scores are 64 bits (an fp64 operation
// takes twice an fp32 one's time here; the exponential of 18 of them is good to 1e-11, so beams
// closer than that may change places).
//
// The best k are found by counting, not by sorting: the 256 lanes form k' >= k groups, each with
// its best element, and the least of those k' is a threshold that at least k elements reach, about
// k' ln k' of them as a rule. Those go to shared memory, where each counts the ones before it:
// its place among the results. Keys hold the value and, below it, the index, so no two are equal,
// and what is chosen does not depend on the order in which lanes run. Where more elements than
// shared memory holds reach the threshold, it is raised by bisection.
#include <type_traits>

#include "kda_elem.h"
#include "kda_ops.h"

namespace kda {
namespace {

using std::integral_constant;

constexpr int HOLD = 512;   // elements that may reach the threshold

// bits that grow with the number, the same for both zeros (-0.0 + 0.0 is +0.0); 0 is below all of them
__device__ __forceinline__ uint32_t ordered(float f) {
  const uint32_t u = __float_as_uint(f + 0.0f);
  return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t u) { return __uint_as_float(u & 0x80000000u ? u & 0x7fffffffu : ~u); }
__device__ __forceinline__ uint64_t ordered(double f) {
  const uint64_t u = __builtin_bit_cast(uint64_t, f + 0.0);
  return u >> 63 ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ double unordered(uint64_t u) {
  return __builtin_bit_cast(double, u >> 63 ? u & ~(1ull << 63) : ~u);
}

// exp(t), t <= 0 or NaN: 2^n 2^f, |f| <= 1/2, a Taylor series of nine terms (7e-12). It is 0 below
// -745, as in 64 bits: masked elements add nothing, and a beam with one other element keeps its
// score to the last bit, which a finished beam's equals. (n stays a number of 32 bits.)
__device__ __forceinline__ double exp_below(double t) {
  t = t < -1100.0 ? -1100.0 : t;
  const double y = t * 1.4426950408889634074, n = __builtin_rint(y), f = (y - n) * 0.69314718055994530942;
  double s = 1.0 / 362880.0;
  s = fma(s, f, 1.0 / 40320.0);
  s = fma(s, f, 1.0 / 5040.0);
  s = fma(s, f, 1.0 / 720.0);
  s = fma(s, f, 1.0 / 120.0);
  s = fma(s, f, 1.0 / 24.0);
  s = fma(s, f, 1.0 / 6.0);
  s = fma(s, f, 0.5);
  s = fma(s, f, 1.0);
  s = fma(s, f, 1.0);
  return __builtin_ldexp(s, (int)n);
}

template <typename T>
__device__ __forceinline__ T from_lane(T v, int mask) {   // of lane ^ mask
  return __shfl_xor(v, mask, 64);
}

// A piece's results: [rows][pieces]
struct BeamWs {
  uint64_t* best;   // [k] keys: value and ~index; 0 where there are fewer
  double* sum;      // of exp(value - top)
  float* top;       // largest value; NaN where one is NaN or +infinity
  int32_t pieces;
  int32_t size;     // elements of a piece
  int32_t groups;   // k': a power of two from 4 to 64, at least k
};

// Least of the groups' largest keys, as KEY has them (an operator > and a zero); the same in all
// lanes. A group is every groups-th lane, so that elements that fill only some of the lanes, as a
// vocabulary's last ones, reach all groups. buf: 256 keys
template <typename KEY>
__device__ __forceinline__ KEY threshold(KEY most, int groups, KEY* buf) {
  const int lane = threadIdx.x & 63;
  for (int o = groups; o < 64; o <<= 1) {
    const KEY other = most.from(o);
    if (other > most) most = other;
  }
  buf[threadIdx.x] = most;
  __syncthreads();
  KEY least = buf[lane];
#pragma unroll
  for (int w = 1; w < 4; ++w)
    if (buf[w * 64 + lane] > least) least = buf[w * 64 + lane];
  for (int o = 1; o < groups; o <<= 1) {
    const KEY other = least.from(o);
    if (least > other) least = other;
  }
  __syncthreads();
  return least;
}

// Sum of v over the workgroup, in all lanes. buf: 4
template <typename T>
__device__ __forceinline__ T wg_sum(T v, T* buf) {
  for (int o = 1; o < 64; o <<= 1) v += from_lane(v, o);
  __syncthreads();
  if ((threadIdx.x & 63) == 0) buf[threadIdx.x >> 6] = v;
  __syncthreads();
  return (buf[0] + buf[1]) + (buf[2] + buf[3]);
}

struct Key64 {
  uint64_t v;
  __device__ __forceinline__ bool operator>(const Key64& o) const { return v > o.v; }
  __device__ __forceinline__ Key64 from(int mask) const { return {from_lane(v, mask)}; }
};

// PER elements of a lane. A workgroup takes a piece of 256 PER elements of a beam's logits.
template <int DT, int PER>
__global__ __launch_bounds__(256, 4) void kda_beam_piece_kernel(BeamParams p, BeamWs w) {
  constexpr int VEC = 16 / elem_size(DT), NV = PER / VEC;
  __shared__ Key64 s_group[256];
  __shared__ uint64_t s_keys[HOLD];
  __shared__ double s_sum[4];
  __shared__ int s_count[4], s_used;
  __shared__ float s_top[4];
  const int tid = threadIdx.x, lane = tid & 63, wave = tid >> 6;
  const int64_t items = (int64_t)p.N * p.W * w.pieces;
  for (int64_t it = blockIdx.x; it < items; it += gridDim.x) {
    const int64_t row = it / w.pieces;
    const int first = (int)(it - row * w.pieces) * 256 * PER;
    if (p.finished && p.finished[row] != 0) continue;   // the same in all lanes
    Pack<DT, VEC> raw[NV];
#pragma unroll
    for (int i = 0; i < NV; ++i) {
      const int at = first + (i * 256 + tid) * VEC;
      raw[i].clear();
      if (at < p.V) load_part<false>(raw[i], p.logits, (size_t)row * p.V + at, p.V - at < VEC ? p.V - at : VEC);
    }
#pragma unroll
    for (int i = 0; i < NV; ++i) {   // nothing behind the last element
      const int at = first + (i * 256 + tid) * VEC;
      if (at + VEC > p.V) {
        float f[VEC];
        raw[i].unpack(f);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f[e] = at + e < p.V ? f[e] : -INFINITY;
        raw[i].pack(f);
      }
    }
    // f(value, index) for the lane's elements in order of their index. They are kept as they lie in
    // memory and taken apart again each time: kept as fp32, or as keys, they would take the registers
    // of all but one wave.
    auto each = [&](auto f) {
      int from = first + tid * VEC;
      asm volatile("" : "+v"(from));   // indices are formed anew each time as well
#pragma unroll
      for (int i = 0; i < NV; ++i) {
        float x[VEC];
        raw[i].opaque();
        raw[i].unpack(x);
#pragma unroll
        for (int e = 0; e < VEC; ++e) f(x[e], from + i * 256 * VEC + e);
        __builtin_amdgcn_sched_barrier(0);
      }
    };
    float own = -INFINITY;
    int own_at = 0;
    each([&](float x, int at) {
      if (x > own) {
        own = x;
        own_at = at;
      }
    });
    float top = own;
    for (int o = 1; o < 64; o <<= 1) top = fmaxf(top, from_lane(top, o));
    __syncthreads();   // the item before has been read
    if (lane == 0) s_top[wave] = top;
    if (tid == 0) s_used = 0;
    __syncthreads();
    top = fmaxf(fmaxf(s_top[0], s_top[1]), fmaxf(s_top[2], s_top[3]));
    double sum = 0.0;   // NaN where an element is NaN or +infinity
    const double dtop = (double)top;
    each([&](float x, int) { sum += exp_below((double)x - dtop); });
    sum = wg_sum(sum, s_sum);
    if (!(top > -INFINITY) || sum != sum) {   // no continuation here: all masked, or one is no number
      bool bad = false;
      each([&](float x, int) { bad = bad || !(x < INFINITY); });
      const bool any = __syncthreads_or(bad);
      if (tid == 0) {
        w.top[it] = any ? __uint_as_float(0x7fc00000u) : -INFINITY;
        w.sum[it] = 0.0;
      }
      for (int i = tid; i < p.k; i += 256) w.best[it * p.k + i] = 0;
      continue;
    }
    auto key_of = [](float x, int at) { return x == -INFINITY ? 0ull : ((uint64_t)ordered(x) << 32) | (uint32_t)~at; };
    uint64_t least = threshold(Key64{key_of(own, own_at)}, w.groups, s_group).v;
    if (least == 0) least = 1;
    // those that reach it to shared memory; returns how many there are, held or not
    auto gather = [&]() {
      const float from = least == 1 ? -INFINITY : unordered((uint32_t)(least >> 32));
      each([&](float x, int at) {
        if (x >= from) {
          const uint64_t q = key_of(x, at);
          if (q >= least) {
            const int to = atomicAdd(&s_used, 1);
            if (to < HOLD) s_keys[to] = q;
          }
        }
      });
      __syncthreads();
      return s_used;
    };
    int count = gather();
    if (count > HOLD) {
      auto reach = [&](uint64_t t) {   // elements with keys of t and more
        int n = 0;
        each([&](float x, int at) { n += key_of(x, at) >= t; });
        return wg_sum(n, s_count);
      };
      for (uint64_t high = ~0ull; count > HOLD;) {   // reach(least) >= k > reach(high)
        const uint64_t mid = least + (high - least) / 2;
        const int n = reach(mid);
        if (n >= p.k) {
          least = mid;
          count = n;
        } else {
          high = mid;
        }
      }
      if (tid == 0) s_used = 0;
      __syncthreads();
      gather();
    }
    for (int i = tid; i < count; i += 256) {
      const uint64_t q = s_keys[i];
      int place = 0;
      for (int j = 0; j < count; ++j) place += s_keys[j] > q;
      if (place < p.k) w.best[it * p.k + place] = q;
    }
    for (int i = count + tid; i < p.k; i += 256) w.best[it * p.k + i] = 0;
    if (tid == 0) {
      w.top[it] = top;
      w.sum[it] = sum;
    }
  }
}

struct Key96 {
  uint64_t s;   // score
  uint32_t i;   // ~(beam V + token)
  __device__ __forceinline__ bool operator>(const Key96& o) const { return s > o.s || (s == o.s && i > o.i); }
  __device__ __forceinline__ Key96 from(int mask) const { return {from_lane(s, mask), from_lane(i, mask)}; }
};

// A logit of a tensor of any type
__device__ __forceinline__ float logit_of(const BeamParams& p, size_t i) {
  float x;
  if (p.dtype == BF16) load_f32<BF16, 1>(p.logits, i, &x);
  else if (p.dtype == FP32) load_f32<FP32, 1>(p.logits, i, &x);
  else load_f32<FP16, 1>(p.logits, i, &x);
  return x;
}

// The pieces' best ones go by their logits. Where different logits have one score (64 bits of a beam's
// score of -1e30, or of the sum, swallow what tells them apart), a piece may so have kept larger logits
// in the place of lower tokens. That matters at the k-th score alone: fewer than k are above it, and
// those are all in their pieces' lists. A list that ends with that score, and whose last logit has a
// neighbour in fp32 of the same score, is the sign of it (no list ends above the k-th score): the
// continuations with the k-th score are then taken from the logits themselves, in order, until there
// are k. (32 x 8 beams of 131072 bf16 tokens, of which all but one do not count: 76 us a call, 60 where all do.)
__global__ __launch_bounds__(256) void kda_beam_join_kernel(BeamParams p, BeamWs w) {
  __shared__ double s_top[64], s_log[64], s_score[64];
  __shared__ bool s_none[64], s_done[64];
  __shared__ Key96 s_group[256], s_keys[HOLD];
  __shared__ unsigned long long s_kth, s_lost;
  __shared__ int s_count[4], s_used, s_above;
  const int tid = threadIdx.x, n = blockIdx.x, lane = tid & 63;
  if (tid == 0) {
    s_used = 0;
    s_kth = s_lost = 0;
    s_above = 0;
  }
  for (int b = tid >> 6; b < p.W; b += 4) {   // a wave: a beam's sum over its pieces
    const int64_t row = (int64_t)n * p.W + b, at = row * w.pieces;
    const bool done = p.finished && p.finished[row] != 0;
    double top = -INFINITY, sum = 0.0;
    bool bad = false;
    if (!done) {
      for (int i = lane; i < w.pieces; i += 64) {
        const float t = w.top[at + i];
        bad = bad || t != t;
        top = t > top ? t : top;
      }
      for (int o = 1; o < 64; o <<= 1) {
        const double t = from_lane(top, o);
        top = t > top ? t : top;
      }
      bad = __any(bad) || top == -INFINITY;
      if (!bad)
        for (int i = lane; i < w.pieces; i += 64) {
          const float t = w.top[at + i];
          if (t != -INFINITY) sum += w.sum[at + i] * exp_below((double)t - top);
        }
      for (int o = 1; o < 64; o <<= 1) sum += from_lane(sum, o);
    }
    if (lane == 0) {
      const float sc = p.scores[row];
      s_top[b] = top;
      s_log[b] = done || bad ? 0.0 : log(sum);
      s_score[b] = (double)sc;
      s_none[b] = bad || !(fabsf(sc) < INFINITY);
      s_done[b] = done;
    }
  }
  __syncthreads();
  // the pieces' best ones first, then their second ones: neighbouring lanes, and so all groups of a
  // threshold, have candidates of the same rank (in the order of the pieces, where a lane's group was
  // the rank, the kernel took 31 us at 32 x 8 beams and not 11)
  const int lists = p.W * w.pieces, total = lists * p.k;
  auto score = [&](int b, float x) { return ordered((((double)x - s_top[b]) - s_log[b]) + s_score[b]); };
  uint64_t lost = 0;   // best score at the end of a list that may have left out others with it
  auto key = [&](int i, auto first) -> Key96 {   // first: its list's end is looked at
    const int j = i / lists, list = i - j * lists, b = list / w.pieces;
    if (s_none[b]) return {0, 0};
    if (s_done[b]) return j == 0 && list == b * w.pieces ? Key96{ordered(s_score[b]), ~((uint32_t)b * p.V + p.eos)} : Key96{0, 0};
    const uint64_t q = w.best[((int64_t)n * lists + list) * p.k + j];
    if (q == 0) return {0, 0};
    const uint32_t x = (uint32_t)(q >> 32);
    const uint64_t v = score(b, unordered(x));
    if (decltype(first)::value && j == p.k - 1 && v > lost &&
        (score(b, unordered(x - 1)) == v || score(b, unordered(x + 1)) == v)) lost = v;
    return {v, ~((uint32_t)b * p.V + ~(uint32_t)q)};
  };
  constexpr int HELD = 8;   // keys of a lane that are kept, where that is all of them: formed once
  const bool held = total <= 256 * HELD;
  Key96 own[HELD];
  auto each = [&](auto f) {
    if (held) {
#pragma unroll
      for (int j = 0; j < HELD; ++j) f(own[j]);
    } else {
      for (int i = tid; i < total; i += 256) f(key(i, std::false_type{}));
    }
  };
  if (held) {
#pragma unroll
    for (int j = 0; j < HELD; ++j) own[j] = tid + 256 * j < total ? key(tid + 256 * j, std::true_type{}) : Key96{0, 0};
  }
  Key96 most{0, 0};
  auto better = [&](const Key96& q) {
    if (q > most) most = q;
  };
  if (held) each(better);
  else
    for (int i = tid; i < total; i += 256) better(key(i, std::true_type{}));
  if (lost != 0) atomicMax(&s_lost, (unsigned long long)lost);
  Key96 least = threshold(most, w.groups, s_group);
  if (least.s == 0) least = {1, 0};
  auto gather = [&]() {   // as in a piece
    each([&](const Key96& q) {
      if (!(least > q)) {
        const int to = atomicAdd(&s_used, 1);
        if (to < HOLD) s_keys[to] = q;
      }
    });
    __syncthreads();
    return s_used;
  };
  int count = gather();
  if (count > HOLD) {   // reach(least) >= k > reach({high, 0}): first by the score, then by the index
    auto reach = [&](const Key96& t) {
      int c = 0;
      each([&](const Key96& q) { c += !(t > q); });
      return wg_sum(c, s_count);
    };
    uint64_t high = ~0ull;
    while (count > HOLD && high - least.s > 1) {
      const Key96 mid{least.s + (high - least.s) / 2, 0};
      const int c = reach(mid);
      if (c >= p.k) {
        least = mid;
        count = c;
      } else {
        high = mid.s;
      }
    }
    uint64_t up = 1ull << 32;   // reach({least.s, up}) < k
    while (count > HOLD) {
      const Key96 mid{least.s, (uint32_t)(least.i + (up - least.i) / 2)};
      const int c = reach(mid);
      if (c >= p.k) {
        least = mid;
        count = c;
      } else {
        up = mid.i;
      }
    }
    if (tid == 0) s_used = 0;
    __syncthreads();
    gather();
  }
  auto put = [&](int place, const Key96& q) {
    const uint32_t at = ~q.i;
    const int64_t to = (int64_t)n * p.k + place;
    p.tokens[to] = (int32_t)(at % (uint32_t)p.V);
    p.parents[to] = (int32_t)(at / (uint32_t)p.V);
    p.new_scores[to] = (float)unordered(q.s);
  };
  for (int i = tid; i < count; i += 256) {
    const Key96 q = s_keys[i];
    int place = 0;
    for (int j = 0; j < count; ++j) place += s_keys[j] > q;
    if (place < p.k) put(place, q);
    if (place == p.k - 1) s_kth = q.s;
  }
  for (int i = count + tid; i < p.k; i += 256) {
    const int64_t to = (int64_t)n * p.k + i;
    p.tokens[to] = p.parents[to] = -1;
    p.new_scores[to] = -INFINITY;
  }
  if (s_lost == 0) return;
  __syncthreads();
  const uint64_t kth = s_kth;
  if (s_lost != kth) return;   // (0 where there are fewer than k: none was left out)
  int above = 0;
  for (int i = tid; i < count; i += 256) above += s_keys[i].s > kth;
  if (above > 0) atomicAdd(&s_above, above);
  __syncthreads();
  int place = s_above;   // of the next one, the same in all lanes
  for (int list = 0; list < lists && place < p.k; ++list) {
    const int b = list / w.pieces, first = (list - b * w.pieces) * w.size;
    if (s_none[b]) continue;
    if (s_done[b]) {
      if (first != 0 || ordered(s_score[b]) != kth) continue;
      if (tid == 0) put(place, {kth, ~((uint32_t)b * p.V + p.eos)});
      ++place;
      continue;
    }
    bool some = false;   // (a piece without one in its list has none)
    for (int j = tid; j < p.k; j += 256) some = some || key(j * lists + list, std::false_type{}).s == kth;
    if (!__syncthreads_or(some)) continue;
    const int end = p.V - first < w.size ? p.V : first + w.size;
    for (int v0 = first; v0 < end && place < p.k; v0 += 256) {
      const int v = v0 + tid;
      const float x = v < end ? logit_of(p, ((size_t)n * p.W + b) * p.V + v) : -INFINITY;
      const bool hit = x > -INFINITY && score(b, x) == kth;
      const uint64_t hits = __ballot(hit);
      __syncthreads();   // the counts before have been read
      if (lane == 0) s_count[tid >> 6] = __popcll(hits);
      __syncthreads();
      int to = place + __popcll(hits & (((uint64_t)1 << lane) - 1));
#pragma unroll
      for (int i = 0; i < 4; ++i) {
        if (i < tid >> 6) to += s_count[i];
        place += s_count[i];
      }
      if (hit && to < p.k) put(to, {kth, ~((uint32_t)b * p.V + (uint32_t)v)});
    }
  }
}

template <typename F>
void by_dtype(int dt, F f) {
  if (dt == BF16) f(integral_constant<int, BF16>{});
  else if (dt == FP32) f(integral_constant<int, FP32>{});
  else f(integral_constant<int, FP16>{});
}

// Elements of a lane: many, or few where the GPU would not be filled so.
int per_lane(int64_t rows, int64_t V) { return rows * ((V + 256 * 32 - 1) / (256 * 32)) >= 512 ? 32 : 8; }

size_t lay_out(BeamWs& w, uint8_t* at, int64_t items, int64_t k) {
  size_t used = 0;
  auto take = [&](size_t bytes) {
    uint8_t* r = at ? at + used : nullptr;
    used += (bytes + 255) / 256 * 256;
    return r;
  };
  w.best = reinterpret_cast<uint64_t*>(take((size_t)items * k * sizeof(uint64_t)));
  w.sum = reinterpret_cast<double*>(take((size_t)items * sizeof(double)));
  w.top = reinterpret_cast<float*>(take((size_t)items * sizeof(float)));
  return used;
}

}  // namespace

// Room for what any call of at most this size takes (few rows have four times as many pieces): a
// workspace for the largest batch serves the smaller ones.
size_t beam_workspace(int64_t N, int64_t W, int64_t V, int64_t k) {
  const int64_t rows = N * W, many = rows * ((V + 256 * 32 - 1) / (256 * 32)), few = rows * ((V + 256 * 8 - 1) / (256 * 8));
  const int64_t most_few = few < 4 * 511 ? few : 4 * 511;   // 8 elements a lane: less than 512 pieces of 32
  BeamWs w{};
  return lay_out(w, nullptr, many > most_few ? many : most_few, k);
}

hipError_t launch_beam_select(const BeamParams& p, void* workspace, hipStream_t stream) {
  if (p.N == 0) return hipSuccess;
  const int64_t rows = (int64_t)p.N * p.W;
  BeamWs w{};
  w.size = 256 * per_lane(rows, p.V);
  w.pieces = (int32_t)(((int64_t)p.V + w.size - 1) / w.size);
  w.groups = 4;
  while (w.groups < p.k) w.groups *= 2;
  const int64_t items = rows * w.pieces;
  lay_out(w, static_cast<uint8_t*>(workspace), items, p.k);
  const unsigned blocks = (unsigned)(items < 65536 ? items : 65536);
  by_dtype(p.dtype, [&](auto dt) {
    constexpr int DT = decltype(dt)::value;
    if (per_lane(rows, p.V) == 32)
      hipLaunchKernelGGL((kda_beam_piece_kernel<DT, 32>), dim3(blocks), dim3(256), 0, stream, p, w);
    else
      hipLaunchKernelGGL((kda_beam_piece_kernel<DT, 8>), dim3(blocks), dim3(256), 0, stream, p, w);
  });
  hipLaunchKernelGGL(kda_beam_join_kernel, dim3((unsigned)p.N), dim3(256), 0, stream, p, w);
  return hipGetLastError();
}

}  // namespace kda
