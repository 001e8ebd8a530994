// kda_seq.h -- the sequences that packed tokens belong to: B rows of T tokens, or packed
// boundaries in device memory (kda_conv.hip, kda_ssm.hip).
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

namespace kda {

// Boundaries' contents are not trusted: clamped into the tokens, so that no access leaves them.
struct Seqs {
  const int64_t* cu;   // boundaries [n + 1], or NULL: rows of T tokens
  int32_t n;           // sequences
  int32_t T;           // tokens of a row; of all sequences with cu
  int32_t tokens;      // all tokens

  __device__ __forceinline__ int32_t begin(int i) const {   // 0 <= i <= n
    if (!cu) return i * T;
    const int64_t v = cu[i];
    return v < 0 ? 0 : v > tokens ? tokens : (int32_t)v;
  }
  // The last sequence that begins at or before token t (the first one where none does)
  __device__ __forceinline__ int find(int32_t t) const {
    if (!cu) return T > 0 ? (int)((uint32_t)t / (uint32_t)T) : 0;
    int lo = 0, hi = n - 1;
    while (lo < hi) {
      const int mid = (lo + hi + 1) >> 1;
      if (cu[mid] <= t) lo = mid;
      else hi = mid - 1;
    }
    return lo;
  }
};

// A place that moves along the tokens: sequence i holds tokens b .. e - 1, and token t is in it
// where b <= t < e.
struct SeqWalk {
  int32_t i, b, e;

  __device__ __forceinline__ void start(const Seqs& s, int32_t t) {
    i = s.find(t);
    b = s.begin(i);
    e = s.begin(i + 1);
  }
  // to the sequence of token t, from one before it
  __device__ __forceinline__ void forward(const Seqs& s, int32_t t) {
    while (t >= e && i + 1 < s.n) {
      ++i;
      b = e > s.begin(i) ? e : s.begin(i);
      e = s.begin(i + 1);
    }
  }
  // to the sequence of token t, from one after it
  __device__ __forceinline__ void back(const Seqs& s, int32_t t) {
    while (t < b && i > 0) {
      --i;
      e = b;
      b = s.begin(i);
    }
  }
  __device__ __forceinline__ bool holds(int32_t t) const { return t >= b && t < e; }
};

}  // namespace kda
