// kda_elem.h -- loads and stores of a few neighbouring elements of bf16, fp32 or fp16
// tensors as fp32, for the kernels that take all three (kda_glr*.hip, kda_layernorm.hip).
#pragma once

#include "kda_device.h"

namespace kda {

// element types (KDA_BF16, KDA_FP32, KDA_FP16 of the public header; the first two are also
// the state codes)
constexpr int BF16 = 1, FP32 = 2, FP16 = 3;
constexpr int elem_size(int dt) { return dt == FP32 ? 4 : 2; }

template <int BYTES>
struct RawOf;
template <>
struct RawOf<2> { using type = uint16_t; };
template <>
struct RawOf<4> { using type = uint32_t; };
template <>
struct RawOf<8> { using type = u32x2; };
template <>
struct RawOf<16> { using type = u32x4; };

template <int DT>
__device__ __forceinline__ float elem_to_f32(uint16_t h) {
  if constexpr (DT == BF16) return bf16_to_f32(h);
  else return (float)__builtin_bit_cast(_Float16, h);
}

// N neighbouring elements of type DT as they lie in memory (at most 16 bytes, aligned to
// their size)
template <int DT, int N>
struct Pack {
  using Raw = typename RawOf<N * elem_size(DT)>::type;
  Raw r;

  __device__ __forceinline__ void load(const void* p, size_t i) {
    r = *reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p) + i * elem_size(DT));
  }
  // at byte `uniform` (the same in every lane) plus a lane's 32-bit offset
  __device__ __forceinline__ void load_at(const void* p, size_t uniform, uint32_t lane) {
    r = *reinterpret_cast<const Raw*>(static_cast<const uint8_t*>(p) + uniform + lane);
  }
  __device__ __forceinline__ void store_at(void* p, size_t uniform, uint32_t lane) const {
    *reinterpret_cast<Raw*>(static_cast<uint8_t*>(p) + uniform + lane) = r;
  }
  // the compiler forgets what it has computed from these registers
  __device__ __forceinline__ void opaque() { asm volatile("" : "+v"(r)); }
  __device__ __forceinline__ void clear() { r = Raw{}; }

  __device__ __forceinline__ void unpack(float* f) const {
    if constexpr (DT == FP32) {
      if constexpr (N == 1) f[0] = __uint_as_float(r);
      else {
#pragma unroll
        for (int i = 0; i < N; ++i) f[i] = __uint_as_float(r[i]);
      }
    } else if constexpr (N == 1) {
      f[0] = elem_to_f32<DT>(r);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        uint32_t w;
        if constexpr (N == 2) w = r;
        else w = r[i];
        if constexpr (DT == BF16) {
          f[2 * i] = bf16_lo(w);
          f[2 * i + 1] = bf16_hi(w);
        } else {
          const f32x2 v = unpack_f16x2(w);
          f[2 * i] = v.x;
          f[2 * i + 1] = v.y;
        }
      }
    }
  }

  __device__ __forceinline__ void pack(const float* f) {
    if constexpr (DT == FP32) {
      if constexpr (N == 1) r = __float_as_uint(f[0]);
      else {
#pragma unroll
        for (int i = 0; i < N; ++i) r[i] = __float_as_uint(f[i]);
      }
    } else if constexpr (N == 1) {
      r = DT == BF16 ? to_bf16(f[0]) : to_f16(f[0]);
    } else {
#pragma unroll
      for (int i = 0; i < N / 2; ++i) {
        const uint32_t w = DT == BF16 ? pack_bf16x2(f[2 * i], f[2 * i + 1]) : pack_f16x2(f[2 * i], f[2 * i + 1]);
        if constexpr (N == 2) r = w;
        else r[i] = w;
      }
    }
  }

  __device__ __forceinline__ void store(void* p, size_t i) const {
    *reinterpret_cast<Raw*>(static_cast<uint8_t*>(p) + i * elem_size(DT)) = r;
  }
};

// elements c .. c + M - 1 of a pack: one 32-bit word of it, or its only element
template <int DT, int N, int M>
__device__ __forceinline__ void unpack_word(const Pack<DT, N>& q, int c, float* f) {
  Pack<DT, M> one;
  if constexpr (N == M) one.r = q.r;
  else one.r = q.r[c / M];
  one.unpack(f);
}
template <int DT, int N, int M>
__device__ __forceinline__ void pack_word(Pack<DT, N>& q, int c, const float* f) {
  Pack<DT, M> one;
  one.pack(f);
  if constexpr (N == M) q.r = one.r;
  else q.r[c / M] = one.r;
}

template <int DT, int N>
__device__ __forceinline__ void load_f32(const void* p, size_t i, float* f) {
  constexpr int M = N * elem_size(DT) > 16 ? 16 / elem_size(DT) : N;
#pragma unroll
  for (int j = 0; j < N; j += M) {
    Pack<DT, M> q;
    q.load(p, i + j);
    q.unpack(f + j);
  }
}

template <int DT, int N>
__device__ __forceinline__ void store_f32(void* p, size_t i, const float* f) {
  constexpr int M = N * elem_size(DT) > 16 ? 16 / elem_size(DT) : N;
#pragma unroll
  for (int j = 0; j < N; j += M) {
    Pack<DT, M> q;
    q.pack(f + j);
    q.store(p, i + j);
  }
}

// c elements (0 <= c <= VEC) from element i on, or from byte a on, zeros behind them, at any
// alignment (the hardware splits what crosses a line): a vector,
// or at most one load of 8, 4 and 2 bytes each (one element after the other, rows of 700 bf16
// elements took 1.5 times as long). EXACT: rows are whole vectors, and c is VEC.
template <bool EXACT, int DT, int VEC>
__device__ __forceinline__ void load_part(Pack<DT, VEC>& q, const uint8_t* a, int c) {
  if (EXACT || c >= VEC) {
    __builtin_memcpy(&q.r, a, 16);
    return;
  }
  if constexpr (DT == FP32) {
    q.r = u32x4{0u, 0u, 0u, 0u};
#pragma unroll
    for (int e = 0; e < VEC - 1; ++e)
      if (e < c) q.r[e] = reinterpret_cast<const uint32_t*>(a)[e];
    return;
  }
  // each piece goes straight to its registers: merging them here would wait for every row's
  // pieces before the next row's loads are issued
  auto w4 = [](const uint8_t* b) { uint32_t v; __builtin_memcpy(&v, b, 4); return v; };
  auto w2 = [](const uint8_t* b) { return (uint32_t)*reinterpret_cast<const uint16_t*>(b); };
  const int bytes = c * elem_size(DT);
  q.r = u32x4{0u, 0u, 0u, 0u};
  if (bytes & 8) {
    u32x2 v;
    __builtin_memcpy(&v, a, 8);
    q.r.x = v.x;
    q.r.y = v.y;
    if (bytes & 4) {
      q.r.z = w4(a + 8);
      if (bytes & 2) q.r.w = w2(a + 12);
    } else if (bytes & 2) {
      q.r.z = w2(a + 8);
    }
  } else if (bytes & 4) {
    q.r.x = w4(a);
    if (bytes & 2) q.r.y = w2(a + 4);
  } else if (bytes & 2) {
    q.r.x = w2(a);
  }
}
// STREAM: not kept in the caches, the inputs stay there instead
template <bool EXACT, bool STREAM = true, int DT, int VEC>
__device__ __forceinline__ void store_part(const Pack<DT, VEC>& q, uint8_t* a, int c) {
  if (EXACT || c >= VEC) {
    using Any = u32x4 __attribute__((aligned(2)));   // any alignment
    if (STREAM) __builtin_nontemporal_store(q.r, reinterpret_cast<Any*>(a));
    else *reinterpret_cast<Any*>(a) = q.r;
    return;
  }
  if constexpr (DT == FP32) {
#pragma unroll
    for (int e = 0; e < VEC - 1; ++e)
      if (e < c) reinterpret_cast<uint32_t*>(a)[e] = q.r[e];
    return;
  }
  const int bytes = c * elem_size(DT);
  const u32x2 head = {q.r.x, q.r.y}, rest = bytes & 8 ? u32x2{q.r.z, q.r.w} : head;
  if (bytes & 8) __builtin_memcpy(a, &head, 8);
  a += bytes & 8;
  if (bytes & 4) __builtin_memcpy(a, &rest, 4);
  if (bytes & 2) *reinterpret_cast<uint16_t*>(a + (bytes & 4)) = (uint16_t)(bytes & 4 ? rest.y : rest.x);
}
template <bool EXACT, int DT, int VEC>
__device__ __forceinline__ void load_part(Pack<DT, VEC>& q, const void* p, size_t i, int c) {
  load_part<EXACT>(q, static_cast<const uint8_t*>(p) + i * elem_size(DT), c);
}
template <bool EXACT, int DT, int VEC>
__device__ __forceinline__ void store_part(const Pack<DT, VEC>& q, void* p, size_t i, int c) {
  store_part<EXACT>(q, static_cast<uint8_t*>(p) + i * elem_size(DT), c);
}

// N elements of a state of dtype code sdt (0: zeros, BF16, FP32); the same branch in every lane
template <int N>
__device__ __forceinline__ void load_state(const void* p, int sdt, size_t i, float* f) {
  if (sdt == FP32) load_f32<FP32, N>(p, i, f);
  else if (sdt == BF16) load_f32<BF16, N>(p, i, f);
  else {
#pragma unroll
    for (int j = 0; j < N; ++j) f[j] = 0.0f;
  }
}
template <int N>
__device__ __forceinline__ void store_state(void* p, int sdt, size_t i, const float* f) {
  if (sdt == FP32) store_f32<FP32, N>(p, i, f);
  else if (sdt == BF16) store_f32<BF16, N>(p, i, f);
}

// the first c of them (EXACT: all; rows of another width are not aligned to vectors)
template <bool EXACT, int N>
__device__ __forceinline__ void load_state_part(const void* p, int sdt, size_t i, int c, float* f) {
  if (EXACT) {
    load_state<N>(p, sdt, i, f);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < c) load_state<1>(p, sdt, i + j, f + j);
  }
}
template <bool EXACT, int N>
__device__ __forceinline__ void store_state_part(void* p, int sdt, size_t i, int c, const float* f) {
  if (EXACT) {
    store_state<N>(p, sdt, i, f);
  } else {
#pragma unroll
    for (int j = 0; j < N; ++j)
      if (j < c) store_state<1>(p, sdt, i + j, f + j);
  }
}

}  // namespace kda
