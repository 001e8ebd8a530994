// kda_api_util.h -- host-side helpers that the C ABI's sources share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdlib>
#include <initializer_list>

#include "../../include/kda.h"

namespace kda {

constexpr size_t ALIGN = 256;   // of workspaces and their regions
constexpr int64_t MAX_SLOTS = (int64_t)1 << 24;

inline size_t align_up(size_t x) { return (x + ALIGN - 1) / ALIGN * ALIGN; }
inline bool aligned(const void* p, size_t a) { return ((uintptr_t)p % a) == 0; }

inline bool env_flag(const char* name) {
  const char* s = std::getenv(name);
  return s && s[0] == '1';
}

// Copies the boundaries to the host in pieces through a stack buffer (no allocation).
inline int validate_cu_on_host(const int64_t* cu, int64_t N, int64_t T, hipStream_t stream) {
  if (hipStreamSynchronize(stream) != hipSuccess) return KDA_ERR_HIP;
  constexpr int64_t PIECE = 512;
  int64_t h[PIECE];
  int64_t prev = 0;
  for (int64_t i0 = 0; i0 <= N; i0 += PIECE) {
    const int64_t n = (N + 1 - i0) < PIECE ? (N + 1 - i0) : PIECE;
    if (hipMemcpy(h, cu + i0, sizeof(int64_t) * (size_t)n, hipMemcpyDeviceToHost) != hipSuccess) return KDA_ERR_HIP;
    for (int64_t i = 0; i < n; ++i) {
      if (i0 + i == 0 ? h[i] != 0 : h[i] < prev) return KDA_ERR_VALUE;
      prev = h[i];
    }
  }
  return prev == T ? KDA_OK : KDA_ERR_VALUE;
}

inline int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

inline bool bad_state_code(int c) { return c != KDA_STATE_NONE && c != KDA_STATE_BF16 && c != KDA_STATE_FP32; }
inline bool bad_dtype(int c) { return c != KDA_BF16 && c != KDA_FP32 && c != KDA_FP16; }

// A state's pointer and its dtype code: both given or neither.
inline int check_state(const void* p, int dtype) {
  if (bad_state_code(dtype)) return KDA_ERR_DTYPE;
  if ((dtype == KDA_STATE_NONE) != (p == nullptr)) return p ? KDA_ERR_DTYPE : KDA_ERR_NULL;
  return KDA_OK;
}

inline bool any_unaligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return true;
  return false;
}

// Whether a state of the recurrence is where the kernels can take it: an element at a time where
// rows are no whole vectors of the token tensors (layers of a cache begin anywhere then), else as
// many elements as such a vector holds.
inline bool state_unaligned(const void* p, int state_dtype, int dtype, int64_t D) {
  if (!p) return false;
  const int64_t vec = dtype == KDA_FP32 ? 4 : 8;
  const size_t elem = state_dtype == KDA_STATE_FP32 ? 4 : 2, all = (size_t)vec * elem;
  return !aligned(p, D % vec != 0 ? elem : all < 16 ? all : 16);
}

inline int check_pool(const void* pool, int64_t L, int64_t S, size_t slot_bytes, int64_t n) {
  if (!pool) return KDA_ERR_NULL;
  if (L < 1 || S < 1 || S > MAX_SLOTS || slot_bytes < 1 || n < 0 || n > INT32_MAX) return KDA_ERR_SHAPE;
  if (L > (int64_t)1 << 32 || (double)L * (double)S * (double)slot_bytes >= 4611686018427387904.0) return KDA_ERR_SHAPE;
  if (!aligned(pool, 16)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

}  // namespace kda
