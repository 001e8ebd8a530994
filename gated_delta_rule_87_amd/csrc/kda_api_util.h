// kda_api_util.h -- host-side helpers that the C ABI's sources share.
#pragma once

#include <hip/hip_runtime.h>

#include <cstdint>
#include <cstdlib>

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

}  // namespace kda
