// kda_ops_api.cpp -- C ABI of the operators beside kda_fwd: argument checks, workspace
// layout and launches of the gated linear recurrence, layer norm and the cache of states.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>
#include <initializer_list>

#include "../../include/kda.h"
#include "kda_api_util.h"
#include "kda_internal.h"
#include "kda_ops.h"

namespace {

using kda::aligned;

using kda::MAX_SLOTS;
constexpr int64_t MAX_D = (int64_t)1 << 24;          // of a row of layer norm
constexpr int64_t MAX_CHANNELS = (int64_t)1 << 22;   // of the recurrence: 32-bit offsets inside a tile

bool bad_state_code(int c) { return c != KDA_STATE_NONE && c != KDA_STATE_BF16 && c != KDA_STATE_FP32; }
bool bad_dtype(int c) { return c != KDA_BF16 && c != KDA_FP32 && c != KDA_FP16; }

// A state's pointer and its dtype code: both given or neither.
int check_state(const void* p, int dtype) {
  if (bad_state_code(dtype)) return KDA_ERR_DTYPE;
  if ((dtype == KDA_STATE_NONE) != (p == nullptr)) return p ? KDA_ERR_DTYPE : KDA_ERR_NULL;
  return KDA_OK;
}

bool any_unaligned(std::initializer_list<const void*> ps, size_t a) {
  for (const void* p : ps)
    if (p && !aligned(p, a)) return true;
  return false;
}

// Whether a state of the recurrence is where the kernels can take it: an element at a time where
// rows are no whole vectors of the token tensors (layers of a cache begin anywhere then), else as
// many elements as such a vector holds.
bool state_unaligned(const void* p, int state_dtype, int dtype, int64_t D) {
  if (!p) return false;
  const int64_t vec = dtype == KDA_FP32 ? 4 : 8;
  const size_t elem = state_dtype == KDA_STATE_FP32 ? 4 : 2, all = (size_t)vec * elem;
  return !aligned(p, D % vec != 0 ? elem : all < 16 ? all : 16);
}

// Checks that both directions of the recurrence share; a, b, c are its token tensors.
int check_glr(const void* a, const void* b, const void* c, int dtype, const int64_t* cu, int64_t N, int64_t B, int64_t T,
              int64_t D) {
  if (T != 0 && (!a || !b || !c)) return KDA_ERR_NULL;
  if (B < 1 || T < 0 || D < 1 || D > MAX_CHANNELS) return KDA_ERR_SHAPE;
  if (cu && (B != 1 || N < 1)) return KDA_ERR_SHAPE;
  if (T > INT32_MAX / 2 || B > INT32_MAX / 2 || B * T >= (int64_t)INT32_MAX / 2) return KDA_ERR_SHAPE;
  if ((cu ? N : B) > INT32_MAX / 2 || !kda::glr_fits(B * T, D, cu ? N : B)) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  return KDA_OK;
}

kda::GlrParams glr_params(const void* x, const void* g, int dtype, const void* init, int init_dtype, const int64_t* cu,
                          int64_t N, int64_t B, int64_t T, int64_t D) {
  kda::GlrParams p{};
  p.x = x;
  p.g = g;
  p.dtype = dtype;
  p.init = init;
  p.init_dtype = init_dtype;
  p.cu = cu;
  p.nseq = (int32_t)(cu ? N : B);
  p.T = (int32_t)T;
  p.tokens = (int32_t)(B * T);
  p.D = (int32_t)D;
  return p;
}

int status(hipError_t e) { return e == hipSuccess ? KDA_OK : KDA_ERR_HIP; }

int check_pool(const void* pool, int64_t L, int64_t S, size_t slot_bytes, int64_t n) {
  if (!pool) return KDA_ERR_NULL;
  if (L < 1 || S < 1 || S > MAX_SLOTS || slot_bytes < 1 || n < 0 || n > INT32_MAX) return KDA_ERR_SHAPE;
  if (L > (int64_t)1 << 32 || (double)L * (double)S * (double)slot_bytes >= 4611686018427387904.0) return KDA_ERR_SHAPE;
  if (!aligned(pool, 16)) return KDA_ERR_ALIGN;
  return KDA_OK;
}

}  // namespace

extern "C" {

int64_t kda_glr_carry_rows(int64_t B, int64_t T) {
  if (B < 1 || T < 0 || T > INT32_MAX || B > INT32_MAX) return 0;
  return (B * T + kda::GLR_TILE - 1) / kda::GLR_TILE;
}

size_t kda_glr_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N) {
  if (B < 1 || T < 0 || D < 1 || N < 0 || D > MAX_CHANNELS || T > INT32_MAX || B > INT32_MAX || N > INT32_MAX) return 0;
  if (B * T >= (int64_t)INT32_MAX / 2 || !kda::glr_fits(B * T, D, N > 0 ? N : B)) return 0;
  return kda::glr_workspace(B * T, D, N > 0 ? N : B);
}

int kda_glr_fwd(const void* x, const void* g, void* y, int dtype, const void* initial_state, int initial_dtype,
                void* final_state, int final_dtype, float* carry, const int64_t* cu_seqlens, int64_t N, int64_t B,
                int64_t T, int64_t D, void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_glr(x, g, y, dtype, cu_seqlens, N, B, T, D);
  if (rc == KDA_OK) rc = check_state(initial_state, initial_dtype);
  if (rc == KDA_OK) rc = check_state(final_state, final_dtype);
  if (rc != KDA_OK) return rc;
  if (initial_state && final_state && initial_dtype != final_dtype) return KDA_ERR_DTYPE;
  if (any_unaligned({x, g, y, carry}, 16) || any_unaligned({cu_seqlens}, 8) ||
      state_unaligned(initial_state, initial_dtype, dtype, D) || state_unaligned(final_state, final_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  if (!workspace || workspace_bytes < kda_glr_workspace_size(B, T, D, cu_seqlens ? N : 0)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, kda::ALIGN)) return KDA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (cu_seqlens && kda::env_flag("KDA_VALIDATE")) {
    rc = kda::validate_cu_on_host(cu_seqlens, N, T, st);
    if (rc != KDA_OK) return rc;
  }
  kda::GlrParams p = glr_params(x, g, dtype, initial_state, initial_dtype, cu_seqlens, N, B, T, D);
  p.y = y;
  p.fin = final_state;
  p.fin_dtype = final_dtype;
  p.carry = carry;
  return status(kda::launch_glr_fwd(p, workspace, st));
}

int kda_glr_bwd(const void* x, const void* g, const void* dy, int dtype, const float* carry, const void* initial_state,
                int initial_dtype, const void* d_final, int d_final_dtype, void* dx, void* dg, void* d_initial,
                int d_initial_dtype, const int64_t* cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t D,
                void* workspace, size_t workspace_bytes, void* stream) {
  int rc = check_glr(x, g, dy, dtype, cu_seqlens, N, B, T, D);
  if (rc == KDA_OK && T != 0 && (!dx || !dg || !carry)) rc = KDA_ERR_NULL;
  if (rc == KDA_OK) rc = check_state(initial_state, initial_dtype);
  if (rc == KDA_OK) rc = check_state(d_final, d_final_dtype);
  if (rc == KDA_OK) rc = check_state(d_initial, d_initial_dtype);
  if (rc != KDA_OK) return rc;
  if (d_initial && (d_initial == d_final || d_initial == initial_state)) return KDA_ERR_VALUE;
  if (any_unaligned({x, g, dy, carry, dx, dg}, 16) || any_unaligned({cu_seqlens}, 8) ||
      state_unaligned(initial_state, initial_dtype, dtype, D) || state_unaligned(d_final, d_final_dtype, dtype, D) ||
      state_unaligned(d_initial, d_initial_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  if (!workspace || workspace_bytes < kda_glr_workspace_size(B, T, D, cu_seqlens ? N : 0)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, kda::ALIGN)) return KDA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (cu_seqlens && kda::env_flag("KDA_VALIDATE")) {
    rc = kda::validate_cu_on_host(cu_seqlens, N, T, st);
    if (rc != KDA_OK) return rc;
  }
  kda::GlrParams p = glr_params(x, g, dtype, initial_state, initial_dtype, cu_seqlens, N, B, T, D);
  p.dy = dy;
  p.dx = dx;
  p.dg = dg;
  p.fin = d_initial;
  p.fin_dtype = d_initial_dtype;
  p.dfin = d_final;
  p.dfin_dtype = d_final_dtype;
  p.carry = const_cast<float*>(carry);
  return status(kda::launch_glr_bwd(p, workspace, st));
}

int kda_glr_step(const void* x, const void* g, void* y, int dtype, void* state, int state_dtype, int64_t S,
                 const int32_t* in_slots, const int32_t* out_slots, int64_t N, int64_t D, void* stream) {
  if (N < 0 || N > INT32_MAX || D < 1 || D > MAX_CHANNELS || S < 1 || S > MAX_SLOTS || !kda::glr_fits(0, D, N)) return KDA_ERR_SHAPE;
  if (!state || (N != 0 && (!x || !g || !y || !in_slots || !out_slots))) return KDA_ERR_NULL;
  if (bad_dtype(dtype) || (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32)) return KDA_ERR_DTYPE;
  if (any_unaligned({x, g, y}, 16) || any_unaligned({in_slots, out_slots}, 4) || state_unaligned(state, state_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  kda::GlrParams p = glr_params(x, g, dtype, state, state_dtype, nullptr, 0, N, 1, D);
  p.y = y;
  p.fin = state;
  p.fin_dtype = state_dtype;
  p.in_slots = in_slots;
  p.out_slots = out_slots;
  p.n_slots = (int32_t)S;
  return status(kda::launch_glr_fwd(p, nullptr, static_cast<hipStream_t>(stream)));
}

size_t kda_layernorm_workspace_size(int64_t M, int64_t D) {
  if (M < 0 || D < 1 || D > MAX_D) return 0;
  return kda::align_up(2 * kda::layernorm_parts(M, D) * (size_t)D * sizeof(float));
}

int kda_layernorm_fwd(const void* x, const float* weight, const float* bias, float eps, void* y, int dtype, float* mean,
                      float* rstd, int64_t M, int64_t D, void* stream) {
  if (M != 0 && (!x || !y)) return KDA_ERR_NULL;
  if (M < 0 || D < 1 || D > MAX_D || (double)M * (double)D >= 1152921504606846976.0) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  if (!std::isfinite(eps) || eps < 0.0f) return KDA_ERR_VALUE;
  if (any_unaligned({x, y, weight, bias, mean, rstd}, 16)) return KDA_ERR_ALIGN;
  kda::NormParams p{};
  p.x = x;
  p.out = y;
  p.dtype = dtype;
  p.weight = weight;
  p.bias = bias;
  p.eps = eps;
  p.mean = mean;
  p.rstd = rstd;
  p.M = M;
  p.D = (int32_t)D;
  return status(kda::launch_layernorm_fwd(p, static_cast<hipStream_t>(stream)));
}

int kda_layernorm_bwd(const void* dy, const void* x, const float* weight, const float* mean, const float* rstd, void* dx,
                      int dtype, float* d_weight, float* d_bias, int64_t M, int64_t D, void* workspace,
                      size_t workspace_bytes, void* stream) {
  if (M != 0 && (!dy || !x || !mean || !rstd)) return KDA_ERR_NULL;
  if (M < 0 || D < 1 || D > MAX_D || (double)M * (double)D >= 1152921504606846976.0) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  if (any_unaligned({dy, x, weight, mean, rstd, dx, d_weight, d_bias}, 16)) return KDA_ERR_ALIGN;
  const bool sums = d_weight || d_bias;
  if (sums && M > 0) {
    if (!workspace || workspace_bytes < kda_layernorm_workspace_size(M, D)) return KDA_ERR_WORKSPACE;
    if (!aligned(workspace, kda::ALIGN)) return KDA_ERR_ALIGN;
  }
  if (!sums && (!dx || M == 0)) return KDA_OK;
  kda::NormParams p{};
  p.dy = dy;
  p.x = x;
  p.out = dx;
  p.dtype = dtype;
  p.weight = weight;
  p.mean = const_cast<float*>(mean);
  p.rstd = const_cast<float*>(rstd);
  p.dw = d_weight;
  p.db = d_bias;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  p.M = M;
  p.D = (int32_t)D;
  return status(kda::launch_layernorm_bwd(p, static_cast<hipStream_t>(stream)));
}

size_t kda_cache_workspace_size(int64_t S) {
  if (S < 1 || S > MAX_SLOTS) return 0;
  return kda::align_up((size_t)(1 + 2 * (S / 2 + 1)) * sizeof(int32_t));
}

int kda_cache_copy(void* pool, int64_t L, int64_t S, size_t slot_bytes, const int32_t* src, const int32_t* dst, int64_t n,
                   void* stream) {
  const int rc = check_pool(pool, L, S, slot_bytes, n);
  if (rc != KDA_OK) return rc;
  if (n != 0 && (!src || !dst)) return KDA_ERR_NULL;
  if (any_unaligned({src, dst}, 4)) return KDA_ERR_ALIGN;
  if (n == 0) return KDA_OK;
  return status(kda::launch_cache_copy({pool, L, S, slot_bytes}, src, dst, n, static_cast<hipStream_t>(stream)));
}

int kda_cache_fork(void* pool, int64_t L, int64_t S, size_t slot_bytes, int32_t* used, const int32_t* src, int32_t* dst,
                   int64_t n, void* stream) {
  const int rc = check_pool(pool, L, S, slot_bytes, n);
  if (rc != KDA_OK) return rc;
  if (!used || (n != 0 && (!src || !dst))) return KDA_ERR_NULL;
  if (any_unaligned({used, src, dst}, 4)) return KDA_ERR_ALIGN;
  if (n != 0 && (dst == src || dst == used || src == used)) return KDA_ERR_VALUE;
  if (n == 0) return KDA_OK;
  return status(kda::launch_cache_fork({pool, L, S, slot_bytes}, used, src, dst, n, static_cast<hipStream_t>(stream)));
}

int kda_cache_free(int32_t* used, int64_t S, const int32_t* slots, int64_t n, void* stream) {
  if (S < 1 || S > MAX_SLOTS || n < 0 || n > INT32_MAX) return KDA_ERR_SHAPE;
  if (!used || (n != 0 && !slots)) return KDA_ERR_NULL;
  if (any_unaligned({used, slots}, 4)) return KDA_ERR_ALIGN;
  if (n != 0 && used == slots) return KDA_ERR_VALUE;
  return status(kda::launch_cache_free(used, S, slots, n, static_cast<hipStream_t>(stream)));
}

int kda_cache_compact(void* pool, int64_t L, int64_t S, size_t slot_bytes, int32_t* used, int32_t* remap, int32_t* table,
                      int64_t n, void* workspace, size_t workspace_bytes, void* stream) {
  const int rc = check_pool(pool, L, S, slot_bytes, n);
  if (rc != KDA_OK) return rc;
  if (!used || !remap) return KDA_ERR_NULL;
  if (!table) n = 0;
  if (any_unaligned({used, remap, table}, 4)) return KDA_ERR_ALIGN;
  if (used == remap || table == remap || table == used) return KDA_ERR_VALUE;
  if (!workspace || workspace_bytes < kda_cache_workspace_size(S)) return KDA_ERR_WORKSPACE;
  if (!aligned(workspace, kda::ALIGN)) return KDA_ERR_ALIGN;
  return status(kda::launch_cache_compact({pool, L, S, slot_bytes}, used, remap, table, n,
                                          static_cast<int32_t*>(workspace), static_cast<hipStream_t>(stream)));
}

}  // extern "C"
