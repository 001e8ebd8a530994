// kda_layer_api.cpp -- C ABI of the short convolution, the selective scan, the root-mean-square
// norm, beam search and the beams' states: argument checks, workspace layout and launches.
#include <hip/hip_runtime.h>

#include <cmath>
#include <cstdint>

#include "../../include/kda.h"
#include "kda_api_util.h"
#include "kda_ops.h"

namespace {

using kda::aligned;
using kda::any_unaligned;
using kda::bad_dtype;
using kda::check_state;
using kda::state_unaligned;
using kda::status;

constexpr int64_t MAX_ROW = (int64_t)1 << 24;         // of the norm
constexpr int64_t MAX_CONV_D = (int64_t)1 << 22;
constexpr int64_t MAX_SSM_D = (int64_t)1 << 20;
constexpr int64_t MAX_BEAM_ROWS = (int64_t)1 << 24;

// Sizes of token tensors [B, T, ...] with rows or packed sequences
int check_tokens(const int64_t* cu, int64_t N, int64_t B, int64_t T) {
  if (B < 1 || T < 0) return KDA_ERR_SHAPE;
  if (cu && (B != 1 || N < 1)) return KDA_ERR_SHAPE;
  if (T > INT32_MAX / 2 || B > INT32_MAX / 2 || B * T >= (int64_t)INT32_MAX / 2) return KDA_ERR_SHAPE;
  if ((cu ? N : B) > INT32_MAX / 2) return KDA_ERR_SHAPE;
  return KDA_OK;
}
bool bad_slots(int64_t N, int64_t S) { return N < 0 || N > INT32_MAX / 2 || S < 1 || S > kda::MAX_SLOTS; }

// initial and final state of a forward pass
int check_states(const void* init, int init_dtype, const void* fin, int fin_dtype) {
  int rc = check_state(init, init_dtype);
  if (rc == KDA_OK) rc = check_state(fin, fin_dtype);
  if (rc == KDA_OK && init && fin && init_dtype != fin_dtype) rc = KDA_ERR_DTYPE;
  return rc;
}
// those of a backward pass
int check_grad_states(const void* init, int init_dtype, const void* dfin, int dfin_dtype, const void* dinit, int dinit_dtype) {
  int rc = check_state(init, init_dtype);
  if (rc == KDA_OK) rc = check_state(dfin, dfin_dtype);
  if (rc == KDA_OK) rc = check_state(dinit, dinit_dtype);
  if (rc == KDA_OK && dinit && (dinit == dfin || dinit == init)) rc = KDA_ERR_VALUE;
  return rc;
}
int check_workspace(const void* workspace, size_t bytes, size_t need) {
  if (need == 0) return KDA_OK;
  if (!workspace || bytes < need) return KDA_ERR_WORKSPACE;
  return aligned(workspace, kda::ALIGN) ? KDA_OK : KDA_ERR_ALIGN;
}
int validate(const int64_t* cu, int64_t N, int64_t T, hipStream_t stream) {
  return cu && kda::env_flag("KDA_VALIDATE") ? kda::validate_cu_on_host(cu, N, T, stream) : KDA_OK;
}

// States of the scan: four elements at once where E is a multiple of 4
bool scan_state_unaligned(const void* p, int dtype, int64_t E) {
  const size_t elem = dtype == KDA_STATE_FP32 ? 4 : 2;
  return p && !aligned(p, E % 4 == 0 ? 4 * elem : elem);
}

bool conv_sizes_ok(int64_t D, int64_t W) { return D >= 1 && D <= MAX_CONV_D && W >= 2 && W <= 4; }
bool ssm_sizes_ok(int64_t D, int64_t E, int64_t G) {
  return D >= 1 && D <= MAX_SSM_D && E >= 1 && E <= 64 && G >= 1 && G <= D && D % G == 0;
}

kda::ConvParams conv_params(const void* x, const float* weight, const float* bias, int dtype, int64_t W, uint32_t flags,
                            const void* init, int init_dtype, const int64_t* cu, int64_t N, int64_t B, int64_t T, int64_t D) {
  kda::ConvParams p{};
  p.x = x;
  p.weight = weight;
  p.bias = bias;
  p.dtype = dtype;
  p.W = (int)W;
  p.silu = (flags & KDA_CONV_SILU) != 0;
  p.init = init;
  p.init_dtype = init_dtype;
  p.cu = cu;
  p.nseq = (int32_t)(cu ? N : B);
  p.T = (int32_t)T;
  p.tokens = (int32_t)(B * T);
  p.D = (int32_t)D;
  return p;
}

kda::SsmParams ssm_params(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* skip,
                          const void* z, const float* dt_bias, int dtype, uint32_t flags, const void* init, int init_dtype,
                          const int64_t* cu, int64_t N, int64_t B, int64_t T, int64_t D, int64_t E, int64_t G) {
  kda::SsmParams p{};
  p.x = x;
  p.dt = dt;
  p.A = A;
  p.Bm = Bm;
  p.Cm = Cm;
  p.skip = skip;
  p.z = z;
  p.dt_bias = dt_bias;
  p.dtype = dtype;
  p.softplus = (flags & KDA_SSM_SOFTPLUS) != 0;
  p.init = init;
  p.init_dtype = init_dtype;
  p.cu = cu;
  p.nseq = (int32_t)(cu ? N : B);
  p.T = (int32_t)T;
  p.tokens = (int32_t)(B * T);
  p.D = (int32_t)D;
  p.E = (int32_t)E;
  p.G = (int32_t)G;
  return p;
}

}  // namespace

extern "C" {

// ---- root-mean-square norm ----

size_t kda_rmsnorm_workspace_size(int64_t M, int64_t D) {
  if (M < 0 || D < 1 || D > MAX_ROW) return 0;
  return kda::align_up(kda::rmsnorm_parts(M, D) * (size_t)D * sizeof(float));
}

int kda_rmsnorm_fwd(const void* x, const void* residual, const float* weight, float eps, void* y, int y_dtype, float* scales,
                    int64_t group, void* residual_out, int dtype, float* rstd, int64_t M, int64_t D, void* stream) {
  if (M != 0 && (!x || !y)) return KDA_ERR_NULL;
  if (M < 0 || D < 1 || D > MAX_ROW || (double)M * (double)D >= 1152921504606846976.0) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype) || (y_dtype != dtype && y_dtype != KDA_E4M3)) return KDA_ERR_DTYPE;
  if (y_dtype == KDA_E4M3) {
    if (group != 128 && group != D) return KDA_ERR_SHAPE;
    if (M != 0 && !scales) return KDA_ERR_NULL;
    if (M != 0 && (y == x || y == residual)) return KDA_ERR_VALUE;   // rows lie elsewhere there
  } else if (group != 0) {
    return KDA_ERR_SHAPE;
  } else if (scales) {
    return KDA_ERR_VALUE;
  }
  if (!std::isfinite(eps) || eps < 0.0f) return KDA_ERR_VALUE;
  if (M != 0 && residual_out == y) return KDA_ERR_VALUE;
  if (any_unaligned({x, residual, weight, y, scales, residual_out, rstd}, 16)) return KDA_ERR_ALIGN;
  kda::RmsParams p{};
  p.x = x;
  p.res = residual;
  p.weight = weight;
  p.eps = eps;
  p.out = y;
  p.scales = scales;
  p.group = (int32_t)group;
  p.res_out = residual_out;
  p.dtype = dtype;
  p.rstd = rstd;
  p.M = M;
  p.D = (int32_t)D;
  return status(kda::launch_rmsnorm_fwd(p, static_cast<hipStream_t>(stream)));
}

int kda_rmsnorm_bwd(const void* dy, const void* x, const float* weight, const float* rstd, const void* d_residual, void* dx,
                    int dtype, float* d_weight, int64_t M, int64_t D, void* workspace, size_t workspace_bytes, void* stream) {
  if (M != 0 && (!dy || !x || !rstd)) return KDA_ERR_NULL;
  if (M < 0 || D < 1 || D > MAX_ROW || (double)M * (double)D >= 1152921504606846976.0) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  if (any_unaligned({dy, x, weight, rstd, d_residual, dx, d_weight}, 16)) return KDA_ERR_ALIGN;
  if (d_weight && M > 0) {
    const int rc = check_workspace(workspace, workspace_bytes, kda_rmsnorm_workspace_size(M, D));
    if (rc != KDA_OK) return rc;
  }
  if (!d_weight && (!dx || M == 0)) return KDA_OK;
  kda::RmsParams p{};
  p.dy = dy;
  p.x = x;
  p.weight = weight;
  p.rstd = const_cast<float*>(rstd);
  p.res = d_residual;
  p.out = dx;
  p.dtype = dtype;
  p.dw = d_weight;
  p.partial = d_weight ? static_cast<float*>(workspace) : nullptr;
  p.M = M;
  p.D = (int32_t)D;
  return status(kda::launch_rmsnorm_bwd(p, static_cast<hipStream_t>(stream)));
}

// ---- short causal convolution ----

size_t kda_conv_workspace_size(int64_t B, int64_t T, int64_t D, int64_t W) {
  if (check_tokens(nullptr, 0, B, T) != KDA_OK || !conv_sizes_ok(D, W) || !kda::conv_fits(B * T, D)) return 0;
  return kda::align_up(kda::conv_workspace(B * T, D, W));
}

int kda_conv_fwd(const void* x, const float* weight, const float* bias, void* y, int dtype, int64_t W, uint32_t flags,
                 const void* initial_state, int initial_dtype, void* final_state, int final_dtype, const int64_t* cu_seqlens,
                 int64_t N, int64_t B, int64_t T, int64_t D, void* stream) {
  if (!weight || (T != 0 && (!x || !y))) return KDA_ERR_NULL;
  int rc = check_tokens(cu_seqlens, N, B, T);
  if (rc != KDA_OK) return rc;
  if (!conv_sizes_ok(D, W) || !kda::conv_fits(B * T, D)) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  rc = check_states(initial_state, initial_dtype, final_state, final_dtype);
  if (rc != KDA_OK) return rc;
  if (flags & ~(uint32_t)KDA_CONV_SILU) return KDA_ERR_VALUE;
  if (T != 0 && x == y) return KDA_ERR_VALUE;
  if (any_unaligned({x, y, weight, bias}, 16) || any_unaligned({cu_seqlens}, 8) ||
      state_unaligned(initial_state, initial_dtype, dtype, D) || state_unaligned(final_state, final_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  hipStream_t st = static_cast<hipStream_t>(stream);
  rc = validate(cu_seqlens, N, T, st);
  if (rc != KDA_OK) return rc;
  kda::ConvParams p = conv_params(x, weight, bias, dtype, W, flags, initial_state, initial_dtype, cu_seqlens, N, B, T, D);
  p.out = y;
  p.fin = final_state;
  p.fin_dtype = final_dtype;
  return status(kda::launch_conv_fwd(p, st));
}

int kda_conv_bwd(const void* x, const float* weight, const float* bias, const void* dy, int dtype, int64_t W, uint32_t flags,
                 const void* initial_state, int initial_dtype, const void* d_final, int d_final_dtype, void* dx, float* d_weight,
                 float* d_bias, void* d_initial, int d_initial_dtype, const int64_t* cu_seqlens, int64_t N, int64_t B, int64_t T,
                 int64_t D, void* workspace, size_t workspace_bytes, void* stream) {
  if (!weight || (T != 0 && (!x || !dy || !dx))) return KDA_ERR_NULL;
  int rc = check_tokens(cu_seqlens, N, B, T);
  if (rc != KDA_OK) return rc;
  if (!conv_sizes_ok(D, W) || !kda::conv_fits(B * T, D)) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  rc = check_grad_states(initial_state, initial_dtype, d_final, d_final_dtype, d_initial, d_initial_dtype);
  if (rc != KDA_OK) return rc;
  if (flags & ~(uint32_t)KDA_CONV_SILU) return KDA_ERR_VALUE;
  if (T != 0 && (dx == x || dx == dy)) return KDA_ERR_VALUE;   // neighbouring tokens read them too
  if (any_unaligned({x, dy, dx, weight, bias, d_weight, d_bias}, 16) || any_unaligned({cu_seqlens}, 8) ||
      state_unaligned(initial_state, initial_dtype, dtype, D) || state_unaligned(d_final, d_final_dtype, dtype, D) ||
      state_unaligned(d_initial, d_initial_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  const bool sums = d_weight || d_bias;
  if (sums) rc = check_workspace(workspace, workspace_bytes, kda_conv_workspace_size(B, T, D, W));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rc == KDA_OK) rc = validate(cu_seqlens, N, T, st);
  if (rc != KDA_OK) return rc;
  kda::ConvParams p = conv_params(x, weight, bias, dtype, W, flags, initial_state, initial_dtype, cu_seqlens, N, B, T, D);
  p.dy = dy;
  p.out = dx;
  p.dfin = d_final;
  p.dfin_dtype = d_final_dtype;
  p.dinit = d_initial;
  p.dinit_dtype = d_initial_dtype;
  p.dw = d_weight;
  p.db = d_bias;
  p.partial = sums ? static_cast<float*>(workspace) : nullptr;
  return status(kda::launch_conv_bwd(p, st));
}

int kda_conv_step(const void* x, const float* weight, const float* bias, void* y, int dtype, int64_t W, uint32_t flags,
                  void* state, int state_dtype, int64_t S, const int32_t* in_slots, const int32_t* out_slots, int64_t N,
                  int64_t D, void* stream) {
  if (bad_slots(N, S) || !conv_sizes_ok(D, W)) return KDA_ERR_SHAPE;
  if (!weight || !state || (N != 0 && (!x || !y || !in_slots || !out_slots))) return KDA_ERR_NULL;
  if (bad_dtype(dtype) || (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32)) return KDA_ERR_DTYPE;
  if (flags & ~(uint32_t)KDA_CONV_SILU) return KDA_ERR_VALUE;
  if (any_unaligned({x, y, weight, bias}, 16) || any_unaligned({in_slots, out_slots}, 4) ||
      state_unaligned(state, state_dtype, dtype, D))
    return KDA_ERR_ALIGN;
  kda::ConvParams p = conv_params(x, weight, bias, dtype, W, flags, state, state_dtype, nullptr, 0, N, 1, D);
  p.out = y;
  p.fin = state;
  p.fin_dtype = state_dtype;
  p.in_slots = in_slots;
  p.out_slots = out_slots;
  p.n_slots = (int32_t)S;
  return status(kda::launch_conv_step(p, static_cast<hipStream_t>(stream)));
}

// ---- selective state space scan ----

int64_t kda_ssm_carry_rows(int64_t B, int64_t T) {
  if (check_tokens(nullptr, 0, B, T) != KDA_OK) return 0;
  return (B * T + kda::SSM_BLOCK - 1) / kda::SSM_BLOCK;
}

size_t kda_ssm_workspace_size(int64_t B, int64_t T, int64_t D, int64_t E, int64_t G, int64_t N, int backward) {
  if (check_tokens(nullptr, 0, B, T) != KDA_OK || N < 0 || N > INT32_MAX / 2 || (N > 0 && B != 1)) return 0;
  if (!ssm_sizes_ok(D, E, G) || !kda::ssm_fits(B * T, D, E, G)) return 0;
  return kda::align_up(kda::ssm_workspace(B * T, D, E, G, backward != 0)) + kda::ALIGN;
}

int kda_ssm_fwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* skip, const void* z,
                const float* dt_bias, void* y, int dtype, uint32_t flags, const void* initial_state, int initial_dtype,
                void* final_state, int final_dtype, float* carry, const int64_t* cu_seqlens, int64_t N, int64_t B, int64_t T,
                int64_t D, int64_t E, int64_t G, void* workspace, size_t workspace_bytes, void* stream) {
  if (!A || (T != 0 && (!x || !dt || !Bm || !Cm || !y))) return KDA_ERR_NULL;
  int rc = check_tokens(cu_seqlens, N, B, T);
  if (rc != KDA_OK) return rc;
  if (!ssm_sizes_ok(D, E, G) || !kda::ssm_fits(B * T, D, E, G)) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  rc = check_states(initial_state, initial_dtype, final_state, final_dtype);
  if (rc != KDA_OK) return rc;
  if (flags & ~(uint32_t)KDA_SSM_SOFTPLUS) return KDA_ERR_VALUE;
  if (T != 0 && (y == x || y == dt || y == z)) return KDA_ERR_VALUE;   // chunks read them more than once
  if (any_unaligned({x, dt, A, Bm, Cm, skip, z, dt_bias, y, carry}, 16) || any_unaligned({cu_seqlens}, 8) ||
      scan_state_unaligned(initial_state, initial_dtype, E) || scan_state_unaligned(final_state, final_dtype, E))
    return KDA_ERR_ALIGN;
  rc = check_workspace(workspace, workspace_bytes, kda_ssm_workspace_size(B, T, D, E, G, cu_seqlens ? N : 0, 0));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rc == KDA_OK) rc = validate(cu_seqlens, N, T, st);
  if (rc != KDA_OK) return rc;
  kda::SsmParams p = ssm_params(x, dt, A, Bm, Cm, skip, z, dt_bias, dtype, flags, initial_state, initial_dtype, cu_seqlens, N, B,
                                T, D, E, G);
  p.y = y;
  p.fin = final_state;
  p.fin_dtype = final_dtype;
  p.carry = carry;
  return status(kda::launch_ssm_fwd(p, workspace, st));
}

int kda_ssm_bwd(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* skip, const void* z,
                const float* dt_bias, const void* dy, int dtype, uint32_t flags, const float* carry, const void* initial_state,
                int initial_dtype, const void* d_final, int d_final_dtype, void* dx, void* d_dt, float* dA, void* dB, void* dC,
                float* d_skip, void* d_z, float* d_dt_bias, void* d_initial, int d_initial_dtype, const int64_t* cu_seqlens,
                int64_t N, int64_t B, int64_t T, int64_t D, int64_t E, int64_t G, void* workspace, size_t workspace_bytes,
                void* stream) {
  if (!A || !dA || (T != 0 && (!x || !dt || !Bm || !Cm || !dy || !carry || !dx || !d_dt || !dB || !dC))) return KDA_ERR_NULL;
  int rc = check_tokens(cu_seqlens, N, B, T);
  if (rc != KDA_OK) return rc;
  if (!ssm_sizes_ok(D, E, G) || !kda::ssm_fits(B * T, D, E, G)) return KDA_ERR_SHAPE;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  rc = check_grad_states(initial_state, initial_dtype, d_final, d_final_dtype, d_initial, d_initial_dtype);
  if (rc != KDA_OK) return rc;
  if (flags & ~(uint32_t)KDA_SSM_SOFTPLUS) return KDA_ERR_VALUE;
  if ((d_skip && !skip) || (T != 0 && d_z && !z) || (d_dt_bias && !dt_bias)) return KDA_ERR_VALUE;
  if (any_unaligned({x, dt, A, Bm, Cm, skip, z, dt_bias, dy, carry, dx, d_dt, dA, dB, dC, d_skip, d_z, d_dt_bias}, 16) ||
      any_unaligned({cu_seqlens}, 8) || scan_state_unaligned(initial_state, initial_dtype, E) ||
      scan_state_unaligned(d_final, d_final_dtype, E) || scan_state_unaligned(d_initial, d_initial_dtype, E))
    return KDA_ERR_ALIGN;
  if (T != 0)
    for (const void* out : {(const void*)dx, (const void*)d_dt, (const void*)d_z})   // chunks read them more than once
      if (out && (out == x || out == dt || out == z || out == dy)) return KDA_ERR_VALUE;
  rc = check_workspace(workspace, workspace_bytes, kda_ssm_workspace_size(B, T, D, E, G, cu_seqlens ? N : 0, 1));
  hipStream_t st = static_cast<hipStream_t>(stream);
  if (rc == KDA_OK) rc = validate(cu_seqlens, N, T, st);
  if (rc != KDA_OK) return rc;
  kda::SsmParams p = ssm_params(x, dt, A, Bm, Cm, skip, z, dt_bias, dtype, flags, initial_state, initial_dtype, cu_seqlens, N, B,
                                T, D, E, G);
  p.dy = dy;
  p.carry = const_cast<float*>(carry);
  p.dfin = d_final;
  p.dfin_dtype = d_final_dtype;
  p.dx = dx;
  p.ddt = d_dt;
  p.dA = dA;
  p.dB = dB;
  p.dC = dC;
  p.dskip = d_skip;
  p.dz = d_z;
  p.dbias = d_dt_bias;
  p.dinit = d_initial;
  p.dinit_dtype = d_initial_dtype;
  return status(kda::launch_ssm_bwd(p, workspace, st));
}

int kda_ssm_step(const void* x, const void* dt, const float* A, const void* Bm, const void* Cm, const float* skip, const void* z,
                 const float* dt_bias, void* y, int dtype, uint32_t flags, void* state, int state_dtype, int64_t S,
                 const int32_t* in_slots, const int32_t* out_slots, int64_t N, int64_t D, int64_t E, int64_t G, void* stream) {
  if (bad_slots(N, S) || !ssm_sizes_ok(D, E, G)) return KDA_ERR_SHAPE;
  if (!A || !state || (N != 0 && (!x || !dt || !Bm || !Cm || !y || !in_slots || !out_slots))) return KDA_ERR_NULL;
  if (bad_dtype(dtype) || (state_dtype != KDA_STATE_BF16 && state_dtype != KDA_STATE_FP32)) return KDA_ERR_DTYPE;
  if (flags & ~(uint32_t)KDA_SSM_SOFTPLUS) return KDA_ERR_VALUE;
  if (any_unaligned({x, dt, A, Bm, Cm, skip, z, dt_bias, y}, 16) || any_unaligned({in_slots, out_slots}, 4) ||
      scan_state_unaligned(state, state_dtype, E))
    return KDA_ERR_ALIGN;
  kda::SsmParams p = ssm_params(x, dt, A, Bm, Cm, skip, z, dt_bias, dtype, flags, state, state_dtype, nullptr, 0, N, 1, D, E, G);
  p.y = y;
  p.fin = state;
  p.fin_dtype = state_dtype;
  p.in_slots = in_slots;
  p.out_slots = out_slots;
  p.n_slots = (int32_t)S;
  return status(kda::launch_ssm_step(p, static_cast<hipStream_t>(stream)));
}

// ---- beam search ----

static bool beam_sizes_ok(int64_t N, int64_t W, int64_t V, int64_t k) {
  return N >= 0 && N <= MAX_BEAM_ROWS && W >= 1 && W <= 64 && V >= 1 && V <= MAX_ROW && k >= 1 && k <= 64 &&
         N * W < MAX_BEAM_ROWS;
}

size_t kda_beam_workspace_size(int64_t N, int64_t W, int64_t V, int64_t k) {
  if (!beam_sizes_ok(N, W, V, k)) return 0;
  return kda::beam_workspace(N, W, V, k) + kda::ALIGN;
}

int kda_beam_select(const void* logits, int dtype, const float* scores, const int32_t* finished, int64_t eos, int32_t* tokens,
                    int32_t* parents, float* new_scores, int64_t N, int64_t W, int64_t V, int64_t k, void* workspace,
                    size_t workspace_bytes, void* stream) {
  if (!beam_sizes_ok(N, W, V, k)) return KDA_ERR_SHAPE;
  if (N != 0 && (!logits || !scores || !tokens || !parents || !new_scores)) return KDA_ERR_NULL;
  if (bad_dtype(dtype)) return KDA_ERR_DTYPE;
  if (finished && (eos < 0 || eos >= V)) return KDA_ERR_VALUE;
  if (N != 0 && (tokens == parents || (new_scores == scores && k != W) || (const void*)tokens == finished ||
                 (const void*)parents == finished))
    return KDA_ERR_VALUE;
  if (any_unaligned({logits}, 16) || any_unaligned({scores, finished, tokens, parents, new_scores}, 4)) return KDA_ERR_ALIGN;
  const int rc = check_workspace(workspace, workspace_bytes, kda_beam_workspace_size(N, W, V, k));
  if (rc != KDA_OK) return rc;
  kda::BeamParams p{};
  p.logits = logits;
  p.dtype = dtype;
  p.scores = scores;
  p.finished = finished;
  p.eos = (int32_t)(finished ? eos : 0);
  p.tokens = tokens;
  p.parents = parents;
  p.new_scores = new_scores;
  p.N = (int32_t)N;
  p.W = (int32_t)W;
  p.V = (int32_t)V;
  p.k = (int32_t)k;
  return status(kda::launch_beam_select(p, workspace, static_cast<hipStream_t>(stream)));
}

int kda_cache_reorder(void* pool, int64_t L, int64_t S, size_t slot_bytes, const int32_t* slots, const int32_t* parents,
                      int32_t* new_slots, int64_t N, int64_t W, void* stream) {
  const int rc = kda::check_pool(pool, L, S, slot_bytes, N);
  if (rc != KDA_OK) return rc;
  if (W < 1 || W > 64 || N > MAX_BEAM_ROWS) return KDA_ERR_SHAPE;
  if (N != 0 && (!slots || !parents || !new_slots)) return KDA_ERR_NULL;
  if (any_unaligned({slots, parents, new_slots}, 4)) return KDA_ERR_ALIGN;
  if (N != 0 && (new_slots == slots || new_slots == parents)) return KDA_ERR_VALUE;
  return status(kda::launch_cache_reorder({pool, L, S, slot_bytes}, slots, parents, new_slots, N, (int)W,
                                          static_cast<hipStream_t>(stream)));
}

}  // extern "C"
