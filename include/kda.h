/*
 * kda.h -- C ABI of the MI355X (gfx950) Kimi Delta Attention forward library
 * (libkda.so), and of the operators beside it that a recurrent layer trains and
 * serves with: the gated linear recurrence (kda_glr_*), layer norm
 * (kda_layernorm_*), and caches of states in slots (kda_cache_*, kda_fwd_slots).
 *
 * The operation (per sequence n and head h, state S of V x K, K contiguous):
 *   q^, k^ = L2-normalised q, k over K (x / sqrt(sum x^2 + 1e-6))
 *   beta   = sigmoid(beta logit)
 *   g~[c]  = lower_bound * sigmoid(exp(A_log[h]) * (g[c] + dt_bias[h][c]))
 *   S      = S * Diag(exp(g~));  S = S - beta (S k^ - v) k^^T;  o = scale * S q^
 * KDA is Gated DeltaNet with a per-channel gate (page "FlashKDA：基於 CUTLASS
 * 的 Kimi Delta Attention CUDA 加速實作", section 背景). The pages print no
 * equation; the gate form, natural exp, the 1e-6 epsilon and the order
 * decay -> delta update -> read-out are this library's stated readings.
 *
 * The argument list mirrors flash_kda.fwd(q, k, v, g, beta, scale, out,
 * A_log, dt_bias, lower_bound, initial_state, final_state, cu_seqlens) and its
 * parameter table ("Kernel API" of the FlashKDA README digest, aiwatch.icu
 * page), with the caller-owned, written-in-place `out` of the 2kiu.com guide
 * (sections 一 and 三).
 *
 * Conventions for every entry point:
 *   - All tensor pointers are DEVICE pointers (hipMalloc'd or from a caching
 *     allocator), row-major and contiguous, aligned to 16 bytes (the state
 *     and fp32 parameters to 16 bytes as well; index arrays to their elements;
 *     states of the gated linear recurrence as said there).
 *   - `stream` is a hipStream_t passed as void* (NULL = the default stream).
 *     Calls are stream-ordered and asynchronous: they return as soon as the
 *     work is enqueued. The library allocates nothing per call and keeps no
 *     pointer after it returns; it is reentrant.
 *   - Errors are detected on the host before anything is launched; on error
 *     nothing is written. cu_seqlens CONTENTS live on the device and are a
 *     caller precondition (cu[0] = 0, non-decreasing, cu[N] = T); the kernels
 *     clamp every sequence into [0, T] so malformed contents cannot make them
 *     access memory out of bounds (results are then unspecified). Setting the
 *     environment variable KDA_VALIDATE=1 makes kda_fwd synchronise the stream
 *     and check the contents on the host (KDA_ERR_VALUE if violated).
 *   - Other environment variables: KDA_LOG=1 prints each kda_fwd call's sizes
 *     and chain segment count to stderr; KDA_CHAIN_SEGMENTS=n caps the number
 *     of segments of the segment-parallel state chain (see
 *     kda_fwd_workspace_size; 1 keeps the plain chain); KDA_GLR_POLLS=n (a whole
 *     number, else ignored) caps the polls of a wait inside kda_glr_fwd and
 *     kda_glr_bwd (see there).
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Status codes. */
enum kda_status {
    KDA_OK = 0,
    KDA_ERR_NULL = 1,      /* a required pointer is NULL                           */
    KDA_ERR_SHAPE = 2,     /* K != 128, V != 128, H < 1, T < 0, B < 1, B != 1 with
                              cu_seqlens, N < 1 with cu_seqlens, D, S, L, M or n
                              out of range, size overflow                           */
    KDA_ERR_DTYPE = 3,     /* unknown dtype or state dtype code, or initial and final
                              state given with different dtypes                     */
    KDA_ERR_VALUE = 4,     /* lower_bound outside [-5, 0] or not finite (safe gate),
                              scale not finite, eps negative or not finite, unknown
                              flag bits, one buffer given twice where the call says
                              so, bad cu_seqlens contents (KDA_VALIDATE=1)          */
    KDA_ERR_ALIGN = 5,     /* a pointer is not aligned as its argument has to be    */
    KDA_ERR_WORKSPACE = 6, /* workspace NULL or too small (kda_fwd_workspace_min, or the
                              operator's own kda_*_workspace_size)                  */
    KDA_ERR_HIP = 7,       /* a HIP runtime call or kernel launch failed            */
    KDA_ERR_CAPACITY = 8   /* kda_fwd_noalloc: the call needs more workspace than
                              its fixed device array holds (KDA_NOALLOC_CAPACITY)   */
};

/*
 * Fusion switches of kda_fwd_ex / kda_fwd_recurrent_ex (the use_gate_in_kernel,
 * use_qk_l2norm_in_kernel and use_beta_sigmoid_in_kernel switches of page
 * "FlashKDA：面向SM90+的高性能KDA CUDA内核库", Q4). A set bit runs that input
 * processing inside the kernels; with a bit clear the input is taken as
 * already processed (this library's reading):
 *   KDA_FUSE_GATE clear          g holds the log-decay g~ itself (bf16), which
 *                                is clamped into [lower_bound, 0]; A_log and
 *                                dt_bias are unused and may be NULL
 *   KDA_FUSE_QK_L2NORM clear     q and k are used as given (expected unit norm)
 *   KDA_FUSE_BETA_SIGMOID clear  beta holds beta itself (expected in [0, 1])
 * KDA_GATE_UNBOUNDED is the safe_gate switch of the same page turned off. The
 * safe gate (bit clear) is the lower_bound form documented at kda_fwd; with the
 * bit set the gate is the plain softplus log-decay, not bounded below, and
 * lower_bound is neither used nor checked (this library's reading):
 *   KDA_FUSE_GATE set            g~ = -exp(A_log[h]) * log(1 + exp(g + dt_bias[h]))
 *   KDA_FUSE_GATE clear          g~ = min(g, 0)
 * Chunks whose 16-token gate sums stay above -80 (natural log) take the same
 * kernel path as the safe gate; others compute their diagonal 16x16 decay
 * blocks pairwise, which costs extra vector work for those chunks only.
 * kda_fwd and kda_fwd_recurrent are the KDA_FUSE_ALL case (safe gate).
 */
enum kda_fuse_flags {
    KDA_FUSE_GATE = 1,
    KDA_FUSE_QK_L2NORM = 2,
    KDA_FUSE_BETA_SIGMOID = 4,
    KDA_FUSE_ALL = 7,
    KDA_GATE_UNBOUNDED = 8,
    KDA_PATH_CHUNKED = 16   /* kda_fwd_ex only: never hand a short call to the
                               token-recurrent kernel (see kda_fwd)             */
};

/* State dtype codes for initial_state / final_state. */
enum kda_state_dtype {
    KDA_STATE_NONE = 0,    /* pointer must be NULL (stateless)  */
    KDA_STATE_BF16 = 1,    /* bfloat16, rounded to nearest-even */
    KDA_STATE_FP32 = 2     /* float32                           */
};

/*
 * kda_fwd_workspace_size -- bytes of device workspace kda_fwd needs.
 *   B, T, H: as for kda_fwd;  N: number of sequences when cu_seqlens is used,
 *   0 otherwise. Returns 0 for invalid sizes (B < 1, T < 0, H < 1, N < 0).
 * The workspace holds the per-chunk intermediates of the chunked (WY) form
 * (74.5 KiB per 64-token chunk and head) and the varlen chunk tables. With few
 * (row or sequence, head) pairs on long rows it also holds the buffers of the
 * segment-parallel state chain: each row's or sequence's chunks are cut into s
 * segments (s chosen from B or N, T and H), with 192 KiB per (row or sequence,
 * segment, head) for the segments' affine maps and initial states.
 * Calls whose full workspace would exceed 4 GiB and that use the plain chain
 * get the size of a windowed run within 4 GiB instead (see
 * kda_fwd_workspace_min; at B = 4, T = 32768, H = 64 that takes the same time
 * as the full 9.5 GiB).
 */
size_t kda_fwd_workspace_size(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * kda_fwd_workspace_min -- the smallest workspace kda_fwd / kda_fwd_ex accept for
 * the same call (same arguments and invalid-size rule as kda_fwd_workspace_size).
 * Calls given less than kda_fwd_workspace_size run in windows, each the
 * intra-chunk pass and the state chain over part of the chunks:
 *   - fixed length (N = 0): chunk columns jb .. jb + w - 1 of every row, with
 *     each row's state carried to the next window in fp32 (in final_state itself
 *     when that is fp32, else in the workspace: 64 KiB per (row, head)); the
 *     minimum holds one chunk column (B * H records of 74.5 KiB) and the carry;
 *   - varlen (N > 0): w consecutive chunk slots of the packed sequences, a
 *     sequence that crosses a window boundary carrying its state in fp32 through
 *     one of two carry slots (64 KiB per head each); the minimum holds the
 *     scheduler's tables, the carry slots and one slot of H records.
 * Windowed calls return the same bits as unwindowed ones; they take more kernel
 * launches and skip the segment-parallel chain.
 */
size_t kda_fwd_workspace_min(int64_t B, int64_t T, int64_t H, int64_t N);

/*
 * kda_fwd -- chunked KDA prefill forward (64-token chunks).
 *
 *   q, k, g      bf16 [B, T, H, K]   query, key, raw gate input (activated inside)
 *   v            bf16 [B, T, H, V]   value
 *   beta         bf16 [B, T, H]      beta logits (sigmoid applied inside)
 *   scale        float               read-out scaling factor (finite)
 *   out          bf16 [B, T, H, V]   OUTPUT, written in place; every element
 *                                    is written, none is read (no need to
 *                                    pre-zero it)
 *   A_log        fp32 [H]            log of each head's gate rate
 *   dt_bias      fp32 [H, K]         per-channel offset added to g
 *   lower_bound  float in [-5, 0]    most negative value the gate can take
 *   initial_state, initial_dtype     NULL/KDA_STATE_NONE (zeros) or
 *                                    [B|N, H, V, K] bf16/fp32
 *   final_state, final_dtype         NULL/KDA_STATE_NONE (not written) or
 *                                    [B|N, H, V, K] bf16/fp32, written for every
 *                                    (sequence, head), zero-length sequences
 *                                    included. May alias initial_state.
 *   cu_seqlens   int64 [N+1] or NULL packed sequence boundaries; requires
 *                                    B == 1 and T the total packed length.
 *                                    Without it, each of the B rows is an
 *                                    independent sequence of length T.
 *   N            number of sequences (ignored without cu_seqlens)
 *   B, T, H, K, V                    sizes; K and V must be 128. T may be 0:
 *                                    then q, k, v, g, beta and out hold no
 *                                    element and may be NULL, and the call
 *                                    only writes final_state (the initial
 *                                    state, or zeros, for every sequence)
 *   workspace, workspace_bytes       caller-owned device scratch of at least
 *                                    kda_fwd_workspace_min(B, T, H, N) bytes
 *                                    (run in windows when below
 *                                    kda_fwd_workspace_size), 256-byte aligned;
 *                                    its contents need no initialisation and
 *                                    are clobbered
 *   stream       hipStream_t as void*
 * Returns a kda_status.
 *
 * Decode-sized calls run on the token-recurrent kernel of kda_fwd_recurrent,
 * which computes the same operation without the chunked form's fixed cost of
 * one 64-token chunk per (sequence, head): fixed-length calls with T <= 8, and
 * varlen calls with T <= 2 N (at most two tokens per sequence on average; the
 * lengths themselves stay on the device). The workspace rules are unchanged.
 * kda_fwd_ex with KDA_PATH_CHUNKED keeps such calls on the chunked kernels.
 */
int kda_fwd(const void *q, const void *k, const void *v, const void *g, const void *beta,
            float scale, void *out, const float *A_log, const float *dt_bias, float lower_bound,
            const void *initial_state, int initial_dtype, void *final_state, int final_dtype,
            const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H, int64_t K,
            int64_t V, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_fwd_recurrent -- the same operation computed token by token (one
 * workgroup per sequence and head, fp32 state in registers). Same arguments
 * and rules as kda_fwd, without a workspace. It is the path for online
 * generation with state passing (decode-sized T; page "FlashKDA：面向SM90+的
 * 高性能KDA CUDA内核库", Q2 on stateful/streaming use) and a reference for the
 * chunked path on long inputs.
 */
int kda_fwd_recurrent(const void *q, const void *k, const void *v, const void *g,
                      const void *beta, float scale, void *out, const float *A_log,
                      const float *dt_bias, float lower_bound, const void *initial_state,
                      int initial_dtype, void *final_state, int final_dtype,
                      const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H,
                      int64_t K, int64_t V, void *stream);

/*
 * kda_fwd_ex, kda_fwd_recurrent_ex -- kda_fwd / kda_fwd_recurrent with the
 * switches in `flags` (KDA_FUSE_* bits, KDA_GATE_UNBOUNDED and, for kda_fwd_ex,
 * KDA_PATH_CHUNKED; other bits: KDA_ERR_VALUE). Every other argument and rule is that of the plain entry
 * point, except that A_log and dt_bias may be NULL when KDA_FUSE_GATE is
 * clear, and lower_bound is ignored when KDA_GATE_UNBOUNDED is set.
 */
int kda_fwd_ex(const void *q, const void *k, const void *v, const void *g, const void *beta,
               float scale, void *out, const float *A_log, const float *dt_bias, float lower_bound,
               const void *initial_state, int initial_dtype, void *final_state, int final_dtype,
               const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H, int64_t K,
               int64_t V, uint32_t flags, void *workspace, size_t workspace_bytes, void *stream);
int kda_fwd_recurrent_ex(const void *q, const void *k, const void *v, const void *g,
                         const void *beta, float scale, void *out, const float *A_log,
                         const float *dt_bias, float lower_bound, const void *initial_state,
                         int initial_dtype, void *final_state, int final_dtype,
                         const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H,
                         int64_t K, int64_t V, uint32_t flags, void *stream);

/*
 * kda_fwd_noalloc -- kda_fwd_ex for callers that cannot allocate device memory
 * (code under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc). The same operation, arguments, switches, rules and errors as
 * kda_fwd_ex, without the workspace arguments: the workspace is a fixed array
 * of KDA_NOALLOC_CAPACITY bytes in device memory that the library holds on
 * every GPU it runs on, from its first use there until the process ends. The
 * call itself allocates nothing and issues no memset or copy.
 *   - Calls whose full workspace exceeds the capacity run in windows (see
 *     kda_fwd_workspace_min); calls whose kda_fwd_workspace_min(B, T, H, N)
 *     exceeds it (fixed length: B * H beyond about 1,890; varlen: H beyond
 *     about 1,300 at moderate T and N) are rejected on the host with
 *     KDA_ERR_CAPACITY, before anything is launched. Decode-sized calls need
 *     no workspace at all.
 *   - The array of the CURRENT device is used: `stream` must belong to it.
 *     The array's device address is looked up once per device, on the first
 *     call there (KDA_ERR_HIP if that fails).
 *   - Every call on one GPU shares that GPU's array and leaves its contents
 *     behind; nothing in it needs clearing (each call writes every word it
 *     reads). Calls that overlap on one device (several streams or host
 *     threads) RACE on the array: the caller must serialise them.
 * kda_noalloc_capacity() returns KDA_NOALLOC_CAPACITY.
 */
#define KDA_NOALLOC_CAPACITY ((size_t)256 << 20)
int kda_fwd_noalloc(const void *q, const void *k, const void *v, const void *g, const void *beta,
                    float scale, void *out, const float *A_log, const float *dt_bias,
                    float lower_bound, const void *initial_state, int initial_dtype,
                    void *final_state, int final_dtype, const int64_t *cu_seqlens, int64_t N,
                    int64_t B, int64_t T, int64_t H, int64_t K, int64_t V, uint32_t flags,
                    void *stream);
size_t kda_noalloc_capacity(void);

/* ---- states in the slots of a cache ----------------------------------------
 *
 * A cache ("pool") holds the states of many sequences in S slots of equal size,
 * for L layers: contiguous [L, S, slot]. The slots' contents are the states that
 * kda_fwd, kda_fwd_recurrent and kda_glr_fwd take and return (for KDA a slot is
 * [H, V, K], for the gated linear recurrence [D]); slot s of a sequence is the
 * same in every layer. Slot numbers are int32 on the device; used[s] is nonzero
 * where slot s is held. Everything runs on the device and in stream order, so
 * the calls can be captured into a graph.
 *
 * Rules of every kda_cache_* call: S <= 2^24, L >= 1, slot_bytes >= 1; pool is
 * aligned to 16 bytes, used, src, dst, slots, remap and table to 4; the arrays do
 * not overlap each other (KDA_ERR_VALUE where one that is written is given twice).
 * n may be 0 (nothing is done; the index arrays may then be NULL). A slot number
 * outside [0, S) is never followed: what it means is said at each call.
 *
 * kda_cache_copy: in every layer, slot dst[i] becomes a copy of slot src[i],
 *   0 <= i < n. Pairs with a number outside [0, S) or with src[i] == dst[i] do
 *   nothing. No slot may be the target of two pairs, or the target of one and the
 *   source of another: the slots concerned then hold unspecified bytes of the
 *   slots involved (no other slot is touched).
 *
 * kda_cache_fork: a new slot for each of n requests. Request i is a used slot
 *   src[i] in [0, S) to copy (several may name the same), or -1 for a slot of
 *   zeros. The requests, in their order, take the free slots in ascending order:
 *   dst[i] is the new slot, its contents are written in every layer and its used
 *   flag becomes 1. dst[i] = -1, and nothing else, where src[i] is neither -1 nor
 *   a slot that was used before the call, and where no free slot is left.
 *
 * kda_cache_free: used[slots[i]] = 0 for every slots[i] in [0, S); others are
 *   passed over, and naming a slot twice is naming it once.
 *
 * kda_cache_compact: moves states to the front, so that the n_used used slots are
 *   slots 0 .. n_used - 1. The free slots below n_used, in ascending order, take
 *   the contents of the used slots from n_used on, in ascending order; all other
 *   slots keep their place. remap[s] (int32 [S], OUTPUT) is the new number of
 *   slot s, or -1 where it was free; used is rewritten (1 below n_used, 0 from
 *   there on). table (int32 [n] or NULL) holds slot numbers that are replaced by
 *   their new ones, -1 for free slots and numbers outside [0, S). workspace:
 *   kda_cache_workspace_size(S) bytes, 256-byte aligned.
 *
 * A pool has slots of one size. Two of them under the same slot numbers (the states
 * of KDA and those of a recurrence) are forked by kda_cache_fork on one and
 * kda_cache_copy with the same src and dst on the other, which leaves the slots of
 * requests -1 there as they were: a sequence begins in them from slot -1 (in_slots
 * of kda_fwd_slots and kda_glr_step: zeros). kda_cache_compact rewrites used, so the
 * second pool's call takes a copy of used from before the first.
 */
size_t kda_cache_workspace_size(int64_t S);
int kda_cache_copy(void *pool, int64_t L, int64_t S, size_t slot_bytes, const int32_t *src, const int32_t *dst,
                   int64_t n, void *stream);
int kda_cache_fork(void *pool, int64_t L, int64_t S, size_t slot_bytes, int32_t *used, const int32_t *src,
                   int32_t *dst, int64_t n, void *stream);
int kda_cache_free(int32_t *used, int64_t S, const int32_t *slots, int64_t n, void *stream);
int kda_cache_compact(void *pool, int64_t L, int64_t S, size_t slot_bytes, int32_t *used, int32_t *remap,
                      int32_t *table, int64_t n, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_fwd_slots -- kda_fwd_recurrent_ex with the states in the slots of a cache's
 * layer: state is [S, H, V, K] (one layer of a pool), sequence n starts from slot
 * in_slots[n] (a number outside [0, S): from zeros) and leaves its state in slot
 * out_slots[n] (outside [0, S): not written), for empty sequences too. in_slots
 * and out_slots are int32 of the number of sequences (N, or B without
 * cu_seqlens) and may be the same array. Several sequences may start from one
 * slot; no slot may be left a state by two sequences, or by one sequence while
 * another starts from it. state_dtype is KDA_STATE_BF16 or KDA_STATE_FP32,
 * 1 <= S <= 2^24. Every other argument and rule is kda_fwd_recurrent_ex's.
 */
int kda_fwd_slots(const void *q, const void *k, const void *v, const void *g, const void *beta,
                  float scale, void *out, const float *A_log, const float *dt_bias, float lower_bound,
                  void *state, int state_dtype, int64_t S, const int32_t *in_slots, const int32_t *out_slots,
                  const int64_t *cu_seqlens, int64_t N, int64_t B, int64_t T, int64_t H, int64_t K,
                  int64_t V, uint32_t flags, void *stream);

/* Element types of the operators below (the state codes' values, and fp16). */
enum kda_dtype {
    KDA_BF16 = 1,
    KDA_FP32 = 2,
    KDA_FP16 = 3
};

/* ---- gated linear recurrence -----------------------------------------------
 *
 * Per sequence and channel, from the state h of before its first token:
 *     h_t = exp(g_t) h_{t-1} + x_t,      y_t = h_t
 * g is the log-decay, as kda_fwd takes it with KDA_FUSE_GATE clear (not clamped
 * here): g <= 0 forgets. A gate whose exponential is below 2^-126 (g < -87.4: -inf
 * and a type's lowest value among them) starts over from x_t, whatever state is
 * before it, infinities and NaN too; no gradient passes it, and its own is 0. All
 * others multiply: an infinite state stays infinite. Gates above 0 are taken as
 * they are; where their exponentials' product over 1024 tokens overflows fp32,
 * results are unspecified. The backward pass, with dy_t
 * and the final state's gradient d_final added at the last token:
 *     G_t = dy_t + exp(g_{t+1}) G_{t+1}
 *     dx_t = G_t,   dg_t = G_t exp(g_t) h_{t-1},   d_initial = exp(g_first) G_first
 * States and sums are fp32 throughout; every output is rounded once.
 *
 *   x, g, y, dy, dx, dg   [B, T, D] in `dtype` (KDA_BF16, KDA_FP32 or KDA_FP16).
 *                         T may be 0 (they hold no element and may be NULL).
 *   D                     channels, 1 <= D <= 2^22, any number (whole multiples
 *                         of 16 bytes are fastest)
 *   initial_state, final_state, their dtypes, cu_seqlens, N, B, T
 *                         as for kda_fwd, with states [B|N, D]. A state is aligned
 *                         to as many of its elements as 16 bytes of x hold (at most
 *                         to 16 bytes) where D is a multiple of that number, else to
 *                         its element: as every layer of a cache [L, S, D] is.
 *                         d_final and d_initial likewise. Tokens of a packed
 *                         batch that no sequence covers are not used, and their
 *                         outputs are left as they were.
 *   carry                 fp32 [kda_glr_carry_rows(B, T), D]: the state that enters
 *                         every 128th of the B * T packed tokens. kda_glr_fwd writes
 *                         it where it is not NULL; kda_glr_bwd needs the one of the
 *                         same x, g, initial_state and boundaries. Its contents
 *                         where a sequence begins are unspecified.
 *   d_final, d_final_dtype, d_initial, d_initial_dtype
 *                         gradient of final_state (NULL/KDA_STATE_NONE: zero) and
 *                         of initial_state (NULL/KDA_STATE_NONE: not written),
 *                         [B|N, D] bf16/fp32 each. An empty sequence's d_initial is
 *                         its d_final. d_initial may be neither d_final nor
 *                         initial_state (KDA_ERR_VALUE).
 *   workspace             caller-owned, kda_glr_workspace_size(B, T, D, N) bytes
 *                         (N = 0 without cu_seqlens) for either direction, 256-byte
 *                         aligned; contents need no initialisation and are clobbered
 * Outputs do not overlap inputs, except that final_state may be initial_state. The
 * workspace is one call's until that call's work is done: calls that overlap in it
 * give unspecified results, NaN among them, after a wait of seconds (workgroups hand
 * states to each other through it; a wait ends after KDA_GLR_POLLS polls of about a
 * microsecond, by default 2^24).
 * Results do not depend on timing: the same call gives the same bits. cu_seqlens'
 * contents are the caller's precondition: non-decreasing, within 0 .. T. KDA_VALIDATE=1
 * checks kda_fwd's rule, with cu[0] = 0 and cu[N] = T, so it also refuses packed
 * batches with tokens that no sequence covers.
 */
int64_t kda_glr_carry_rows(int64_t B, int64_t T);   /* 0 for invalid sizes, as below */
size_t kda_glr_workspace_size(int64_t B, int64_t T, int64_t D, int64_t N);
int kda_glr_fwd(const void *x, const void *g, void *y, int dtype, const void *initial_state, int initial_dtype,
                void *final_state, int final_dtype, float *carry, const int64_t *cu_seqlens, int64_t N, int64_t B,
                int64_t T, int64_t D, void *workspace, size_t workspace_bytes, void *stream);
int kda_glr_bwd(const void *x, const void *g, const void *dy, int dtype, const float *carry,
                const void *initial_state, int initial_dtype, const void *d_final, int d_final_dtype, void *dx,
                void *dg, void *d_initial, int d_initial_dtype, const int64_t *cu_seqlens, int64_t N, int64_t B,
                int64_t T, int64_t D, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_glr_step -- one token for each of N sequences, the states in the slots of a
 * cache's layer [S, D] (bf16/fp32): y[n] = exp(g[n]) state[in_slots[n]] + x[n], left
 * in slot out_slots[n]. x, g, y are [N, D] in `dtype`; the rules for slots are
 * kda_fwd_slots', the state's alignment kda_glr_fwd's. N >= 0.
 */
int kda_glr_step(const void *x, const void *g, void *y, int dtype, void *state, int state_dtype, int64_t S,
                 const int32_t *in_slots, const int32_t *out_slots, int64_t N, int64_t D, void *stream);

/* ---- layer norm --------------------------------------------------------------
 *
 * Per row of D elements, with the row's mean m and r = 1 / sqrt(variance + eps)
 * (variance over D, not D - 1):
 *     y = (x - m) r weight + bias
 *     a = dy weight,  c1 = mean(a),  c2 = mean(a (x - m) r)
 *     dx = r (a - c1 - (x - m) r c2)
 *     d_weight = sum over rows of dy (x - m) r,   d_bias = sum over rows of dy
 * Statistics and sums are fp32; every output is rounded once.
 *
 *   x, y, dy, dx      [M, D] in `dtype` (KDA_BF16, KDA_FP32 or KDA_FP16), M >= 0,
 *                     1 <= D <= 2^24. A row per token (D the model's width), or per
 *                     token and head (D = 128 and M = B * T * H on kda_fwd's out).
 *   weight, bias      fp32 [D], or NULL (ones, zeros)
 *   eps               finite, >= 0
 *   mean, rstd        fp32 [M]: written by kda_layernorm_fwd where not NULL, read
 *                     by kda_layernorm_bwd (needed there where M > 0). The forward
 *                     pass centres rows beyond fp32's step of their mean; the
 *                     backward pass takes mean and rstd as they are given, rounded.
 *   d_weight, d_bias  fp32 [D] or NULL, overwritten (zeros where M = 0). Their sums
 *                     have an order of their own that no timing changes.
 *   dx                may be NULL (only the weight's and bias's gradients are wanted)
 *   workspace         caller-owned, kda_layernorm_workspace_size(M, D) bytes,
 *                     256-byte aligned, needed where d_weight or d_bias is given
 * y may be x, and dx may be dy or x; other outputs do not overlap inputs.
 */
size_t kda_layernorm_workspace_size(int64_t M, int64_t D);
int kda_layernorm_fwd(const void *x, const float *weight, const float *bias, float eps, void *y, int dtype,
                      float *mean, float *rstd, int64_t M, int64_t D, void *stream);
int kda_layernorm_bwd(const void *dy, const void *x, const float *weight, const float *mean, const float *rstd,
                      void *dx, int dtype, float *d_weight, float *d_bias, int64_t M, int64_t D, void *workspace,
                      size_t workspace_bytes, void *stream);

/* kda_status_string -- static description of a status code (never NULL). */
const char *kda_status_string(int status);

/* kda_version -- library version string, e.g. "0.1.0 gfx950". */
const char *kda_version(void);

/*
 * Per-kernel timing of kda_fwd (a measurement hook; results are unchanged).
 *
 * kda_profile_start(max_calls): from now on, each of the next max_calls
 *   kda_fwd calls records HIP events on its stream before its first kernel and
 *   after each kernel (the events are created here, not per call, with
 *   hipEventDisableSystemFence: they only measure time and add no cache
 *   write-back to the timed work, so they must not be used to order anything
 *   with the host or other devices). Calls
 *   beyond max_calls are not timed. Starting again discards earlier recordings.
 *   Returns KDA_ERR_VALUE unless 1 <= max_calls <= 65536, KDA_ERR_HIP if an
 *   event cannot be created.
 * kda_profile_stop(total_ms, launches, n_kernels): waits for the recorded
 *   events and writes, for each kernel i < kda_profile_kernel_count(), the
 *   summed milliseconds over the timed calls into total_ms[i] and the number
 *   of timed calls that launched it into launches[i] (host arrays of
 *   n_kernels >= the kernel count); then stops timing and frees the events.
 *   Returns KDA_ERR_NULL, KDA_ERR_SHAPE (n_kernels too small), KDA_ERR_VALUE
 *   (timing not started) or KDA_ERR_HIP.
 * kda_profile_kernel_name(i): static name of kernel i ("" when out of range).
 * One interval runs from one event to the next on the same stream: the
 * kernel's execution plus its launch gap.
 */
int kda_profile_start(int max_calls);
int kda_profile_stop(double *total_ms, int *launches, int n_kernels);
int kda_profile_kernel_count(void);
const char *kda_profile_kernel_name(int i);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
