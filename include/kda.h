/*
 * kda.h -- C ABI of libkda: Kimi Delta Attention (KDA) prefill and decode on
 * AMD Instinct MI355X (gfx950).
 *
 * The method (Kimi K3 explainer, SemiAnalysis, Chinese translation):
 *   DeltaNet section: delta rule S_t = S_{t-1} - beta_t (S_{t-1} k_t - v_t) k_t^T;
 *   GDN/KDA paragraph: a forget gate alpha is applied to S, and KDA makes
 *   alpha a diagonal matrix (one decay per key channel);
 *   FlashKDA paragraph: the recurrence written with D_t = Diag(alpha_t) and
 *   the delta u_t (decode follows it); prefill unrolls it over chunks of C
 *   tokens (Q_decay, K_restore, causal M_qk, UT transform for the
 *   pseudo-values U), the cumulative decay a being one value per token.
 *
 * Per (sequence, head) chain and token t, with alpha_t = exp(g_t):
 *     S'  = S_{t-1} Diag(alpha_t)
 *     u_t = beta_t (v_t - S' k_t)
 *     S_t = S' + u_t k_t^T
 *     o_t = S_t q_t
 * The state S is stored as written here: shape [Dv][Dk], row = value
 * channel, Dk contiguous, fp32 (so a row's reductions over the key channels
 * read contiguous memory). No 1/sqrt(D) scale and no normalisation is applied;
 * q and k arrive already normalised if the model wants them so.
 *
 * Conventions for every call
 *   - All tensor pointers are DEVICE pointers, dense and contiguous, in the
 *     layouts given below; q, k, v, g and out of kda_prefill must be
 *     16-byte aligned. The caller owns every buffer; the library never allocates or
 *     frees device memory and keeps no mutable global state, with one stated
 *     exception: kda_prefill_noalloc's fixed per-device workspace. Calls from
 *     several host threads at once are safe.
 *   - Calls are asynchronous on `stream` (a hipStream_t; NULL = the null
 *     stream). Nothing is synchronised and no device memory is read on the
 *     host. Kernel faults surface at the caller's next synchronisation.
 *   - Argument checks run on the host before any launch. A negative
 *     kda_status is returned, no kernel is launched and no output is
 *     touched. Launch failures return KDA_ERR_HIP. Nothing throws.
 *   - NaN/Inf inputs give unspecified outputs but no fault.
 */
#ifndef KDA_H
#define KDA_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    KDA_OK = 0,
    KDA_ERR_INVALID_ARG = -1,   /* NULL required pointer, bad size, bad dtype */
    KDA_ERR_UNSUPPORTED = -2,   /* valid but outside the support matrix below */
    KDA_ERR_WORKSPACE = -3,     /* workspace missing or smaller than required */
    KDA_ERR_HIP = -4            /* a HIP launch or query failed */
} kda_status;

typedef enum {
    KDA_F32 = 0,
    KDA_BF16 = 1
} kda_dtype;

/* Layout of the decay gate g (kda_options.gate). */
typedef enum {
    KDA_GATE_CHANNEL = 0,   /* g [..][H][Dk]: one log-decay per key channel (KDA) */
    KDA_GATE_HEAD = 1       /* g [..][H]: one per token and head (Gated DeltaNet);
                               g NULL: no decay (DeltaNet) */
} kda_gate;

/*
 * Options of kda_prefill_ex and kda_decode_ex. A zero-initialised struct (or
 * a NULL pointer) gives kda_prefill's / kda_decode's behaviour.
 *   gate           kda_gate value (else KDA_ERR_INVALID_ARG)
 *   qk_l2norm      nonzero: q and k are L2-normalised over Dk inside the
 *                  kernels, x <- x / sqrt(sum_c x_c^2 + l2norm_eps), as the
 *                  explainer's KDA block does before the recurrence (its
 *                  input-processing paragraph); the inputs are not modified
 *   l2norm_eps     > 0 when qk_l2norm is set (else KDA_ERR_INVALID_ARG)
 *   snapshot_every, max_snapshots, snapshots
 *                  prefill only, as for kda_prefill_snapshots; snapshots NULL
 *                  = none (decode: must be NULL)
 */
typedef struct {
    int gate;
    int qk_l2norm;
    float l2norm_eps;
    int snapshot_every;
    int max_snapshots;
    float *snapshots;
} kda_options;

/* Library version, (major << 16) | (minor << 8) | patch. */
int kda_version(void);

/* Human-readable name of a kda_status value (static string, never NULL). */
const char *kda_status_string(int status);

/*
 * Bytes of device workspace kda_prefill needs for these sizes. A pure host
 * function of its arguments (0 is a valid answer). T_total is the number of
 * tokens over all sequences (B*T for dense input). Returns 0 for sizes
 * kda_prefill would reject. On the MFMA shapes it is about 66 KB per
 * (chunk, head), except for one long sequence (see kda_prefill), where it is
 * that of two windows of 512 chunks plus one fp32 state per head.
 */
size_t kda_prefill_workspace_size(int N, int T_total, int H, int Dk, int Dv, int C,
                                  kda_dtype io_dtype);

/*
 * kda_prefill -- chunked prefill over whole sequences, dense or packed
 * (varlen), with an optional initial state (append-prefill after a cached
 * prefix: the prefix cache of the explainer's KV-cache section stores
 * exactly this state).
 *
 * Layouts (token-major, T_total = B*T):
 *   q, k   [T_total][H][Dk]   io_dtype
 *   v      [T_total][H][Dv]   io_dtype
 *   g      [T_total][H][Dk]   fp32, natural-log decay (alpha = exp(g); g <= 0
 *                              is the intended domain, g = -inf wipes a channel)
 *   beta   [T_total][H]       beta_dtype
 *   S0     [N][H][Dv][Dk]     fp32 initial state, or NULL for a zero state
 *   out    [T_total][H][Dv]   out_dtype, o_t for every token
 *   S_out  [N][H][Dv][Dk]     fp32 final state, or NULL to skip it; may be
 *                              the same pointer as S0 (updated in place)
 *   cu_seqlens  int32 [N+1] device array of token offsets with
 *               cu_seqlens[0] = 0 and cu_seqlens[N] = T_total (varlen, then
 *               B must be 1), or NULL: then N must equal B and sequence n
 *               is tokens [n*T, (n+1)*T).
 * Chunks of C tokens restart at every sequence start; the last chunk of a
 * sequence may be short; a zero-length sequence gives S_out = S0. Results do
 * not depend on C beyond rounding.
 *
 * Support matrix (else KDA_ERR_UNSUPPORTED):
 *   Dk == Dv in {64, 128}; C in {16, 32, 64}; H * Dv * C * 4 <= INT_MAX (the
 *     kernels address one chunk of a token-major tensor with 32-bit offsets);
 *   io_dtype KDA_F32: fp32 arithmetic throughout, beta_dtype and out_dtype
 *     must be KDA_F32;
 *   io_dtype KDA_BF16: bf16 q/k/v, beta_dtype KDA_BF16 or KDA_F32, out_dtype
 *     KDA_BF16 or KDA_F32 (a bf16 `out` is the round-to-nearest-even of the
 *     fp32 value the same kernel would store). At Dk = Dv = 128, C = 64 the
 *     contractions run on fp16 MFMA (the state and U split into fp16 hi + lo
 *     parts, about 22 significant bits, where they feed the state) and fp32
 *     MFMA, with fp32 accumulation and an fp32 state; other bf16 shapes run
 *     fp32 arithmetic.
 *   Value range of the bf16 path: v and S0 of any magnitude (each (sequence,
 *     head, value-column tile) is scaled internally by a power of two from the
 *     running maximum of |S0| and |v|; tested from 1e-7 to 1e3). q and k rows
 *     of L2 norm at most 16 (their products are held in fp16; L2-normalised
 *     inputs, or the qk_l2norm option, satisfy this). As for the recurrence
 *     itself, a step is a contraction only while beta_t ||k_t||^2 <= 2.
 *
 * workspace: device buffer of at least kda_prefill_workspace_size(...) bytes
 * (may be NULL when that size is 0), 256-byte aligned. Its contents on entry
 * are ignored; it must not be used by anything else until the call's work
 * on `stream` has finished.
 *
 * One long sequence (N == 1 with at least 2,048 chunks, on the fp16/fp32 MFMA
 * shapes) runs as a pipeline over windows of 512 chunks: the per-chunk
 * operands of only two windows exist at a time, so the workspace stops
 * growing with T_total. Where the scan (64 workgroups per 8 heads) leaves at
 * least half of the CUs free (H <= 16 on 256 CUs), the preparation of the next window
 * runs on a second HIP stream beside the scan of the current one; that stream
 * and five events are created by the call and released by the runtime once
 * their work has completed, all of the call's work is ordered after earlier
 * work on `stream`, and later work on `stream` after all of it. Otherwise, and
 * while `stream` is being captured into a HIP graph, the windows run in order
 * on `stream` alone (same results).
 */
int kda_prefill(const void *q, const void *k, const void *v, const float *g,
                const void *beta, const float *S0, void *out, float *S_out,
                const int32_t *cu_seqlens, int N, int B, int T, int H, int Dk, int Dv,
                int C, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_prefill_noalloc -- kda_prefill without a caller workspace, for callers
 * that cannot allocate device memory: code under HIP graph capture, tight
 * serving loops, harnesses that forbid hipMalloc. It calls no allocator.
 *
 * All arguments, layouts, the support matrix and the results as for
 * kda_prefill (the same kernels run). The workspace is instead a fixed array
 * of KDA_NOALLOC_SCRATCH_BYTES (128 MiB) in the library's device memory, one
 * per GPU, held from the library's first use on that GPU until the process
 * ends. Sizes whose workspace (kda_prefill_workspace_size) exceeds it return
 * KDA_ERR_WORKSPACE before anything is launched. It creates no stream or
 * event either: one long sequence runs its windows in order on `stream`.
 * The array is looked up on
 * the device current at the call, and `stream` must belong to that device.
 * Every call on one GPU shares the array: calls that overlap in time on the
 * same GPU (different streams, or host threads without ordering) race and
 * give undefined results. Calls ordered on one stream are safe; nothing in
 * the array needs to be cleared between them.
 */
#define KDA_NOALLOC_SCRATCH_BYTES (128u << 20)
int kda_prefill_noalloc(const void *q, const void *k, const void *v, const float *g,
                        const void *beta, const float *S0, void *out, float *S_out,
                        const int32_t *cu_seqlens, int N, int B, int T, int H, int Dk, int Dv,
                        int C, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                        void *stream);

/*
 * kda_prefill_snapshots -- kda_prefill that also saves intermediate states
 * for prefix caching. Linear attention keeps one fixed-size state per chain
 * instead of a growing KV cache, so a prefix cache must hold the state at
 * chosen token offsets (Explainer, KV-cache section: coarse fixed intervals
 * plus prompt boundaries, the latter being S_out).
 *
 * All arguments as for kda_prefill, plus:
 *   snapshot_every  tokens between snapshots, a multiple of C (else
 *                   KDA_ERR_UNSUPPORTED), >= 1
 *   max_snapshots   capacity per sequence, >= 1
 *   snapshots       [N][H][max_snapshots][Dv][Dk] fp32 device buffer (not NULL).
 *                   Slot k-1 of sequence n receives the state after its first
 *                   k * snapshot_every tokens, for every k >= 1 with
 *                   k * snapshot_every <= length(n) and k <= max_snapshots.
 *                   Other slots are not written.
 * Snapshots are exact intermediate states of the same computation (the values
 * S_out would have for the truncated sequence, up to rounding).
 */
int kda_prefill_snapshots(const void *q, const void *k, const void *v, const float *g,
                          const void *beta, const float *S0, void *out, float *S_out,
                          const int32_t *cu_seqlens, int N, int B, int T, int H, int Dk, int Dv,
                          int C, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                          int snapshot_every, int max_snapshots, float *snapshots,
                          void *workspace, size_t workspace_bytes, void *stream);

/*
 * gdn_prefill -- the same chunked prefill with the scalar forget gate of Gated
 * DeltaNet, or with no gate (DeltaNet). Per the explainer's GDN/KDA paragraph,
 * GDN applies one forget gate alpha to the whole state, which KDA refines into
 * one decay per key channel; the DeltaNet section's delta rule is the case
 * alpha = 1. The recurrence above holds with Diag(alpha_t) = alpha_t I.
 *
 * All arguments and the support matrix as for kda_prefill, except:
 *   g   [B][T][H] fp32 (with cu_seqlens: [1][T_total][H]): the natural-log
 *       decay of each token and head, alpha_t = exp(g_t) for every key channel;
 *       or NULL: alpha_t = 1 (DeltaNet). 4-byte aligned; no 16-byte rule.
 * kda_prefill_workspace_size gives the workspace. The kernels are kda_prefill's,
 * reading one decay per token and head.
 */
int gdn_prefill(const void *q, const void *k, const void *v, const float *g,
                const void *beta, const float *S0, void *out, float *S_out,
                const int32_t *cu_seqlens, int N, int B, int T, int H, int Dk, int Dv,
                int C, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_decode -- one token per sequence, state updated in place. This is one
 * step of the recurrence above (the explainer's decode paragraph: about
 * 7*D^2 FLOPs and about 8*D^2 bytes per head, the fp32 state being read and
 * written once).
 *
 *   q, k   [N][H][Dk]  io_dtype        v    [N][H][Dv]  io_dtype
 *   g      [N][H][Dk]  fp32            beta [N][H]      beta_dtype
 *   S      [N][H][Dv][Dk] fp32, read and overwritten with the new state
 *   out    [N][H][Dv]  out_dtype, o_t = S_t q_t
 * Support: Dk == Dv in {64, 128}; io_dtype KDA_BF16 or KDA_F32; beta_dtype
 * and out_dtype either; N*H >= 1.
 */
int kda_decode(const void *q, const void *k, const void *v, const float *g,
               const void *beta, float *S, void *out, int N, int H, int Dk, int Dv,
               kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype, void *stream);

/*
 * gdn_decode -- kda_decode with the scalar gate of Gated DeltaNet (g [N][H]
 * fp32, alpha = exp(g) for every key channel) or none (g NULL: DeltaNet,
 * alpha = 1). Otherwise as kda_decode.
 */
int gdn_decode(const void *q, const void *k, const void *v, const float *g,
               const void *beta, float *S, void *out, int N, int H, int Dk, int Dv,
               kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype, void *stream);

/*
 * kda_prefill_ex -- kda_prefill with options (gate layout, fused q/k L2
 * normalisation, snapshots). The g layout follows opt->gate (see gdn_prefill
 * for KDA_GATE_HEAD); everything else as kda_prefill, with the same workspace.
 */
int kda_prefill_ex(const void *q, const void *k, const void *v, const float *g,
                   const void *beta, const float *S0, void *out, float *S_out,
                   const int32_t *cu_seqlens, int N, int B, int T, int H, int Dk, int Dv,
                   int C, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                   const kda_options *opt, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_decode_ex -- kda_decode with options (gate layout as for gdn_decode
 * when KDA_GATE_HEAD, fused q/k L2 normalisation; no snapshots).
 */
int kda_decode_ex(const void *q, const void *k, const void *v, const float *g,
                  const void *beta, float *S, void *out, int N, int H, int Dk, int Dv,
                  kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype out_dtype,
                  const kda_options *opt, void *stream);

/*
 * kda_output_gate -- the output side of the KDA block: per-head RMS norm of
 * the attention output, a per-channel weight and a sigmoid output gate. The
 * explainer's KDA section (its input/output paragraph) says KDA's output is
 * normalised per head and controlled by an output forget gate computed by a
 * projection; the projection needs trained weights, so the caller passes its
 * result (the gate pre-activation z). Per row r, head h and channel j:
 *     out[r][h][j] = o[r][h][j] / sqrt(mean_j' o[r][h][j']^2 + eps)
 *                    * weight[j] * 1 / (1 + exp(-z[r][h][j]))
 *   o        [rows][H][Dv] o_dtype (e.g. kda_prefill's out, rows = tokens, or
 *            kda_decode's out, rows = sequences)
 *   gate     [rows][H][Dv] gate_dtype, the pre-activation z
 *   weight   [Dv] fp32, shared by the heads; NULL = all ones
 *   out      [rows][H][Dv] out_dtype; may be o itself when out_dtype ==
 *            o_dtype (in place), no other overlap is allowed
 *   eps      > 0
 * o, gate, out and weight must be 16-byte aligned. Supported: Dv in {64, 128}
 * (else KDA_ERR_UNSUPPORTED); rows == 0 launches nothing (o, gate and out may
 * then be NULL). Arithmetic in fp32; a bf16 out is the round-to-nearest-even
 * of the fp32 result. Errors:
 * KDA_ERR_INVALID_ARG for NULL o / gate / out with rows > 0, rows < 0, H < 1, Dv < 1,
 * eps <= 0 or NaN, a bad dtype, misalignment, rows * H > INT_MAX, or an
 * in-place call that changes the dtype.
 */
int kda_output_gate(const void *o, const void *gate, const float *weight, void *out, int rows, int H,
                    int Dv, float eps, kda_dtype o_dtype, kda_dtype gate_dtype, kda_dtype out_dtype,
                    void *stream);

/*
 * kda_recurrent -- the recurrence over a few tokens of each sequence, with the
 * states in a pool of slots: checking draft tokens (the state after every one
 * is kept, and decoding goes on from the accepted one), continuing a shared
 * prefix without copying its state, or a step of ragged length per sequence.
 *
 *   q, k   [T_total][H][Dk] io_dtype      v    [T_total][H][Dv] io_dtype
 *   g      [T_total][H][Dk] fp32, or with opt->gate == KDA_GATE_HEAD
 *          [T_total][H], NULL = no decay
 *   beta   [T_total][H] beta_dtype        out  [T_total][H][Dv] out_dtype
 *   S      [slots][H][Dv][Dk] fp32, the pool, 16-byte aligned
 *   cu_seqlens  int32 [N+1]: sequence n is tokens cu_seqlens[n] up to
 *          cu_seqlens[n+1]. It may be empty; out rows (and states) of tokens
 *          that belong to no sequence are left as they were. Offsets outside
 *          [0, T_total] are cut to it. Offsets that fall make sequences share
 *          tokens: their out rows are then undefined (no fault).
 *   slot_in   int32 [N]: the slot a sequence starts from; a value outside
 *          [0, slots), or slot_in NULL: the zero state
 *   slot_out  int32 [T_total]: the slot that receives the state after a token;
 *          outside [0, slots), or slot_out NULL: that state is not kept
 * cu_seqlens, slot_in and slot_out are device arrays. A sequence may keep a
 * state in the slot it started from (in place), and several sequences may start
 * from one slot. A slot that one sequence writes must not be the start, nor be
 * written by, another sequence of the call: those contents are undefined (no
 * fault). Slots that no token names are not written. If one sequence names a
 * slot for several tokens, the last one stays.
 *
 * Arithmetic in fp32. opt: gate and qk_l2norm as for kda_decode_ex; snapshots
 * must be NULL; opt may be NULL. Support: Dk == Dv in {64, 128}; N * H * Dk^2 / 16
 * below 2^32. q, k, v, a per-channel g, S and out 16-byte aligned; out must be none
 * of the other buffers. T_total == 0 launches nothing.
 */
int kda_recurrent(const void *q, const void *k, const void *v, const float *g, const void *beta, float *S,
                  void *out, const int32_t *cu_seqlens, const int32_t *slot_in, const int32_t *slot_out, int N,
                  int T_total, int H, int Dk, int Dv, int slots, kda_dtype io_dtype, kda_dtype beta_dtype,
                  kda_dtype out_dtype, const kda_options *opt, void *stream);

/*
 * kda_recurrent_padded -- kda_recurrent for an out whose contents on entry mean nothing:
 * with zero_rows 1, rows before cu_seqlens[0] and from cu_seqlens[N] on become zero (0: they
 * are left as they were; else KDA_ERR_INVALID_ARG). All else as there.
 */
int kda_recurrent_padded(const void *q, const void *k, const void *v, const float *g, const void *beta, float *S,
                         void *out, const int32_t *cu_seqlens, const int32_t *slot_in, const int32_t *slot_out, int N,
                         int T_total, int H, int Dk, int Dv, int slots, kda_dtype io_dtype, kda_dtype beta_dtype,
                         kda_dtype out_dtype, int zero_rows, const kda_options *opt, void *stream);

/*
 * kda_prefill_backward -- the gradient of kda_prefill (and, with
 * opt->gate == KDA_GATE_HEAD, of gdn_prefill; with qk_l2norm, through the
 * normalisation): from dout, the gradient of out, and dS_out, the gradient of
 * S_out, to those of every input. Nothing of the forward call is needed: the
 * states at the chunk borders are computed again.
 *
 *   q, k, v, g, beta, S0, cu_seqlens, N, B, T, H, Dk, Dv  as for kda_prefill;
 *          cu_seqlens may end before T_total, offsets below the one before them or
 *          outside [0, T_total] are cut
 *   dout    [T_total][H][Dv] dout_dtype
 *   dS_out  [N][H][Dv][Dk] fp32, or NULL: the final state has no gradient
 *   dq, dk  [T_total][H][Dk], dv [T_total][H][Dv]   io_dtype
 *   dg      fp32, g's layout; NULL exactly when g is
 *   dbeta   [T_total][H] beta_dtype
 *   dS0     [N][H][Dv][Dk] fp32, or NULL to skip it (S0 may be NULL, a zero state)
 * Rows of tokens in no sequence of a packed batch are left as they were. A
 * sequence of length zero gives dS0 = dS_out.
 *
 * Arithmetic, states and their gradients in fp32 (matrix products on fp32
 * instructions, or on bf16 ones with every operand cut in three), for any magnitude
 * of dout whose products stay between about 1e-33 and 3.3e38; a bf16 gradient
 * is the rounded fp32 value. A log-decay of -104 or less
 * (exp is 0 in fp32; -inf wipes a channel) has gradient 0. Results repeat bit for
 * bit.
 * Support: Dk == Dv in {64, 128}; io_dtype KDA_F32 with fp32 beta and dout, or
 * KDA_BF16 with either; (T_total / 64 + N + 1) * H below 2^23. opt->snapshots
 * must be NULL; opt may be NULL. All tensors but beta, dbeta and a per-head g, dg
 * must be 16-byte aligned. No gradient may be any other buffer of the call.
 * workspace: kda_prefill_backward_workspace_size bytes, 256-byte aligned, its contents
 * ignored, not used by anything else until the call's work has finished. That is about
 * (ceil(T_total / 64) + N) * H times 381 KB at Dk = 128, 169 KB at 64: every sequence,
 * an empty one too, adds a chunk's share for each head.
 * The size function returns 0 for sizes that the call rejects.
 */
size_t kda_prefill_backward_workspace_size(int N, int T_total, int H, int Dk, int Dv);
int kda_prefill_backward(const void *q, const void *k, const void *v, const float *g, const void *beta,
                         const void *dout, const float *S0, const float *dS_out, void *dq, void *dk, void *dv,
                         float *dg, void *dbeta, float *dS0, const int32_t *cu_seqlens, int N, int B, int T, int H,
                         int Dk, int Dv, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype dout_dtype,
                         const kda_options *opt, void *workspace, size_t workspace_bytes, void *stream);

/*
 * kda_prefill_backward_padded -- kda_prefill_backward for buffers whose contents on
 * entry mean nothing: rows of tokens in no sequence of a packed batch, whose gradient is
 * zero, become zero in the gradients that zero_rows names (KDA_ZERO_* added up; other
 * bits: KDA_ERR_INVALID_ARG), and are left as they were in the others. All else as there.
 */
typedef enum {
    KDA_ZERO_DQ = 1,
    KDA_ZERO_DK = 2,
    KDA_ZERO_DV = 4,
    KDA_ZERO_DG = 8,
    KDA_ZERO_DBETA = 16,
    KDA_ZERO_ALL = 31
} kda_zero_rows;
int kda_prefill_backward_padded(const void *q, const void *k, const void *v, const float *g, const void *beta,
                                const void *dout, const float *S0, const float *dS_out, void *dq, void *dk, void *dv,
                                float *dg, void *dbeta, float *dS0, const int32_t *cu_seqlens, int N, int B, int T,
                                int H, int Dk, int Dv, kda_dtype io_dtype, kda_dtype beta_dtype, kda_dtype dout_dtype,
                                int zero_rows, const kda_options *opt, void *workspace, size_t workspace_bytes,
                                void *stream);

/*
 * kda_output_gate_backward -- the gradient of kda_output_gate. With
 * r = 1 / sqrt(mean_j o_j^2 + eps), n = o r, s = sigmoid(z) and x = dout s w:
 *     d_o = r (x - n mean_j(x n)),  dgate = dout n w s (1 - s),
 *     dweight = sum over rows and heads of dout s n
 *   o, gate, weight, rows, H, Dv, eps  as for kda_output_gate
 *   dout [rows][H][Dv] dout_dtype;  d_o o_dtype;  dgate gate_dtype
 *   dweight [Dv] fp32, or NULL to skip it (weight may be NULL, ones)
 * fp32 arithmetic (o of at most 1e18 in magnitude: its squares are summed); dweight's sum has a
 * fixed order. rows == 0 gives dweight = 0.
 * No gradient may be any other buffer of the call. Alignment, support and errors
 * as for kda_output_gate. workspace: kda_output_gate_backward_workspace_size bytes
 * (at most 1 MiB), 256-byte aligned; may be NULL when that is 0 or dweight is NULL.
 */
size_t kda_output_gate_backward_workspace_size(int rows, int H, int Dv);
int kda_output_gate_backward(const void *o, const void *gate, const void *dout, const float *weight, void *d_o,
                             void *dgate, float *dweight, int rows, int H, int Dv, float eps, kda_dtype o_dtype,
                             kda_dtype gate_dtype, kda_dtype dout_dtype, void *workspace, size_t workspace_bytes,
                             void *stream);

/*
 * kda_layer_norm -- the block's input norm: layer norm of every row of W
 * channels, or its RMS norm (rms nonzero):
 *     mean = sum_c x_c / W (0 for RMS),  rstd = 1 / sqrt(sum_c (x_c - mean)^2 / W + eps)
 *     out_c = (x_c - mean) rstd weight_c + bias_c
 *   x    [rows][W] x_dtype;  out [rows][W] out_dtype, may be x itself when the
 *        dtypes are the same
 *   weight, bias  [W] fp32; NULL = ones, zeros
 *   mean, rstd    [rows] fp32, kept for the backward pass; NULL to skip (mean
 *        must be NULL for RMS)
 *   eps  > 0
 * fp32 arithmetic (x of at most 1e17 in magnitude: its squares are summed); the variance
 * is the mean square of centred values. Any W from 1
 * to 16384 (above: KDA_ERR_UNSUPPORTED) and any alignment of the element type;
 * fastest with W a multiple of 8 and 16-byte aligned x, out, weight and bias.
 * rows == 0 launches nothing.
 */
int kda_layer_norm(const void *x, const float *weight, const float *bias, void *out, float *mean, float *rstd,
                   int rows, int W, float eps, int rms, kda_dtype x_dtype, kda_dtype out_dtype, void *stream);

/*
 * kda_layer_norm_backward -- its gradient. With n = (x - mean) rstd and h = dy weight:
 *     dx = rstd (h - n mean_c(h n) - mean_c(h))      (RMS: without the last term)
 *     dweight = sum over rows of dy n,  dbias = sum over rows of dy
 *   mean, rstd  as kda_layer_norm left them (mean NULL for RMS)
 *   dy [rows][W] dy_dtype;  dx [rows][W] x_dtype
 *   dweight, dbias  [W] fp32, or NULL to skip
 * The sums over rows have a fixed order. rows == 0 gives zeros. No gradient may be
 * any other buffer of the call. Sizes and alignment as for kda_layer_norm.
 * workspace: kda_layer_norm_backward_workspace_size bytes (at most 4 KiB x W),
 * 256-byte aligned; may be NULL when that is 0 or dweight and dbias are NULL.
 */
size_t kda_layer_norm_backward_workspace_size(int rows, int W);
int kda_layer_norm_backward(const void *x, const void *dy, const float *mean, const float *rstd, const float *weight,
                            void *dx, float *dweight, float *dbias, int rows, int W, int rms, kda_dtype x_dtype,
                            kda_dtype dy_dtype, void *workspace, size_t workspace_bytes, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* KDA_H */
