/*
 * gdn.h -- C ABI of the Gated DeltaNet (GDN) token-mixer library for AMD
 * Instinct MI355X (gfx950).
 *
 * The calls that form the GDN layer's data-parallel hot path:
 *
 *   gdn_build_conv_chunks       host: exact (sequence, 8-token chunk) list
 *   gdn_causal_conv1d_varlen    GPU: width-4 causal conv over packed prefill
 *   gdn_causal_conv1d_varlen_tiles
 *                               GPU: the same, 8- or 16-token programs
 *   gdn_causal_conv1d_update    GPU: single-token conv for decode
 *   gdn_fused_recurrent_decode  GPU: gated delta rule over packed tokens
 *   gdn_chunk_gated_delta_rule  GPU: the same rule over prefill tokens,
 *                               chunkwise on the matrix cores
 *   gdn_chunk_workspace_size    host: scratch bytes the chunkwise call needs
 *   gdn_fused_conv_decode       GPU: conv update + gated delta rule, one launch
 *   gdn_chunk_rule_and_fused_decode
 *                               GPU: the chunkwise rule on a step's prefill
 *                               tokens and the fused decode of its decode
 *                               rows, sharing one grid
 *
 * and those of the hybrid model's other layers on the same engine step:
 *
 *   gdn_build_step_tables       GPU: a step's query_start_loc, positions,
 *                               cache slots, pages and conv descriptors from
 *                               the requests' lengths
 *   gdn_rope_frequencies        host: rotary frequencies, scaled for long
 *                               contexts
 *   gdn_rope_append_kv8         GPU: rotary positions on q and k; k and v
 *                               written into the 8-bit paged cache
 *   gdn_paged_attention_kv8     GPU: attention over that cache, any mix of
 *                               decode rows and prompt chunks
 *   gdn_paged_attention_kv8_workspace_size
 *                               host: scratch bytes the attention needs
 *   gdn_rope_append_kv4         GPU: the same, into the 4-bit paged cache
 *   gdn_paged_read_kv4          GPU: ranges of keys and values out of that
 *                               cache, as packed bf16 rows
 *   gdn_paged_attention_kv4     GPU: attention over the 4-bit cache
 *   gdn_paged_attention_kv4_workspace_size
 *                               host: scratch bytes the attention needs
 *   gdn_gated_rms_norm          GPU: norm of each head with its output gate
 *   gdn_residual_rms_norm       GPU: norm after a block, its gate, residual
 *                               scale and sum, and the next block's norm
 *
 * Conventions shared by every call
 * --------------------------------
 * - bf16 values travel as raw 16-bit patterns (gdn_bf16).  fp32 -> bf16
 *   rounding is round-to-nearest-even.  Arithmetic is fp32.
 * - Unless marked "host", a pointer is a device pointer (HBM of the current
 *   HIP device).  The caller owns every buffer, scratch workspaces included.
 *   The library never allocates or frees device memory and caches no caller
 *   pointers; its only global state is the static scratch of
 *   gdn_chunk_rule_and_fused_decode_noalloc (and that scratch's per-device
 *   address).  It may be called from several threads, each on its own
 *   buffers.
 * - GPU calls validate their arguments on the host, then enqueue kernels on
 *   `stream` (a hipStream_t; NULL = the default stream) and return without
 *   waiting.  A call that returns an error enqueued nothing.
 * - "Stride" arguments count elements, not bytes, between consecutive token
 *   rows.  Within a row, channels (or heads, then head elements) are packed.
 * - Vector-access contract: bf16 row pointers and strides are multiples of
 *   8 elements (16 bytes); fp32 state pointers are 16-byte aligned.
 * - Sequences are packed back to back.  query_start_loc[s] .. [s+1] is the
 *   token range of sequence s; it must be non-decreasing with
 *   query_start_loc[0] == 0 and query_start_loc[num_seqs] == num_tokens
 *   (device-side preconditions: not checked, but the kernels clamp every
 *   range to [0, num_tokens), so a malformed array gives wrong results,
 *   never an access outside the buffers).  state_indices[s] selects the
 *   state slot of sequence s; a negative index marks padding: that sequence
 *   is skipped, its outputs and every slot are left untouched.  An index at
 *   or past num_slots is skipped the same way (the kernels check it).  Slots
 *   used in one call must be distinct.
 *
 * Return values: GDN_OK or a negative gdn_status; gdn_last_error() then
 * describes the failure (thread-local, valid until the thread's next call).
 */
#ifndef GDN_H
#define GDN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef uint16_t gdn_bf16;

/* Tokens per conv program: one descriptor covers tokens
 * [qsl[seq] + 8*chunk, min(qsl[seq] + 8*chunk + 8, qsl[seq+1])). */
#define GDN_CONV_CHUNK_TOKENS 8
/* The only conv width the library implements. */
#define GDN_CONV_WIDTH 4

typedef struct gdn_conv_chunk {
    int32_t seq;    /* sequence index into query_start_loc */
    int32_t chunk;  /* 8-token chunk index within that sequence */
} gdn_conv_chunk;

typedef enum gdn_status {
    GDN_OK = 0,
    GDN_ERR_INVALID = -1,      /* NULL pointer, bad count, bad pair, aliasing */
    GDN_ERR_UNSUPPORTED = -2,  /* width != 4, misaligned, unsupported head dim */
    GDN_ERR_CAPACITY = -3,     /* descriptor buffer or workspace too small */
    GDN_ERR_HIP = -4           /* the HIP runtime reported an error */
} gdn_status;

/* Text of the last error on the calling thread ("" after a success). */
const char *gdn_last_error(void);

/*
 * gdn_build_conv_chunks -- host only, synchronous.
 *
 * Source: page "perf(gdn): dispatch exact causal-conv chunks", section "What
 * changed": the conv is dispatched as one program per exact (sequence,
 * 8-token chunk) pair; the list is built once per engine step, uploaded once
 * and reused by every GDN layer of the step.
 *
 * For s = 0 .. num_seqs-1 and c = 0 .. ceil(L_s / 8) - 1 (L_s =
 * qsl_host[s+1] - qsl_host[s]) appends {s, c}: sequences in order, chunks
 * ascending; empty sequences contribute nothing.
 *
 *   qsl_host   host, int32 [num_seqs + 1], non-decreasing (checked)
 *   out_host   host, gdn_conv_chunk [capacity]; may be NULL if capacity == 0
 *   n_out      host, receives the number of descriptors needed
 *
 * Errors: GDN_ERR_INVALID (NULL qsl_host/n_out, num_seqs < 0, capacity < 0,
 * decreasing qsl, count overflow); GDN_ERR_CAPACITY when the list does not
 * fit: *n_out then holds the required count and out_host[0 .. capacity) holds
 * the first descriptors.  Pass capacity 0 to query the count.
 */
int gdn_build_conv_chunks(const int32_t *qsl_host, int32_t num_seqs,
                          gdn_conv_chunk *out_host, int32_t capacity, int32_t *n_out);

/*
 * gdn_causal_conv1d_varlen -- depthwise causal conv1d over packed prefill
 * tokens, width 4, optional SiLU, per-sequence carried state.
 *
 * Sources: page "perf(gdn): dispatch exact causal-conv chunks", section "What
 * changed" (one program per exact chunk descriptor; the descriptor is
 * optional and its (buffer, count) pair is validated together, reviewer
 * comment on the same page); page "RTX 5070 Ti: close Qwen3.5-4B TTFT, TPOT,
 * and VRAM gaps vs vLLM", section "Existing evidence" (width-4 conv).
 *
 * For each sequence s with slot = state_indices[s] >= 0, tokens [a, a+L):
 *   window e = h || x[a .. a+L), h = conv_state[slot] if has_initial_state[s]
 *             else 3 zero rows (oldest first)
 *   y[a+p][c] = act(bias[c] + sum_{j<4} weight[c][j] * e[p+j][c])
 *             (weight[c][3] multiplies the current token; act = SiLU if silu)
 *   conv_state[slot] <- e[L .. L+3)   (the three newest window rows)
 *
 *   x                 bf16 [num_tokens][x_stride], channels [0, channels)
 *   weight            bf16 [channels][4]
 *   bias              bf16 [channels], or NULL for no bias
 *   conv_state        bf16 [num_slots][3][channels], read and written in place
 *   query_start_loc   int32 [num_seqs + 1]
 *   state_indices     int32 [num_seqs]
 *   has_initial_state uint8 [num_seqs], or NULL (= every sequence has one)
 *   chunks, n_chunks  descriptors from gdn_build_conv_chunks on the same
 *                     query_start_loc, copied to the device: the only
 *                     dispatch, so required whenever num_tokens > 0.  Both
 *                     NULL/0 is valid only with num_tokens == 0 (the call
 *                     then enqueues nothing); exactly one of them set is an
 *                     error.  A descriptor whose seq is not in [0, num_seqs)
 *                     or whose chunk lies past its sequence is skipped.
 *   y                 bf16 [num_tokens][y_stride]; must not overlap x,
 *                     conv_state, weight or bias
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative count,
 * (chunks == NULL) != (n_chunks == 0), num_tokens > 0 without descriptors,
 * fewer than ceil(num_tokens / 8) or more than num_tokens descriptors,
 * stride < channels, y overlapping x, conv_state, weight or bias,
 * num_slots < 1); GDN_ERR_UNSUPPORTED (width != 4, channels % 8, strides or
 * pointers off the 16-byte contract); GDN_ERR_HIP (launch failure).
 */
int gdn_causal_conv1d_varlen(const gdn_bf16 *x, int64_t x_stride,
                             const gdn_bf16 *weight, const gdn_bf16 *bias,
                             gdn_bf16 *conv_state, int32_t num_slots,
                             const int32_t *query_start_loc,
                             const int32_t *state_indices,
                             const uint8_t *has_initial_state,
                             const gdn_conv_chunk *chunks, int32_t n_chunks,
                             gdn_bf16 *y, int64_t y_stride,
                             int32_t num_seqs, int32_t num_tokens, int32_t channels,
                             int32_t width, int32_t silu, void *stream);

/*
 * gdn_causal_conv1d_varlen_tiles -- gdn_causal_conv1d_varlen with a choice of
 * program size: each program takes descriptors_per_program consecutive
 * entries of the descriptor list (1: 8-token programs, exactly
 * gdn_causal_conv1d_varlen; 2: 16-token programs).  The descriptors stay the
 * exact 8-token ones; when a program's second descriptor continues its first
 * (same sequence, next chunk), its 3-row halo is the first's last rows, so a
 * 16-token program reads 19 rows where two 8-token programs read 22.
 * Results are bit-identical to gdn_causal_conv1d_varlen for every input.
 *
 * Sources: page "RTX 5070 Ti: close Qwen3.5-4B TTFT, TPOT, and VRAM gaps vs
 * vLLM", section "Existing evidence" (the multi-token tile arm of the conv);
 * page "perf(gdn): dispatch exact causal-conv chunks", section "What changed"
 * (exact 8-token descriptors).
 *
 * Arguments, layouts and errors as gdn_causal_conv1d_varlen, plus:
 *   descriptors_per_program  1 or 2, else GDN_ERR_UNSUPPORTED; with 2, x_stride
 *                            and y_stride must be at most 2^26 elements
 *                            (GDN_ERR_UNSUPPORTED otherwise)
 */
int gdn_causal_conv1d_varlen_tiles(const gdn_bf16 *x, int64_t x_stride,
                                   const gdn_bf16 *weight, const gdn_bf16 *bias,
                                   gdn_bf16 *conv_state, int32_t num_slots,
                                   const int32_t *query_start_loc,
                                   const int32_t *state_indices,
                                   const uint8_t *has_initial_state,
                                   const gdn_conv_chunk *chunks, int32_t n_chunks,
                                   gdn_bf16 *y, int64_t y_stride,
                                   int32_t num_seqs, int32_t num_tokens, int32_t channels,
                                   int32_t width, int32_t silu,
                                   int32_t descriptors_per_program, void *stream);

/*
 * gdn_causal_conv1d_update -- the same conv for one new token per sequence
 * (decode): row b uses slot state_indices[b] (negative: row skipped).
 *
 *   y[b][c] = act(bias[c] + sum_{j<3} weight[c][j] * conv_state[slot][j][c]
 *                 + weight[c][3] * x[b][c])
 *   conv_state[slot] <- (conv_state[slot][1], conv_state[slot][2], x[b])
 *
 * Identical arithmetic to gdn_causal_conv1d_varlen, so a sequence advanced
 * by this call gives bit-identical outputs to the varlen call on the whole
 * sequence.  Layouts as above with num_tokens = batch.
 *
 * Errors: as gdn_causal_conv1d_varlen (minus the descriptor pair).
 */
int gdn_causal_conv1d_update(const gdn_bf16 *x, int64_t x_stride,
                             const gdn_bf16 *weight, const gdn_bf16 *bias,
                             gdn_bf16 *conv_state, int32_t num_slots,
                             const int32_t *state_indices,
                             gdn_bf16 *y, int64_t y_stride,
                             int32_t batch, int32_t channels, int32_t width,
                             int32_t silu, void *stream);

/*
 * gdn_fused_recurrent_decode -- the gated delta rule, fused per (sequence,
 * v-head), token by token, over packed tokens (decode: one token each).
 *
 * Sources: the fused GDN decode with a register-resident state named on page
 * "RTX 5070 Ti: close Qwen3.5-4B TTFT, TPOT, and VRAM gaps vs vLLM", section
 * "Existing evidence"; the rule itself from Yang, Kautz, Hatamizadeh, "Gated
 * Delta Networks: Improving Mamba2 with Delta Rule" (ICLR 2025).
 *
 * For each sequence s with slot = state_indices[s] >= 0 and v-head h (q/k
 * head hk = h / (num_v_heads / num_k_heads)):
 *   S = has_initial_state[s] ? state[slot][h] : 0      (dv x dk, fp32)
 *   for each token t of s:
 *     qh, kh = q[t][hk], k[t][hk], each divided by sqrt(sum x^2 + 1e-6)
 *              when qk_l2norm != 0
 *     a = exp(g[t][h]),  b = beta[t][h]
 *     S = a * S * (I - b kh kh^T) + b v[t][h] kh^T
 *     o[t][h] = scale * S qh
 *   state[slot][h] = S
 *
 *   q, k     bf16, token t head j at q + t*q_stride + j*head_k_dim
 *   v        bf16, token t head h at v + t*v_stride + h*head_v_dim
 *            (q, k and v may be column views of one conv output row)
 *   g, beta  fp32 [num_tokens][num_v_heads]  (g = log decay)
 *   state    fp32 [num_slots][num_v_heads][head_v_dim][head_k_dim], in place;
 *            row i (one v channel) is contiguous along head_k_dim
 *   query_start_loc  int32 [num_seqs + 1], or NULL: one token per sequence
 *            (then num_tokens == num_seqs and token s belongs to sequence s)
 *   o        bf16, token t head h at o + t*o_stride + h*head_v_dim
 *
 * Launch shape: with query_start_loc == NULL the call is laid out for
 * bandwidth (every state row streamed once); with it, for per-token
 * latency.  Both shapes do identical per-token arithmetic, so splitting a
 * sequence across calls gives bit-identical results.
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative count,
 * num_v_heads % num_k_heads, strides too small, num_tokens != num_seqs
 * without query_start_loc, o overlapping q/k/v/g/beta/state); GDN_ERR_UNSUPPORTED
 * (head_k_dim not in {16, 32, 64, 128}, head_v_dim not a positive multiple
 * of 8 up to 256, alignment contract); GDN_ERR_HIP.
 */
int gdn_fused_recurrent_decode(const gdn_bf16 *q, int64_t q_stride,
                               const gdn_bf16 *k, int64_t k_stride,
                               const gdn_bf16 *v, int64_t v_stride,
                               const float *g, const float *beta,
                               float *state, int32_t num_slots,
                               const int32_t *query_start_loc,
                               const int32_t *state_indices,
                               const uint8_t *has_initial_state,
                               gdn_bf16 *o, int64_t o_stride,
                               int32_t num_seqs, int32_t num_tokens,
                               int32_t num_k_heads, int32_t num_v_heads,
                               int32_t head_k_dim, int32_t head_v_dim,
                               float scale, int32_t qk_l2norm, void *stream);

/*
 * gdn_chunk_gated_delta_rule -- the same gated delta rule as
 * gdn_fused_recurrent_decode over packed prefill tokens, evaluated chunk by
 * chunk (64 tokens) in the equivalent matrix form on the matrix cores.
 *
 * Sources: the rule from Yang, Kautz, Hatamizadeh, "Gated Delta Networks:
 * Improving Mamba2 with Delta Rule" (ICLR 2025); its chunkwise form follows
 * from unrolling the recurrence over a chunk: with u_t the per-token update
 * vector, (I + A) U = R for a unit lower-triangular A built from the chunk's
 * keys, gates and betas (the pages name the prefill GDN path only by its
 * test, page "Qwen3.5-4b BF16 optimization and correctness (sm_120)",
 * section "Evidence").
 *
 * Two kernels run on `stream`: one prepares, for every (64-token chunk,
 * v-head) in parallel, the parts that do not depend on the state (the
 * inverse of I + A, the masked decayed Q K^T, per-token factors) in
 * `workspace`; the second walks each sequence's chunks in order.
 *
 * Arguments, layouts, state semantics and errors are those of
 * gdn_fused_recurrent_decode, except:
 *   query_start_loc  required (int32 [num_seqs + 1])
 *   head_k_dim       must be 128
 *   head_v_dim       a positive multiple of 32 up to 256
 *   q/k/v/o_stride   below 2^24 elements (32-bit offsets within a chunk)
 *   workspace        device scratch owned by the caller, 256-byte aligned,
 *                    at least gdn_chunk_workspace_size(num_seqs, num_tokens,
 *                    num_k_heads, num_v_heads) bytes; its contents on entry
 *                    do not matter and are overwritten.  Calls that share a
 *                    workspace must not overlap in time.
 * Errors beyond those: GDN_ERR_INVALID (NULL workspace, or a workspace
 * whose first gdn_chunk_workspace_size bytes overlap q, k, v, g, beta,
 * state or o), GDN_ERR_UNSUPPORTED
 * (misaligned workspace, a token stride of 2^24 elements or more),
 * GDN_ERR_CAPACITY (workspace_bytes too small).
 * Results equal the per-token recurrence up to fp32 rounding (a different
 * association of the same sums); sequence lengths need not be multiples of
 * 64.  Splitting a sequence across calls moves the chunk boundaries, so it
 * changes results only within that rounding.
 */
size_t gdn_chunk_workspace_size(int32_t num_seqs, int32_t num_tokens,
                                int32_t num_k_heads, int32_t num_v_heads);

int gdn_chunk_gated_delta_rule(const gdn_bf16 *q, int64_t q_stride,
                               const gdn_bf16 *k, int64_t k_stride,
                               const gdn_bf16 *v, int64_t v_stride,
                               const float *g, const float *beta,
                               float *state, int32_t num_slots,
                               const int32_t *query_start_loc,
                               const int32_t *state_indices,
                               const uint8_t *has_initial_state,
                               gdn_bf16 *o, int64_t o_stride,
                               int32_t num_seqs, int32_t num_tokens,
                               int32_t num_k_heads, int32_t num_v_heads,
                               int32_t head_k_dim, int32_t head_v_dim,
                               void *workspace, size_t workspace_bytes,
                               float scale, int32_t qk_l2norm, void *stream);

/*
 * gdn_fused_conv_decode -- one decode step of the whole mixer: the
 * single-token conv update of every channel fused with the gated delta rule
 * on its output, in one launch.
 *
 * Sources: the width-4 conv and the fused GDN decode of page "RTX 5070 Ti:
 * close Qwen3.5-4B TTFT, TPOT, and VRAM gaps vs vLLM", section "Existing
 * evidence"; the rule from Yang, Kautz, Hatamizadeh, "Gated Delta Networks"
 * (ICLR 2025).
 *
 * Equivalent, bit for bit, to
 *   gdn_causal_conv1d_update(x, ..., y_tmp, ...)      (y_tmp in bf16)
 *   gdn_fused_recurrent_decode(q = y_tmp[:, 0 : HK dk],
 *                              k = y_tmp[:, HK dk : 2 HK dk],
 *                              v = y_tmp[:, 2 HK dk :], ...)
 * where the conv row is laid out q | k | v (channels = 2 HK dk + HV dv) and
 * batch row b uses slot state_indices[b] in both pools (negative: skipped).
 * The conv output is written to y only when y is not NULL.
 *
 *   x            bf16 [batch][x_stride]
 *   conv_weight  bf16 [channels][4];  conv_bias bf16 [channels] or NULL
 *   conv_state   bf16 [num_conv_slots][3][channels], in place
 *   g, beta      fp32 [batch][num_v_heads]
 *   state        fp32 [num_slots][num_v_heads][head_v_dim][head_k_dim], in place
 *   o            bf16, row b head h at o + b*o_stride + h*head_v_dim
 *   y            bf16 [batch][y_stride] or NULL
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative batch, slot
 * counts < 1, num_v_heads % num_k_heads, strides too small, o or y
 * overlapping x, state or conv_state, o overlapping g or beta, y
 * overlapping o); GDN_ERR_UNSUPPORTED (head dims as for
 * gdn_fused_recurrent_decode, more than 8192 conv channels read by one q/k
 * head group, alignment contract); GDN_ERR_HIP.
 */
int gdn_fused_conv_decode(const gdn_bf16 *x, int64_t x_stride,
                          const gdn_bf16 *conv_weight, const gdn_bf16 *conv_bias,
                          gdn_bf16 *conv_state, int32_t num_conv_slots,
                          const float *g, const float *beta,
                          float *state, int32_t num_slots,
                          const int32_t *state_indices,
                          gdn_bf16 *o, int64_t o_stride,
                          gdn_bf16 *y, int64_t y_stride,
                          int32_t batch, int32_t num_k_heads, int32_t num_v_heads,
                          int32_t head_k_dim, int32_t head_v_dim, int32_t silu,
                          float scale, int32_t qk_l2norm, void *stream);

/*
 * gdn_chunk_rule_and_fused_decode -- the recurrence of one engine step that
 * holds both prefill tokens and decode rows (after the prefill tokens' conv):
 * gdn_chunk_gated_delta_rule on the prefill tokens and gdn_fused_conv_decode
 * on the decode rows, with the chunkwise form's serial scan and the decode
 * sharing one grid.
 *
 * Sources: the serving workload of page "RTX 5070 Ti: close Qwen3.5-4B
 * TTFT, TPOT, and VRAM gaps vs vLLM", section "Problem" (concurrency 32, a
 * 2048-token batch budget), whose engine steps batch decode rows with
 * chunked-prefill tokens; the two operations are those of the two calls
 * named above.
 *
 * Why one grid: the scan walks each sequence's chunks in order on one
 * workgroup per (sequence, v-head, 64 v rows) and leaves most CUs idle for
 * its whole run; the decode is bandwidth-bound and independent of it.  The
 * scan's workgroups are placed first, the decode units take the CUs left,
 * then each CU a scan workgroup releases.
 *
 * Arguments:
 *   q .. workspace_bytes  the prefill tokens, exactly as the same-named
 *                         arguments of gdn_chunk_gated_delta_rule
 *   dec_x .. silu         the decode rows, as the arguments x .. silu of
 *                         gdn_fused_conv_decode (dec_g, dec_beta,
 *                         dec_state_indices, dec_o, dec_y, dec_batch for its
 *                         g, beta, state_indices, o, y, batch)
 *   state .. qk_l2norm    shared by both: the layer's recurrent-state pool
 *                         and head shape
 * The two halves run concurrently: a state slot may be used by only one of
 * them (state_indices and dec_state_indices disjoint, apart from negative
 * entries; a device-side precondition, not checked).  Every result --
 * o, dec_o, dec_y, the state slots and conv_state -- is bit-identical to
 * calling gdn_chunk_gated_delta_rule and then gdn_fused_conv_decode (either
 * order) with the same arguments.  An empty half (num_seqs or num_tokens 0,
 * dec_batch 0) is skipped: its other arguments are not checked (pointers
 * may be NULL) and overlap nothing; the call with both empty enqueues
 * nothing.  Shapes the shared grid does not take
 * (head_v_dim not a multiple of 64) run the two operations as consecutive
 * launches on `stream`.
 *
 * Errors: every error of either call, with its arguments; GDN_ERR_INVALID
 * when what one half writes (o, the workspace; dec_o, dec_y, conv_state)
 * overlaps an operand of the other half (q, k, v, g, beta, o, workspace;
 * dec_x, conv_weight, conv_bias, conv_state, dec_g, dec_beta, dec_o, dec_y).
 */
int gdn_chunk_rule_and_fused_decode(
    /* prefill tokens */
    const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
    const gdn_bf16 *v, int64_t v_stride, const float *g, const float *beta,
    const int32_t *query_start_loc, const int32_t *state_indices,
    const uint8_t *has_initial_state, gdn_bf16 *o, int64_t o_stride,
    int32_t num_seqs, int32_t num_tokens, void *workspace, size_t workspace_bytes,
    /* decode rows */
    const gdn_bf16 *dec_x, int64_t dec_x_stride,
    const gdn_bf16 *conv_weight, const gdn_bf16 *conv_bias,
    gdn_bf16 *conv_state, int32_t num_conv_slots,
    const float *dec_g, const float *dec_beta, const int32_t *dec_state_indices,
    gdn_bf16 *dec_o, int64_t dec_o_stride, gdn_bf16 *dec_y, int64_t dec_y_stride,
    int32_t dec_batch, int32_t silu,
    /* both */
    float *state, int32_t num_slots, int32_t num_k_heads, int32_t num_v_heads,
    int32_t head_k_dim, int32_t head_v_dim, float scale, int32_t qk_l2norm,
    void *stream);

/* Bytes of the static device scratch gdn_chunk_rule_and_fused_decode_noalloc
 * uses as its chunk workspace (one copy per GPU). */
#define GDN_NOALLOC_SCRATCH_BYTES ((size_t)64 << 20)

/*
 * gdn_chunk_rule_and_fused_decode_noalloc -- gdn_chunk_rule_and_fused_decode
 * without the workspace arguments, for callers that cannot allocate device
 * memory: code under HIP graph capture, tight serving loops, harnesses that
 * forbid allocation.  The chunk workspace is instead a static device array
 * of GDN_NOALLOC_SCRATCH_BYTES bytes inside the library, one per GPU, held
 * until the process ends.
 *
 * Arguments, results and errors are those of gdn_chunk_rule_and_fused_decode
 * (which it calls with that array as the workspace); results are
 * bit-identical to it.  The call allocates nothing: no hipMalloc, no
 * hipFree, no allocating library routine.  Its first call on a device looks
 * up that device's copy of the array (hipGetSymbolAddress) and keeps the
 * address.
 *
 * Limit: a prefill half whose gdn_chunk_workspace_size(num_seqs, num_tokens,
 * num_k_heads, num_v_heads) exceeds GDN_NOALLOC_SCRATCH_BYTES is refused
 * with GDN_ERR_CAPACITY (at 16 q/k and 32 v heads that is about 96 chunks of
 * 64 tokens, e.g. 2048 tokens in up to 64 sequences).
 *
 * Sharing: every call on one GPU uses that GPU's one array, which keeps what
 * the last call wrote (nothing in it needs to start cleared: each call
 * writes every record it reads).  Calls that overlap in time on one GPU --
 * on different streams or from different threads -- race on the array and
 * give wrong results; the caller must order them, e.g. on one stream.
 */
int gdn_chunk_rule_and_fused_decode_noalloc(
    /* prefill tokens */
    const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
    const gdn_bf16 *v, int64_t v_stride, const float *g, const float *beta,
    const int32_t *query_start_loc, const int32_t *state_indices,
    const uint8_t *has_initial_state, gdn_bf16 *o, int64_t o_stride,
    int32_t num_seqs, int32_t num_tokens,
    /* decode rows */
    const gdn_bf16 *dec_x, int64_t dec_x_stride,
    const gdn_bf16 *conv_weight, const gdn_bf16 *conv_bias,
    gdn_bf16 *conv_state, int32_t num_conv_slots,
    const float *dec_g, const float *dec_beta, const int32_t *dec_state_indices,
    gdn_bf16 *dec_o, int64_t dec_o_stride, gdn_bf16 *dec_y, int64_t dec_y_stride,
    int32_t dec_batch, int32_t silu,
    /* both */
    float *state, int32_t num_slots, int32_t num_k_heads, int32_t num_v_heads,
    int32_t head_k_dim, int32_t head_v_dim, float scale, int32_t qk_l2norm,
    void *stream);

/* ------------------------------------------------------------------------
 * The full-attention layers' side of an engine step, and the norms between
 * blocks.  A call without tokens (rows, requests) is valid, enqueues nothing
 * and checks no more than its counts; gdn_build_step_tables fills its outputs
 * still.
 * ------------------------------------------------------------------------ */

/* Sequences one gdn_build_step_tables call takes at most. */
#define GDN_STEP_MAX_SEQS 4096

/*
 * gdn_build_step_tables -- what every layer of an engine step needs to know
 * about its requests, built on the GPU from their lengths in one launch:
 * nothing is read back to the host, so the call can sit in a captured graph.
 *
 * With c = context_lens[s] tokens of request s already in the cache, n =
 * query_lens[s] new ones (negative lengths count as 0) and P = page_size:
 *   query_start_loc[s] = sum of n over the requests before s;  seq_lens[s] = c + n
 *   request s holds ceil(c / P) pages, the first entries of its block_table
 *   row, and takes ceil((c + n) / P) - ceil(c / P) more.  The pages taken,
 *   counted p = 0, 1, ... over the requests in order, come off the end of the
 *   free list, free_pages[num_free[0] - 1 - p], and are appended to the rows.
 *   positions[t] = c + i and slot_mapping[t] = block_table[s][(c + i) / P] * P
 *   + (c + i) % P for t = query_start_loc[s] + i
 *   chunks: {s, i} for i < ceil(n / 8), sequences in order: the list that
 *   gdn_build_conv_chunks makes of query_start_loc
 *   counts[0..3] = tokens, descriptors, pages taken, pages missing
 * The caller's free list is not changed: the last counts[2] of its first
 * num_free[0] entries are in use after the call.
 *
 * Room: tokens past num_tokens and descriptors past n_chunks are not written
 * (counts still has the full numbers).  Entries past the step's own are
 * filled: positions and slot_mapping with -1, descriptors with {-1, 0}, which
 * the conv calls skip.  When the free list runs out, or a row of max_pages
 * entries is full, the missing page's entry (inside the row) and its tokens'
 * slots are -1 and counts[3] counts it.  Sums past 2^31 - 1 saturate.
 *
 *   context_lens, query_lens  int32 [num_seqs]
 *   free_pages                int32 [free_capacity];  num_free: int32 [1],
 *                             on the device, clamped to [0, free_capacity]
 *   block_table               int32 [num_seqs][block_table_stride], in place,
 *                             max_pages entries of a row in use
 *   query_start_loc           int32 [num_seqs + 1];  seq_lens: int32 [num_seqs]
 *   positions                 int32 [num_tokens];  slot_mapping: int64 [num_tokens]
 *   chunks                    gdn_conv_chunk [n_chunks], or NULL/0
 *   counts                    int32 [4]
 *
 * Errors: GDN_ERR_INVALID (a pointer NULL that its count needs, negative
 * counts, page_size not a power of two from 1 to 1024, max_pages < 1,
 * block_table_stride < max_pages, (chunks == NULL) != (n_chunks == 0), an
 * output overlapping an input or another output); GDN_ERR_UNSUPPORTED (more
 * than GDN_STEP_MAX_SEQS requests, a pointer off its type's alignment);
 * GDN_ERR_HIP.
 */
int gdn_build_step_tables(const int32_t *context_lens, const int32_t *query_lens, int32_t num_seqs,
                          const int32_t *free_pages, const int32_t *num_free, int32_t free_capacity,
                          int32_t *block_table, int64_t block_table_stride, int32_t max_pages,
                          int32_t page_size, int32_t *query_start_loc, int32_t *seq_lens,
                          int32_t *positions, int64_t *slot_mapping, int32_t num_tokens,
                          gdn_conv_chunk *chunks, int32_t n_chunks, int32_t *counts, void *stream);

typedef enum gdn_rope_scaling {
    GDN_ROPE_PLAIN = 0,    /* f_i = base^(-2i / rotary_dim) */
    GDN_ROPE_LINEAR = 1,   /* positions interpolated: f_i / factor */
    GDN_ROPE_NTK = 2,      /* base raised to base * factor^(r / (r - 2)), r = rotary_dim */
    GDN_ROPE_YARN = 3      /* slow frequencies divided by factor, fast ones kept, a ramp between */
} gdn_rope_scaling;

/*
 * gdn_rope_frequencies -- host only, synchronous: the rotary_dim / 2 rotary
 * frequencies in 64 bits, and the factor of the rotated elements that goes
 * with them (1 but for YaRN).
 *
 * Sources: Su et al., "RoFormer" (2021) for the frequencies; Peng et al.,
 * "YaRN: Efficient Context Window Extension of Large Language Models" (2023)
 * for the scalings: with r_i = original_context f_i / 2pi turns over the
 * original context, f_i gamma + (f_i / factor) (1 - gamma), gamma = clamp((r_i
 * - beta_slow) / (beta_fast - beta_slow), 0, 1), and the factor 0.1 ln(factor)
 * + 1.  The ramp is that paper's, linear in turns.  A model that was trained with
 * another one (linear in the pair's number i between the two borders, rounded or
 * not) has other frequencies: pass its own to gdn_rope_append_kv8, which takes
 * any, with its own factor.
 *
 *   out           host, double [rotary_dim / 2]
 *   rope_scale    host, receives the factor
 *   factor        >= 1 (ignored by GDN_ROPE_PLAIN); original_context, beta_fast
 *                 and beta_slow are GDN_ROPE_YARN's (customary: 32 and 1)
 *
 * Errors: GDN_ERR_INVALID (NULL pointers, rotary_dim odd or < 2, base <= 1,
 * an unknown scaling, factor < 1, for NTK rotary_dim 2, for YaRN
 * original_context < 1 or beta_fast <= beta_slow).
 */
int gdn_rope_frequencies(int32_t rotary_dim, double base, int32_t scaling, double factor,
                         double original_context, double beta_fast, double beta_slow,
                         double *out, double *rope_scale);

/*
 * The 8-bit paged cache of gdn_rope_append_kv8 and gdn_paged_attention_kv8:
 *   k_cache  e4m3 (OCP: 4 exponent bits, bias 7, 3 mantissa bits, no
 *            infinities) [num_pages][num_kv_heads][page_size][head_dim]
 *   v_cache  e4m3 [num_pages][num_kv_heads][head_dim][page_size]: a page's
 *            tokens are contiguous for each element, the order in which the
 *            products of weights and values read them
 *   k_scale, v_scale  fp32 [num_pages][num_kv_heads]
 * An element is its code times its page's and head's scale.  page_size is 16,
 * 32 or 64; head_dim 64, 128 or 256.  The caches are 16-byte aligned.
 */

/*
 * gdn_rope_append_kv8 -- rotary positions on q and k, and the new k and v
 * written into the cache, in one launch.
 *
 * For token t and pair i < rotary_dim / 2, with angle positions[t] *
 * frequencies[i]: (a, b) -> rope_scale (a cos - b sin, b cos + a sin), where
 * (a, b) are elements (i, i + rotary_dim / 2) of a head, or (2i, 2i + 1) with
 * interleaved != 0; elements from rotary_dim on are kept.  Angles and products
 * are in 64 bits: a position of a million costs no accuracy.  q_out is rounded
 * to bf16, k to fp32 before it is coded.
 *
 * Cache: token t goes to slot slot_mapping[t] = page * page_size + offset; a
 * slot outside [0, num_pages * page_size) (padding, -1) is not written.  The
 * tokens of one page must be consecutive in the call, at consecutive offsets
 * (the order gdn_build_step_tables gives; otherwise the codes of that page are
 * undefined, but nothing outside the cache is accessed).  With m the largest
 * finite magnitude among a page's and head's new elements, the scale is the
 * least power of two s >= 2^-100 with m <= 448 s -- or the page's present
 * scale, where its tokens begin at an offset above 0 and that is larger.
 * Codes are rounded to nearest even.  Where a page's scale grows, the codes
 * below the first new offset are rounded again to the new one, exact for
 * powers of two but for codes that leave e4m3's normal range.  Infinities and
 * NaN are coded as NaN.  Codes past the last new offset stay as they are.
 *
 *   q, k, v       bf16, token t head j at q + t*q_stride + j*head_dim (may be
 *                 column views of one projection's output); k_stride and
 *                 v_stride below 2^24 elements
 *   q_out         bf16 [.][q_out_stride]: not overlapping q, k or v, or q itself
 *                 with the same stride; q NULL (and q_out NULL): no q
 *   positions     int32 [num_tokens]
 *   slot_mapping  int64 [num_tokens]
 *   frequencies   fp64 [rotary_dim / 2], device; NULL with rotary_dim 0
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative counts, head
 * counts < 1, num_pages < 1, strides too small, q without q_out, an output
 * overlapping an input); GDN_ERR_UNSUPPORTED (page_size, head_dim, rotary_dim
 * not a multiple of 16 from 0 to head_dim, strides or pointers off the
 * alignment contract); GDN_ERR_HIP.
 */
int gdn_rope_append_kv8(const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
                        const gdn_bf16 *v, int64_t v_stride, const int32_t *positions,
                        const int64_t *slot_mapping, const double *frequencies, int32_t rotary_dim,
                        int32_t interleaved, double rope_scale, gdn_bf16 *q_out, int64_t q_out_stride,
                        uint8_t *k_cache, uint8_t *v_cache, float *k_scale, float *v_scale,
                        int32_t num_pages, int32_t page_size, int32_t num_tokens,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void *stream);

/*
 * gdn_paged_attention_kv8 -- attention of a step's tokens over the cache.
 *
 * Request s owns the tokens [a, a + n) of query_start_loc and keys j in [0,
 * L), L = seq_lens[s] (its own new tokens among them); key j is row j %
 * page_size of page block_table[s][j / page_size].  For its token i, at
 * position p = L - n + i, and q head h (kv head h / (num_q_heads /
 * num_kv_heads)):
 *   x_j = scale * (q . k_j);  w = softmax of x over the keys with j <= p if
 *   causal, j > p - window if window > 0;  o = sum_j w_j v_j
 * A token that sees no key gets o = 0.  Keys of a page outside [0, num_pages)
 * (-1 in the block table) or past max_pages are not seen.  Masked keys have
 * no influence whatever their codes and scales hold, NaN included; cache
 * bytes past L are free to hold anything.
 *
 * Scores are products of the cache's codes with q in two 8-bit parts (exact
 * for elements of at least 2^-14 of their head's largest, within 2^-22 of that
 * largest for smaller ones), summed in fp32; softmax statistics and sums are
 * fp32.  A weight is rounded to bf16 in its product with a value, with the
 * values' scale in it: off by at most 2^-8 of itself, however light beside
 * others, while that product is above bf16's least normal value, 2^-126.  o is
 * rounded to bf16.  Its sums are finite where the keys seen times the largest
 * magnitude among their values stay below 2^128.  A token that sees a key of a
 * page whose v_scale is infinite or NaN gets infinite or NaN elements there.
 * Results do not change from call to call (no atomics).
 *
 * With at most as many tokens as requests (num_tokens <= num_seqs) the call
 * takes each request for a few rows, as a decode step's are.  Requests without
 * new tokens count there: a prompt in a batch padded with empty ones up to that
 * point is right but slower (2,000 tokens among 2,000 requests: 171 us at heads
 * of 256 and 195 us at 128; among 1,999: 92 and 79 us; alone: 84 and 62 us).  Leave
 * empty requests out of num_seqs where prompts are among the others.
 *
 *   q            bf16, token t head h at q + t*q_stride + h*head_dim
 *   block_table  int32 [num_seqs][block_table_stride], max_pages entries used
 *   seq_lens     int32 [num_seqs] (negative counts as 0)
 *   max_seq_len  the largest of seq_lens as the caller knows it; it decides
 *                how the work is split, and results do not depend on it but
 *                for rounding (0 < it; a request may be longer).  A bound far
 *                above the lengths costs time: parts come out too long, and few
 *   o            bf16 [.][o_stride], rows of tokens that no request owns are
 *                left as they are; must not overlap an input
 *   workspace    device scratch of gdn_paged_attention_kv8_workspace_size
 *                bytes for these sizes, 256-byte aligned, contents free (may
 *                be NULL when that is 0).  Calls that share one must not
 *                overlap in time.
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative counts,
 * num_q_heads not a positive multiple of num_kv_heads, num_pages or max_pages
 * < 1, max_seq_len < 1, window < 0, strides too small, o or the workspace
 * overlapping an operand); GDN_ERR_UNSUPPORTED (page_size, head_dim, a page of
 * all heads or a row of max_pages pages past 32-bit offsets, alignment
 * contract); GDN_ERR_CAPACITY (workspace too small); GDN_ERR_HIP.
 */
size_t gdn_paged_attention_kv8_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len);

int gdn_paged_attention_kv8(const gdn_bf16 *q, int64_t q_stride, const uint8_t *k_cache,
                            const uint8_t *v_cache, const float *k_scale, const float *v_scale,
                            int32_t num_pages, int32_t page_size, const int32_t *block_table,
                            int64_t block_table_stride, int32_t max_pages, const int32_t *seq_lens,
                            const int32_t *query_start_loc, int32_t max_seq_len,
                            gdn_bf16 *o, int64_t o_stride, int32_t num_seqs, int32_t num_tokens,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                            int32_t causal, int32_t window, void *workspace, size_t workspace_bytes,
                            void *stream);

/*
 * The 4-bit paged cache of gdn_rope_append_kv4, gdn_paged_read_kv4 and
 * gdn_paged_attention_kv4: 4.25 bits per element of a key and 4 bits and two
 * bytes per head of a value, where the 8-bit cache has 8.
 *   k_cache  e2m1 codes (2 exponent bits, 1 mantissa bit: 0, 0.5, 1, 1.5, 2, 3,
 *            4, 6 and a sign) [num_pages][num_kv_heads][page_size][head_dim / 2]:
 *            two elements of a key to a byte, the even one in the low half
 *   k_scale  e8m0 (2^(byte - 127), 255: NaN), one of 32 elements of a key
 *            [num_pages][num_kv_heads][head_dim / 32][page_size]
 *   v_cache  e2m1 codes [num_pages][num_kv_heads][page_size / 16][head_dim][8]:
 *            an element's codes of 16 neighbouring tokens (a granule), two
 *            tokens to a byte, the even one in the low half
 *   v_scale  bf16 [num_pages][num_kv_heads][page_size], one of a token's value
 * An element is its code times its scale.  page_size is 16, 32 or 64; head_dim
 * 64, 128 or 256.  All four are 16-byte aligned.
 */

/*
 * gdn_rope_append_kv4 -- rotary positions on q and k, and the new k and v
 * written into the cache, in one launch.
 *
 * Rotation, positions and frequencies are those of gdn_rope_append_kv8, and so is
 * the order that slot_mapping has to have; angles, sines and cosines times
 * rope_scale, and k's products are in 64 bits, q's products in fp32.
 *
 * Cache: k and v are rounded to nearest even at their scale.  A key's 32
 * elements' scale is the power of two below which their largest magnitude m has
 * two bits: 2^(e - 2), m between 1 and 1.75 times 2^e, or between 0.875 and 1 (so m
 * is met by 3.5 to 7 scales, 7 excluded); 2^-100 at least.  A value's scale is
 * m / 6 rounded to bf16, m the largest magnitude of the token's head; 2^-100 at
 * least.  A block or head with an infinity or NaN has a scale of NaN, and all of
 * it reads as NaN.  (m above 1.75 2^127 reads as infinite.)  What was stored
 * before keeps its codes and scales: a token's do not depend on its neighbours'.
 * New tokens of one granule (16 neighbouring slots) that do not follow each other in
 * the call, with others or padding between them, in another order or with a slot
 * named twice, leave the codes of all that granule's values undefined, those of
 * tokens stored before too; nothing outside the cache is accessed.
 *
 *   q, k, v, q_out, positions, slot_mapping, frequencies, rotary_dim,
 *   interleaved, rope_scale   as gdn_rope_append_kv8's
 *
 * Errors: as gdn_rope_append_kv8's.
 */
int gdn_rope_append_kv4(const gdn_bf16 *q, int64_t q_stride, const gdn_bf16 *k, int64_t k_stride,
                        const gdn_bf16 *v, int64_t v_stride, const int32_t *positions,
                        const int64_t *slot_mapping, const double *frequencies, int32_t rotary_dim,
                        int32_t interleaved, double rope_scale, gdn_bf16 *q_out, int64_t q_out_stride,
                        uint8_t *k_cache, uint8_t *v_cache, uint8_t *k_scale, gdn_bf16 *v_scale,
                        int32_t num_pages, int32_t page_size, int32_t num_tokens,
                        int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, void *stream);

/*
 * gdn_paged_read_kv4 -- ranges of keys and values read back out of the cache:
 * contexts for another attention, another cache or another engine.
 *
 * Request s fills the rows [a, b) of out_start_loc[s], out_start_loc[s + 1]: row
 * a + i is key key_starts[s] + i, as it lies at its row of its page of the block
 * table.  k is exact in bf16, v rounded once.  Rows whose key has no page (-1 in
 * the block table, or outside [0, num_pages), or past max_pages), and rows that no
 * request owns, are left as they are.
 *
 *   block_table    int32 [num_seqs][block_table_stride], max_pages entries used
 *   key_starts     int32 [num_seqs] (negative counts as 0), or NULL: from key 0 on
 *   out_start_loc  int32 [num_seqs + 1], as query_start_loc, clamped to [0, num_rows)
 *   k_out, v_out   bf16, row r head h at k_out + r*k_out_stride + h*head_dim; one
 *                  of them may be NULL: not read
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative counts, num_kv_heads,
 * num_pages or max_pages < 1, strides too small, an output overlapping an input or
 * the other one); GDN_ERR_UNSUPPORTED (page_size, head_dim, alignment contract);
 * GDN_ERR_HIP.
 */
int gdn_paged_read_kv4(const uint8_t *k_cache, const uint8_t *v_cache, const uint8_t *k_scale,
                       const gdn_bf16 *v_scale, int32_t num_pages, int32_t page_size,
                       const int32_t *block_table, int64_t block_table_stride, int32_t max_pages,
                       const int32_t *key_starts, const int32_t *out_start_loc, gdn_bf16 *k_out,
                       int64_t k_out_stride, gdn_bf16 *v_out, int64_t v_out_stride, int32_t num_seqs,
                       int32_t num_rows, int32_t num_kv_heads, int32_t head_dim, void *stream);

/*
 * gdn_paged_attention_kv4 -- attention of a step's tokens over the 4-bit cache.
 *
 * Tokens, requests, masks, pages and what comes of rows that see no key are those
 * of gdn_paged_attention_kv8; a masked key has no influence whatever its codes
 * and scales hold.
 *
 * Scores are products of the cache's codes and scales with q in three 6-bit parts
 * per 32 elements (exact for elements of at least 2^-7 of those 32's largest,
 * within 2^-15 of that largest for smaller ones: bf16 itself is off by up to 2^-9
 * of it there; where that largest is below 2^-110, within 2^-125), summed in fp32;
 * softmax statistics and sums are fp32.  A weight (the heaviest key's is 1) is
 * rounded to bf16 in its product with a value, with the value's scale in it: off
 * by at most 2^-8 of itself while weight times scale is above 2^-118.  o is rounded
 * to bf16.  A head of q with an infinity or NaN gives NaN, and so does a seen key or
 * value whose scale is NaN.  Products of q and k, and scores in units of log2, of
 * 2^127 and more overflow.  Results do not change from call to call (no atomics).
 *
 * The keys of a call with at most as many tokens as requests are divided into
 * parts by max_seq_len and the numbers of requests and kv heads, not by the lengths:
 * - A bound above the lengths costs a second launch and parts without keys (32
 *   requests of 1,100 keys, 16/4 heads of 256: 13.5 us, and 17 with any bound from
 *   4,096 on), and from about 2^20 on the order by length (200 of 1 to 8,000, 32/8 of
 *   128: 139 us, 140 at 131,072 and 151 at 2^20).
 * - With more than 128 (request, kv head) pairs nothing is divided, however long one
 *   request is: 31 of 1,100 keys and one of 131,072, 32/8 of 128, take 676 us.  Such
 *   a request is better off in a call of its own (36 us, and 11 for the others).
 * - A window of more than 1,024 keys is divided as the whole request would be (one
 *   request of 131,072 keys, 32/8 of 128: 18.5 us in a window of 4,096; one of 4,096 keys
 *   11.2).
 * A prompt among as many requests as tokens, empty ones, is right but slower: 2,000
 * tokens among 2,000 requests 92 us at 16/4 heads of 256 and 87 at 32/8 of 128, among
 * 1,999 88 and 102 us, alone 63 and 54 us.
 *
 *   scale        finite, and so its product with log2(e) (below 2^127.47)
 *   others       as gdn_paged_attention_kv8's, the workspace of
 *                gdn_paged_attention_kv4_workspace_size bytes
 *
 * Errors: as gdn_paged_attention_kv8's, and GDN_ERR_INVALID where scale or its
 * product with log2(e) is not finite.
 */
size_t gdn_paged_attention_kv4_workspace_size(int32_t num_tokens, int32_t num_seqs, int32_t num_q_heads,
                                              int32_t num_kv_heads, int32_t head_dim, int32_t max_seq_len);

int gdn_paged_attention_kv4(const gdn_bf16 *q, int64_t q_stride, const uint8_t *k_cache,
                            const uint8_t *v_cache, const uint8_t *k_scale, const gdn_bf16 *v_scale,
                            int32_t num_pages, int32_t page_size, const int32_t *block_table,
                            int64_t block_table_stride, int32_t max_pages, const int32_t *seq_lens,
                            const int32_t *query_start_loc, int32_t max_seq_len,
                            gdn_bf16 *o, int64_t o_stride, int32_t num_seqs, int32_t num_tokens,
                            int32_t num_q_heads, int32_t num_kv_heads, int32_t head_dim, float scale,
                            int32_t causal, int32_t window, void *workspace, size_t workspace_bytes,
                            void *stream);

/*
 * gdn_gated_rms_norm -- root-mean-square norm of each head, times its output
 * gate (the GDN mixer's output norm; without a gate, the norm of q and k
 * heads):
 *   y = x / sqrt(mean(x^2) + eps) * (weight_offset + weight) * silu(gate)
 * over head_dim elements, in fp32, rounded once.  (A head whose sum of squares
 * passes fp32's range, with elements of 2^60 and more, comes out as zeros.)
 *
 *   x, gate, y  bf16, token t head h at x + t*x_stride + h*head_dim; gate may
 *               be NULL; y may be x itself with the same stride
 *   weight      bf16 [head_dim] (weight_offset 1: stored about zero)
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative num_tokens,
 * num_heads < 1, strides too small, y overlapping x otherwise, gate or
 * weight); GDN_ERR_UNSUPPORTED (head_dim not a multiple of 8 up to 512,
 * alignment contract); GDN_ERR_HIP.
 */
int gdn_gated_rms_norm(const gdn_bf16 *x, int64_t x_stride, const gdn_bf16 *gate, int64_t gate_stride,
                       const gdn_bf16 *weight, gdn_bf16 *y, int64_t y_stride, int32_t num_tokens,
                       int32_t num_heads, int32_t head_dim, float eps, float weight_offset, void *stream);

/*
 * gdn_residual_rms_norm -- between two blocks, in one pass over each row:
 *   u = x;  with post_weight: u = u / sqrt(mean(u^2) + eps) * (weight_offset + post_weight)
 *   with gate: u = u * sigmoid(gate)
 *   h = residual + residual_scale * u;  new_residual = h (rounded to bf16)
 *   y = h / sqrt(mean(h^2) + eps) * (weight_offset + weight)
 * in fp32; y is formed from h before its rounding, so the sum's rounding does
 * not enter the next block.  (Sums of squares past fp32's range: as above.)
 *
 *   x, residual, gate, new_residual, y  bf16 [rows][stride], hidden elements
 *               used; gate may be NULL; new_residual may be residual or x, and
 *               y may be x, each itself with the same stride
 *   weight, post_weight  bf16 [hidden]; post_weight may be NULL
 *
 * Errors: GDN_ERR_INVALID (required pointer NULL, negative rows, strides too
 * small, an output overlapping an operand otherwise, or the other output);
 * GDN_ERR_UNSUPPORTED (hidden not a multiple of 8 up to 16384, alignment
 * contract); GDN_ERR_HIP.
 */
int gdn_residual_rms_norm(const gdn_bf16 *x, int64_t x_stride, const gdn_bf16 *residual, int64_t residual_stride,
                          const gdn_bf16 *post_weight, const gdn_bf16 *gate, int64_t gate_stride,
                          const gdn_bf16 *weight, gdn_bf16 *new_residual, int64_t new_residual_stride,
                          gdn_bf16 *y, int64_t y_stride, int32_t rows, int32_t hidden,
                          float residual_scale, float eps, float weight_offset, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* GDN_H */
