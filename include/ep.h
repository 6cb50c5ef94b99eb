/*
 * ep.h — MoE dispatch / combine on one MI355X (gfx950): the C ABI.
 *
 * The operations follow the DeepEP README (community translation),
 * section "Interfaces and examples":
 *   - dispatch (README "Example use in model training or inference
 *     prefilling", dispatch_forward): route each token's hidden row to the
 *     experts of its top-k choice, into expert-contiguous receive rows whose
 *     per-expert counts are padded to expert_alignment for the grouped GEMM;
 *     x may be BF16 or FP8 with per-token scale factors;
 *   - combine (combine_forward): reduce each token's k expert outputs back
 *     into one BF16 row;
 *   - dispatch_backward is a combine (also returning the combined weight
 *     gradients); combine_backward is a dispatch that reuses the handle;
 *   - handle caching for decode (README "Example use in inference decoding"):
 *     a handle is reused across calls and skips the layout and the CPU sync.
 * This library computes one GPU's share of that work: every receive row
 * lives in this GPU's memory; there is no transport.
 *
 * Conventions for every entry point:
 *   - Pointers marked "device" are HIP device pointers (or host pointers the
 *     device can access); "host" pointers are ordinary host memory.
 *   - The caller owns every buffer: inputs, outputs and the workspace. The
 *     library allocates no device memory, keeps no pointer after returning
 *     and holds no global state except a thread-local error message, each
 *     device's CU count (queried once) and the fixed 1 MiB device array of
 *     ep_dispatch_forward_static_scratch (one per GPU, for the process's
 *     lifetime).
 *   - `stream` is a hipStream_t (NULL = the null stream). All work is
 *     enqueued on it and runs asynchronously; only ep_handle_read_counts and
 *     ep_handle_check wait for the stream.
 *   - Argument errors (NULL or misaligned pointer, sizes out of range,
 *     workspace too small) return EP_ERR_INVALID_ARG / EP_ERR_WORKSPACE /
 *     EP_ERR_UNSUPPORTED immediately and enqueue nothing;
 *     ep_last_error_message() says what was wrong. A failed launch returns
 *     EP_ERR_HIP.
 *   - Data errors found on the device (an expert id outside [0, E) that is
 *     not -1; a fixed-capacity overflow) do not fail the call: the pair is
 *     skipped (its slot is -1, it is copied nowhere and contributes nothing
 *     to combine) and a sticky bit is set in the handle's error word, read
 *     with ep_handle_check.
 *   - Alignment: x, recv, y, out and their FP8 counterparts must be 16-byte
 *     aligned; hidden must be a multiple of 8 (BF16) or 128 (FP8).
 *   - Numbers: bf16 = bfloat16 bit patterns (uint16); FP8 = OCP E4M3FN bytes;
 *     scales and weights are IEEE binary32.
 *   - Environment (read at each launch):
 *       EP_BUFFER_DEBUG=1  print, to stderr, the launch geometry each call
 *                          picks (kernel, grid, block, rows per zero-fill
 *                          piece, row pieces per token): the library's form
 *                          of the README's EP_BUFFER_DEBUG (section
 *                          "Environment variables": print buffer set-up and
 *                          SM-count choices).
 *       EP_LAUNCH_CUS=n    size grids as if the device had n compute units
 *                          (1 <= n <= 4096). Results never depend on launch
 *                          geometry; this knob exists so tests can show it.
 */
#ifndef EP_H
#define EP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    EP_OK = 0,
    EP_ERR_INVALID_ARG = 1,
    EP_ERR_UNSUPPORTED = 2,
    EP_ERR_HIP = 3,
    EP_ERR_WORKSPACE = 4
} ep_status;

/* Receive layout.
 * EP_MODE_COMPACT: expert-major rows, expert e owns
 *   [expert_off[e], expert_off[e] + pad[e]) with pad[e] = ceil(cnt[e]/A)*A;
 *   its first cnt[e] rows hold the pairs routed to e, the rest are padding.
 * EP_MODE_FIXED: expert e owns [e*C, e*C + C) (a [E, C, hidden] buffer, the
 *   decode layout); its first min(cnt[e], C) rows are written, the others
 *   are left untouched. */
typedef enum { EP_MODE_COMPACT = 0, EP_MODE_FIXED = 1 } ep_mode;

/* Payload type of a dispatch.
 * EP_BF16: x is bf16 [T, hidden]; recv is bf16 [rows, hidden].
 * EP_FP8_QUANTIZE: x is bf16 [T, hidden]; each 1x128 block of a token is
 *   quantised once (amax = max |x|, scale = amax / 448, code =
 *   E4M3FN(x / scale) rounded to nearest even and saturated to +-448; an
 *   all-zero block has scale 0 and zero codes); recv is E4M3FN
 *   [rows, hidden], recv_scales is binary32 [rows, hidden/128] row-major.
 * EP_FP8_PREQUANT: x is already E4M3FN [T, hidden] with x_scales binary32
 *   [T, hidden/128] (the README's (data, scale_factors) tuple); codes and
 *   scales are copied bitwise.
 * Entry points take the payload type as an int32_t holding one of these
 * values (any other value is EP_ERR_INVALID_ARG), so that a caller's
 * out-of-range value is an error rather than an invalid enum. */
typedef enum { EP_BF16 = 0, EP_FP8_QUANTIZE = 1, EP_FP8_PREQUANT = 2 } ep_dtype;

/* ep_config.flags */
#define EP_FLAG_NO_ZERO_PAD 1u /* COMPACT: leave padding rows unwritten */

/* Bits of the device error word (ep_handle_check). */
#define EP_ERRFLAG_BAD_ID 1u   /* an id outside [0, E) other than -1 */
#define EP_ERRFLAG_OVERFLOW 2u /* FIXED: more than C pairs for an expert */

/* Static sizes of one layout; the README's buffer arguments
 * (num_max_tokens_per_rank, hidden, num_topk, expert_alignment).
 * Limits: 1 <= num_experts <= 1024, 1 <= num_topk <= 32,
 * num_experts % num_dests == 0, max_tokens * num_topk < 2^31,
 * 8 <= hidden <= 2^24 and hidden % 8 == 0 (hidden % 128 == 0 for FP8),
 * expert_alignment >= 1 (must be 1 in FIXED mode), capacity >= 1 in FIXED
 * mode, idx_bits 64 (int64 topk_idx, torch.topk's type) or 32. */
typedef struct {
    int32_t max_tokens;       /* T_max: tokens a layout may hold */
    int32_t hidden;           /* H */
    int32_t num_experts;      /* E */
    int32_t num_topk;         /* k */
    int32_t num_dests;        /* D: experts grouped in D contiguous ranges */
    int32_t expert_alignment; /* A */
    int32_t capacity;         /* C: rows per expert in FIXED mode */
    int32_t mode;             /* ep_mode */
    int32_t idx_bits;         /* 64 or 32 */
    uint32_t flags;           /* EP_FLAG_* */
} ep_config;

/* Routing metadata shared by dispatch, combine and the duals (the README's
 * EPHandle). Plain data: copying it is fine. Every pointer points into the
 * caller's workspace (device memory) and is valid while the workspace
 * lives and no other ep_layout writes into it. Contents after the layout
 * has run on the stream:
 *   cnt[E]         pairs routed to each expert (before any capacity limit)
 *   pad[E]         rows of expert e in the receive buffer (COMPACT: padded
 *                  count; FIXED: min(cnt, C)) — the GEMM row counts
 *   expert_off[E+1] first row of each expert (COMPACT: exclusive scan of pad;
 *                  FIXED: e*C); expert_off[E] is the row total R
 *   dest_off[D+1]  first row of each destination: expert_off[d*E/D]
 *   dest_tokens[D] distinct tokens with a routed pair into destination d
 *   slot[T*k]      receive row of pair (t, j) or -1 when skipped; rows of
 *                  one expert are in ascending (t, j) order
 *   row_src[Rcap]  pair index t*k + j held by each row; -1 on padding rows
 *                  (COMPACT); FIXED rows past pad[e] are not written
 *   row_w[Rcap]    topk_w of the pair held by each row, 0 on padding rows;
 *                  written only when ep_layout got topk_w
 *   err_flags[1]   EP_ERRFLAG_* bits raised by this layout
 *   topk_idx       the caller's topk_idx the layout was built from (not a
 *                  copy: the README's decode example returns
 *                  cached_handle.topk_idx in place of a new recv_topk_idx,
 *                  "Example use in inference decoding"); valid while the
 *                  caller keeps that buffer, NULL for an empty batch */
typedef struct {
    ep_config cfg;
    int32_t num_tokens;
    int32_t num_blocks; /* internal: layout partition of the pairs */
    int32_t* cnt;
    int32_t* pad;
    int32_t* expert_off;
    int32_t* dest_off;
    int32_t* dest_tokens;
    int32_t* slot;
    int32_t* row_src;
    float* row_w;
    uint32_t* err_flags;
    void* internal; /* workspace scratch for the layout kernels */
    const void* topk_idx;
} ep_handle;

/* Bytes of workspace one layout needs (the README's get_buffer_size_hint).
 * Returns 0 when the config is invalid (see ep_last_error_message). */
size_t ep_workspace_bytes(const ep_config* cfg);

/* Rows a receive buffer must have to hold any layout of this config without
 * knowing the counts: max_tokens*k + E*(A-1) (COMPACT) or E*C (FIXED). The
 * README sizes its buffer from num_max_tokens_per_rank and hidden before any
 * routing is known (section "Interfaces and examples", "Buffer
 * initialization": get_buffer_size_hint); this is the same bound for the
 * receive rows, so a caller allocates them once and never waits for counts.
 * Returns -1 when the config is invalid. */
int64_t ep_recv_rows_bound(const ep_config* cfg);

/* Builds the layout of `num_tokens` tokens (README dispatch_forward: the
 * per-expert counts and padded offsets; the stable slot of every pair).
 *   cfg        host; copied into *out.
 *   num_tokens 0 <= num_tokens <= cfg->max_tokens.
 *   topk_idx   device [num_tokens, k], int64 or int32 per cfg->idx_bits;
 *              -1 masks a pair.
 *   topk_w     device [num_tokens, k] binary32, or NULL (row_w not written).
 *   workspace  device, >= ep_workspace_bytes(cfg) bytes, 256-byte aligned;
 *              must not be in use by another in-flight layout.
 *   out        host; receives the handle (valid once the stream reaches it).
 * Enqueues one kernel for small layouts (num_tokens * k <= 4096 and
 * E <= 512), three otherwise. Never synchronises. */
ep_status ep_layout(const ep_config* cfg, int32_t num_tokens, const void* topk_idx,
                    const float* topk_w, void* workspace, size_t workspace_bytes,
                    ep_handle* out, void* stream);

/* Layout and dispatch in one call: the README's dispatch_forward, which
 * builds the handle (per-expert counts, padded offsets, stable slots) and
 * moves the hidden states in the same call. Arguments are those of
 * ep_layout followed by those of ep_dispatch; every argument of both is
 * checked before anything is enqueued. The results (handle contents, recv,
 * recv_scales) are bit-identical to ep_layout followed by ep_dispatch.
 * Small batches (num_tokens * k <= 4096 and E <= 512, the decode sizes of
 * README "Example use in inference decoding", whose zero-fill of padding
 * rows, if any, fits the CUs beside one block per token) take a single
 * kernel launch:
 * every block derives its rows from all the batch's ids (the whole small
 * layout in LDS, or, in FIXED mode and with expert_alignment 1, only the
 * counts that place its own pairs), so no block waits on another. Larger batches enqueue the layout kernels and then the dispatch
 * kernel. Never synchronises. */
ep_status ep_dispatch_forward(const ep_config* cfg, int32_t num_tokens, const void* topk_idx,
                              const float* topk_w, void* workspace, size_t workspace_bytes,
                              int32_t dtype, const void* x, const float* x_scales, void* recv,
                              float* recv_scales, ep_handle* out, void* stream);

/* ep_dispatch_forward for callers that cannot allocate device memory: code
 * under HIP graph capture, tight serving loops, harnesses that forbid
 * hipMalloc. Same arguments, checks and results (bit-identical handle,
 * recv and recv_scales), except where the multi-block layout keeps its
 * per-block partials (counts [nblk, E], distinct tokens [nblk, D], error
 * bits [nblk]; nblk = ceil(num_tokens * k / 1024), each region rounded up
 * to 256 bytes): in a static device array the library holds (1 MiB per
 * GPU, kept until the process ends) instead of the workspace. The
 * workspace then needs only the handle's arrays; ep_workspace_bytes(cfg)
 * always suffices. Allocates nothing, on the host or the device. The first
 * call on each device looks up the array's address (hipGetSymbolAddress,
 * not a stream operation). A layout whose partials exceed 1 MiB returns
 * EP_ERR_WORKSPACE and enqueues nothing. Every call on one GPU shares the
 * array: calls whose work overlaps on one GPU (concurrent streams) race and
 * must be ordered by the caller; consecutive calls on one stream are safe,
 * since every entry a call reads is written earlier in that call. Small
 * batches (the single launch) use no partials. */
ep_status ep_dispatch_forward_static_scratch(const ep_config* cfg, int32_t num_tokens, const void* topk_idx,
                                             const float* topk_w, void* workspace, size_t workspace_bytes,
                                             int32_t dtype, const void* x, const float* x_scales, void* recv,
                                             float* recv_scales, ep_handle* out, void* stream);

/* Dispatch on an existing handle (README dispatch_forward, or dispatch with a
 * cached handle: no layout work, no synchronisation).
 *   x          device [T, hidden]: bf16 (EP_BF16, EP_FP8_QUANTIZE) or E4M3FN
 *              (EP_FP8_PREQUANT).
 *   x_scales   device [T, hidden/128] binary32 for EP_FP8_PREQUANT, else NULL.
 *   recv       device [ep_recv_rows_bound, hidden] bf16 or E4M3FN. Row
 *              slot[t, j] receives token t's row. COMPACT padding rows are
 *              zero-filled unless EP_FLAG_NO_ZERO_PAD; rows at or past
 *              expert_off[E] are not touched.
 *   recv_scales device [rows bound, hidden/128] binary32 for the FP8 types
 *              (padding rows get 0), else NULL. */
ep_status ep_dispatch(const ep_handle* h, int32_t dtype, const void* x, const float* x_scales,
                      void* recv, float* recv_scales, void* stream);

/* Combine (README combine_forward): for every token t and channel c,
 *   acc = +0; for j = 0..k-1 with slot[t, j] >= 0:
 *       acc = fmaf(topk_w[t, j], float(y[slot[t, j], c]), acc)
 *   (acc = acc + float(y[...]) when topk_w is NULL);
 *   out[t, c] = bf16(acc), round to nearest even.
 *   y          device bf16 [rows bound, hidden] (expert outputs, receive
 *              layout).
 *   topk_w     device [T, k] binary32 or NULL.
 *   out        device bf16 [T, hidden].
 *   row_vals   device [rows bound] binary32 or NULL; with out_vals given,
 *              out_vals[t, j] = row_vals[slot[t, j]] (0 for skipped pairs).
 *   out_vals   device [T, k] binary32 or NULL. */
ep_status ep_combine(const ep_handle* h, const void* y, const float* topk_w, void* out,
                     const float* row_vals, float* out_vals, void* stream);

/* README dispatch_backward: the backward of a dispatch is a combine without
 * weights; grad_row_w (per receive row, e.g. the gradient of row_w) is
 * gathered back to grad_topk_w [T, k] when both are given. */
ep_status ep_dispatch_backward(const ep_handle* h, const void* grad_recv, const float* grad_row_w,
                               void* grad_x, float* grad_topk_w, void* stream);

/* README combine_backward: the backward of a combine is a dispatch of the
 * output gradient on the same handle, which the README lets arrive in BF16
 * or as an FP8 (data, scale_factors) pair. dtype, grad_out, grad_out_scales,
 * grad_y and grad_y_scales are as ep_dispatch's dtype, x, x_scales, recv and
 * recv_scales (grad_out_scales: EP_FP8_PREQUANT only, device [T, hidden/128]
 * binary32; NULL otherwise). With topk_w, the copy for pair (t, j) is the
 * gradient of the weighted combine, bf16(topk_w[t, j] * float(grad_out[t, c]))
 * (one binary32 multiply, round to nearest even); with EP_FP8_QUANTIZE that
 * BF16 copy is then quantised per 1x128 block as ep_dispatch quantises x,
 * each pair with its own scales. EP_FP8_PREQUANT with topk_w returns
 * EP_ERR_UNSUPPORTED (weighting codes would need them re-quantised). */
ep_status ep_combine_backward(const ep_handle* h, int32_t dtype, const void* grad_out,
                              const float* grad_out_scales, const float* topk_w, void* grad_y,
                              float* grad_y_scales, void* stream);

/* Gradient of the weighted combine with respect to its weights (the part of
 * README combine_backward that a weighted combine adds; the gradient with
 * respect to the expert outputs is ep_combine_backward with topk_w):
 *   grad_topk_w[t, j] = sum_c float(grad_out[t, c]) * float(y[slot[t, j], c])
 * in binary32, 0 for skipped pairs.
 *   grad_out     device bf16 [T, hidden] (gradient of combine's out).
 *   y            device bf16 [rows bound, hidden]: the expert outputs the
 *                forward combine read.
 *   grad_topk_w  device binary32 [T, k].
 * The sum is taken in a fixed order (per lane over its channels, then a
 * butterfly over the 64 lanes of a wave, then over the waves in order), so
 * results are deterministic; each product passes through at most
 * 8 * ceil((hidden / 8) / 1024) + 6 + 15 binary32 additions, which bounds
 * the error against the exact sum by that count times 2^-24 times
 * sum_c |grad_out[t, c] * y[slot, c]|. */
ep_status ep_combine_weight_grad(const ep_handle* h, const void* grad_out, const void* y,
                                 float* grad_topk_w, void* stream);

/* FP8 grouped GEMM over the receive layout: the consumer the layout is built
 * for (README: per-expert received-token counts meant for the expert GEMM, rows padded to
 * expert_alignment; "New features": EPv2's new GEMM layout). For every row r
 * of expert e and output channel c < n:
 *   out[r, c] = bf16( sum_kb a_scales[r, kb] * b_scales[e, c/128, kb]
 *                            * sum_{k in block kb} a[r, k] * b[e, c, k] )
 * accumulated in binary32 (MFMA partial sums per 128-wide K block, each
 * promoted with one binary32 product of the two scales and one FMA), rounded
 * to nearest even.
 *   a          device E4M3FN [rows bound, hidden]: the FP8 dispatch's recv.
 *   a_scales   device binary32 [rows bound, hidden/128]: its recv_scales.
 *   b          device E4M3FN [E, n, hidden]: expert e's weights, one row of
 *              hidden codes per output channel.
 *   b_scales   device binary32 [E, n/128, hidden/128]: 128x128 block scales.
 *   out        device bf16 [rows bound, n]. COMPACT: every row below
 *              expert_off[E] is written; padding rows (past expert_off[e] +
 *              cnt[e]) are zero when the receive padding rows are zero (the
 *              default; unspecified under EP_FLAG_NO_ZERO_PAD). FIXED: expert
 *              e's rows [e*C, e*C + ceil(pad[e]/128)*128) are written; those
 *              at or past e*C + pad[e] are unspecified. Other rows are not
 *              touched.
 * a, b and out must be 16-byte aligned, the scale arrays 4-byte aligned
 * (EP_ERR_INVALID_ARG otherwise). Requires hidden % 128 == 0, n % 128 == 0,
 * and expert_alignment % 128 == 0 (COMPACT) or capacity % 128 == 0 (FIXED),
 * so that every 128-row tile belongs to one expert; otherwise
 * EP_ERR_UNSUPPORTED. */
ep_status ep_grouped_gemm_fp8(const ep_handle* h, const void* a, const float* a_scales, const void* b,
                              const float* b_scales, int32_t n, void* out, void* stream);

/* BF16 products grouped by expert over the receive layout, for any
 * expert_alignment or capacity: the experts' products of a training step, in
 * its three directions. Live rows are those that hold a pair: expert e's first
 * cnt[e] rows (FIXED: pad[e]). Only live rows are read as operands, so the
 * contents of padding rows, and of experts without a pair, never matter. n
 * (output channels) and k (input channels; not tied to cfg.hidden, so that an
 * expert's second layer is the same call) are multiples of 8, at most 2^20
 * (EP_ERR_UNSUPPORTED above). Products of bf16 values are summed in binary32
 * by the MFMA and rounded once, to nearest even. The order of a sum depends on
 * n, k, the config, num_tokens and the counts, never on the device, the launch
 * or other experts' rows: the same call gives the same bits again.
 *
 * Forward: for every live row r of expert e and c < n,
 *   out[r, c] = bf16( sum_j a[r, j] * b[e, c, j] ),  j < k.
 *   a    device bf16 [rows bound, k].
 *   b    device bf16 [E, n, k]: one row of k weights per output channel, as
 *        ep_grouped_gemm_fp8's.
 *   out  device bf16 [rows bound, n]. COMPACT padding rows are zero-filled
 *        unless EP_FLAG_NO_ZERO_PAD; no other row is touched. Must not overlap
 *        an operand (also below).
 * More than 2^31 - 2^24 pairs (P = num_tokens * num_topk) are EP_ERR_UNSUPPORTED
 * (also below), and so is a product of more tiles than one launch holds: with
 * tiles of R rows, P / R + min(P, E) row tiles times the column tiles may be at
 * most 2^23 - 1. Forward: for P <= 16 E tiles are 128 columns by R = 16 (32 for
 * P > 6 E), otherwise 256 columns by R = 256. */
ep_status ep_grouped_gemm_bf16(const ep_handle* h, const void* a, const void* b, int32_t n, int32_t k, void* out,
                               void* stream);

/* Gradient of ep_grouped_gemm_bf16 with respect to a: for every live row r of
 * expert e and j < k,
 *   grad_a[r, j] = bf16( sum_c grad_out[r, c] * b[e, c, j] ),  c < n.
 *   grad_out  device bf16 [rows bound, n].
 *   b         device bf16 [E, n, k], the forward's.
 *   grad_a    device bf16 [rows bound, k]; padding rows as the forward's.
 * Tiles: 256 columns (of k) by R = 256. */
ep_status ep_grouped_gemm_bf16_grad_input(const ep_handle* h, const void* grad_out, const void* b, int32_t n,
                                          int32_t k, void* grad_a, void* stream);

/* Gradient of ep_grouped_gemm_bf16 with respect to b, whole: for every expert
 * e, c < n and j < k,
 *   grad_b[e, c, j] = sum_r grad_out[r, c] * a[r, j] over e's live rows,
 * zero for an expert without a live row.
 *   grad_out  device bf16 [rows bound, n].
 *   a         device bf16 [rows bound, k], the forward's.
 *   grad_b    device [E, n, k]: binary32 when grad_b_f32 is 1, bf16 when 0.
 * Tiles: E * ceil(n / 256) * ceil(k / 128), at most 2^24 - 1. */
ep_status ep_grouped_gemm_bf16_grad_weight(const ep_handle* h, const void* grad_out, const void* a, int32_t n,
                                           int32_t k, int32_t grad_b_f32, void* grad_b, void* stream);

/* Products with 4-bit weights grouped by expert, for serving: as
 * ep_grouped_gemm_bf16, with the weights held as MXFP4 (OCP Microscaling
 * Formats: E2M1 codes with one E8M0 scale for each 32 of them along k),
 *   out[r, c] = bf16( sum_j a[r, j] * e2m1(code[e, c, j]) * 2^(scale[e, c, j / 32] - 127) ).
 *   a         device bf16 [rows bound, k]; k is a multiple of 32.
 *   b         device bytes [E, n, k / 2]: code j in byte j / 2, even j in the
 *             low nibble; a code is sign, two exponent bits, one mantissa bit
 *             (0, 0.5, 1, 1.5, 2, 3, 4, 6 and their negatives).
 *   b_scales  device bytes [E, n, k / 32], any alignment. 255 is NaN: its 32
 *             weights, and so the sums they enter, are NaN.
 *   out       as ep_grouped_gemm_bf16's, and likewise n.
 * A weight is a bf16 value (weights past bf16's largest finite value are
 * infinite, as in binary32), products are summed in binary32 by the MFMA and
 * rounded once. Tiles: 128 columns by R = 16 for P <= 6 E, 256 columns by 32 for
 * P <= 20 E, otherwise 256 columns by 64. */
ep_status ep_grouped_gemm_mxfp4(const ep_handle* h, const void* a, const void* b, const void* b_scales, int32_t n,
                                int32_t k, void* out, void* stream);

/* Quantises rows to MXFP4 (OCP Microscaling Formats), the operands of
 * ep_grouped_gemm_mxfp4 and ep_grouped_gemm_mxfp4_rows. For each 32 consecutive
 * values of a row, with m = max|x|,
 *   X = max(floor(log2 m) - 2, -127), scale = X + 127 (0 for 32 zeros),
 *   code = E2M1(x / 2^X), rounded to nearest even, at most 6 in magnitude, the
 *          sign kept;
 * a NaN or an infinity among them: scale 255 (NaN) and zero codes.
 *   h       NULL: all rows. Otherwise x has the receive layout, rows is
 *           ep_recv_rows_bound(&h->cfg), and only rows that hold a pair are read
 *           and written.
 *   k       a multiple of 32, at most 2^20 (EP_ERR_UNSUPPORTED above); rows * k
 *           at most 2^42.
 *   x       device [rows, k], bf16, or binary32 when x_f32 is 1.
 *   codes   device bytes [rows, k / 2]: value j in byte j / 2, even j in the low
 *           nibble.
 *   scales  device bytes [rows, k / 32], any alignment.
 *   values  device bf16 [rows, k]: what the codes stand for, exactly (NaN where the
 *           scale is), or NULL. The operand of the BF16 products in the backward
 *           pass of training with 4-bit operands. May be x's own buffer when x is bf16. */
ep_status ep_quantize_mxfp4(const ep_handle* h, int64_t rows, int32_t k, int32_t x_f32, const void* x, void* codes,
                            void* scales, void* values, void* stream);

/* ep_grouped_gemm_mxfp4 with the rows in MXFP4 as well, on the matrix unit's 4-bit
 * form:
 *   out[r, c] = bf16( sum_j av[r, j] * bv[e, c, j] ),
 * av and bv the values that codes and scales stand for.
 *   a         device bytes [rows bound, k / 2], codes as ep_quantize_mxfp4 writes
 *             them; k is a multiple of 32.
 *   a_scales  device bytes [rows bound, k / 32], any alignment. 255 is NaN, as in b_scales.
 *   b, b_scales, out  as ep_grouped_gemm_mxfp4's, and likewise n.
 * Products are exact, and summed in binary32 by the MFMA (a sum's terms more than
 * 23 binary places below its largest are cut off), rounded once. Tiles: 256 columns by
 * R = 256 (192 for k no multiple of 128) where k is at least 128, the scales are 4-byte
 * aligned and there are enough of them; otherwise 128 columns by R = 16 for P <= 6 E, by
 * R = 64 above. */
ep_status ep_grouped_gemm_mxfp4_rows(const ep_handle* h, const void* a, const void* a_scales, const void* b,
                                     const void* b_scales, int32_t n, int32_t k, void* out, void* stream);

/* RMS norm with the residual's addition: the norm before the router and the
 * dispatch, whose FP8 output is an EP_FP8_PREQUANT dispatch's input. For every
 * token t < num_tokens and channel c < hidden:
 *   s[c] = bf16(x[t, c] + residual[t, c]), written to total (without a
 *          residual s = x, and total must be NULL);
 *   rstd[t] = 1 / sqrt(mean_c s[c]^2 + eps), in binary32;
 *   u[c] = s[c] * weight[c], exact in binary32;
 * EP_BF16: y[t, c] = bf16(u[c] * rstd[t]);
 * EP_FP8_QUANTIZE, for each 128 channels: q = max|u| / 448,
 *   y[t, c] = E4M3FN(u[c] / q) rounded to nearest even and saturated to +-448,
 *   y_scales = q * rstd[t] (q = 0: zero codes, scale 0). rstd multiplies a
 *   whole row and so enters the scale alone.
 *   Infinities and NaN go by the same formulas, a NaN among the |u| being their
 *   maximum: its 128 channels have NaN codes and a NaN scale; beside an infinite
 *   u, which has a NaN code, the others have zero codes, and the scale is q * rstd
 *   likewise, infinite (NaN where rstd is 0).
 *   x, residual, total  device bf16 [num_tokens, hidden]; total may be x's or
 *                       residual's own buffer.
 *   weight    device bf16 [hidden].
 *   eps       positive.
 *   y         device bf16 or E4M3FN [num_tokens, hidden].
 *   y_scales  device binary32 [num_tokens, hidden / 128] for FP8, else NULL.
 *   rstd      device binary32 [num_tokens].
 * hidden is a multiple of 8 (FP8: of 128), at most 32768, num_tokens below 2^22
 * (EP_ERR_UNSUPPORTED above). y must not overlap an input. */
ep_status ep_rms_norm(int32_t num_tokens, int32_t hidden, int32_t dtype, const void* x, const void* residual,
                      const void* weight, float eps, void* total, void* y, float* y_scales, float* rstd,
                      void* stream);

/* Bytes of workspace ep_rms_norm_backward needs; 0 when the sizes are invalid
 * (see ep_last_error_message). */
size_t ep_rms_norm_workspace_bytes(int32_t num_tokens, int32_t hidden);

/* Backward of ep_rms_norm (of y before an FP8 output's rounding): with s and
 * rstd the forward's, g = grad_y[t] and m = mean_c(g[c] * weight[c] * s[c] * rstd[t]),
 *   grad_x[t, c] = bf16( rstd[t] * (g[c] * weight[c] - s[c] * rstd[t] * m) + grad_total[t, c] ),
 *   grad_weight[c] = sum_t g[c] * s[c] * rstd[t].
 * grad_x is the gradient of x and of residual alike.
 *   total       device bf16 [num_tokens, hidden]: the forward's total (x when
 *               it had no residual).
 *   rstd        device binary32 [num_tokens]: the forward's.
 *   grad_y      device bf16 [num_tokens, hidden].
 *   grad_total  device bf16 [num_tokens, hidden], the gradient that reaches
 *               total by other ways than y, or NULL.
 *   grad_x      device bf16 [num_tokens, hidden]; may be grad_total's own buffer.
 *   grad_weight device binary32 [hidden]; zeros for an empty batch.
 *   workspace   device, >= ep_rms_norm_workspace_bytes, 256-byte aligned; not
 *               to be shared by calls that may overlap.
 * Sums are taken in binary32 in an order that depends on the sizes alone. */
ep_status ep_rms_norm_backward(int32_t num_tokens, int32_t hidden, const void* total, const void* weight,
                               const float* rstd, const void* grad_y, const void* grad_total, void* grad_x,
                               float* grad_weight, void* workspace, size_t workspace_bytes, void* stream);

/* ---- The router: what stands between the norm and the layout. ---- */

/* Scores of a token's experts from its logits l. */
typedef enum { EP_SCORE_SOFTMAX = 0, EP_SCORE_SIGMOID = 1 } ep_score;

/* Sizes and rule of a router. Limits: 1 <= num_experts <= 1024,
 * 1 <= num_topk <= 32, num_groups divides num_experts and is at most 64,
 * 1 <= topk_groups <= num_groups, group_best 1 or 2 and at most the
 * num_experts / num_groups experts of a group, num_topk at most the
 * topk_groups * num_experts / num_groups experts that stay, scale finite. */
typedef struct {
    int32_t num_experts;  /* E */
    int32_t num_topk;     /* k */
    int32_t score;        /* ep_score */
    int32_t num_groups;   /* G: experts in G contiguous groups; 1 = no groups */
    int32_t topk_groups;  /* groups whose experts a token may choose */
    int32_t group_best;   /* a group goes by the sum of its 1 or 2 highest keys */
    int32_t renormalize;  /* 1: a token's weights are divided by their sum */
    int32_t idx_bits;     /* 64 or 32: type of topk_idx */
    int32_t logits_f32;   /* 1: logits (and their gradient) binary32, 0: bf16 */
    float scale;          /* factor of the weights */
} ep_router;

/* Chooses each token's experts: the topk_idx and topk_w that ep_layout and
 * ep_combine take. For every token, with l its logits and e < E,
 *   s[e] = exp(l[e] - max l) / sum_i exp(l[i] - max l)   (EP_SCORE_SOFTMAX)
 *        = 1 / (1 + exp(-l[e]))                           (EP_SCORE_SIGMOID);
 *   key[e] = s[e] + bias[e], in binary64; the logit itself when there is no bias
 *        and group_best is 1, where scores order as logits do;
 * the topk_groups groups with the largest sums of their group_best highest keys
 * stay (num_groups > 1), and of their experts the k with the highest keys are
 * chosen, highest first; among equals the lowest index goes first. Then
 *   topk_w[j] = scale * s[i_j]  or, with renormalize,
 *               scale * s[i_j] / (sum_m s[i_m] + 1e-20),
 * in binary32, where a score below 2^-126 may count as 0: the bias steers the choice alone.
 * An expert whose logit or bias is -infinity is never chosen. Where that
 * leaves fewer than k (a group none), the remaining topk_idx are -1 and their
 * weights 0: ep_layout skips such pairs. A key that is NaN counts as the lowest
 * finite number; NaN and +infinity reach the weights by the formulas.
 *   logits      device [num_tokens, E], binary32 or bf16.
 *   bias        device binary32 [E], or NULL.
 *   token_mask  device bytes [num_tokens], or NULL: a token whose byte is 0
 *               (padding of a batch) gets topk_idx -1 and weights 0, and its
 *               logits are not read.
 *   topk_idx    device [num_tokens, k], int64 or int32 per idx_bits.
 *   topk_w      device binary32 [num_tokens, k].
 * num_tokens is at most 2^25. One launch. */
ep_status ep_route(const ep_router* r, int32_t num_tokens, const void* logits, const float* bias,
                   const uint8_t* token_mask, void* topk_idx, float* topk_w, void* stream);

/* Bytes of workspace ep_balance_loss needs; 0 when the arguments are invalid
 * (see ep_last_error_message). */
size_t ep_balance_loss_workspace_bytes(const ep_router* r, int32_t num_tokens, int32_t num_seqs);

/* The balance loss of a batch, for every sequence of it, with the counts. A token
 * is routed when one of its topk_idx lies in [0, E); others (padding) enter
 * nothing. With p the shares of a token's scores (softmax: s; sigmoid:
 * s / sum_i s[i], also where the scores themselves underflow), for every sequence q and
 * expert e
 *   counts[q, e] = pairs of q's tokens with topk_idx = e,
 *   N_q          = routed tokens of q, Q = sequences with N_q > 0,
 *   coef[q]      = E / (k N_q^2 Q), 0 where N_q is 0;
 *   loss         = sum_q coef[q] * sum_e counts[q, e] * sum_t p[t, e]
 * over q's routed tokens t: 1 where scores and counts are even.
 *   topk_idx    device [num_tokens, k] per idx_bits; ids outside [0, E) are no pairs.
 *   seq_off     device int32 [num_seqs + 1], ascending: sequence q has tokens
 *               [seq_off[q], seq_off[q + 1]), as far as they lie in [0, num_tokens);
 *               tokens before the first and past the last enter nothing. NULL: one
 *               sequence of all tokens, num_seqs 1.
 *   loss        device binary32 [1].
 *   counts      device int32 [num_seqs, E].
 *   coef        device binary32 [num_seqs].
 *   workspace   device, >= ep_balance_loss_workspace_bytes, 256-byte aligned; not
 *               to be shared by calls that may overlap.
 * Sums over tokens are taken in an order that depends on the sizes, seq_off and which
 * tokens' sigmoids are all tiny. num_tokens is at most 2^25, num_seqs 2^17. Two launches. */
ep_status ep_balance_loss(const ep_router* r, int32_t num_tokens, const void* logits, const void* topk_idx,
                          const int32_t* seq_off, int32_t num_seqs, float* loss, int32_t* counts, float* coef,
                          void* workspace, size_t workspace_bytes, void* stream);

/* Gradient of ep_route's weights and of ep_balance_loss with respect to the
 * logits (the choice and the counts are constants). With n[e] how often e stands
 * in a token's topk_idx, g[e] the sum of its grad_topk_w there, and
 * D = sum_e n[e] s[e] + 1e-20,
 *   u[e] = scale * g[e]  or, with renormalize,
 *          scale * (g[e] - n[e] * (sum_i g[i] s[i]) / D) / D;
 *   b[e] = grad_loss * coef[q] * counts[q, e], q the token's sequence;
 * softmax: grad_logits = s[e] * (u[e] + b[e] - sum_i s[i] (u[i] + b[i]));
 * sigmoid: grad_logits = s[e] (1 - s[e]) * (u[e] + (b[e] - sum_i p[i] b[i]) / sum_i s[i]).
 * A token that is not routed gets zeros. Ids outside [0, E) add nothing.
 *   grad_topk_w  device binary32 [num_tokens, k], or NULL (the loss's gradient alone).
 *   counts, coef, grad_loss  ep_balance_loss's, and the loss's gradient (device
 *                binary32 [1]); all three or none of them (the weights' gradient alone).
 *   seq_off, num_seqs  as ep_balance_loss's (NULL and 1 without counts).
 *   grad_logits  device [num_tokens, E], binary32 or bf16 as logits; may be the
 *                logits' own buffer.
 * num_tokens is at most 2^25. One launch. */
ep_status ep_route_backward(const ep_router* r, int32_t num_tokens, const void* logits, const void* topk_idx,
                            const float* grad_topk_w, const int32_t* counts, const float* coef,
                            const float* grad_loss, const int32_t* seq_off, int32_t num_seqs, void* grad_logits,
                            void* stream);

/* Copies cnt and pad (host arrays of E, either may be NULL) and the row
 * total R (host, may be NULL) to the host. Synchronises the stream: this is
 * the README's CPU synchronisation of a non-cached dispatch. */
ep_status ep_handle_read_counts(const ep_handle* h, int32_t* cnt, int32_t* pad, int64_t* rows,
                                void* stream);

/* Reads the handle's error word (EP_ERRFLAG_* bits) to host *flags.
 * Synchronises the stream. No passage of the pages defines this call: their
 * API has no device-side data errors; it reports the two this library
 * defines (an out-of-range expert id, a fixed-capacity overflow). */
ep_status ep_handle_check(const ep_handle* h, uint32_t* flags, void* stream);

/* Static text for a status code (an ep_status value; any other value
 * gives "EP_ERR_UNKNOWN"). No passage of the pages defines this call: it
 * belongs to this C ABI's error convention. */
const char* ep_status_string(int32_t s);

/* Message of the last failed call on this thread ("" if none). No passage
 * of the pages defines this call: it belongs to this C ABI's error
 * convention (the pages' Python API raises exceptions instead). */
const char* ep_last_error_message(void);

#ifdef __cplusplus
}
#endif

#endif /* EP_H */
