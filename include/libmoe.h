/* libmoe — the routed mixture-of-experts expert layer of a Kolibri-style model on one
 * NVIDIA GB300 (sm_103a), as a C ABI over hand-written CUDA kernels.
 *
 * The layer (page "We Ported Aleph Alpha's Kolibri to a MacBook. Our Own Gate Said No.",
 * section "The gate", and section 1 for the bias and the forced ids; section 3 for the
 * SwitchGLU expert layer): for every token a float32 router scores the routed experts
 * (384 in Kolibri-1), the top k = 6 are selected and weighted, one shared expert runs for
 * every token, and the weighted expert outputs are summed.  The expert choices can instead
 * be forced from a supplied id tensor (page "We Stopped the Kolibri Benchmark Before Scoring
 * One Answer", section "The gate, forced").  Numerical recipe of this library (the pages
 * leave it open):
 *   logits[t,e] = sum_k x[t,k] Wr[e,k] + b[e]                       (fp32)
 *   ids[t]      = the k largest softmax probabilities, lowest index on ties, in descending
 *                 order;  w[t,i] = p[ids_i] / sum_j p[ids_j]
 *   expert e    = W8A8 SwiGLU: x is quantised per token to E4M3 (scale max|x|/448),
 *                 g = (qx . Wg[e,n]) sx sg[e,n], u likewise, h = silu(g) u, h quantised per
 *                 row the same way, y_e[m] = (qh . Wd[e,m]) sh sd[e,m], stored as a bf16
 *                 activation (round to nearest even) before the combine
 *   y[t]        = y_shared[t] + sum_{i=0..k-1} w[t,i] y_{ids_i}[t]  (slot order, fp32)
 * With fp32 weights (MOE_F32) the experts run in fp32 without quantisation.
 *
 * Conventions for every call:
 *  - Every pointer argument is device memory owned by the caller, unless stated.  The
 *    library allocates nothing and keeps no state between calls.
 *  - Calls are asynchronous on `stream`; host-side validation errors return at once and
 *    launch nothing.  Device-side errors (bad forced ids, a wait that timed out) are
 *    recorded in the workspace and reported by moe_get_status().  Nothing traps.
 *  - T == 0 is a no-op returning MOE_OK.
 *  - Alignment: x, y, weights, scales and the workspace 16-byte aligned.
 *  - Shapes: top_k == 6 (else MOE_ERR_UNSUPPORTED), n_experts <= 1024, T <= 2^20;
 *    E4M3 or E2M1 weights in the tiled layout: d_model % 128 == 0 and ffn % 128 == 0 (E2M1
 *    weights only in the tiled layout); E4M3 weights
 *    in the row layout: d_model % 256 == 0, d_model <= 2048, ffn % 64 == 0, ffn <= 640;
 *    fp32 weights: d_model % 128 == 0 and ffn % 32 == 0.
 *  - Layout: row-major, last index contiguous.
 */
#ifndef LIBMOE_H
#define LIBMOE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* A cudaStream_t (0 = the legacy default stream) and a cudaEvent_t. */
typedef struct CUstream_st* moe_stream_t;
typedef struct CUevent_st* moe_event_t;

typedef enum {
  MOE_OK = 0,
  MOE_ERR_INVALID_ARG = -1,   /* null/misaligned pointer, bad dtype or shape */
  MOE_ERR_UNSUPPORTED = -2,   /* valid request this library does not implement (e.g. k != 6) */
  MOE_ERR_WORKSPACE = -3,     /* ws_bytes < moe_workspace_bytes() */
  MOE_ERR_BAD_FORCED_ID = -4, /* a forced id was out of range or repeated within a token */
  MOE_ERR_TIMEOUT = -5,       /* a device-side wait gave up */
  MOE_ERR_CUDA = -6,          /* a CUDA runtime call failed */
  MOE_ERR_INDEX = -7,         /* MOE_DEBUG builds only: a kernel's index check failed (an internal
                                 error of the library; the access was kept inside its buffer) */
  MOE_ERR_BAD_PAGE = -8,      /* a token's sequence, position or page was outside the page table or
                                 the cache */
  MOE_ERR_NO_PAGES = -9       /* a sequence's new tokens did not fit: the pool had too few free pages, or
                                 its row of the page table or the token list no room */
} moe_status;

/* MOE_E2M1: 4-bit weights (OCP E2M1 codes: sign bit 3, magnitudes 0, 0.5, 1, 1.5, 2, 3, 4,
 * 6), two per byte, element 2i in the low nibble of byte i, with one fp32 scale per output row
 * like MOE_E4M3 (this library's reading of the 4-bit "K4" builds of page "We Stopped the
 * Kolibri Benchmark Before Scoring One Answer", section "What this means if you want Kolibri
 * on a Mac"; the pages give no format).  Weight matrices keep their row count and halve their
 * bytes per row; activations enter the contractions as E4M3 as for MOE_E4M3 (W4A8). */
/* MOE_INT4: rows of a key-value cache in 4 bits (moe_kv_cache below), not a type of weights. */
typedef enum { MOE_F32 = 0, MOE_BF16 = 1, MOE_E4M3 = 2, MOE_E2M1 = 3, MOE_INT4 = 4 } moe_dtype;

/* Byte order of the E4M3 expert weight tensors (w_gate_up, w_down, sh_gate_up, sh_down).
 *   MOE_LAYOUT_ROWS   the shapes below, row-major (a checkpoint's order).
 *   MOE_LAYOUT_TILED  the same bytes regrouped by moe_pack_weights into 16 KB tiles of 128
 *                     rows x 128 bytes of k, each tile stored in the 128-byte-swizzled order
 *                     the tensor cores read, and ordered so that the tiles one GEMM step
 *                     needs are contiguous:
 *                     gate/up tile (e, n, j, half) at byte ((((e * F/128) + n) * d/128 + j) * 2 + half) * 16384
 *                       = rows half*F + 128 n .. +127 of expert e's [2F, d] matrix, k = 128 j .. 128 j + 127
 *                     down tile (e, m, j) at byte (((e * d/128) + m) * F/128 + j) * 16384
 *                       = rows 128 m .. +127 of expert e's [d, F] matrix, k = 128 j .. +127
 *                     inside a tile, byte (r, c) sits at r*128 + 16*((c/16) ^ (r%8)) + c%16.
 *                     The shared expert's tensors are tiled the same way (as expert 0).
 *                     Requires E4M3 or E2M1, d_model % 128 == 0 and ffn % 128 == 0.
 *                     E2M1 weights use the same tile order with 8 KB tiles (tile index
 *                     x 8192 in place of x 16384): 128 rows of 64 bytes (128 codes of k)
 *                     each, rows in order and unswizzled (the tensor cores' swizzle is
 *                     applied when a tile is copied to shared memory).
 * The tensor-core expert kernels read the tiled layout (each pipeline stage is then one
 * contiguous copy of 32-80 KB); the weight-streaming kernels read the row layout.  E2M1
 * layers run only on the tensor-core kernels, so moe_forward takes them tiled. */
typedef enum { MOE_LAYOUT_ROWS = 0, MOE_LAYOUT_TILED = 1 } moe_layout;

/* How router_bias enters the routing (page "We Ported Aleph Alpha's Kolibri to a MacBook.
 * Our Own Gate Said No.", section 1: "router score plus a per-expert selection bias").
 *   MOE_BIAS_SCORE   logits = x Wr^T + b: the bias shifts both the selection and the weights.
 *   MOE_BIAS_SELECT  logits = x Wr^T: the experts are ranked on logits + b, and the weights are
 *                    the softmax of the unbiased logits renormalised over the selected six. */
typedef enum { MOE_BIAS_SCORE = 0, MOE_BIAS_SELECT = 1 } moe_bias_mode;

/* One layer: borrowed device pointers.  Shapes with d = d_model, F = ffn, E = n_experts.
 *   w_router     [E, d]  fp32            router_bias [E] fp32 or NULL
 *   w_gate_up    [E, 2, F, d]            gate rows (index 0) then up rows (index 1)
 *                (E2M1: the last dimension of each weight tensor holds two codes per byte)
 *   s_gate_up    [E, 2, F] fp32          per-output-row scales (E4M3 only, else NULL)
 *   w_down       [E, d, F]               s_down [E, d] fp32 (E4M3 only)
 *   sh_gate_up   [2, F, d]               sh_s_gate_up [2, F] (E4M3 only)
 *   sh_down      [d, F]                  sh_s_down [d] (E4M3 only)
 * Weights are E4M3 codes (w_dtype = MOE_E4M3, one byte each), E2M1 codes (MOE_E2M1, two
 * per byte) or fp32 (MOE_F32). */
typedef struct {
  int d_model, ffn, n_experts, top_k;
  moe_dtype w_dtype;
  const float* w_router;
  const float* router_bias;
  const void* w_gate_up;
  const float* s_gate_up;
  const void* w_down;
  const float* s_down;
  const void* sh_gate_up;
  const float* sh_s_gate_up;
  const void* sh_down;
  const float* sh_s_down;
  moe_layout w_layout; /* order of the four E4M3 weight tensors (MOE_LAYOUT_ROWS for fp32) */
  moe_bias_mode bias_mode; /* MOE_BIAS_SCORE (a zero-initialised struct) or MOE_BIAS_SELECT */
} moe_layer;

/* Flags for moe_forward / moe_forward_stack: which expert kernels run.  0 = automatic: the
 * tcgen05 grouped GEMMs for tiled E4M3 weights, the weight-streaming kernels otherwise. */
#define MOE_PATH_AUTO 0u
#define MOE_PATH_STREAM 1u /* weight-streaming kernels (row layout; any T) */
#define MOE_PATH_TC 2u     /* tcgen05 grouped GEMMs (tiled layout; any T) */

/* Writes the tiled layout (MOE_LAYOUT_TILED above) of src's four E4M3 (or E2M1) weight
 * tensors, which must be in the row layout, into gate_up [E*2*F*d], down [E*d*F], sh_gate_up
 * [2*F*d] and sh_down [d*F] bytes (half as many for E2M1) of caller-owned device memory
 * (16-byte aligned, not overlapping the sources).  The scales and the router are unchanged; a moe_layer with the four pointers
 * replaced and w_layout = MOE_LAYOUT_TILED then describes the same layer.  Asynchronous on
 * `stream`.  MOE_ERR_UNSUPPORTED unless E4M3 or E2M1 with d_model % 128 == 0 and
 * ffn % 128 == 0. */
moe_status moe_pack_weights(const moe_layer* src, void* gate_up, void* down, void* sh_gate_up, void* sh_down,
                            moe_stream_t stream);

/* Bytes of workspace the calls below need for T tokens of this layer (host only). */
size_t moe_workspace_bytes(const moe_layer* layer, int T);

/* Clears the workspace's status record.  Call once after allocating a workspace (or use
 * zero-filled memory).  Asynchronous on `stream`. */
moe_status moe_workspace_init(void* ws, size_t ws_bytes, moe_stream_t stream);

/* Router and selection (free routing) for T tokens: a float32 router scores every routed
 * expert and the top k = 6 are kept and weighted (page "We Ported Aleph Alpha's Kolibri to a
 * MacBook. Our Own Gate Said No.", section "The gate": 384 experts, top 6, a float32 router; the
 * per-expert bias: section 1).
 *   x           [T, d]  bf16 or fp32 (x_dtype)
 *   k           must equal layer->top_k (6)
 *   ids_out     [T, k] int32: selected experts, descending probability, lowest index on ties
 *   w_out       [T, k] fp32: renormalised softmax weights of the selected experts
 *   logits_out  [T, E] fp32 router logits (bias included under MOE_BIAS_SCORE, not under
 *               MOE_BIAS_SELECT), or NULL */
moe_status moe_route(const void* x, moe_dtype x_dtype, int T, const moe_layer* layer, int k,
                     int32_t* ids_out, float* w_out, float* logits_out, void* ws, size_t ws_bytes,
                     moe_stream_t stream);

/* Grouping of the T*k routed (token, slot) rows by expert, shared expert last: the sorted
 * grouping that turns the experts into one grouped GEMM (page "We Ported Aleph Alpha's Kolibri
 * to a MacBook. Our Own Gate Said No.", section 3, update of 5 October: the sorted path and its
 * row-count edge cases).
 *   counts  [E + 1]   rows per expert; counts[E] = T (the shared expert's rows)
 *   offsets [E + 2]   exclusive prefix sum of counts; offsets[E] = T*k, offsets[E+1] = T*k + T
 *   perm    [T*k + T] token of each row; tokens ascend within each expert (stable)
 *   pos     [T, k]    row holding (token t, slot i)
 * ids [T, k] must be valid (distinct within a token, in [0, E)). */
moe_status moe_dispatch(const int32_t* ids, int T, int n_experts, int k, int32_t* counts, int32_t* offsets,
                        int32_t* perm, int32_t* pos, void* ws, size_t ws_bytes, moe_stream_t stream);

/* The whole layer for T tokens.
 *   x            [T, d] bf16 or fp32 (x_dtype)
 *   forced_ids   [T, k] int32 or NULL: use these experts in this order instead of selecting.
 *                Ids out of range or repeated within a token contribute nothing and set
 *                MOE_ERR_BAD_FORCED_ID in the status record.
 *   forced_w     [T, k] fp32 or NULL (only with forced_ids): use these weights as given;
 *                without it the weights are the renormalised softmax over the forced ids.
 *   ids_out, w_out  [T, k] or NULL: the ids and weights used
 *   y            [T, d] bf16 or fp32 (y_dtype)
 *   flags        MOE_PATH_* */
moe_status moe_forward(const void* x, moe_dtype x_dtype, int T, const moe_layer* layer,
                       const int32_t* forced_ids, const float* forced_w, int32_t* ids_out, float* w_out,
                       void* y, moe_dtype y_dtype, unsigned flags, void* ws, size_t ws_bytes,
                       moe_stream_t stream);

/* L layers on a bf16 residual stream, free routing: for l = 0..L-1,
 * r <- bf16_round_nearest_even(r + layer_l(r)).  Kolibri-1 stacks 50 such MoE layers (page "We
 * Ported Aleph Alpha's Kolibri to a MacBook. Our Own Gate Said No.", section "The gate"); the
 * bf16 residual with one rounding per layer after an fp32 add is this library's reading of the
 * pages' bf16 activations.
 *   layers    host array of L layer descriptors (read during the call only)
 *   residual  [T, d] bf16, updated in place
 *   ids_out   [L, T, k] int32 or NULL: the experts each layer selected
 * ws must hold moe_workspace_bytes() of the largest layer; layers share it in turn. */
moe_status moe_forward_stack(const moe_layer* layers, int L, void* residual, int T, int32_t* ids_out,
                             unsigned flags, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Stage boundaries recorded by the *_traced calls: before the router, then after the router,
 * selection, dispatch, activation quantisation, gate/up, h quantisation, down, combine. */
#define MOE_TRACE_POINTS 9

/* moe_forward, recording `events` (MOE_TRACE_POINTS caller-created CUDA events, or NULL) on
 * `stream` at the stage boundaries, so the caller can time each kernel stage. */
moe_status moe_forward_traced(const void* x, moe_dtype x_dtype, int T, const moe_layer* layer,
                              const int32_t* forced_ids, const float* forced_w, int32_t* ids_out, float* w_out,
                              void* y, moe_dtype y_dtype, unsigned flags, void* ws, size_t ws_bytes,
                              moe_stream_t stream, moe_event_t* events);

/* moe_forward_stack with events [L][MOE_TRACE_POINTS] (or NULL) recorded per layer. */
moe_status moe_forward_stack_traced(const moe_layer* layers, int L, void* residual, int T, int32_t* ids_out,
                                    unsigned flags, void* ws, size_t ws_bytes, moe_stream_t stream,
                                    moe_event_t* events);

/* Synchronises `stream`, returns a device-side error recorded in the workspace since the last
 * call (MOE_OK if none; of several MOE_ERR_INDEX before MOE_ERR_TIMEOUT, and that before refused
 * ids and pages) and clears the record. */
moe_status moe_get_status(void* ws, moe_stream_t stream);

/* moe_route without a workspace, for callers that cannot allocate device memory (a host
 * runtime that owns all device memory through its own pool and forbids side allocations, or a
 * serving loop where an allocation, which may synchronise the device, is not allowed).  The
 * pages have no counterpart: this is a deployment variant of the router and selection.
 *   Same arguments and results as moe_route, minus logits_out and the workspace.
 *   Scratch: a fixed 4 MiB + 768 B array inside the library, resident on every GPU that loads
 *   it until the process exits; T * n_experts must be <= 1,048,576, else MOE_ERR_WORKSPACE.
 *   The first call on a device looks up the array's device address (once per device, with
 *   that device current); make that first call before any stream capture.  A device reset or
 *   another CUDA context on the device moves the array: the first call made under the new
 *   context looks the address up again.
 *   All calls on a device share the array: calls that overlap on the GPU race; serialise them.
 *   No device-side error can arise in this call (no forced ids, no device-side waits), so it
 *   has no status record to read: host-side errors are its return value, as for moe_route.
 *   Allocates nothing (no cudaMalloc, no cudaFree). */
moe_status moe_route_noalloc(const void* x, moe_dtype x_dtype, int T, const moe_layer* layer, int k,
                             int32_t* ids_out, float* w_out, moe_stream_t stream);

/* ---- the decode step between two expert layers: paged cache, attention, norms -----------------
 *
 * A Kolibri-style decoder layer is attention and then the expert layer on one residual stream,
 * 40 layers with a 513-token sliding window and every fifth with full context (page "We Ported
 * Aleph Alpha's Kolibri to a MacBook. Our Own Gate Said No.", section "The gate").  The calls
 * below are what a decode step needs around moe_forward and the two projections.  They follow
 * the conventions at the top; device-side errors go to the status record of the workspace they
 * are given. */

/* A paged key-value cache: n_pages pages of page_size tokens, each token with n_kv_heads keys and
 * values of head_dim elements.
 *   k, v          [n_pages, n_kv_heads, page_size, head_dim]  bf16, or E4M3 codes; 4-bit codes
 *                 (MOE_INT4): [.., head_dim / 2] bytes
 *   k_exp, v_exp  [n_pages, n_kv_heads, page_size] uint8 (E4M3 and INT4, else NULL): a row's values
 *                 are its codes (INT4: times their scales) times 2^(exp - 127)
 *   k_scale, v_scale  [n_pages, n_kv_heads, page_size, 4 ceil(head_dim / 64)] uint8 (INT4 only, else not
 *                 read): byte b of each 16 elements is their scale (1 + (b % 8) / 8) 2^(b / 8 - 12), from
 *                 2^-12 to 15; the bytes past head_dim / 16 are zeros
 * INT4: element i is n_i scale(i / 16) 2^(exp - 127) with n_i a whole number from -7 to 7.  Elements 4u ..
 * 4u + 3 are bytes 2u and 2u + 1 of their row: the codes n_i + 8, the first in the lowest four bits of
 * 16, and those 16 bits turned left by 3 (the order that attention takes apart in the fewest steps).  A row is
 * 0.57 bytes an element, against 1.01 in E4M3 and 2 in bf16.
 * Position p of sequence s lives in row p % page_size of page page_table[s, p / page_size], of a
 * page_table [n_seqs, max_pages] int32 on the device that the caller fills as it hands out pages
 * (entries beyond a sequence's length are not read).
 * dtype MOE_BF16, MOE_E4M3 or MOE_INT4; page_size a multiple of 16, up to 4096; head_dim a multiple of 16
 * (INT4: of 32), up to 256; n_kv_heads up to 1024; n_pages * n_kv_heads * page_size below 2^31; all pointers
 * 16-byte aligned.  (k_scale and v_scale are looked at for MOE_INT4 alone.) */
typedef struct {
  int n_pages, page_size, n_kv_heads, head_dim;
  moe_dtype dtype;
  void* k;
  void* v;
  uint8_t* k_exp;
  uint8_t* v_exp;
  uint8_t* k_scale;
  uint8_t* v_scale;
} moe_kv_cache;

/* Writes T tokens' keys and values into the cache.
 *   k, v      T rows of [n_kv_heads, head_dim], bf16 or fp32 (kv_dtype), the rows k_stride and
 *             v_stride elements apart (a fused projection's output is taken as it lies); both a
 *             multiple of 16 bytes
 *   seq, pos  [T] int32: each token's sequence and position; seq NULL: token t is sequence t's.
 *             A negative position skips the token.  Two tokens of one call must not be given one
 *             place (its row is then undefined).
 * bf16 cache: values rounded to nearest even.  E4M3 cache: a row's exponent is the smallest power
 * of two (2^-127 at least) that brings its largest magnitude to 448 at most, and its codes are the
 * scaled values rounded to nearest even: scaling by a power of two is exact, so each value is
 * rounded once and moe_kv_read returns it without another rounding.  A NaN stays one; an infinity is
 * stored as 448 times 2^120, beyond fp32, reads back as an infinity, and sets its row's exponent.
 * INT4 cache: a row's exponent is the smallest power of two, from 2^-111 to 2^119, that brings its largest
 * magnitude to 105 at most; then the scale of 16 elements is the smallest that brings theirs to 7 at most; then
 * each element is rounded once, to the nearest of -7 .. 7, ties to the even one.  So it is off by at most half its
 * group's scale; magnitudes above 105 times 2^119 become that.  A row with an infinity or a NaN in it reads back
 * as NaN (exponent byte 255).
 * A sequence outside [0, n_seqs), a position past the page table or a page outside [0, n_pages)
 * writes nothing and records MOE_ERR_BAD_PAGE in ws (any workspace of this library). */
moe_status moe_kv_write(const moe_kv_cache* cache, const void* k, const void* v, moe_dtype kv_dtype, int64_t k_stride,
                        int64_t v_stride, int T, const int32_t* seq, const int32_t* pos, const int32_t* page_table,
                        int n_seqs, int max_pages, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Reads T tokens' keys and values back: k_out, v_out [T, n_kv_heads, head_dim] bf16 or fp32
 * (out_dtype), token t from sequence seq[t] (NULL: t) and position pos[t].  A skipped or refused
 * token (as for moe_kv_write) reads as zeros. */
moe_status moe_kv_read(const moe_kv_cache* cache, int T, const int32_t* seq, const int32_t* pos,
                       const int32_t* page_table, int n_seqs, int max_pages, void* k_out, void* v_out,
                       moe_dtype out_dtype, void* ws, size_t ws_bytes, moe_stream_t stream);

/* Bytes of workspace moe_attn_decode needs for up to B sequences of n_heads query heads on this
 * cache's shape (host only; 0 for a shape it refuses). */
size_t moe_attn_workspace_bytes(const moe_kv_cache* cache, int n_heads, int B);

/* Clears an attention workspace's status record and join counters.  Call once after allocating
 * it, and again after MOE_ERR_TIMEOUT.  An attention workspace serves moe_attn_decode calls of any
 * size that fits, one at a time, and no moe_forward (which would overwrite the counters).
 * Asynchronous on `stream`. */
moe_status moe_attn_workspace_init(void* ws, size_t ws_bytes, moe_stream_t stream);

/* Attention of one new token a sequence over the paged cache.  Query head h reads kv head
 * h / (n_heads / n_kv_heads); for sequence b with n = lens[b] cached tokens (the new one among
 * them: moe_kv_write first) and j from max(0, n - window) (window 0: from 0) to n - 1,
 *   out[b,h] = sum_j p_j v_j / sum_j p_j,  p_j = exp(scale q[b,h].k_j - max),
 *   lse[b,h] = log sum_j exp(scale q[b,h].k_j)
 *   q           B rows of [n_heads, head_dim] bf16, q_stride elements apart (a multiple of 8)
 *   lens        [B] int32 on the device; sequence b is row b of page_table [B, max_pages]
 *   out         [B, n_heads, head_dim] bf16, not overlapping q
 *   lse         [B, n_heads] fp32 or NULL: joins this result with another part of the context
 * n <= 0 gives zeros and an lse of -infinity.  n beyond the page table is cut to it, and a page
 * outside [0, n_pages) is left out as if masked; both record MOE_ERR_BAD_PAGE.  What lies in the
 * cache outside the window (NaN and infinity included) has no effect.  Scores, sums and the
 * accumulators are fp32; the results do not depend on the order in which CTAs finish.
 * Weights p_j are rounded before they multiply the values, and unrounded in the sum: to bf16 (off by
 * 2^-8 of themselves at most) over a bf16 cache; as closely over an E4M3 cache, where those below 2^-75
 * of the largest among 32 tokens lose bits.  Over an E4M3 cache query elements below 2^-14 of their
 * head's largest are held to 2^-22 of that one.  So before its own rounding to bf16 an output is off by
 * up to 2^-8 of sum_j p_j |v_j| / sum_j p_j.  An INT4 cache's values are exact in bf16, and attention over it is
 * that over a bf16 cache of the same values.  A weight below 2^-126 of the row's largest is 0.
 * n_heads a multiple of n_kv_heads, up to 1024; B up to 65536; max_pages * page_size up to 2^28, and
 * (max_pages * page_size / 32 + 1) * B * n_kv_heads * ceil(n_heads / n_kv_heads / 4) below 2^31. */
moe_status moe_attn_decode(const moe_kv_cache* cache, const void* q, int64_t q_stride, int n_heads, int B,
                           const int32_t* lens, const int32_t* page_table, int max_pages, float scale, int window,
                           void* out, float* lse, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---- the pages and places of new tokens ----------------------------------------------------------
 *
 * A serving step knows how many tokens each sequence has in the cache and how many it gets.  The calls
 * below keep the page table, the pool of free pages and the lengths on the device, so that a step that
 * a CUDA graph replays hands out pages by itself.
 *   lens        [B] int32: tokens that each sequence has in the cache (a negative one counts as 0)
 *   page_table  [B, max_pages] int32 as above; a sequence holds the first ceil(len / page_size) entries, and no
 *               page belongs to two sequences
 *   free_pages  [n_pages] int32: a stack, whose first n_free[0] entries are the free pages
 * Both calls are given the workspace of moe_pages_workspace_bytes and report to its status record. */
size_t moe_pages_workspace_bytes(int B);

/* Room for new tokens.
 *   new_tokens  [B] int32: tokens to come for each sequence (negative: 0); NULL: one each
 *   lens_out    [B], n_free_out [1]: the lengths and the count of free pages afterwards (may be lens and
 *               n_free themselves)
 *   starts      [B + 1] int32: where each sequence's tokens begin on the list of all new tokens (in the order of
 *               sequences), cut to max_tokens
 *   seq, pos, slot  [max_tokens] int32, 16-byte aligned: each new token's sequence and position, and its place in
 *               the cache, page * page_size + row; -1 in all three behind the last token
 * A sequence that needs pages takes them from the top of the stack, sequences in order, and its entries of the
 * page table are written.  A sequence gets nothing if its tokens would go past its row of the page table or past
 * max_tokens, or if it needs pages and those of the sequences before it (served or not for want of pages) leave too
 * few (so one that is refused for want of pages holds up those behind it that need some: places are handed out in order):
 * its tokens keep their place on the list with pos and slot -1 (moe_kv_write and moe_rope_kv_write skip those), its
 * length stays, and MOE_ERR_NO_PAGES is recorded.  A page outside [0, n_pages) in the table or in the pool gives
 * slots of -1, and an n_free outside [0, n_pages] counts as the nearest; both record MOE_ERR_BAD_PAGE.
 * B up to 65536, max_tokens up to 2^20, page_size 1 to 4096, max_pages * page_size up to 2^28, n_pages *
 * page_size below 2^31; lens_out, n_free_out, starts, seq, pos, slot apart from each other and from every input but
 * as above. */
moe_status moe_page_plan(const int32_t* lens, const int32_t* new_tokens, int B, int32_t* page_table, int max_pages,
                         const int32_t* free_pages, const int32_t* n_free, int n_pages, int page_size, int max_tokens,
                         int32_t* lens_out, int32_t* n_free_out, int32_t* starts, int32_t* seq, int32_t* pos,
                         int32_t* slot, void* ws, size_t ws_bytes, moe_stream_t stream);

/* The pages of ended sequences back to the pool: each sequence with ended[b] != 0 ([B] bytes) puts its pages on
 * the stack, sequences in order, and has length 0 afterwards; the page table stays as it is.  Lengths past the page table
 * are cut to it, pages that the stack of n_pages entries has no room for are dropped, and an entry of the table outside
 * [0, n_pages) goes on the stack as it is (a plan that comes to it gives no place there); each of these records
 * MOE_ERR_BAD_PAGE.  lens_out and n_free_out as above. */
moe_status moe_page_release(const int32_t* lens, const uint8_t* ended, int B, const int32_t* page_table, int max_pages,
                            int32_t* free_pages, const int32_t* n_free, int n_pages, int page_size, int32_t* lens_out,
                            int32_t* n_free_out, void* ws, size_t ws_bytes, moe_stream_t stream);

/* ---- rotary positions ------------------------------------------------------------------------------
 *
 * The first `dim` elements of a head are pairs, each turned by an angle that grows with the token's position p:
 *   (a, b) -> m (a cos t - b sin t, b cos t + a sin t),   t = p f_i,   i = 0 .. dim / 2 - 1
 * with pair i the elements i and i + dim / 2, or 2i and 2i + 1 (interleaved); elements from dim on stay.
 *   turns      [dim / 2] uint64 on the device: f_i as a fraction of a turn in units of 2^-64.  p times that, modulo
 *              2^64, is the angle however far the position is, without 64-bit floating point (kernels take it to
 *              fp32 with an error below 2^-27 of a turn)
 *   magnitude  m, which some of the ways to stretch a context come with */
typedef struct {
  int dim, interleaved;
  float magnitude;
  const uint64_t* turns;
} moe_rope_table;

/* The frequencies f_i = base^(-2i / dim), as trained for a context of `original` positions, or changed for one
 * `factor` times as long:
 *   MOE_ROPE_LINEAR    f_i / factor (positions moved closer together)
 *   MOE_ROPE_BASE      base * factor^(dim / (dim - 2)) in place of base (dim > 2)
 *   MOE_ROPE_BY_INDEX  f_i (1 - r_i) + f_i / factor r_i with r_i = clamp((i - i0) / max(i1 - i0, 0.001), 0, 1):
 *                      pairs that turn more than `high` times in the original context stay, those below `low`
 *                      turns are slowed; i(x) = dim ln(original / (2 pi x)) / (2 ln base) is the index of x turns,
 *                      i0 = max(floor(i(high)), 0), i1 = min(ceil(i(low)), dim - 1); magnitude 0.1 ln factor + 1
 *   MOE_ROPE_BY_TURNS  the same blend with 1 - r_i = clamp((x_i - low) / (high - low), 0, 1), x_i = original f_i /
 *                      (2 pi) the pair's turns in the original context; magnitude 1 */
typedef enum {
  MOE_ROPE_PLAIN = 0,
  MOE_ROPE_LINEAR = 1,
  MOE_ROPE_BASE = 2,
  MOE_ROPE_BY_INDEX = 3,
  MOE_ROPE_BY_TURNS = 4
} moe_rope_scaling;

/* turns_out [dim / 2] and magnitude_out [1] of those frequencies (host memory; a host computation in 64 bits).
 * dim even, 2 to 256; base > 1; factor >= 1; original, low and high above 0 and low < high where they are used. */
moe_status moe_rope_frequencies(int dim, double base, moe_rope_scaling scaling, double factor, double original, double low,
                                double high, uint64_t* turns_out, float* magnitude_out);

/* turns_out [n] of frequencies [n] in radians a position (host memory), for any other rule.  Finite, of magnitude
 * below 2^31. */
moe_status moe_rope_turns(const double* frequencies, int n, uint64_t* turns_out);

/* x turned: rows of [n_heads, head_dim] bf16 or fp32 (dtype), x_stride elements apart, to out, likewise with
 * out_stride (out may be x, with its stride; else apart from it).  pos [T] int32, any value; inverse != 0 turns back
 * (with the same magnitude): the gradient of the operator, and, with it, positions moved by a difference.
 * Products and sums are fp32, rounded once.  head_dim a multiple of 8, up to 256; rope->dim a multiple of 8, up to
 * head_dim; n_heads up to 1024; strides a multiple of 16 bytes; x and out 16-byte aligned. */
moe_status moe_rope_apply(const moe_rope_table* rope, const void* x, int64_t x_stride, void* out, int64_t out_stride,
                          moe_dtype dtype, int T, int n_heads, int head_dim, const int32_t* pos, int inverse,
                          moe_stream_t stream);

/* A step's queries and keys turned, and keys and values into the cache, in one launch.
 *   q       rows of [n_heads, head_dim], k, v rows of [n_kv_heads, head_dim], bf16 or fp32 (dtype), q_stride,
 *           k_stride and v_stride elements apart (multiples of 16 bytes)
 *   q_out   bf16 rows of [n_heads, head_dim], q_out_stride elements apart: what moe_attn_decode takes (may be q, with its
 *           stride, where that is bf16; else apart from it); apart from k, v and the cache
 *   pos     [T] int32: for the angles (a negative one too)
 *   slot    [T] int32: page * page_size + row of each token's place (moe_page_plan); negative: the key and value are
 *           not written.  A slot past the cache writes nothing and records MOE_ERR_BAD_PAGE in ws.  Two tokens of one call
 *           must not be given one place.
 * Keys are rounded, or quantised as by moe_kv_write, once, from their turned fp32 values. */
moe_status moe_rope_kv_write(const moe_rope_table* rope, const moe_kv_cache* cache, const void* q, int64_t q_stride,
                             int n_heads, void* q_out, int64_t q_out_stride, const void* k, const void* v,
                             moe_dtype dtype, int64_t k_stride, int64_t v_stride, int T, const int32_t* pos,
                             const int32_t* slot, void* ws, size_t ws_bytes, moe_stream_t stream);

/* What stands between two blocks on the residual stream, in one pass over [T, d]:
 *   z  = y * rsqrt(mean(y^2) + eps) * w_post     (w_post NULL: z = y)
 *   z  = z * gate                                (gate NULL: no gate)
 *   r' = residual + alpha * z                    (y NULL: r' = residual)
 *   x  = r' * rsqrt(mean(r'^2) + eps) * w_pre    (the next block's input)
 *   y             [T, d] bf16 or fp32 (y_dtype): the block's output, or NULL
 *   w_post, w_pre [d] fp32
 *   gate          rows of d elements, bf16 or fp32 (gate_dtype), gate_stride elements apart (a
 *                 multiple of 8; 0: one row for all tokens), or NULL
 *   residual      [T, d] bf16 or fp32 (r_dtype); residual_out likewise (may be residual itself)
 *   x             [T, d] bf16 or fp32 (x_dtype), or NULL (then w_pre is not read)
 * All sums are fp32; r' and x are each rounded once, x from the fp32 r'.  residual_out may be NULL
 * when y is (the residual then stays as it is).  d a multiple of 8, up to 16384; y, residual,
 * w_post, w_pre, gate, x 16-byte aligned; alpha finite, eps >= 0. */
moe_status moe_block_norm(const void* y, moe_dtype y_dtype, const float* w_post, const void* gate,
                          moe_dtype gate_dtype, int64_t gate_stride, float alpha, const void* residual,
                          void* residual_out, moe_dtype r_dtype, const float* w_pre, void* x, moe_dtype x_dtype, int T,
                          int d, float eps, moe_stream_t stream);

/* Exercises the device-side timeout path: launches one CTA whose wait on a barrier can never
 * complete; the wait gives up after timeout_us (<= 1 s) and records MOE_ERR_TIMEOUT in the
 * workspace's status record, which moe_get_status() then returns.  The GPU context stays
 * usable.  For failure-detection tests. */
moe_status moe_selftest_wait_timeout(void* ws, size_t ws_bytes, unsigned timeout_us, moe_stream_t stream);

/* Static description of a status code. */
const char* moe_status_string(moe_status status);

/* The device E4M3 encoder the kernels use (round to nearest even, saturating at +-448),
 * on n fp32 values: out[i] = code(in[i]).  For codec tests. */
moe_status moe_e4m3_encode(const float* in, uint8_t* out, int64_t n, moe_stream_t stream);

#ifdef __cplusplus
}
#endif

#endif /* LIBMOE_H */
