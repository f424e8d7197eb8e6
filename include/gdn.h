/*
 * gdn.h -- C ABI of the GB300 (sm_103a) Gated DeltaNet recurrence library
 *          (libgdn_gb300.so).
 *
 * The operation.  For every sequence s and value head vh, with the D_v x D_k
 * f32 state S of that pair (row i = d_v index, column j = d_k index) and for
 * tokens t = 0 .. n_tokens-1 in order:
 *
 *     alpha    = exp(-g_t)
 *     S        = alpha * S                       (decay-first, flags bit0 = 0)
 *     sk[i]    = sum_j S[i][j] * k_t[j]
 *     delta[i] = (v_t[i] - sk[i]) * beta_t
 *     S[i][j] += delta[i] * k_t[j]
 *     y_t[i]   = q_scale * sum_j S[i][j] * q_t[j]
 *
 * This is the step order of the kernel body of
 * "gated_delta_net_decode_capture.metal" (mlx-native 0.9.2), steps
 * "decay + partial s_k" and "state update + output partial".  With flags
 * bit0 = 1 the state is decayed after S@k instead, as in the recurrence of
 * the module doc of "gated_delta_net.rs" (mlx-native 0.4.0):
 * S' = alpha*S + beta*outer(v - S@k, k), y = S'@q.
 *
 * k_head, the key/query head read by value head vh ("GQA broadcast",
 * gated_delta_net.rs): vh % n_k_heads (flags bit1 = 0, the capture kernel's
 * head setup) or vh / (n_v_heads / n_k_heads) (flags bit1 = 1).
 *
 * Layouts, innermost (fastest) dimension first, all f32, densely packed
 * ("Memory layouts" table of gated_delta_net.rs; "Memory layout for
 * state_capture" section of the capture kernel page):
 *     q, k            [D_k, n_k_heads, n_tokens, n_seqs]
 *     v, output       [D_v, n_v_heads, n_tokens, n_seqs]
 *     g, beta         [n_v_heads, n_tokens, n_seqs]
 *     state_in/out    [D_k, D_v, n_v_heads, n_seqs]
 *     state_capture   [D_k, D_v, n_v_heads, n_tokens, n_seqs]
 *
 * Parameters: a HOST array of at least 9 uint32 ("Buffer bindings" section of
 * the capture kernel page; "Buffer / params contract" of
 * gated_delta_net_decode.rs, mlx-native 0.21.1):
 *     params[0..5] = D_k, D_v, n_k_heads, n_v_heads, n_tokens, n_seqs
 *     params[6]    = flags (the pages always write 0 here; see GDN_FLAG_*)
 *     params[7]    = reserved, must be 0
 *     params[8]    = q_scale_bits: the f32 bit pattern of q_scale, applied to
 *                    y at writeback; 0 means q_scale = 1.0.
 *
 * Ownership and lifetime.  Every buffer pointer is a DEVICE pointer owned by
 * the caller; the library allocates no memory, keeps no state between calls
 * (apart from the device status word of gdn_device_status) and never
 * synchronises (apart from gdn_device_status).  All work is enqueued on `stream` (NULL = the
 * legacy default stream) and is asynchronous: buffers must stay valid until
 * the stream reaches the call.  Calls on different streams with disjoint
 * buffers may run concurrently.
 *
 * Errors.  Arguments are checked on the host before anything is enqueued; a
 * failed check returns GDN_ERR_INVALID_ARGUMENT or GDN_ERR_UNSUPPORTED and
 * enqueues nothing.  A failed launch returns GDN_ERR_CUDA.  Faults during
 * kernel execution surface through the stream like any CUDA error.  After a
 * non-OK status, gdn_last_error() gives a message (per calling thread).
 *
 * Device-side failures.  The chunked prefill kernels (the chunked path of
 * gdn_forward, gdn_forward_ws, gdn_forward_chunked_noalloc) wait on
 * asynchronous copies and tensor-core work through barriers, and every such
 * wait is bounded (about a second of GPU clock).  A wait that runs out does
 * not hang or fault the GPU: the kernel writes NaN into the affected
 * (seq, value head) state_out (the two-pass form also into its chunk
 * matrices, so the outputs that depend on them become NaN), releases its
 * tensor memory, returns, and sets GDN_DEVICE_WAIT_TIMEOUT in the library's
 * device status word.  The call itself has already returned GDN_OK by then;
 * gdn_device_status() reads the word, which tells a timed-out wait from NaN
 * inputs.  The other kernels have no waits of this kind.
 */
#ifndef GDN_GB300_H
#define GDN_GB300_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as CUDA's cudaStream_t / CUstream. */
typedef struct CUstream_st *gdn_stream_t;

typedef enum gdn_status {
  GDN_OK = 0,
  GDN_ERR_INVALID_ARGUMENT = 1, /* the pages' InvalidArgument cases, and ours */
  GDN_ERR_UNSUPPORTED = 2,      /* valid for the method, no kernel for it here */
  GDN_ERR_CUDA = 3              /* a CUDA runtime call failed */
} gdn_status;

#define GDN_N_PARAMS 9

/* params[6] flag bits.  0 selects the behaviour of the pages' kernel. */
#define GDN_FLAG_DECAY_AFTER 0x1u /* decay after S@k (gated_delta_net.rs)  */
#define GDN_FLAG_KHEAD_DIV 0x2u   /* k_head = vh / (n_v/n_k)               */
#define GDN_PATH_SHIFT 2u         /* bits 2-3: path choice                 */
#define GDN_PATH_MASK 0xCu
#define GDN_PATH_AUTO 0u          /* the library picks by shape            */
#define GDN_PATH_SCAN 1u          /* token-by-token scan kernel            */
#define GDN_PATH_CHUNKED 2u       /* chunked tensor-core prefill, split-bf16
                                     operands                              */
#define GDN_PATH_CHUNKED_TF32 3u  /* the same with TF32 operands (faster,
                                     about 1e-3 less accurate)             */

/*
 * gdn_forward -- run the recurrence over n_tokens tokens for every
 * (seq, value head) pair, write y to `output` and the final state to
 * `state_out`.  Follows dispatch_gated_delta_net_decode
 * (gated_delta_net_decode.rs, mlx-native 0.21.1) and dispatch_gated_delta_net
 * (gated_delta_net.rs, mlx-native 0.4.0); buffer order is the pages' buffer
 * slots 0-8.
 *
 * Checks (mirroring `validate` and `validate_params_buf` of
 * gated_delta_net_decode.rs):
 *   INVALID_ARGUMENT: params == NULL or n_params < 9; any of D_k, D_v,
 *     n_k_heads, n_v_heads, n_tokens, n_seqs == 0; n_v_heads % n_k_heads != 0;
 *     D_k % 32 != 0 or D_k > 128; D_v % (D_k/32) != 0; params[7] != 0;
 *     unknown flag bits; a NULL buffer; q, k, state_in or state_out
 *     not 16-byte aligned, or v, g, beta, output not 4-byte aligned;
 *     state_in and state_out overlapping without being the same pointer
 *     (state_in == state_out, an in-place update, is allowed); output
 *     overlapping any other buffer; on a forced chunked path, v not 16-byte
 *     aligned (its rows are copied 16 bytes at a time).
 *   UNSUPPORTED: D_k = 96 (D_k/32 = 3 has no kernel, as on the pages);
 *     the chunked path forced for a shape it does not cover.
 *
 * Path choice (params[6] bits 2-3).  GDN_PATH_AUTO runs the token-loop
 * kernel for n_tokens <= 16 and for every capture call; for longer windows
 * without capture it runs the tensor-core
 * chunked form when that form covers the call (D_k = D_v = 128, f32
 * activations, no capture, v 16-byte aligned) and n_tokens >= 48, and the
 * token-by-token FP32 scan otherwise.  GDN_PATH_SCAN forces the scan;
 * GDN_PATH_CHUNKED and GDN_PATH_CHUNKED_TF32 force the chunked form
 * (UNSUPPORTED for a shape it does not cover).
 * Accuracy against a double-precision evaluation of the recurrence (rel-L2,
 * 4 x 4096-token windows): the token-loop kernel and the scan compute every
 * product in f32, about 1e-7; the chunked form takes each tensor-core
 * product as three bf16 products of split operands (x = hi + lo), about
 * 1e-5 (3e-5 for negative gates, whose states grow by e^20 over the
 * window); GDN_PATH_CHUNKED_TF32 rounds the operands to TF32 instead, one
 * product each, about 5e-4 (3e-3 for those negative gates).
 * gdn_forward runs the chunked form in one pass; gdn_forward_ws, given a
 * workspace, in two (faster from about 512 tokens on; under GDN_PATH_AUTO it
 * keeps the one pass below that).
 * Buffer sizes cannot be checked through raw pointers: each buffer must hold
 * the element count its layout above gives.
 */
gdn_status gdn_forward(const float *q, const float *k, const float *v, const float *g,
                       const float *beta, const float *state_in, float *output,
                       float *state_out, const uint32_t *params, size_t n_params,
                       gdn_stream_t stream);

/*
 * gdn_forward_capture -- gdn_forward, plus the state after every token
 * written to `state_capture` (slot 9 of the capture kernel page):
 * state_capture[:, :, vh, t, s] = S after token t.  Slice n_tokens-1 is
 * bit-identical to state_out (the "Determinism contract" of
 * dispatch_gated_delta_net_decode_with_capture).  For speculative-decode
 * rollback the caller takes slice `accepted_idx` as the new state.
 *
 * Extra checks (dispatch_gated_delta_net_decode_with_capture):
 *   INVALID_ARGUMENT: state_capture == NULL or not 16-byte aligned, or
 *     overlapping any other buffer; state_capture_elems !=
 *     n_tokens*D_k*D_v*n_v_heads*n_seqs when n_seqs > 1, or smaller than it
 *     when n_seqs == 1 (elements past that count are left untouched).
 *   UNSUPPORTED: the chunked path forced (it keeps no per-token state).
 */
gdn_status gdn_forward_capture(const float *q, const float *k, const float *v, const float *g,
                               const float *beta, const float *state_in, float *output,
                               float *state_out, const uint32_t *params, size_t n_params,
                               float *state_capture, size_t state_capture_elems,
                               gdn_stream_t stream);

/* The buffers of one problem (e.g. one linear-attention layer) for
 * gdn_forward_layers; every pointer is a DEVICE pointer, as in gdn_forward. */
typedef struct gdn_layer_buffers {
  const float *q, *k, *v, *g, *beta, *state_in;
  float *output, *state_out;
  float *state_capture; /* read only when with_capture != 0 */
} gdn_layer_buffers;

/*
 * gdn_forward_layers -- gdn_forward (or gdn_forward_capture when with_capture
 * != 0) on n_layers problems of the same shape and flags (`params`), such as
 * the linear-attention layers of one forward pass, which the pages run one
 * dispatch per layer ("Memory cost" of gated_delta_net_decode_capture.metal:
 * 30+ linear-attention layers per forward).  On the decode path (n_tokens <=
 * 16, automatic path) all layers run in one launch per 64 layers, so a
 * small-batch decode step is not paid for in launch latency; otherwise the
 * layers are launched one after another.  `layers` is a HOST array of
 * n_layers entries (1 <= n_layers <= 1024) that the call reads before it
 * returns.
 *
 * Checks: those of gdn_forward / gdn_forward_capture for every layer (the
 * message names the layer), plus INVALID_ARGUMENT when a layer's output,
 * state_out or state_capture overlaps any buffer of another layer.
 * Results are bit-identical to calling gdn_forward once per layer.
 */
gdn_status gdn_forward_layers(const gdn_layer_buffers *layers, size_t n_layers,
                              const uint32_t *params, size_t n_params, int with_capture,
                              size_t state_capture_elems, gdn_stream_t stream);

/*
 * gdn_commit_capture -- speculative-decode rollback.  After gdn_forward_capture
 * verified n_tokens tokens, make the state after each sequence's last
 * accepted token the active state:
 *     for every s with 0 <= accepted_idx[s] < n_tokens:
 *         state[:, :, :, s] = state_capture[:, :, :, accepted_idx[s], s]
 * Sequences with an index outside [0, n_tokens) (e.g. -1: nothing accepted)
 * keep their state.  The pages leave this step to the caller
 * (dispatch_gated_delta_net_decode_with_capture, gated_delta_net_decode.rs:
 * "the caller reads state_capture[..., accepted_idx, ...] as the new active
 * state"); here it is one launch that reads the indices on the device.
 *
 * state_capture: DEVICE, [D_k, D_v, n_v_heads, n_tokens, n_seqs] f32 as written by
 *   gdn_forward_capture with the same params; state_capture_elems as there.
 * accepted_idx:  DEVICE, n_seqs int32.
 * state:         DEVICE, [D_k, D_v, n_v_heads, n_seqs] f32, updated in place.
 * params:        HOST, the same 9-u32 block as the capture call (n_k_heads and
 *   the flags are checked but not used).
 * Checks: the params checks of gdn_forward; NULL pointers; state_capture and
 *   state 16-byte aligned, accepted_idx 4-byte aligned; the capture size rule
 *   of gdn_forward_capture; state overlapping state_capture or accepted_idx.
 */
gdn_status gdn_commit_capture(const float *state_capture, size_t state_capture_elems,
                              const int32_t *accepted_idx, float *state, const uint32_t *params,
                              size_t n_params, gdn_stream_t stream);

/*
 * bf16 activations with f32 state.  The prefill page ("Dtype / precision" of
 * gated_delta_net.rs, mlx-native 0.4.0) keeps all accumulation in f32 and
 * names bf16 inputs and outputs as a later variant.  These entry points are
 * that variant: q, k, v and output hold bfloat16 (the upper half of an f32
 * bit pattern, as torch.bfloat16 / __nv_bfloat16), in the same layouts as
 * above; g, beta, state_in, state_out and state_capture stay f32.  Each
 * bf16 value is widened exactly to f32 on load, every product and sum is f32
 * as in gdn_forward, and y is rounded once, to nearest-even bf16, when it is
 * stored.  Results for the same widened inputs therefore equal gdn_forward's
 * up to that final rounding of y (state and capture are bit-identical).
 *
 * Extra checks: v 4-byte aligned and output 2-byte aligned (q and k stay
 * 16-byte); UNSUPPORTED when D_v is odd (v is staged two rows at a time) or
 * when the TF32 chunked path is forced.  The chunked path (forced, or chosen
 * by GDN_PATH_AUTO) runs with split operands; bf16 inputs are their own hi
 * halves, so its products leave out the terms with a zero lo half, which
 * add nothing in the f32 form: results keep the equalities above.
 */
typedef uint16_t gdn_bf16; /* bfloat16 bit pattern */

gdn_status gdn_forward_bf16(const gdn_bf16 *q, const gdn_bf16 *k, const gdn_bf16 *v,
                            const float *g, const float *beta, const float *state_in,
                            gdn_bf16 *output, float *state_out, const uint32_t *params,
                            size_t n_params, gdn_stream_t stream);

gdn_status gdn_forward_capture_bf16(const gdn_bf16 *q, const gdn_bf16 *k, const gdn_bf16 *v,
                                    const float *g, const float *beta, const float *state_in,
                                    gdn_bf16 *output, float *state_out, const uint32_t *params,
                                    size_t n_params, float *state_capture,
                                    size_t state_capture_elems, gdn_stream_t stream);

/*
 * Two-pass chunked prefill with a caller-provided workspace.
 *
 * The chunked (WY / UT) form of the recurrence over 64-token chunks splits
 * into a part that does not depend on the state -- per chunk, the Gram
 * products, A, T = (I + A)^-1 and the masked decay-weighted Q K^T -- and the
 * state pass.  gdn_forward_ws runs the first part for every (seq, chunk) in
 * parallel -- the products of K and Q once per key head, the gated parts per
 * value head -- writes it to `workspace`, then runs the state pass (one CTA
 * per (seq, value head)).  The pages have no chunked kernel:
 * the chunk equations are the delta rule's published chunkwise form derived
 * from the recurrence of gated_delta_net.rs (mlx-native 0.4.0) and of the
 * capture kernel page, with the operands of the path bits (split bf16 for
 * GDN_PATH_AUTO and GDN_PATH_CHUNKED, TF32 for GDN_PATH_CHUNKED_TF32).
 *
 * gdn_workspace_size: *bytes = the workspace gdn_forward_ws needs for
 *   `params` -- on the chunked path (forced, or chosen by GDN_PATH_AUTO for
 *   the shape, assuming a 16-byte-aligned v, with at least 512 tokens: the
 *   automatic choice keeps the one-pass form for shorter windows, where it
 *   is the faster one), per (seq, 64-token chunk),
 *   32 KB per value head plus 96 KB per key head (the K and Q operands and K^T,
 *   shared by the value heads that read the key head); 0 on every other
 *   path, and 0 when a key head has more than 32 value heads (the two-pass
 *   form takes at most 32; gdn_forward_ws then runs the one-pass chunked
 *   form of gdn_forward).  Same params checks and status as gdn_path_name.
 *
 * gdn_forward_ws: gdn_forward, plus `workspace` (DEVICE, caller-owned,
 *   at least gdn_workspace_size bytes, 16-byte aligned, overlapping no other
 *   buffer; may be NULL when the size is 0).  The call overwrites the
 *   workspace; its contents afterwards are unspecified.  On the chunked
 *   path (forced, or chosen by GDN_PATH_AUTO for 512 tokens or more) the
 *   two-pass form runs; otherwise the call runs exactly as gdn_forward and
 *   does not touch the workspace.  Extra checks: INVALID_ARGUMENT for a NULL, misaligned,
 *   short or overlapping workspace when the size is > 0.
 */
gdn_status gdn_workspace_size(const uint32_t *params, size_t n_params, size_t *bytes);

gdn_status gdn_forward_ws(const float *q, const float *k, const float *v, const float *g,
                          const float *beta, const float *state_in, float *output,
                          float *state_out, const uint32_t *params, size_t n_params,
                          void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/*
 * gdn_forward_ws_bf16 -- gdn_forward_ws with bf16 q, k, v and output, as
 * gdn_forward_bf16 is to gdn_forward (same layouts, f32 g, beta and state;
 * y rounded once to nearest-even bf16 when stored).  The workspace size is
 * gdn_workspace_size's for the same params; the two-pass form stores only
 * the hi halves of K, Q and K^T (bf16 inputs are exact), using part of it.
 * Results: the state equals gdn_forward_ws's on the same widened inputs bit
 * for bit, and the output equals its output rounded to bf16.  Checks as
 * gdn_forward_bf16 plus the workspace checks of gdn_forward_ws; the TF32
 * chunked path (GDN_PATH_CHUNKED_TF32) is UNSUPPORTED with bf16 activations.
 */
gdn_status gdn_forward_ws_bf16(const gdn_bf16 *q, const gdn_bf16 *k, const gdn_bf16 *v,
                               const float *g, const float *beta, const float *state_in,
                               gdn_bf16 *output, float *state_out, const uint32_t *params,
                               size_t n_params, void *workspace, size_t workspace_bytes,
                               gdn_stream_t stream);

/*
 * gdn_forward_chunked_noalloc -- the two-pass chunked prefill of
 * gdn_forward_ws, for callers that cannot allocate device memory: its chunk
 * scratch lives in a fixed array inside this library instead of a
 * caller-provided workspace.  The pages have no counterpart; it exists for
 * code that only ever receives device buffers from a host framework that
 * owns all device memory (a plugin or an embedded runtime whose memory pool
 * offers it no allocation hook), and for loops that must not pay for
 * cudaMalloc, which can synchronise the device.  Nothing here allocates:
 * no cudaMalloc, no cudaFree, no allocating library routine.
 *
 * Limit: the fixed scratch is 32 MiB, and a problem needs, per (seq,
 * 64-token chunk), 32 KB per value head plus 96 KB per key head (what
 * gdn_workspace_size reports) -- e.g. one sequence of 1024 tokens with 16
 * value and 16 key heads, or of 640 tokens with 48 value and 16 key heads;
 * every GPU on which the library's chunked kernels are loaded holds it until
 * the process exits.  Larger problems return
 * GDN_ERR_INVALID_ARGUMENT with the numbers; use gdn_forward_ws for them.
 *
 * Arguments, layouts and checks as gdn_forward (f32 activations), for the
 * chunked path: the params path bits must not be GDN_PATH_SCAN
 * (GDN_PATH_AUTO means GDN_PATH_CHUNKED here), the chunked path's shape rules apply (D_k = D_v = 128,
 * else GDN_ERR_UNSUPPORTED), and v must be 16-byte aligned as for
 * gdn_forward_ws (INVALID_ARGUMENT otherwise).  Results equal
 * gdn_forward_ws's on the chunked path.  With more than 32 value heads per
 * key head it runs the one-pass chunked form of gdn_forward, which needs no
 * scratch (as gdn_forward_ws does).
 *
 * The first call on a device looks up the device address of the scratch
 * (once per device and context, with that device current; if the context is
 * destroyed and created again, e.g. by cudaDeviceReset, the next call looks
 * it up again); make that first call before any stream capture.  Every call
 * on a device shares the one scratch array:
 * each call writes all of it that it reads, so nothing carries over between
 * calls, but calls that overlap on the GPU (e.g. on two streams at once)
 * race on it and must be ordered by the caller.
 */
gdn_status gdn_forward_chunked_noalloc(const float *q, const float *k, const float *v,
                                       const float *g, const float *beta, const float *state_in,
                                       float *output, float *state_out, const uint32_t *params,
                                       size_t n_params, gdn_stream_t stream);

/* gdn_layer_buffers with bf16 q, k, v and output. */
typedef struct gdn_layer_buffers_bf16 {
  const gdn_bf16 *q, *k, *v;
  const float *g, *beta, *state_in;
  gdn_bf16 *output;
  float *state_out;
  float *state_capture; /* read only when with_capture != 0 */
} gdn_layer_buffers_bf16;

/* gdn_forward_layers on bf16 activations (gdn_forward_bf16 per layer). */
gdn_status gdn_forward_layers_bf16(const gdn_layer_buffers_bf16 *layers, size_t n_layers,
                                   const uint32_t *params, size_t n_params, int with_capture,
                                   size_t state_capture_elems, gdn_stream_t stream);

/*
 * ======================================================================
 * The full-attention layers of a hybrid model's serving step.
 *
 * Hybrid LLMs put a full-attention layer between their Gated DeltaNet
 * layers.  The calls below are that layer's part of a step over a paged
 * key-value cache: gdn_kv_plan assigns pages and slots from the request
 * lengths, gdn_rope_store rotates q and k and stores k and v, gdn_attn_paged
 * attends.  All three read the lengths on the device, so a whole step can be
 * enqueued or graph-captured without a host round trip.  Ownership, streams
 * and errors are those of the calls above; the params structs are HOST memory
 * that the call reads before it returns.  The source pages have no counterpart
 * of these calls.
 *
 * The cache.  k_cache and v_cache (same layout, f32 or bf16) hold, for page p,
 * key head h and position o within the page, head_dim contiguous elements at
 *     p * cache_page_stride + h * cache_head_stride + o * cache_slot_stride
 * (strides in elements; [head_dim, page_size, n_kv_heads, n_pages] or
 * [head_dim, n_kv_heads, page_size, n_pages], innermost first, or a view of a
 * larger array).  Slot number: p * page_size + o.  Any page_size >= 1.
 *
 * Rows of q, k, v and of the outputs: per token, [head_dim, n_heads] contiguous
 * elements; tokens lie a token stride apart, so views of a fused projection's
 * output are taken as they are.
 */
#define GDN_DTYPE_F32 0u
#define GDN_DTYPE_BF16 1u

typedef struct gdn_kv_plan_params {
  uint32_t n_seqs;     /* requests */
  uint32_t page_size;
  uint32_t n_pages;    /* pages of the cache */
  uint32_t max_pages;  /* entries of a block-table row */
  uint32_t n_free_max; /* entries of free_pages */
  uint32_t n_slots;    /* entries of slot_map and positions */
} gdn_kv_plan_params;

/*
 * gdn_kv_plan -- the bookkeeping of one step, on the device.  All arrays are
 * DEVICE int32; request s has ctx_lens[s] cached tokens, adds new_lens[s]
 * (0: an idle slot), and holds the pages block_table[s][0 .. owned[s]).
 * free_pages[0 .. n_free[0]) is a stack of unused pages, taken from its end.
 *
 *   need[s]   = max(owned[s], ceil((ctx_lens[s] + new_lens[s]) / page_size))
 *   block_table[s][owned[s] .. need[s]) = the next pages of the stack, request
 *               after request (updated in place; other entries are kept)
 *   owned_out[s] = need[s];  kv_lens[s] = ctx_lens[s] + new_lens[s]
 *   n_free_out[0] = n_free[0] - pages taken
 *   token_start[s] (n_seqs + 1 entries) = new tokens of the requests before s
 *   positions[i], slot_map[i] of the step's token i (the requests' new tokens,
 *               packed): its position in its request and its cache slot;
 *               entries past the step's tokens are 0 and -1
 *
 * After a rollback to a shorter ctx_lens the pages beyond stay owned and are
 * filled again.  A request whose pages the stack cannot give is not served: its
 * tokens' slots are -1, its kv_lens stays ctx_lens, its table row and owned
 * stay, and GDN_DEVICE_OUT_OF_PAGES is set; once one was not served, no later
 * request that needs a page is.  A request with impossible numbers (negative,
 * more cached tokens than its pages hold, more pages than max_pages) is not
 * served either (its kv_lens is 0 where the cached part itself is impossible),
 * and GDN_DEVICE_BAD_REQUEST is set, as it is when the step has more than
 * n_slots tokens (the first n_slots are written) or n_free is out of range.
 *
 * Checks: INVALID_ARGUMENT for NULL or not 4-byte-aligned pointers, zero
 * n_seqs, page_size, n_pages or max_pages, page counts times page_size at 2^31
 * or above, and an output that overlaps another array.
 * One launch; results do not depend on its shape.
 */
gdn_status gdn_kv_plan(const int32_t *ctx_lens, const int32_t *new_lens, const int32_t *owned,
                       const int32_t *free_pages, const int32_t *n_free, int32_t *block_table,
                       int32_t *kv_lens, int32_t *owned_out, int32_t *n_free_out,
                       int32_t *token_start, int32_t *slot_map, int32_t *positions,
                       const gdn_kv_plan_params *params, gdn_stream_t stream);

#define GDN_ROPE_INTERLEAVED 0x1u /* pairs (2j, 2j+1) instead of (j, j + rot_dim/2) */
#define GDN_ROPE_INVERSE 0x2u     /* the inverse rotation, which is the gradient's */
#define GDN_ROPE_MAX_DIM 256u     /* largest head_dim */

typedef struct gdn_rope_params {
  uint32_t dtype; /* of q, k, v, outputs and caches */
  uint32_t head_dim, rot_dim; /* the first rot_dim elements of a head are rotated, the rest copied */
  uint32_t n_q_heads, n_kv_heads, n_tokens;
  uint32_t n_axes, n_positions; /* rows of `positions`; rows of cos_sin */
  uint32_t flags;
  uint32_t page_size, n_pages; /* gdn_rope_store only, as the cache strides */
  int64_t q_stride, k_stride, v_stride, q_out_stride, k_out_stride; /* token strides */
  int64_t positions_stride; /* elements between axes; 0: every axis reads the same row */
  int64_t cache_page_stride, cache_head_stride, cache_slot_stride;
  uint8_t axis_of_pair[GDN_ROPE_MAX_DIM / 2]; /* the axis of each of the rot_dim/2 pairs */
} gdn_rope_params;

/*
 * gdn_rope -- rotary positions with one or more axes (time; time, height,
 * width; ...).  Pair j of every q and k head, at the token's position
 * p = positions[axis_of_pair[j]][token]:
 *     (a, b) -> (a c - b s, b c + a s),   c = cos_sin[p][j], s = cos_sin[p][rot_dim/2 + j]
 * cos_sin: DEVICE f32 [rot_dim, n_positions], innermost first.  Computed in
 * f32 and rounded once when stored.  q_out and k_out may be q and k (in place).
 * The gradients of q and k are the same call on the outputs' gradients with
 * GDN_ROPE_INVERSE.
 *
 * gdn_rope_store -- gdn_rope whose k goes to the cache, with v beside it: token
 * i's rows are stored at slot_map[i] (-1: nowhere; DEVICE int32).  Two tokens
 * of a call must not share a slot.
 *
 * A position outside [0, n_positions) makes the token's rotated elements NaN
 * and sets GDN_DEVICE_BAD_POSITION; a slot past the cache stores nothing and
 * sets GDN_DEVICE_BAD_PAGE.
 *
 * Checks: INVALID_ARGUMENT for NULL pointers, zero sizes (n_tokens may be 0:
 * nothing is done), head_dim odd, 0 or above GDN_ROPE_MAX_DIM, rot_dim odd or
 * outside (0, head_dim], an axis_of_pair entry >= n_axes, unknown flags or
 * dtype, pointers not aligned to an element, token strides below a row's
 * length, an output that overlaps another buffer (other than exactly its own
 * input; k_cache and v_cache may lie among one another, as views of one array,
 * while no row of one shares a byte with one of the other), cache strides of which one
 * is below what the smaller ones and a row cover (gdn_rope_store; strides over an
 * extent of 1 do not count); UNSUPPORTED for GDN_ROPE_INVERSE with gdn_rope_store.  Any alignment
 * and strides are taken; 16-byte aligned rows go 16 bytes at a time.
 */
gdn_status gdn_rope(const void *q, const void *k, const int32_t *positions, const float *cos_sin,
                    void *q_out, void *k_out, const gdn_rope_params *params, gdn_stream_t stream);

gdn_status gdn_rope_store(const void *q, const void *k, const void *v, const int32_t *positions,
                          const float *cos_sin, const int32_t *slot_map, void *q_out, void *k_cache,
                          void *v_cache, const gdn_rope_params *params, gdn_stream_t stream);

typedef struct gdn_attn_params {
  uint32_t dtype; /* of q, the caches and the output */
  uint32_t head_dim; /* 64, 128 or 256 */
  uint32_t n_q_heads, n_kv_heads;
  uint32_t n_seqs, n_tokens; /* requests; rows of q */
  uint32_t page_size, n_pages, max_pages;
  uint32_t window; /* > 0: a token sees its last `window` keys only */
  float scale;     /* of the scores, e.g. 1/sqrt(head_dim) */
  int64_t q_stride, out_stride; /* token strides */
  int64_t cache_page_stride, cache_head_stride, cache_slot_stride;
} gdn_attn_params;

/*
 * gdn_attn_paged -- attention of each request's newest tokens over its cached
 * keys and values.  Request s has kv_lens[s] keys, the step's among them, in
 * the pages of block_table row s (max_pages entries), and the q rows
 * token_start[s] .. token_start[s + 1] (NULL: row s).  Its row t of T sees
 * keys j <= kv_lens[s] - T + t, and of those the last `window` if window > 0:
 *     output = sum_j p_j v_j,   p = softmax over the seen j of scale * q.k_j
 * per query head h, with key head h / (n_q_heads / n_kv_heads).  A row that
 * sees no key is zero.  Cache contents that a row does not see do not reach it,
 * NaN and infinities included; infinities that it does see give NaN or
 * infinities.  One token per request (decode) or a window of a few
 * (verification of drafted tokens) is what it is built for; longer windows are
 * right but read the keys once per block of 8 to 64 rows (tokens times query
 * heads per key head), and every block reads all keys that any of the request's
 * rows sees: a prompt of T tokens costs T times its length, and a sliding window
 * far shorter than the prompt does not change that.  Rows of q that no request has
 * are not written.
 *
 * The running maximum, the sums and the result are f32, rounded once at the end.
 * f32 operands are split so that a product is good to 2^-20 of its factors'
 * magnitudes; bf16 q, k and v are exact, and each probability is good to 2^-16
 * where the result's rounding takes 2^-8.  Sums are kept relative to a maximum that
 * may lag by a factor of 2^8: values above 2^119 may give infinities.  Results do
 * not vary from run to run.
 *
 * workspace: DEVICE, at least gdn_attn_workspace_size bytes, 16-byte aligned,
 * contents irrelevant before and unspecified after; concurrent calls need one
 * each.  The size depends on dtype, head_dim, heads, n_seqs and n_tokens only,
 * and not on the lengths.
 *
 * A table entry outside [0, n_pages) for a key that one of the request's rows sees makes
 * the rows of that request's key head NaN and sets GDN_DEVICE_BAD_PAGE (entries of pages
 * that the window has left may hold anything); a length outside
 * [0, max_pages * page_size] or a token_start that does not ascend within
 * [0, n_tokens] is clipped and sets GDN_DEVICE_BAD_REQUEST.
 *
 * Checks: INVALID_ARGUMENT for NULL pointers, zero sizes (n_tokens may be 0),
 * n_q_heads % n_kv_heads != 0, unknown dtype, a scale that is not finite, caches
 * not 16-byte aligned or their strides not multiples of 16 bytes, bf16 q not
 * 4-byte aligned or with an odd stride, other pointers not aligned to an
 * element, token strides below a row's length, page counts times page_size at
 * 2^31 - 2^16 or above, n_tokens < n_seqs without token_start, output
 * overlapping any other buffer, the workspace rules; UNSUPPORTED for a head_dim
 * other than 64, 128, 256.
 */
gdn_status gdn_attn_workspace_size(const gdn_attn_params *params, size_t *bytes);

gdn_status gdn_attn_paged(const void *q, const void *k_cache, const void *v_cache,
                          const int32_t *block_table, const int32_t *kv_lens,
                          const int32_t *token_start, void *output, const gdn_attn_params *params,
                          void *workspace, size_t workspace_bytes, gdn_stream_t stream);

/* Message for the last non-OK status returned on the calling thread ("" if
 * none).  The pointer stays valid until the thread's next call. */
const char *gdn_last_error(void);

/* Bits of the device status word. */
#define GDN_DEVICE_WAIT_TIMEOUT 0x1u /* a chunked kernel's bounded wait ran out */
#define GDN_DEVICE_OUT_OF_PAGES 0x2u /* gdn_kv_plan: the free stack could not serve a request */
#define GDN_DEVICE_BAD_REQUEST 0x4u  /* gdn_kv_plan, gdn_attn_paged: impossible lengths or offsets */
#define GDN_DEVICE_BAD_PAGE 0x8u     /* a page number or slot outside the cache */
#define GDN_DEVICE_BAD_POSITION 0x10u /* gdn_rope*: a position outside the cos/sin table */

/*
 * gdn_device_status -- the library's device-side failure channel (see
 * "Device-side failures" above).  The pages report errors as a Result from
 * validation on the host ("validate", gated_delta_net_decode.rs); a failure
 * that can only happen while a kernel runs needs a channel of its own, and
 * this is it.
 *
 * Waits for all work enqueued on `stream` so far (it synchronises the
 * stream), then stores in *status (HOST pointer) the OR of the GDN_DEVICE_*
 * bits set by any kernel of this library on the CURRENT device since the
 * word was last cleared (0 = no failure); with reset != 0 the word is
 * cleared afterwards.  One word per device, shared by every stream and
 * thread: read it after the calls of interest have been enqueued on
 * `stream`, and order work on other streams yourself.  Allocates nothing.
 * Returns INVALID_ARGUMENT for status == NULL, GDN_ERR_CUDA if the read
 * fails (e.g. an earlier fault left the context unusable).
 */
gdn_status gdn_device_status(uint32_t *status, int reset, gdn_stream_t stream);

/* The kernel path the library would run for `params` (with or without
 * capture): on GDN_OK, *name points to a static string such as
 * "token_loop_decode".  Runs the same params checks as gdn_forward and returns
 * the same status for invalid params.  Host-only: enqueues nothing. */
gdn_status gdn_path_name(const uint32_t *params, size_t n_params, int capture,
                         const char **name);

#ifdef __cplusplus
}
#endif

#endif /* GDN_GB300_H */
