/*
 * kda_recoverssm.h -- C ABI of the MI355X (gfx950) KDA RecoverSSM library.
 *
 * The library implements, for Kimi Delta Attention (KDA) layers served with
 * speculative decoding, the two device operations the vLLM Kimi-K3 pages
 * describe:
 *
 *   kda_conv_update_verify  -- the speculative verify of one KDA layer with
 *       the depthwise causal short convolution fused in.  Per request and
 *       head it runs the gated delta rule over the draft positions starting
 *       from the request's checkpoint state, writes the outputs, the per-
 *       position correction and [raw key | raw gate] records, and rolls the
 *       conv state in place.  The checkpoint is only read.
 *       (kernels page `vllm.models.kimi_k3.nvidia.recoverssm.kernels`,
 *       class `CuteRecoverSSMVerify`, method `__call__`; ops page
 *       `vllm/models/kimi_k3/nvidia/ops/recoverssm.py`, functions
 *       `_kda_gate`, `_kda_recurrent_step`, `_kda_recoverssm_verify_kernel`,
 *       `kda_recoverssm_verify`.)
 *
 *   kda_recoverssm_commit   -- folds each request's first n accepted
 *       positions, from those records, into its checkpoint state, for every
 *       layer in one launch; in align mode (prefix caching) it also stores
 *       the state at a completed block boundary.
 *       (kernels page, function `cute_recoverssm_commit`; ops page,
 *       `_commit_kda_state_kernel` and `KDARecoverSSMCommitContext`.)
 *
 *   kda_commit_plan, kda_compact_conv_state -- the two launches that the
 *       ops page's `KDARecoverSSMCommitContext.commit` runs before the
 *       state commit: the per-request plan (commit lengths, final and
 *       boundary slots) and the conv-state compaction.
 *
 *   kda_recoverssm_commit_step -- those three (plan, compaction, commit)
 *       with the same results, in one launch.
 *
 *   kda_conv_prefill, kda_conv_update_decode -- the layer on prompts (the
 *       chunked form, from a zero or given state) and on single tokens (the
 *       recurrent form), which produce and advance the checkpoints that the
 *       verify starts from.
 *
 *   kda_step_tables -- a step's index arrays built on the GPU from request
 *       lengths: token offsets, new blocks, state slots, cache slots.
 *
 *   kda_sample -- tokens from logits and given random numbers, and the
 *       accepted counts of draft windows that the commit plan reads.
 *
 *   kda_latent_write, kda_latent_attention -- the attention layers between
 *       KDA layers, over a paged cache of one latent vector a token, for
 *       single tokens and draft windows.
 *
 *   kda_latent_expand, kda_latent_prefill -- the same layers on prompts: keys
 *       and values of every head from the cached latents, and the causal
 *       attention over them.
 *
 *   kda_copy_blocks, kda_fork_blocks, kda_free_blocks, kda_compact_blocks --
 *       blocks shared, copied, given back and moved, over the states, conv
 *       states and caches that share a block table.
 *
 *   kda_adjust_logits -- biases, penalties for repeated tokens and grammar
 *       masks on the logits that kda_sample takes.
 *
 * plus host-only argument checks mirroring the pages' validation
 * (kernels page `_check_layouts`, `can_use_cute_recoverssm`; ops page
 * `kda_recoverssm_verify`, `KDARecoverSSMCommitContext.create/commit`).
 *
 * Conventions shared by every entry point
 * ---------------------------------------
 *  - Tensors are described by kda_tensor: a device pointer, a dtype, and up
 *    to four sizes and strides, strides counted in ELEMENTS.  Every pointer
 *    handed to the library is a device pointer unless stated otherwise.
 *  - The caller owns every buffer.  The library allocates no device memory,
 *    keeps no pointer after a call returns and performs no host/device
 *    synchronisation.  Launches are asynchronous on the given stream (a
 *    hipStream_t passed as void*; NULL = the null stream), so every launch
 *    may be captured in a HIP graph.
 *  - Every entry point returns KDA_OK (0) or a kda_status code; a failing
 *    call launches nothing and leaves a message for kda_last_error() in the
 *    calling thread.  Zero-sized work (batch 0, or no tokens for a verify
 *    without pending_lens) returns KDA_OK without launching.
 *  - Values that live on the device (query lengths, slots, accepted counts,
 *    commit lengths, record rows) are never read by the host.  The kernels
 *    clamp them instead: query length to [0, Q], accepted count to [1, Q],
 *    commit length to [0, Q]; a slot <= null_block_id or >= the pool size is
 *    null; a record row outside [0, rows) writes (verify) or reads (commit)
 *    no records.
 *  - Two requests of one launch must not name the same non-null slot, and a
 *    commit's final slot must not be another request's source slot; the
 *    pages leave these cases undefined and so does this library.
 */
#ifndef KDA_RECOVERSSM_H
#define KDA_RECOVERSSM_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#define KDA_ABI_VERSION 6

/* Status codes. */
typedef enum {
  KDA_OK = 0,
  KDA_E_SHAPE = 1,       /* sizes disagree with each other */
  KDA_E_DTYPE = 2,       /* an element type that is not accepted */
  KDA_E_LAYOUT = 3,      /* strides or alignment of a cache page or
                            parameter tensor (kernels page `_check_layouts`) */
  KDA_E_UNALIGNED = 4,   /* a per-step activation does not start on a
                            16-byte boundary; nothing is launched and the
                            caller may run another implementation (kernels
                            page, `CuteRecoverSSMVerify.__call__` returns
                            False in that case) */
  KDA_E_UNSUPPORTED = 5, /* head dim not in {16,32,64,128}, conv width not
                            4, window Q not in 1..16 */
  KDA_E_CAPACITY = 6,    /* more tokens than batch * Q (ops page,
                            `kda_recoverssm_verify`) */
  KDA_E_DEVICE = 7,      /* a HIP runtime error */
  KDA_E_ARG = 8          /* a required pointer is NULL or a count is
                            negative */
} kda_status;

/* Element types. */
typedef enum { KDA_F32 = 0, KDA_BF16 = 1 } kda_dtype;

/* How the verify hands out its (request, head) work items. */
typedef enum {
  KDA_SCHEDULE_DEFAULT = 0,    /* the library's choice (the fastest measured
                                  for the shape: PER_ITEM up to 65535
                                  requests, else TICKETS) */
  KDA_SCHEDULE_PER_ITEM = 1,   /* one workgroup per item, handed out by the
                                  hardware dispatcher (each XCD takes one
                                  contiguous eighth of the items) */
  KDA_SCHEDULE_TICKETS = 2,    /* persistent workgroups drawing tickets of
                                  items_per_ticket items from work_counter
                                  (the kernels page's design) */
  KDA_SCHEDULE_V_TILES = 3     /* v_tiles workgroups per item, each taking
                                  head_dim / v_tiles rows of the state (the
                                  ops page's verify grid over V blocks,
                                  requests and heads), for batches too small
                                  to fill the GPU; the conv roll of the q
                                  and k channels waits for every V-tile of
                                  the item through an arrival counter in
                                  work_counter.  Head dims 64 and 128,
                                  windows up to 8, no pending_lens.  Same
                                  results, bit for bit, as PER_ITEM. */
} kda_schedule;

/* A strided tensor view.  `stride` is in elements; unused trailing entries
   of shape/stride are ignored. */
typedef struct {
  void* data;
  int32_t dtype;     /* kda_dtype */
  int32_t ndim;
  int64_t shape[4];
  int64_t stride[4];
} kda_tensor;

/* Arguments of kda_conv_update_verify.  H = number of heads, D = head dim
   (= key dim = value dim), T = token rows, Q = spec_query_len (draft window),
   W = 4 conv taps, Lc = Q + W - 2 conv-state length, N state slots, R record
   rows.  "act" is the activation dtype (F32 or BF16) shared by mixed_qkv,
   raw_gate, raw_beta and conv_state. */
typedef struct {
  kda_tensor mixed_qkv;    /* act [T, 3HD]: raw q|k|v projections before the
                              convolution; channel = part*H*D + h*D + d */
  kda_tensor raw_gate;     /* act [T, HD]: gate input before dt_bias */
  kda_tensor raw_beta;     /* act [T, H]: beta before the sigmoid */
  kda_tensor A_log;        /* F32 [H], contiguous */
  kda_tensor dt_bias;      /* F32 [H, D] (or [H*D]), contiguous */
  kda_tensor state;        /* F32 [N, H, D(v), D(k)]: checkpoint pool, read
                              only; strides (any, D*D, D, 1), slot stride a
                              multiple of 16 bytes */
  kda_tensor correction;   /* F32 [R, H, Q, D]: correction record */
  kda_tensor key_gate;     /* F32 or act [R, H, Q, 2D]: [0,D) post-conv raw
                              key, [D,2D) raw gate */
  kda_tensor out;          /* F32 or act [T, HD] */
  kda_tensor conv_state;   /* act; dim-first [N, 3HD, Lc] or token-first
                              [N, Lc, 3HD] (see conv_dim_first); rolled in
                              place */
  kda_tensor conv_weight;  /* F32 or act [3HD, W]; weight[:, W-1] multiplies
                              the newest input */
  const int32_t* query_start_loc;      /* [batch+1] token offsets */
  const int32_t* state_indices;        /* [batch] checkpoint slots */
  const int32_t* num_accepted_tokens;  /* [batch] conv history offset + 1 */
  const int32_t* record_rows;          /* [batch] record row, or NULL: the
                                          request's state slot */
  int32_t* work_counter;   /* device int32[work_counter_len]: [0] is the
                              ticket counter of the ticket schedule,
                              [1 + b * H + h] the arrival counter of request
                              b, head h under the V-tile schedule (fused
                              conv only).  Must be 0 before the first
                              launch; every launch leaves it at 0.  One
                              counter array per launch in flight.  May be
                              NULL for the other schedules. */
  int32_t batch;
  int32_t spec_query_len;  /* Q */
  int32_t null_block_id;   /* slots <= this are null (the ops page imports
                              the value without printing it; the tests
                              use 0) */
  int32_t conv_dim_first;  /* 1: conv_state is [N, 3HD, Lc]; 0: [N, Lc, 3HD] */
  int32_t use_lower_bound; /* 1: g = lower_bound*sigmoid(A x); 0: softplus */
  float lower_bound;
  int32_t max_workgroups;  /* ticket schedule: at most this many
                              workgroups (0 = as many as are resident at
                              once); ignored by the per-item schedule */
  int32_t items_per_ticket; /* ticket schedule: (request, head) items
                               claimed per ticket; 0 = library default */
  int32_t schedule;        /* kda_schedule */
  const int32_t* pending_lens; /* device [batch] or NULL.  When given, the
                              launch first performs the deferred commit of
                              the previous step (state page, deferred
                              commit; ops page `_commit_kda_state_kernel`):
                              the first pending_lens[b] positions (clamped
                              to [0, Q]) recorded in request b's record row
                              are folded into its checkpoint, which is
                              written back in place, and the verify then
                              starts from the updated state and overwrites
                              that row with this step's records.  A request
                              with a live slot and an empty window (no
                              tokens, or T = 0) still folds its pending
                              positions.  Uses the per-item schedule
                              (batch <= 65535). */
  int32_t work_counter_len; /* elements of work_counter; 0 with a counter
                               means 1.  The V-tile schedule of the fused
                               conv verify needs 1 + batch * H. */
  int32_t v_tiles;         /* V-tile schedule: 2, 4 or 8 workgroups per
                              (request, head); 0 = the library's choice */
} kda_verify_args;

/* Arguments of kda_recoverssm_commit.  Per-layer tensors are described by
   device tables of int64 base byte addresses and slot (row) strides in
   elements, as the ops page's commit context builds them; inner strides
   are shared by all layers. */
typedef struct {
  int32_t num_layers;          /* L >= 1 */
  int32_t batch;
  int32_t num_heads;           /* H */
  int32_t head_dim;            /* D */
  int32_t spec_query_len;      /* Q */
  int32_t null_block_id;
  int64_t num_slots;           /* N of every layer's state pool */
  int64_t num_record_rows;     /* R of every layer's records */
  /* device int64[L] tables */
  const int64_t* state_base_addrs;          /* F32 [N, H, D, D] views */
  const int64_t* state_block_strides;
  const int64_t* correction_base_addrs;     /* F32 [R, H, Q, D] views */
  const int64_t* correction_block_strides;
  const int64_t* key_gate_base_addrs;       /* [R, H, Q, 2D] views */
  const int64_t* key_gate_block_strides;
  int64_t state_strides[2];       /* head, row; must be (D*D, D) */
  int64_t correction_strides[2];  /* head, position; dim stride is 1 */
  int64_t key_gate_strides[2];    /* head, position; dim stride is 1 */
  int32_t key_gate_dtype;         /* kda_dtype */
  int32_t max_workgroups;         /* 0: one workgroup per (layer, request,
                                     head); > 0: a persistent grid of at
                                     most this many workgroups */
  const float* A_log;             /* device F32 [L, H] */
  int64_t A_log_strides[2];
  const float* dt_bias;           /* device F32 [L, H, D] */
  int64_t dt_bias_strides[3];
  const int32_t* use_lower_bound; /* device int32 [L]: gate kind per layer */
  const float* lower_bound;       /* device F32 [L] */
  const int32_t* state_indices;   /* device [batch] source slots */
  const int32_t* commit_lens;     /* device [batch] accepted positions */
  const int32_t* final_state_indices; /* device [batch] or NULL: in place */
  const int32_t* record_rows;     /* device [batch] or NULL: source slot */
  /* Optional HOST copy of the six device tables, laid out as int64[6][L] in
     the order above (state bases, state strides, correction bases,
     correction strides, key/gate bases, key/gate strides).  When given,
     the checks verify every layer's alignment; NULL skips those checks. */
  const int64_t* host_tables;
  /* Align mode (ops page `_commit_kda_state_kernel` with ALIGN_MODE): both
     NULL, or both device int32 [batch].  A request that commits and whose
     boundary slot is live also stores, before its final state, the state
     after its first m = boundary_recovery_lens[b] (clamped to [0, n])
     positions at that slot.  Both states come from the source checkpoint
     as it was before the launch; a request's boundary and final slots must
     not be another request's source or destination in the same launch. */
  const int32_t* boundary_state_indices;
  const int32_t* boundary_recovery_lens;
} kda_commit_args;

/* Arguments of kda_commit_plan (ops page: `_prepare_commit_plan_kernel`,
   launched by `KDARecoverSSMCommitContext.commit`; its body is not on the
   pages).  For row b of the batch, with row = request_indices[b] (or b):
     n = num_accepted_tokens[row] clamped to [0, q_b], q_b the window of b
         (0 when state_indices[b] <= null_block_id);
   without a block table: final = state_indices[b], boundary = null id,
   boundary length 0.  With one (prefix caching, one state block per
   mamba_block_size tokens), for c = num_computed_tokens[row] (tokens before
   the window, clamped to >= 0) and n >= 1:
     final = block_table[row][(c + n) / bs], the block that will hold the
             next token (null id when past the table's width);
     when that block starts at P with c < P (the committed tokens completed
     the block before it) and P / bs - 1 is inside the table,
     boundary = block_table[row][P / bs - 1] with boundary length P - c;
     otherwise boundary = null id, length 0.
   A row outside [0, num_request_rows) plans no commit (n = 0). */
typedef struct {
  int32_t batch;
  int32_t spec_query_len;          /* Q */
  int32_t null_block_id;
  int32_t mamba_block_size;        /* align mode: tokens per block, >= Q */
  int32_t num_request_rows;        /* rows of the per-request arrays */
  int32_t block_table_width;       /* align mode: blocks per row */
  int64_t block_table_strides[2];  /* align mode: row, column (elements) */
  const int32_t* num_accepted_tokens;  /* device, per request row */
  const int32_t* request_indices;      /* device [batch] or NULL */
  const int32_t* state_indices;        /* device [batch] */
  const int32_t* query_start_loc;      /* device [batch + 1] */
  const int32_t* block_table;          /* device or NULL (no align) */
  const int32_t* num_computed_tokens;  /* device per request row, or NULL;
                                          given iff block_table is */
  int32_t* commit_lens;                /* device [batch] outputs */
  int32_t* final_state_indices;
  int32_t* boundary_state_indices;
  int32_t* boundary_recovery_lens;
} kda_plan_args;

/* Arguments of kda_compact_conv_state (ops page: `_compact_conv_state_kernel`,
   launched by `KDARecoverSSMCommitContext.commit`; its body is not on the
   pages).  The verify leaves a request's conv state rolled: entry 2 + t
   holds window input t, entries 0 and 1 the two inputs before the window.
   For every layer and every request with a live source slot, n =
   commit_lens[b] (clamped to [0, Q]) >= 1 and a live final slot, entries
   [n - 1, n + 2) of the source (the three inputs before token n of the
   window) are copied to entries [0, 3) of the final slot, so that the next
   verify reads its history with accepted count 1.  In align mode the
   entries [m - 1, m + 2) go to a live boundary slot the same way, when
   m = boundary_recovery_lens[b] (clamped to [0, n]) >= 1.  Other entries
   are not touched; values are copied bit for bit; everything is read
   before anything is written, and the boundary is written first. */
typedef struct {
  int32_t num_layers;
  int32_t batch;
  int32_t spec_query_len;       /* Q: the conv state holds Q + 2 entries */
  int32_t null_block_id;
  int64_t num_slots;            /* N */
  int64_t conv_dim;             /* channels, 3 * H * D */
  int32_t conv_dtype;           /* kda_dtype of every layer's conv state */
  int32_t pad_;
  /* device int64 [4][L]: per layer, the base byte address, then the slot,
     channel and token strides (elements) of its conv state seen dim-first
     as [N, conv_dim, Q + 2] (a token-first state is its transpose). */
  const int64_t* conv_tables;
  const int64_t* host_conv_tables;  /* optional HOST copy, for the checks */
  const int32_t* state_indices;           /* device [batch] */
  const int32_t* commit_lens;             /* device [batch] */
  const int32_t* final_state_indices;     /* device [batch] or NULL */
  const int32_t* boundary_state_indices;  /* both NULL or both given */
  const int32_t* boundary_recovery_lens;
} kda_compact_args;

/* Arguments of kda_conv_prefill and kda_prefill_qkv: the KDA layer over whole
   prompts, B requests of any lengths laid end to end in T token rows.  Per
   request and head, from S_0 (the initial slot's state, or zero), with
   q, k, v, g, beta formed exactly as in the verify:
     c_t = beta_t (v_t - S_{t-1} diag(e^g_t) k_hat_t),
     S_t = S_{t-1} diag(e^g_t) + c_t k_hat_t^T,  out_t = S_t q_t.
   The last state goes to the request's state slot and, with the fused conv,
   its last three raw inputs to entries [0, 3) of that slot's conv state (read
   back with accepted count 1); other entries stay.  A request without tokens
   changes nothing, its state slot included.  Tokens are taken 32 at a time: an
   input that is not finite spoils its request's outputs from up to 31 tokens
   before it on, and no other request's.  Arithmetic is fp32-like, its errors
   going by the largest value that a row v of the state, or that v, has within
   the 32 tokens. */
typedef struct {
  kda_tensor mixed_qkv;    /* act [T, 3HD]: raw q|k|v (kda_conv_prefill) or
                              convolved q|k|v (kda_prefill_qkv) */
  kda_tensor raw_gate;     /* act [T, HD] */
  kda_tensor raw_beta;     /* act [T, H] */
  kda_tensor A_log;        /* F32 [H], contiguous */
  kda_tensor dt_bias;      /* F32 [H, D] (or [H*D]), contiguous */
  kda_tensor state;        /* F32 [N, H, D(v), D(k)], as for the verify */
  kda_tensor out;          /* F32 or act [T, HD] */
  kda_tensor conv_state;   /* act; as for the verify (conv only) */
  kda_tensor conv_weight;  /* F32 or act [3HD, W] (conv only) */
  const int32_t* query_start_loc;       /* [batch+1] token offsets, clamped
                                           to [0, T]; not decreasing */
  const int32_t* state_indices;         /* [batch] slots that receive the
                                           states; a request whose slot is
                                           null gets +0.0 outputs and
                                           nothing else */
  const int32_t* initial_state_indices; /* [batch] slots the requests start
                                           from (state and conv history), a
                                           null slot meaning zeros; may name
                                           the request's own slot.  NULL:
                                           every request starts from zero */
  const int32_t* num_accepted_tokens;   /* [batch] conv history offset + 1 in
                                           the initial slot, clamped to
                                           [1, Q], or NULL: 1 */
  void* workspace;         /* device, 16-byte aligned, at least
                              kda_prefill_workspace_size(...) bytes; not
                              shared by launches in flight together */
  int64_t workspace_bytes;
  int32_t batch;
  int32_t spec_query_len;  /* Q: the conv state holds Q + 2 entries */
  int32_t null_block_id;
  int32_t conv_dim_first;
  int32_t use_lower_bound;
  float lower_bound;       /* at most 0 (a bound above 0 lets states grow past
                              the operands' range and is refused here, not by
                              the decode) */
} kda_prefill_args;

/* Arguments of kda_conv_update_decode and kda_decode_qkv: one token for each
   of `batch` requests (row b of the activations is request b's), one step of
   the recurrence from the request's state slot, with q, k, v, g, beta formed
   exactly as in the verify:
     c = beta (v - S diag(e^g) k_hat),  S' = S diag(e^g) + c k_hat^T,
     out = S' q.
   The new state goes to the final slot (NULL: in place); with the fused conv,
   the newest three raw inputs go to entries [0, 3) of the final slot's conv
   state, other entries stay.  A request whose state slot is null gets +0.0
   outputs and nothing else; one whose final slot alone is null gets its output
   and no state. */
typedef struct {
  kda_tensor mixed_qkv;    /* act [B, 3HD] */
  kda_tensor raw_gate;     /* act [B, HD] */
  kda_tensor raw_beta;     /* act [B, H] */
  kda_tensor A_log;        /* as kda_verify_args, down to state */
  kda_tensor dt_bias;
  kda_tensor state;
  kda_tensor out;          /* F32 or act [B, HD] */
  kda_tensor conv_state;
  kda_tensor conv_weight;
  const int32_t* state_indices;        /* [batch] */
  const int32_t* final_state_indices;  /* [batch] or NULL: in place */
  const int32_t* num_accepted_tokens;  /* [batch] conv history offset + 1,
                                          or NULL: 1 */
  int32_t batch;
  int32_t spec_query_len;  /* Q: the conv state holds Q + 2 entries */
  int32_t null_block_id;
  int32_t conv_dim_first;
  int32_t use_lower_bound;
  float lower_bound;
} kda_decode_args;

/* Arguments of kda_step_tables: the index arrays of one step, from request
   lengths.  Request b runs q_b = max(query_lens[b], 0) tokens after its
   c = max(num_computed_tokens[row], 0) computed ones, row =
   request_indices[b] (or b); one block holds block_size tokens, and block i
   of a request is block_table[row][i] (its state slot and its cache block).
   After the step a request holds the block of its next token, that is
   (c + q_b) / block_size + 1 blocks, at most the table's width; what
   num_blocks[row] lacks is taken from free_blocks in batch order and written
   to the row, the null id once the free blocks run out.  Then
     query_start_loc[b] = q_0 + .. + q_{b-1} (sums are held to max_tokens),
     state_indices[b]   = block of token c,
     initial_state_indices[b] = the same when c > 0, else the null id,
     final_state_indices[b] = block of token c + q_b,
   (the null id past the width), and for token t of request b, in token order,
     positions[t]    = c + t - query_start_loc[b],
     slot_mapping[t] = block * block_size + position % block_size,
   -1 where the block is null; behind the last token, up to max_tokens,
   positions are 0 and slots -1.  A request whose row is outside
   [0, num_request_rows) runs its tokens with null blocks.  Two requests of
   a launch must not name the same row. */
typedef struct {
  const int32_t* query_lens;           /* [batch] */
  const int32_t* num_computed_tokens;  /* per request row */
  const int32_t* num_blocks;           /* per request row: blocks held */
  const int32_t* request_indices;      /* [batch] or NULL: row = b */
  const int32_t* free_blocks;          /* [num_free] */
  int32_t* block_table;                /* [num_request_rows, width] */
  int64_t block_table_strides[2];      /* row, column (elements) */
  int32_t batch;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t block_size;
  int32_t num_free;
  int32_t max_tokens;                  /* size of positions, slot_mapping */
  int32_t null_block_id;
  int32_t pad_;
  int32_t* query_start_loc;            /* [batch + 1] outputs from here on */
  int32_t* new_num_blocks;             /* per request row, written for the
                                          batch's rows: live blocks held;
                                          may be num_blocks itself */
  int32_t* state_indices;              /* [batch] */
  int32_t* initial_state_indices;      /* [batch] */
  int32_t* final_state_indices;        /* [batch] */
  int32_t* positions;                  /* [max_tokens] */
  int64_t* slot_mapping;               /* [max_tokens] */
  int32_t* num_allocated;              /* [1] blocks the step asked for; over
                                          num_free when they ran out */
} kda_tables_args;

/* Arguments of kda_sample.  For each row x of logits (V values), with the
   parameters of its request (row m belongs to the request b with
   query_start_loc[b] <= m < query_start_loc[b+1]; without query_start_loc,
   b = m), over the order of falling x, ties by rising index:
     w_i = exp((x_i - max x) / temperature);
     the longest prefix with every w_i >= min_p and at most top_k tokens is
     kept, then its shortest prefix with at least top_p of its mass;
     token = the lowest kept i with sum of w_j over kept j <= i  >  u * mass,
   u = uniform[m].  temperature <= 0: the lowest index of the maximum.
   top_k <= 0, top_p >= 1, min_p <= 0, NaN parameters and NULL arrays leave
   their filter (or temperature 1) out; top_p <= 0 keeps one token; u is
   held to [0, 1 - 2^-24] (NaN: 0).  NaN logits count as -inf; a row without
   any value above -inf gives token -1.  Each w is rounded to 46 binary places
   (62 - ceil(log2 V) where that is fewer; formed in fp64, so that one next to
   the middle of two may go to either) and summed as an integer: no order of
   additions changes a token.  V up to 2^20.
   Rows before query_start_loc[0] or from query_start_loc[batch] on are not
   touched.
   Acceptance (draft_tokens given): request b's window holds the tokens
   draft_tokens[s .. e) (s, e from query_start_loc); row m's token is checked
   against draft_tokens[m + 1], and num_accepted[b] = 1 + the number of
   leading matches, in [1, e - s] (0 for an empty window): what
   kda_commit_plan takes as num_accepted_tokens (with request_indices it reads
   that array by request row, this one is in batch order).  next_tokens[b] is
   the token of row s + num_accepted[b] - 1 (-1 for an empty window). */
typedef struct {
  kda_tensor logits;              /* F32 or BF16 [M, V], rows contiguous */
  const float* uniform;           /* [M] */
  const float* temperature;       /* [batch] each, or NULL */
  const int32_t* top_k;
  const float* top_p;
  const float* min_p;
  const int32_t* query_start_loc; /* [batch + 1], or NULL: batch = M */
  const int32_t* draft_tokens;    /* [M] or NULL */
  int32_t* tokens;                /* [M] output */
  int32_t* num_accepted;          /* [batch] outputs, given iff draft_tokens */
  int32_t* next_tokens;
  void* workspace;                /* device, 16-byte aligned, at least
                                     kda_sample_workspace_size(M, V) bytes;
                                     not shared by launches in flight
                                     together */
  int64_t workspace_bytes;
  int32_t batch;
  int32_t pad_;
} kda_sample_args;

/* Arguments of kda_latent_write: token t's latent and rope key go to place
   slot_mapping[t] of a paged cache (block slot / block_size, token slot %
   block_size of it, as kda_step_tables numbers them), bit for bit.  R = latent
   dim, P = rope dim.  A slot in a block <= null_block_id or past the cache
   writes nothing.  Two tokens must not name the same slot. */
typedef struct {
  kda_tensor latent;             /* act [T, R] */
  kda_tensor rope_key;           /* act [T, P]; empty for P = 0 */
  kda_tensor cache;              /* act [N, block_size, R + P] */
  const int64_t* slot_mapping;   /* [T] */
  int32_t null_block_id;
  int32_t pad_;
} kda_latent_write_args;

/* Arguments of kda_latent_attention: attention in latent space (the absorbed
   form) over a paged cache.  Token t of request b (its rows follow
   query_start_loc, clamped to [0, T]) stands at position c + i, c =
   max(num_computed_tokens[row], 0), i = t - query_start_loc[b], row =
   request_indices[b] (or b), and sees the cache entries e_j = (c_j | r_j) of
   positions j = 0 .. c + i, its own included (kda_latent_write comes first):
     s_j = softmax_scale * q_th . e_j,   p = softmax over j,
     out_th = sum_j p_j c_j,             lse_th = ln sum_j e^(s_j).
   Position j lies in block block_table[row][j / block_size]; positions of a
   null block (<= null_block_id or >= N) or past the table's width are not
   seen.  A query that sees nothing, or whose row is outside
   [0, num_request_rows), gets +0.0 outputs and lse -inf.  An entry that is not
   finite reaches the queries that see it, no others.  Arithmetic is fp32; with
   bf16 a weight p weighs the latents as two bf16 values, off by 2^-15 of it at
   most.  Token rows outside all requests are not touched. */
typedef struct {
  kda_tensor q;                  /* act [T, H, R + P] */
  kda_tensor cache;              /* act [N, block_size, R + P]; R is 128, 256
                                    or 512, P is 0 or 64 */
  kda_tensor out;                /* act [T, H, R] */
  kda_tensor lse;                /* F32 [T, H], or empty */
  const int32_t* query_start_loc;      /* [batch + 1], not decreasing */
  const int32_t* num_computed_tokens;  /* per request row */
  const int32_t* request_indices;      /* [batch] or NULL: row = b */
  const int32_t* block_table;          /* [num_request_rows, width] */
  int64_t block_table_strides[2];      /* row, column (elements) */
  void* workspace;               /* device, 16-byte aligned, at least
                                    kda_latent_attention_workspace_size(...)
                                    bytes; not shared by launches in flight
                                    together */
  int64_t workspace_bytes;
  int32_t batch;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t null_block_id;
  float softmax_scale;           /* finite */
  int32_t pad_;
} kda_latent_args;

/* Arguments of kda_latent_expand: keys and values of every head from cached
   latents.  Request b's key rows key_start_loc[b] .. key_start_loc[b + 1]
   (clamped to [0, S]; not decreasing) are its positions 0, 1, ..; for the
   entry (c_j | r_j) of such a position,
     key[s, h] = W_h[0 .. D) c_j,  value[s, h] = W_h[D .. 2D) c_j,
     rope_key[s] = r_j,
   with fp32 sums, rounded once.  Positions of null blocks, past the block
   table or of rows outside [0, num_request_rows) give +0.0.  Rows outside all
   requests are not touched. */
typedef struct {
  kda_tensor cache;              /* act [N, block_size, R + P]; R is 128, 256
                                    or 512, P a multiple of 16 bytes */
  kda_tensor weight;             /* act [H, 2 D, R] */
  kda_tensor key;                /* act [S, H, D]; D is 64 or 128 */
  kda_tensor rope_key;           /* act [S, P], or empty: not gathered */
  kda_tensor value;              /* act [S, H, D] */
  const int32_t* key_start_loc;  /* [batch + 1] */
  const int32_t* request_indices;      /* [batch] or NULL: row = b */
  const int32_t* block_table;          /* [num_request_rows, width] */
  int64_t block_table_strides[2];      /* row, column (elements) */
  int32_t batch;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t null_block_id;
} kda_latent_expand_args;

/* Arguments of kda_latent_prefill: causal attention with a key and a value
   for every head and one rope key for all of them.  Request b has the queries
   query_start_loc[b] .. query_start_loc[b + 1] (clamped to [0, T]) and the
   keys key_start_loc[b] .. key_start_loc[b + 1] (clamped to [0, S]); the
   queries stand at its last positions: query i of n_q sees the keys j <= n_k -
   n_q + i,
     s_j = softmax_scale * (q_th[0 .. D) . key[j, h] + q_th[D ..) . rope[j]),
     out_th = sum_j softmax(s)_j value[j, h],  lse_th = ln sum_j e^(s_j).
   A query without keys (n_k < n_q) gets +0.0 outputs and lse -inf.  A key or
   value that is not finite reaches the queries that see it, no others.
   Arithmetic is fp32; with bf16 a weight weighs the values as two bf16 values,
   off by 2^-15 of it at most.  Token rows outside all requests are not
   touched. */
typedef struct {
  kda_tensor q;                  /* act [T, H, D + P]; D 64 or 128, P 0 or 64 */
  kda_tensor key;                /* act [S, H, D] */
  kda_tensor rope_key;           /* act [S, P]; empty for P = 0 */
  kda_tensor value;              /* act [S, H, D] */
  kda_tensor out;                /* act [T, H, D] */
  kda_tensor lse;                /* F32 [T, H], or empty */
  const int32_t* query_start_loc;  /* [batch + 1], not decreasing, both */
  const int32_t* key_start_loc;
  int32_t batch;
  float softmax_scale;           /* finite */
} kda_latent_prefill_args;

/* Arguments of kda_adjust_logits: logits changed in place, before kda_sample.
   For the entry x of token v in row m, which belongs to request b as in
   kda_sample:
     y = x + bias (the last entry of b's list that names v, if one does);
     v seen:     y = y / r where y > 0, else y * r;
     count > 0:  y = y - frequency_penalty * count - presence_penalty;
     v not allowed by m's grammar mask: y = -inf.
   A history is row request_indices[b] (or b) of token_ids, its first
   token_lens[row] entries (held to [0, max_len]); the first
   prompt_lens[row] of them are the prompt.  A token is seen if it is among
   them, and its count is how often it occurs behind the prompt.  With
   draft_tokens, row m of the window that starts at s also counts (and has
   seen) draft_tokens[s + 1 .. m]; draft_tokens[s] is the history's last token.
   r <= 0, NaN parameters and NULL arrays leave their change out; a request
   without a row of token_ids (NULL, or outside [0, num_request_rows)) has an
   empty history.  Tokens outside [0, V) are ignored.  Arithmetic is fp32,
   rounded once.  Entries that nothing changes keep their bits; rows that belong
   to no request are not touched.  V is at most 2^20, batch 65535 and M 2^31 -
   64.
   A mask row holds a bit for each token, bit v % 32 of word v / 32, 1 =
   allowed; row m's is mask_rows[m] (NULL: m), outside [0, num_masks): none. */
typedef struct {
  kda_tensor logits;               /* F32 or BF16 [M, V], rows contiguous */
  const int32_t* query_start_loc;  /* [batch + 1], or NULL: batch = M */
  const int32_t* draft_tokens;     /* [M] or NULL */
  const int32_t* request_indices;  /* [batch] or NULL: row = b */
  const int32_t* token_ids;        /* [num_request_rows, max_len] or NULL */
  int64_t token_ids_stride;        /* of a row; columns are contiguous */
  const int32_t* prompt_lens;      /* per request row */
  const int32_t* token_lens;       /* per request row */
  const float* repetition_penalty; /* [batch] each, or NULL */
  const float* frequency_penalty;
  const float* presence_penalty;
  const int32_t* bias_start;       /* [batch + 1] or NULL, not decreasing */
  const int32_t* bias_tokens;      /* [num_biases] */
  const float* bias_values;        /* [num_biases] */
  const int32_t* mask;             /* [num_masks, >= ceil(V / 32)] or NULL */
  int64_t mask_stride;             /* of a row; words are contiguous */
  const int32_t* mask_rows;        /* [M] or NULL */
  int32_t batch;
  int32_t num_request_rows;
  int32_t max_len;
  int32_t num_biases;
  int32_t num_masks;
  int32_t pad_;
} kda_logits_args;

/* Arguments of kda_copy_blocks: for each pair (source, destination) and every
   pool (a layer's state, conv state or cache; block i lies at base + i *
   stride), the block's bytes copied bit for bit.  A pair with a null id
   (<= null_block_id or >= num_blocks) or with source = destination copies
   nothing.  A destination must not be another pair's source or destination. */
typedef struct {
  const int64_t* tables;         /* device int64 [3][num_pools]: base byte
                                    addresses, block strides and block sizes
                                    in bytes */
  const int64_t* host_tables;    /* optional HOST copy, for the checks and the
                                    launch's size */
  const int32_t* copy_pairs;     /* device [max_pairs][2] */
  const int32_t* num_pairs;      /* device [1] or NULL: max_pairs; held to
                                    [0, max_pairs] */
  int64_t num_blocks;            /* N of every pool */
  int32_t num_pools;
  int32_t max_pairs;
  int32_t null_block_id;
  int32_t pad_;
} kda_copy_args;

/* Arguments of kda_fork_blocks: request rows that continue another row's
   tokens.  Fork f makes child row b = child_rows[f] hold the first c =
   max(num_computed_tokens[a], 0) tokens of parent row a = parent_rows[f]:
     blocks 0 .. k - 1, k = c / block_size, are the parent's (shared),
     block k, which the next token goes to and which holds the running state,
     is taken from free_blocks in the order of the forks (the null id once
     they run out),
     copy_pairs[f] = (the parent's block k, the new one) for kda_copy_blocks,
     num_computed_tokens[b] = c, num_blocks[b] = k + 1 (at most the width).
   A pair is (null, null) where the parent does not hold block k or there is
   no new block.  Where k is past the table (a request at its full length)
   the fork shares the table's blocks and takes none.  A fork with a row
   outside [0, num_request_rows) or with a = b does nothing and takes none.
   Entries of the child's row behind block k stay.  A child row must not be
   another fork's row; a parent may have many forks.  num_forks is below
   2^24. */
typedef struct {
  const int32_t* parent_rows;    /* [num_forks] */
  const int32_t* child_rows;     /* [num_forks] */
  int32_t* num_computed_tokens;  /* per request row, read and written */
  int32_t* num_blocks;           /* per request row, read and written */
  int32_t* block_table;          /* [num_request_rows, width], as well */
  int64_t block_table_strides[2];      /* row, column (elements) */
  const int32_t* free_blocks;    /* [num_free] */
  int32_t* copy_pairs;           /* [num_forks][2] output */
  int32_t* num_allocated;        /* [1] output: blocks the forks asked for, 0
                                    without forks (which may leave it NULL) */
  int32_t num_forks;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t block_size;
  int32_t num_free;
  int32_t null_block_id;
} kda_fork_args;

/* Arguments of kda_free_blocks: rows released, references counted anew, free
   blocks listed.
     new_num_blocks[r] = 0 for released rows, else num_blocks[r] held to
     [0, width] (may be num_blocks itself);
     ref_counts[i] = pinned[i] (0 where negative; NULL: 0) + how often the rows
     hold block i (their first new_num_blocks entries; null ids are none);
     free_blocks = the blocks i > null_block_id with no reference, in rising
     order, null ids behind them up to N;  num_free = how many they are.
   `pinned` is by block id, and follows the moves of kda_compact_blocks only
   where its holder moves it.
   Released rows outside [0, num_request_rows) are ignored; one may be named
   twice.  N is at most 2^28, num_request_rows below 2^24. */
typedef struct {
  const int32_t* released_rows;  /* [num_released] */
  const int32_t* block_table;    /* [num_request_rows, width] */
  int64_t block_table_strides[2];      /* row, column (elements) */
  const int32_t* num_blocks;     /* per request row: entries held */
  const int32_t* pinned;         /* [N] references of other holders, or NULL */
  int32_t* new_num_blocks;       /* per request row; outputs from here on */
  int32_t* ref_counts;           /* [N] */
  int32_t* free_blocks;          /* [N] */
  int32_t* num_free;             /* [1] */
  void* workspace;               /* kda_blocks_workspace_size(N) bytes, 4-byte
                                    aligned */
  int64_t workspace_bytes;
  int32_t num_released;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t total_blocks;          /* N */
  int32_t null_block_id;
  int32_t pad_;
} kda_free_args;

/* Arguments of kda_compact_blocks: live blocks (ref_counts > 0) moved to the
   lowest ids behind the null one.  With n live blocks, those above
   null_block_id + n move, in rising order, to the free ids up to there, in
   rising order:
     copy_pairs lists the moves (kda_copy_blocks makes them), null pairs
     behind them;  num_pairs = how many (of more than max_pairs moves the
     first max_pairs are made; N / 2 are always enough);
     new_block_table is the block table with the new ids in the first
     num_blocks[r] entries of each row, other entries as they were (may be
     block_table itself);
     new_ref_counts the counts by new id (may be ref_counts itself).
   Blocks that kda_free_blocks found pinned move as the others do: whoever holds
   ids outside the block table puts destinations for sources in them, and moves
   the entries of `pinned` likewise, before the next kda_free_blocks.
   With all moves made, the free blocks are null_block_id + n + 1 .. N - 1.
   Limits as in kda_free_args. */
typedef struct {
  const int32_t* ref_counts;     /* [N] */
  const int32_t* block_table;    /* [num_request_rows, width] */
  int64_t block_table_strides[2];      /* row, column (elements) */
  const int32_t* num_blocks;     /* per request row: entries held */
  int32_t* new_block_table;      /* outputs from here on */
  int64_t new_block_table_strides[2];
  int32_t* new_ref_counts;       /* [N] */
  int32_t* copy_pairs;           /* [max_pairs][2] */
  int32_t* num_pairs;            /* [1] */
  void* workspace;               /* kda_blocks_workspace_size(N) bytes, 4-byte
                                    aligned */
  int64_t workspace_bytes;
  int32_t max_pairs;
  int32_t num_request_rows;
  int32_t block_table_width;
  int32_t total_blocks;          /* N */
  int32_t null_block_id;
  int32_t pad_;
} kda_compact_blocks_args;

/* Library ABI version (KDA_ABI_VERSION). */
int kda_abi_version(void);

/* Message of the last failing call in this thread ("" if none). */
const char* kda_last_error(void);

/* Name of a status code. */
const char* kda_status_string(int status);

/* Host-only validation of verify arguments: shapes, dtypes, strides,
   alignment and supported sizes.  Reads no device memory, launches nothing.
   (kernels page `_check_layouts`, `can_use_cute_recoverssm`; ops page
   `kda_recoverssm_verify`.) */
int kda_check_verify(const kda_verify_args* args);

/* Validate, then launch the fused conv update + speculative verify on
   `stream`.  Writes out, correction/key_gate records of the written
   positions, and the rolled conv state; leaves state and every other byte
   unchanged; null requests get +0.0 outputs and nothing else. */
int kda_conv_update_verify(const kda_verify_args* args, void* stream);

/* kda_conv_update_verify for callers that cannot allocate device memory
   (code under HIP graph capture, tight serving loops, harnesses that forbid
   allocation): the same checks, kernels and results, except that the work
   counters (the ticket counter, and the V-tile schedule's arrival counters)
   live in a scratch array of the library instead of args->work_counter,
   which is ignored.  The array holds 1 + 65536 int32 per GPU, is looked up
   (and cleared by a kernel on `stream`) on the first call on each device,
   and is kept until the process ends.  Every launch leaves it at zero, but
   it is shared: calls that overlap on one GPU (two streams, or two threads)
   race on it.  A V-tile launch of more than 65536 (request, head) items is
   refused with KDA_E_CAPACITY before any device call.  Allocates nothing. */
int kda_conv_update_verify_noalloc(const kda_verify_args* args, void* stream);

/* The unfused verify (ops page, `kda_recoverssm_verify` and
   `_kda_recoverssm_verify_kernel`): the same as kda_conv_update_verify
   except that mixed_qkv [T, 3HD] already holds the convolved q | k | v
   (the three column blocks, channel = part*H*D + h*D + d) and the key
   record stores that k as given.  conv_state, conv_weight and
   num_accepted_tokens are not used (they may be empty / NULL). */
int kda_check_verify_qkv(const kda_verify_args* args);
int kda_recoverssm_verify_qkv(const kda_verify_args* args, void* stream);

/* Host-only validation of commit arguments (ops page
   `KDARecoverSSMCommitContext.create` and `.commit`). */
int kda_check_commit(const kda_commit_args* args);

/* Validate, then launch the multi-layer commit on `stream`: for every layer
   and request with a non-null source slot, a non-null final slot, a valid
   record row and n = commit length > 0, the checkpoint of every head
   becomes S_n = S_0 * prod_t diag(exp g_t) + sum_t c_t k_hat_t^T
   * prod_{s>t} diag(exp g_s) over t < n, stored at the final slot. */
int kda_recoverssm_commit(const kda_commit_args* args, void* stream);

/* Host-only validation of the plan arguments, then its launch on `stream`
   (one thread per request; writes only the four output arrays). */
int kda_check_commit_plan(const kda_plan_args* args);
int kda_commit_plan(const kda_plan_args* args, void* stream);

/* Host-only validation of the compaction arguments, then its launch on
   `stream` (one thread per layer, request and channel). */
int kda_check_compact_conv(const kda_compact_args* args);
int kda_compact_conv_state(const kda_compact_args* args, void* stream);

/* The whole of the ops page's `KDARecoverSSMCommitContext.commit` in one
   launch: the results of kda_commit_plan(plan), then, when `compact` is not
   NULL, kda_compact_conv_state(compact), then kda_recoverssm_commit(commit),
   bit for bit.  Every (layer, request, head) workgroup of the commit plans
   its request itself (the layer-0, head-0 one writes the plan's four
   outputs) and copies that head's conv histories (its q, k and v channels)
   before its state fold.
   The three blocks must describe the calls the separate path would make:
   one batch, window and null id; the commit's state_indices, commit_lens
   and final_state_indices (and, iff the plan has a block table, its
   boundary pair) are the plan's state_indices and output pointers, and so
   are the compaction's; the compaction covers the commit's layers and slot
   count with conv_dim = 3 * num_heads * head_dim.  Otherwise KDA_E_ARG.
   The plan's output arrays are written, never read, by the launch.  The
   slot rules of the separate calls hold: no request's final or boundary
   slot is another request's source or destination. */
int kda_check_commit_step(const kda_commit_args* commit,
                          const kda_plan_args* plan,
                          const kda_compact_args* compact);
int kda_recoverssm_commit_step(const kda_commit_args* commit,
                               const kda_plan_args* plan,
                               const kda_compact_args* compact,
                               void* stream);

/* Of the calls below, no output may share memory with an input, except where
   an argument says so (states and conv states of one slot, num_blocks).  The
   squares of a head's q and k are summed in fp32. */

/* Bytes of workspace that a prefill of `tokens` rows and `batch` requests
   needs (0 for sizes that the checks refuse); the activation dtype is
   act_dtype, out's is out_dtype (kda_dtype). */
int64_t kda_prefill_workspace_size(int64_t tokens, int64_t batch,
                                   int64_t num_heads, int64_t head_dim,
                                   int32_t act_dtype, int32_t out_dtype);

/* Host-only validation of prefill arguments, then the launches (two kernels
   on `stream`): with the fused short convolution, or on convolved q|k|v
   (conv_state, conv_weight and num_accepted_tokens are then not used).  A
   request's state slot must not be another request's state or initial
   slot. */
int kda_check_prefill(const kda_prefill_args* args);
int kda_conv_prefill(const kda_prefill_args* args, void* stream);
int kda_check_prefill_qkv(const kda_prefill_args* args);
int kda_prefill_qkv(const kda_prefill_args* args, void* stream);

/* Host-only validation of decode arguments, then the launch (one kernel).  A
   request's final slot must not be another request's state or final slot. */
int kda_check_decode(const kda_decode_args* args);
int kda_conv_update_decode(const kda_decode_args* args, void* stream);
int kda_check_decode_qkv(const kda_decode_args* args);
int kda_decode_qkv(const kda_decode_args* args, void* stream);

/* Host-only validation of the step tables' arguments, then the launches. */
int kda_check_step_tables(const kda_tables_args* args);
int kda_step_tables(const kda_tables_args* args, void* stream);

/* Bytes of workspace that sampling `rows` rows of `vocab` logits needs (0
   for sizes that the checks refuse). */
int64_t kda_sample_workspace_size(int64_t rows, int64_t vocab);

/* Host-only validation of the sampling arguments, then the launches. */
int kda_check_sample(const kda_sample_args* args);
int kda_sample(const kda_sample_args* args, void* stream);

/* Host-only validation of the cache write's arguments, then its launch. */
int kda_check_latent_write(const kda_latent_write_args* args);
int kda_latent_write(const kda_latent_write_args* args, void* stream);

/* Bytes of workspace of a latent attention over `tokens` rows of `batch`
   requests (0 for sizes that the checks refuse); act_dtype a kda_dtype. */
int64_t kda_latent_attention_workspace_size(int64_t tokens, int64_t batch,
                                            int64_t num_heads,
                                            int64_t latent_dim,
                                            int64_t rope_dim,
                                            int32_t act_dtype);

/* Host-only validation of the latent attention's arguments, then the
   launches (two kernels). */
int kda_check_latent_attention(const kda_latent_args* args);
int kda_latent_attention(const kda_latent_args* args, void* stream);

/* Host-only validation of the expansion's arguments, then its launch. */
int kda_check_latent_expand(const kda_latent_expand_args* args);
int kda_latent_expand(const kda_latent_expand_args* args, void* stream);

/* Host-only validation of the prompt attention's arguments, then its
   launch. */
int kda_check_latent_prefill(const kda_latent_prefill_args* args);
int kda_latent_prefill(const kda_latent_prefill_args* args, void* stream);

/* Host-only validation of the logits' changes, then their launch. */
int kda_check_adjust_logits(const kda_logits_args* args);
int kda_adjust_logits(const kda_logits_args* args, void* stream);

/* Host-only validation of the block operators' arguments, then their launches
   (copies and forks one kernel, the other two several).  The workspace of the
   last two is scratch memory for `total_blocks` blocks (0 for sizes that the
   checks refuse), not shared by launches in flight together. */
int kda_check_copy_blocks(const kda_copy_args* args);
int kda_copy_blocks(const kda_copy_args* args, void* stream);
int kda_check_fork_blocks(const kda_fork_args* args);
int kda_fork_blocks(const kda_fork_args* args, void* stream);
int64_t kda_blocks_workspace_size(int64_t total_blocks);
int kda_check_free_blocks(const kda_free_args* args);
int kda_free_blocks(const kda_free_args* args, void* stream);
int kda_check_compact_blocks(const kda_compact_blocks_args* args);
int kda_compact_blocks(const kda_compact_blocks_args* args, void* stream);

/* Launch a one-workgroup kernel that sets counter[0..n) to 0 on `stream`
   (for a counter left non-zero by an aborted launch).  Uses no memset
   node, so it may be captured in a graph. */
int kda_reset_counter(int32_t* counter, int32_t n, void* stream);

/* Kernel timing without a profiler, for callers that measure each kernel's
   own duration (an event recorded on the stream around a launch also counts
   the gap the event's own marker adds before the next dispatch).  Arms the
   calling thread: the next `launches` kernels that library calls on this
   thread launch (a prefill takes two, the step tables two or, without
   tokens, one, sampling three to eight, the latent attention two, the
   changes of logits one to three (masks one for each 65535 rows), free lists
   and compactions one to five, the other operators on caches and blocks one) are dispatched with hipExtLaunchKernel, `start_event` (a hipEvent_t,
   may be NULL) recording the start of the first of them and `stop_event` (may
   be NULL) the end of the last.  The counter-clearing kernels
   (kda_reset_counter, the first use of the no-allocation entry point's array
   on a device) are not counted.  launches = 0 disarms.  If `pending` is not NULL it receives
   the number of launches the previous arming was still waiting for (0 when
   every armed launch happened, so its stop event was recorded).  The
   events stay the caller's; do not arm the thread while it captures a
   graph.  KDA_E_ARG if launches < 0 (the previous arming is then kept). */
int kda_set_launch_events(void* start_event, void* stop_event,
                          int32_t launches, int32_t* pending);

#ifdef __cplusplus
}
#endif
#endif /* KDA_RECOVERSSM_H */
