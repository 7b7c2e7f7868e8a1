/*
 * dflash_attn.h -- C ABI of the GB300 DFlash draft attention library
 * (libdflash_attn.so).
 *
 * One draft attention layer of a DFlash block-diffusion drafter
 * (Qwen3DFlashAttention): queries from a block of noise tokens (one anchor
 * plus mask tokens), keys and values from the projected target-model context
 * followed by the block, per-head q/k RMSNorm, RoPE over the
 * [context | block] window, grouped KV heads, non-causal softmax (optionally
 * a symmetric sliding-window band), o_proj, and a draft KV cache that is
 * cropped back to the accepted prefix after verification.  Around it: the
 * context K/V of several layers from one projection, the rest of the draft
 * decoder layer (norms, residual stream, SwiGLU MLP), a paged cache with a
 * slot mapping and block tables, causal layers, the attention core of
 * the packed training layout with its backward, and what training needs
 * around it (head norm and rotation, the head's loss, clipping).
 *
 * Page citations name the page by title and the section or symbol on it:
 *   [P3] "DFlash源码导读（二）：Qwen3DFlashAttention注意力实现全解析"
 *   [P4] "nemo_automodel.components.speculative.dflash.draft_qwen3"
 *   [P5] "vllm.model_executor.models.qwen3_dflash"
 *
 * Conventions for every call:
 *  - Every entry point returns an int status: DFLASH_OK (0) or a negative
 *    DFLASH_ERR_* code; dflash_last_error() then returns a message for the
 *    calling thread.  No C++ exception crosses this boundary.
 *  - Arguments are checked on the host before anything is enqueued.  A call
 *    that fails a check enqueues no work and leaves every object unchanged.
 *  - "device" pointers are CUDA device memory of the device that was current
 *    when the layer was created; "host" pointers are ordinary CPU memory that
 *    is read only during the call.  The caller owns every pointer it passes.
 *    Device tensors handed to a bf16 layer must start on a 16-byte boundary.
 *  - Tensors are dense, row-major, in the layer's dtype (DFLASH_BF16 or
 *    DFLASH_FP32) unless stated otherwise; integer tensors are int32.
 *  - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *    stream) and runs asynchronously; outputs are valid once the stream has
 *    reached that point.
 *  - Handles are not thread-safe: one thread (or external locking) per layer
 *    handle and per cache at a time.  One layer's calls share its scratch, so
 *    calls of one layer must not run concurrently on different streams.
 *  - Faults found on the device (a position outside [0, max_position), an
 *    anchor outside [0, seq], a paged-cache slot or block-table entry outside
 *    the cache, a bounded wait that ran out) do not stop the kernels: the
 *    offending value is clamped or the access skipped, a code is recorded in
 *    the layer's device error word, and dflash_device_error() reports it.
 */
#ifndef DFLASH_ATTN_H
#define DFLASH_ATTN_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct dflash_attn dflash_attn;   /* one layer: weights + scratch */
typedef struct dflash_cache dflash_cache; /* one draft KV cache */
typedef struct dflash_kv_group dflash_kv_group; /* context K/V of several layers */
typedef struct dflash_mlp dflash_mlp;     /* norms + MLP of a decoder layer */
typedef struct dflash_paged_cache dflash_paged_cache; /* paged KV storage */
typedef struct dflash_q8_cache dflash_q8_cache; /* draft KV cache in 8 bits */
typedef void* dflash_stream;              /* a cudaStream_t */

enum {
  DFLASH_OK = 0,
  DFLASH_ERR_ARG = -1,         /* null pointer, bad enum, non-positive size  */
  DFLASH_ERR_SHAPE = -2,       /* sizes inconsistent with the layer/cache    */
  DFLASH_ERR_CAPACITY = -3,    /* cache rows would exceed its capacity       */
  DFLASH_ERR_RANGE = -4,       /* crop length above the current length, ...  */
  DFLASH_ERR_CUDA = -5,        /* a CUDA runtime call failed                 */
  DFLASH_ERR_DEVICE = -6,      /* a kernel recorded a device-side fault      */
  DFLASH_ERR_UNSUPPORTED = -7, /* valid request the library does not handle */
  DFLASH_ERR_MEMORY = -8       /* device allocation failed                   */
};

enum { DFLASH_BF16 = 0, DFLASH_FP32 = 1 };

/* Device-side fault codes reported by dflash_device_error(). */
enum {
  DFLASH_DEV_OK = 0,
  DFLASH_DEV_WAIT_TIMEOUT = 1, /* a pipeline wait gave up (kernel returned)  */
  DFLASH_DEV_POSITION = 2,     /* position outside [0, max_position)         */
  DFLASH_DEV_ANCHOR = 3,       /* anchor outside [0, seq]                    */
  DFLASH_DEV_SLOT = 4          /* paged cache: a slot outside the cache (the
                                  row was not written), or a block-table entry
                                  of a page holding the sequence's keys outside
                                  the cache (page 0 read in its place)        */
};

/* Layer scalars.  [P3] step 1: head_dim is the explicit value, else
 * hidden / n_heads; num_key_value_groups = n_heads / n_kv_heads.
 * [P4] Qwen3DFlashAttention: scaling = head_dim^-0.5; sliding_window only on
 * sliding-attention layers ([P3] step 5).  [P5] DFlashQwen3Model: fc takes
 * n_target_layers * hidden concatenated features. */
typedef struct {
  int32_t hidden;          /* H                                              */
  int32_t n_heads;         /* query heads                                    */
  int32_t n_kv_heads;      /* key/value heads; divides n_heads               */
  int32_t head_dim;        /* d; 0 -> hidden / n_heads                       */
  int32_t n_target_layers; /* fc input width = n_target_layers * hidden; 0 = no fc */
  float rms_eps;           /* eps of q_norm, k_norm and hidden_norm          */
  float rope_theta;        /* RoPE base                                      */
  int32_t sliding_window;  /* 0 = full attention; W > 0 keeps keys with
                              |query key index - key index| < W ([P4]
                              _sliding_window_mask)                          */
  int32_t max_position;    /* positions must lie in [0, max_position);
                              0 -> 131072                                    */
  int32_t dtype;           /* DFLASH_BF16 or DFLASH_FP32                     */
  int32_t causal;          /* 1: block row t sees the keys at or before its
                              own key index (every cached and context row,
                              block rows 0..t), with the band on sliding
                              layers ([P5] _dflash_layer_causal); 0: the
                              block is bidirectional.  Inference only: the
                              packed training forward is _UNSUPPORTED on a
                              causal layer                                   */
} dflash_attn_config;

/* Message for the last failed call on this thread ("" if none). */
const char* dflash_last_error(void);

/* ABI version of this header (major * 100 + minor): 105. */
int dflash_abi_version(void);

/* Create one layer on the current CUDA device.
 * [P4] Qwen3DFlashAttention members q_proj, k_proj, v_proj, o_proj, q_norm,
 * k_norm; [P5] DFlashQwen3Attention (no biases); [P5] DFlashQwen3Model fc and
 * hidden_norm.
 *   wq [n_heads*d, H], wk [n_kv*d, H], wv [n_kv*d, H], wo [H, n_heads*d],
 *   q_norm_w [d], k_norm_w [d], fc_w [H, n_target_layers*H] (may be NULL when
 *   n_target_layers == 0), hidden_norm_w [H] (NULL iff fc_w is NULL).
 * All are device pointers in cfg->dtype, nn.Linear [out, in] layout.  They
 * are copied into library-owned memory before the call returns; the caller
 * may free them afterwards.
 * Errors: _ARG (null out/weights, bad dtype), _SHAPE (non-positive sizes,
 * n_heads % n_kv_heads != 0, odd head_dim; bf16 layers need head_dim 128 and
 * hidden % 128 == 0), _CUDA, _MEMORY.  On error *out is set to NULL. */
int dflash_attn_create(const dflash_attn_config* cfg, const void* wq,
                       const void* wk, const void* wv, const void* wo,
                       const void* q_norm_w, const void* k_norm_w,
                       const void* fc_w, const void* hidden_norm_w,
                       dflash_attn** out);

/* Free the layer and its scratch.  Waits for the device to finish the
 * layer's outstanding work.  NULL is accepted (no-op). */
int dflash_attn_destroy(dflash_attn* attn);

/* Optional: size the layer's scratch for calls up to these sizes now, so
 * that later calls of at most that size allocate nothing.
 * Scratch that a dflash_attn_forward, _paged or _q8 captured into a CUDA graph
 * uses stays allocated until the layer is destroyed, also when a larger call
 * later needs more.
 * max_rows = largest (batch*q_len + total new context rows) of a forward, or
 * rows of a ctx_project; max_keys = largest total key rows of one sequence;
 * max_batch = largest batch. */
int dflash_attn_reserve(dflash_attn* attn, int max_batch, int max_rows,
                        int max_keys);

/* Draft KV cache for `batch` sequences of up to `capacity_rows` rows each.
 * [P3] step 4 (DynamicCache update/crop).  Layout of the device storage:
 * K and V each [batch][n_kv_heads][capacity_rows][head_dim] in the layer
 * dtype; K rows are stored after k_norm and RoPE, V rows raw.  Lengths start
 * at 0 and are mirrored on the host.  The cache may be used with any layer
 * whose n_kv_heads, head_dim and dtype match the one given here. */
int dflash_cache_create(const dflash_attn* attn, int batch, int capacity_rows,
                        dflash_cache** out);
int dflash_cache_destroy(dflash_cache* cache);

/* Copy the current row counts into host_len[batch] (host memory). */
int dflash_cache_lengths(const dflash_cache* cache, int32_t* host_len);

/* Device pointers to the K and V storage (layout above), and the geometry.
 * For inspection and tests; writing through them is the caller's risk. */
int dflash_cache_data(const dflash_cache* cache, void** k, void** v,
                      int32_t* batch, int32_t* n_kv_heads,
                      int32_t* capacity_rows, int32_t* head_dim);

/* Copy the whole K and V storage (layout above) into caller device buffers
 * k_dst and v_dst, each batch*n_kv_heads*capacity_rows*head_dim elements,
 * on `stream`.  For inspection and tests. */
int dflash_cache_read(const dflash_cache* cache, void* k_dst, void* v_dst,
                      dflash_stream stream);

/* Crop each sequence b to its first host_keep[b] rows (host memory).
 * [P3] step 4: after verification the cache is cut back to the accepted
 * prefix.  No data moves: rows at or beyond the new length are dead and are
 * overwritten by the next append.  keep == len is a no-op.
 * Errors: _RANGE if any keep < 0 or keep > current length (nothing changes). */
int dflash_cache_crop(dflash_cache* cache, const int32_t* host_keep);

/* Context projection ([P3] 看懂注意力数据流; [P5] combine_hidden_states and
 * precompute_and_store_context_kv's hidden_norm):
 *   target_hidden = hidden_norm(fc(target_layers))
 * target_layers [rows, n_target_layers*H] and target_hidden [rows, H] are
 * device tensors.  rows may be 0 (nothing is enqueued).
 * Errors: _UNSUPPORTED if the layer has no fc, _ARG, _SHAPE. */
int dflash_ctx_project(dflash_attn* attn, const void* target_layers, int rows,
                       void* target_hidden, dflash_stream stream);

/* The same context projection as dflash_ctx_project, for callers that must
 * not have device memory allocated on their behalf.  The pages have no
 * counterpart: this is a property of this library, not of the method.
 * Who needs it: serving processes that fix all device memory at start-up
 * and treat any later allocation as a failure, and hosts whose memory pool
 * must be the only allocator on the GPU.  dflash_ctx_project may grow
 * layer-owned scratch with cudaMalloc; this entry point never allocates and
 * never frees.
 * Its scratch (the fp32 fc output, the split-K partial tiles and their
 * counters) lives in one fixed 16 MiB array inside the library's device
 * image, present on every GPU that loads the library until the process
 * exits.  The scratch a request needs is rows * H * 4 bytes for the fc
 * output plus the split-K tiles of the projection kernel the row count
 * selects: up to 384 rows that kernel needs no split-K tiles, from 385 rows
 * the persistent kernel may split K and then needs 128 KB per (tile, split).
 * At H = 4096 (fc 20480 -> 4096) that admits up to 384 rows and rejects
 * 385 and more.  A request above 16 MiB is rejected with
 * DFLASH_ERR_CAPACITY and enqueues nothing.
 * The first call on a device looks up the array's device address (which may
 * load the library's device code on that device): make that first call
 * before any stream capture.  Every call on a device shares the one array
 * and the array keeps the previous call's contents; the call clears the
 * parts that must start at zero on `stream` itself.  Calls whose work can
 * overlap on the GPU (different streams, or other threads) race on the
 * array: serialise them.  Arguments, layouts and other errors are those of
 * dflash_ctx_project; the layer's device must be the current device. */
int dflash_ctx_project_noalloc(dflash_attn* attn, const void* target_layers,
                               int rows, void* target_hidden,
                               dflash_stream stream);

/* One inference step of the layer for `batch` sequences.
 * [P3] steps 1-4 and 关键设计; [P4] Qwen3DFlashAttention.forward,
 * apply_rotary_pos_emb, _sliding_window_mask; [P5] DFlashQwen3Attention.forward.
 *   noise_hidden  device [batch, q_len, H]: the block embeddings
 *   target_hidden device [sum_b n_ctx[b], H]: new context rows, sequence-major
 *                 (may be NULL when every n_ctx is 0)
 *   host_n_ctx    host   [batch]: new context rows per sequence (>= 0)
 *   positions     device [sum_b (n_ctx[b] + q_len)]: per sequence its context
 *                 rows' positions, then the block's q_len positions
 *   out           device [batch, q_len, H]
 * For sequence b with L_b cached rows, the call appends n_ctx[b] context rows
 * and then the q_len block rows (K after k_norm + RoPE, V raw) at cache rows
 * L_b .. L_b + n_ctx[b] + q_len - 1, sets its length to that sum, and attends
 * every block query to all rows of the sequence (non-causal; on a layer with
 * sliding_window W only to keys whose index is within W of the query's index
 * L_b + n_ctx[b] + t).  The block rows stay in the cache until a crop.
 * Requires batch == cache batch <= 512; bf16 layers also need
 * (n_heads/n_kv_heads) * q_len <= 128.
 * Errors: _ARG, _SHAPE, _CAPACITY (L_b + n_ctx[b] + q_len > capacity; nothing
 * is appended for any sequence), _CUDA. */
int dflash_attn_forward(dflash_attn* attn, dflash_cache* cache, int batch,
                        int q_len, const void* noise_hidden,
                        const void* target_hidden, const int32_t* host_n_ctx,
                        const int32_t* positions, void* out,
                        dflash_stream stream);

/* Paged draft KV cache ([P5] precompute_and_store_context_kv: the context
 * K/V go into the layer's paged cache through do_kv_cache_update with a
 * slot_mapping; the draft's attention reads the pages through the batch's
 * block table).  Storage: K and V each [n_pages][n_kv_heads][page_size]
 * [head_dim] bf16, zeroed at creation; page p row r is slot p*page_size + r.
 * page_size is 16, 32, 64 or 128.  The cache holds no lengths: which pages
 * belong to which sequence, their order and each sequence's length are the
 * caller's (block table, slot mapping, host_len_before), so crop and
 * reuse are the caller's bookkeeping.  bf16 layers only (else _UNSUPPORTED).
 * dflash_paged_cache_data returns the storage and its geometry (for
 * inspection and tests; writing through it is the caller's risk);
 * dflash_paged_cache_read copies the whole K and V storage into caller
 * device buffers of n_pages*n_kv_heads*page_size*head_dim elements each, on
 * `stream`. */
int dflash_paged_cache_create(const dflash_attn* attn, int n_pages,
                              int page_size, dflash_paged_cache** out);
int dflash_paged_cache_destroy(dflash_paged_cache* cache);
int dflash_paged_cache_data(const dflash_paged_cache* cache, void** k,
                            void** v, int32_t* n_pages, int32_t* n_kv_heads,
                            int32_t* page_size, int32_t* head_dim);
int dflash_paged_cache_read(const dflash_paged_cache* cache, void* k_dst,
                            void* v_dst, dflash_stream stream);

/* dflash_attn_forward over a paged cache.  Arguments, outputs and errors are
 * those of dflash_attn_forward, with the cache replaced by:
 *   host_len_before host   [batch]: rows each sequence already holds
 *   slot_mapping    device [sum_b (n_ctx[b] + q_len)]: the slot each new
 *                   row's K and V are written to, in the order of positions
 *   block_table     device [batch][bt_stride]: sequence b's key row k lives
 *                   in page block_table[b][k / page_size], row k % page_size
 * The new rows of sequence b take key indices len_before[b] .. len_before[b]
 * + n_ctx[b] + q_len - 1; the call attends over indices 0 .. that end
 * through the block table.  The slots must be the ones the block table gives
 * for those indices (the kernels trust it).  A slot outside the cache skips
 * that row's write and records DFLASH_DEV_SLOT; a block-table entry outside
 * the cache for a page that holds keys of the sequence reads page 0 in its
 * place and records DFLASH_DEV_SLOT.  Block-table entries past a sequence's
 * last row may hold anything.
 * Errors: _ARG, _SHAPE, _UNSUPPORTED, _CAPACITY (a sequence's rows exceed
 * bt_stride pages), _CUDA. */
int dflash_attn_forward_paged(dflash_attn* attn, dflash_paged_cache* cache,
                              int batch, int q_len, const void* noise_hidden,
                              const void* target_hidden,
                              const int32_t* host_n_ctx,
                              const int32_t* host_len_before,
                              const int32_t* positions,
                              const int32_t* slot_mapping,
                              const int32_t* block_table, int bt_stride,
                              void* out, dflash_stream stream);

/* Context K/V of several draft layers in one projection ([P5]
 * precompute_and_store_context_kv: the context K/V of all layers come from one
 * GEMM over their stacked k_proj/v_proj weights, then each layer's k_norm,
 * RoPE and cache insert).
 *
 * dflash_kv_group_create stacks the K and V weights of n_layers (1..16) bf16
 * layers that share hidden, n_kv_heads, head_dim, device, max_position,
 * rms_eps and rope_theta (else _SHAPE; fp32 layers _UNSUPPORTED).  The group
 * owns a copy of those weights; the layers must outlive it.
 *
 * dflash_kv_group_append projects the batch's new context rows once for all
 * layers and appends, for layer l, K = RoPE(k_norm_l(T Wk_l^T)) and
 * V = T Wv_l^T to caches[l] at its current lengths, exactly as
 * dflash_attn_forward appends context rows.  Afterwards call each layer's
 * dflash_attn_forward with host_n_ctx all zero (and positions for the block
 * rows only): it appends the block rows and attends over every cached row.
 *   caches          host array of n_layers cache handles (same batch and
 *                   lengths; geometry of the layers)
 *   target_hidden   device [sum n_i, H] bf16, sequence-major (may be NULL
 *                   when every n_i is 0)
 *   host_n_ctx      host [batch] new context rows per sequence
 *   positions       device [sum n_i] int32, the context rows' positions
 * Errors: _ARG (nulls, negative counts), _SHAPE (batch, geometry or lengths
 * differ between caches), _CAPACITY (a cache would overflow; nothing is
 * appended). */
int dflash_kv_group_create(dflash_attn* const* layers, int n_layers,
                           dflash_kv_group** out);
int dflash_kv_group_destroy(dflash_kv_group* group);
int dflash_kv_group_append(dflash_kv_group* group, dflash_cache* const* caches,
                           int batch, const void* target_hidden,
                           const int32_t* host_n_ctx, const int32_t* positions,
                           dflash_stream stream);

/* The rest of a draft decoder layer ([P4] Qwen3DFlashDecoderLayer:
 * input_layernorm, self_attn, post_attention_layernorm, mlp = Qwen3MLP; [P5]
 * stacks gate_proj/up_proj into gate_up_proj).  Reading taken (the pages name
 * Qwen3MLP without printing it): mlp(y) = down(silu(gate(y)) * up(y)).
 * Weights bf16 device, nn.Linear layout: gate_w, up_w [intermediate, hidden],
 * down_w [hidden, intermediate]; input_norm_w, post_norm_w [hidden] bf16.
 * hidden % 128 == 0 (<= 8192), intermediate % 128 == 0, else _SHAPE.  The
 * handle owns copies of the weights. */
int dflash_mlp_create(int hidden, int intermediate, float rms_eps,
                      const void* gate_w, const void* up_w, const void* down_w,
                      const void* input_norm_w, const void* post_norm_w,
                      dflash_mlp** out);
int dflash_mlp_destroy(dflash_mlp* mlp);

/* One draft decoder layer in the residual-stream form of [P5]'s draft model
 * (each layer returns (hidden_states, residual); the next one adds them):
 *   r1 = hidden_in + residual_in   (residual_in NULL: r1 = hidden_in)
 *   r2 = r1 + attn(input_norm(r1))   -- dflash_attn_forward on the normed rows
 *   hidden_out = mlp(post_norm(r2)),  residual_out = r2
 * hidden_in, residual_in, hidden_out, residual_out: device bf16
 * [batch, q_len, hidden] (residual_out may alias residual_in); the other
 * arguments and the cache update are those of dflash_attn_forward.  bf16
 * layers only (_UNSUPPORTED otherwise); the MLP's hidden must equal the
 * layer's (_SHAPE). */
int dflash_decoder_layer_forward(dflash_attn* attn, dflash_mlp* mlp,
                                 dflash_cache* cache, int batch, int q_len,
                                 const void* hidden_in, const void* residual_in,
                                 const void* target_hidden,
                                 const int32_t* host_n_ctx,
                                 const int32_t* positions, void* hidden_out,
                                 void* residual_out, dflash_stream stream);

/* Training-layout forward with no cache ([P4] module docstring: each block's
 * queries see the context strictly before its anchor plus their own block,
 * bidirectionally; training is one forward with no cache).
 *   noise_hidden  device [batch, n_blocks*block_size, H]
 *   target_hidden device [batch, seq, H]  (projected context)
 *   anchors       device [batch, n_blocks]  int32, each in [0, seq]
 *   out           device [batch, n_blocks*block_size, H]
 * Context row j sits at position j, row t of block k at anchors[k] + t.
 * Blocks may share positions; anchors need not be sorted (sorted anchors
 * balance the work best).  Layers with sliding_window > 0 are _UNSUPPORTED.
 * bf16 layers need (n_heads/n_kv_heads) * block_size <= 128. */
int dflash_attn_forward_packed(dflash_attn* attn, int batch, int seq,
                               int n_blocks, int block_size,
                               const void* noise_hidden,
                               const void* target_hidden,
                               const int32_t* anchors, void* out,
                               dflash_stream stream);

/* Kernel kinds of the per-launch event trace. */
enum {
  DFLASH_K_FC = 0,     /* fc projection GEMM of dflash_ctx_project        */
  DFLASH_K_NORM = 1,   /* hidden_norm row RMSNorm of dflash_ctx_project   */
  DFLASH_K_QKV = 2,    /* QKV projection + norm + RoPE + cache append     */
  DFLASH_K_ATTN = 3,   /* attention (with the split merge)                */
  DFLASH_K_OPROJ = 4,  /* o_proj GEMM                                     */
  DFLASH_K_MISC = 5,   /* packed-layout positions                         */
  DFLASH_K_MLP = 6,    /* decoder layer: add+norm kernels and MLP GEMMs    */
  DFLASH_K_BWD = 7,    /* packed attention core backward (dK/dV and dQ)   */
  DFLASH_K_COUNT = 8
};

/* Attention core of the packed training layout, forward and backward
 * ([P4] module docstring: block k's queries see the context strictly before
 * anchors[k] and their own block; the draft is trained by backpropagation
 * through that masked attention).  These take Q, K and V directly (after
 * the projections, norms and RoPE), so a training framework can run its own
 * projections and autograd around them.  The layer handle supplies
 * n_heads, n_kv_heads, head_dim and scratch; its weights are not used.
 *   q, out, d_out, dq  device [batch][n_blocks*block_size][n_heads][head_dim]
 *                      bf16 (block k's rows at k*block_size ..)
 *   k, v, dk, dv       device [batch][n_kv_heads][seq + n_blocks*block_size]
 *                      [head_dim] bf16: per (sequence, kv head) the seq
 *                      context rows, then every block's rows in block order
 *   lse                device [batch][n_blocks*block_size][n_heads] fp32:
 *                      natural log of each query row's softmax normaliser,
 *                      log(sum over visible keys of exp(q.k / sqrt(head_dim)))
 *   anchors            device [batch][n_blocks] int32 in [0, seq]
 * dflash_packed_attn_core writes out = softmax(q k^T / sqrt(d), masked) v and
 * lse.  dflash_packed_attn_core_backward takes the forward's q, k, v, out,
 * lse and the output gradient d_out and writes the gradients dq, dk, dv
 * (each KV head's gradient sums over the query heads that read it; key rows
 * no query sees get 0).  Every output element is written exactly once (no
 * atomics; reruns are bitwise identical).
 * Requires a bf16 layer without sliding window or causal flag, and
 * (n_heads / n_kv_heads) * block_size == 64.  An anchor outside [0, seq] is
 * clamped and recorded (DFLASH_DEV_ANCHOR) by the forward.
 * Errors: _ARG, _SHAPE, _UNSUPPORTED, _CUDA. */
int dflash_packed_attn_core(dflash_attn* attn, int batch, int seq,
                            int n_blocks, int block_size, const void* q,
                            const void* k, const void* v,
                            const int32_t* anchors, void* out, float* lse,
                            dflash_stream stream);
int dflash_packed_attn_core_backward(dflash_attn* attn, int batch, int seq,
                                     int n_blocks, int block_size,
                                     const void* q, const void* k,
                                     const void* v, const void* out,
                                     const float* lse, const void* d_out,
                                     const int32_t* anchors, void* dq,
                                     void* dk, void* dv,
                                     dflash_stream stream);

/* Draft KV cache in 8 bits (the pages have no counterpart: a property of this
 * library, not of the method).  A row of a KV head is 128 code bytes and one
 * scale byte per group of 32 channels, 132 bytes instead of 256, which is what
 * a decode step reads per key.
 *
 * Value of a channel = code * 2^e, e = scale byte - 127, where for the group's
 * largest magnitude amax
 *   DFLASH_Q8_INT8: code a whole number of magnitude at most 127, and
 *   DFLASH_Q8_E4M3: code an e4m3 number (3 fraction bits) of magnitude at
 *                   most 448;
 *   e = the smallest integer with amax <= 127 * 2^e (448 * 2^e), at least
 *       -117; code = x * 2^-e rounded to nearest, ties to even.  Scale byte 0
 *   marks a group of zeros.
 * Values read back are exact in bf16.  The error of a channel is at most
 * 2^(e-1) with int8 (at most amax / 127), and with e4m3 at most 2^-4 of
 * itself or 2^(e-10): int8 is the finer one for rows whose channels are of one
 * size, e4m3 keeps the small channels of rows with a few large ones.
 * Magnitudes above 2^126 are stored as 2^126; a group with an infinity or NaN
 * reads back as NaN in all of its channels.
 *
 * Storage: codes [batch][n_kv_heads][rows][128] (int8: the number plus 128)
 * and scale bytes [batch][n_kv_heads][rows][4], K and V each, rows
 * = capacity_rows rounded up to a multiple of 128, zeroed at creation.
 * Lengths start at 0 and are kept on the host, as in dflash_cache; crop moves
 * no data.  bf16 layers only (else _UNSUPPORTED).
 *
 * Every call that enqueues work needs the layer's device to be the current
 * one (_ARG).  The cache owns the scratch of the attention over it, sized once
 * at creation: calls on one cache must not run concurrently on different
 * streams.  In a CUDA graph a call keeps the lengths, and so the rows it
 * writes and reads, of the moment of its capture; what a replayed call reads has
 * to be rows that the cache still holds or that a replay wrote.
 *
 * The cache keeps the range of the scales written to every (sequence, KV head).
 * The attention reads a head's codes as fp16 numbers while its scales lie within
 * 20 binades of one another (K and V each) and no group reads NaN, otherwise as
 * bf16 numbers, which takes about 1.4 times as long.  Either is exact; the
 * probabilities are rounded to the same type.  A range widens with every row
 * that is written, also with one that is cropped later, and starts again when an
 * append outside a CUDA graph begins at row 0. */
enum { DFLASH_Q8_E4M3 = 0, DFLASH_Q8_INT8 = 1 };

int dflash_q8_cache_create(const dflash_attn* attn, int batch,
                           int capacity_rows, int format,
                           dflash_q8_cache** out);
int dflash_q8_cache_destroy(dflash_q8_cache* cache);

/* As dflash_cache_lengths and dflash_cache_crop. */
int dflash_q8_cache_lengths(const dflash_q8_cache* cache, int32_t* host_len);
int dflash_q8_cache_crop(dflash_q8_cache* cache, const int32_t* host_keep);

/* Device pointers to the storage (layout above) and its geometry
 * (stored_rows: the rounded capacity); any output may be NULL.  For
 * inspection; writing through them is the caller's risk. */
int dflash_q8_cache_data(const dflash_q8_cache* cache, void** k_codes,
                         void** v_codes, void** k_scales, void** v_scales,
                         int32_t* batch, int32_t* n_kv_heads,
                         int32_t* stored_rows, int32_t* head_dim);

/* Size the cache's scratch for dflash_attn_forward_q8 calls that append at
 * most max_new_rows rows (context and block) to any sequence, so that they
 * allocate nothing for it: 4 * batch * n_kv_heads * 128 * max_new_rows bytes
 * (K and V in bf16, every sequence's rows at the same distance). */
int dflash_q8_cache_reserve(dflash_q8_cache* cache, int max_new_rows);

/* Encode host_n[b] rows of K and V behind the rows sequence b holds.
 *   k, v    device bf16, row r (the sequences' new rows one after another)
 *           at k + r * k_row_stride elements: [n_kv_heads][128], dense; rows
 *           may be slices of a wider tensor (strides multiples of 8, at least
 *           n_kv_heads * 128).  May be NULL when every count is 0.
 *   host_n  host [batch]
 * Errors: _ARG, _SHAPE, _CAPACITY (nothing is appended for any sequence),
 * _CUDA. */
int dflash_q8_cache_append(dflash_q8_cache* cache, const void* k, const void* v,
                           int64_t k_row_stride, int64_t v_row_stride,
                           const int32_t* host_n, dflash_stream stream);

/* Decode rows host_first[b] .. host_first[b] + host_n[b] - 1 of every
 * sequence, one sequence after another, into the dense device tensors k_dst
 * and v_dst [sum host_n][n_kv_heads][128] bf16.
 * Errors: _ARG, _SHAPE, _RANGE (rows the sequence does not hold), _CUDA. */
int dflash_q8_cache_read(const dflash_q8_cache* cache, const int32_t* host_first,
                         const int32_t* host_n, void* k_dst, void* v_dst,
                         dflash_stream stream);

/* Attention of a block's queries over an 8-bit cache, without the layer's
 * projections (its weights are not used; its head counts, window and causal
 * flag are).
 *   q    device bf16 [batch][q_len][n_heads][128], after norm and RoPE
 *   out  device bf16, as q
 *   lse  device fp32 [batch][q_len][n_heads] or NULL: natural log of the sum
 *        over the row's keys of exp(q.k / sqrt(128))
 * The q_len queries stand at the sequence's last q_len key indices (block row
 * t at length - q_len + t, which only a window or the causal flag look at); K
 * and V are the rows the cache holds.  A row that sees no key gets out = 0 and
 * lse = -infinity; a row of q with an infinity or NaN, NaN.  Scores are held in
 * fp32: beyond its range one counts as the largest number, or as not seen below.
 * Any q_len; at most 128 query heads per KV head (_UNSUPPORTED).  The cached
 * rows are decoded once per 64 query rows of a KV head (q_len * n_heads /
 * n_kv_heads), which bounds long calls: up to 64 rows take one time, up to 128
 * nearly twice that.
 * After a bounded wait that ran out (DFLASH_DEV_WAIT_TIMEOUT, which only
 * dflash_device_error() reports) rows of out and lse may be zero, -infinity or
 * lack some of their keys.
 * Errors: _ARG, _SHAPE, _UNSUPPORTED, _CUDA. */
int dflash_q8_attn_core(dflash_attn* attn, dflash_q8_cache* cache, int batch,
                        int q_len, const void* q, void* out, float* lse,
                        dflash_stream stream);

/* dflash_attn_forward over an 8-bit cache: arguments, outputs, appended rows,
 * lengths and errors are those of dflash_attn_forward.  K (after k_norm and
 * RoPE) and V are rounded to bf16 and encoded as they are appended, and the
 * queries see the encoded rows, the block's own included.  Any q_len.
 * Before a call is captured into a CUDA graph its scratch has to have the size
 * it needs (a call of that size before, or dflash_attn_reserve and
 * dflash_q8_cache_reserve).  The scratch of the layer and of the cache that a
 * captured call uses stays allocated until they are destroyed, also when a
 * larger call later needs more; they have to outlive the graph. */
int dflash_attn_forward_q8(dflash_attn* attn, dflash_q8_cache* cache, int batch,
                           int q_len, const void* noise_hidden,
                           const void* target_hidden, const int32_t* host_n_ctx,
                           const int32_t* positions, void* out,
                           dflash_stream stream);

/* Verification of drafted tokens against the target's probabilities, from
 * given uniform numbers ([P3] 关键设计: the target accepts a prefix of the
 * block, to which the draft cache is then cropped).  Needs no layer.
 *
 * Sequence b has drafted tokens x_0 .. x_{n-1}, drawn from the distributions
 * q_i, and the target's distributions p_0 .. p_n (p_i: after i of them).
 * Draft i is accepted when every one before it is and
 *     u_accept[i] * q_i(x_i) < p_i(x_i)        (compared without rounding).
 * With a the number of accepted drafts, one more token follows them: drawn
 * from max(p_a - q_a, 0) when draft a was rejected, from p_n when a = n, as
 * the first token whose cumulative weight exceeds floor(u_sample * sum of the
 * weights), the product not rounded before.  Weights are whole multiples of 2^-44: a probability is taken as
 * floor(min(max(p, 0), 1) * 2^44), NaN as 0.  If the difference leaves no
 * weight the token is drawn from p_a; if that has none either it is -1.  The
 * result does not depend on the GPU's order of summation.
 *
 * draft_probs NULL: the drafts were chosen without sampling (the largest
 * logit, say), so q_i is 1 at x_i and 0 elsewhere.
 *
 *   dtype         of the probabilities, DFLASH_BF16 or DFLASH_FP32
 *   draft_tokens  device int32 [batch][n_draft]; a token outside [0, vocab)
 *                 is rejected
 *   draft_probs   device: p of token v at batch_stride * b + row_stride * i
 *                 + v elements, i < n_draft; may be NULL
 *   target_probs  the same, i <= n_draft.  Rows on 16-byte boundaries are
 *                 read with wider loads.
 *   u_accept      device fp32 [batch][n_draft], u_sample fp32 [batch], in
 *                 [0, 1) (a u_sample outside is moved to the nearest end, NaN
 *                 to 0)
 *   seq_drafts    device int32 [batch] or NULL: drafts of each sequence,
 *                 moved into [0, n_draft]; NULL: n_draft for all
 *   accepted      device int32 [batch]: a
 *   tokens        device int32 [batch][n_draft + 1]: the accepted drafts, the
 *                 token that follows, then -1
 * n_draft may be 0 (a token is drawn from p_0); draft_tokens and u_accept may
 * then be NULL.  Work goes to the current device.
 * Errors: _ARG, _SHAPE (vocab >= 2^19, too many tokens), _CUDA. */
int dflash_verify(int batch, int n_draft, int vocab, int dtype,
                  const int32_t* draft_tokens, const void* draft_probs,
                  int64_t draft_batch_stride, int64_t draft_row_stride,
                  const void* target_probs, int64_t target_batch_stride,
                  int64_t target_row_stride, const float* u_accept,
                  const float* u_sample, const int32_t* seq_drafts,
                  int32_t* accepted, int32_t* tokens, dflash_stream stream);

/* Per-head RMSNorm and rotation of queries and keys, outside the QKV
 * projection, and its gradient: with dflash_packed_attn_core what a training
 * framework needs between its projections and the attention ([P3] step 1,
 * [P4] apply_rotary_pos_emb; the pages leave the gradient to autograd).  Per
 * head x of a row at position p, with r = 1 / sqrt(mean(x^2) + rms_eps):
 *   y = rotation(p) (gain * x * r)      (pairs j, j + head_dim / 2)
 * and back, with w = rotation(-p) d_y:
 *   d_x = r * (w * gain - x * r^2 * mean(w * gain * x)),
 *   d_gain = sum over rows and heads of w * x * r.
 * The layer gives head counts, head_dim, rms_eps, rope_theta, max_position and
 * its type; of its weights only the gains are used, and only where q_norm_w or
 * k_norm_w is NULL. */
typedef struct {
  void* data;                /* [batch][rows][heads][head_dim], channels dense */
  int64_t batch_stride, row_stride, head_stride; /* in elements, >= 0        */
} dflash_heads;

/*   q, k          device, n_heads and n_kv_heads heads; NULL: none of them
 *                 (the keys of context rows, say), not both
 *   q_norm_w      device [head_dim] in the layer's type, or NULL
 *   positions     device int32 [batch][rows]; one outside [0, max_position) is
 *                 clamped and recorded (DFLASH_DEV_POSITION)
 *   q_out, k_out  device, as q and k; may be q and k themselves (not overlap
 *                 them otherwise), or any layout whose heads do not overlap,
 *                 such as rows of the packed core's keys; not one another
 * Strides of inputs may be 0.  bf16: 16-byte boundaries, strides multiples of
 * 8 elements; 32-bit tensors: 4-byte boundaries.  A head's sum of squares has to
 * lie in fp32's range.  batch or rows may be 0.  The layer's device has to be current.
 * Errors: _ARG, _SHAPE, _CUDA. */
int dflash_qk_norm_rope(dflash_attn* attn, int batch, int rows, const dflash_heads* q,
                        const dflash_heads* k, const void* q_norm_w, const void* k_norm_w,
                        const int32_t* positions, const dflash_heads* q_out,
                        const dflash_heads* k_out, dflash_stream stream);

/* Bytes of the workspace of dflash_qk_norm_rope_backward. */
int dflash_qk_norm_rope_workspace(const dflash_attn* attn, size_t* bytes);

/*   q, k            as given to dflash_qk_norm_rope (before norm and rotation)
 *   d_q, d_k        device, as q and k: gradients of its outputs
 *   dq_out, dk_out  device: gradients of q and k; may be d_q and d_k or q and k
 *                   themselves
 *   d_q_norm,       device fp32 [head_dim]: the gains' gradients, written (not
 *   d_k_norm        added to); NULL iff q (k) is
 *   workspace       device, 16-byte aligned, the caller's until the work is done
 * Every sum is taken in an order that depends on the sizes and the tensors'
 * alignment alone.
 * Errors: _ARG, _SHAPE, _CAPACITY (workspace), _CUDA. */
int dflash_qk_norm_rope_backward(dflash_attn* attn, int batch, int rows, const dflash_heads* q,
                                 const dflash_heads* k, const void* q_norm_w,
                                 const void* k_norm_w, const int32_t* positions,
                                 const dflash_heads* d_q, const dflash_heads* d_k,
                                 const dflash_heads* dq_out, const dflash_heads* dk_out,
                                 float* d_q_norm, float* d_k_norm, void* workspace,
                                 size_t workspace_bytes, dflash_stream stream);

/* Cross entropy of a linear head over a vocabulary, and its gradients, for
 * training a draft against the target's tokens, without holding the logits
 * (no counterpart on the pages).  Needs no layer.  With z = x w^T:
 *   nll = logsumexp(z) - z[target],   lse = logsumexp(z)   (natural logs)
 *   dx = d_nll * (sum_v p_v w_v - w[target]),
 *   dw[v] = sum over rows of d_nll * (p_v - [v = target]) * x,   p = exp(z - lse):
 * the gradients of sum(d_nll * nll), so that d_nll holds the loss' weights.
 *   x        device bf16: row r at x + r * x_stride elements, channels dense
 *   w        device bf16 [vocab][hidden], rows w_stride elements apart
 *   targets  device int32 [rows]; one outside [0, vocab) marks a row without a
 *            target: nll, lse and dx are 0, and nothing of the row is looked at
 *   d_nll    device fp32 [rows]
 *   nll, lse device fp32 [rows]
 *   dx       device bf16 [rows][hidden]; dw device bf16 [vocab][hidden] or NULL
 *            (a head that is not trained).  Written, not added to; must not
 *            overlap the inputs.
 * hidden is a multiple of 8 (at most 2^16), row strides too; rows may be 0 (dw
 * is then zero).  Products are of bf16 with fp32 sums; exponentials relative to
 * a reference, and d_nll * p for dw, are rounded to bf16 once before the second
 * product.  Sums are taken in an order that depends on the sizes and on which
 * rows have a target alone.
 * A logit that is NaN or +infinity, or the target's where it is -infinity,
 * leaves the row's nll not finite; an x that is not finite changes dw, but
 * nothing else of other rows.
 *   workspace  device, 256-byte aligned, the caller's until the work is done;
 *              dflash_linear_ce_workspace gives its size for grads = 0 (nll and
 *              lse), 1 (dx) or 2 (dx and dw).  With R the rows rounded up to
 *              256 and H hidden rounded up to 64 it is, in bytes, 2 R H and R *
 *              vocab / 32 (twice that for grads = 0); with gradients also up to
 *              64 R H of fp32 sums (few rows: 64, many: 4) and a piece's
 *              exponentials, at most about 1 GiB (or 4096 columns' worth, if
 *              that is more; half as much again with dw and all columns in one
 *              piece); with dw 8 vocab; a few words a row and piece.
 * After a bounded wait that ran out nll and lse are NaN.  Work goes to the
 * current device.
 * Errors: _ARG, _SHAPE, _CAPACITY (workspace), _CUDA. */
int dflash_linear_ce_workspace(int rows, int vocab, int hidden, int grads, size_t* bytes);
int dflash_linear_ce(int rows, int vocab, int hidden, const void* x, int64_t x_stride,
                     const void* w, int64_t w_stride, const int32_t* targets, float* nll,
                     float* lse, void* workspace, size_t workspace_bytes, dflash_stream stream);
int dflash_linear_ce_grad(int rows, int vocab, int hidden, const void* x, int64_t x_stride,
                          const void* w, int64_t w_stride, const int32_t* targets,
                          const float* d_nll, float* nll, float* lse, void* dx, void* dw,
                          void* workspace, size_t workspace_bytes, dflash_stream stream);

/* Global norm of many gradients, and clipping by it.  Needs no layer (no
 * counterpart on the pages).
 *   norm = sqrt(sum over all tensors of g^2)
 *   clipping: where norm > max_norm, out = g * (max_norm / norm); otherwise,
 *   and where an infinity or NaN is among the gradients (the caller finds it in
 *   `norm`), out = g.  A norm of finite gradients above fp32's range, which
 *   `norm` gives as infinite, clips like any other.
 *   n_tensors   at most 2^20; may be 0 (norm 0)
 *   grads, out  host arrays of device pointers, aligned to their types; out
 *               NULL: in place.  What is written must not overlap anything
 *               else that is read or written (_ARG): each tensor is given once.
 *   counts      host: elements of each tensor, dense; may be 0 (the pointer
 *               may then be NULL)
 *   dtypes      host: DFLASH_BF16 or DFLASH_FP32 each; out has the same
 *   max_norm    >= 0; may be infinite
 *   norm        device fp32
 *   workspace   device, 16-byte aligned, the caller's until the work is done
 * Squares are added in fp64 above groups of 64, in an order that depends on
 * the sizes and addresses' alignment alone; magnitudes over the whole fp32
 * range count.  Gradients that need no clipping in place are only read.
 * Work goes to the current device.
 * Errors: _ARG, _CAPACITY (workspace), _MEMORY, _CUDA. */
int dflash_grad_norm_workspace(int n_tensors, size_t* bytes);
int dflash_grad_norm(int n_tensors, const void* const* grads, const int64_t* counts,
                     const int32_t* dtypes, float* norm, void* workspace,
                     size_t workspace_bytes, dflash_stream stream);
int dflash_clip_grad_norm(int n_tensors, const void* const* grads, void* const* out,
                          const int64_t* counts, const int32_t* dtypes, double max_norm,
                          float* norm, void* workspace, size_t workspace_bytes,
                          dflash_stream stream);

/* Kernels this library has launched in this process so far, over every
 * layer, cache and device (a launch that returned an error counts too).  A
 * caller reads it before and after a region to count that region's kernels. */
int dflash_kernel_launches(uint64_t* count);

/* Launch tracing for measurement: while enabled, every kernel launch of the
 * layer is bracketed by two CUDA events recorded on its own stream.
 * dflash_trace_enable(attn, 1) starts a fresh trace, (attn, 0) stops it.
 * dflash_trace_read waits for the recorded events and returns, for one
 * kernel kind, the summed device time in milliseconds and the launch count.
 * Not for use while a stream is being captured into a CUDA graph. */
int dflash_trace_enable(dflash_attn* attn, int enable);
int dflash_trace_read(dflash_attn* attn, int kind, double* total_ms,
                      int32_t* launches);

/* Wait for the device, then report and clear the layer's device error word
 * (DFLASH_DEV_*).  Returns DFLASH_ERR_DEVICE when the word was non-zero. */
int dflash_device_error(dflash_attn* attn, int32_t* code);

/* Check of the bounded device waits (no counterpart on the pages: failure
 * handling of this library).  Enqueues one kernel on `stream` in which one
 * thread waits on a shared-memory mbarrier with the same routine every
 * pipeline wait of the library uses, but for at most limit_ns nanoseconds of
 * GPU global time instead of the pipelines' 2 s.
 *   arrive = 1: the barrier's one expected arrival is made first; the wait
 *               completes at once and nothing is recorded.
 *   arrive = 0: nothing ever arrives; the wait runs out, records
 *               DFLASH_DEV_WAIT_TIMEOUT in the layer's device error word and
 *               the kernel returns normally (no trap, no fault): the context
 *               stays usable and dflash_device_error() reports the code.
 * limit_ns must lie in [1e3, 1e8].  Errors: _ARG, _CUDA. */
int dflash_wait_probe(dflash_attn* attn, int64_t limit_ns, int arrive,
                      dflash_stream stream);

/* Measurement aid (no counterpart on the pages): the rate at which TMA alone
 * reads a projection's weights.  Enqueues one kernel on `stream` that streams
 * the rows x cols bf16 row-major device matrix `matrix` (caller-owned, 16-byte
 * aligned) once into shared memory in the boxes the GEMMs read weights in
 * (128 rows x 64 columns, 128-byte swizzle) and discards it.  The boxes, in
 * (row block, column block) order, are split into `ctas` contiguous shares,
 * one per CTA; each CTA keeps `stages` boxes (16 KB each) in flight and
 * reuses a slot as soon as its box has landed.  Nothing is written.  Time it
 * with events on `stream`.  rows: a positive multiple of 128; cols: a
 * positive multiple of 64; stages in [1, 12]; ctas in [1, 2 x SMs], and at
 * most 6 stages when ctas exceeds the SM count (two CTAs per SM).  Its
 * bounded waits record DFLASH_DEV_WAIT_TIMEOUT in the layer's device error
 * word like every pipeline of the library.  Errors: _ARG, _CUDA. */
int dflash_read_stream_probe(dflash_attn* attn, const void* matrix, int64_t rows,
                             int64_t cols, int ctas, int stages, dflash_stream stream);

#ifdef __cplusplus
}
#endif

#endif /* DFLASH_ATTN_H */
