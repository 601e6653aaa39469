/*
 * pi.h -- C ABI of the neuron-aware sparse FFN decode path (one GPU, sm_103a).
 *
 * Per decode layer the path computes, for each token x (length d):
 *   1. predictor:  u = P1 x,  s = P2 u + b,  neuron k predicted active iff s_k > tau
 *   2. compaction: the ascending list of predicted-active storage rows
 *   3. FC1:        h_j = ReLU(W1[idx_j] . x + b1[idx_j])     (gated: * (Wu[idx_j] . x))
 *   4. FC2:        y = b2 + sum_j h_j * W2t[idx_j, :]
 * following the pages describing PowerInfer (PowerInfer summary (CSDN)):
 * section "Background" (FC1, ReLU, FC2 as products of the input with neurons,
 * i.e. rows/columns of the weight matrices), section "Adaptive sparse
 * predictor" (an input/hidden/output predictor of which neurons fire),
 * section "Neuron-aware operator" (decide whether a neuron is active, then
 * process only its row or column, with no dense-format conversion) and section
 * "Neuron placement and management" (a table maps each stored neuron to its
 * original position).
 *
 * Conventions for every entry point:
 *  - Every pointer argument except the descriptors is DEVICE memory owned by
 *    the caller; the library allocates nothing and keeps no pointer after the
 *    call returns.  Descriptors (pi_layer_desc, pi_layer_weights) are HOST
 *    structs read during the call only.
 *  - All calls are asynchronous on `stream` (a cudaStream_t passed as void*;
 *    NULL = the legacy default stream).  Device-side counts stay on the device:
 *    no call synchronises the host except pi_last_device_status.
 *  - Arguments are validated on the host before anything is launched; a bad
 *    argument returns PI_ERR_INVALID_ARG and launches nothing.  A failed launch
 *    returns PI_ERR_CUDA.
 *  - Binary16 data is passed as pi_half (IEEE 754 binary16 bit patterns).
 *  - Per-neuron arrays (W1, Wu, W2t, their scales, b1, P2 rows, table) are in
 *    STORAGE order: storage row k holds original neuron table[k].
 *  - Masks: bit k of a mask is bit (k % 32) of 32-bit word k / 32; a batch of
 *    B masks is B consecutive runs of ceil(F/32) words.
 *  - Alignment: every weight, x and workspace pointer 16-byte aligned;
 *    d % 8 == 0 (fp16) and d % 32 == 0 (INT4); rank % 8 == 0.
 *  - Calls on distinct streams with distinct outputs and workspaces may run
 *    concurrently; calls sharing a workspace must be stream-ordered.
 *  - A workspace must be zero-filled (e.g. cudaMemset) before its first use;
 *    the library keeps it consistent from then on.  pi_ffn_layer and
 *    pi_ffn_stack exchange data between thread blocks through it with bounded
 *    waits: a wait that exceeds 2 s makes the kernel return early and sets the
 *    device status read by pi_last_device_status (PI_ERR_TIMEOUT).
 */
#ifndef PI_H
#define PI_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

#if defined(PI_BUILD) && defined(__GNUC__)
#define PI_API __attribute__((visibility("default")))
#else
#define PI_API
#endif

typedef uint16_t pi_half; /* IEEE 754 binary16 bit pattern */

typedef enum {
    PI_OK = 0,
    PI_ERR_INVALID_ARG = 1, /* bad pointer, size, alignment or descriptor      */
    PI_ERR_UNSUPPORTED = 2, /* valid request this build does not implement       */
    PI_ERR_CUDA = 3,        /* a CUDA runtime call or launch failed              */
    PI_ERR_TIMEOUT = 4,     /* a bounded device-side wait expired                */
    PI_ERR_WORKSPACE = 5    /* workspace NULL, misaligned or smaller than needed */
} pi_status;

typedef enum {
    PI_W_F16 = 0,     /* rows of d binary16 values                                    */
    PI_W_INT4_G32 = 1 /* rows of d/2 bytes of INT4 codes (even element in the low      */
                      /* nibble, two's complement, value q*scale) + d/32 binary16 scales */
} pi_wdtype;

typedef struct {
    int d;            /* model width                                  */
    int ffn;          /* FFN width F (number of neurons)              */
    int rank;         /* predictor rank r                             */
    int batch;        /* tokens B processed together (1..32)          */
    pi_wdtype wdtype; /* FC1/FC2 weight format (Wu is always fp16)    */
    int gated;        /* 1: h = ReLU(Wg x + bg) * (Wu x)              */
} pi_layer_desc;

typedef struct {
    const void *w1;          /* [F, d] fp16, or [F, d/2] INT4 codes (gate rows when gated) */
    const pi_half *w1_scales; /* [F, d/32] (INT4 only, else NULL)                           */
    const pi_half *b1;       /* [F]  FC1 (gate) bias, also the predictor bias              */
    const pi_half *wu;       /* [F, d] fp16 up-projection rows (gated only, else NULL)     */
    const void *w2t;         /* [F, d] fp16 or INT4 codes: row k = neuron k's FC2 column   */
    const pi_half *w2t_scales; /* [F, d/32] (INT4 only, else NULL)                         */
    const pi_half *b2;       /* [d]                                                        */
    const pi_half *p1;       /* [r, d] predictor input layer                               */
    const pi_half *p2;       /* [F, r] predictor output layer (storage order)              */
    const int32_t *table;    /* [F] storage row -> original neuron id                      */
} pi_layer_weights;

/* Bytes of workspace pi_predict, pi_sparse_fc1, pi_sparse_fc2 and pi_ffn_layer need for
 * `desc` (0 if the descriptor is invalid). */
PI_API size_t pi_workspace_bytes(const pi_layer_desc *desc);

/*
 * Predictor (PowerInfer summary (CSDN), section "Adaptive sparse predictor").
 *   u_b = P1 x_b (fp32), s_b = P2 u_b + bpred (fp32), mask_b bit k = s_bk > tau.
 * x: [B, d] fp16.  mask: [B, ceil(F/32)] uint32 (bits past F are 0).
 * workspace: >= pi_workspace_bytes(desc) bytes, 16-byte aligned.
 * For 16 <= B <= 32, fp16 weights, d % 128 == 0 and rank % 16 == 0 both
 * products run on the tcgen05 tensor cores; u enters P2 u as two fp16 halves
 * hi = fp16(u), lo = fp16(u - hi), which keeps fp32 accuracy.
 */
PI_API pi_status pi_predict(const pi_layer_desc *desc, const pi_half *x, const pi_half *p1,
                     const pi_half *p2, const pi_half *bpred, float tau, uint32_t *mask,
                     void *workspace, size_t ws_bytes, void *stream);

/*
 * Active-neuron compaction (section "Neuron-aware operator": first decide
 * which neurons are active; section "Neuron placement and management": the
 * table gives each stored neuron's original position).
 * For B == 1 compacts mask; for B > 1 compacts the union (bitwise OR) of the
 * B masks.  idx: [F] int32, ascending storage rows, first *d_count valid.
 * orig_idx (nullable, requires table): table[idx].  d_count: [1] int32.
 */
PI_API pi_status pi_compact(const pi_layer_desc *desc, const uint32_t *mask, const int32_t *table,
                     int32_t *idx, int32_t *orig_idx, int32_t *d_count, void *stream);

/*
 * Row-gathered FC1 with fused bias and ReLU (section "Background"; section
 * "Neuron-aware operator": only the rows of active neurons are read).
 *   h[j*B + b] = ReLU(W1[idx_j] . x_b + b1[idx_j])  (gated: times Wu[idx_j] . x_b)
 * for j < *d_count; when B > 1 and mask != NULL, h[j*B+b] = 0 wherever token
 * b's own mask bit idx_j is 0.  h: [F*B] fp32 (neuron-major).
 * For 16 <= B <= 32, fp16 weights and d % 128 == 0 the rows are gathered once
 * for all B tokens and multiplied on the tcgen05 tensor cores (fp16 x fp16
 * products, fp32 accumulation); so are INT4 rows of a ReLU layer at B = 16
 * with d % 256 == 0 (codes as exact fp16 integers, group scales applied per
 * 32-element group); INT4 at 2 <= B <= 16 otherwise streams on CUDA cores;
 * the rest runs on CUDA cores in chunks of <= 8 tokens.
 * workspace: >= pi_workspace_bytes(desc) bytes, 16-byte aligned (partial
 * sums of the tensor-core split).
 */
PI_API pi_status pi_sparse_fc1(const pi_layer_desc *desc, const pi_half *x, const pi_layer_weights *w,
                        const int32_t *idx, const int32_t *d_count, const uint32_t *mask,
                        float *h, void *workspace, size_t ws_bytes, void *stream);

/*
 * FC2 as a gather-accumulate over W2t rows (section "Background"; section
 * "Neuron-aware operator": only the columns of active neurons, stored as rows).
 *   y[b*d + c] = b2[c] + sum_{j < *d_count} h[j*B + b] * W2t[idx_j, c]   (fp32)
 * Reduced without atomics in a fixed order (bitwise reproducible).
 * Under the same conditions as pi_sparse_fc1 the tensor cores take it, with h
 * split into fp16 hi = fp16(h) and lo = fp16(h - hi) so that fp32 accuracy is
 * kept.  INT4 rows at B = 16: the codes are the exact fp16 A operand and the
 * row's group scale moves into B, one (hi, lo) pair of h * scale per token and
 * 32-column group, lo = fp16((h * scale - hi) * 2^11) (scaled out again in the
 * epilogue).
 */
PI_API pi_status pi_sparse_fc2(const pi_layer_desc *desc, const float *h, const int32_t *idx,
                        const int32_t *d_count, const pi_layer_weights *w, float *y,
                        void *workspace, size_t ws_bytes, void *stream);

/*
 * pi_sparse_fc2 for callers that cannot allocate device memory.  The pages
 * have no counterpart to this entry point: it exists for callers such as a
 * plug-in inside a host framework that owns the whole device memory pool and
 * offers no allocation hook, or a service with a fixed device-memory budget
 * that forbids allocation after start-up, which therefore cannot pass the
 * workspace pi_sparse_fc2 needs.  Same arguments and result as pi_sparse_fc2
 * without the workspace; the FC2 partial sums live in an 8 MiB array inside
 * the library that every GPU loading the library holds until process exit.
 *  - Returns PI_ERR_WORKSPACE when the FC2 partial sums of `desc` exceed that
 *    array (2 Mi floats).  They are, with G the SM count: splits x batch x d
 *    floats on the per-token path; G x (ceil(d/128/G) + 2) x T x 128 floats on
 *    the streamed fp16 path (T = 2, 4 or 8 tokens) and on the batch 16..32
 *    tensor-core path (T = 16 or 32) and on the INT4 tensor-core path at 16
 *    tokens (T = 16); G x (ceil(d/256/G) + 2) x T x 256 on the streamed INT4
 *    path (T = 4, 8 or 16).  Allocates nothing in any case.
 *  - The first call on a device looks up the array's device address (once per
 *    device, with that device current); make that first call before any
 *    stream capture.
 *  - All calls share the one array: calls whose executions overlap on the GPU
 *    (different streams, or concurrent host threads) race and give wrong
 *    results; keep them ordered on one stream.
 */
PI_API pi_status pi_sparse_fc2_noalloc(const pi_layer_desc *desc, const float *h, const int32_t *idx,
                                       const int32_t *d_count, const pi_layer_weights *w, float *y,
                                       void *stream);

/*
 * Second tier of a layer's FC rows (PowerInfer summary (CSDN), sections
 * "Neuron placement and management" and "GPU-CPU hybrid execution": the hot
 * neurons stay in GPU memory and the cold ones in the host's memory).  Storage
 * rows 0 .. n_hot-1 (the hot prefix of the neuron table) are read from the
 * pi_layer_weights arrays, rows n_hot .. F-1 from these arrays at row
 * k - n_hot.  The arrays may be host memory that the GPU addresses directly
 * (pinned and mapped, as from cudaHostAlloc; on a Grace-Blackwell system the
 * Grace memory, read over NVLink-C2C) or device memory; they are read with
 * plain 16-byte loads, never with bulk copies.  Same element layout as the
 * pi_layer_weights arrays; 16-byte aligned.
 */
typedef struct {
    int n_hot;                 /* 0 .. F                                              */
    const void *w1;            /* [F - n_hot, d] fp16 or [F - n_hot, d/2] INT4 codes   */
    const pi_half *w1_scales;  /* [F - n_hot, d/32] (INT4 only, else NULL)             */
    const pi_half *wu;         /* [F - n_hot, d] fp16 (gated only, else NULL)          */
    const void *w2t;           /* [F - n_hot, d] fp16 or INT4 codes                    */
    const pi_half *w2t_scales; /* [F - n_hot, d/32] (INT4 only, else NULL)             */
} pi_cold_tier;

/*
 * pi_sparse_fc1 / pi_sparse_fc2 with the rows of `cold` for the storage rows
 * from cold->n_hot on (same results; the per-token CUDA-core kernels, in
 * chunks of <= 8 tokens, for every batch size).  pi_sparse_fc1_tiered needs no
 * workspace; pi_sparse_fc2_tiered takes pi_workspace_bytes(desc) bytes.
 * PI_ERR_INVALID_ARG if n_hot is outside 0..F or a needed pointer is NULL or
 * misaligned.
 */
PI_API pi_status pi_sparse_fc1_tiered(const pi_layer_desc *desc, const pi_half *x, const pi_layer_weights *w,
                                      const pi_cold_tier *cold, const int32_t *idx, const int32_t *d_count,
                                      const uint32_t *mask, float *h, void *stream);
PI_API pi_status pi_sparse_fc2_tiered(const pi_layer_desc *desc, const float *h, const int32_t *idx,
                                      const int32_t *d_count, const pi_layer_weights *w, const pi_cold_tier *cold,
                                      float *y, void *workspace, size_t ws_bytes, void *stream);
/* One decode layer whose cold FC rows live in `cold`: predictor (weights in
 * w) -> compaction -> pi_sparse_fc1_tiered -> pi_sparse_fc2_tiered.  The
 * workspace holds the same intermediates as for pi_ffn_layer. */
PI_API pi_status pi_ffn_layer_tiered(const pi_layer_desc *desc, const pi_half *x, const pi_layer_weights *w,
                                     const pi_cold_tier *cold, float tau, void *workspace, size_t ws_bytes,
                                     float *y, void *stream);

/*
 * One whole decode layer: predictor -> compaction -> FC1 -> FC2 on `stream`.
 * x: [B, d] fp16; y: [B, d] fp32.  The per-token masks, the union index list
 * and its count are left in the workspace (see pi_workspace_layout).
 */
PI_API pi_status pi_ffn_layer(const pi_layer_desc *desc, const pi_half *x, const pi_layer_weights *w,
                       float tau, void *workspace, size_t ws_bytes, float *y, void *stream);

/*
 * One decode step through a stack of n_layers (1..96) layers that share d,
 * ffn, wdtype and gated; desc->rank is the largest rank and ranks[l] (NULL:
 * all desc->rank) the rank of layer l.  Layer l computes y_l from x_l exactly
 * as pi_ffn_layer does, and the next layer's input is the normalisation of
 * its output, x_{l+1} = fp16(y_l / sqrt(mean(y_l^2) + eps)) (as
 * pi_rmsnorm_half).  layers: HOST array of n_layers weight sets (device
 * pointers inside).  x: [B, d] fp16 input of layer 0; y: [B, d] fp32 output
 * of the last layer; x_trace (nullable): [n_layers-1, B, d] fp16, the inputs
 * of layers 1..n_layers-1; layer_counts (nullable): [n_layers, 2] int32, per
 * layer the number of predicted-active neurons and the number of those whose
 * FC1 output is non-zero (for any token of the batch).  The workspace
 * intermediates are the last layer's.
 */
PI_API pi_status pi_ffn_stack(const pi_layer_desc *desc, int n_layers, const pi_layer_weights *layers,
                              const int *ranks, const pi_half *x, float tau, float eps, void *workspace,
                              size_t ws_bytes, float *y, pi_half *x_trace, int32_t *layer_counts,
                              void *stream);

/* Offsets (bytes) of the intermediates pi_ffn_layer leaves in the workspace. */
typedef struct {
    size_t mask;  /* uint32 [B, ceil(F/32)] per-token masks         */
    size_t idx;   /* int32 [F] ascending active rows (union if B>1) */
    size_t count; /* int32 [1]                                      */
    size_t h;     /* float [F*B] FC1 outputs                        */
    size_t total; /* == pi_workspace_bytes                          */
} pi_workspace_layout_t;
PI_API pi_status pi_workspace_layout(const pi_layer_desc *desc, pi_workspace_layout_t *out);

/*
 * Inter-layer normalisation of a decode stack: x_out[b, c] =
 * fp16(y[b, c] / sqrt(mean_c(y[b, :]^2) + eps)) with round-to-nearest-even.
 * y: [B, d] fp32, 16-byte aligned; x_out: [B, d] fp16, 8-byte aligned; d a
 * multiple of 4 (else PI_ERR_INVALID_ARG).  One block per token.
 */
PI_API pi_status pi_rmsnorm_half(int d, int batch, const float *y, float eps, pi_half *x_out,
                          void *stream);

/*
 * Head-sparse self-attention block of one decode step (PowerInfer summary
 * (CSDN), section "Background", paragraph on activation sparsity: in the
 * self-attention block about half of the heads contribute little for a given
 * input; unite.ai page, section on adaptive sparsity predictors: each layer
 * has one activity predictor for its MLP block and one for its self-attention
 * block, and only the neurons predicted active are computed).  The block's
 * neurons are its heads.  For each sequence b (one new token x_b at cache
 * position pos[b]):
 *   1. head mask: u = P1 x_b, s = P2 u + bp, head h active iff s_h > tau
 *      (the predictor of pi_predict with F = heads);
 *   2. k_g = Wk_g x_b + bk_g and v_g = Wv_g x_b + bv_g for EVERY KV head g,
 *      stored as binary16 (round to nearest even) at position pos[b] of the
 *      caches, so later tokens find a complete cache;
 *   3. for each active head h (KV head g = h / (heads / kv_heads)):
 *      q = Wq_h x_b + bq_h;  a_t = softmax_t(q . K_g[t] / sqrt(head_dim)) over
 *      t = 0 .. pos[b] (the token's own key included);  o_h = sum_t a_t V_g[t];
 *   4. y_b = bo + sum over active h of Wo[:, h*dh .. h*dh+dh-1] o_h.
 * A head that is not active for the token adds nothing to y_b: its query,
 * its pass over the cache and its Wo columns are skipped.  Arithmetic in fp32
 * on fp16 weights and caches; the output projection is reduced in a fixed
 * order (bitwise reproducible).
 */
typedef struct {
    int d;         /* model width (multiple of 8)                                  */
    int heads;     /* query heads H (1 .. 1024)                                    */
    int kv_heads;  /* key/value heads KVH, dividing H (H: multi-head attention)    */
    int head_dim;  /* dh: 64 or 128                                                */
    int rank;      /* head predictor rank (multiple of 8)                          */
    int batch;     /* sequences B, one new token each (1 .. 32)                    */
    int max_seq;   /* cache capacity smax per sequence and KV head                 */
} pi_attn_desc;

typedef struct {
    const pi_half *wqkv; /* [(H + 2 KVH) dh, d]: query rows of head h at h*dh, key rows of KV
                            head g at (H + g) dh, value rows at (H + KVH + g) dh            */
    const pi_half *bqkv; /* [(H + 2 KVH) dh] (zeros for a model without biases)           */
    const pi_half *wot;  /* [H dh, d]: Wo transposed, row j = column j of Wo              */
    const pi_half *bo;   /* [d]                                                           */
    const pi_half *p1;   /* [rank, d]  head predictor input layer                         */
    const pi_half *p2;   /* [H, rank]  head predictor output layer                        */
    const pi_half *bp;   /* [H]        head predictor bias                                */
} pi_attn_weights;

/* Bytes of workspace pi_attn_heads needs for `desc` (0 if it is invalid). */
PI_API size_t pi_attn_workspace_bytes(const pi_attn_desc *desc);

/*
 * x: [B, d] fp16.  kcache, vcache: [B, KVH, max_seq, head_dim] fp16 (in:
 * positions below pos[b] of sequence b; out: position pos[b] written).
 * pos: [B] int32 on the device.  head_mask: [B, ceil(H/32)] uint32 out (the
 * predicted-active heads).  y: [B, d] fp32 out.  All 16-byte aligned.
 * The workspace needs no zero fill.  A pos[b] outside 0 .. max_seq-1 leaves
 * sequence b's cache untouched and its y equal to bo, and sets the device
 * status read by pi_last_device_status to PI_ERR_INVALID_ARG.
 */
PI_API pi_status pi_attn_heads(const pi_attn_desc *desc, const pi_half *x, const pi_attn_weights *w,
                               pi_half *kcache, pi_half *vcache, const int32_t *pos, float tau,
                               uint32_t *head_mask, float *y, void *workspace, size_t ws_bytes,
                               void *stream);

/* ------------------------------------------------------------------------
 * Paged serving: block tables, rotary positions with the store into a paged
 * key/value cache, and attention of new tokens over that cache.
 *
 * A request is a row b of a batch.  Its keys and values live in pages of
 * page_size positions; block_table[b * max_pages + j] is the page of its
 * positions j * page_size .. (j + 1) * page_size - 1.  The tokens of a step
 * are packed: those of request b are rows cu_new[b] .. cu_new[b + 1] - 1.  A
 * slot names a position of the cache: page * page_size + position % page_size.
 * ---------------------------------------------------------------------- */
typedef enum { PI_T_F16 = 0, PI_T_BF16 = 1, PI_T_F32 = 2 } pi_dtype;

/* Rows, pages and capacities of a step. */
typedef struct {
    int batch;      /* rows B (1 .. 4096)                                              */
    int page_size;  /* positions per page: 16, 32, 64 or 128                           */
    int num_pages;  /* pages of the cache = capacity of the free list (1 .. 2^26)       */
    int max_pages;  /* entries per block-table row (1 .. 2^20; max_pages * page_size   */
                    /* <= 2^30)                                                        */
    int max_tokens; /* capacity of slots and positions (0 .. 2^24)                      */
} pi_tables_desc;

/*
 * Block tables, page accounting, slots and positions of one step, from the
 * request lengths alone.  Row b keeps cached_len[b] positions and receives
 * new_len[b] tokens; it holds held[b] pages now and needs
 * ceil((cached_len + new_len) / page_size).
 *   - Pages a row no longer needs (its request ended, was replaced by a
 *     shorter one, or was rolled back) are pushed on the free list in row
 *     order, then in column order: free_list[*free_count + i].
 *   - Rows that need more take theirs off the top in row order.  A row is
 *     served iff it needs none or the pages wanted up to and including it
 *     are there; the others keep the pages they hold, get kv_len 0 and their
 *     tokens slot -1.  Running out of pages is not an error: read kv_len.
 * Out: held_out [B] (may be held), free_count_out [1] (may be free_count),
 * cu_new [B + 1], kv_len [B] (cached + new of a served row), slots
 * [max_tokens] and positions [max_tokens] (cached_len + i of a row's i-th
 * token; entries past cu_new[B]: slot -1, position 0).  In and out:
 * block_table [B, max_pages] (only entries of newly taken pages are written)
 * and free_list [num_pages].  All int32 but slots (int64), on the device.
 * A row with a negative length or page count, with more positions than a
 * table row holds, or whose tokens pass max_tokens is not served, keeps its
 * pages and sets the device status to PI_ERR_INVALID_ARG.  The tokens of a
 * row whose positions leave its table row (cached_len negative, or too many
 * with the new ones) are counted in cu_new, so that the rows after it find
 * theirs in the packed projections, where all rows' tokens are max_tokens at
 * most; where they are more, and where new_len (negative, or above what a table
 * row holds) or held itself is out of range, the row's tokens are not counted.
 * cu_new stays within max_tokens.  A free count outside 0 .. num_pages (taken
 * as the nearest bound) and a push past num_pages (dropped) set the same status.
 */
PI_API pi_status pi_block_tables(const pi_tables_desc *desc, const int32_t *cached_len, const int32_t *new_len,
                                 const int32_t *held, int32_t *held_out, int32_t *block_table, int32_t *free_list,
                                 const int32_t *free_count, int32_t *free_count_out, int32_t *cu_new,
                                 int32_t *kv_len, int64_t *slots, int32_t *positions, void *stream);

/* A paged cache (keys and values are two arrays of this shape).  Element
 * (page, head, position, i) is at page * page_stride + head * head_stride +
 * position * token_stride + i (in elements), so both [pages, heads, page_size,
 * head_dim] and [pages, page_size, heads, head_dim] are described.  Strides
 * are at least head_dim and multiples of 8 (head_stride of 64); base pointers
 * 16-byte aligned. */
typedef struct {
    int kv_heads;   /* 1 .. 1024                       */
    int head_dim;   /* 64 or 128                       */
    int page_size;  /* 16, 32, 64 or 128               */
    int num_pages;  /* 1 .. 2^26                       */
    int dtype;      /* PI_T_F16 or PI_T_BF16           */
    long long page_stride, head_stride, token_stride;
} pi_page_desc;

/* How the frequencies base^(-2 i / rot_dim) become longer-range ones. */
typedef enum {
    PI_ROPE_NONE = 0,
    PI_ROPE_LINEAR = 1, /* f / factor (positions interpolated)                            */
    PI_ROPE_BLEND = 2,  /* by wavelengths per original length, r = original_max f / 2 pi:  */
                        /* f / factor below `low`, f above `high`, linear in r between     */
    PI_ROPE_RAMP = 3    /* by pair index: f up to the pair that turns `high` times within */
                        /* original_max positions, f / factor from the one that turns     */
                        /* `low` times, linear in the index between                        */
} pi_rope_scaling;

typedef struct {
    int head_dim;      /* 64 or 128                                               */
    int rot_dim;       /* leading elements that turn: 0 .. head_dim, multiple of 16 */
    int interleaved;   /* 0: pairs (i, i + rot_dim/2); 1: pairs (2i, 2i + 1)      */
    int scaling;       /* pi_rope_scaling                                         */
    double base;       /* > 1                                                     */
    double factor;     /* > 0 (scaled forms)                                      */
    double original_max, low, high; /* blend and ramp: 0 < original_max, 0 < low < high */
    double mscale;     /* factor on cos and sin (1: none), finite                 */
} pi_rope_desc;

/* What pi_rope_store needs of a pi_rope_desc: host memory, filled once by
 * pi_rope_plan_init and passed to every call.  turns[i] is the angle of pair i
 * per position as a fraction of a turn in 64-bit fixed point, so that position
 * p turns by p * turns[i] modulo 2^64 with no loss at far positions. */
typedef struct {
    int head_dim, rot_dim, interleaved;
    float mscale;
    uint64_t turns[64];
} pi_rope_plan;
PI_API pi_status pi_rope_plan_init(const pi_rope_desc *desc, pi_rope_plan *plan);

/* The projections of a step: token t's head h starts at t * stride + h *
 * head_dim (in elements; strides multiples of 8, at least heads * head_dim). */
typedef struct {
    int tokens;        /* 0 .. 2^24                                         */
    int heads;         /* query heads (1 .. 1024)                           */
    int dtype;         /* of q, k, v: PI_T_F16, PI_T_BF16 or PI_T_F32       */
    long long q_stride, k_stride, v_stride, out_stride;
} pi_qkv_desc;

/*
 * Rotary positions and the store into the cache, one launch.  With a =
 * positions[t] * f_i, each pair (x1, x2) of a query or key head becomes
 *   mscale (x1 cos a - x2 sin a), mscale (x2 cos a + x1 sin a);
 * the rest of the head and the values pass unchanged.  Arithmetic in fp32,
 * rounded once to the cache's type.  q_out [tokens, heads, head_dim] (type of
 * the cache; may be q where the types and strides agree, and shares no other
 * memory with q, k or v); keys and values go to slots[t] of kcache and
 * vcache.  A token with slot -1 is rotated and not stored; a slot past the
 * cache or below -1 is not stored and sets the device status to
 * PI_ERR_INVALID_ARG.  q and q_out may both be NULL (store only), or k, v,
 * slots, kcache and vcache (rotate only).  All 16-byte aligned.
 */
PI_API pi_status pi_rope_store(const pi_rope_plan *plan, const pi_page_desc *cache, const pi_qkv_desc *desc,
                               const void *q, const void *k, const void *v, const int32_t *positions,
                               const int64_t *slots, void *q_out, void *kcache, void *vcache, void *stream);

typedef struct {
    int heads;      /* query heads, a multiple of the cache's kv_heads, at most 128 per KV head */
    int batch;      /* requests (1 .. 4096)                                                    */
    int max_tokens; /* rows of q and out (0 .. 2^24)                                            */
    int max_new;    /* most new tokens of one request (1 .. max_tokens)                         */
    int max_pages;  /* entries per block-table row (max_pages * page_size <= 2^30)             */
    int window;     /* 0: none; else a position sees itself and the window - 1 before it        */
    float scale;    /* of the scores; 0: 1 / sqrt(head_dim)                                    */
} pi_paged_desc;

/* Bytes of workspace pi_paged_attn needs (0 if a descriptor is invalid). */
PI_API size_t pi_paged_workspace_bytes(const pi_paged_desc *desc, const pi_page_desc *cache);

/*
 * Causal attention of the new tokens over the paged cache, which holds their
 * own keys and values already.  Request b has n = cu_new[b+1] - cu_new[b] new
 * tokens, the last of its kv_len[b] positions; its i-th token is at position
 * p = kv_len[b] - n + i and sees t = max(0, p - window + 1) .. p:
 *   a_t = scale q . k_t,  out = sum_t e^{a_t} v_t / sum_t e^{a_t},
 *   lse = log sum_t e^{a_t}
 * for each query head h with key/value head h / (heads / kv_heads).  A token
 * that sees nothing (its request has fewer positions than tokens, e.g. kv_len
 * 0) gets zeros and lse -inf.  q [max_tokens, heads, head_dim] and out have the
 * cache's type, rows q_stride and out_stride elements apart (multiples of 8),
 * and share no memory (they may lie side by side in rows of one stride);
 * lse [max_tokens, heads] fp32, or NULL.  Rows past cu_new[batch] are left
 * alone.  Positions that no token of the request sees are not used, whatever
 * they hold: an infinity or NaN reaches the tokens that see it and no others.
 * A call that meets any takes longer, since the rows that are not finite are
 * looked at again by the block that wrote them: 7 ms instead of 0.3 for a token
 * behind 131 thousand keys, 5 ms instead of 1.1 for a chunk of 4096 tokens
 * behind 12288.  Products of 16-bit values are summed in fp32; the weights
 * e^{a_t - m} enter the second product rounded to the cache's type.  The result
 * does not depend on timing (bitwise reproducible on one device).
 * An inconsistent row (cu_new decreasing or past max_tokens, more than max_new
 * tokens, kv_len outside 0 .. max_pages * page_size) is taken as one without
 * tokens (kv_len: without keys) and a page id outside the cache reads as
 * zeros; both set the device status to PI_ERR_INVALID_ARG.
 * workspace: pi_paged_workspace_bytes, 16-byte aligned, zero-filled before its
 * first use (and again after a PI_ERR_TIMEOUT).
 */
PI_API pi_status pi_paged_attn(const pi_paged_desc *desc, const pi_page_desc *cache, const void *q,
                               long long q_stride, const void *kcache, const void *vcache,
                               const int32_t *block_table, const int32_t *cu_new, const int32_t *kv_len, void *out,
                               long long out_stride, float *lse, void *workspace, size_t ws_bytes, void *stream);

/* ------------------------------------------------------------------------
 * The paged cache in 8 bits.  Keys and values are held as e4m3 codes (one
 * byte: sign, 4 bits of exponent, 3 of fraction; no infinities), and each
 * block of 16 positions and each KV head has an exponent e for its keys and
 * one for its values: a code c stands for c 2^e.  A cache takes half the
 * bytes of a 16-bit one (and 1 / 128 more for heads of 128, 1 / 64 for 64: an
 * int8 exponent for 16 head_dim codes).  Block tables, slots and positions are
 * those of pi_block_tables.
 *
 * Element (page, head, position, i) of a code array is the byte at page *
 * page_stride + head * head_stride + position * token_stride + i, so both
 * [pages, heads, page_size, head_dim] and [pages, page_size, heads, head_dim]
 * are described.  Strides are at least head_dim and multiples of 16; base
 * pointers 16-byte aligned.  The exponents are int8 [num_pages, kv_heads,
 * page_size / 16], kept apart for keys and for values, in the range -32 .. 32
 * (others are taken as the nearest).
 * ---------------------------------------------------------------------- */
typedef struct {
    int kv_heads;   /* 1 .. 1024                       */
    int head_dim;   /* 64 or 128                       */
    int page_size;  /* 16, 32, 64 or 128               */
    int num_pages;  /* 1 .. 2^26                       */
    long long page_stride, head_stride, token_stride;   /* bytes */
} pi_page8_desc;

/*
 * Rotary positions and the store into an 8-bit cache: pi_rope_store with the
 * rotated keys and the values quantised as they are written.  The new tokens
 * of a block and head have the largest finite magnitude A; its exponent is the
 * smallest e in -32 .. 32 with A <= 448 2^e, and no smaller than the block's
 * present one where the block keeps earlier positions (the new tokens' first
 * place in the block is not 0).  Where that raises it, the codes of those
 * earlier positions are rounded again under the new exponent.  A code is x /
 * 2^e rounded to nearest even, x in fp32 (magnitudes above 448 2^32 are held as
 * that); an infinity or NaN is stored as NaN.  What a block holds behind the
 * new tokens is given up.
 *   The new tokens of a block are consecutive rows at consecutive slots, as
 * pi_block_tables lists them: a row whose slot does not follow the row
 * before's begins a block's new tokens, and a block has one such row in a call
 * (of several, the block's contents are undefined).  Slots are as for
 * pi_rope_store: -1 is not stored; below that or past the cache is not stored
 * and sets the device status to PI_ERR_INVALID_ARG.
 *   out_dtype is the type of q_out, PI_T_F16 or PI_T_BF16.  q_out may be q where
 * types and strides agree, and shares no other memory with q, k or v.  q and
 * q_out may both be NULL (store only), or k, v, slots, caches and exponents
 * (rotate only).  All but the exponents 16-byte aligned.
 */
PI_API pi_status pi_rope_store8(const pi_rope_plan *plan, const pi_page8_desc *cache, const pi_qkv_desc *desc,
                                int out_dtype, const void *q, const void *k, const void *v,
                                const int32_t *positions, const int64_t *slots, void *q_out, void *kcache,
                                void *vcache, int8_t *kexp, int8_t *vexp, void *stream);

/* Rows that are read back from an 8-bit cache. */
typedef struct {
    int batch;      /* requests (1 .. 4096)                                      */
    int max_pages;  /* entries per block-table row (max_pages * page_size <= 2^30) */
    int max_rows;   /* rows of the outputs (0 .. 2^30)                            */
    int dtype;      /* of the outputs: PI_T_F16, PI_T_BF16 or PI_T_F32            */
    long long k_stride, v_stride;   /* elements from row to row, multiples of 8, at least kv_heads * head_dim */
} pi_read8_desc;

/*
 * Keys and values of requests as rows of 16 or 32 bits.  Row cu_rows[b] + i of
 * k_out and v_out becomes position start[b] + i of request b (start NULL: 0) for
 * all KV heads [kv_heads, head_dim]: c 2^e rounded to the type (fp16 values that
 * would round past 65504 are 65504).  Rows past cu_rows[batch] are left alone.
 * A position outside 0 .. max_pages * page_size - 1 or a page id outside the
 * cache reads as zeros, and an inconsistent request (cu_rows decreasing,
 * negative or past max_rows) is not read, while the others are (a row of several
 * becomes one of theirs); each sets the device status to PI_ERR_INVALID_ARG.  k_out or v_out may be NULL (with its codes and exponents).
 */
PI_API pi_status pi_page_read8(const pi_read8_desc *desc, const pi_page8_desc *cache, const void *kcache,
                               const void *vcache, const int8_t *kexp, const int8_t *vexp,
                               const int32_t *block_table, const int32_t *start, const int32_t *cu_rows,
                               void *k_out, void *v_out, void *stream);

/* Bytes of workspace pi_paged_attn8 needs (0 if a descriptor is invalid). */
PI_API size_t pi_paged8_workspace_bytes(const pi_paged_desc *desc, const pi_page8_desc *cache);

/*
 * pi_paged_attn over an 8-bit cache: the same outputs from keys and values
 * c 2^e.  q and out are of type `dtype`, PI_T_F16 or PI_T_BF16.  Rows of
 * requests without tokens, rows past cu_new[batch], inconsistent rows and page
 * ids are as for pi_paged_attn; a NaN in the cache reaches the tokens that see
 * it and no others.  The result does not depend on timing (bitwise
 * reproducible on one device).
 *   Where max_new is above 64 / (heads / kv_heads) (and 1), requests of more than
 * 8 / (heads / kv_heads) tokens (and 1) go over a 16-bit copy of the pages they
 * see, which the call makes in the workspace (c 2^e rounded to `dtype`, fp16
 * values past 65504 as that); the workspace of such a descriptor has room for
 * one of the whole cache, twice its bytes.  max_new is the descriptor's: a step
 * whose requests are all short is quicker with a descriptor that says so.  fp16
 * outputs that would round past 65504 are 65504.
 * workspace: pi_paged8_workspace_bytes, 16-byte aligned, zero-filled before its
 * first use (and again after a PI_ERR_TIMEOUT); one workspace serves any number
 * of calls that are stream-ordered, whatever their descriptors, where it has the
 * bytes of each.
 */
PI_API pi_status pi_paged_attn8(const pi_paged_desc *desc, const pi_page8_desc *cache, int dtype, const void *q,
                                long long q_stride, const void *kcache, const void *vcache, const int8_t *kexp,
                                const int8_t *vexp, const int32_t *block_table, const int32_t *cu_new,
                                const int32_t *kv_len, void *out, long long out_stride, float *lse,
                                void *workspace, size_t ws_bytes, void *stream);

/* How one pi_ffn_stack step of `desc` (n_layers layers with the given ranks,
 * NULL: all desc->rank) is executed on the current device.  Diagnostics: lets a
 * caller or a test see which streaming mode the batch-1 persistent kernel
 * takes for a shape.  Host only, launches nothing. */
typedef struct {
    int fused;         /* 1: one persistent launch per decode step (batch 1)      */
    int ctas;          /* its thread blocks (one per SM)                          */
    int pred_in_smem;  /* 1: a block's share of the predictor is copied whole into
                          shared memory before it is used                         */
    int p2_ring_slots; /* else: a block's P2 rows stream through this many slots of
                          16 rows (a rank whose ring cannot hold two slots runs
                          on the per-step kernels: fused = 0)                     */
    int fc_row_slots;  /* FC weight rows a block holds in shared memory at once; a
                          block whose predicted neurons need more rows (gated: 3
                          per neuron, else 2) streams them through a ring          */
    int smem_bytes;    /* dynamic shared memory per block                         */
} pi_stack_plan_t;
PI_API pi_status pi_stack_plan(const pi_layer_desc *desc, int n_layers, const int *ranks, pi_stack_plan_t *out);
/* The same plan for a device with `sm_count` SMs (1..4096) instead of the
 * current device: host only, no device is queried, so the plan can be checked
 * where there is no GPU.  PI_ERR_INVALID_ARG for a bad descriptor, layer count,
 * rank or SM count. */
PI_API pi_status pi_stack_plan_for(const pi_layer_desc *desc, int n_layers, const int *ranks, int sm_count,
                                   pi_stack_plan_t *out);

/* Number of kernel launches one pi_ffn_layer call issues for `desc` (-1 if
 * the descriptor is invalid). */
PI_API int pi_launches_per_layer(const pi_layer_desc *desc);

PI_API const char *pi_status_string(pi_status s);

/* Synchronises `stream`, then returns and clears the device status word set
 * by bounded device-side waits (PI_OK or PI_ERR_TIMEOUT). */
PI_API pi_status pi_last_device_status(void *stream);

/* Diagnostics: sets the limit of the bounded device-side waits of the launches
 * that follow (grid barriers and copy/MMA stage waits; 1 ns .. 10 s; 0 restores
 * the default 2 s).  Process-wide, for every device.  A short limit makes the
 * kernels take their failure path: the wait gives up, the device status
 * becomes PI_ERR_TIMEOUT, the block waits (always up to 2 s) for its own copies
 * and tensor-core operations in flight, frees its tensor memory and returns.
 * For testing that path; outputs of a call that timed out are undefined, and
 * a workspace used by pi_ffn_layer or pi_ffn_stack must be zero-filled again
 * before its next use. */
PI_API pi_status pi_debug_set_wait_timeout(long long timeout_ns);

/* Diagnostics: launches one wait on a word that nothing writes, bounded by
 * timeout_ns (1 ns .. 10 s).  The wait gives up, and the device status becomes
 * PI_ERR_TIMEOUT (read it with pi_last_device_status); the GPU context stays
 * usable.  For testing the bounded-wait path. */
PI_API pi_status pi_debug_wait_timeout(long long timeout_ns, void *stream);

#ifdef __cplusplus
}
#endif

#endif /* PI_H */
