/*
 * salad.h -- C ABI of the SALAD hybrid-attention forward library (sm_100a).
 *
 * SALAD runs two attention branches on shared Q, K, V and mixes them with a
 * gated, projected residual:
 *     O = O_sparse + s_b * ((phi(Q) H / (phi(Q) Z + eps)) W_lin[h])
 * with phi = ReLU, H = phi(K)^T V, Z = phi(K)^T 1 and
 * s_b = sigmoid(w . mean_tokens(X[b]) + bias).
 * Sources, by page title and section:
 *   "SALAD ... (paper.rainbus.top)": 前置知识 (sparse mask, linear attention),
 *       方法步骤详情 steps 2-6 (parallel branches, zero-init projection, gate,
 *       residual sum).
 *   "视频扩散模型中的稀疏注意力机制解析 (ijyty.com)": 1.1 (ST-SWA token
 *       regrouping + sliding window), 1.2 (Top-K block selection from block
 *       means), 2.3 (gate: token mean, linear, sigmoid).
 *
 * Conventions shared by every entry point
 *   - Tensors Q, K, V, O are bf16, contiguous, [B, H, N, d] with the exact
 *     token count N (no caller padding).  d must be 64 or 128; the block
 *     size must be 64.  N must be in [1, 262144].  (salad_rope takes other types
 *     and sizes, and it and the cache operators take strides; see there.)
 *   - All tensor pointers are DEVICE pointers, 16-byte aligned, owned by the
 *     caller.  Pointers documented as HOST are read during the call only.
 *   - The library never allocates or frees device memory and never
 *     synchronises.  Scratch memory is a caller-provided device workspace
 *     whose size is returned by the matching *_workspace_bytes query;
 *     256-byte alignment is required.  salad_forward alone creates, on its
 *     first call on each caller stream, two streams and three events of its
 *     own (kept until the process exits) to run independent steps side by
 *     side.
 *   - Work is enqueued on `stream` (a cudaStream_t; NULL = legacy default
 *     stream) in call order.  All argument checks run on the host before any
 *     launch: an invalid call returns an error and enqueues nothing.
 *   - Waits inside the kernels are bounded.  A wait that runs out sets a
 *     device-side error word instead of trapping; salad_check_error() reads
 *     it (and is the only call that synchronises).
 */
#ifndef SALAD_H_
#define SALAD_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int salad_status;
#define SALAD_OK                0
#define SALAD_ERR_INVALID_ARG  (-1)   /* null pointer, bad size, misaligned */
#define SALAD_ERR_UNSUPPORTED  (-2)   /* d not in {64,128}, block != 64, no sm_100 device */
#define SALAD_ERR_CUDA         (-3)   /* a CUDA runtime call or launch failed */
#define SALAD_ERR_TIMEOUT      (-4)   /* a bounded device-side wait ran out */
#define SALAD_ERR_WORKSPACE    (-5)   /* workspace missing, too small or misaligned */

/* Sparse-branch patterns. */
#define SALAD_MODE_TOPK   0   /* Top-K block-sparse (ijyty.com 1.2) */
#define SALAD_MODE_SWA    1   /* spatio-temporal sliding window (ijyty.com 1.1) */
#define SALAD_MODE_DENSE  2   /* every key (the full-attention special case) */

typedef void* salad_stream;   /* cudaStream_t */

/* Human-readable text of a status code; never NULL. */
const char* salad_status_string(salad_status status);

/* Library version as MAJOR*10000 + MINOR*100 + PATCH. */
int salad_version(void);

/*
 * Gate (paper.rainbus.top 方法步骤详情 step 5; ijyty.com 2.3):
 *   s[b] = sigmoid( sum_c w[c] * (1/N) sum_n x[b,n,c] + bias ).
 * x: bf16 [B, N, D] device; w: bf16 [D] device; s: float32 [B] device (out).
 * D must be a multiple of 8.  Workspace: salad_gate_workspace_bytes(B, N, D).
 */
size_t salad_gate_workspace_bytes(int B, int N, int D);
salad_status salad_gate(const void* x, const void* w, float bias, int B, int N, int D,
                        float* s, void* workspace, size_t workspace_bytes,
                        salad_stream stream);

/*
 * Gate with no scratch argument, for callers that cannot allocate device
 * memory at all (a plug-in that receives only its input and output buffers,
 * or code on a path where an allocator call is not permitted).  No passage of
 * the paper corresponds to it.  It keeps its per-CTA partial sums in a fixed
 * 64 KB array inside the library (present on every GPU that loads the
 * library, until the process exits) instead of a caller workspace.
 *   - Result: the value salad_gate computes, from the same kernels and the
 *     same partition of the tokens whenever that partition's B x parts
 *     partial sums fit the array's 16384 floats -- on a 148-SM B200 that
 *     holds for every accepted B, N and D, and the two results are then
 *     bit-identical.  (Were it not to fit, fewer parts per sample would be
 *     used, which changes only the float32 rounding of the partial sums.)
 *   - B may be at most 256; larger batches return SALAD_ERR_INVALID_ARG
 *     before any launch.  Other arguments as for salad_gate.
 *   - The first call on each device looks up the array's device address;
 *     make that first call before capturing the stream into a CUDA graph.
 *   - All calls share the one array, and each call overwrites the slots it
 *     reads, so no clearing is needed -- but two calls whose kernels overlap
 *     on the GPU (different streams without ordering) race on it.
 *   - Allocates nothing: no cudaMalloc, no cudaFree, no allocating library.
 */
salad_status salad_gate_noalloc(const void* x, const void* w, float bias, int B, int N, int D,
                                float* s, salad_stream stream);

/*
 * Top-K block selection (ijyty.com 1.2): split tokens into blocks of `block`
 * rows, average each block over its valid rows (float64), score every
 * query-block mean against every key-block mean (float64 dot product), keep
 * the `topk` largest per query block (ties: lower block index first).
 * q, k: bf16 [B, H, N, d] device.  idx: int32 [B, H, nb, topk] device (out),
 * nb = ceil(N/block), each row in ascending block order.  1 <= topk <= nb.
 * The float64 decision is reached by tensor-core scores of a two-term bf16
 * split of the means with a certified error bound, and a float64 rescoring
 * of the blocks the bound leaves undecided (the bound assumes float32
 * accumulation in the tensor core no worse than float32 additions).
 * Workspace: salad_select_workspace_bytes(B, H, N, d, block); it holds the
 * float32 score matrix [B, H, nb, ceil(nb/128)*128] among others.
 */
size_t salad_select_workspace_bytes(int B, int H, int N, int d, int block);
salad_status salad_select_blocks(const void* q, const void* k, int B, int H, int N, int d,
                                 int block, int topk, int32_t* idx,
                                 void* workspace, size_t workspace_bytes,
                                 salad_stream stream);

/*
 * Linear-attention state (paper.rainbus.top 前置知识 Linear Attention):
 *   Hst[b,h] = relu(K[b,h])^T V[b,h]   float32 [B, H, d, d] device (out)
 *   Z[b,h]   = relu(K[b,h])^T 1        float32 [B, H, d]    device (out)
 * Hst is row-major: Hst[b,h][c][j] = sum_n relu(k[n][c]) v[n][j].
 * Workspace: salad_linear_state_workspace_bytes(B, H, N, d).
 */
size_t salad_linear_state_workspace_bytes(int B, int H, int N, int d);
salad_status salad_linear_state(const void* k, const void* v, int B, int H, int N, int d,
                                float* Hst, float* Z, void* workspace, size_t workspace_bytes,
                                salad_stream stream);

/*
 * Linear-attention output (paper.rainbus.top 前置知识 Linear Attention, the
 * output phi(Q) H / (phi(Q) Z) of the state above; 方法步骤详情 step 3, the
 * linear branch on the layer's own Q):
 *   o_lin[b,h,n,:] = relu(q) Hst / (relu(q) . Z + eps).
 * eps (>= 0, finite) keeps a row with relu(q) = 0 at zero instead of 0/0.
 * q: bf16 [B,H,N,d] device; Hst, Z: float32 device, as produced by
 * salad_linear_state; o_lin: bf16 [B,H,N,d] device (out), must not overlap q.
 * Needs no workspace.  Errors: SALAD_ERR_INVALID_ARG for a null or
 * misaligned pointer, a bad size or eps; nothing is enqueued then.
 */
salad_status salad_linear_apply(const void* q, const float* Hst, const float* Z, float eps,
                                int B, int H, int N, int d, void* o_lin, salad_stream stream);

/*
 * Token permutation of the ST-SWA heads (ijyty.com 1.1).  The latent grid
 * F x Hh x Wh (N = F*Hh*Wh) is flattened frame-major, t = (f*Hh + y)*Wh + x;
 * the space-major order is r = (y*Wh + x)*F + f.
 * src, dst: bf16 [S, N, d] device, S = number of (batch, head) slabs,
 * 1 <= S <= 65535.
 * inverse = 0: dst[s][r] = src[s][t(r)] (frame-major -> space-major);
 * inverse = 1: dst[s][t(r)] = src[s][r] (space-major -> frame-major).
 * src and dst must not overlap.
 */
salad_status salad_permute_tokens(const void* src, void* dst, int S, int N, int d,
                                  int F, int Hh, int Wh, int inverse, salad_stream stream);

/*
 * Sparse branch alone: normalised softmax attention over the pattern,
 * o_sparse = softmax(Q K^T / sqrt(d) + M) V, bf16 [B,H,N,d] (out).
 *   mode SALAD_MODE_TOPK : M keeps, for query block i, the key blocks
 *                          idx[b,h,i,0..topk) (device int32, ascending).
 *   mode SALAD_MODE_SWA  : M keeps |r - c| <= window in each head's order;
 *                          heads with space_major_heads[h] != 0 (HOST uint8
 *                          [H], may be NULL = none) are regrouped
 *                          space-major with the (F, Hh, Wh) grid and their
 *                          output rows are returned in frame-major order.
 *   mode SALAD_MODE_DENSE: every key.
 * Workspace: salad_sparse_attn_workspace_bytes(...).
 */
size_t salad_sparse_attn_workspace_bytes(int B, int H, int N, int d, int mode, int topk,
                                         const uint8_t* space_major_heads);
salad_status salad_sparse_attn(const void* q, const void* k, const void* v,
                               int B, int H, int N, int d, int mode, int block, int topk,
                               const int32_t* idx, int window,
                               const uint8_t* space_major_heads, int F, int Hh, int Wh,
                               void* o_sparse, void* workspace, size_t workspace_bytes,
                               salad_stream stream);

/*
 * Dense flash attention on the same shapes (the comparator the method is
 * measured against): o = softmax(Q K^T / sqrt(d)) V, bf16 [B,H,N,d] (out).
 * Needs no workspace.
 */
salad_status salad_dense_attn(const void* q, const void* k, const void* v,
                              int B, int H, int N, int d, void* o, salad_stream stream);

/*
 * Full-width projection of concatenated heads with a gated residual
 * (paper.rainbus.top 方法步骤详情 step 4, the linear branch's projection read
 * as one layer over all heads, and step 7, the output projection):
 *   out[b,n,:] = resid[b,n,:] + s_b * (A_cat[b,n,:] W)
 * A: bf16 [B,H,N,d] device; A_cat[b,n, h*d + c] = A[b,h,n,c] (the heads of a
 * token concatenated, head-major; no copy is made).  W: bf16 row-major
 * [H*d, n_out] device, n_out a positive multiple of 64.
 * out_per_head = 1: out (and resid) are bf16 [B,H,N,d] (n_out must equal
 *   H*d; column h*d + c of a token is out[b,h,n,c]).
 * out_per_head = 0: out (and resid) are bf16 [B,N,n_out], token-major.
 * resid: device, same layout as out, or NULL (no residual).  It may be the
 *   same pointer as out (in place); otherwise it must not overlap out.
 * s: device float32 [B] or NULL (s_b = 1).  Samples with s_b < drop_threshold
 *   are skipped: their out is not written (0 or NaN never skips).
 * out must not overlap A or W.  Needs no workspace.  tcgen05 GEMM with fp32
 * accumulation; the result is rounded once to bf16.
 */
salad_status salad_project(const void* a, int B, int H, int N, int d, const void* w, int n_out,
                           void* out, int out_per_head, const void* resid, const float* s,
                           float drop_threshold, salad_stream stream);

/*
 * The whole hybrid layer (paper.rainbus.top 方法步骤详情 steps 2-6, 8):
 * gate, sparse branch, linear branch, per-head projection W_lin (d x d,
 * right-multiplying row vectors: O_l' = O_l W_lin[h]), gated residual sum.
 * The sparse pattern runs on `stream`; the gate and the linear branch run on
 * two streams of the library forked from `stream` by an event and joined
 * back to it before the attention kernel, so all work is ordered after the
 * caller's earlier work on `stream` and before its later work.
 * Reentrant: each caller stream gets its own two side streams and fork/join
 * events (created by the first call on that stream -- make it before the
 * stream is captured into a CUDA graph -- and kept until the process exits;
 * up to 32 caller streams per device, after which a call enqueues every step
 * on `stream` itself, in order).  So calls from several threads on different
 * streams neither wait for one another on the host nor depend on one another
 * on the GPU; calls on the same stream are serialised while they enqueue.
 * Concurrent calls must not share a workspace or an output buffer.
 */
typedef struct salad_forward_args {
    const void* q;              /* bf16 [B,H,N,d] device */
    const void* k;              /* bf16 [B,H,N,d] device */
    const void* v;              /* bf16 [B,H,N,d] device */
    const void* x;              /* bf16 [B,N,D] device: gate input (time-modulated hidden state) */
    const void* w_gate;         /* bf16 [D] device */
    float gate_bias;
    const void* w_lin;          /* bf16 [H,d,d] device */
    void* o;                    /* bf16 [B,H,N,d] device (out) */
    int B, H, N, d, D;
    int mode;                   /* SALAD_MODE_* */
    int block;                  /* must be 64 */
    int topk;                   /* TOPK mode: key blocks per query block, 1..nb */
    int window;                 /* SWA mode: half-width, >= 0 */
    const uint8_t* space_major_heads;  /* SWA mode: HOST uint8 [H] or NULL */
    int F, Hh, Wh;              /* SWA mode: latent grid, F*Hh*Wh == N */
    float eps;                  /* linear-attention denominator eps (1e-6) */
    float gate_override;        /* NaN: use the gate; otherwise s_b = this value */
    /* Post-training branch dropping ("SALAD ... (paper.rainbus.top)" 方法步骤详情
     * step 8; "视频扩散模型中的稀疏注意力机制解析" 3.1-3.2): the linear branch
     * of sample b (state, fold and linear term) is skipped, on the device,
     * when s_b < drop_threshold; that sample's output is then O_sparse.  The
     * threshold is calibrated offline (a percentile of gate values).  0 or
     * NaN: never drop.  +-inf is rejected. */
    float drop_threshold;
    /* 3-D rotary position encoding in the linear branch ("SALAD ...
     * (paper.rainbus.top)" 方法步骤详情 step 3): 1 = on, 0 = off.  Adjacent
     * channel pairs of phi(q) and phi(k) turn by the token's frame, row and
     * column positions on the F x Hh x Wh grid (F*Hh*Wh == N required; the
     * tokens are frame-major) over three channel groups of d - 4*floor(d/6),
     * 2*floor(d/6), 2*floor(d/6) channels, pair i of a g-channel group at
     * rate rope_base^(-2i/g).  The rotation enters the numerator only:
     * O_l = (R phi(q)) H_R / (phi(q) Z + eps) with H_R = sum_j R_j phi(k_j) v_j^T
     * and Z = sum_j phi(k_j). */
    int rope3d;
    float rope_base;            /* > 1, usually 10000 */
    /* Full-width projection of the linear branch (paper.rainbus.top 方法步骤详情
     * step 4 read as one layer over all heads): bf16 [H*d, H*d] device, or
     * NULL for the per-head w_lin.  When set, w_lin is not read and
     *   O[b,:,n,:] = O_sparse + s_b * split_heads(cat_heads(O_l[b,:,n,:]) w_lin_full)
     * with cat_heads putting column h*d + c = O_l[b,h,n,c] (see
     * salad_project).  With rope3d, O_l carries the rotation as above. */
    const void* w_lin_full;
    /* Output projection (step 7): bf16 [H*d, d_out] device, or NULL.  When
     * set, out[b,n,:] = cat_heads(O[b,:,n,:]) w_out is written too; o still
     * receives O. */
    const void* w_out;
    int d_out;                  /* multiple of 64 when w_out is set */
    void* out;                  /* bf16 [B,N,d_out] device (out) when w_out is set */
    float* s_out;               /* optional device float32 [B] (out), may be NULL */
    int32_t* idx_out;           /* optional device int32 [B,H,nb,topk] (out), may be NULL */
    void* workspace;            /* device scratch, >= salad_forward_workspace_bytes() */
    size_t workspace_bytes;
    /* Optional profiling hook: NULL, or a HOST array of 5 cudaEvent_t,
     * recorded at the start (on `stream`), when the gate ends, when the
     * sparse-pattern step (selection or regrouping) ends, when the attention
     * kernel starts (every input ready), and when it ends (the full-width
     * projections, if any, follow that last event).  The gate and the
     * linear branch run on two library-owned streams forked from `stream`
     * and joined back before the attention, so only the last two events
     * bound one kernel. */
    void* const* phase_events;
    /* SWA mode, heads regrouped space-major ("视频扩散模型中的稀疏注意力机制解析
     * (ijyty.com)" 1.1): 0 (default) copies their Q, K, V space-major into
     * the workspace first; 1 regroups them inside the attention's TMA loads
     * instead (no copy): their work items and key tiles are floor(128/F)
     * whole spatial positions, floor(128/F)*F of the 128 MMA rows (requires
     * F <= 128, else SALAD_ERR_UNSUPPORTED).  Same results within rounding
     * (frame-major heads bit-identical); no copy workspace.  On a B200 the
     * copy is faster (480p ST-SWA layer: 1.02 ms with the copy, 1.63 ms in
     * the loads), so 1 exists for memory-tight callers. */
    int regroup_in_load;
} salad_forward_args;

size_t salad_forward_workspace_bytes(const salad_forward_args* args);
salad_status salad_forward(const salad_forward_args* args, salad_stream stream);

/*
 * Rotary positions with several axes (time, height, width) on queries and
 * keys, and the backward pass.  Every channel pair of a token turns by
 * angle = position[axis] * rate:
 *   y_u = x_u cos(angle) - x_w sin(angle),  y_w = x_u sin(angle) + x_w cos(angle).
 * The d channels belong to three axes, split[0] + split[1] + split[2] = d
 * (each even and >= 0; an unused axis has 0): pair i of a group of g channels
 * turns at rate base^(-2i/g).  This is the encoding that salad_forward's
 * rope3d option applies inside the linear branch ("SALAD ...
 * (paper.rainbus.top)" 方法步骤详情 step 3), for the tensors that enter the
 * sparse branch or a cache, with any split, on any axes.
 *   pairing SALAD_PAIR_ADJACENT: pair m is channels (2m, 2m + 1);
 *           SALAD_PAIR_HALVES:   pair m is channels (m, m + d/2).
 *   The first split[0]/2 pairs are axis 0's, then axis 1's, then axis 2's.
 * Positions: `positions`, or, where it is NULL, the latent grid: token n of
 * every sample stands at p = offset + n, position (p / (Hh Wh), p / Wh % Hh,
 * p % Wh) (frame-major).
 * inverse = 1 turns by -angle: the backward pass, since dx = R^T dy.
 * Angles are formed and reduced in float64, products are float32, and the
 * result is rounded once to the tensors' type.
 * Layout: rows of d contiguous elements; strides in elements of the batch,
 * head and token dimensions (multiples of 16 bytes; 0 in an input where it
 * is broadcast).  q_out may be q itself (same pointer and strides), likewise
 * k_out and k; outputs otherwise overlap no input, nor each other.  q and k
 * may be interleaved slices of one buffer.
 * d: a multiple of 16 from 16 to 256.  Needs no workspace.
 */
#define SALAD_BF16 0
#define SALAD_F16  1
#define SALAD_F32  2
#define SALAD_PAIR_ADJACENT 0
#define SALAD_PAIR_HALVES   1

typedef struct salad_strides {
    int64_t b, h, n;            /* elements between samples, heads, tokens */
} salad_strides;

typedef struct salad_rope_args {
    const void* q;              /* [B,Hq,N,d] device */
    void* q_out;                /* [B,Hq,N,d] device (out) */
    const void* k;              /* [B,Hk,N,d] device, or NULL with Hk = 0 */
    void* k_out;                /* [B,Hk,N,d] device (out), or NULL */
    salad_strides q_st, qo_st, k_st, ko_st;
    int dtype;                  /* SALAD_BF16, SALAD_F16 or SALAD_F32, of all four tensors */
    int B, Hq, Hk, N, d;
    const int32_t* positions;   /* device [N,3], or [B,N,3] with positions_batched = 1; or NULL */
    int positions_batched;
    int Hh, Wh, offset;         /* the grid, where positions is NULL; offset >= 0 */
    int split[3];
    float base;                 /* > 1 */
    int pairing;
    int inverse;
} salad_rope_args;

salad_status salad_rope(const salad_rope_args* args, salad_stream stream);

/*
 * A block cache of keys and values in 8 bits, for video generated chunk by
 * chunk (and for single tokens): tokens of a sequence are held in blocks of
 * 64.  A full ("closed") block is an e4m3 page of a shared pool with one
 * power-of-two scale for its keys and one for its values per head; the open
 * block behind it is kept in bf16, so that nothing is rounded twice.
 *   k_pages, v_pages  uint8 (e4m3 codes) [pages, H, 64, d]
 *   k_scale, v_scale  float32 [pages, H]: 2^e with the smallest e >= -100
 *                     for which every |x| <= 448 * 2^e; a value is
 *                     code * scale.  A block and head with an infinity or a
 *                     NaN gets a NaN scale and reads as NaN.
 *   k_tail, v_tail    bf16 [B, 2, H, 64, d]: the open block of each
 *                     sequence, in one of two slots
 *   page_table        int32 [B, blocks]: page of block j of sequence b
 *   seq               int32 [B, 2]: tokens held (>= 0), tail slot (0 or 1)
 * All are device pointers, contiguous, the pages and tails 16-byte aligned.
 * d is 64 or 128, pages * H below 2^31.  An appended chunk goes to the other
 * tail slot when it closes the open block, so (seq, tail) still describe the
 * cache as it was: a chunk may be appended again at the same seq (each
 * denoising step of a chunk does) and is kept by taking seq_out for the next
 * seq.
 * Pages that a call writes must differ from one another and from the pages
 * of blocks that are to be kept.
 * Table entries that are read and lie outside [0, pages) are skipped on the
 * device; lengths, slots and counts out of range are forced into it, and
 * tokens that the table has no room for (it holds 64 * blocks, and the open
 * block 63 more) are dropped.  salad_check_error then returns
 * SALAD_ERR_INVALID_ARG.
 */
typedef struct salad_cache {
    void* k_pages;
    void* v_pages;
    float* k_scale;
    float* v_scale;
    void* k_tail;
    void* v_tail;
    const int32_t* page_table;
    int B, H, d;                /* H: key/value heads */
    int pages, blocks;
} salad_cache;

/*
 * Append: token i < counts[b] of sequence b becomes token seq[b].len + i of
 * the cache.  Keys are turned by salad_rope's encoding on the way where
 * `rotate` is 1 (float32 products, rounded to bf16 before they are held): the
 * positions of the new tokens, or, where positions is NULL, the grid
 * position of p = seq[b].len + i.  Values are not turned.
 * k, v: bf16 [B,H,N,d] with strides as in salad_rope.  counts: int32 [B]
 * device or NULL (N each); rows behind a count are not read.
 * seq_out: int32 [B,2], seq after the append; may be seq itself (a second,
 * small launch advances it then) and may be NULL; it overlaps nothing else.
 */
typedef struct salad_cache_append_args {
    salad_cache cache;
    const int32_t* seq;
    int32_t* seq_out;
    const void* k;
    const void* v;
    salad_strides k_st, v_st;
    int N;
    const int32_t* counts;
    int rotate;
    const int32_t* positions;   /* device [N,3], or [B,N,3] with positions_batched = 1; or NULL */
    int positions_batched;
    int Hh, Wh;
    int split[3];
    float base;
    int pairing;
} salad_cache_append_args;

salad_status salad_cache_append(const salad_cache_append_args* args, salad_stream stream);

/*
 * Attention over the cache: o = softmax(scale q k^T + M) v, the queries being
 * the last counts[b] tokens that sequence b holds (append them first):
 * query i < counts[b] stands at p = seq[b].len - counts[b] + i.
 *   frame = F > 0: tokens come in groups of F (a latent frame; 1: one token).
 *                  A query sees its own group, as far as it is held, and
 *                  what is before it: keys j < min(len, (floor(p / F) + 1) F).
 *   frame = 0:     every query sees all held keys.
 *   window >= 0:   of the keys before the query's group (before the first
 *                  query, for frame = 0) only the last `window` are seen;
 *                  window < 0: all of them.
 * Blocks that no row sees are not read: pages before the window of the first
 * row may have been given back.
 * A row that sees no key (an empty sequence, or p < 0) is 0 with lse = -inf.
 * q, o: bf16 [B,Hq,N,d], strides as in salad_rope; Hq a multiple of the
 * cache's H, query head h reading key/value head h / (Hq / H).  lse (may be
 * NULL): float32 [B,Hq,N] contiguous, natural log of the sum of exponentials.
 * Rows behind a count are left as they are.  o and lse overlap nothing else.
 * Closed blocks are read as their exact values (code * scale), so scales are
 * powers of two from 2^-100 up, or NaN with NaN codes, as the append writes
 * them.  Softmax statistics and sums are float32.  P is rounded for the
 * product with the values: to fp16, by 2^-11 of itself, or, where it is below
 * 2^-25 of a row's largest product of weight and block scale, by 2^-36 of that.
 * In calls of few rows (up to 32 of a key head, and up to 64 where
 * B * H * blocks is small) these are 2^-29 and 2^-40, and P is rounded to bf16
 * (2^-8) with the open block's values: with 33 to 64 rows the width of the
 * table decides, and with it the last bits.  In calls of few rows on more than
 * 512 sequences the keys of a sequence and head are not split over the GPU.
 * (Rows of a key head / 256) * (blocks / 2) stays below 2^31.  Workspace:
 * salad_cache_attn_workspace_bytes(args); two calls that may overlap on the
 * GPU need two workspaces.
 */
typedef struct salad_cache_attn_args {
    salad_cache cache;
    const int32_t* seq;
    const void* q;
    void* o;
    salad_strides q_st, o_st;
    float* lse;
    int Hq, N;
    const int32_t* counts;
    int frame, window;
    float scale;                /* > 0, usually 1/sqrt(d) */
    void* workspace;
    size_t workspace_bytes;
} salad_cache_attn_args;

size_t salad_cache_attn_workspace_bytes(const salad_cache_attn_args* args);
salad_status salad_cache_attn(const salad_cache_attn_args* args, salad_stream stream);

/*
 * Reads and clears the device-side error word after synchronising `stream`.
 * Returns SALAD_ERR_TIMEOUT if any kernel gave up a bounded wait since the
 * last check; SALAD_ERR_CUDA if the stream reports an error or a kernel
 * refused to run (the attention kernel does when its dynamic shared memory
 * is not 1024-byte aligned); SALAD_ERR_INVALID_ARG if a cache operator met
 * a page, length, slot or count out of range; else SALAD_OK.
 */
salad_status salad_check_error(salad_stream stream);

/*
 * Test hook for the bounded-wait machinery: launches one CTA that waits on
 * an mbarrier nothing will ever arrive on, with a limit of `timeout_ns`
 * nanoseconds, then records SALAD_ERR_TIMEOUT in the device error word and
 * exits.  Used to check that a wait which runs out surfaces as an error
 * status rather than a hang or a trap.
 */
salad_status salad_debug_wait_timeout(unsigned long long timeout_ns, salad_stream stream);

#ifdef __cplusplus
}  /* extern "C" */
#endif

#endif  /* SALAD_H_ */
