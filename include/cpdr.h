/*
 * cpdr.h -- C ABI of the segmented ("True CP") gated delta-rule forward for
 * GB300 (sm_103a).
 *
 * The operation is the one described in the article
 *   "flash-linear-attention 上下文并行CP从 CP2TP、Ring CP 到 True CP 的设计取舍
 *    与源码实现"                                     (cited below as [FLA-CP])
 * run on ONE GPU with the sequence cut into R contiguous segments that play
 * the role of context-parallel ranks:
 *
 *   per token      S_t = (I - beta_t k_t k_t^T) Diag(alpha_t) S_{t-1} + beta_t k_t v_t^T
 *                  o_t = scale * S_t^T q_t                      alpha_t = exp(g_t)
 *   preprocess     every segment j computes, from a zero state, the state of
 *                  its trailing fragment S_ext,j (dk x dv) and the product of
 *                  that fragment's transfer matrices M_j (dk x dk), in the
 *                  chunk (WY) form with 64-token chunks    ([FLA-CP] §2.1-§2.3)
 *   merge          S_init,r = sum over predecessors: S <- M_j S + S_ext,j
 *                                                          ([FLA-CP] §2.1, §5.2)
 *   fwd            every fragment restarts from S_init (its segment's first
 *                  fragment, when it continues a sequence) or zero, and emits
 *                  o and the final state of sequences ending in it
 *                                                          ([FLA-CP] §4, §5.2)
 *
 * Conventions shared by every entry point
 * ----------------------------------------
 * Layout.  q: [B, T, Hq, dk]; k: [B, T, H, dk]; v: [B, T, H, dv];
 *          o: [B, T, Hq, dv] (Hq == H unless desc.Hq asks for grouped query
 *          heads); beta: [B, T, H];
 *          gate: [B, T, H] (scalar, GDN) or [B, T, H, dk] (per key dim, KDA),
 *          all contiguous, row-major.  Packed variable-length batches use
 *          B == 1 and global cu_seqlens ([FLA-CP] §3.1, §4 NOTE).
 *          S_ext, S_init: [R, B, H, dk, dv] fp32; M: [R, B, H, dk, dk] fp32
 *          (entry (r, b, h) belongs to segment r of row b; the layout of the
 *          gathered buffer of [FLA-CP] §2.4 with world_size = R);
 *          final_state: [N, H, dk, dv] fp32 ([N, HV, K, V] of the KDA
 *          initial_state description in hyper-parallel issue #7).  With
 *          CPDR_FLAG_STATE_V_FIRST the dk x dv states are [.., dv, dk]; with
 *          CPDR_FLAG_LAYOUT_ZIGZAG the token axis is in zigzag order and the
 *          segment axis has 2R entries.
 * Types.   q, k, v, beta, o share the input dtype (fp32 or bf16); gates are
 *          fp32 natural-log gates g = log(alpha).  Arithmetic is fp32 or
 *          bf16 tensor-core products with fp32 accumulation; the M chain is
 *          kept at fp32 accuracy ([FLA-CP] §2.2).
 * Memory.  Every tensor argument is a DEVICE pointer owned by the caller, and
 *          must be 16-byte aligned.  The library owns only the cpdr_ctx
 *          (host tables plus small device metadata allocated at create,
 *          and two copy streams and twelve events for cpdr_forward_host).
 *          No call below allocates device memory.
 * Streams. `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *          stream).  Calls enqueue work and return; they never synchronise.
 *          Every stage runs on `stream` (cpdr_forward_host also uses the
 *          context's copy streams, ordered against `stream` by events); a
 *          context must not be used from two host threads at once.
 * Errors.  Every call validates its arguments on the host before any
 *          launch and returns a cpdr_status; on failure nothing is launched
 *          and cpdr_last_error() gives a message (thread-local).  Launch
 *          failures come back as CPDR_ERR_CUDA.
 */
#ifndef CPDR_H_
#define CPDR_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    CPDR_OK = 0,
    CPDR_ERR_INVALID = 1,      /* bad shapes, cut rule violated, null/misaligned pointers */
    CPDR_ERR_UNSUPPORTED = 2,  /* valid but not implemented (e.g. dk != dv, d not in {64,128}) */
    CPDR_ERR_CUDA = 3,         /* a CUDA runtime call or kernel launch failed */
    CPDR_ERR_WORKSPACE = 4,    /* a caller-provided buffer is too small */
    CPDR_ERR_TIMEOUT = 5       /* a bounded device-side wait gave up (see cpdr_check_device_status) */
} cpdr_status;

/* desc.flags */
#define CPDR_FLAG_HOST_ONLY   (1u << 0)  /* plan only: no device tables; launch calls are rejected */
#define CPDR_FLAG_FORCE_SIMT  (1u << 1)  /* use the fp32 CUDA-core kernels even where tensor cores apply */
/* Zigzag token layout ([FLA-CP] §3.2).  Each row (or the packed batch) is cut
 * into 2R equal parts; virtual rank r holds part r followed by part 2R-1-r, and
 * the tensors q, k, v, beta, gate and o hold the R ranks' [front; back] inputs
 * side by side, rank 0 first (for R = 2: parts 0, 3, 1, 2 in memory).
 * cu_seqlens stays in sequence order.  Every part is a segment of its own, so
 * the exchange buffers have 2R entries, indexed by part in sequence order, and
 * the cut rule becomes "tokens >= 2R and divisible by 2R". */
#define CPDR_FLAG_LAYOUT_ZIGZAG (1u << 2)
/* state_v_first ([FLA-CP] §5.1; [N, HV, V, K] of hyper-parallel issue #7):
 * every dk x dv state buffer -- S_ext, S_init and final_state -- is stored
 * transposed, [.., dv, dk].  M keeps its [.., dk, dk] layout. */
#define CPDR_FLAG_STATE_V_FIRST (1u << 3)

/* desc.gate_kind */
#define CPDR_GATE_SCALAR  0   /* GDN: g [B, T, H] */
#define CPDR_GATE_PER_DIM 1   /* KDA: gk [B, T, H, dk] */

/* desc.in_dtype */
#define CPDR_DTYPE_F32  0
#define CPDR_DTYPE_BF16 1

typedef struct {
    int32_t B, H, dk, dv;   /* batch rows, heads, key dim, value dim */
    int32_t R;              /* virtual context ranks: R contiguous segments per row (or 2R
                               zigzag pieces, see CPDR_FLAG_LAYOUT_ZIGZAG) */
    int32_t num_seqs;       /* N: sequences (== B without cu_seqlens) */
    int64_t T;              /* tokens per row, or total tokens when packed */
    const int64_t *cu_seqlens_host; /* NULL: B rows of T tokens; else N+1 global offsets
                                       (host memory, read during create only), B == 1 */
    int32_t gate_kind;      /* CPDR_GATE_* */
    int32_t in_dtype;       /* CPDR_DTYPE_* */
    uint32_t flags;         /* CPDR_FLAG_* */
    float scale;            /* output scale */
    int32_t Hq;             /* query heads of q and o (GQA, [FLA-CP] §5.1): 0 or H for none,
                               else a multiple G*H; q head hq reads the state of head hq / G,
                               while k, v, beta, gate and every state keep H heads */
    int32_t conv_width;     /* causal conv1d kernel size W for cpdr_conv1d_fwd (the
                               conv1d_kernel_size of [FLA-CP] §3.1-§3.2): 0 = no conv path,
                               else 1..8 */
} cpdr_desc;

typedef struct cpdr_ctx cpdr_ctx;

/* One local fragment: the intersection of a segment with a sequence. */
typedef struct {
    int64_t tok0;    /* first token on the flattened [B*T] token axis, where it is in
                        memory (zigzag layout: its memory position, not its sequence position) */
    int32_t len;     /* tokens (>= 1) */
    int32_t seg;     /* segment buffer index r*B + b */
    int32_t seq;     /* sequence index */
    int32_t flags;   /* CPDR_FRAG_* */
} cpdr_fragment;

#define CPDR_FRAG_CONT_PREV 1   /* continues a sequence from segment r-1: starts from S_init[seg] */
#define CPDR_FRAG_CONT_NEXT 2   /* continues into segment r+1: pre-processed into S_ext/M[seg] */
#define CPDR_FRAG_ENDS_SEQ  4   /* the sequence ends here: final_state[seq] is written */

/*
 * Build the partition plan ([FLA-CP] §3.2-§3.3: contiguous layout, the cut
 * rule "tokens >= R and divisible by R" per row, searchsorted-style
 * intersection of the global cu_seqlens with each segment) and upload its
 * small device tables (unless CPDR_FLAG_HOST_ONLY).  The plan is built once
 * and reused, like the memoised context of [FLA-CP] §3.3.
 * Errors: CPDR_ERR_INVALID (cut rule, non-monotone cu_seqlens, B != 1 with
 * cu_seqlens, non-positive sizes), CPDR_ERR_UNSUPPORTED (dk != dv or
 * d not in {64, 128}), CPDR_ERR_CUDA (table upload).  *out is NULL on error.
 */
cpdr_status cpdr_ctx_create(const cpdr_desc *desc, cpdr_ctx **out);

/* Free the context and its device tables.  NULL is accepted. */
void cpdr_ctx_destroy(cpdr_ctx *ctx);

/* Byte sizes of the caller-owned exchange buffers S_ext, M, S_init and of
 * final_state.  Any pointer may be NULL. */
cpdr_status cpdr_buffer_sizes(const cpdr_ctx *ctx, size_t *sext_bytes, size_t *m_bytes,
                              size_t *sinit_bytes, size_t *final_bytes);

/* Plan introspection (host memory): number of fragments, and a copy of the
 * fragment table into out[0 .. min(cap, n)). */
cpdr_status cpdr_plan_num_fragments(const cpdr_ctx *ctx, int32_t *n);
cpdr_status cpdr_plan_fragments(const cpdr_ctx *ctx, cpdr_fragment *out, int32_t cap);

/* Plan counters (host memory): out[0] fragments, [1] pre-processed
 * fragments, [2] merge chains, [3] segments with zeroed S_ext/M, [4]
 * segments with zeroed S_init, [5] empty sequences, [6] kernel launches per
 * preprocess+merge+fwd step, [7] 1 if the tensor-core kernels are selected. */
cpdr_status cpdr_plan_counts(const cpdr_ctx *ctx, int32_t out[8]);

/*
 * WY build ([FLA-CP] §2.2 and the recompute_w_u step of its §4 Code Flow):
 * for every 64-token chunk of every fragment and every head,
 *     A_ij = beta_i exp(G_i - G_j) k_i . k_j  (j < i),   T = (I + A)^-1,
 * with G the in-chunk cumulative log gate, and the tiles W and U are built
 * from:  T' = T diag(beta)  (U = T' V)  and  T'' = T diag(beta gamma)
 * (W = T'' K, gamma_j = exp(G_j)).  Each (chunk, head) gets three 64 x 64
 * bf16 tiles -- T', T'' rounded (hi) and T'' - hi rounded (lo) -- stored as
 * 8 KiB 128-byte-swizzled images, in the chunk order of the plan's fragment
 * table, heads innermost.  The chunk recurrences of cpdr_preprocess and
 * cpdr_fwd read them (the triangular solve is independent across chunks, so
 * it runs here once, fully parallel, instead of inside every chain).
 * cpdr_wy_bytes() gives the workspace size: 24 KiB per (chunk, head) on the
 * tensor-core path (bf16, dk = dv = 128, scalar gate), 0 otherwise (then
 * this call does nothing and `wy` may be NULL).
 * Per-dim gate (KDA) on the tensor-core path: the gate cannot be applied
 * inside the chunk recurrence as a scalar, so this step also pre-gates the
 * operands, as [FLA-CP] §2.3 does at the WY stage (kg = k 2^(g_last - g),
 * qg = q 2^g): per (chunk, head) it writes, after the three tiles above
 * (built with gamma = 1), the per-dim chunk decay 2^(G_C), the bf16 tiles
 * k 2^G (hi, lo), k 2^(G_C - G) (hi, lo), q 2^G and the masked intra-chunk
 * product (Q K^T ⊙ Lambda) -- 113 KiB per (chunk, head).  With grouped
 * query heads (Hq = G H) the unit holds q 2^G and the product of its state's
 * first query head; those of query heads 1 .. G-1 (24 KiB each) follow all
 * units, [chunk][head][G - 1].
 * In: q (device; read only for the per-dim gate, else may be NULL), k,
 * beta, gate (device).  Out: wy (device, caller-owned).
 */
cpdr_status cpdr_wy_bytes(const cpdr_ctx *ctx, size_t *bytes);
cpdr_status cpdr_wy_build(const cpdr_ctx *ctx, const void *q, const void *k, const void *beta,
                          const float *gate, void *wy, void *stream);

/*
 * Pre-process ([FLA-CP] §2.1-§2.3, pre_process_fwd in its Code Flow of §4):
 * for every segment whose trailing fragment continues into the next
 * segment, S_ext = state of that fragment from zero, M = chained transfer
 * matrix  M <- (Diag(gamma^C) - (Gamma ⊙ K)^T W) M  over its 64-token
 * chunks.  Entries of segments with no continuing fragment are zeroed.
 * In: k, v, beta, gate (device); wy: the tiles cpdr_wy_build wrote for the
 * same k, beta and gate (NULL when cpdr_wy_bytes() is 0).  Out: S_ext, M
 * (device, sizes from cpdr_buffer_sizes).
 */
cpdr_status cpdr_preprocess(const cpdr_ctx *ctx, const void *k, const void *v, const void *beta,
                            const float *gate, const void *wy, float *S_ext, float *M, void *stream);

/*
 * Merge ([FLA-CP] §2.1; ownership rule of §5.2): for every segment r whose
 * first fragment continues a sequence begun in segment r - n_pre,
 *     S = 0;  for j = r - n_pre .. r - 1:  S <- M_j S + S_ext,j
 * and S_init[r] = S; all other entries are zeroed.  Evaluated as one
 * sequential scan per sequence (equal in exact arithmetic).  Precision: on
 * the tensor-core path (bf16 inputs, d = 128) each product M_j S runs on the
 * tensor cores with M_j and S split into bf16 hi/lo pairs and fp32
 * accumulation (about 2^-16 relative per step); otherwise all fp32.
 * In: S_ext, M (device, as cpdr_preprocess wrote them).  Out: S_init
 * (device).  Errors: CPDR_ERR_INVALID, CPDR_ERR_CUDA.
 */
cpdr_status cpdr_merge(const cpdr_ctx *ctx, const float *S_ext, const float *M, float *S_init,
                       void *stream);

/*
 * Forward ([FLA-CP] §4, chunk_gated_delta_rule_fwd_h plus the output step):
 * every fragment runs the 64-token chunk recurrence from S_init[seg] (first
 * fragment continuing a sequence) or zero, writes o = scale * S_t^T q_t per
 * token and, when its sequence ends there, final_state[seq].
 * wy: as for cpdr_preprocess.  final_state may be NULL.
 */
cpdr_status cpdr_fwd(const cpdr_ctx *ctx, const void *q, const void *k, const void *v,
                     const void *beta, const float *gate, const void *wy, const float *S_init, void *o,
                     float *final_state, void *stream);

/*
 * Causal depthwise conv1d over the token axis, the layer step before the
 * delta rule, on the context's segments ([FLA-CP] §2.4: the conv sees only
 * the W - 1 tokens before each token, so a rank takes the tail of the
 * previous rank's tokens; §3.2-§3.3: conv1d_kernel_size, pre_num_conv_tokens).
 * Per channel c and token t of a sequence (positions before the sequence
 * start read as zero):
 *     y[t, c] = act( bias[c] + sum_{i=0}^{W-1} weight[c, i] * x[t - (W-1) + i, c] )
 * act = identity (activation 0) or SiLU, z * sigmoid(z) (activation 1).
 * On one device the previous segment's tail is read where it lies in memory
 * (in the zigzag layout, another rank's part), so no exchange buffer exists.
 * Layout: x, y [B, T, channels] in the context's token order and input dtype
 * (fp32 or bf16), contiguous; weight [channels, W] fp32; bias [channels] fp32
 * or NULL.  W = desc.conv_width (> 0).  channels % 8 == 0, 1 <= channels.
 * Arithmetic in fp32, y rounded once.  y must not overlap x.
 * Errors: CPDR_ERR_INVALID (context without a conv width, bad channels or
 * activation, null or misaligned pointers), CPDR_ERR_CUDA.
 */
cpdr_status cpdr_conv1d_fwd(const cpdr_ctx *ctx, const void *x, const float *weight, const float *bias,
                            int32_t channels, int32_t activation, void *y, void *stream);

/*
 * Backward ([FLA-CP] §2.2 and §4 split it into a pre-process, the merge run
 * in reverse with the transposed transfer matrices, and state-gradient
 * chains): the gradients of  sum_t <do_t, o_t> + sum_n <dht_n, final_state_n>
 * with respect to q, k, v, beta and the gate, for the same inputs the
 * forward ran on.
 *   1. each segment's first fragment that continues a sequence runs the
 *      reverse chain from its local end gradient (dht if its sequence ends
 *      there, else 0) and keeps the state gradient at its start, dS_ext;
 *   2. per sequence crossing cuts:  G = dS_ext[r1];
 *      for j = r1-1 .. r0+1:  G <- M_j^T G + dS_ext[j]  (the gradient at the
 *      end of every continuing fragment);
 *   3. every fragment runs the reverse chain from that end gradient (or dht,
 *      or 0) and writes the input gradients.
 * For bf16 inputs and dk = dv = 128 (either gate) the chains run in chunk form on the tensor
 * cores: the forward is recomputed with every chunk's starting state and
 * Delta kept, the state-gradient chain runs chunk by chunk in reverse
 * (tcgen05), the reverse merge on the tensor cores, and a parallel kernel
 * forms the input gradients of every (chunk, head) (for the per-dim gate
 * with its factors folded into the operands); the workspace then holds the
 * WY tiles (the per-dim gate's units), the fp32 inverse T and four fp32
 * tensors per (chunk, head) (about 216 KiB each).  Otherwise the reverse
 * chain is the per-token chain rule, on CUDA cores in fp32, with the
 * forward states recomputed from S_init per token.  With grouped query
 * heads (Hq = G H) each state's chain takes the G query heads that read it
 * ([FLA-CP] §5.1): its state gradient collects scale q do^T of every one of
 * them, and each gets its own dq (on the tensor cores the chunk-form
 * state-gradient chain, linear in those terms, runs once per query head and
 * sums, and the input-gradient kernel makes a pass per query head).
 * In (device): q, k, v, beta, gate and do ([B, T, Hq, dv], the input dtype)
 * as for cpdr_fwd; dht [N, H, dk, dv] fp32 (with CPDR_FLAG_STATE_V_FIRST
 * [N, H, dv, dk]) or NULL (zero); S_init and M as cpdr_merge and
 * cpdr_preprocess left them for these inputs.  Out (device, fp32, written
 * here): dq [B, T, Hq, dk], dk [B, T, H, dk], dv [B, T, H, dv], dbeta
 * [B, T, H], dgate (the gate's shape).  workspace: device memory of
 * cpdr_bwd_workspace_bytes() bytes, 256-byte aligned.
 * Errors: CPDR_ERR_UNSUPPORTED when the G query heads' rows of one chunk do
 * not fit the CUDA-core chain's shared memory (at d = 128: G above 8 for
 * bf16 with the scalar gate, 6 with the per-dim gate; 4 and 3 for fp32);
 * CPDR_ERR_WORKSPACE; CPDR_ERR_INVALID; CPDR_ERR_CUDA.
 */
cpdr_status cpdr_bwd_workspace_bytes(const cpdr_ctx *ctx, size_t *bytes);
cpdr_status cpdr_bwd(const cpdr_ctx *ctx, const void *q, const void *k, const void *v, const void *beta,
                     const float *gate, const void *dout, const float *dht, const float *S_init, const float *M,
                     float *dq, float *dk, float *dv, float *dbeta, float *dgate, void *workspace,
                     size_t workspace_bytes, void *stream);

/*
 * Layer steps around the token mixers
 * -----------------------------------
 * The calls below are the steps a layer takes before, beside and after the
 * delta rule (no counterpart in the article).  They take the context for its
 * input dtype (and, for the recurrence, its sequences and token layout), its
 * device and its status word.  Unlike cpdr_bwd, whose gradients are all fp32,
 * the gradient of a tensor has the tensor's own type here, so that it feeds
 * the step before it as it is.  Sums, statistics and states are fp32 and run
 * in a fixed order: the same call on the same inputs gives the same bits.
 * All tensors are contiguous; outputs must not overlap inputs or one another
 * except where "in place" is said.  The calls allocate nothing, keep nothing
 * between calls and can be captured into a graph; calls that share a
 * workspace must not overlap on the GPU.
 */

/*
 * Gated linear recurrence, the diagonal sibling of the delta rule: per
 * channel c and token t of a sequence, with a_t = exp(gate_t),
 *     h_t = a_t h_{t-1} + x_t,    y_t = h_t,
 * from h0 (or zero) at the sequence's start; hT is the state behind its last
 * token (h0, or zero, for an empty sequence).  gate is a natural-log gate, at
 * most 88; -infinity is one (a_t = 0: the state is dropped); from -87.4 down
 * a_t is 0.  x and h0 are finite.  Positive gates that sum to more than 1 over
 * 16 tokens cost time: up to 1024 tokens around them run 16 at a time, one group
 * behind the other (so do all that follow a state that is not finite).  What
 * falls below 1e-17 of the largest state of the last 1024 tokens counts as zero.
 * Sequences and token layout are the context's (packed batches, zigzag); its
 * segments play no part.
 * Layout: x, y [B, T, channels] in the context's token order and input dtype;
 * gate [B, T, channels] fp32; h0, hT [N, channels] fp32, either may be NULL
 * (hT may be h0 itself); channels % 8 == 0, at most 2^24.
 * carry (NULL, or cpdr_glr_carry_bytes() bytes): what cpdr_glr_bwd needs of
 * the forward, fp32 [groups, channels]: the state before every 16th token of
 * each sequence (its tokens 0, 16, 32, ...), sequence after sequence.
 */
cpdr_status cpdr_glr_carry_bytes(const cpdr_ctx *ctx, int32_t channels, size_t *bytes);
cpdr_status cpdr_glr_fwd(const cpdr_ctx *ctx, const void *x, const float *gate, const float *h0, int32_t channels,
                         void *y, float *hT, float *carry, void *stream);

/*
 * Plan introspection: how cpdr_glr_fwd (backward 0) or cpdr_glr_bwd (1) runs
 * over the context's sequences with that many channels.  out = {CTAs of a
 * cluster, CTAs of an SM that the choice counts on, CTAs of an SM that the
 * device holds (0 for a host-only context)}.
 */
cpdr_status cpdr_plan_glr(const cpdr_ctx *ctx, int32_t channels, int32_t backward, int32_t out[3]);

/*
 * Its backward: the gradients of  sum_t <dy_t, y_t> + sum_n <dhT_n, hT_n>,
 *     dh_t = dy_t + a_{t+1} dh_{t+1}  (dhT in the place of the last product),
 *     dx_t = dh_t,   dgate_t = dh_t a_t h_{t-1},   dh0 = a_0 dh_0.
 * x, gate and carry as the forward took and left them; dy, dx [B, T,
 * channels] in the input dtype; dgate [B, T, channels] fp32; dhT (NULL: zero)
 * and dh0 (or NULL) [N, channels] fp32 (dh0 may be dhT itself).
 */
cpdr_status cpdr_glr_bwd(const cpdr_ctx *ctx, const void *x, const float *gate, const float *carry, const void *dy,
                         const float *dhT, int32_t channels, void *dx, float *dgate, float *dh0, void *stream);

/*
 * Its single-token form, for decoding over a pool of state slots: row i of x,
 * gate and y [n, channels] is the next token of the sequence whose state is
 * slot slots[i] (int32, device; NULL: slot i) of state [num_slots, channels]
 * fp32.  state_out gets the new states of the slots that occur; it may be
 * state itself (in place), and its other slots are left as they were.  Rows
 * whose slot is outside 0 .. num_slots - 1 (padding, -1) do nothing: their y
 * is left as it was.  Rows of the same slot are consecutive tokens of its
 * sequence, in row order.  0 <= n <= 65535.  The context's sequences play no
 * part, only its dtype.
 */
cpdr_status cpdr_glr_step(const cpdr_ctx *ctx, const void *x, const float *gate, const float *state,
                          float *state_out, const int32_t *slots, int32_t n, int32_t num_slots, int32_t channels,
                          void *y, void *stream);

/*
 * RMS norm with the residual's addition.  Per row of `width` elements, with
 * s = x + residual (s = x when residual is NULL),
 *     y_i = s_i weight_i / sqrt(mean(s^2) + eps).
 * x, residual, sum_out, y [rows, width] in the context's input dtype; weight
 * [width] fp32.  sum_out (or NULL) receives s, rounded once; y is computed
 * from the unrounded sum.  y8 and scale (both or neither; y may be NULL then,
 * or given too): y in 8 bits, e4m3 [rows, width], with one fp32 scale per row,
 *     scale = max(max_i |y_i| / 448, 2^-126),   y8_i = e4m3(y_i (1 / scale)),
 * rounded to nearest even, 1 / scale rounded to fp32 first (a quotient next to a
 * tie may go the other way); a row with a NaN or an infinity has a NaN scale.
 * Squares are summed in fp32: |s| up to 1e17 (a row whose sum passes fp32's
 * range gives y = 0), and with eps = 0 from 1e-18 up.
 * sum_out and y may each be x or residual (in place; not both the same).
 * rows >= 0, width % 8 == 0, width <= 16384, 0 <= eps <= 1.  A row is
 * anything that is normalised as one: a token, or a head of d elements.
 */
cpdr_status cpdr_rmsnorm_fwd(const cpdr_ctx *ctx, int64_t rows, int32_t width, const void *x, const void *residual,
                             const float *weight, float eps, void *sum_out, void *y, void *y8, float *scale,
                             void *stream);

/*
 * Its backward, from s (sum_out, or x where there was no residual), dy and,
 * unless NULL, the gradient dsum that reaches s past the norm:
 *     ds_i = rstd (w_i dy_i - s_i rstd^2 mean(s w dy)) + dsum_i,
 *     dweight_i = sum over rows of dy_i s_i rstd,   rstd = 1/sqrt(mean(s^2)+eps).
 * ds is the gradient of x and of residual alike; it may be dy or dsum (in
 * place).  dy, dsum, ds [rows, width] in the input dtype; dweight [width]
 * fp32.  workspace: cpdr_rmsnorm_bwd_workspace_bytes() bytes, 16-byte
 * aligned.
 */
cpdr_status cpdr_rmsnorm_bwd_workspace_bytes(const cpdr_ctx *ctx, int64_t rows, int32_t width, size_t *bytes);
cpdr_status cpdr_rmsnorm_bwd(const cpdr_ctx *ctx, int64_t rows, int32_t width, const void *s, const float *weight,
                             float eps, const void *dy, const void *dsum, void *ds, float *dweight, void *workspace,
                             size_t workspace_bytes, void *stream);

/*
 * Layer norm with the residual's addition.  Per row of `width` elements, with
 * s = x + residual (s = x when residual is NULL) and m = mean(s),
 *     y_i = (s_i - m) weight_i / sqrt(mean((s - m)^2) + eps) + bias_i.
 * As cpdr_rmsnorm_fwd in all else: types, sum_out, the 8-bit output with its
 * scales, the in-place forms, sizes and |s|; weight [width] and bias [width]
 * fp32, bias or NULL.  With eps = 0 a row without variance has no value.
 */
cpdr_status cpdr_layernorm_fwd(const cpdr_ctx *ctx, int64_t rows, int32_t width, const void *x, const void *residual,
                               const float *weight, const float *bias, float eps, void *sum_out, void *y, void *y8,
                               float *scale, void *stream);

/*
 * Its backward, from s (sum_out, or x where there was no residual), dy and,
 * unless NULL, the gradient dsum that reaches s past the norm: with
 * rstd = 1/sqrt(mean((s - m)^2) + eps), xh = (s - m) rstd and u = weight dy,
 *     ds_i = rstd (u_i - mean(u) - xh_i mean(u xh)) + dsum_i,
 *     dweight_i = sum over rows of dy_i xh_i,   dbias_i = sum over rows of dy_i.
 * ds is the gradient of x and of residual alike; it may be dy or dsum (in
 * place).  dy, dsum, ds [rows, width] in the input dtype; dweight and dbias
 * [width] fp32, dbias or NULL.  workspace: cpdr_layernorm_bwd_workspace_bytes()
 * bytes, 16-byte aligned.
 */
cpdr_status cpdr_layernorm_bwd_workspace_bytes(const cpdr_ctx *ctx, int64_t rows, int32_t width, size_t *bytes);
cpdr_status cpdr_layernorm_bwd(const cpdr_ctx *ctx, int64_t rows, int32_t width, const void *s, const float *weight,
                               float eps, const void *dy, const void *dsum, void *ds, float *dweight, float *dbias,
                               void *workspace, size_t workspace_bytes, void *stream);

/*
 * Embedding lookup with scaling:  y_i = scale table[tokens_i].
 * tokens [n] int32 (4-byte aligned); table [vocab, width] and y [n, width] in
 * the context's input dtype; a row whose token lies outside 0 .. vocab - 1
 * (padding, -1) is zero.  scale is finite; y is rounded once.
 * 0 <= n <= 2^30; 1 <= vocab <= 2^30; width % 8 == 0, at most 2^20.
 */
cpdr_status cpdr_embed_fwd(const cpdr_ctx *ctx, const int32_t *tokens, int64_t n, const void *table, int32_t vocab,
                           int32_t width, float scale, void *y, void *stream);

/*
 * Its gradient:  dtable_v = scale times the sum over the rows with tokens_i = v
 * of dy_i.  The whole of dtable [vocab, width] is written, zeros where v does
 * not occur; rows whose token lies outside the table add nothing.  dy [n,
 * width] and dtable in the input dtype; sums in fp32, rounded once.  A token's
 * rows are added in the order of the batch, in groups that depend on the
 * tokens, the sizes and the GPU's number of multiprocessors alone.  workspace:
 * cpdr_embed_bwd_workspace_bytes() bytes, 16-byte aligned.
 */
cpdr_status cpdr_embed_bwd_workspace_bytes(const cpdr_ctx *ctx, int64_t n, int32_t vocab, int32_t width, size_t *bytes);
cpdr_status cpdr_embed_bwd(const cpdr_ctx *ctx, const int32_t *tokens, int64_t n, int32_t vocab, int32_t width,
                           float scale, const void *dy, void *dtable, void *workspace, size_t workspace_bytes,
                           void *stream);

/*
 * The gated delta rule token by token, its serving form, over a pool of state
 * slots: row i of q [n, Hq, dk], k [n, H, dk], v [n, H, dv], beta [n, H], gate
 * ([n, H] or [n, H, dk]) and o [n, Hq, dv] is the next token of the sequence
 * whose states are slot slots[i] (int32, device; NULL: slot i) of state
 * [num_slots, H, dk, dv] fp32 ([.., dv, dk] with CPDR_FLAG_STATE_V_FIRST): what
 * cpdr_fwd leaves in final_state, and goes on from.  Per state head,
 *     S <- (I - beta k k^T) Diag(alpha) S + beta k v^T,   o = scale S^T q,
 * alpha = exp(gate) (-infinity: the state is dropped).  Heads, dims, gate kind,
 * input dtype, scale and state layout are the context's; its sequences and
 * segments play no part.  state_out gets the new states of the slots that
 * occur; it may be state itself (in place), and its other slots are left as
 * they were.  Rows whose slot is outside 0 .. num_slots - 1 (padding, -1) do
 * nothing: their o is left as it was.  Rows of the same slot are consecutive
 * tokens of its sequence, in row order; its states stay on the chip between
 * them.  0 <= n <= 65535.  States and sums are fp32, o is rounded once; states
 * and inputs are finite (a dropped infinity is 0 times infinity).  All rows'
 * slots are looked through for each row that the one before does not tell of:
 * past some thousand rows that shows (one token a slot, H = 1, dk = 64: 4096
 * rows 29 us and 24 without slots, 65535 rows 1170 and 320).  A state is read
 * by one row of its slot alone, whatever the rows' order.
 */
cpdr_status cpdr_delta_step(const cpdr_ctx *ctx, const void *q, const void *k, const void *v, const void *beta,
                            const float *gate, const float *state, float *state_out, const int32_t *slots, int32_t n,
                            int32_t num_slots, void *o, void *stream);

/*
 * The causal conv1d token by token, over a pool of windows: row i of x and y
 * [n, channels] is the next token of the sequence whose last W - 1 inputs,
 * oldest first (zeros before its start), are slot slots[i] of state
 * [num_slots, W - 1, channels] in the input dtype,
 *     y = act( bias + sum_{i<W-1} weight[c, i] state[i, c] + weight[c, W-1] x[c] ),
 * and the window moves on by one.  weight, bias, activation and W =
 * desc.conv_width as for cpdr_conv1d_fwd; slots, state_out, n and rows without
 * a slot as for cpdr_delta_step (the search here: 512 channels, one token a
 * slot, 8192 rows 26 us and 13 without slots, 65535 rows 1030 and 82).  With
 * W = 1 there is no state: state and state_out may be NULL.  channels % 8 == 0,
 * at most 2^24.
 */
cpdr_status cpdr_conv1d_step(const cpdr_ctx *ctx, const void *x, const float *weight, const float *bias,
                             const void *state, void *state_out, const int32_t *slots, int32_t n, int32_t num_slots,
                             int32_t channels, int32_t activation, void *y, void *stream);

/*
 * Matrix product with bias, activation and residual in its epilogue:
 *     z = x w^T + bias,   y = act(z) + residual,
 * x [rows, K], w [N, K], y and residual [rows, N], z [rows, N] or NULL (the
 * value before the activation, which cpdr_linear_bwd takes), bias [N] fp32 or
 * NULL, residual or NULL (y may be residual: in place); act = identity (0),
 * SiLU (1) or GELU z Phi(z) (2).  bf16 contexts only; x and w are bf16, or,
 * when x_scale [rows] and w_scale [N] (fp32, both or neither) are given,
 * e4m3, standing for x[i, k] x_scale[i] and w[n, k] w_scale[n] (what
 * cpdr_rmsnorm_fwd leaves in y8 and scale is such an x).  The products are
 * accumulated in fp32; y and z are rounded once (act itself is off by up to
 * 1e-6 |z|, and where it falls off, z < -3, by up to 2e-4 of its value; SiLU
 * below z = -87 and GELU below z = -13 are 0).
 * rows >= 0; K % 8 == 0 (e4m3: K % 16 == 0); N % 8 == 0; both at most 2^23.
 * Errors: CPDR_ERR_UNSUPPORTED (an fp32 context), CPDR_ERR_INVALID,
 * CPDR_ERR_CUDA.
 */
cpdr_status cpdr_linear_fwd(const cpdr_ctx *ctx, int64_t rows, int32_t K, int32_t N, const void *x, const void *w,
                            const float *x_scale, const float *w_scale, const float *bias, int32_t activation,
                            const void *residual, void *z, void *y, void *stream);

/*
 * Plan introspection: the form in which cpdr_linear_fwd runs these sizes (and
 * cpdr_linear_bwd the input gradient of w [K, N]).  out = {rows of x in a tile
 * of the form for few rows, 0: the form for many; CTAs that K is split over}.
 */
cpdr_status cpdr_plan_linear(const cpdr_ctx *ctx, int64_t rows, int32_t K, int32_t N, int32_t e4m3, int32_t out[2]);

/*
 * Its backward for bf16 operands, from dy [rows, N] bf16 (which is also the
 * residual's gradient):
 *     dz = dy act'(z),   dx = dz w,   dw = dz^T x,   dbias = sum over rows of dz.
 * z as the forward left it (NULL without an activation); dx [rows, K] and dw
 * [N, K] bf16, dbias [N] fp32, each NULL where it is not wanted (then the
 * operand that it alone needs may be NULL too).  dz is rounded to bf16 for
 * the two products; dbias is summed from the unrounded dz.  workspace:
 * cpdr_linear_bwd_workspace_bytes() bytes, 16-byte aligned.
 */
cpdr_status cpdr_linear_bwd_workspace_bytes(const cpdr_ctx *ctx, int64_t rows, int32_t K, int32_t N,
                                            int32_t activation, size_t *bytes);
cpdr_status cpdr_linear_bwd(const cpdr_ctx *ctx, int64_t rows, int32_t K, int32_t N, const void *x, const void *w,
                            const void *z, const void *dy, int32_t activation, void *dx, void *dw, float *dbias,
                            void *workspace, size_t workspace_bytes, void *stream);

/* pre_num_conv_tokens ([FLA-CP] §3.3) per segment, host memory: how many of
 * the W - 1 tokens before segment s's start belong to its first sequence
 * (0 when the segment starts a sequence), out[0 .. min(cap, nseg)). */
cpdr_status cpdr_plan_conv_tokens(const cpdr_ctx *ctx, int32_t *out, int32_t cap);

/*
 * Whole path from HOST memory: copies q, k, v, beta, gate into the
 * caller-provided device workspace, runs the WY build, preprocess, merge and fwd on
 * `stream`, and copies o and final_state back (host pointers; use pinned
 * memory for asynchronous copies).  Returns after enqueuing; the caller
 * synchronises the stream before reading o.  The workspace must hold
 * cpdr_host_workspace_bytes() bytes (256-byte aligned device memory).
 * The host-to-device copies run on the context's copy stream, ordered after
 * all work enqueued on `stream` before the call, in the order the stages
 * need them (k, beta, gate, then v, then q in four groups of consecutive
 * tokens); each stage waits on `stream` for its own inputs only, the
 * forward runs group by group, and each group's o is copied back on the
 * context's output stream while the next group runs; `stream` waits for
 * the last copy before anything later on it.
 */
cpdr_status cpdr_host_workspace_bytes(const cpdr_ctx *ctx, size_t *bytes);
cpdr_status cpdr_forward_host(const cpdr_ctx *ctx, const void *q, const void *k, const void *v,
                              const void *beta, const float *gate, void *o, float *final_state,
                              void *device_workspace, size_t workspace_bytes, void *stream);

/*
 * Allocation-free whole path (no counterpart in the article: it is an
 * interface for callers that cannot allocate device memory, e.g. code inside
 * a runtime that owns all device memory through its own pool or static
 * memory plan).  Runs the WY build, preprocess, merge and fwd like the calls
 * above, but keeps everything except the caller's inputs and outputs -- the
 * WY tiles, the exchange buffers S_ext, M, S_init, the plan tables and the
 * status word of the bounded waits -- in one file-scope device array of
 * 32 MiB per device
 * (held by every GPU that loads the library until the process exits).  It
 * calls no cudaMalloc, cudaFree or other allocating routine, and accepts a
 * context created with CPDR_FLAG_HOST_ONLY.
 * In: q, k, v, beta, gate (device).  Out: o, final_state (device; final_state
 * may be NULL).  Errors: CPDR_ERR_WORKSPACE when the problem needs more than
 * the array holds (R*B*H*dk*(2*dv + dk)*4 bytes of exchange buffers, the WY
 * tiles of cpdr_wy_bytes() and the plan tables), CPDR_ERR_INVALID / CPDR_ERR_CUDA as for the other calls.
 * Set-up: the first call on a device looks up the array's device address
 * (cudaGetSymbolAddress) with that device current; make that first call
 * before any stream capture.  Every call shares the one array and overwrites
 * it: calls whose work overlaps on the GPU (other streams, other contexts)
 * race.  The context is only read (the call runs its stages on a private
 * view of it that shares the plan), so other calls may use the context
 * meanwhile.  The plan tables are copied into the array from pageable host
 * memory on `stream`, so the call may block the host until those small
 * copies are staged.  A bounded wait that expires inside this call records
 * its code in the context's status word when the context has one, else (a
 * CPDR_FLAG_HOST_ONLY context) in the array's status word, which is cleared
 * at the start of every call: read it with cpdr_check_device_status on the
 * same context and device before the next allocation-free call there.
 */
cpdr_status cpdr_forward_noalloc(const cpdr_ctx *ctx, const void *q, const void *k, const void *v,
                                 const void *beta, const float *gate, void *o, float *final_state, void *stream);

/*
 * Device status: kernels that wait on an mbarrier do so for a bounded number
 * of polls; when a wait gives up, the kernel records a nonzero code in the
 * context's device status word and returns instead of hanging.  This call
 * synchronises `stream`, reads and clears that word, and returns
 * CPDR_ERR_TIMEOUT (with the code in the message) if it was set.  For a
 * context created with CPDR_FLAG_HOST_ONLY, whose kernels can only have run
 * through cpdr_forward_noalloc, it reads and clears the status word of that
 * entry point's array on the current device (CPDR_OK if the entry point has
 * not run on this device).
 */
cpdr_status cpdr_check_device_status(const cpdr_ctx *ctx, void *stream);

/*
 * Self-test of the bounded-wait failure path (no counterpart in the article):
 * launches one warp that waits, for at most `max_cycles` SM clock cycles
 * (0 < max_cycles <= 4e9, about 2 s at the maximum clock), on an mbarrier
 * phase that nothing completes, then records code 1 at site 99 in the
 * context's device status word and returns -- what every bounded wait of the
 * library does when it gives up.  cpdr_check_device_status then reports
 * CPDR_ERR_TIMEOUT and clears the word; the context stays usable.  No fault,
 * trap or unbounded wait is involved.
 */
cpdr_status cpdr_selftest_wait_timeout(const cpdr_ctx *ctx, long long max_cycles, void *stream);

/* Thread-local message for the last non-OK status of this thread. */
const char *cpdr_last_error(void);

/* Library version string. */
const char *cpdr_version(void);

#ifdef __cplusplus
}
#endif
#endif /* CPDR_H_ */
