/*
 * cpattn.h - C ABI of libcpattn.so: context-parallel causal attention run as a
 * Q-KV task graph on one GB300 GPU (sm_103a).
 *
 * The method, in the words of the pages it follows:
 *  - "Context Parallelism (CP)" (llm-infra-atlas, parallel/04_cp), §2.1: the
 *    query sequence is cut into Q blocks and the key/value sequence into KV
 *    segments; every (Q block, KV segment) pair that the mask does not empty
 *    is an edge of a bipartite task graph, and each edge is one
 *    TileAttention(Q_i, K_j, V_j, M_ij) that yields a partial state
 *    (O_ij, L_ij): O normalised inside the segment, L the row log-sum-exp of
 *    the masked Q_i K_j^T / sqrt(d).
 *  - same page, §2.2: partial states are merged by
 *    L_i = log sum_j exp L_ij,  O_i = sum_j exp(L_ij - L_i) O_ij.
 *  - "04 · Megatron-LM 实现" (llm-infra-atlas, 04_cp/04_megatron_cp_integration),
 *    §1.1 and §1.2: the zigzag split (rank r keeps chunks r and 2cp-1-r of
 *    2cp equal chunks) and its per-sub-sequence form for packed (THD) input.
 *  - "上下文并行：一条序列跨卡，仍算同一个目标" (glenzli.com, context-parallel),
 *    01 and 02: the online recurrence (m, l, a) inside a tile, and the backward
 *    replay from the full-row LSE with dK/dV summed at the key owner.
 *  - "Sequence Parallelism + Ring Attention" (naphjohn LLM-blog), §2: ranks
 *    keep their queries and receive the K/V blocks in ring order.
 * The cp "ranks" are logical: all of them run on one GPU, in ring order, with
 * no collective.
 *
 * Conventions shared by every entry point
 *  - Every tensor pointer is DEVICE memory owned by the caller.  The library
 *    never allocates or frees device memory; scratch space is the caller's
 *    workspace (ws, ws_bytes).
 *  - `stream` is a cudaStream_t passed as void* (NULL = legacy default
 *    stream).  Every call only enqueues work on that stream and returns; the
 *    status reports host-side validation and launch errors.  Faults detected
 *    on the device (a bounded wait that ran out) are reported later through
 *    cp_get_device_error().
 *  - Layouts are contiguous, row-major:
 *      BSHD: q, o, dout, dq  [batch][seqlen][heads_q][head_dim]
 *            k, v, dk, dv    [batch][seqlen][heads_kv][head_dim]
 *      THD (cu_seqlens given, batch = 1): the same with seqlen = T.
 *      lse                   [batch][seqlen][heads_q], float32, natural log.
 *    Element type of q/k/v/o/dout/dq/dk/dv: desc->dtype (float32 or bf16).
 *  - Token order: CP_ORDER_ORIGINAL (the sequence as written) or
 *    CP_ORDER_RANK_LOCAL (rank 0's tokens, then rank 1's, ... each rank in the
 *    order of cp_partition_indices), applying to every token-indexed tensor of
 *    a call.
 *  - Grouped heads: q-head h reads kv-head h / (heads_q / heads_kv).
 *  - Attention kernels (cp_tile_attn_fwd, cp_ring_attn_fwd, cp_ring_attn_bwd,
 *    cp_ring_attn_fwd_static_ws) are fixed by the element type: float32 runs
 *    on CUDA-core FFMA kernels (float32 arithmetic, head_dim 64 or 128), bf16
 *    on the tcgen05 tensor-core kernels, built for head_dim 128 only.  bf16
 *    with another head_dim, or a driver that does not export the tensor-map
 *    encoder the tcgen05 kernels need, returns CP_ERR_UNSUPPORTED; no call
 *    switches to another kernel class.  The token gathers and the partition
 *    take both element types at head_dim 64 and 128.
 *  - Status codes are the cp_status values below; no call aborts the process.
 */
#ifndef CPATTN_H_
#define CPATTN_H_

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
  CP_OK = 0,
  CP_ERR_INVALID_ARG = -1, /* null pointer, bad size, bad cu_seqlens        */
  CP_ERR_ALIGNMENT = -2,   /* a length is not a multiple of 2*cp (striped: cp);
                              serving: a pointer or stride off 16 bytes    */
  CP_ERR_UNSUPPORTED = -3, /* head_dim, dtype or head grouping not built
                              (bf16 attention: head_dim 128 only), or
                              batch * seqlen >= 2^31 token rows           */
  CP_ERR_WORKSPACE = -4,   /* ws too small (see cp_ring_attn_workspace_bytes) */
  CP_ERR_CUDA = -5,        /* a CUDA runtime call failed                   */
  CP_ERR_TIMEOUT = -6      /* a device-side bounded wait ran out           */
} cp_status;

typedef enum { CP_F32 = 0, CP_BF16 = 1 } cp_dtype;

typedef enum { CP_ORDER_ORIGINAL = 0, CP_ORDER_RANK_LOCAL = 1 } cp_order;

/* How a sequence (each packed sub-sequence) is split over the cp ranks. */
typedef enum {
  CP_PARTITION_ZIGZAG = 0,  /* 2cp chunks, rank r holds chunks r and 2cp-1-r
                               ("04 · Megatron-LM 实现" §1.1, §1.2)          */
  CP_PARTITION_STRIPED = 1  /* interleaved: token i on rank i mod cp
                               ("Sequence Parallelism + Ring Attention" §5);
                               lengths a multiple of cp, and the token tensors
                               of the ring entry points in rank-local order  */
} cp_partition_scheme;

/* Problem description.  Sizes are in elements. */
typedef struct {
  int32_t batch;       /* BSHD batch; must be 1 for THD                      */
  int32_t heads_q;     /* H                                                  */
  int32_t heads_kv;    /* Hkv, divides H                                     */
  int32_t head_dim;    /* d: 64 or 128                                       */
  int32_t cp;          /* logical context-parallel ranks, >= 1               */
  int32_t causal;      /* 1: causal by original position; 0: full (THD still
                          block-diagonal)                                    */
  int64_t seqlen;      /* BSHD: tokens per batch entry; THD: total tokens T  */
  const int32_t* cu_seqlens_host; /* THD boundaries, HOST memory, [n_seqs+1],
                          cu[0] = 0, cu[n_seqs] = T; NULL for BSHD          */
  const int32_t* cu_seqlens_dev;  /* the same array in DEVICE memory (used by
                          cp_partition_indices); NULL for BSHD             */
  int32_t n_seqs;      /* number of packed sub-sequences (THD), else 0      */
  cp_dtype dtype;      /* element type of the token tensors                 */
  cp_order order;      /* token order of the token tensors                  */
  float softmax_scale; /* 0 -> 1/sqrt(head_dim)                              */
  cp_partition_scheme partition; /* CP_PARTITION_ZIGZAG (0) or _STRIPED     */
  int32_t window;      /* sliding-window width W ("Context Parallelism (CP)"
                          §2.1: a sparser edge set); 0: none.  W > 0 (causal
                          only): the query at position i sees the keys at
                          positions i-W+1 .. i of its (sub-)sequence        */
  /* Hybrid CP ("04 · Megatron-LM 实现" §7, one round of cp_hybrid_schedule;
     THD, zigzag split): sub-sequence k is split by the zigzag rule with
     cp = seq_cp[k] over ranks seq_rank0[k] .. seq_rank0[k] + seq_cp[k] - 1
     (seq_cp[k] a power of two <= cp, seq_rank0[k] a multiple of it), and
     rank r's stream holds, sub-sequence by sub-sequence, the parts of the
     sub-sequences whose group contains r (ranks of different lengths).
     NULL: every sub-sequence spans all cp ranks.                           */
  const int32_t* seq_cp_host;    /* [n_seqs], HOST memory                    */
  const int32_t* seq_rank0_host; /* [n_seqs], HOST memory                    */
  const int32_t* seq_cp_dev;     /* the same arrays in DEVICE memory (used by */
  const int32_t* seq_rank0_dev;  /* cp_partition_indices)                     */
} cp_attn_desc;

/* Human-readable name of a status code (static string). */
const char* cp_status_string(cp_status status);

/* Validate a descriptor without touching the GPU (host logic only).
 * Checks: sizes positive, H % Hkv == 0, d in {64, 128}, batch == 1 for THD,
 * cu_seqlens_host non-decreasing from 0 to T, every sub-sequence length (and
 * the BSHD seqlen) a multiple of 2*cp ("04 · Megatron-LM 实现" §1.1: the
 * sequence length must be divisible by 2*cp); under CP_PARTITION_STRIPED a
 * multiple of cp and order CP_ORDER_RANK_LOCAL (a rank's tokens are strided
 * in the original order), else CP_ERR_UNSUPPORTED.  window: 0 <= W < 2^30
 * (CP_ERR_INVALID_ARG), and W > 0 needs causal = 1 (CP_ERR_UNSUPPORTED).
 * Hybrid CP (seq_cp_host set): THD, zigzag, seq_rank0_host set, every
 * seq_cp[k] a power of two <= cp and seq_rank0[k] a multiple of it with
 * seq_rank0[k] + seq_cp[k] <= cp (else CP_ERR_INVALID_ARG), every length a
 * multiple of 2 * seq_cp[k] (else CP_ERR_ALIGNMENT). */
cp_status cp_validate_desc(const cp_attn_desc* desc);

/* Zigzag / packed partition ("04 · Megatron-LM 实现" §1.1 and §1.2; "Context
 * Parallelism (CP)" §4) or striped partition ("Sequence Parallelism + Ring
 * Attention" §5), as desc->partition says.
 *  idx      [cp][L/cp] int32, device, written: idx[r][t] = original token index
 *           (within one batch entry) held at slot t of rank r.  L = seqlen.
 *           Zigzag BSHD: chunk r then chunk 2cp-1-r of 2cp chunks of L/(2cp)
 *           tokens.  Zigzag THD: for every sub-sequence k in order, its chunk r
 *           then its chunk 2cp-1-r (chunk length len_k / (2cp)).
 *           Striped: for every sub-sequence k (BSHD: the one sequence) in
 *           order, its tokens r, r + cp, r + 2cp, ... (len_k / cp of them).
 *           Hybrid CP: rank r's stream (see cp_attn_desc), ranks in order;
 *           rank r's slice of sub-sequence k is its chunk o = r - seq_rank0[k]
 *           then chunk 2 seq_cp[k] - 1 - o of len_k / (2 seq_cp[k]) tokens.
 *  local_cu [n_seqs+1] int32, device, optional (NULL): boundaries of the
 *           sub-sequences inside one rank's local stream (cu / cp; identical
 *           for every rank).  THD only.  Hybrid CP: [cp][n_seqs+1], REQUIRED:
 *           local_cu[r][k] = the idx slot where rank r's slice of
 *           sub-sequence k starts (empty when r is not in k's group),
 *           local_cu[r][n_seqs] = the end of rank r's stream.
 * Uses desc->cu_seqlens_dev on the device and desc->cu_seqlens_host for
 * validation.  Errors: CP_ERR_ALIGNMENT when a length is not a multiple of
 * 2*cp (striped: cp); CP_ERR_INVALID_ARG for null idx or bad cu_seqlens. */
cp_status cp_partition_indices(const cp_attn_desc* desc, int32_t* idx, int32_t* local_cu,
                               void* stream);

/* Token gather along the sequence (the index_select of "04 · Megatron-LM 实现"
 * §1.1/§1.2) applied to a [batch][seqlen][heads][head_dim] tensor of
 * desc->dtype.  inverse = 0: dst[b][t] = src[b][idx[t]] (original -> rank
 * local); inverse = 1: dst[b][idx[t]] = src[b][t] (rank local -> original).
 * idx is the [cp][seqlen/cp] array of cp_partition_indices.  src and dst must
 * not overlap. */
cp_status cp_permute_tokens(const cp_attn_desc* desc, const int32_t* idx, int32_t heads,
                            const void* src, void* dst, int32_t inverse, void* stream);

/* Per-token metadata of the rank-local order ("04 · Megatron-LM 实现" §1.2:
 * each packed sub-sequence keeps its own positions, counted from 0):
 *  seq_pos [seqlen][2] int32, device, written: for slot t, the index k of the
 *          sub-sequence holding token idx[t] and that token's position in it
 *          (BSHD: k = 0 and the position in the sequence).
 * idx is the array of cp_partition_indices (any split); THD reads
 * desc->cu_seqlens_dev.  Errors: validation errors, CP_ERR_INVALID_ARG for
 * null pointers. */
cp_status cp_token_seq_pos(const cp_attn_desc* desc, const int32_t* idx, int32_t* seq_pos, void* stream);

/* cp_permute_tokens with the rotary position embedding fused in ("04 ·
 * Megatron-LM 实现" §5: the positions must be split by the same zigzag as the
 * tokens; position_ids travel with the tokens).  For a [batch][seqlen][heads]
 * [head_dim] tensor of desc->dtype, pos = the position of token idx[t] in its
 * sequence (BSHD: idx[t]; THD: idx[t] minus the start of its sub-sequence in
 * desc->cu_seqlens_dev), theta_i = pos * rope_base^(-2i/head_dim), i <
 * head_dim/2, and R rotates each pair (x_i, x_{i+head_dim/2}) (the
 * rotate-half pairing) by theta_i:
 *   inverse = 0: dst[b][t] = R(pos) src[b][idx[t]]        (original -> rank local)
 *   inverse = 1: dst[b][idx[t]] = R(pos)^T src[b][t]      (rank local -> original;
 *                the transpose, as for a gradient)
 * Angles are formed and reduced to [-pi, pi] in float64, rotated in float32.
 * Errors: CP_ERR_INVALID_ARG for null pointers, src == dst, heads < 1 or
 * rope_base <= 0; head_dim other than 64/128 is rejected by validation. */
cp_status cp_permute_rope(const cp_attn_desc* desc, const int32_t* idx, int32_t heads, float rope_base,
                          const void* src, void* dst, int32_t inverse, void* stream);

/* One TileAttention edge ("Context Parallelism (CP)" §2.1, A_ij):
 * queries  rows [q_row0, q_row0 + q_len)  of every batch entry of q,
 * keys     rows [kv_row0, kv_row0 + kv_len) of k and v.
 * q_pos0 / kv_pos0 are the ORIGINAL positions of the first row of each range
 * (rows are consecutive positions): with desc->causal, key j is visible to
 * query i iff kv_pos0 + j <= q_pos0 + i, and with desc->window = W > 0 also
 * q_pos0 + i - (kv_pos0 + j) < W.  Both ranges must lie in one sequence (one
 * batch entry, or one packed sub-sequence).
 * Output partial state, float32, device:
 *   o_part   [batch][q_len][heads_q][head_dim]: output normalised over the
 *            visible keys of this segment (0 for a row that sees none);
 *   lse_part [batch][q_len][heads_q]: natural-log LSE of the scaled masked
 *            scores (-inf for a row that sees no key).
 * Errors: CP_ERR_INVALID_ARG if a range leaves the tensor or a length is < 0. */
cp_status cp_tile_attn_fwd(const cp_attn_desc* desc, const void* q, const void* k, const void* v,
                           int64_t q_row0, int64_t q_pos0, int64_t q_len, int64_t kv_row0,
                           int64_t kv_pos0, int64_t kv_len, float* o_part, float* lse_part,
                           void* stream);

/* The LSE merge of n_parts partial states ("Context Parallelism (CP)" §2.2):
 *   o_parts   [n_parts][rows][heads][head_dim] float32, device
 *   lse_parts [n_parts][rows][heads]           float32, device
 *   o_out     [rows][heads][head_dim] of out_dtype (float32 or bf16, rounded
 *             to nearest even), lse_out [rows][heads] float32 (may be NULL).
 * L = log sum_j exp L_j (max-shifted), O = sum_j exp(L_j - L) O_j.  Partials
 * with L = -inf weigh 0; if all are -inf the row is O = 0, L = -inf.
 * head_dim must be 64 or 128; n_parts >= 1. */
cp_status cp_merge_partials(int32_t n_parts, int64_t rows, int32_t heads, int32_t head_dim,
                            const float* o_parts, const float* lse_parts, void* o_out,
                            cp_dtype out_dtype, float* lse_out, void* stream);

/* Bytes of workspace cp_ring_attn_fwd (backward = 0) or cp_ring_attn_bwd
 * (backward = 1) needs for this descriptor; 0 if the descriptor is invalid
 * or names an attention shape that is not built (bf16 with head_dim != 128).
 * The workspace must be 256-byte aligned. */
size_t cp_ring_attn_workspace_bytes(const cp_attn_desc* desc, int32_t backward);

/* Context-parallel forward over the whole task graph.
 * For every logical rank r, ring step t = 0..cp-1 (key owner s = (r - t) mod cp,
 * "Sequence Parallelism + Ring Attention" §2), every Q chunk of r and the two
 * KV chunks of s form one edge when some query sees some key; each edge runs
 * TileAttention into a float32 partial state in ws, and the partials of each
 * query row are merged (§2.2 of "Context Parallelism (CP)") into
 *   o   (layout of q, desc->dtype)  and  lse ([batch][seqlen][heads_q] f32).
 * Inputs and outputs are in desc->order.  ws: device, at least
 * cp_ring_attn_workspace_bytes(desc, 0) bytes, 256-byte aligned; its contents
 * need no initialisation and are clobbered.  Calls that share a workspace must
 * not overlap on the GPU.  A descriptor with no tokens (seqlen 0) returns
 * CP_OK at once without reading any pointer; empty sub-sequences of a packed
 * batch own no token and no edge. */
cp_status cp_ring_attn_fwd(const cp_attn_desc* desc, const void* q, const void* k, const void* v,
                           void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Context-parallel backward ("上下文并行" 01 BACKWARD/REPLAY and
 * GRADIENT/RETURN, 02 second aligned equations).  Rebuilds the probabilities
 * of every edge from the merged row LSE (P = exp(S - lse)), uses
 * D_i = <dO_i, O_i>, and writes
 *   dq (layout of q), dk, dv (layout of k); dK/dV contributions of every query
 *   rank are summed at the key owner, grouped heads summed into their kv-head.
 * o and lse are cp_ring_attn_fwd's outputs for the same inputs; dout has the
 * layout of q.  ws: at least cp_ring_attn_workspace_bytes(desc, 1) bytes,
 * 256-byte aligned; its contents need no initialisation and are clobbered.
 * For bf16 with head_dim 128 the dq contributions of the key owners are added
 * into a float32 accumulator in ws by hardware reductions whose order is not
 * fixed, so dq may differ in the last bits between calls; dk and dv are
 * summed in a fixed order.  seqlen 0: CP_OK at once, as for the forward. */
cp_status cp_ring_attn_bwd(const cp_attn_desc* desc, const void* q, const void* k, const void* v,
                           const void* o, const float* lse, const void* dout, void* dq, void* dk,
                           void* dv, void* ws, size_t ws_bytes, void* stream);

/* cp_ring_attn_fwd without a caller workspace, for callers that cannot
 * allocate device memory (no cudaMalloc allowed or available to them).  The
 * pages have no counterpart: this is a property of this library's interface.
 * The scratch is a static device array of cp_static_ws_capacity() bytes
 * (64 MiB) inside the library; every GPU that loads the library keeps it until
 * the process exits.  Same arguments, layouts and results as
 * cp_ring_attn_fwd, minus ws / ws_bytes.
 *  - Returns CP_ERR_WORKSPACE, launching nothing, when the problem needs more
 *    than the static scratch (cp_ring_attn_workspace_bytes(desc, 0) >
 *    cp_static_ws_capacity()).
 *  - Calls no cudaMalloc, cudaFree or other allocating routine.  The first
 *    call in a context (normally once per device, in its primary context)
 *    looks up the scratch's device address (cudaGetSymbolAddress) with that
 *    context current.  A new context (for instance after cudaDeviceReset)
 *    counts as a first call again: the address is looked up anew, never
 *    reused from the old one.
 *  - Every call on a device shares the one scratch array, which keeps the
 *    last call's contents: calls that overlap on the GPU (different streams,
 *    no ordering between them) race and give wrong results. */
cp_status cp_ring_attn_fwd_static_ws(const cp_attn_desc* desc, const void* q, const void* k,
                                     const void* v, void* o, float* lse, void* stream);

/* Size in bytes of the static scratch of cp_ring_attn_fwd_static_ws. */
size_t cp_static_ws_capacity(void);

/* Waits for `stream`, then reads and clears the library's device error word.
 * Returns CP_OK, or CP_ERR_TIMEOUT if a kernel gave up on a bounded wait since
 * the last call (its outputs are then invalid), CP_ERR_INVALID_ARG if a paged
 * attention met a page number outside its cache, or CP_ERR_CUDA. */
cp_status cp_get_device_error(void* stream);

/* Failure-detection check: sets the cycle budget of the main-loop waits
 * (mbarrier and pacing waits) of the tcgen05 kernels and of the paged
 * attention for launches made after this call, process-wide.  cycles <= 0
 * restores the default of 4e9 cycles (about two seconds); more than the default
 * returns CP_ERR_INVALID_ARG.  While a shorter budget is set, launches run a
 * separately compiled copy of each of these kernels (the default copies never
 * read the budget, so the setting costs nothing when unused) whose waits probe
 * their barrier without suspending and give up once `cycles` have passed: a
 * budget of a few cycles makes any wait that is not already complete run out.
 * The block then raises its abort flag, its other roles leave their loops, its
 * TMA copies and MMAs are drained with the default budget, TMEM is freed, and
 * cp_get_device_error reports CP_ERR_TIMEOUT (the outputs of that call are
 * invalid).  The pages have no counterpart ("04 · Megatron-LM 实现" §7.2 shows
 * only the deadlock a missing barrier participant causes).  Not for production
 * use.  (cp_cross_attn_fwd and cp_cross_attn_bwd keep the default budget.) */
cp_status cp_debug_set_wait_limit(int64_t cycles);

/* Host-only statistics of the task graph built for a descriptor (no GPU use):
 * out[0] forward work items (Q tile x key owner), out[1] partial-state rows
 * per batch entry, out[2] merge segments (Q chunks), out[3] backward work items
 * (KV tile), out[4] unmasked (query, key) pairs per batch entry and head,
 * out[5] forward key-tile visits (128 x 128 tiles) per batch entry and head.
 * Returns CP_OK or the validation error. */
cp_status cp_ring_plan_stats(const cp_attn_desc* desc, int64_t out[6]);

/* Host-only view of the schedule of the tensor-core backward (no GPU use).
 * *grid: CTAs of the launch; *n_work: work indices, w = (batch entry *
 * heads_kv + kv-head) * (backward work items, out[3] of cp_ring_plan_stats)
 * + item.  CTA c runs work[cta[c]] .. work[cta[c + 1] - 1] in that order;
 * load[c] is its planned cost (query tiles x heads per group + 1 per item).
 * Any output pointer may be null; cta holds *grid + 1 entries, work *n_work,
 * load *grid (query the sizes with null arrays first).  Returns CP_OK or the
 * validation error. */
cp_status cp_ring_bwd_schedule(const cp_attn_desc* desc, int32_t* grid, int64_t* n_work, int32_t* cta,
                               int32_t* work, int64_t* load);

/* Hybrid CP schedule ("04 · Megatron-LM 实现" §7.1, the balanced scheduler;
 * §2.3, aligned power-of-two rank groups).  Host only, no GPU.
 * Assigns every sequence a round, a CP size (power of two) and the first
 * rank of its group, longest sequence first:
 *  - a sequence needs the smallest power of two g of ranks with
 *    len <= g * capacity (max(1, 2^ceil(log2(len / capacity)))); its cost on
 *    g ranks is len^2 / g;
 *  - per round: buckets of about equal cost, one per distinct need (closed
 *    past 1.1x the equal share); a sequence joins the least loaded group of
 *    its size with room for len / g more tokens per rank, else opens a group
 *    on the lowest aligned idle block, else waits for the next round; the
 *    round stops at a bucket step once every rank is busy and the loads are
 *    within 5%; the last placed sequences wait while that cuts the spread
 *    of the busy ranks' loads; groups then double over idle buddy blocks,
 *    most loaded first.
 *  lens     [n] HOST, sequence lengths, each a multiple of 2 * world
 *  world    ranks (a power of two); capacity: tokens per rank per round
 *  round, cp, rank0  [n] HOST, written; n_rounds HOST, written
 * Errors: CP_ERR_INVALID_ARG (null pointers, n < 0, world not a power of two,
 * capacity < 1, a negative length), CP_ERR_ALIGNMENT (a length not a
 * multiple of 2 * world), CP_ERR_UNSUPPORTED (a sequence longer than
 * world * capacity). */
cp_status cp_hybrid_schedule(const int32_t* lens, int32_t n, int32_t world, int64_t capacity,
                             int32_t* round, int32_t* cp, int32_t* rank0, int32_t* n_rounds);

/* Host only: the planner's task-graph tables, for tests and tools.
 *  which 0: forward items of 128 query rows (one per Q tile and streaming
 *           part; the FFMA forward), 1: the same parts in 256-row items (the
 *           tensor-core forward), 2: backward items (one K/V tile and every
 *           query range that sees it), 3: dQ items of the FFMA backward (one
 *           Q tile and every key range it sees), 4: merge segments (no
 *           segs; items [n][8]: output row, rows, first partial row, parts,
 *           partial stride, merge row, 0, 0 - output row r + i merges partial
 *           rows first + e * stride + i, e < parts).
 *  items [n_items][8] int32 (which 0-3): stationary tile row, position,
 *           length, first segment, segment count, partial-state row
 *           (forward), cost, 0;
 *  segs  [n_segs][4] int32: streamed range row, position, length, band
 *           (the sliding-window width in the range's positions; 0 none).
 * Rows index the token tensors (desc->order); positions are those the
 * kernels' masks compare (causal: key position <= query position, and
 * query - key < band when band > 0).  Pass null arrays to read the sizes
 * first.  Errors: validation errors, CP_ERR_INVALID_ARG for a bad `which`. */
cp_status cp_ring_plan_tables(const cp_attn_desc* desc, int32_t which, int64_t* n_items, int64_t* n_segs,
                              int32_t* items, int32_t* segs);

/* ------------------------------------------------------------------------
 * Serving: the K/V of running requests live in the pages of a cache, and a
 * step takes some new tokens of each request: cp_kv_extend gives them pages,
 * slots and positions, cp_kv_append rotates them and writes their K/V into
 * the cache, cp_paged_attn_fwd attends over the pages.  All lengths live in
 * device memory and are read there: no call waits for the host, and each
 * can be captured into a CUDA graph and replayed on new lengths.  Every call
 * follows the shared conventions above (caller's memory, caller's stream,
 * 16-byte aligned rows).
 * ------------------------------------------------------------------------ */

/* The pages of a cache, for K and V alike: element i of head g of token t of
 * page n is at n * page_stride + t * token_stride + g * head_stride + i
 * (strides in elements, multiples of 16 bytes; head_dim contiguous), so that
 * pages, tokens and heads may lie in any order, [page][token][head] and
 * [page][head][token] among them, and K and V side by side in one allocation.  Slot n * page_size + t names a token. */
typedef struct {
  void* k;
  void* v;
  int32_t n_pages;
  int32_t page_size;    /* a power of two, 8 to 256                          */
  int32_t heads_kv;
  int32_t head_dim;     /* 64 or 128                                         */
  int64_t page_stride;
  int64_t token_stride;
  int64_t head_stride;
  cp_dtype dtype;
} cp_kv_cache;

/* Block tables and slot maps from the lengths of the requests.
 *  lens, add     [n_reqs] device: tokens that request r has in the cache, and
 *                tokens that it brings; its pages are the first
 *                ceil(lens / page_size) entries of its table row.
 *  free_pages    [n_pool] device: numbers of unused pages, n_free [1] of them
 *                counted from the front, taken from the back.
 *  block_table   [n_reqs][max_blocks] device, in place: the new pages are
 *                written behind the request's pages, nothing else changes.
 *  lens_out      [n_reqs]: lens + add, cu_new [n_reqs + 1]: the first row of
 *                each request's new tokens, n_free_out [1].
 *  slots, pos    [max_rows]: slot and position of every new token; -1 and 0
 *                behind the last.
 * Requests are served in order: from the first one that does not fit (free
 * pages, max_blocks, max_rows, a negative length) on, none is: their lengths
 * stay and they own no row, which cu_new shows.  The outputs must not overlap
 * the inputs.  n_reqs <= 16384, max_blocks * page_size <= 2^30.
 * Errors: CP_ERR_INVALID_ARG (null pointers, sizes), CP_ERR_UNSUPPORTED. */
cp_status cp_kv_extend(int32_t n_reqs, int32_t max_blocks, int32_t page_size, int64_t max_rows, int32_t n_pool,
                       const int32_t* lens, const int32_t* add, const int32_t* free_pages, const int32_t* n_free,
                       int32_t* block_table, int32_t* lens_out, int32_t* cu_new, int32_t* slots, int32_t* pos,
                       int32_t* n_free_out, void* stream);

/* Gives the pages of the requests with done[r] != 0 back: they are appended
 * to free_pages (request by request, in table order; what n_pool cannot hold
 * is dropped), their table entries become -1 and lens_out[r] = 0; the others
 * keep theirs.  A negative entry holds no page and is passed over, so pages in
 * front of a window that the caller gave back to the pool before are marked
 * by -1; every other entry has to be a page of this request alone (one that is
 * in the pool already, or in another row too, would be handed out twice).
 * block_table and free_pages change in place. */
cp_status cp_kv_release(int32_t n_reqs, int32_t max_blocks, int32_t page_size, int32_t n_pool, const int32_t* lens,
                        const int32_t* done, int32_t* free_pages, const int32_t* n_free, int32_t* block_table,
                        int32_t* lens_out, int32_t* n_free_out, void* stream);

/* Rotary positions with n_axes axes (time, height, width of images and video;
 * one axis is cp_permute_rope's embedding).  n = the sum of section pairs are
 * rotated, the last head_dim - 2 n elements of a head are left as they are.
 *  axis of pair i: section[0] pairs of axis 0, then section[1] of axis 1, ...;
 *    interleaved: the axes take turns, those that have used up their section
 *    are passed over.
 *  angle of pair i: position on its axis times base^(-i / n); restart: times
 *    base^(-j / section[axis]), j = the pairs of its axis before it.
 *  pair i: elements (i, i + n), or with adjacent (2 i, 2 i + 1).
 * n must be a multiple of 8. */
typedef struct {
  int32_t n_axes;       /* 1 to 4                                            */
  int32_t section[4];   /* pairs of each axis                                */
  int32_t interleaved;
  int32_t restart;
  int32_t adjacent;
  float base;           /* > 0                                               */
} cp_rope;

/* Rotates q [rows][heads_q][head_dim] and, with heads_k > 0, k [rows][heads_k]
 * [head_dim] by the positions pos [n_axes][rows] (device, any sign) in one
 * launch; q_stride, k_stride: elements between rows of the inputs (slices of
 * one projection), outputs contiguous.  inverse = 1 applies the transpose
 * R(pos)^T, which is the gradient.  A contiguous input may be its own output.
 * An angle is off by at most 2^-26 + 2^-32 + |position| 2^-53 turns for bases
 * from 1 on (its rounding to float32, the bits below 2^-32 turns, and base^-e / 2 pi in 53
 * bits): 1.1e-7 rad up to positions of 2^24, 1.6e-6 at 2^31.
 * Errors: CP_ERR_INVALID_ARG, CP_ERR_UNSUPPORTED (head_dim, n % 8 != 0),
 * CP_ERR_ALIGNMENT (a pointer or stride off 16 bytes). */
cp_status cp_rope_axes(const cp_rope* rope, const int32_t* pos, int64_t rows, int32_t head_dim, cp_dtype dtype,
                       int32_t heads_q, const void* q, int64_t q_stride, void* q_out, int32_t heads_k, const void* k,
                       int64_t k_stride, void* k_out, int32_t inverse, void* stream);

/* Writes k and v [rows][heads_kv][head_dim] (row strides in elements) into the
 * slots [rows] (device) of the cache.  With rope, k is rotated by pos on the way, and q (heads_q > 0)
 * into q_out [rows][heads_q][head_dim] in the same launch.  A row
 * whose slot is negative or behind the last page is left out: nothing of it
 * is written, q_out's row neither.  Slots that are named twice hold one of
 * the rows, or 16-byte pieces of both.  The inputs must not lie in the cache.
 * Errors as above. */
cp_status cp_kv_append(const cp_kv_cache* cache, const int32_t* slots, int64_t rows, const void* k, int64_t k_stride,
                       const void* v, int64_t v_stride, const cp_rope* rope, const int32_t* pos, int32_t heads_q,
                       const void* q, int64_t q_stride, void* q_out, void* stream);

/* Attention over a paged cache.  The cache holds every visible token, the
 * new ones among them (cp_kv_append comes first). */
typedef struct {
  cp_kv_cache kv;
  int32_t heads_q;      /* a multiple of kv.heads_kv                         */
  int32_t max_new;      /* about how many new tokens a request brings at most:
                           chooses the kernel, any number is computed right; 0: many */
  int32_t causal;       /* 1: new token i of n, at position len - n + i, sees
                           the keys up to its own; 0: all of its request     */
  int32_t window;       /* W > 0: keys at positions > own - W only; 0: none   */
  float softmax_scale;  /* 0 -> 1/sqrt(head_dim)                              */
} cp_paged_desc;

/* Host-only check of a descriptor (the errors that the calls below return). */
cp_status cp_validate_paged_desc(const cp_paged_desc* desc);

/* Bytes of workspace of cp_paged_attn_fwd: fixed by the descriptor, whatever
 * the lengths.  0 if it is invalid.  256-byte aligned. */
size_t cp_paged_attn_workspace_bytes(const cp_paged_desc* desc);

/* For request r, with new tokens in rows cu_new[r] .. cu_new[r + 1] - 1 of q
 * and kv_lens[r] cached tokens (new ones included) in the pages that its row of
 * block_table [n_reqs][max_blocks] names:
 *   o [rows][heads_q][head_dim] (kv.dtype), lse [rows][heads_q] float32, natural
 * log, as cp_tile_attn_fwd gives them (0 and -inf where a row sees no key), so
 * that they merge with other partial states by cp_merge_partials.
 * q: [rows][heads_q][head_dim], q_stride elements between rows.  Rows from
 * cu_new[n_reqs] on are left as they were.  o and lse must not overlap the inputs.
 * Lengths are clamped to the table and to the rows of q.  Only pages with a visible key are
 * looked at: entries behind the last key, or in front of every row's window, may
 * hold anything, and so may the rest of the last page.  A page number outside
 * the cache where a key is visible reads as zeros and is reported: cp_get_device_error then
 * returns CP_ERR_INVALID_ARG.  A K/V value that is not finite reaches every
 * row whose tile of keys holds it, as in the other attention calls.
 * A row with a NaN score has NaN in o and lse.
 * Results do not depend on timing: the same call gives the same bits.
 * Calls that share a workspace must not overlap on the GPU.
 * Errors: CP_ERR_INVALID_ARG, CP_ERR_UNSUPPORTED (sizes, heads), CP_ERR_ALIGNMENT,
 * CP_ERR_WORKSPACE. */
cp_status cp_paged_attn_fwd(const cp_paged_desc* desc, int32_t n_reqs, int64_t rows, int32_t max_blocks,
                            const void* q, int64_t q_stride, const int32_t* block_table, const int32_t* cu_new,
                            const int32_t* kv_lens, void* o, float* lse, void* ws, size_t ws_bytes, void* stream);

/* Host only: how cp_paged_attn_fwd divides a call with these lengths (HOST
 * arrays cu_new [n_reqs + 1] and kv_lens [n_reqs]) over the *grid blocks of its
 * launches on the current device (without a device: as if every pair of 148 SMs could run
 * a pair of blocks), for tests and tools.  pieces [*n][8] int32, in the order of the
 * blocks: block, request, kv-head, first packed row of the tile (token * group + head
 * in group, counted in the request), packed rows, first key and end of the
 * piece's keys, and the slot of its partial state (-1: the tile is whole and goes to
 * the outputs).  Pass null arrays to read the sizes first.  n_reqs >= 1; it
 * refuses the sizes that cp_paged_attn_fwd refuses. */
cp_status cp_paged_schedule(const cp_paged_desc* desc, int32_t n_reqs, int64_t rows, int32_t max_blocks,
                            const int32_t* cu_new, const int32_t* kv_lens, int32_t* grid, int64_t* n,
                            int32_t* pieces);

/* ------------------------------------------------------------------------
 * Cross attention: packed query sequences attend over packed key sequences of
 * other lengths (a decoder over its encoder's states; with equal lengths self
 * attention), with an optional bias of the relative position and optional dropout,
 * forward and backward.  Lengths live in device memory and are read there: no call waits for
 * the host, and each can be captured into a CUDA graph and replayed on new lengths,
 * biases and random numbers.
 *
 * Sequence b has the nq queries in rows cu_q[b] .. cu_q[b + 1] - 1 of q (with len_q
 * the first len_q[b] of them only) and the nk keys in rows cu_k[b] .. cu_k[b + 1] - 1
 * of k and v (with len_k the first len_k[b] only: a padded batch).  cu_q and
 * cu_k do not decrease; what lies outside the tensors is left out.
 *  score  s_ij = softmax_scale q_i . k_j [+ bias[bucket(j - (i + nk - nq))][h]];
 *  mask   causal: j <= i + nk - nq, so that the ends are aligned (new queries
 *         behind cached keys); else every query sees all nk keys;
 *  P      = exp(s - lse), lse_i = log sum_j exp s_ij; a row that sees no key has o = 0, lse = -inf;
 *  o_i    = sum_j P_ij keep_ij / (1 - p) v_j.
 * Grouped heads as everywhere: q-head h reads kv-head h / (heads_q / heads_kv).
 *
 * Buckets of a relative position x = j - (i + nk - nq): rel_both = 0 counts the
 * distance n = max(-x, 0) in `per` = rel_buckets buckets; rel_both = 1 the distance n = |x| in
 * per = rel_buckets / 2, with the keys behind the query (x > 0) in the second half.  With
 * e = per / 2, distances below e have a bucket each, and bucket e + t starts at the distance
 * ceil(e (rel_max_distance / e)^(t / (per - e)) (1 - 1e-12)), t = 0 .. per - e - 1
 * (floating point; the last factor puts a distance that lies on a border behind it).
 * Table entries below -1e30 mask their pairs (a row of only such sees no key, and
 * their gradient is 0); the others are 1e30 at most.
 *
 * Dropout: keep_ij comes from Philox4x32 with 7 rounds (Salmon et al., 2011), drawn
 * again wherever it is needed and never stored: counter words (j / 8, i,
 * b * heads_q + h, low half of rng[1]), key rng[0] (low half first); of the four words of a draw,
 * element e = j % 8 takes the low 15 bits of half e % 2 (0: low) of word e / 2, and is
 * kept iff that number >= round(dropout * 2^15) (to the nearest, halves to even; dropout is a float: a caller who holds a
 * double rounds it to a multiple of 2^-15 first, which a float holds exactly).  1 - p is taken after
 * that rounding.  rng [2] (seed, offset) lies in device memory; the backward takes the same two numbers.
 * ------------------------------------------------------------------------ */
typedef struct {
  int32_t heads_q;
  int32_t heads_kv;        /* divides heads_q                                  */
  int32_t head_dim;        /* 64 or 128                                        */
  cp_dtype dtype;          /* of q, k, v, o, their gradients and the bias table */
  int32_t causal;
  int32_t max_q;           /* about how many queries a sequence has at most:
                              chooses the forward's kernel, any number is computed right; 0: many */
  int32_t rel_buckets;     /* 0: no bias; up to 64, even with rel_both, 2 or more a direction */
  int32_t rel_max_distance; /* where the last bucket begins at the latest: half of a
                              direction's buckets to 65536                     */
  int32_t rel_both;        /* keys behind the query have buckets of their own  */
  float dropout;           /* 0 <= p < 1; 0: none, rng is not read             */
  float softmax_scale;     /* 0 -> 1/sqrt(head_dim)                            */
} cp_cross_desc;

/* Host-only check of a descriptor (the errors that the calls below return). */
cp_status cp_validate_cross_desc(const cp_cross_desc* desc);

/* Bytes of workspace of cp_cross_attn_fwd (backward = 0), or of both calls
 * (backward = 1), whatever the lengths.  0 if the arguments are invalid.  256-byte aligned;
 * contents need no initialisation and are clobbered. */
size_t cp_cross_attn_workspace_bytes(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k,
                                     int32_t backward);

/* Forward: o [rows_q][heads_q][head_dim], lse [rows_q][heads_q] float32, natural log (as cp_tile_attn_fwd gives
 * them, and without dropout fit to be merged by cp_merge_partials).  q [rows_q][heads_q][head_dim], k and v
 * [rows_k][heads_kv][head_dim] with row strides in elements (slices of one projection).  bias
 * [rel_buckets][heads_q] (NULL iff rel_buckets is 0).  rest (bf16 only, layout of o, with a bias up to 128 q-heads
 * a kv-head; NULL: not wanted): what o lost, for cp_cross_attn_bwd.  With a bias o + rest is the output to at most
 * 2^-16 of sum_j P_ij keep_ij / (1 - p) |v_j| (in the mean 2^-17 of the output): P goes into the second product in
 * two parts.  Without one P is rounded to bf16 there (2^-8 of P at most, as in every call without rest) and rest is
 * what o's own rounding took.  Rows that no sequence owns are not read, and
 * left as they were in o, rest and lse.  o and lse must not overlap the inputs.  A K/V value that is not finite reaches
 * every row of its sequence whose tile of keys holds it, as in the other attention calls, but no
 * other sequence.  A row with a NaN score has NaN in o and lse.  Results do not depend on
 * timing: the same call gives the same bits.  Calls that share a workspace must not overlap on the GPU.
 * Errors: CP_ERR_INVALID_ARG, CP_ERR_UNSUPPORTED (sizes, heads; dropout in bf16 with more than 128 q-heads
 * a kv-head), CP_ERR_ALIGNMENT (a pointer or stride off 16 bytes), CP_ERR_WORKSPACE. */
cp_status cp_cross_attn_fwd(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* len_q, const int32_t* len_k,
                            const void* bias, const uint64_t* rng, void* o, void* rest, float* lse, void* ws,
                            size_t ws_bytes, void* stream);

/* Backward: with dS_ij = P_ij (keep_ij / (1 - p) dO_i . v_j - dO_i . o_i),
 *   dq_i = softmax_scale sum_j dS_ij k_j,  dk_j = softmax_scale sum_i dS_ij q_i,  dv_j = sum_i P_ij keep_ij / (1 - p) dO_i,
 *   dbias[b][h] = sum of dS_ij over the pairs of bucket b, all sequences,
 * grouped heads summed into their kv-head.  o, rest and lse are the forward's for the same inputs and rng.  A row's
 * dS sums to 0, so that a bucket that holds all but w of n pairs keeps what dO . o is off by: dbias is off, beyond
 * its own rounding, by sqrt(n / w) of its norm times 2^-18 in bf16 with rest and 2^-21 in float32, as a rule (at
 * most four times that), and by 2^-9 sqrt(n / w) in bf16 without rest, whose dS has the error that the roundings
 * of P and of o make in dO . o, up to 2^-8 P_ij (|dO_i| |o_i| + sum_j P_ij |dO_i . v_j|).
 * dout has the layout of q (row stride in elements).
 * dq, dk and dv [rows][heads][head_dim] are contiguous; rows that no sequence owns (and keys that no query
 * sees) get zeros.  dbias [rel_buckets][heads_q], given iff bias is.  The outputs must not overlap the inputs.
 * In bf16 P is rounded before dv's product, and dS before dq's and dk's.  A value of q, k, v or dout that is not
 * finite reaches the gradients of its sequence whose tiles hold it, and dbias, but no other sequence's dq, dk and
 * dv.
 * In bf16 the dq contributions of the key tiles are added in float32 by hardware reductions whose order is not
 * fixed, so dq may differ in the last bits between calls; all other sums have a fixed order.  ws: as for the
 * forward, with backward = 1.  Errors: as for the forward; CP_ERR_UNSUPPORTED for a bias in bf16 with more than
 * 128 q-heads a kv-head too, whose forward leaves no rest. */
cp_status cp_cross_attn_bwd(const cp_cross_desc* desc, int32_t n_seqs, int64_t rows_q, int64_t rows_k, const void* q,
                            int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                            const void* o, const void* rest, const float* lse, const void* dout, int64_t dout_stride,
                            const int32_t* cu_q, const int32_t* cu_k, const int32_t* len_q, const int32_t* len_k,
                            const void* bias, const uint64_t* rng, void* dq, void* dk, void* dv, void* dbias, void* ws,
                            size_t ws_bytes, void* stream);

/* Kernel classes reported by cp_profile_read. */
typedef enum {
  CP_K_PARTITION = 0, /* partition index kernel                          */
  CP_K_PERMUTE = 1,   /* token gather                                    */
  CP_K_TILE_FWD = 2,  /* tile-attention forward over all edges           */
  CP_K_MERGE = 3,     /* LSE merge                                       */
  CP_K_DELTA = 4,     /* backward preprocess D = rowsum(dO * O)          */
  CP_K_TILE_BWD = 5,  /* tile-attention backward                         */
  CP_K_CONVERT = 6,   /* float32 accumulator -> output dtype             */
  CP_K_TABLES = 7,    /* task-graph table upload (pinned host -> workspace) */
  CP_K_ROPE = 8,      /* token gather with rotary position embedding     */
  CP_K_KV_TABLES = 9, /* request tables of a paged cache                 */
  CP_K_HEAD_ROWS = 10, /* multi-axis rotation, rows into a paged cache   */
  CP_K_PAGED = 11,    /* attention over a paged cache                    */
  CP_K_PAGED_MERGE = 12, /* join of its cut tiles                        */
  CP_K_CROSS = 13,       /* cross attention forward                      */
  CP_K_CROSS_MERGE = 14, /* join of its cut tiles                        */
  CP_K_CROSS_PREP = 15,  /* its bias spread, its backward's preparation  */
  CP_K_CROSS_BWD = 16,   /* cross attention backward                     */
  CP_K_CROSS_POST = 17,  /* its sums and conversions                     */
  CP_K_COUNT = 18
} cp_kernel_class;

/* Benchmark instrumentation (no effect on results).  With timing on, every
 * kernel the library launches is bracketed by two CUDA events recorded on the
 * stream it runs on.  Launch counts are always kept. */
cp_status cp_profile_enable(int32_t on);

/* Waits for the recorded events, writes per-class total device milliseconds
 * (ms[CP_K_COUNT]) and launch counts (launches[CP_K_COUNT]) since the last
 * read, and resets both.  Either pointer may be NULL. */
cp_status cp_profile_read(double* ms, int64_t* launches);

#ifdef __cplusplus
}
#endif

#endif /* CPATTN_H_ */
