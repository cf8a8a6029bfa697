/*
 * vg.h — C ABI of the Vegas hot path on one GB300 (sm_103a).
 *
 * Verification-guided sparse self-speculative decoding, as described on the page
 * "Resumo Técnico: Vegas – Decodificação Auto-Especulativa com Atenção Esparsa
 * Guiada por Verificação" (gist.science summary of paper 2602.07223), cited below
 * as "Vegas §<section>".  One iteration has three device steps:
 *
 *   vg_verify_attn        full attention of the gamma+1 verify rows over the KV cache
 *                         (Vegas §2 step 1), which also sums the pre-softmax logits of
 *                         every prefix entry over the chosen rows and all query heads
 *                         (Vegas §2.A formula, §2.B Collect-2-Query, §3 instrumentation);
 *   vg_topk_select        the k prefix entries with the largest summed logit
 *                         (Vegas §2 step 2, the argmax of §2.A);
 *   vg_sparse_draft_attn  one draft step's attention over the selected entries plus the
 *                         draft tokens appended so far, gathered token by token
 *                         (Vegas §2 step 3; §3 sparse execution, page size one).
 *   vg_iteration          verify -> select -> gamma draft steps, in stream order.
 *   vg_iteration_plan_*   the same iteration captured once as a CUDA graph and
 *                         launched step after step.
 * Around a batch of such sequences:
 *   vg_shared_verify_attn verification for sequences that share a prefix, read once for all;
 *   vg_rope_append        rotary positions of new q and k rows; k and v enter the cache;
 *   vg_pages_resize, vg_pages_fork, vg_pages_compact
 *                         the page pool behind a block table: rows grown, cut and freed,
 *                         branches that share a parent's pages, live pages moved together.
 *
 * Conventions shared by every call
 *   - All tensor arguments are DEVICE pointers to caller-owned memory, unless a
 *     comment says "host".  The library never allocates, frees or synchronises,
 *     and never keeps a pointer after a call returns (except the plans of
 *     vg_iteration_plan_create, which allocate and keep theirs).
 *   - bf16 is IEEE bfloat16 (uint16 storage); fp32 is IEEE binary32.
 *   - Every call only enqueues work on `stream` (0 = legacy default stream) and
 *     returns.  Arguments are validated on the host before anything is enqueued;
 *     a call that returns an error has enqueued nothing.
 *   - Device-side checks (a prefix length above max_len, an index outside the
 *     allowed range, a bounded wait that ran out) never fault: the kernel skips the
 *     offending item and writes a VG_ERR_* code into *dev_status (if dev_status is
 *     non-NULL; the first error wins, the caller zeroes it).  Results for a sequence
 *     whose inputs failed a device check are unspecified.
 *   - Alignment: every device pointer must be 16-byte aligned (dev_status: 4-byte).
 *   - Workspace: `ws` is caller-owned device scratch of at least
 *     vg_workspace_size(...) bytes, 256-byte aligned.  Its contents need no
 *     initialisation and are garbage after a call.  Calls that share a workspace
 *     must be ordered on one stream.
 *   - Thread safety: calls may be made from several host threads; vg_last_error()
 *     is per thread.
 *
 * KV cache (Vegas §1: one K and one V entry per token, growing with the context)
 *   Token-granular slot pool: K and V are bf16 [capacity_slots][H_kv][d], one slot
 *   per token holding all KV heads contiguously (the "page size of one token" of
 *   Vegas §3).  Sequence b's token i lives in slot seq_offset[b] + i.  The caller
 *   reserves, after each prefix, room for the gamma+1 verify rows.
 *
 * Shapes supported by this build: d in {64, 128}; H_kv in [1, 16]; H_q = G * H_kv
 * with G in [1, 16]; gamma in [0, 15]; G * (gamma+1) <= 64; 1 <= B <= 1024;
 * max_len <= 262144 for vg_topk_select; k >= 1; H_kv * d <= 1024 for
 * vg_sparse_draft_attn (one token's page of K and of V is staged whole).
 */
#ifndef VG_H
#define VG_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t vg_status;

#define VG_OK 0
#define VG_ERR_INVALID_ARG (-1)        /* null pointer, bad value, misalignment      */
#define VG_ERR_UNSUPPORTED_SHAPE (-2)  /* outside the shapes listed above             */
#define VG_ERR_WORKSPACE (-3)          /* ws NULL or smaller than vg_workspace_size  */
#define VG_ERR_CUDA (-4)               /* a CUDA runtime call failed                 */
#define VG_ERR_DEVICE_TIMEOUT (-5)     /* device: a bounded wait ran out             */
#define VG_ERR_DEVICE_BOUNDS (-6)      /* device: length or index out of range       */
#define VG_ERR_DEVICE_PAGES (-7)       /* device: the page pool has too few free pages */

/* Problem dimensions (host struct). */
typedef struct vg_dims {
  int32_t B;       /* sequences in the batch                                          */
  int32_t H_q;     /* query heads                                                     */
  int32_t H_kv;    /* key/value heads; query head h reads KV head h / (H_q/H_kv)      */
  int32_t d;       /* head dimension                                                  */
  int32_t gamma;   /* draft tokens per iteration; verification has gamma+1 rows,     */
                   /* row gamma being the bonus token (Vegas §2.B)                    */
  int32_t max_len; /* host-side upper bound on every prefix length (sizes grids and  */
                   /* the workspace; longer device lengths are reported, not read)   */
  float scale;     /* logit scale; 0 means 1/sqrt(d)                                  */
} vg_dims;

/* The KV cache of one layer (host struct holding device pointers).
 *
 * Two layouts of the same slot pool (one slot = one token's keys of every KV head):
 *   page_table == NULL: sequence b's token i lives in slot seq_offset[b] + i;
 *   page_table != NULL: the vLLM-style block table of Vegas §3 (the draft runs as a
 *     paged attention whose pages are tokens): the pool is cut into pages of page_size
 *     slots (page p = slots p * page_size .. p * page_size + page_size - 1) and token i
 *     of sequence b lives in row i % page_size of page page_table[b][i / page_size].
 *     seq_offset is then unused (may be NULL).  Page entries outside the pool are
 *     reported on the device as VG_ERR_DEVICE_BOUNDS and their tokens skipped.
 *     vg_sparse_draft_attn reads any page_size >= 1; vg_verify_attn and vg_iteration
 *     need page_size 8, 16, 32 or a multiple of 64 (VG_ERR_UNSUPPORTED_SHAPE otherwise).
 *     pages_per_seq (>= 1) is the row stride of page_table; a sequence's prefix plus
 *     its gamma+1 verify rows must fit pages_per_seq * page_size tokens. */
typedef struct vg_kv_cache {
  void* K;                    /* bf16 [capacity_slots][H_kv][d]                       */
  void* V;                    /* bf16 [capacity_slots][H_kv][d]                       */
  const int64_t* seq_offset;  /* device int64 [B]: slot of token 0 of sequence b      */
  int64_t capacity_slots;     /* slots in K and V                                     */
  const int32_t* page_table;  /* device int32 [B][pages_per_seq], or NULL             */
  int32_t page_size;          /* tokens per page (page_table only)                    */
  int32_t pages_per_seq;      /* row stride of page_table (page_table only)          */
} vg_kv_cache;

/*
 * Verification attention with fused logit aggregation (Vegas §2 step 1; §2.A; §2.B; §3).
 *
 * For sequence b with prefix length n_b = prefix_len[b], verify row t in [0, gamma]
 * and query head h (KV head g = h / G):
 *   out[b][t][h] = softmax_j(l_j) . V_j over j in {prefix 0..n_b-1} U {verify rows u <= t},
 *   l_j = scale * q[b][t][h] . K_j   (causal among the verify rows, itself included);
 * and for every prefix entry i < n_b and each enabled mask (row_mask0, row_mask1):
 *   scores[b][i] = sum over rows t with bit t set, over all H_q heads, of
 *                  scale * q[b][t][h] . K[seq_offset[b] + i][h / G]
 * i.e. the objective of the Vegas §2.A selection formula, before any softmax.  The
 * verify rows' own keys are not scored (T is a subset of the prefix P).
 *
 *   q        bf16 [B][gamma+1][H_q][d]
 *   k_new    bf16 [B][gamma+1][H_kv][d] — the verify rows' keys and values.  They are
 *   v_new        appended to the cache at slots seq_offset[b] + n_b + t.  Pass both
 *                NULL when those slots already hold them.
 *   prefix_len  device int32 [B], each in [0, max_len]
 *   row_mask0/1 bit t selects verify row t; 0 disables that output.  Collect-2-Query
 *               is (1 | 1 << gamma); all rows is (1 << (gamma+1)) - 1.
 *   scores0/1   fp32 [B][score_stride] (score_stride >= max_len); NULL iff its mask is 0.
 *               Entries at positions >= n_b are left untouched.
 *   out      bf16 [B][gamma+1][H_q][d]
 */
vg_status vg_verify_attn(const vg_dims* dims, const vg_kv_cache* cache, const void* q,
                         const void* k_new, const void* v_new, const int32_t* prefix_len,
                         uint32_t row_mask0, uint32_t row_mask1, float* scores0, float* scores1,
                         int64_t score_stride, void* out, void* ws, size_t ws_bytes,
                         int32_t* dev_status, void* stream);

/*
 * Per-sequence top-k of the aggregated scores (Vegas §2 step 2, the argmax of §2.A).
 *
 * T_b = the k positions i < len[b] with the largest scores[b][i]; equal scores
 * prefer the lower position; -0.0 equals +0.0 (NaN scores: unspecified order).
 *   idx[b][0..count_b) = T_b in ascending order, count_b = min(k, len[b]);
 *   idx[b][count_b..k) = -1;  count[b] = count_b.
 *
 *   scores  fp32 [B][score_stride];  len  device int32 [B], each in [0, max_len]
 *   idx     int32 [B][k];            count  int32 [B]
 * Uses no workspace (ws may be NULL).
 */
vg_status vg_topk_select(const float* scores, int64_t score_stride, const int32_t* len, int32_t B,
                         int32_t max_len, int32_t k, int32_t* idx, int32_t* count, void* ws,
                         size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * Sliding-window selection: the query-agnostic comparison policy of Vegas §1 (simple
 * query-agnostic methods such as sliding windows select cheaply but draft poorly).
 * No counterpart in the Vegas method itself; it gives drafts a baseline selection in
 * the same form as vg_topk_select, whose overlap with the verification-guided one can
 * be measured.
 *
 *   T_b = the last min(k, len[b]) prefix positions, len[b] - count_b .. len[b] - 1,
 *   idx[b][0..count_b) = T_b ascending, idx[b][count_b..k) = -1, count[b] = count_b.
 *
 *   len  device int32 [B], each in [0, max_len] (others: VG_ERR_DEVICE_BOUNDS, count 0)
 *   idx  int32 [B][k];  count  int32 [B];  1 <= k <= 2^24
 */
vg_status vg_window_select(const int32_t* len, int32_t B, int32_t max_len, int32_t k, int32_t* idx,
                           int32_t* count, int32_t* dev_status, void* stream);

/*
 * One sparse draft step (Vegas §2 step 3; §3 sparse execution with page size one).
 *
 * For sequence b the attended set is
 *   A_b = { idx[b][j] : j < count[b] }  U  { tail_start[b] + u : u < tail_len[b] },
 * positions relative to seq_offset[b].  out[b][h] = softmax over A_b of
 * scale * q[b][h] . K_j, applied to V_j, on KV head h / G.
 * If k_new / v_new (bf16 [B][H_kv][d]) are non-NULL they are the current draft
 * token's key and value: they are appended at slot tail_start[b] + tail_len[b] - 1
 * (tail_len[b] >= 1 is then required) and attended from the inputs directly.
 * tail_len[b] <= 16 (a draft phase appends at most gamma + 1 <= 16 tokens); a longer
 * tail is reported as VG_ERR_DEVICE_BOUNDS.  k_stride <= 2^24.
 * Selected positions must be < tail_start[b]; entries outside [0, tail_start[b]) are
 * skipped and reported as VG_ERR_DEVICE_BOUNDS.
 *
 *   q      bf16 [B][H_q][d]             idx  int32 [B][k_stride], count int32 [B] (<= k_stride)
 *   tail_start, tail_len  device int32 [B]   out  bf16 [B][H_q][d]
 *   flags  0, or VG_DRAFT_SELECTION_SETTLED (below); other bits are VG_ERR_INVALID_ARG.
 */
/* The caller vouches that idx, count, seq_offset or page_table, tail_start, tail_len and the
 * cache entries at the selected positions were all written before the kernel that precedes
 * this call in the stream began.  That holds for every draft step of a phase after the
 * first: the selection is made once per verification and the steps in between only
 * append draft tokens (Vegas §2 step 3).  The call then starts gathering the selected
 * entries before its dependency on that preceding kernel resolves, overlapping the
 * end of the previous step; the draft-token tail still waits for it.  Results are
 * unspecified if the promise does not hold. */
#define VG_DRAFT_SELECTION_SETTLED 1u

vg_status vg_sparse_draft_attn(const vg_dims* dims, const vg_kv_cache* cache, const void* q,
                               const void* k_new, const void* v_new, const int32_t* idx,
                               const int32_t* count, int32_t k_stride, const int32_t* tail_start,
                               const int32_t* tail_len, uint32_t flags, void* out, void* ws,
                               size_t ws_bytes, int32_t* dev_status, void* stream);

/* Inputs of one iteration (host struct of device pointers). */
typedef struct vg_iter_inputs {
  const void* q_verify;        /* bf16 [B][gamma+1][H_q][d]                              */
  const void* k_verify;        /* bf16 [B][gamma+1][H_kv][d], appended at n_b + t         */
  const void* v_verify;
  const void* q_draft;         /* bf16 [gamma][B][H_q][d]                                */
  const void* k_draft;         /* bf16 [gamma][B][H_kv][d]; step s appended at n_b + s    */
  const void* v_draft;
  const int32_t* prefix_len;   /* device int32 [B]                                       */
} vg_iter_inputs;

/* Outputs of one iteration (host struct of device pointers). */
typedef struct vg_iter_outputs {
  void* out_verify;            /* bf16 [B][gamma+1][H_q][d]                              */
  float* scores0;              /* fp32 [B][score_stride], rows of row_mask0 (selection)   */
  float* scores1;              /* fp32 [B][score_stride] or NULL (row_mask1 == 0)         */
  int64_t score_stride;
  int32_t* idx;                /* int32 [B][k]: selection on scores0                      */
  int32_t* count;              /* int32 [B]                                              */
  int32_t* idx1;               /* int32 [B][k] selection on scores1, or NULL              */
  int32_t* count1;             /* int32 [B], or NULL                                     */
  void* out_draft;             /* bf16 [gamma][B][H_q][d]                                */
} vg_iter_outputs;

/*
 * One Vegas round (Vegas §2 steps 1-3), enqueued in order on `stream`:
 *   vg_verify_attn (appends k_verify/v_verify) -> vg_topk_select on scores0
 *   (and on scores1 if idx1 != NULL) -> for s = 0..gamma-1: vg_sparse_draft_attn
 *   with q_draft[s], appending k_draft[s] at slot n_b + s and attending
 *   T_b U {n_b .. n_b + s} (the draft tokens so far, the current one included).
 * Draft tokens reuse the verify rows' slots.  k >= 1.
 */
vg_status vg_iteration(const vg_dims* dims, const vg_kv_cache* cache, const vg_iter_inputs* in,
                       int32_t k, uint32_t row_mask0, uint32_t row_mask1, vg_iter_outputs* out,
                       void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * vg_iteration (Vegas §2 steps 1-3), captured once and launched many times.  This
 * has no counterpart in the paper, which runs inside a serving framework's loop.  A
 * decode loop calls the same iteration with the same buffers step after step;
 * launching its ~3 + 2*gamma kernels one by one costs the GPU a fraction of a
 * microsecond each.  A plan records the launch sequence of one argument set as a CUDA
 * graph, and each launch replays it in a single call, with the same results as
 * vg_iteration on the buffers' contents at launch time.
 *
 * vg_iteration_plan_create: same arguments and validation as vg_iteration (returns
 *   the same codes, enqueues nothing, writes *plan = NULL on error) plus
 *   plan (out): receives an opaque handle owned by the caller.
 *   The plan keeps every pointer it was given, and the values of *dims, *cache, *in
 *   and *out at creation: each launch reads and writes those same buffers, which
 *   must stay allocated, at the same addresses, until vg_iteration_plan_destroy.
 *   Put new inputs in those buffers between launches.  Unlike every other call,
 *   creating a plan allocates: host memory and the CUDA graph's resources
 *   (VG_ERR_CUDA if the CUDA runtime refuses).  Do not call it while this
 *   thread is capturing a stream.  The plan belongs to the current device.
 * vg_iteration_plan_launch: enqueues one iteration on `stream`, in stream order
 *   with the work before and after it.  VG_ERR_INVALID_ARG for a NULL plan or a
 *   current device other than the plan's; VG_ERR_CUDA if the launch fails.  Launches
 *   of one plan on different streams race on its buffers: order them.
 * vg_iteration_plan_destroy: frees the plan (NULL is a no-op).  Launches already
 *   enqueued still complete.
 */
typedef struct vg_iteration_plan vg_iteration_plan;
vg_status vg_iteration_plan_create(const vg_dims* dims, const vg_kv_cache* cache, const vg_iter_inputs* in,
                                   int32_t k, uint32_t row_mask0, uint32_t row_mask1,
                                   const vg_iter_outputs* out, void* ws, size_t ws_bytes,
                                   int32_t* dev_status, vg_iteration_plan** plan);
vg_status vg_iteration_plan_launch(const vg_iteration_plan* plan, void* stream);
vg_status vg_iteration_plan_destroy(vg_iteration_plan* plan);

/*
 * vg_sparse_draft_attn without a workspace argument.  This entry point has no
 * counterpart in the paper; it exists for callers that cannot hand the library
 * device memory, for example a host that must not call cudaMalloc during decoding
 * (the call can synchronise the device and stall other streams) or that has no
 * workspace to offer.  Same computation, arguments and results as
 * vg_sparse_draft_attn with flags 0; the scratch space comes from an 8 MiB area
 * inside the library that every GPU using the library keeps until the process exits.
 *   - It allocates and frees nothing.
 *   - Dimensions whose draft scratch exceeds 8 MiB are rejected with
 *     VG_ERR_WORKSPACE (for 152 SMs: about H_q * (152 + B) * (d + 2) * 4 bytes).
 *   - The first call on each device looks up the area's device address and keeps
 *     it for the life of the process; make that first call before any stream
 *     capture, and do not reset a device (cudaDeviceReset) while the library is
 *     loaded, since the kept address would then be stale.
 *   - All calls share the one area, which keeps the last call's contents (nothing
 *     in it needs to start at zero).  Calls that may overlap on the GPU - on
 *     different streams, or from different host threads - race on it; order them.
 */
vg_status vg_sparse_draft_attn_noalloc(const vg_dims* dims, const vg_kv_cache* cache, const void* q,
                                       const void* k_new, const void* v_new, const int32_t* idx,
                                       const int32_t* count, int32_t k_stride, const int32_t* tail_start,
                                       const int32_t* tail_len, void* out, int32_t* dev_status, void* stream);

/*
 * Acceptance of the draft chain (Vegas §2 step 1: the verification pass accepts or
 * rejects the draft tokens; §5: lossless, what is committed follows the target model).
 * The page leaves the rule to standard speculative decoding; this is that rule on
 * given logits.  For sequence b:
 *   p_logits  fp32 [B][gamma+1][V]  row t: the target's logits for the token after t
 *                                     accepted drafts (row gamma: the bonus position)
 *   q_logits  fp32 [B][gamma][V]    the draft's logits of draft token t (sampling only)
 *   draft_tokens  int32 [B][gamma]  in [0, V) (others: rejected, VG_ERR_DEVICE_BOUNDS)
 *   mode VG_ACCEPT_GREEDY: draft t survives while it is the most likely token of row t
 *     (ties: lowest token); the next token is the most likely token of row a.
 *   mode VG_ACCEPT_SAMPLE: draft t survives iff u_accept[b][t] * q_t(x_t) < p_t(x_t), p and
 *     q the softmax of the rows; at the first rejection a the next token is drawn from
 *     max(0, p_a - q_a) (from p_a if that is zero everywhere), after gamma acceptances
 *     from p_gamma.  A draw with weights w takes the smallest v whose running sum of
 *     weights exceeds u_resample[b] times their total.  u values in [0, 1), fp32.
 *   n_accept  int32 [B]: a, the drafts accepted (0 .. gamma);  next_token int32 [B].
 *   advance_len  int32 [B] or NULL: if given, increased by a + 1 (the verified row before
 *     the drafts and the a accepted drafts join the prefix; their keys and values are
 *     already in the cache).
 * Computed in fp32 with fixed summation orders (deterministic).  B <= 1024, gamma <= 15,
 * V <= 2^20; V % 4 == 0 reads the rows with 16-byte loads.  Workspace: at least
 * vg_accept_workspace_size(B, gamma, V) bytes, 256-byte aligned, no initialisation.
 */
#define VG_ACCEPT_GREEDY 0u
#define VG_ACCEPT_SAMPLE 1u
size_t vg_accept_workspace_size(int32_t B, int32_t gamma, int32_t V);
vg_status vg_accept(int32_t B, int32_t gamma, int32_t V, const float* p_logits, const float* q_logits,
                    const int32_t* draft_tokens, const float* u_accept, const float* u_resample,
                    uint32_t mode, int32_t* n_accept, int32_t* next_token, int32_t* advance_len,
                    void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * vg_verify_attn for a batch whose sequences share prefixes: samples, branches or requests of
 * one prompt.  No counterpart in the page, which treats each sequence by itself; the results
 * are those of vg_verify_attn (up to rounding), the shared tokens' keys and values being read
 * once for a whole group instead of once a sequence.
 *
 *   groups->n_groups     groups of consecutive sequences, 1 .. 1024
 *   groups->group_start  device int32 [n_groups + 1], ascending from 0 to B: group j is
 *                        sequences group_start[j] .. group_start[j + 1] - 1 (it may be empty);
 *                        NULL with n_groups == 1: the whole batch
 *   groups->shared_len   device int32 [n_groups]: the first shared_len[j] tokens of all members
 *                        are the same, 0 <= shared_len[j] <= every member's prefix_len.  They
 *                        are read where the group's first member has them; a remainder past a
 *                        multiple of 128 tokens is read where each member has it, so every
 *                        member's own table row (or slots) must hold all of its tokens, as
 *                        after vg_pages_fork.  A bad page of the first member among them is a
 *                        failed check of every member.
 *   row_mask, scores     as row_mask0, scores0 of vg_verify_attn: scores for every prefix entry
 *                        of every sequence, shared ones included; both 0 / NULL to leave out
 *   others               as vg_verify_attn (page_size 8, 16, 32 or a multiple of 64)
 * With d = 128, 5 * n_groups + 4 * B beyond about 8500 is refused (VG_ERR_UNSUPPORTED_SHAPE): the
 * batch's layout has to fit beside the tiles in shared memory.
 * A group_start that is not such a list, or a shared_len out of range, is reported as
 * VG_ERR_DEVICE_BOUNDS, and the group's (or every) sequence is then read by itself.
 * Workspace: at least vg_shared_verify_workspace_size(dims, groups) bytes (only n_groups is
 * read; 0 on bad arguments or no device), 256-byte aligned, contents arbitrary.
 * Launches: 3, or 4 with scores.
 */
typedef struct vg_prefix_groups {
  int32_t n_groups;
  const int32_t* group_start;
  const int32_t* shared_len;
} vg_prefix_groups;
size_t vg_shared_verify_workspace_size(const vg_dims* dims, const vg_prefix_groups* groups);
vg_status vg_shared_verify_attn(const vg_dims* dims, const vg_kv_cache* cache, const vg_prefix_groups* groups,
                                const void* q, const void* k_new, const void* v_new, const int32_t* prefix_len,
                                uint32_t row_mask, float* scores, int64_t score_stride, void* out, void* ws,
                                size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * Rotary positions of new q and k rows, and the append of k and v to the cache.  No
 * counterpart in the page, whose engine rotates inside the model; it is the step before
 * vg_verify_attn (which then takes k_new = v_new = NULL) and before a prompt's attention.
 *
 * Row r of the packed rows belongs to sequence b at position pos = prefix_len[b] + t, t its
 * index among b's rows.  In every q and k head each pair (x, y) of the first rot_dim
 * elements becomes (x c - y s, x s + y c), c and s being mscale times the cosine and sine of
 * pos * f_i; the elements from rot_dim on are copied.  q goes to q_out, k and v (as it is)
 * to the cache slot of position pos.
 *
 *   rope->freq     device uint64 [rot_dim / 2]: f_i as a fraction of a turn per position,
 *                  round(f_i / 2pi * 2^64) (vg_rope_freqs fills a host array).  The angle is
 *                  exact to pos * 2^-65 of a turn at any position.
 *   rope->rot_dim  even, 2 .. d.   rope->layout  VG_ROPE_HALF: pairs (i, i + rot_dim / 2);
 *                  VG_ROPE_INTERLEAVED: pairs (2i, 2i + 1).
 *   rope->mscale   finite; 0 means 1.
 *   q, k, v, q_out bf16 [n_rows][H_q or H_kv][d] with row strides in elements (multiples of
 *                  8, at least heads * d), so that the three may be slices of one projection's
 *                  output.  q_out may be q itself with the same stride; else it overlaps
 *                  none of the inputs, and no input overlaps the cache.
 *   row_start      device int32 [B + 1], ascending from 0: b's rows are row_start[b] ..
 *                  row_start[b + 1] - 1 (none, if equal).  Rows from row_start[B] on, up to
 *                  n_rows, are padding: nothing is read or written for them.  NULL: every
 *                  sequence has gamma + 1 rows, and n_rows must be B * (gamma + 1).
 *   prefix_len     device int32 [B], each in [0, max_len]: tokens in the cache before the rows.
 * A row whose prefix length is out of range is left alone, one whose slot lies outside the
 * cache is not appended (its q is still rotated); both report VG_ERR_DEVICE_BOUNDS.  Any
 * page_size >= 1.  n_rows in [0, 2^24]; uses no workspace; one launch (none for 0 rows, for which
 * q, k, v and q_out may be NULL).
 */
#define VG_ROPE_HALF 0
#define VG_ROPE_INTERLEAVED 1
typedef struct vg_rope {
  const uint64_t* freq;
  int32_t rot_dim;
  int32_t layout;
  float mscale;
} vg_rope;
vg_status vg_rope_append(const vg_dims* dims, const vg_kv_cache* cache, const vg_rope* rope, const void* q,
                         int64_t q_stride, const void* k, int64_t k_stride, const void* v, int64_t v_stride,
                         const int32_t* row_start, int32_t n_rows, const int32_t* prefix_len, void* q_out,
                         int64_t q_out_stride, int32_t* dev_status, void* stream);

/*
 * The frequencies of vg_rope_append, computed on the host in 64 bits into freq (HOST memory,
 * rot_dim / 2 entries; the caller copies them to the device).  f_i = base^(-2i / rot_dim), then
 *   VG_ROPE_PLAIN   as it is;
 *   VG_ROPE_LINEAR  f_i / factor (positions compressed by factor);
 *   VG_ROPE_BASE    base * factor^(rot_dim / (rot_dim - 2)) instead of base (rot_dim > 2), which
 *                   leaves the fastest pair and divides the slowest by factor;
 *   VG_ROPE_RAMP    by parts: a pair that turns r = orig_len * f_i / 2pi times within the
 *                   original context keeps f_i if r >= fast, gets f_i / factor if r <= slow, and
 *                   a blend linear in r between.  (A common choice of mscale beside it is
 *                   0.1 ln(factor) + 1.)  A blend linear in the pair's index i, as some models
 *                   were trained with, is another: fill freq by that formula.
 * base > 0, factor > 0 (finite, the base of BASE too), every f_i below 2pi; RAMP: orig_len > 0 and
 * 0 <= slow < fast.  Arguments that a kind does not name are ignored.  No device needed.
 */
#define VG_ROPE_PLAIN 0u
#define VG_ROPE_LINEAR 1u
#define VG_ROPE_BASE 2u
#define VG_ROPE_RAMP 3u
vg_status vg_rope_freqs(int32_t rot_dim, double base, uint32_t scaling, double factor, double orig_len, double slow,
                        double fast, uint64_t* freq);

/*
 * The page pool behind a block table (vg_kv_cache.page_table), kept on the device and
 * changed there, so that a decode loop never waits for the host.  No counterpart in the
 * page, whose engine manages its pages itself.  A host struct of device pointers:
 *   page_table  int32 [n_seqs][pages_per_seq], as vg_kv_cache reads it (the first rows of a
 *               table of n_seqs rows serve a batch of B <= n_seqs sequences);
 *   held        int32 [n_seqs]: row s holds its first held[s] entries; later ones are not read;
 *   refs        int32 [n_pages]: how often a page is held, 0 (or less): free.
 * One table serves every layer: page p of a layer is its slots p * page_size and on.  A new
 * pool is held = 0 and refs = 0; a page that must never be handed out keeps refs > 0.
 * page_size in [1, 2^20], n_pages <= 2^30, n_pages * page_size < 2^31, n_seqs <= 65536,
 * pages_per_seq <= 2^30, n_seqs * pages_per_seq < 2^31.
 *
 * Requests are served in order, all releases before any page is handed out, the lowest free
 * pages first: the result depends on the state and the request alone.  Reported on the
 * device, the request then changing nothing: VG_ERR_DEVICE_BOUNDS for a row outside the table
 * or named twice (the first one counts), a length that does not fit pages_per_seq pages (or is
 * negative, or longer than what the parent holds).  VG_ERR_DEVICE_PAGES: the pool ran out; the
 * request keeps what it had after releases, and so do all later ones that need pages.  Calls
 * that share a pool or a workspace must be ordered on one stream.
 * Workspace: vg_pages_workspace_size bytes (0 on a bad pool), 256-byte aligned, contents
 * arbitrary before and after.  All pointers 16-byte aligned.  A request of no rows (n = 0) does
 * nothing; its lists may be NULL.
 */
typedef struct vg_page_pool {
  int32_t* page_table;
  int32_t* held;
  int32_t* refs;
  int32_t n_seqs;
  int32_t pages_per_seq;
  int32_t n_pages;
  int32_t page_size;
} vg_page_pool;
size_t vg_pages_workspace_size(const vg_page_pool* pool);

/*
 * Rows grown, cut or freed: row seq[j] holds ceil(length[j] / page_size) pages afterwards
 * (j < n; length 0 frees it).  Pages past that are given back (their entries become -1);
 * missing ones are appended.  Cutting a row inside a page that other rows hold leaves that
 * page shared: fork the row before tokens are appended there.
 *   seq  device int32 [n], or NULL for rows 0 .. n-1;  length  device int32 [n];  0 <= n <= n_seqs
 */
vg_status vg_pages_resize(const vg_page_pool* pool, const int32_t* seq, const int32_t* length, int32_t n, void* ws,
                          size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * Branches: row child[j] becomes a copy of the first length[j] tokens of row parent[j], with
 * room for `room` more.  What the child held is given back; whole pages are shared (their
 * references counted); the page that length[j] ends inside is copied, the tokens in use only,
 * in every layer, so that both rows may append; ceil((length + room) / page_size) pages are
 * held.  A row may be the parent of many, but not parent and child in one call.  If the pool
 * runs out, the child holds nothing.
 *   caches  host array of n_layers caches (1 .. 128): K, V and capacity_slots are read, each
 *           with at least n_pages * page_size slots;  token_bytes  bytes of one slot of K
 *           (H_kv * d * 2), a multiple of 16, up to 2^20
 *   parent, child, length  device int32 [n], 0 <= n <= n_seqs;  room >= 0
 */
vg_status vg_pages_fork(const vg_page_pool* pool, const vg_kv_cache* caches, int32_t n_layers, int32_t token_bytes,
                        const int32_t* parent, const int32_t* child, const int32_t* length, int32_t n, int32_t room,
                        void* ws, size_t ws_bytes, int32_t* dev_status, void* stream);

/*
 * Holes closed: with n_live pages in use, the ones from index n_live on move into the free
 * ones below it (ascending into ascending), contents of every layer included; afterwards
 * pages 0 .. n_live - 1 are in use.  Entries of the rows that held a moved page name its new
 * place in page_table_out, and its references are in refs_out; both may be the pool's own
 * arrays (in place) or must not overlap them.  Entries past held are copied as they are.  A
 * page kept from use by a reference of its own moves like any other: keep such pages at the front.
 * Moved pages' old contents stay where they were.  n_live: device int32 (the count).
 */
vg_status vg_pages_compact(const vg_page_pool* pool, const vg_kv_cache* caches, int32_t n_layers, int32_t token_bytes,
                           int32_t* page_table_out, int32_t* refs_out, int32_t* n_live, void* ws, size_t ws_bytes,
                           int32_t* dev_status, void* stream);

/* Bytes of workspace any call of an iteration (verify, select, draft) needs for these
 * dimensions on the current device (0 on invalid dims or no device; see vg_last_error()). */
size_t vg_workspace_size(const vg_dims* dims, int32_t k);

/* Kernels one vg_sparse_draft_attn call with these dimensions enqueues on the current
 * device: 1 when every sequence's entries fall to a single CTA of the step's grid
 * (that CTA finishes the sequence), else 2 (a second kernel merges the partials).  tail_len_max is the
 * longest tail the call may attend, 0 for the bound of a device tail_len array (16).
 * Returns 0 on invalid arguments or when no device is present (see vg_last_error()).
 * vg_iteration enqueues 3 (verify, its merge, the selection; 4 with a second
 * selection) plus gamma times this number for tail_len_max = 1 .. gamma. */
int32_t vg_sparse_draft_launches(const vg_dims* dims, int32_t k_stride, int32_t tail_len_max);

/* Human-readable description of the last error on this host thread ("" if none). */
const char* vg_last_error(void);

/* Library version, as major * 10000 + minor * 100 + patch. */
int32_t vg_version(void);

/* Self-test of the device-side failure path (no part of the method): launches one
 * CTA of two warps on `stream`; each waits on an mbarrier that nothing arrives on.
 * The first wait gives up after limit_us microseconds (1 .. 1000000), writes
 * VG_ERR_DEVICE_TIMEOUT into *dev_status (if it holds 0) and raises the CTA's abort
 * flag, on which the second wait (whose own limit is the library's 2 s) gives up at
 * once.  *elapsed_ns (device memory, may be NULL) receives the time from the start
 * of the waits to the end of both, so a caller can check that neither a lost wait
 * nor its abort leaves a kernel running.  No copy or tensor-core operation is
 * involved.  Returns VG_ERR_INVALID_ARG for a limit out of range or a NULL or
 * misaligned dev_status / elapsed_ns, VG_ERR_CUDA if the launch fails. */
vg_status vg_selftest_lost_wait(uint32_t limit_us, int32_t* dev_status, uint64_t* elapsed_ns, void* stream);

#ifdef __cplusplus
}
#endif

#endif /* VG_H */
