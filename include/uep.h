/*
 * uep.h -- C-ABI of libuep.so, the MI355X (gfx950) real-time MoE expert
 * load-balancing path: load matrix -> quota solve -> local-first reroute and
 * token assignment -> permute -> redundant-slot staging, plus Waterfill
 * shared-expert placement and the LPLB min-max replica split.
 *
 * Sources (the pages the method comes from):
 *   [UEP]  "300 微秒调平 MoE 专家负载！小红书 UltraEP 逼近 94.3% 理想训推吞吐"
 *          (UltraEP technical article, m.163.com)
 *   [BLOG] "Improving DeepEP MoE Load Balance in SGLang with Waterfill and LPLB"
 *          (papercache notes of the lmsys blog)
 *
 * Conventions shared by every call
 *   - Every array argument is a DEVICE pointer owned by the caller, except where a
 *     call says "host".  The library never allocates, frees or synchronises on
 *     these calls; work is enqueued on `stream` (a hipStream_t; NULL = the null
 *     stream) and ordered with the caller's other work on that stream.
 *   - Integer arrays are int32, row-major, with the shapes given below.
 *     bf16 data is passed as raw uint16 bits and moved bit for bit; calls with a
 *     dtype argument take void pointers to UEP_F32 or UEP_BF16 elements.
 *   - Geometry: R virtual EP ranks, T tokens per rank, K routing slots per token,
 *     E logical experts, home(e) = e / (E / R) for the routed experts.  A physical
 *     instance id is i = r * inst_per_rank + j (rank r, local slot j); instance
 *     tables `inst_expert[I]` give each instance's logical expert or -1.
 *   - A top-k id of -1 is an empty routing slot (a padded or absent token).  It is
 *     not counted and gets bucket position, instance and row -1.
 *   - Return value: uep_status.  Argument checks run on the host before anything
 *     is enqueued; on an error nothing is enqueued.  UEP_EHIP reports a launch
 *     failure (hipGetLastError).
 *   - Content errors (bad ids, quotas that do not match the load, ...) are found
 *     on the device and OR-ed as UEP_ERR_* bits into the optional device word
 *     `err` (may be NULL).  The caller clears it beforehand and reads it after its
 *     own synchronisation.  Outputs are unspecified when a bit is set.
 *   - Calls are stateless and re-entrant.  Calls that overlap on one stream-less
 *     set of buffers race like any other kernels writing the same memory.
 *   - Limits: R <= 64, E <= 4096, K <= 64, R*T*K < 2^31, total load < 2^31,
 *     hidden size H <= 2^29 for the row moves (a row is one store span).
 */
#ifndef UEP_H
#define UEP_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef int32_t uep_status;
enum {
  UEP_OK = 0,
  UEP_EINVAL = 1,      /* null pointer, negative size, r_begin/r_end out of range */
  UEP_EGEOM = 2,       /* unsupported geometry (limits above, E % R != 0, H % 8 != 0 ...) */
  UEP_EWORKSPACE = 3,  /* workspace missing or smaller than the *_workspace_size query */
  UEP_EHIP = 4         /* a kernel launch or HIP runtime call failed */
};

/* device-side content error bits */
enum {
  UEP_ERR_ID_RANGE = 1,     /* a top-k id outside [-1, E) */
  UEP_ERR_DUP_ID = 2,       /* an expert twice in one token's top-k */
  UEP_ERR_QUOTA_SUM = 4,    /* an expert's instance quotas do not sum to its load */
  UEP_ERR_INST_DUP = 8,     /* two instances of one expert on one rank */
  UEP_ERR_BAD_QUOTA = 16,   /* negative quota, or quota on an unused instance */
  UEP_ERR_COVER = 32,       /* a bucket position not covered by the transfer plan */
  UEP_ERR_LP = 64,          /* LPLB: an expert with load but no instance */
  UEP_ERR_ROW_RANGE = 128,  /* a dest_row entry outside [-1, out_rows) */
  UEP_ERR_LOGIT = 256,      /* a router logit (or logit's bias) that is NaN or +infinity */
  UEP_ERR_GRAD = 512,       /* AdamW: a gradient element that is not finite */
  UEP_ERR_PLAN = 1024,      /* AdamW: not a plan for this call, or a step below 1 */
  UEP_ERR_OFFSET = 2048,    /* an offset table that falls or leaves its rows or tokens */
  UEP_ERR_VALUE = 4096      /* rows to 8 bits: an element that is NaN or infinite */
};

/* element types of the calls that take more than one */
enum { UEP_F32 = 0, UEP_BF16 = 1 };

/* Library version string and a static text for a status code (host). */
const char* uep_version(void);
const char* uep_status_string(uep_status s);

/* ------------------------------------------------------------------------- *
 * uep_device_copy -- plain device-to-device copy, the measured HBM reference line.
 * Not a step of the balancing path: it is the "achievable bandwidth" kernel against
 * which the permute and staging kernels are read, and the known-size kernel that
 * calibrates hardware byte counters.  Each workgroup copies 16 KiB with 16-byte
 * vector loads, all issued before its stores.
 *
 *   src   [bytes]  in   device memory, 16-byte aligned
 *   dst   [bytes]  out  device memory, 16-byte aligned, not overlapping src
 *   bytes               multiple of 16; 0 is a no-op
 * Returns UEP_EINVAL for null pointers or negative size, UEP_EGEOM for misaligned
 * pointers or a size that is not a multiple of 16.
 * ------------------------------------------------------------------------- */
uep_status uep_device_copy(const void* src, void* dst, int64_t bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_device_fill -- writes a 32-bit pattern over device memory.  Not a step of the
 * balancing path: the write-only HBM reference line (the permute and staging
 * streams are mostly writes), and a fill kernel for callers that clear buffers
 * inside a captured graph and want no memset node there.  Same workgroup shape as
 * uep_device_copy (16 KiB per workgroup, 16-byte vector stores).
 *
 *   dst    [bytes]  out  device memory, 16-byte aligned
 *   bytes                multiple of 16; 0 is a no-op
 *   value                the 32-bit word written at every 4-byte offset
 * Returns UEP_EINVAL for a null pointer or negative size, UEP_EGEOM for a misaligned
 * pointer or a size that is not a multiple of 16.
 * ------------------------------------------------------------------------- */
uep_status uep_device_fill(void* dst, int64_t bytes, uint32_t value, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_load_matrix -- the global load matrix of one layer.
 * [UEP] section "在 Gate 之后获取当前层真实负载" (real load after Gate): once the Gate
 * has run, every expert's exact token count for this microbatch and layer is known;
 * the routing metadata of the whole EP group forms the global load matrix.
 *
 *   topk_ids   [R][T][K]  in   expert ids in [-1, E), distinct within a token
 *   counts     [R][E]     out  counts[r][e] = number of (t, k) on rank r routed to e
 *   bucket_pos [R][T][K]  out  number of tokens t' < t on rank r whose top-k holds
 *                              the same expert (stable position in its bucket);
 *                              may be NULL: then only counts are computed (a layer
 *                              that needs the loads but no positions, e.g. the routed
 *                              loads Waterfill starts from), and duplicate ids are
 *                              not checked
 *   err                   out  optional; UEP_ERR_ID_RANGE, UEP_ERR_DUP_ID
 *   ws, ws_bytes               device workspace of uep_load_matrix_workspace_size()
 * ------------------------------------------------------------------------- */
size_t uep_load_matrix_workspace_size(int32_t R, int32_t T, int32_t K, int32_t E);
uep_status uep_load_matrix(const int32_t* topk_ids, int32_t R, int32_t T, int32_t K,
                           int32_t E, int32_t* counts, int32_t* bucket_pos, int32_t* err,
                           void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_load_matrix_noalloc -- uep_load_matrix without a caller workspace, for callers
 * that cannot allocate device memory (code under HIP graph capture, tight serving
 * loops, harnesses that forbid allocation).  Same arguments, outputs and errors as
 * uep_load_matrix minus ws / ws_bytes; the chunk histograms live in an 8 MiB array the
 * library holds on each GPU it runs on, until the process ends.  Geometries whose
 * uep_load_matrix_workspace_size() exceeds 8 MiB return UEP_EWORKSPACE (the layers
 * here need 0.5-5 MiB).  All calls on one GPU share that array: calls that overlap on
 * one GPU (several streams or host threads) race and must be ordered by the caller.
 * Allocates and frees nothing; the first call on a device looks up the array's device
 * address once (UEP_EHIP if that fails).
 * ------------------------------------------------------------------------- */
uep_status uep_load_matrix_noalloc(const int32_t* topk_ids, int32_t R, int32_t T, int32_t K,
                                   int32_t E, int32_t* counts, int32_t* bucket_pos,
                                   int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_solve_quota -- joint replica placement and quota solve.
 * [UEP] section "Quota 同时决定专家副本与 token 分流": a quota is the token load an
 * expert instance receives after rerouting; each search step may instantiate a
 * replica and updates the quota distribution; at most S redundant slots per rank,
 * no logical expert twice on one rank, and a new replica gets at least q_min
 * tokens.  Section "共享冗余 slot 管理动态专家副本": mains never move.
 * Every caller with the same counts gets the same plan (deterministic, ties to
 * the lowest index).  Search ("fill to the waterline", T* = ceil(sum c / R),
 * every step opens one replica, so at most R*S steps):
 *   1. h = the most loaded rank; stop if L_h <= T*, or if L_h - T* < q_min.
 *   2. Plain step: h's mains with quota left, quota descending (id ascending on
 *      ties), each tried in turn: a new replica in the lowest free slot of the
 *      least loaded rank t with L_t < T*, a free slot and no copy of the expert,
 *      taking d = min(q_main, L_h - T*, T* - L_t) if d >= q_min.
 *   3. Relay, when no main of h can move (the quota-distribution update): for h's
 *      mains in the same order, the lowest-index rank x != h with L_x >= T*, a free
 *      slot and no copy of the donor e, one of whose mains f (quota left) has a
 *      replica on a rank y with L_y < T*.  d2 = min(q_f, T* - L_y) moves from f's
 *      main to y's replica, then e opens on x with d = min(q_e, L_h - T*,
 *      T* - (L_x - d2)) if d >= q_min.  Such an x sits exactly at T* and has one
 *      such (f, y) only (a lemma of the search), so no further order applies.
 *   4. Neither moves: stop (stats[3] = 1).
 * No rank ever rises above T*; h's excess falls every step.
 *
 *   counts      [R][E]           in   load matrix (E % R == 0, E_loc = E / R)
 *   S, q_min                          redundant slots per rank (0..8), minimum quota
 *   slot_expert [R][S]           out  expert held by each slot, -1 if empty
 *   inst_expert [R*(E_loc+S)]    out  instance table: j < E_loc main of r*E_loc + j,
 *                                     j >= E_loc slot j - E_loc
 *   inst_quota  [R*(E_loc+S)]    out  tokens each instance takes
 *   rank_load   [R]              out  load per rank after the plan
 *   stats       [4]              out  {replicas placed, steps, T*, 1 if stopped early}
 * ------------------------------------------------------------------------- */
uep_status uep_solve_quota(const int32_t* counts, int32_t R, int32_t E, int32_t S,
                           int32_t q_min, int32_t* slot_expert, int32_t* inst_expert,
                           int32_t* inst_quota, int32_t* rank_load, int32_t* stats,
                           void* stream);

/* ------------------------------------------------------------------------- *
 * uep_identity_quota -- quotas when every expert has exactly one instance
 * (used with the Waterfill layout of [BLOG] section "共享专家融合作为启用机制",
 * where each rank has one shared-expert slot next to its routed experts).
 *
 *   counts      [R][E]     in   R <= 64
 *   inst_expert [n_inst]   in   each expert at most once
 *   inst_quota  [n_inst]   out  total load of the instance's expert (0 if unused)
 * Returns UEP_EINVAL for null pointers or non-positive sizes, UEP_EGEOM for R > 64.
 * ------------------------------------------------------------------------- */
uep_status uep_identity_quota(const int32_t* counts, int32_t R, int32_t E, int32_t n_inst,
                              const int32_t* inst_expert, int32_t* inst_quota, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_reroute_assign -- local-first reroute and per-token realisation.
 * [UEP] section "Quota 同时决定专家副本与 token 分流": tokens first use the instance of
 * their expert on their own rank; what the local quota cannot take goes to remote
 * instances by their remaining quota; the aggregate quotas are then realised per
 * token.  Remote fill = interval overlap: residual demands laid end to end in
 * ascending source rank against remaining capacities in ascending instance id.
 * Dispatch layout: instance blocks in instance-id order; inside a block source
 * rank ascending, then token ascending.  The tokens of (r, e) in token order fill
 * the local instance first, then the remote instances in ascending id.
 *
 *   counts, topk_ids, bucket_pos      in   from uep_load_matrix
 *   inst_per_rank, inst_expert[I],
 *   inst_quota[I]                     in   the plan; I = R * inst_per_rank
 *   r_begin, r_end                    in   per-token outputs only for sources in
 *                                          [r_begin, r_end); xfer/inst_offset always whole
 *   xfer        [R][I]                out  tokens of source r served by instance i
 *   inst_offset [I+1]                 out  first dispatch row of every instance
 *   dest_inst, dest_row [R][T][K]     out  instance and dispatch row of every pair
 *   err                               out  optional; QUOTA_SUM, INST_DUP, BAD_QUOTA, COVER
 *   ws, ws_bytes                           uep_reroute_workspace_size()
 * ------------------------------------------------------------------------- */
size_t uep_reroute_workspace_size(int32_t R, int32_t E, int32_t inst_per_rank);
uep_status uep_reroute_assign(const int32_t* counts, const int32_t* topk_ids,
                              const int32_t* bucket_pos, int32_t R, int32_t T, int32_t K,
                              int32_t E, int32_t inst_per_rank, const int32_t* inst_expert,
                              const int32_t* inst_quota, int32_t r_begin, int32_t r_end,
                              int32_t* xfer, int32_t* inst_offset, int32_t* dest_inst,
                              int32_t* dest_row, int32_t* err, void* ws, size_t ws_bytes,
                              void* stream);

/* ------------------------------------------------------------------------- *
 * uep_plan -- uep_load_matrix, uep_solve_quota and uep_reroute_assign of one layer in
 * one call ([UEP] sections "在 Gate 之后获取当前层真实负载" and "Quota 同时决定专家副本与
 * token 分流": the solve sits on the forward critical path between the Gate and the
 * dispatch).  Outputs and errors are those of the three calls, bit for bit; the solve
 * runs on the finished load matrix concurrently with the bucket-position ranking,
 * which it does not need.  Arguments are the union of the three calls' (S, q_min as
 * uep_solve_quota; r_begin / r_end restrict the assignment as in uep_reroute_assign;
 * inst_per_rank = E / R + S); ws is one workspace of uep_plan_workspace_size() bytes.
 * Geometries off the ranking fast path (E > 1024 or K > 16) run the three calls in
 * sequence.
 * ------------------------------------------------------------------------- */
size_t uep_plan_workspace_size(int32_t R, int32_t T, int32_t K, int32_t E, int32_t S);
uep_status uep_plan(const int32_t* topk_ids, int32_t R, int32_t T, int32_t K, int32_t E,
                    int32_t S, int32_t q_min, int32_t r_begin, int32_t r_end, int32_t* counts,
                    int32_t* bucket_pos, int32_t* slot_expert, int32_t* inst_expert,
                    int32_t* inst_quota, int32_t* rank_load, int32_t* stats, int32_t* xfer,
                    int32_t* inst_offset, int32_t* dest_inst, int32_t* dest_row, int32_t* err,
                    void* ws, size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_permute -- scatter token activations into the per-instance dispatch buffer.
 * [UEP] section "流式通信算子加速动态权重分发": once replica weights are in place,
 * token dispatch follows the reroute plan; this is its on-device permutation.
 * Each source row is read once and written to each of its K rows.
 *
 *   x        [R][T][H] bf16 bits  in   activations (H % 8 == 0, rows 16-byte aligned)
 *   dest_row [R][T][K]            in   from uep_reroute_assign (-1: no row)
 *   r_begin, r_end                     only sources in [r_begin, r_end) are moved
 *   out      [out_rows][H] bf16   out  dispatch buffer, out_rows >= the routed pairs
 *                                      (inst_offset[I] of uep_reroute_assign)
 *   row_src  [out_rows]           out  optional; (r*T + t)*K + k of the pair in each row
 *   err                           out  optional; UEP_ERR_ROW_RANGE: a dest_row entry
 *                                      outside [-1, out_rows), that pair is not moved
 * ------------------------------------------------------------------------- */
uep_status uep_permute(const uint16_t* x, const int32_t* dest_row, int32_t R, int32_t T,
                       int32_t K, int32_t H, int32_t r_begin, int32_t r_end, uint16_t* out,
                       int64_t out_rows, int32_t* row_src, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_combine -- expert outputs from the dispatch buffer back to token order.
 * [BLOG] section "背景知识与设计原则": DeepEP's combine brings each token's routed-
 * expert outputs back after dispatch; section "共享专家融合作为启用机制": a fused
 * shared slot is one more column of the same layout and goes through the same
 * combine.  The pages do not write it out; this is the standard MoE output with the
 * router weights as input:
 *   y[r][t] = bf16( sum_k w[r][t][k] * out[dest_row[r][t][k]] ),  slots with row -1 skipped,
 * each product and addition rounded to nearest even in fp32, k ascending from +0.0,
 * no fused multiply-add, then nearest-even rounding to bf16 (a NaN stays a NaN).
 *
 *   out      [out_rows][H] bf16   in   dispatch buffer (layout of uep_permute's out),
 *                                      16-byte aligned; NULL is taken if out_rows is 0
 *   dest_row [R][T][K]            in   from uep_reroute_assign
 *   gate_w   [R][T][K] fp32       in   combine weights
 *   r_begin, r_end                     only tokens of ranks in [r_begin, r_end) are written
 *   y        [R][T][H] bf16 bits  out  16-byte aligned; other ranks' rows are untouched
 *   err                           out  optional; UEP_ERR_ROW_RANGE: a dest_row entry
 *                                      outside [-1, out_rows), taken as no row
 * Returns UEP_EINVAL / UEP_EGEOM like uep_permute.
 * ------------------------------------------------------------------------- */
uep_status uep_combine(const uint16_t* out, int64_t out_rows, const int32_t* dest_row,
                       const float* gate_w, int32_t R, int32_t T, int32_t K, int32_t H,
                       int32_t r_begin, int32_t r_end, uint16_t* y, int32_t* err,
                       void* stream);

/* ------------------------------------------------------------------------- *
 * uep_stage_replica_weights -- redundant-slot weight staging / gradient reduction.
 * [UEP] section "共享冗余 slot 管理动态专家副本": each rank has S fixed redundant slots
 * (weights + gradient buffer, no optimizer state) shared by every MoE layer; the
 * current layer's replica weights are written into them before dispatch.
 * Section "复用前向方案，完成权重恢复与梯度归约": backward reuses the forward plan,
 * writes the replica weights again, reduces replica gradients into the main's
 * gradient buffer and clears the redundant gradient buffer.
 * Section "流式通信算子加速动态权重分发": fixed-size tiles pulled by a persistent
 * kernel from a device-side task list derived from the plan.
 *
 *   mode = UEP_STAGE_WEIGHTS:     slot_w[r][s] = main_w[slot_expert[r][s]] (bit copy)
 *                                 for used slots of ranks in [r_begin, r_end)
 *   mode = UEP_STAGE_GRAD_REDUCE: for each expert e homed in [r_begin, r_end) with
 *                                 replicas on ranks r1 < r2 < ...:
 *                                 main_grad[e] = ((main_grad[e] + g_r1) + g_r2) + ...
 *                                 in fp32 round-to-nearest-even, then those slot
 *                                 gradients are set to +0.0
 *   slot_expert [R][S]                       in   from uep_solve_quota; entries outside
 *                                                 [0, E) are empty slots (skipped)
 *   main_w  [E][expert_elems] bf16, slot_w [R][S][expert_elems] bf16   (WEIGHTS)
 *   main_grad [E][expert_elems] f32, slot_grad [R][S][expert_elems] f32 (GRAD_REDUCE)
 *   expert_elems % 8 == 0; unused pointers of the other mode may be NULL.
 * ------------------------------------------------------------------------- */
enum { UEP_STAGE_WEIGHTS = 0, UEP_STAGE_GRAD_REDUCE = 1 };
uep_status uep_stage_replica_weights(int32_t mode, int32_t R, int32_t E, int32_t S,
                                     const int32_t* slot_expert, int32_t r_begin,
                                     int32_t r_end, const uint16_t* main_w, uint16_t* slot_w,
                                     float* main_grad, float* slot_grad,
                                     int64_t expert_elems, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_waterfill -- place every token's shared-expert slot on a rank.
 * [BLOG] section "Waterfill算法执行步骤": L_r = routed load on rank r; N shared slots;
 * waterline H = ceil((sum_r L_r + N) / R); slack S_r = max(H - L_r, 0); each token's
 * shared slot goes to a candidate rank sampled in proportion to slack with a small
 * local preference; with zero slack everywhere, a clearly lighter candidate, else
 * the local rank.  Section "通信权衡与模式选择": candidates are the ranks the token
 * already visits plus its own rank (all_ranks = 0), or every rank of the EP group in
 * the all-rank mode (all_ranks != 0).
 * Constants: weights (2^p + 1) * S_r0 for the source rank r0 and 2^p * S_c for the
 * others (p = local_pref_shift, 0..8); draw = word 0 of Philox4x64-10 with counter
 * (r0*T + t, 0, 0, 0) and key (seed, layer), v = floor(draw * W / 2^64); the first
 * candidate (order: r0, then ascending rank) whose running weight exceeds v wins.
 * Zero total weight: the lightest candidate c with (2^p+1) L_c < 2^p L_r0, else r0.
 *
 *   counts     [R][E]      in   routed load matrix (E % R == 0)
 *   topk_ids   [R][T][K]   in
 *   batch_size [R]         in   live tokens per rank B_r <= T (N = sum B_r); tokens
 *                               t >= B_r get shared rank -1
 *   shared_rank[R][T]      out
 *   waterline  [1], slack [R], rank_load [R]  out  H, S_r, L_r
 *   ext_topk   [R][T][K+1] out  optional: top-k plus the column E + shared_rank
 *                               (-1 for absent tokens), i.e. the fused layout
 * ------------------------------------------------------------------------- */
uep_status uep_waterfill(const int32_t* counts, const int32_t* topk_ids,
                         const int32_t* batch_size, int32_t R, int32_t T, int32_t K,
                         int32_t E, uint64_t seed, uint64_t layer, int32_t local_pref_shift,
                         int32_t all_ranks, int32_t* shared_rank, int32_t* waterline,
                         int32_t* slack, int32_t* rank_load, int32_t* ext_topk, void* stream);

/* ------------------------------------------------------------------------- *
 * LPLB -- min-max split of replicated experts' load over their copies.
 * [BLOG] sections "线性规划（LP）公式化构建" and "决策变量与矩阵规模优化": minimise
 * the peak rank load M subject to, per rank, copy allocation + fixed single-copy
 * load + slack = M and, per replicated expert, the split summing to its true count;
 * the structural matrix depends only on the placement and is built once offline,
 * only the right-hand side changes per batch; a Big-M auxiliary column keeps the
 * system feasible and is driven to zero.  Section "从全局计数到LP求解的工程实现":
 * every rank solves the same LP on the GPU with an interior-point method into
 * preallocated buffers.  Section "从LP解决方案到Token调度": the split decides how a
 * replicated expert's tokens go to its copies (here: integer quotas by largest
 * remainder on rint(x * 256), then uep_reroute_assign).
 *
 * uep_lplb_prepare (offline): builds the LP structure from a HOST instance table
 *   inst_expert_host [R*inst_per_rank] (every expert with load needs >= 1 instance,
 *   at most one per rank) and copies it into the device buffer `lp` of
 *   uep_lplb_struct_size() bytes (synchronous copy; call outside the hot loop).
 * uep_lplb (per batch): fp32 Mehrotra predictor-corrector steps, at most `iters`.
 *   counts     [R][E]     in   load matrix
 *   iters                 in   iteration cap (0..200; the solve stops earlier once the
 *                              duality gap is at most 1e-4 of M; 30 is plenty)
 *   x          [n_copies] out  split per copy (token units, copies ordered by expert,
 *                              then instance id), normalised to sum to each count
 *   m          [1]        out  max rank load of that split
 *   inst_quota [I]        out  integer quotas for every instance
 *   stats      [4]        out  optional: {n_replicated, n_copies, iterations run, solve:
 *                              8 or 16 = block solve with lane groups of that size, 0 = dense}
 *   err                   out  optional; UEP_ERR_LP: an expert with load but no instance
 *                              or a column sum of 2^27 or more (the solve still runs), or
 *                              `lp` not a structure from uep_lplb_prepare (then nothing
 *                              else is written)
 * ------------------------------------------------------------------------- */
size_t uep_lplb_struct_size(int32_t R, int32_t E, int32_t inst_per_rank);
uep_status uep_lplb_prepare(const int32_t* inst_expert_host, int32_t R, int32_t E,
                            int32_t inst_per_rank, void* lp, size_t lp_bytes, void* stream);
uep_status uep_lplb(const int32_t* counts, const void* lp, int32_t iters, float* x, float* m,
                    int32_t* inst_quota, int32_t* stats, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_lplb_plan -- uep_load_matrix, uep_lplb and uep_reroute_assign of one layer in one
 * call ([BLOG] sections "从全局计数到LP求解的工程实现" and "从LP解决方案到Token调度": the LP
 * runs on the global counts, then its split decides the token dispatch).  Outputs and
 * errors are those of the three calls, bit for bit; the LP runs on the finished load
 * matrix concurrently with the bucket-position ranking, which it does not need.
 *
 *   topk_ids, R, T, K, E              in   as uep_load_matrix
 *   lp                                in   structure from uep_lplb_prepare for R, E and
 *                                          inst_per_rank; iters as uep_lplb
 *   inst_per_rank, inst_expert[I]     in   the static instance table the structure was
 *                                          built from (I = R * inst_per_rank)
 *   r_begin, r_end                    in   as uep_reroute_assign
 *   counts, bucket_pos                out  as uep_load_matrix
 *   x, m, inst_quota, stats           out  as uep_lplb
 *   xfer, inst_offset, dest_inst,
 *   dest_row                          out  as uep_reroute_assign
 *   err                               out  optional; every bit the three calls set
 *   ws, ws_bytes                           uep_lplb_plan_workspace_size()
 * Geometries off the ranking fast path (E > 1024 or K > 16) run the three calls in
 * sequence.
 * ------------------------------------------------------------------------- */
size_t uep_lplb_plan_workspace_size(int32_t R, int32_t T, int32_t K, int32_t E,
                                    int32_t inst_per_rank);
uep_status uep_lplb_plan(const int32_t* topk_ids, int32_t R, int32_t T, int32_t K, int32_t E,
                         const void* lp, int32_t inst_per_rank, const int32_t* inst_expert,
                         int32_t iters, int32_t r_begin, int32_t r_end, int32_t* counts,
                         int32_t* bucket_pos, float* x, float* m, int32_t* inst_quota,
                         int32_t* stats, int32_t* xfer, int32_t* inst_offset,
                         int32_t* dest_inst, int32_t* dest_row, int32_t* err, void* ws,
                         size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_lplb_sample -- LPLB's per-token copy draw.
 * [BLOG] section "从LP解决方案到Token调度": the split, normalised per replicated expert,
 * is a probability distribution over its physical copies; every token routed to a
 * replicated expert draws one copy from it, and a single-copy expert keeps its only
 * instance.  Weights are the integers w_p = rint(max(x_p, 0) * 256) of uep_lplb's
 * quota step; the draw for slot k of global token g = r*T + t is word k mod 4 u of
 * Philox4x64-10 at counter (g, k div 4, 1, 0), key (seed, layer) (one block of the
 * generator per four slots of a token); v = floor(u * W / 2^64)
 * with W = sum w_p, and the first copy (instance order) whose running weight exceeds
 * v wins; W = 0: copy floor(u * n / 2^64) of the expert's n copies.
 * The dispatch layout then follows from uep_load_matrix on dest_inst (instances as
 * experts, E' = I), uep_identity_quota with the identity table and
 * uep_reroute_assign.
 *
 *   topk_ids  [R][T][K]   in   expert ids (-1: empty slot -> -1)
 *   lp                    in   device structure from uep_lplb_prepare (same R)
 *   x         [n_copies]  in   per-copy split (uep_lplb's x, same copy order)
 *   dest_inst [R][T][K]   out  physical instance of every pair
 *   err                   optional: UEP_ERR_ID_RANGE, UEP_ERR_LP (an expert with no
 *                         instance; or `lp` not a structure from uep_lplb_prepare for R
 *                         ranks, and then every pair is -1)
 * ------------------------------------------------------------------------- */
uep_status uep_lplb_sample(const int32_t* topk_ids, int32_t R, int32_t T, int32_t K,
                           const void* lp, const float* x, uint64_t seed, uint64_t layer,
                           int32_t* dest_inst, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_gate -- the router gate: top-k expert ids and combine weights from the logits.
 * [UEP] section "在 Gate 之后获取当前层真实负载": the path starts where the Gate has run;
 * this is that Gate, so that a layer goes from router logits to the load matrix
 * (topk_ids) and the combine (gate_w) without leaving the library.
 *   scores     softmax: s_e = exp(l_e) / sum_j exp(l_j);  sigmoid: s_e = 1/(1 + exp(-l_e))
 *   selection  the K largest of l_e, or of s_e + bias_e (fp32) where a bias is given, in
 *              descending order, ties to the lowest expert id
 *   weights    w_k = scale * s_k, or with renorm scale * s_k / sum over the selected s
 *              (all weights 0 if that sum is 0)
 * Only finite logits are eligible (and enter the softmax's sum): -infinity, of the logit
 * or of the bias, masks an expert; NaN and +infinity do too and are flagged.  A token with
 * fewer than K eligible experts gets id -1 and weight 0 in the remaining slots.  The selection is
 * over all experts; a selection by groups of experts (some routers take the best groups first)
 * is the caller's, as -infinity in the logits of the groups left out.
 *
 *   logits     [R][T][E]  in   dtype UEP_F32 or UEP_BF16
 *   bias       [E] fp32   in   optional, sigmoid only: enters the selection, not the weights
 *   batch_size [R]        in   optional: tokens t >= batch_size[r] are absent (ids -1,
 *                              weights 0, their logits are not read)
 *   score                      UEP_GATE_SOFTMAX or UEP_GATE_SIGMOID
 *   scale                      finite, not 0
 *   topk_ids   [R][T][K]  out
 *   gate_w     [R][T][K]  out  fp32; sums and exponentials are fp32 (a sigmoid score below
 *                              2^-126 counts as 0).  Neither may overlap another array
 *   err                   out  optional; UEP_ERR_LOGIT
 * Returns UEP_EINVAL for null pointers, sizes < 1 (T may be 0), an unknown dtype or
 * score, a bias with softmax, a bad scale, overlapping outputs; UEP_EGEOM for R > 64, E > 4096, K > 64,
 * K > E, R*T >= 2^26 or R*T*K >= 2^31.
 * ------------------------------------------------------------------------- */
enum { UEP_GATE_SOFTMAX = 0, UEP_GATE_SIGMOID = 1 };
uep_status uep_gate(const void* logits, int32_t dtype, const float* bias,
                    const int32_t* batch_size, int32_t R, int32_t T, int32_t E, int32_t K,
                    int32_t score, int32_t renorm, float scale, int32_t* topk_ids,
                    float* gate_w, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_gate_grad -- gradient of uep_gate's weights with respect to the logits (the
 * selection is piecewise constant, the bias gets no gradient).  With g_k = scale * dw_k
 * and u_k = gate_w_k / scale over the selected slots:
 *   softmax, renorm   dl_k = u_k (g_k - sum_j u_j g_j)
 *   softmax           dl_e = s_e (g_e - sum_j u_j g_j), g_e = 0 unless e is selected
 *   sigmoid, renorm   dl_k = u_k (1 - s_k) (g_k - sum_j u_j g_j)
 *   sigmoid           dl_k = u_k (1 - s_k) g_k
 * with 1 - s_k = 1/(1 + exp(l_k)), which keeps its digits near s_k = 1,
 * and 0 for every other expert.  Slots with id -1 take no part; a token whose slots are
 * all -1 gets zeros.
 *
 *   dgate_w    [R][T][K] fp32  in   gradient of the weights (uep_combine_grad's dgate_w)
 *   logits     [R][T][E]       in   as given to uep_gate
 *   topk_ids, gate_w           in   as written by uep_gate with the same score, renorm
 *                                   and scale
 *   dlogits    [R][T][E]       out  the logits' dtype; every element is written; not
 *                                   overlapping an input (UEP_EINVAL)
 *   err                        out  optional; UEP_ERR_ID_RANGE: an id outside [-1, E),
 *                                   taken as -1
 * Returns UEP_EINVAL / UEP_EGEOM like uep_gate.
 * ------------------------------------------------------------------------- */
uep_status uep_gate_grad(const float* dgate_w, const void* logits, int32_t dtype,
                         const int32_t* topk_ids, const float* gate_w, int32_t R, int32_t T,
                         int32_t E, int32_t K, int32_t score, int32_t renorm, float scale,
                         void* dlogits, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_permute_grad -- gradient of uep_permute: every token sums the gradients of the
 * dispatch rows that hold a copy of it,
 *   dx[r][t] = bf16( sum_k dout[dest_row[r][t][k]] ), slots with row -1 skipped,
 * k ascending from +0.0, additions rounded to nearest even in fp32, then nearest-even
 * rounding to bf16.  [UEP] section "复用前向方案，完成权重恢复与梯度归约": backward reuses
 * the forward plan, here its dest_row.
 *
 *   dout     [out_rows][H] bf16   in   gradient of the dispatch buffer, 16-byte aligned
 *   dest_row [R][T][K]            in   as given to uep_permute
 *   r_begin, r_end                     only tokens of ranks in [r_begin, r_end) are written
 *   dx       [R][T][H] bf16 bits  out  16-byte aligned; other ranks' rows are untouched; not
 *                                      overlapping an input (UEP_EINVAL)
 *   err                           out  optional; UEP_ERR_ROW_RANGE, taken as no row
 * Returns UEP_EINVAL / UEP_EGEOM like uep_permute; dout may be NULL if out_rows is 0.
 * ------------------------------------------------------------------------- */
uep_status uep_permute_grad(const uint16_t* dout, int64_t out_rows, const int32_t* dest_row,
                            int32_t R, int32_t T, int32_t K, int32_t H, int32_t r_begin,
                            int32_t r_end, uint16_t* dx, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_combine_grad -- gradient of uep_combine with respect to the expert outputs and
 * to the combine weights, one pass over both:
 *   dout[dest_row[r][t][k]] = bf16( w[r][t][k] * dy[r][t] )     (one fp32 product)
 *   dgate_w[r][t][k]        = sum_h dy[r][t][h] * out[dest_row[r][t][k]][h]
 * the sum in fp32, in an order that depends on the geometry alone (the same call gives the
 * same bits).  Slots with row -1 move nothing and get dgate_w 0.  Rows of dout that no
 * slot names are left as they are.
 *
 *   dy       [R][T][H] bf16       in   gradient of the combined output, 16-byte aligned
 *   out      [out_rows][H] bf16   in   uep_combine's dispatch buffer; may be NULL together
 *                                      with dgate_w (then only dout is computed)
 *   dest_row [R][T][K]            in   as given to uep_combine (no row named twice)
 *   gate_w   [R][T][K] fp32       in
 *   r_begin, r_end                     only tokens of ranks in [r_begin, r_end)
 *   dout     [out_rows][H] bf16   out  16-byte aligned; may be `out` itself (in place), but
 *                                      overlap it or another array in no other way (UEP_EINVAL)
 *   dgate_w  [R][T][K] fp32       out  slots of other ranks are untouched; not overlapping any
 *                                      other array, gate_w among them (UEP_EINVAL)
 *   err                           out  optional; UEP_ERR_ROW_RANGE, taken as no row
 * Returns UEP_EINVAL / UEP_EGEOM like uep_permute; out and dout may be NULL if out_rows is 0
 * (dgate_w, if given, gets its zeros).
 * ------------------------------------------------------------------------- */
uep_status uep_combine_grad(const uint16_t* dy, const uint16_t* out, int64_t out_rows,
                            const int32_t* dest_row, const float* gate_w, int32_t R, int32_t T,
                            int32_t K, int32_t H, int32_t r_begin, int32_t r_end,
                            uint16_t* dout, float* dgate_w, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * AdamW -- one optimizer step over many tensors in one launch.
 * [UEP] section "共享冗余 slot 管理动态专家副本": redundant slots hold weights and gradients
 * but no optimizer state; after the gradient reduction the mains alone are stepped.
 * For every element, with t the step, lr = sched[0] * lr_scale, g = sched[1] * grad:
 *   m = b1 m + (1 - b1) g;   v = b2 v + (1 - b2) g^2
 *   p = p (1 - lr wd) - lr / (1 - b1^t) * m / (sqrt(v / (1 - b2^t)) + eps)
 * in fp32 (every product and sum of m and v rounded on its own; the quotient within a few
 * units in the last place).  An element whose g is not finite takes g = 0 and is flagged.
 *
 * States are fp32 or 8 bits.  8-bit states keep the upper bits of the fp32 number (its 8
 * exponent bits and 3 mantissa bits: its level), as a distance from the largest level of
 * each block of 256 elements: m in sign and 7 bits, v (never negative) in 8 bits.
 *   code 0 = zero; v code c = level top_v - 255 + c, m code c = level top_m - 127 + c
 *   tops[block] = top_m | top_v << 16; an m below the window becomes 0, a v above 0 never
 *   falls below code 1, so no quotient grows by rounding
 * Both are rounded stochastically (added to the lower 20 bits before they are cut), since
 * a second moment that moves by 1 - b2 of itself a step would otherwise stay where it is
 * for ever.  bf16 parameters are rounded the same way from the fp32 result.  The random
 * bits are a function of (seed, t, the tensor's index, the element's index) alone:
 *   key = mix(mix(t * 0x9E3779B9 + seed) ^ (index + 1));  for the elements 4i .. 4i+3
 *   w0 = mix(i * 0x9E3779B9 ^ key), w1..w5 each the next xorshift (13, 17, 5) of the last
 *   element 4i+j: parameter the lower (j even) or upper half of w[j / 2], m the lower and v
 *   the upper half of w[2 + j];  all 32-bit;
 *   mix(x): x ^= x >> 16; x *= 0x9E3779B9; x ^= x >> 15; x *= 0xBB67AE85; x ^= x >> 16
 * with half a step = 2^15, added in units of 2^-16 of a step.
 *
 * uep_adamw_prepare (offline): copies a HOST table of tensors into the device buffer
 *   `plan` of uep_adamw_plan_size() bytes (synchronous copy; outside the hot loop) and
 *   writes the number of work tiles to *n_tiles (host).  The tensors stay where they are.
 *   Every tensor of a plan has the same types: param_dtype and grad_dtype UEP_F32 or
 *   UEP_BF16, state_bits 32 (m, v fp32) or 8 (m, v uint8, with tops); states start as
 *   zeros.  `copy` is optional with fp32 parameters: the new value rounded to nearest bf16.
 *   Pointers need the alignment of their own type only; tensors in which every group of four
 *   elements is aligned (16 bytes of fp32, 8 of bf16, 4 of codes) are faster.
 *   At most 65535 tensors of at most 2^33 elements, 1.7e10 together.
 * uep_adamw: one step.  n_tiles and the types as given to and by uep_adamw_prepare.
 *   step   [1] int32  in   t >= 1, device memory
 *   sched  [2] fp32   in   {learning rate, factor on every gradient}, device memory, so a
 *                          captured graph can be replayed with new values
 *   0 <= beta1, beta2 < 1, 2^-126 <= eps <= 2^126 (double: 1 - beta is formed before it is
 *   rounded)
 *   err               out  optional; UEP_ERR_GRAD, UEP_ERR_PLAN (then nothing else is written)
 * uep_adamw_decode: the values that 8-bit states stand for (checkpoints), n elements from
 *   the start of a tensor or of several whose starts are multiples of 256 apart;
 *   m, v [n] of dtype UEP_F32 or UEP_BF16 (both hold them exactly); n < 1.7e10
 * ------------------------------------------------------------------------- */
typedef struct uep_adamw_tensor {
  void* param;          /* [n] param_dtype, updated */
  const void* grad;     /* [n] grad_dtype */
  void* m;              /* [n] fp32 or uint8, updated */
  void* v;              /* [n] fp32 or uint8, updated */
  int32_t* tops;        /* [ceil(n / 256)], 8-bit states only (else NULL), updated */
  uint16_t* copy;       /* [n] bf16 bits, written; optional, fp32 parameters only */
  int64_t n;            /* elements, may be 0 */
  float weight_decay;   /* wd */
  float lr_scale;       /* this tensor's factor on the learning rate */
} uep_adamw_tensor;
size_t uep_adamw_plan_size(const uep_adamw_tensor* tensors_host, int32_t count);
uep_status uep_adamw_prepare(const uep_adamw_tensor* tensors_host, int32_t count,
                             int32_t param_dtype, int32_t grad_dtype, int32_t state_bits,
                             void* plan, size_t plan_bytes, int64_t* n_tiles, void* stream);
uep_status uep_adamw(const void* plan, int64_t n_tiles, int32_t param_dtype,
                     int32_t grad_dtype, int32_t state_bits, const int32_t* step,
                     const float* sched, double beta1, double beta2, double eps,
                     uint32_t seed, int32_t* err, void* stream);
uep_status uep_adamw_decode(const uint8_t* m_codes, const uint8_t* v_codes,
                            const int32_t* tops, int64_t n, int32_t dtype, void* m, void* v,
                            void* stream);

/* ------------------------------------------------------------------------- *
 * uep_balance_loss -- the router's balance loss over sequences of tokens, with the per-expert
 * counts and mean scores it is made of.  [UEP] section "在 Gate 之后获取当前层真实负载" balances
 * the load that the Gate produced; the auxiliary loss that keeps that load near even is the
 * page's point of comparison, not written out there; this is the standard one.  Over the
 * tokens of sequence g, of which n_g are present (some id is not -1):
 *   p_te       softmax: exp(l_e) / sum_j exp(l_j);  sigmoid: s_e / sum_j s_j, s = 1/(1 + exp(-l))
 *   counts_ge  ids of expert e;   prob_ge = (sum of p_te over the present tokens) / n_g
 *   loss_g     E / (K n_g) * sum_e counts_ge prob_ge     (1 where both are even; 0 if n_g is 0)
 * A call without seq_offset has n_seq equal sequences of the R*T tokens in order (n_seq = R: a
 * loss for each rank's microbatch; 1: for the whole group).  -infinity masks an expert; NaN
 * and +infinity do too and are flagged, except in an absent token, whose logits may be anything;
 * a token without a finite logit has p = 0.  A sigmoid score below 2^-126 counts as 0.
 *
 *   logits     [R][T][E]    in   dtype UEP_F32 or UEP_BF16
 *   topk_ids   [R][T][K]    in   -1: empty slot
 *   seq_offset [n_seq + 1]  in   optional: sequence g is the tokens r*T + t in
 *                                [seq_offset[g], seq_offset[g+1]), may be empty; tokens outside
 *                                of all belong to none.  Not falling, within [0, R*T]
 *   score                        UEP_GATE_SOFTMAX or UEP_GATE_SIGMOID
 *   loss [n_seq] fp32, counts [n_seq][E], prob [n_seq][E] fp32, tokens [n_seq]    out
 *                                (n_g).  None may overlap another array
 *   err                     out  optional; UEP_ERR_LOGIT, UEP_ERR_ID_RANGE (such an id is taken
 *                                as -1), UEP_ERR_OFFSET
 *   ws, ws_bytes                 uep_balance_loss_workspace_size(), 16-byte aligned; calls that may
 *                                overlap need one each
 * Sums over tokens are fp32 within a block of tokens and 64 bits across blocks, in an order that
 * depends on the geometry and seq_offset alone (the same call gives the same bits).
 * Returns UEP_EINVAL for null pointers, sizes < 1 (T may be 0: every output is 0), an unknown
 * dtype or score, overlapping outputs; UEP_EGEOM for R > 64, E > 4096, K > 64, n_seq > 65535,
 * n_seq*E >= 2^31, R*T >= 2^26, R*T*K >= 2^31, or R*T no multiple of n_seq without seq_offset.
 * ------------------------------------------------------------------------- */
size_t uep_balance_loss_workspace_size(int32_t R, int32_t T, int32_t E, int32_t n_seq);
uep_status uep_balance_loss(const void* logits, int32_t dtype, const int32_t* topk_ids,
                            const int32_t* seq_offset, int32_t n_seq, int32_t R, int32_t T,
                            int32_t E, int32_t K, int32_t score, float* loss, int32_t* counts,
                            float* prob, int32_t* tokens, int32_t* err, void* ws,
                            size_t ws_bytes, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_balance_loss_grad -- gradient of uep_balance_loss with respect to the logits (the
 * counts are piecewise constant).  For a present token of sequence g
 *   dl_e = dloss_g E / (K n_g^2) p_e (counts_ge - sum_j counts_gj p_j)      softmax
 *   the same times 1 - s_e                                                  sigmoid
 * and 0 for other tokens.  With counts and tokens summed over more microbatches than the
 * logits' own, dloss is scaled by their ratio n_own / n_all by the caller.
 *
 *   dloss      [n_seq] fp32    in   gradient of each sequence's loss (device memory)
 *   logits, topk_ids, seq_offset, score    as given to uep_balance_loss
 *   counts [n_seq][E], tokens [n_seq]      as written by it
 *   add        [R][T][E]       in   optional: what the gradient is added to, e.g. that of
 *                                   uep_gate_grad; the logits' dtype; may be `dlogits` itself
 *   dlogits    [R][T][E]       out  the logits' dtype; every element is written (one rounding);
 *                                   overlapping an input in no other way (UEP_EINVAL)
 *   err                        out  optional; UEP_ERR_LOGIT, UEP_ERR_ID_RANGE, UEP_ERR_OFFSET
 * Returns UEP_EINVAL / UEP_EGEOM like uep_balance_loss.
 * ------------------------------------------------------------------------- */
uep_status uep_balance_loss_grad(const float* dloss, const void* logits, int32_t dtype,
                                 const int32_t* topk_ids, const int32_t* counts,
                                 const int32_t* tokens, const int32_t* seq_offset,
                                 int32_t n_seq, int32_t R, int32_t T, int32_t E, int32_t K,
                                 int32_t score, const void* add, void* dlogits, int32_t* err,
                                 void* stream);

/* ------------------------------------------------------------------------- *
 * Rows in 8 bits.  A bf16 row x becomes integers q in [-127, 127] and one fp32 scale:
 *   scale = max(fp32(max_h |x_h| / 127), 2^-126),   q_h = x_h / scale to the nearest integer,
 * the exact quotient, ties to even.  A NaN becomes 0 and an infinity +-127, are flagged and
 * take no part in the maximum.
 *
 * uep_quant_rows: rows in place of each other (expert outputs between two products; the output
 *   channels of a weight matrix, once).
 *     x [rows][H] bf16   in   16-byte aligned, H % 16 == 0, H <= 65536
 *     live_rows [1]      in   optional, device memory: rows at or past it are neither read nor
 *                             written (inst_offset[I] of uep_reroute_assign)
 *     q [rows][H] int8, scale [rows] fp32   out   q 16-byte aligned; not overlapping each other
 *                             or an input
 * uep_permute_quant: the dispatch in 8 bits, uep_permute with half the bytes written: every
 *   token's row is put into 8 bits once and goes to each of its K dispatch rows.
 *     x, dest_row, R, T, K, r_begin, r_end   as uep_permute
 *     q [out_rows][H], scale [out_rows]      out; rows that no slot names are left as they are
 * err   optional; UEP_ERR_VALUE, UEP_ERR_ROW_RANGE (such an entry is taken as no row)
 * Returns UEP_EINVAL for null pointers, negative sizes, overlaps; UEP_EGEOM for H or an
 * alignment that does not fit, and the limits above.
 * ------------------------------------------------------------------------- */
uep_status uep_quant_rows(const uint16_t* x, int64_t rows, int32_t H, const int32_t* live_rows,
                          int8_t* q, float* scale, int32_t* err, void* stream);
uep_status uep_permute_quant(const uint16_t* x, const int32_t* dest_row, int32_t R, int32_t T,
                             int32_t K, int32_t H, int32_t r_begin, int32_t r_end, int8_t* q,
                             float* scale, int64_t out_rows, int32_t* err, void* stream);

/* ------------------------------------------------------------------------- *
 * uep_expert_product -- the experts' matrix product over the dispatch buffer, in 8-bit
 * integers with a scale for each row and each output channel.  [UEP] section "共享冗余 slot
 * 管理动态专家副本": an instance is its rank's main or a replica in a redundant slot, each with
 * weights of its own; this runs all of them on the rows that the plan gave them.
 *   z[p][n] = sum_d q[p][d] w[n][d]  (exact, int32);  y[p][n] = z w_scale[n] q_scale[p]  in fp32
 *   UEP_PRODUCT_PLAIN    out[p][n] = bf16(y[p][n])                                      n < N
 *   UEP_PRODUCT_SWIGLU   out[p][n] = bf16(silu(y[p][n]) y[p][N/2 + n])                n < N/2
 * with silu(g) = g / (1 + exp(-g)) (hardware exp2 and reciprocal, each within a unit in the last
 * place; 0 for gates below -174) and w those of the row's instance i = r * (E/R + S) + j: main r*E/R + j for j < E/R,
 * slot (r, j - E/R) otherwise.  S = 0 and R = 1: one matrix per expert; E = 1 then: a plain
 * product of all rows (a shared expert).
 *
 *   q [rows][D] int8, q_scale [rows] fp32    in   from uep_quant_rows or uep_permute_quant
 *   inst_offset [I+1]         in   first row of every instance, I = R * (E/R + S); from
 *                                  uep_reroute_assign.  NULL if I is 1: all rows.  Rows outside
 *                                  [inst_offset[0], inst_offset[I]) are left as they are
 *   main_w [E][N][D] int8, main_scale [E][N] fp32    in
 *   slot_w [R][S][N][D], slot_scale [R][S][N]        in   NULL if S is 0
 *                                  (uep_stage_replica_weights moves both: N*D/2 and 2*N of its
 *                                  16-bit elements an expert)
 *   out [rows][N or N/2] bf16 bits  out   not overlapping an input (UEP_EINVAL)
 *   err                       out  optional; UEP_ERR_OFFSET: a table that falls or leaves
 *                                  [0, rows]
 * How the work is cut goes by `rows` and the number of instances, on the host: a buffer with many
 * more rows than its table names takes longer than one of the table's size.
 * q, weights and out 16-byte aligned.  D % 16 == 0, D <= 65536, N % 8 == 0 (SwiGLU: 16),
 * N*D < 2^31, S <= 8, rows <= 2^29; otherwise UEP_EGEOM.
 * ------------------------------------------------------------------------- */
enum { UEP_PRODUCT_PLAIN = 0, UEP_PRODUCT_SWIGLU = 1 };
uep_status uep_expert_product(const int8_t* q, const float* q_scale, int64_t rows,
                              const int32_t* inst_offset, int32_t R, int32_t E, int32_t S,
                              const int8_t* main_w, const float* main_scale,
                              const int8_t* slot_w, const float* slot_scale, int32_t N,
                              int32_t D, int32_t act, uint16_t* out, int32_t* err,
                              void* stream);

#ifdef __cplusplus
}
#endif

#endif /* UEP_H */
