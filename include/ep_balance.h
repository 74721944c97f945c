/*
 * ep_balance.h -- real-time MoE expert load balancing on one AMD MI355X (gfx950).
 *
 * The calls follow the problem as the UltraEP pages state it:
 *   - the gate emits top-k *logical* expert IDs per token; experts run as
 *     *physical* instances: each expert's native instance plus copies placed
 *     in a fixed number of reserved spare slots per EP rank, with no runtime
 *     allocation (UltraEP news article, m.youleyou.com, section on the key
 *     designs; UltraEP digest, agihunt.info, "What UltraEP does");
 *   - balancing reads the exact load after the gate, then solves how much load
 *     (a quota) every expert instance receives, jointly with where replicas go
 *     (UltraEP article, key designs, control-plane paragraph);
 *   - tokens of one logical expert are rerouted over its instances (same
 *     section, forward-pass paragraph); the three mapping tables are those of
 *     EPLB: physical slot -> logical expert, logical expert -> replica slots,
 *     replica count per expert (EPLB tutorial, t6page.pages.dev, section on the
 *     mapping tables);
 *   - replica weights are gathered into slot buffers that every layer reuses
 *     (UltraEP article, key designs, memory paragraph);
 *   - imbalance = load of the most loaded rank / mean rank load (UltraEP
 *     digest, "Reported results"); balancedness = its reciprocal (EPLB
 *     tutorial, measured-speedup section).
 *
 * All EP ranks of one layer are simulated on one GPU: the rank is an array
 * axis.  One "plan" is one (microbatch, layer); calls take P plans at once.
 *
 * Departures from the plain five-call sketch of this interface: the layout is
 * one packed device table built by ep_layout_init; ep_plan_quota also returns
 * each plan's move count; ep_balance_stats returns four int64 columns plus the
 * two imbalances as doubles (the move count and the step-cap flag come from
 * the planner); ep_route_noalloc serves callers that cannot allocate.
 *
 * Conventions shared by every call
 *   - Pointers named as device data are device pointers owned by the caller;
 *     the library allocates and frees nothing.
 *   - Every call only enqueues work on `stream` (a hipStream_t; NULL = the
 *     null stream) and returns; it never synchronises.  Calls on different
 *     streams are safe when their outputs do not alias.
 *   - The return value reports errors detectable on the host:
 *       EP_OK, EP_ERR_INVALID_ARG (null/misaligned pointer, bad size, workspace
 *       too small, unsupported shape), EP_ERR_HIP (a HIP runtime call failed).
 *     Data errors found on the device never force a sync: they are reported
 *     in the per-plan status words (EP_STATUS_*).
 *   - The balancing path is integer work throughout; no call's results depend on
 *     scheduling (no order-dependent atomics), so every output is bit-reproducible.
 */
#ifndef EP_BALANCE_H
#define EP_BALANCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef void *ep_stream_t; /* a hipStream_t */

enum {
    EP_OK = 0,
    EP_ERR_INVALID_ARG = -1,
    EP_ERR_HIP = -2,
    EP_ERR_TOO_LARGE = -3, /* ep_route_noalloc: the batch needs more than its scratch */
};

/* bits of the per-plan status word */
enum {
    EP_STATUS_BAD_ID = 1u,   /* an expert ID >= E was seen; such pairs count nowhere */
    EP_STATUS_STEP_CAP = 2u, /* the planner stopped at its step cap                  */
    EP_STATUS_BAD_LOAD = 4u, /* the planner got a load < 0 or a total above INT32_MAX */
};

/*
 * Physical layout of one EP group: native placement + spare slots per rank.
 *
 * Physical slots are numbered rank-major; inside rank r the native experts come
 * first in ascending logical ID, then the rank's spare slots.  The o-th spare
 * slot in that order owns row o of the slot buffer.
 *
 * `tables` points to device memory holding ep_layout_table_ints() int32 values
 * written by ep_layout_init(); the struct itself lives in host memory and is
 * read by every call at enqueue time.
 */
typedef struct ep_layout {
    int32_t num_experts;  /* E: logical experts                                   */
    int32_t num_ranks;    /* R: EP ranks                                          */
    int32_t num_phys;     /* Phi = E + S physical slots                           */
    int32_t num_spare;    /* S: spare slots over all ranks                        */
    int32_t max_replicas; /* rho = min(R, 1 + S): row width of log2phy            */
    int32_t max_rank_natives; /* most native experts on one rank                  */
    int32_t max_rank_spares;  /* most spare slots on one rank                     */
    int32_t ranks_per_domain; /* D > 0: replicas stay in the scale-up domain of     */
                              /* their expert's native rank (rank r is in domain    */
                              /* r / D; an 8-GPU xGMI node on MI355X); 0: anywhere. */
                              /* ep_layout_init sets 0; the caller may change it.   */
    const int32_t *tables;/* device, packed tables (see ep_layout_init)           */
} ep_layout_t;

/* Number of int32 values ep_layout_init writes for (E, R, S). */
size_t ep_layout_table_ints(int32_t num_experts, int32_t num_ranks, int32_t num_spare);

/*
 * Validate a placement, pack its tables on the host and copy them with a
 * blocking hipMemcpy into `device_tables` (caller-owned, at least
 * ep_layout_table_ints(E, R, sum(spare_count)) int32 values).  Fills *out.
 *   native_count  host [R]: native experts of each rank (>= 0, sum = E)
 *   native_experts host [E]: rank-major lists, rank r's block of native_count[r]
 *                  IDs in any order (each logical ID exactly once)
 *   spare_count   host [R]: spare slots of each rank (>= 0)
 * Setup only (once per EP group), not part of the per-plan path.
 * Returns EP_ERR_INVALID_ARG for an invalid placement or a rank count above
 * EP_MAX_RANKS, EP_ERR_HIP if the copy fails.
 */
#define EP_MAX_RANKS 4096
#define EP_MAX_EXPERTS 16384
int ep_layout_init(int32_t num_experts, int32_t num_ranks, const int32_t *native_count,
                   const int32_t *native_experts, const int32_t *spare_count,
                   int32_t *device_tables, size_t device_table_ints, ep_layout_t *out);

/*
 * Workspace for one (ep_load_histogram, ep_reroute) pair, in bytes.  It carries
 * per-expert pair counts from the histogram to the reroute (and the dispatch
 * layout): for every sub-block of consecutive pairs, how many pairs of each
 * expert come before it in the plan, stored as a count within a segment of
 * sub-blocks plus a per-segment base.  With E <= 256 it also holds a one-byte
 * copy of every ID and a flag per sub-block (padding or IDs >= E present),
 * which the reroute reads in place of the int32 IDs of unflagged sub-blocks.
 * Pass the same buffer, untouched in between, with the same N and P.  Grows
 * as P * (sub-blocks + segments + 1) * (E + 1) * 4, about 1/8 to 1/4 byte per
 * pair, plus about 1 byte per pair with E <= 256.
 */
size_t ep_workspace_bytes(int64_t pairs_per_plan, int32_t num_plans, int32_t num_experts);

/*
 * Pairs per sub-block for a launch of P plans of N pairs with E experts: the
 * unit of work of one wave in the histogram, the reroute and the dispatch
 * layout, and the unit of the workspace's count rows (one row of E + 1 int32
 * per sub-block).  A power of two from 1024 up; 0 for invalid sizes.  For
 * callers that account for the workspace's traffic; no call needs it.
 */
int64_t ep_sub_block_pairs(int64_t pairs_per_plan, int32_t num_plans, int32_t num_experts);

/*
 * A1 -- exact per-expert load of every plan (UltraEP article, key designs:
 * the global load is read after the gate and before dispatch).
 *   topk_ids  device int32 [P][N]: N = R*T*k pairs per plan in (source rank,
 *             token, k) order.  ID < 0 is padding (ignored); ID >= E is an
 *             error: status bit EP_STATUS_BAD_ID, the pair is ignored.
 *   load      device int32 [P][E] (written)
 *   ws        device, >= ep_workspace_bytes(N, P, E) bytes, 16-byte aligned
 *   status    device uint32 [P] (written: EP_STATUS_BAD_ID or 0)
 * N may be 0 (loads become 0).  Requires N < 2^31, 1 <= P <= 65535 and
 * E <= 5119 (eight LDS histograms of E + 1 counters in a workgroup's 160 KiB).
 */
int ep_load_histogram(const int32_t *topk_ids, int64_t pairs_per_plan, int32_t num_plans,
                      const ep_layout_t *layout, int32_t *load, void *ws, size_t ws_bytes,
                      uint32_t *status, ep_stream_t stream);

/*
 * A2 -- joint replica placement and per-instance quotas, one independent plan
 * per (microbatch, layer) starting from the native placement (UltraEP article,
 * key designs: each exploration step may create a replica and move load; the
 * pages do not print the solver, so the rule below is this library's reading).
 *
 * Greedy, capped at 2*S + R committed moves (status EP_STATUS_STEP_CAP):
 *   h = most loaded rank (lowest index on ties); candidates = loaded instances
 *   on h by (quota desc, expert asc).  First try to re-level a candidate that
 *   already has replicas, else replicate one onto the least loaded rank (lowest
 *   index on ties) that has a free spare slot and no instance of it, into that
 *   rank's lowest free spare slot.  Every move water-fills the expert's load
 *   over its instances: with other-expert loads b_i sorted by (b, rank), the m*
 *   largest-prefix instances with m*b_(m) < load + sum_{j<=m} b_(j) end at
 *   floor(S/m*) or one more (the extra units to the first S mod m* of them).
 *   With layout->ranks_per_domain = D > 0 the replica rank must also share the
 *   expert's native domain (UltraEP article, section on why it reaches the
 *   optimum: replication stays inside the high-bandwidth scale-up domain).
 *   A move is kept only if it lowers h's load; the loop stops when no move
 *   does.  Replicas left with quota 0 are freed.
 *   load      device int32 [P][E]
 *   phy2log   device int32 [P][Phi]: logical expert of each slot, -1 = empty
 *   phy_quota device int32 [P][Phi]: pairs each instance receives (0 if empty)
 *   logcnt    device int32 [P][E]: instances per expert (>= 1)
 *   log2phy   device int32 [P][E][rho]: instance slots in ascending order, -1 padded
 *   steps     device int32 [P] or NULL: committed moves
 *   status    device uint32 [P] or NULL: EP_STATUS_STEP_CAP and
 *             EP_STATUS_BAD_LOAD are OR-ed in
 * Every load must be >= 0 and a plan's total at most INT32_MAX (true of any
 * histogram of fewer than 2^31 pairs).  A plan that breaks this makes no move:
 * it keeps the native placement (quota = load) and gets EP_STATUS_BAD_LOAD.
 * Requires rho <= 64 (at most 64 instances of one expert), 1 <= P <= 65535,
 * and either R <= 64 with at most 8 natives and 16 spare slots per rank, or
 * tables that fit the generic kernel's 160 KiB of LDS (about 60 bytes per rank
 * and per expert: R = E up to about 2700); other layouts return
 * EP_ERR_INVALID_ARG.
 */
int ep_plan_quota(const int32_t *load, int32_t num_plans, const ep_layout_t *layout,
                  int32_t *phy2log, int32_t *phy_quota, int32_t *logcnt, int32_t *log2phy,
                  int32_t *steps, uint32_t *status, ep_stream_t stream);

/*
 * A3 -- order-preserving reroute of every (token,k) pair to a physical instance
 * of its own logical expert (UltraEP article, key designs: reroute splits one
 * native expert's tokens over its replicas; EPLB tutorial: the physical ID is
 * looked up from the top-k logical ID).  The j-th pair (0-based, flat order)
 * of expert e goes to the instance i (ascending slot order) with
 * Q_i <= j < Q_i + quota_i, Q_i the sum of the quotas of the instances before i.
 *   topk_ids  device int32 [P][N], the same IDs the histogram saw (with
 *             E <= 256 most pairs are read from the workspace's byte copy;
 *             pairs are read here only in sub-blocks that hold padding or bad
 *             IDs, where phys_ids is not 16-byte aligned, and after a
 *             sub-block's last whole 256-pair tile)
 *   phy_quota, log2phy, logcnt: a plan as ep_plan_quota writes it (each
 *             instance a distinct slot in [0, Phi), logcnt in [0, rho])
 *   ws        the workspace filled by ep_load_histogram for these IDs
 *   phys_ids  device int32 [P][N] (written): physical slot, -1 for padding,
 *             invalid IDs and pairs beyond the expert's total quota
 * phys_ids 4-byte aligned.  LDS bounds the shape: 16 E + 8 Phi + 256 bytes
 * must fit 160 KiB (E up to about 6800 at Phi = E); otherwise, and for a ws
 * smaller than ep_workspace_bytes(N, P, E), EP_ERR_INVALID_ARG.
 */
int ep_reroute(const int32_t *topk_ids, int64_t pairs_per_plan, int32_t num_plans,
               const ep_layout_t *layout, const int32_t *phy_quota, const int32_t *log2phy,
               const int32_t *logcnt, const void *ws, size_t ws_bytes, int32_t *phys_ids,
               ep_stream_t stream);

/*
 * A1 -> A2 -> A3 over a batch of plans (e.g. every MoE layer of a microbatch)
 * cut into chunks that overlap across three streams: one planner launch lasts
 * about as long as its slowest plan, so the planner of chunk c runs while the
 * histogram of chunk c + 1 streams, and the reroute of chunk c while the
 * planner of chunk c + 1 runs.  The outputs are exactly those of
 * ep_load_histogram, ep_plan_quota and ep_reroute made in order on one stream
 * (arguments and layouts as there, P plans).  Kernels of two streams run side
 * by side only when the streams sit on different hardware queues; the HIP
 * runtime spreads streams over its queues (GPU_MAX_HW_QUEUES of them, 4 by
 * default) in creation order, so three streams created one after another get
 * three queues, whereas a side stream that shares the queue of the caller's
 * busy stream loses the overlap.
 *   chunk_plans  host int32 [num_chunks]: plans per chunk, each >= 1, summing
 *                to P; 1 <= num_chunks <= EP_MAX_CHUNKS
 *   ws           device, >= ep_pipeline_workspace_bytes(N, chunk_plans,
 *                num_chunks, E) bytes, 16-byte aligned: one histogram
 *                workspace per chunk
 *   stream       the caller's stream: the chain starts after the work already
 *                enqueued there and later work there waits for all of it
 *   side_streams host array of three distinct streams of the caller, none of
 *                them `stream`, default priority: histograms run on [0],
 *                planners on [1], reroutes on [2]
 *   events       2 + 2 * num_chunks events of the caller (hipEvent_t, e.g.
 *                created with hipEventDisableTiming), recorded and waited on
 *                here; no other work may use them until the chain completes
 * Returns EP_ERR_INVALID_ARG (nothing enqueued) for bad arguments, including
 * any that one of the three calls would reject for a chunk.
 */
#define EP_MAX_CHUNKS 16
size_t ep_pipeline_workspace_bytes(int64_t pairs_per_plan, const int32_t *chunk_plans, int32_t num_chunks,
                                   int32_t num_experts);
int ep_route_pipelined(const int32_t *topk_ids, int64_t pairs_per_plan, int32_t num_plans,
                       const ep_layout_t *layout, const int32_t *chunk_plans, int32_t num_chunks,
                       int32_t *load, uint32_t *status, int32_t *phy2log, int32_t *phy_quota,
                       int32_t *logcnt, int32_t *log2phy, int32_t *steps, int32_t *phys_ids, void *ws,
                       size_t ws_bytes, ep_stream_t stream, const ep_stream_t *side_streams,
                       void *const *events);

/*
 * Next row after A3 -- dispatch layout for the token all-to-all (EPLB
 * tutorial, EPLB / DeepEP section: dispatch sends each pair to its physical
 * replica; combine gathers results back to the logical expert).  Pairs are
 * laid out physical-slot-major: slot s owns positions [off_s, off_s + quota_s)
 * with off the exclusive prefix of the quotas in slot order, and the j-th pair
 * of expert e, served by the instance whose quota range starts at Q, sits at
 * off_s + (j - Q): for plans whose quotas cover the loads, the stable counting
 * sort of the pairs by physical slot.
 *   topk_ids, plan tables, ws  as for ep_reroute (the same histogram workspace)
 *   slot_offsets  device int32 [P][Phi+1] (written): off_s, last entry = total
 *   dispatch_pos  device int32 [P][N] (written): position of each pair, -1 for
 *                 padding, invalid IDs and pairs past the expert's quotas
 *   dispatch_src  device int32 [P][N] (written): pair index (within the plan)
 *                 at each position, -1 for positions no pair takes
 * All output arrays 4-byte aligned.  LDS bounds the shape: 24 E + 12 Phi + 20
 * bytes must fit 160 KiB (about E <= 4500 at Phi = E).
 */
int ep_dispatch_layout(const int32_t *topk_ids, int64_t pairs_per_plan, int32_t num_plans,
                       const ep_layout_t *layout, const int32_t *phy_quota, const int32_t *log2phy,
                       const int32_t *logcnt, const void *ws, size_t ws_bytes,
                       int32_t *slot_offsets, int32_t *dispatch_pos, int32_t *dispatch_src,
                       ep_stream_t stream);

/*
 * A4 -- weight distribution on one GPU: gather the weights of every expert that
 * occupies a spare slot into that slot's row of the cross-layer slot buffer
 * (UltraEP article, key designs: reserved slots, weight buffers reused across
 * layers).  One plan (one layer) per call; empty spare slots are not written.
 * Each distinct expert is read once (with a workspace: once per group of up to
 * 4 of its slots) and stored into every slot that holds it.
 *   expert_weights device [E][bytes_per_expert], one layer (16-byte aligned)
 *   phy2log        device int32 [Phi], that layer's plan
 *   slot_buf       device [S][bytes_per_expert] (16-byte aligned)
 *   ws             device, ep_slot_fill_workspace_bytes(layout) bytes (16-byte
 *                  aligned), or NULL: with it the call first lists the plan's
 *                  distinct experts and their slots there (a one-workgroup
 *                  kernel) and then streams each expert's weights in address
 *                  order, the faster form; without it every workgroup finds
 *                  its slot's expert itself.  The workspace holds no state
 *                  between calls; calls in flight at once need their own.
 * bytes_per_expert must be a positive multiple of 16.  A spare slot whose
 * phy2log entry lies outside [0, E) is empty: its row is not written.
 */
size_t ep_slot_fill_workspace_bytes(const ep_layout_t *layout);
int ep_slot_fill(const void *expert_weights, int64_t bytes_per_expert, const int32_t *phy2log,
                 const ep_layout_t *layout, void *slot_buf, void *ws, size_t ws_bytes,
                 ep_stream_t stream);

/*
 * Next row -- replica gradient reduction in backward (UltraEP article, key
 * designs: replicas keep no optimizer state and their gradients are reduced
 * back to the native expert; backward paragraph: accumulation keeps a fixed
 * order so the reduction is deterministic).  One plan (one layer) per call:
 * for every expert with logcnt >= 2, its native row becomes the fp32 fold of
 * its instances' gradient rows in ascending physical-slot order
 *     acc = g(inst 0); acc = acc + g(inst 1); ...
 * reading native_grads[e] for the native instance and slot_grads[o] for the
 * replica in the o-th spare slot.  Other rows and slot_grads are not written.
 *   native_grads device float [E][n] (in/out), 16-byte aligned
 *   slot_grads   device float [S][n], the gradient half of the slot buffer
 *   log2phy, logcnt  that layer's plan (ep_plan_quota)
 * n = elems_per_expert must be a positive multiple of 4; requires rho <= 64 and
 * E <= 65535.  Rows of experts whose instance list names a slot outside
 * [0, Phi) are left unchanged.
 */
int ep_replica_grad_reduce(float *native_grads, int64_t elems_per_expert, const float *slot_grads,
                           const int32_t *log2phy, const int32_t *logcnt, const ep_layout_t *layout,
                           ep_stream_t stream);

/*
 * A5 -- balance statistics per plan (UltraEP digest, "Reported results":
 * most loaded rank over the mean).
 *   stats      device int64 [P][4]: max rank load before (native placement),
 *              max rank load after (sum of quotas per rank), total load,
 *              replicas in use (spare slots with a positive quota)
 *   imbalance  device double [P][2]: before, after = max * R / total (exactly
 *              rounded; 1.0 when total == 0)
 *   rank_load  device int32 [P][2][R] or NULL: per-rank loads before / after
 */
int ep_balance_stats(const int32_t *load, const int32_t *phy_quota, int32_t num_plans,
                     const ep_layout_t *layout, int64_t *stats, double *imbalance,
                     int32_t *rank_load, ep_stream_t stream);

/*
 * For callers that cannot allocate device memory (code under graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): ep_load_histogram,
 * ep_plan_quota and ep_reroute in one call, with the workspace that carries
 * the histogram's per-sub-block counts (and byte copy) to the reroute held in
 * a device array of the library instead of a caller buffer.  The outputs are
 * exactly those of the three calls (same arguments, same meaning, same
 * layouts; status is written as the histogram writes it, then the planner's
 * flag is OR-ed in).  The call allocates nothing and never synchronises.
 *
 * The array is EP_NOALLOC_SCRATCH_BYTES (64 MiB) per GPU, held by every GPU
 * the library runs this call on until the process ends.  A batch whose
 * workspace, ep_workspace_bytes(N, P, E), is larger returns EP_ERR_TOO_LARGE
 * and enqueues nothing; 64 MiB holds, for example, 14 plans of 4.2M pairs at
 * E = 128 (a plan = one layer of an EP64 group with 8192 tokens per rank,
 * top-8) or 75 such plans at E = 384.  All argument checks of the three calls run before
 * anything is enqueued.  Every call on one GPU shares that GPU's array, so
 * calls whose work overlaps on one GPU (other streams, other host threads)
 * race and corrupt each other's results: serialise them (one stream, or
 * events) on each GPU.
 */
#define EP_NOALLOC_SCRATCH_BYTES (64u << 20)
int ep_route_noalloc(const int32_t *topk_ids, int64_t pairs_per_plan, int32_t num_plans,
                     const ep_layout_t *layout, int32_t *load, uint32_t *status, int32_t *phy2log,
                     int32_t *phy_quota, int32_t *logcnt, int32_t *log2phy, int32_t *steps,
                     int32_t *phys_ids, ep_stream_t stream);

/* ---------------------------------------------------------------------------
 * The layer around the balancer: the gate that makes the expert IDs, the
 * experts' products over the dispatch order, the layer for a few tokens and
 * the optimizer step on the folded gradients.  The conventions above hold:
 * device pointers of the caller, no allocation, enqueue only, results that do
 * not depend on scheduling.
 * ------------------------------------------------------------------------- */
enum {
    EP_DTYPE_F32 = 0,
    EP_DTYPE_BF16 = 1,
    EP_DTYPE_FP8 = 2, /* OCP e4m3 with power-of-two block scales, see ep_quant_rows */
};

/*
 * Gate: the top-k experts of every token and their weights.
 *   score  s_e = logit_e + bias_e in fp32; NaN counts as -inf, and -inf (an
 *          expert switched off, a padded token) is never chosen
 *   groups num_groups > 1: experts form equal consecutive groups, a group's
 *          score is its best s, and only the topk_groups best groups stay
 *          (equal ones: lowest group)
 *   chosen the top_k largest s, in descending order (equal ones: lowest
 *          expert); where fewer are left, ID -1 (padding to the calls above)
 *          and weight 0
 *   weight w_j = scale * exp(logit_j) / sum_i exp(logit_i) over the chosen
 *          (without the bias), computed from the largest one on
 * num_experts <= 1024, top_k <= 16, num_groups <= 16 and dividing num_experts.
 */
typedef struct ep_gate {
    int32_t num_experts, top_k;
    int32_t num_groups, topk_groups; /* 1, 1: no group limit */
    int32_t logits_dtype;            /* EP_DTYPE_F32 or EP_DTYPE_BF16 */
    float scale;                     /* finite */
    const float *bias;               /* device [E] or NULL; moves the choice, not the weights */
} ep_gate_t;

/*
 *   logits   device [T][stride], stride >= E elements
 *   ids      device int32 [T][k], weights device float [T][k] (written)
 */
int ep_gate_topk(const void *logits, int64_t stride, int64_t num_tokens, const ep_gate_t *gate, int32_t *ids,
                 float *weights, ep_stream_t stream);

/*
 * Gradient of the weights with respect to the logits:
 *   dl_j = w_j (g_j - sum_i w_i g_i / scale) at the chosen experts, 0 elsewhere.
 * gate: num_experts, top_k, scale and logits_dtype (of grad_logits) are used.
 *   ids, weights  as ep_gate_topk wrote them; grad_weights device float [T][k]
 *   grad_logits   device [T][E], every element written
 */
int ep_gate_topk_backward(const int32_t *ids, const float *weights, const float *grad_weights, int64_t num_tokens,
                          const ep_gate_t *gate, void *grad_logits, ep_stream_t stream);

/*
 * 8-bit floating point with a scale for each block of 128: values are OCP e4m3
 * bytes, and a block's scale is the byte c, standing for 2^(c - 127), the
 * smallest power of two that brings the block's largest finite magnitude to 448
 * at most.  Rounding is to nearest, ties to even; NaN and infinities become NaN.
 *
 * ep_quant_rows: blocks of 128 columns of one row, for activations.
 *   x      device [rows][stride] fp32 or bf16
 *   q      device bytes [rows][cols up to a multiple of 128], zeros past cols, 16-byte aligned
 *   scale  device bytes [rows][ep_scale_stride(cols)] (the number of blocks up
 *          to a multiple of 4; the bytes past the blocks are 127), 4-byte aligned
 * ep_swiglu_quant: the same for silu(g) * u, where a bf16 row of 2 * inter
 * values holds g and then u.
 * ep_quant_blocks: blocks of 128 rows x 128 columns, for weights.
 *   w      device [groups][rows][cols], group_stride elements between groups
 *   q      bytes [groups][rows][cols up to 128], scale bytes
 *          [groups][row blocks][column blocks]; with transpose != 0 those of
 *          the transposed matrices: q [groups][cols][rows up to 128], scale
 *          [groups][column blocks][row blocks], the same values
 */
int64_t ep_scale_stride(int64_t cols);
int ep_quant_rows(const void *x, int32_t dtype, int64_t rows, int64_t cols, int64_t stride, uint8_t *q,
                  uint8_t *scale, ep_stream_t stream);
int ep_swiglu_quant(const void *gate_up, int64_t rows, int64_t inter, uint8_t *q, uint8_t *scale,
                    ep_stream_t stream);
int ep_quant_blocks(const void *w, int32_t dtype, int32_t groups, int64_t group_stride, int64_t rows, int64_t cols,
                    int32_t transpose, uint8_t *q, uint8_t *scale, ep_stream_t stream);

/* The matrices of a set of experts; `stride` bytes and `scale_stride` bytes from
 * one expert to the next, so that a matrix may be a part of a packed expert row.
 * data 16-byte aligned, stride a multiple of 16.  scale: NULL unless the data
 * are EP_DTYPE_FP8. */
typedef struct ep_matrix {
    const void *data;
    const uint8_t *scale;
    int64_t stride, scale_stride;
} ep_matrix_t;

/*
 * Grouped product: y[i] = w_g x[r(i)] for the output rows i of group g, the
 * consecutive rows offsets[g] .. offsets[g + 1] - 1, offsets[0] = 0.  Rows from
 * offsets[groups] on become 0.  Offsets live on the device and cannot be refused:
 * values outside [0, m] are brought into it and a group that ends before its start
 * is empty, so that no access leaves a buffer.  Groups that overlap for that
 * reason each multiply their rows; a row of several holds one of their products.
 *   x, x_scale  as ep_quant_rows writes them: k columns, x_rows rows
 *   rows        device int32 [m] or NULL: r(i) = rows[i] / rows_div (the pair
 *               that a dispatch position serves, rows_div = top-k); a negative
 *               or too large row gives y[i] = 0.  NULL: r(i) = i, x_rows >= m
 *   offsets     device int32 [groups + 1], or NULL with one group: all rows
 *   w           [groups][n][k], as ep_quant_blocks writes them
 *   layout      NULL, or the layout whose physical slots are the groups: then w
 *               holds the native experts [E] and slot_w the spare slots [S]
 *               (the slot buffer), and slot_offsets of ep_dispatch_layout are
 *               the offsets
 *   y           device bf16 [m][n], every element written (with such offsets)
 * The input gradient is the same call on the quantised output gradient with
 * weights from ep_quant_blocks(transpose = 1).  m < 2^31 - 1024.
 */
typedef struct ep_grouped_matmul {
    const void *x;
    const uint8_t *x_scale;
    int64_t x_rows;
    const int32_t *rows;
    int32_t rows_div;
    int32_t groups;
    const int32_t *offsets;
    int64_t m, n, k;
    ep_matrix_t w, slot_w;
    const ep_layout_t *layout;
    void *y;
} ep_grouped_matmul_t;
int ep_grouped_matmul(const ep_grouped_matmul_t *p, ep_stream_t stream);

/*
 * Weight gradient of the grouped product: out_g[n][k] = sum over the rows i of
 * group g of dy[i][n] x[i][k], fp32, every element written (0 for an empty
 * group).  dy, x: device bf16 [m][dy_stride], [m][x_stride] (elements).
 * groups, offsets as above.  With a layout the physical slots' gradients go to
 * out [E] (native) and slot_out [S], the two inputs of ep_replica_grad_reduce.
 * out_stride, slot_out_stride: floats from one group to the next.
 */
typedef struct ep_grouped_wgrad {
    const void *dy, *x;
    int64_t dy_stride, x_stride;
    int64_t m, n, k;
    int32_t groups;
    const int32_t *offsets;
    const ep_layout_t *layout;
    float *out, *slot_out;
    int64_t out_stride, slot_out_stride;
} ep_grouped_wgrad_t;
int ep_grouped_wgrad(const ep_grouped_wgrad_t *p, ep_stream_t stream);

/*
 * The same from rows of x that are held in 8 bits, as ep_quant_rows or
 * ep_grouped_swiglu wrote them, each operand gathered or not:
 *   out_g[n][k] = sum over the rows i of group g of dy[d(i)][n] x[r(i)][k]
 * fp32, every element written.  d(i) = dy_places[i] / rows_div, or i without dy_places;
 * r(i) likewise with x_places.  Given both, they are one and the same list.  A row whose
 * place is negative or too large adds nothing.
 *   dy       device bf16 [dy_rows][dy_stride], dy_stride < 2^31; dy_rows >= m without
 *            dy_places
 *   x, x_scale  rows of k values in 8 bits, x_rows of them; x_rows >= m without x_places
 *   dy_places, x_places  device int32 [m] or NULL
 *   ws       ep_wgrad_mixed_workspace_bytes(x_rows, k) bytes, 16-byte aligned: x in
 *            bf16, twice its bytes; no state between calls, calls in flight at once
 *            need their own.  bf16 holds x's values under scale bytes from 3 to 246
 *            exactly; under smaller ones those below 2^-133 are rounded to multiples of
 *            it, under larger ones those from 2^128 on are infinite
 */
typedef struct ep_grouped_wgrad_mixed {
    const void *dy;
    int64_t dy_rows, dy_stride;
    const void *x;
    const uint8_t *x_scale;
    int64_t x_rows;
    const int32_t *dy_places, *x_places;
    int32_t rows_div;
    int32_t groups;
    const int32_t *offsets;
    int64_t m, n, k;
    const ep_layout_t *layout;
    float *out, *slot_out;
    int64_t out_stride, slot_out_stride;
    void *ws;
    size_t ws_bytes;
} ep_grouped_wgrad_mixed_t;
size_t ep_wgrad_mixed_workspace_bytes(int64_t x_rows, int64_t k);
int ep_grouped_wgrad_mixed(const ep_grouped_wgrad_mixed_t *p, ep_stream_t stream);

/*
 * The gated feed-forward block over the same groups of rows.  For output row i of
 * group g with the input row r(i), as in ep_grouped_matmul:
 *   a = gate_g x[r(i)],  b = up_g x[r(i)],  h[i] = w_i silu(a) b   (fp32, then 8 bits)
 * with w_i = weights[rows[i]] (rows NULL: weights[i]; weights NULL: 1).  With the
 * combine's weights here, the combine after the product of h with the matrices
 * back takes weights of 1.
 *   gate, up, slot_gate, slot_up   [groups][inter][k], as ep_quant_blocks writes each
 *   weights  device float [weights_count] or NULL; a row of a pair past them has no
 *            input (rows NULL: weights_count >= m)
 *   h, h_scale  rows of inter values in 8 bits (the layout of ep_quant_rows), every
 *            byte written; rows without an input (rows[i] negative or too large) and rows
 *            from offsets[groups] on are rows of zeros
 *   keep     NULL, or what ep_grouped_swiglu_backward needs of a and b, keep_dtype:
 *            EP_DTYPE_BF16  bf16 [m][2 * inter], a and then b
 *            EP_DTYPE_FP8   in 8 bits: bytes [m][2 * I], I = inter up to a multiple of
 *                           128: a, zeros, b, zeros, and keep_scale with
 *                           ep_scale_stride(2 * I) bytes a row
 *            rows without an input and past the groups: zeros
 * Roundings of h (and of q below) are to nearest as in ep_quant_rows, but ties go
 * away from zero; a and b in 8 bits are rounded as there.
 *   sums8    0: the sums are of fp32's precision, so that few values are rounded to
 *            8 bits another way than the sums' exact values.  1: those of
 *            ep_grouped_matmul, in little more than half the time for many rows; they
 *            are off by up to 6e-5 of a result where some columns of x are much larger
 *            than others, and send one value in 300 the other way, by a sixteenth of it
 * A row's outputs do not depend on the other rows.  With sums8 = 0 both operands are
 * taken in bf16, which holds their values under scale bytes from 3 to 246 exactly; under
 * smaller ones those below 2^-133 are rounded to multiples of it, under larger ones
 * those from 2^128 on are infinite.
 */
typedef struct ep_grouped_swiglu {
    const void *x;
    const uint8_t *x_scale;
    int64_t x_rows;
    const int32_t *rows;
    int32_t rows_div;
    int32_t groups;
    const int32_t *offsets;
    int64_t m, inter, k;
    ep_matrix_t gate, up, slot_gate, slot_up;
    const ep_layout_t *layout;
    const float *weights;
    int64_t weights_count;
    uint8_t *h, *h_scale;
    int32_t keep_dtype;
    void *keep;
    uint8_t *keep_scale;
    int32_t sums8;
} ep_grouped_swiglu_t;
int ep_grouped_swiglu(const ep_grouped_swiglu_t *p, ep_stream_t stream);

/*
 * Its gradient, from the gradient dy of the block's output (a row for each token)
 * and from a, b as they were kept.  With d = down_g^T dy[r(i)], s = sigmoid(a):
 *   da = w_i d b s (1 + a (1 - s)),  db = w_i d a s,  dw_i = sum over inter of d a s b
 *   dy, dy_scale, dy_rows, rows, rows_div, groups, offsets, m, layout  as x and the
 *            rest there; k columns (the block's output)
 *   down, slot_down   [groups][inter][k]: the matrices back as ep_quant_blocks(transpose = 1)
 *            writes them
 *   keep, keep_dtype, keep_scale, weights  as ep_grouped_swiglu wrote or took them
 *   grad     device bf16 [m][2 * inter]: da and then db, the dy of the weight gradient; or NULL
 *   q, q_scale  the same in 8 bits in the layout of keep: the x of the grouped product
 *            that gives the input gradient, with the matrices [groups][hidden][2 * I];
 *            or NULL
 *   grad_weights  device float or bf16 (grad_weights_dtype) [pairs], or NULL: dw at
 *            i = pos[pair], 0 where pos is outside [0, m); pos NULL: dw_i, pairs == m
 *   ws       with grad_weights: ep_swiglu_backward_workspace_bytes(m, inter) bytes, 16-byte
 *            aligned; no state between calls, calls in flight at once need their own
 *   sums8    as there; with 1, d and so dw keep about 16 bits
 * Every element of the outputs is written; rows without a dy are zeros.
 */
typedef struct ep_grouped_swiglu_backward {
    const void *dy;
    const uint8_t *dy_scale;
    int64_t dy_rows;
    const int32_t *rows;
    int32_t rows_div;
    int32_t groups;
    const int32_t *offsets;
    int64_t m, inter, k;
    ep_matrix_t down, slot_down;
    const ep_layout_t *layout;
    const float *weights;
    int64_t weights_count;
    int32_t keep_dtype;
    const void *keep;
    const uint8_t *keep_scale;
    void *grad;
    uint8_t *q, *q_scale;
    void *grad_weights;
    int32_t grad_weights_dtype;
    const int32_t *pos;
    int64_t pairs;
    void *ws;
    size_t ws_bytes;
    int32_t sums8;
} ep_grouped_swiglu_backward_t;
size_t ep_swiglu_backward_workspace_bytes(int64_t m, int64_t inter);
int ep_grouped_swiglu_backward(const ep_grouped_swiglu_backward_t *p, ep_stream_t stream);

/*
 * Combine: out_t = sum_j weights[t][j] * y[pos[t][j]] in fp32, j ascending,
 * rounded to bf16 once.  pos: device int32 [T][k] (dispatch_pos of
 * ep_dispatch_layout); positions outside [0, rows) give nothing.  y: bf16
 * [rows][hidden], out: bf16 [T][hidden].
 */
int ep_moe_combine(const void *y, int64_t rows, const int32_t *pos, const float *weights, int64_t num_tokens,
                   int32_t top_k, int64_t hidden, void *out, ep_stream_t stream);

/*
 * A whole mixture-of-experts layer for up to EP_MAX_FEW_TOKENS tokens:
 *   ids, w  as ep_gate_topk
 *   out_t = sum_j w_tj down_e (silu(gate_e x_t) * (up_e x_t)),  e = ids_tj >= 0
 * summed in fp32 and rounded to bf16 once; between the products h is held as the
 * sum of two bf16, 16 bits of mantissa.  With up to 8 tokens every distinct expert's
 * weights are read once; with more, gate and up once for every 32 of its tokens
 * and down once for every 16.  The experts are the native ones: there is no layout.
 *   x        device bf16 [T][x_stride], 16-byte aligned, x_stride a multiple of 8
 *   logits   as for ep_gate_topk
 *   experts  bf16 matrices gate, up [E][inter][hidden], down [E][hidden][inter],
 *            or the same in 8 bits as ep_quant_blocks writes them (x stays bf16;
 *            bytes past a row's columns must be 0); hidden and inter multiples of 8
 *   out      device bf16 [T][out_stride] (written)
 *   ids, weights  device [T][k] (written)
 *   ws       device, ep_few_tokens_workspace_bytes(T, k, hidden, inter) bytes, 16-byte
 *            aligned; no state between calls, calls in flight at once need their own
 */
#define EP_MAX_FEW_TOKENS 64
typedef struct ep_experts {
    int32_t hidden, inter;
    int32_t dtype; /* EP_DTYPE_BF16 or EP_DTYPE_FP8 */
    ep_matrix_t gate, up, down;
} ep_experts_t;
size_t ep_few_tokens_workspace_bytes(int32_t num_tokens, int32_t top_k, int32_t hidden, int32_t inter);
int ep_moe_few_tokens(const void *x, int64_t x_stride, int32_t num_tokens, const void *logits, int64_t logits_stride,
                      const ep_gate_t *gate, const ep_experts_t *experts, void *out, int64_t out_stride, int32_t *ids,
                      float *weights, void *ws, size_t ws_bytes, ep_stream_t stream);

/*
 * AdamW over many tensors in one launch (one for every 48 tensors), in place:
 *   g = grad * grad_scale,  m = beta1 m + (1 - beta1) g,  v = beta2 v + (1 - beta2) g^2
 *   p = p (1 - lr wd) - lr / (1 - beta1^step) * m / (sqrt(v) / sqrt(1 - beta2^step) + eps)
 * in fp32, each operation rounded.  state_bits 32: exp_avg, exp_avg_sq are
 * float [numel].  state_bits 8: they are bytes [numel] with a scale byte c
 * (2^(c - 127)) for each 128 elements in exp_avg_scale, exp_avg_sq_scale
 * [ceil(numel / 128)]; m as sign, 4 bits of exponent, 3 of mantissa, v as 5 bits
 * of exponent, 3 of mantissa (never 0 for v > 0), rounded stochastically from a
 * hash of (seed, step, index of the tensor, element), so that a run repeats bit
 * for bit.  Fresh states are all 0 with scale bytes 1.  The codes hold no infinity
 * and no NaN: an infinite or NaN gradient shows in its parameter, which is NaN from
 * then on; its moments become 0 and leave the rest of their block alone.
 * The array of descriptors is host memory and read at enqueue time.
 */
typedef struct ep_adamw_tensor {
    float *param;
    const void *grad;           /* fp32 or bf16, grad_dtype */
    void *exp_avg, *exp_avg_sq;
    uint8_t *exp_avg_scale, *exp_avg_sq_scale;
    void *copy;                 /* bf16 [numel] of the new parameters, or NULL */
    int64_t numel;              /* 0: skipped */
} ep_adamw_tensor_t;
typedef struct ep_adamw {
    double lr, beta1, beta2, eps, weight_decay, grad_scale;
    int64_t step;               /* from 1 */
    uint32_t seed;
    int32_t state_bits, grad_dtype;
} ep_adamw_t;
int ep_adamw_step(const ep_adamw_tensor_t *tensors, int32_t num_tensors, const ep_adamw_t *hp, ep_stream_t stream);

/* The fp32 values of 8-bit states: exp_avg[i], exp_avg_sq[i] device float
 * [numel] of tensor i (host arrays of pointers). */
int ep_adamw_values(const ep_adamw_tensor_t *tensors, int32_t num_tensors, float *const *exp_avg,
                    float *const *exp_avg_sq, ep_stream_t stream);

/* Human-readable name of a return code. */
const char *ep_status_string(int code);

#ifdef __cplusplus
}
#endif

#endif /* EP_BALANCE_H */
