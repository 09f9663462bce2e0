/*
 * zero_mi355x.h - C ABI of the per-rank partitioned mixed-precision optimizer
 * step (ZeRO / FSDP data parallelism) on AMD MI355X (gfx950).
 *
 * Cited page: "Zero Redundancy Optimizer (ZeRO) and Fully Sharded Data
 * Parallelism (FSDP): Mathematical Foundations of Memory Partitioning,
 * Communication Complexity, and Overlapped Execution" (llms.blog), written
 * [ZF] below with the section name.
 *
 * One rank's step, as [ZF] "Execution Flow for ZeRO-1" (steps 2-4) and
 * "ZeRO-Stage 2" lay it out, maps onto these calls:
 *   zero_partition_plan     flat padded buffer cut into N_d equal shards
 *   zero_grad_reduce_shard  the rank's averaged gradient slice (reduce-scatter,
 *                           seen from the receiving rank)
 *   zero_grad_sqnorm        squared-norm partial of a gradient shard
 *   zero_clip_scale         global-norm clip coefficient from all partials
 *   zero_shard_adamw_step   fp32 master/m/v update and bf16 parameter emit
 *   zero_multi_tensor_adamw_step  the same over a ragged list of tensors
 *                           (FSDP-2's per-parameter shards)
 *   zero_mt_table_*         the same list described once in device memory,
 *                           stepped in one launch
 *   zero_reduce_adamw_step  the reduce and the update in one pass, for a step
 *                           with no global norm between them
 *   zero_shard_adamw8_step, zero_multi_tensor_adamw8_step, zero_mt8_table_*,
 *   zero_reduce_adamw8_step  the AdamW forms with the moments held in 8 bits
 *   zero_state8_quantize, zero_state8_dequantize  those moments from and to fp32
 *   zero_orthogonalize      a stack of matrices, orthogonalised by Newton-Schulz
 *                           steps
 *   zero_muon_step, zero_muon_table_*  Muon's update of weight matrices: momentum,
 *                           orthogonalisation, weight update and bf16 emit
 *   zero_gather_params      bf16 shards back to per-tensor parameters
 *                           (all-gather output layout, then un-flatten)
 *   zero_flatten_params     per-tensor bf16 buffers into the padded flat buffer
 *                           (the step before the reduce; inverse of the gather)
 *   zero_*_table_create, zero_copy_table_run  the gather or flatten of fixed
 *                           buffers, described once in device memory
 *   zero_reduce_table_*     the reduce straight from per-tensor replicas of
 *                           fixed buffers (no flatten of each replica first)
 *   zero_offload_adamw_step ZeRO-Offload: the update on the host CPU, with the
 *                           gradient and parameter transfers overlapped
 *   zero_adamw_schedule_*, zero_*_scheduled  AdamW with the step number counted
 *                           on the device, so a step captured in a HIP graph
 *                           replays successive steps
 *
 * Conventions, for every function below:
 *   - bf16 values travel as raw uint16_t bit patterns; fp32 as float.
 *   - "device" pointers address GPU memory of the current HIP device; the
 *     caller allocates and owns them. The library never frees them and keeps
 *     no reference to them after the call returns.
 *   - "host" pointers are read during the call only.
 *   - Device work is enqueued on `stream` (0 = the legacy default stream) and
 *     runs asynchronously; the function returns once the work is enqueued.
 *     Results are visible to later work on the same stream.
 *   - Every function returns a zero_status; nothing aborts or throws across
 *     the ABI. On failure nothing has been enqueued, unless the status is
 *     ZERO_EHIP from a failed launch. zero_last_error() gives a readable
 *     detail for the last failure on the calling thread.
 *   - Element counts and offsets are int64_t; buffers beyond 2^32 elements
 *     are supported everywhere.
 *   - Any device pointer that is not 16-byte aligned is accepted; such calls
 *     run a slower scalar path with identical results.
 */
#ifndef ZERO_MI355X_H
#define ZERO_MI355X_H

#include <stddef.h>
#include <stdint.h>

#include <hip/hip_runtime_api.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum zero_status {
    ZERO_OK = 0,
    ZERO_EINVAL = 1,    /* an argument is invalid (null, negative, out of range) */
    ZERO_ERANGE = 2,    /* a size overflows int64 or exceeds a documented maximum */
    ZERO_ENOMEM = 3,    /* host memory allocation failed */
    ZERO_EHIP = 4,      /* a HIP runtime call or kernel launch failed */
    ZERO_ENOSPACE = 5   /* the caller's workspace is smaller than required */
} zero_status;

/* Largest number of gradient replicas one zero_grad_reduce_shard call reduces. */
#define ZERO_MAX_REPLICAS 64

/* Opaque partition plan: host memory owned by the library, immutable after
 * zero_partition_plan returns, safe to read from several threads. */
typedef struct zero_plan zero_plan;

/* The part of tensor `tensor` that lies in rank `rank`'s shard:
 * tensor elements [tensor_offset, tensor_offset + length) are shard elements
 * [shard_offset, shard_offset + length). */
typedef struct zero_segment {
    int32_t tensor;
    int32_t rank;
    int64_t tensor_offset;
    int64_t shard_offset;
    int64_t length;
} zero_segment;

/* ------------------------------------------------------------------ plan (host only)
 *
 * [ZF] "FSDP-1: FlatParameter and Module-Level Wrapping": a unit's tensors are
 * flattened into one contiguous 1-D buffer, padded to a length divisible by
 * the world size, and cut into N_d equal chunks; [ZF] "ZeRO-Stage 1" gives
 * each rank a Phi/N_d slice of the optimizer state.
 *
 * numels       host [n_tensors]: element count of each tensor, in flat order
 *              (each >= 0; zero-sized tensors are allowed and own no elements).
 * n_tensors    >= 0.
 * n_ranks      N_d >= 1.
 * align_elems  A >= 1: every shard length is a multiple of A, so the padded
 *              length P = ceil(Phi / (N_d*A)) * N_d*A and the shard length
 *              S = P / N_d. Tensor t starts at flat element sum(numels[<t]);
 *              elements [Phi, P) are padding. Rank r owns [r*S, (r+1)*S).
 * out          receives the new plan; free it with zero_plan_free.
 * Errors: ZERO_EINVAL for a null pointer, a negative count, n_ranks < 1 or
 * align_elems < 1; ZERO_ERANGE if P would overflow int64; ZERO_ENOMEM. */
zero_status zero_partition_plan(const int64_t* numels, int32_t n_tensors, int32_t n_ranks,
                                int32_t align_elems, zero_plan** out);
void zero_plan_free(zero_plan* plan);                       /* accepts NULL */

/* FSDP-2 per-parameter layout. [ZF] "FSDP-2: Per-Parameter Sharding via
 * DTensor (fully_shard)": each tensor is sharded on its own along its leading
 * dimension (a Shard(0) placement) instead of being flattened with the others,
 * and the shards of one unit travel in a coalesced communication buffer.
 *
 * Tensor t (numels[t] elements, dim0[t] >= 1 rows of inner_t = numels[t]/dim0[t]
 * elements; dim0[t] must divide numels[t]; a zero-sized tensor may give 0)
 * is cut into N_d chunks of c_t = ceil(dim0[t] / N_d) rows, as torch.chunk
 * cuts it: rank r holds rows [r*c_t, min((r+1)*c_t, dim0[t])), possibly none.
 * A rank's coalesced buffer holds its chunk of every tensor in order, each
 * padded to c_t*inner_t elements, the whole padded to a multiple of
 * align_elems: S = that length. The N_d coalesced buffers side by side form
 * the plan's flat buffer of P = N_d*S elements, so zero_grad_reduce_shard,
 * zero_shard_adamw_step, zero_gather_params and zero_flatten_params apply
 * unchanged; padding positions hold zeros. zero_plan_tensor_offset(t) gives
 * the start of tensor t's chunk inside every rank's buffer.
 * Errors as zero_partition_plan, plus ZERO_EINVAL when dim0 does not divide
 * a numel. */
zero_status zero_partition_plan_shard0(const int64_t* numels, const int64_t* dim0,
                                       int32_t n_tensors, int32_t n_ranks, int32_t align_elems,
                                       zero_plan** out);

/* 0 for a flat (FSDP-1 / ZeRO) plan, 1 for a Shard(0) plan, -1 for NULL. */
int32_t zero_plan_kind(const zero_plan* plan);

int64_t zero_plan_numel(const zero_plan* plan);             /* Phi, or -1 if plan is NULL */
int64_t zero_plan_padded_numel(const zero_plan* plan);      /* P,   or -1 */
int64_t zero_plan_shard_numel(const zero_plan* plan);       /* S,   or -1 */
int32_t zero_plan_num_tensors(const zero_plan* plan);       /* T,   or -1 */
int32_t zero_plan_num_ranks(const zero_plan* plan);         /* N_d, or -1 */
int64_t zero_plan_tensor_offset(const zero_plan* plan, int32_t tensor);  /* -1 if out of range;
                                                                           flat plans: the tensor's
                                                                           flat start */
int64_t zero_plan_tensor_numel(const zero_plan* plan, int32_t tensor);   /* -1 if out of range */
int32_t zero_plan_num_segments(const zero_plan* plan, int32_t rank);     /* -1 if out of range */

/* Copies rank's segments, in flat order, into host array out[capacity].
 * *count receives the number of segments; ZERO_ENOSPACE (with *count set) if
 * capacity is too small. */
zero_status zero_plan_segments(const zero_plan* plan, int32_t rank, zero_segment* out,
                               int32_t capacity, int32_t* count);

/* Static training-state bytes per GPU. [ZF] "Static Memory Allocation"
 * (16 bytes per parameter: 2 bf16 param, 2 bf16 grad, 12 fp32 master/m/v)
 * and the stage formulas of [ZF] "ZeRO-Stage 1" (4 Phi + 12 Phi/N_d),
 * "ZeRO-Stage 2" (2 Phi + 14 Phi/N_d) and "ZeRO-Stage 3 and Fully Sharded Data
 * Parallelism" (16 Phi/N_d). stage: 0 = DDP, 1, 2, 3. padded != 0 counts the
 * flat buffers at P and the shards at S (stage 0 stays 16 Phi). */
zero_status zero_plan_memory_bytes(const zero_plan* plan, int32_t stage, int32_t padded,
                                   double* bytes);

/* ------------------------------------------------------------------ gradient reduction
 *
 * [ZF] "Execution Flow for ZeRO-1", step 2: rank i receives the gradient of
 * its own partition averaged over the data-parallel ranks; [ZF] "ZeRO-Stage 2":
 * gradients are reduced into their owners' slices bucket by bucket as backward
 * produces them. On one GPU the R replicas sit in one HBM; this call is the
 * receiving rank's arithmetic of that reduce-scatter.
 *
 * replicas     host [n_replicas] of device pointers; replicas[k] points at
 *              replica k's bf16 gradient for global flat elements
 *              [begin, begin + count) (a whole flat buffer, or one bucket).
 * n_replicas   R, 1 <= R <= ZERO_MAX_REPLICAS.
 * begin,count  the global flat window the replica buffers cover (count >= 0,
 *              begin >= 0, begin + count <= P).
 * shard_grad   device [S]: element i is global element rank*S + i. Only the
 *              window's intersection with rank's shard is written; that slice
 *              must not overlap the replicas' slices the call reads, or the
 *              workspace:
 *              out = bf16_rne( (sum over k = 0..R-1, in order, of fp32(rep_k)) / R ),
 *              the sum and the division in IEEE fp32.
 * sqnorm_out   device, nullable: receives the fp64 sum of squares of the bf16
 *              values this call wrote (0 if it wrote nothing). Deterministic for a
 *              given window and workspace size.
 * workspace    device, required when sqnorm_out is non-null; at least
 *              zero_sqnorm_workspace_bytes() bytes, 8-byte aligned, owned by
 *              the caller. It holds the per-workgroup partials between the
 *              call's kernels; it needs no initialisation and its contents
 *              on return are unspecified. Calls that may run
 *              at the same time (on different streams) need separate
 *              workspaces; calls on one stream may share one.
 *              With zero_reduce_workspace_bytes(n) bytes or more, where n is
 *              the number of elements written (at most count), a window of
 *              2^24 elements or more, of at most 8 replicas, whose slices are
 *              4-byte aligned takes the one-pass kernel: one workgroup per 512 elements, a partial per
 *              workgroup and a two-level final sum. It is faster on windows too
 *              large for the caches. The bf16 output is the same either way.
 *              The fp64 sum is grouped differently, so its last bits may
 *              differ. Without a norm the one-pass kernel needs no workspace.
 * Errors: ZERO_EINVAL (null plan/replicas/shard_grad, a null replica pointer,
 * R out of range, rank out of range, bad window, workspace not 8-byte
 * aligned, the written slice overlapping a replica's slice or the workspace,
 * named in zero_last_error()); ZERO_ENOSPACE; ZERO_EHIP. */
zero_status zero_grad_reduce_shard(const zero_plan* plan, int32_t rank,
                                   const uint16_t* const* replicas, int32_t n_replicas,
                                   int64_t begin, int64_t count, uint16_t* shard_grad,
                                   double* sqnorm_out, void* workspace, size_t workspace_bytes,
                                   hipStream_t stream);

/* For callers that cannot allocate device memory (code under HIP graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): zero_grad_reduce_shard
 * with the same arguments except the workspace, which is a device array the
 * library owns, ZERO_NOALLOC_SCRATCH_BYTES bytes on each device, kept from the
 * library's load until the process ends. The call allocates nothing: no
 * hipMalloc, no hipFree, no allocating library routine. The first call on a
 * device looks up that device's copy of the array (hipGetSymbolAddress) with
 * the device current; a caller that captures graphs makes that first call
 * before capturing. The bf16 output is zero_grad_reduce_shard's. The norm
 * equals zero_grad_reduce_shard's with a workspace of
 * ZERO_NOALLOC_SCRATCH_BYTES bytes: windows of 2^24 elements or more whose
 * one-pass partials fit the array (up to about 2.7e8 elements) take the
 * one-pass kernel, larger windows the grid-stride kernel and its fixed 2,048
 * partials, so no window size is refused. Every call on one device shares
 * that device's array: calls that may overlap on one device (other streams,
 * other host threads) race on it and must be ordered by the caller; calls in
 * order on one stream are safe. Errors: as zero_grad_reduce_shard (no
 * workspace errors); ZERO_ERANGE for a device index above 63; ZERO_EHIP. */
#define ZERO_NOALLOC_SCRATCH_BYTES (4u << 20)
zero_status zero_grad_reduce_shard_noalloc(const zero_plan* plan, int32_t rank,
                                           const uint16_t* const* replicas, int32_t n_replicas,
                                           int64_t begin, int64_t count, uint16_t* shard_grad,
                                           double* sqnorm_out, hipStream_t stream);

/* ------------------------------------------------------------------ squared norm
 *
 * Sum of squares of n bf16 values (device [n]), accumulated in fp64 (each
 * square is exact), written to device sqnorm_out[0]. Two fixed-order
 * reduction levels, no floating-point atomics: the result is reproducible on
 * a given device. The norm clip is not on the cited pages; the global norm it
 * needs is the sum of these partials over every rank. workspace as for
 * zero_grad_reduce_shard; with zero_reduce_workspace_bytes(n) bytes or more, a
 * 16-byte-aligned input of 2^24 elements or more takes a one-pass kernel (a
 * partial per 16,384 elements, two-level final sum; the fp64 grouping differs,
 * so the last bits may too).
 * Errors: ZERO_EINVAL (null pointers with n > 0, n < 0, workspace not 8-byte
 * aligned); ZERO_ENOSPACE; ZERO_EHIP. */
zero_status zero_grad_sqnorm(const uint16_t* grad, int64_t n, double* sqnorm_out,
                             void* workspace, size_t workspace_bytes, hipStream_t stream);

/* Workspace bytes that zero_grad_sqnorm and zero_grad_reduce_shard need: a
 * fixed bound, independent of n and of the device. */
size_t zero_sqnorm_workspace_bytes(void);

/* Workspace bytes with which zero_grad_reduce_shard (with the norm) and
 * zero_grad_sqnorm can take their one-pass kernels on up to count elements:
 * about 8 bytes per 512 elements, never less than zero_sqnorm_workspace_bytes().
 * Host only. */
size_t zero_reduce_workspace_bytes(int64_t count);

/* ------------------------------------------------------------------ clip coefficient
 *
 * partials     device [n_partials] fp64 squared-norm partials (one per rank, or
 *              per bucket), summed in index order in fp64.
 * max_norm     clip threshold; <= 0 disables clipping (coefficient 1).
 * scale_out    device float: min(1, max_norm / (sqrt(total) + 1e-6)) rounded
 *              once to fp32; NaN when the total is not finite, which makes
 *              zero_shard_adamw_step skip its update.
 * Errors: ZERO_EINVAL (null pointers, n_partials < 1 or > 65536); ZERO_EHIP. */
zero_status zero_clip_scale(const double* partials, int32_t n_partials, double max_norm,
                            float* scale_out, hipStream_t stream);

/* ------------------------------------------------------------------ AdamW shard update
 *
 * [ZF] "Static Memory Allocation": fp32 master weights, fp32 first moment m_t
 * and fp32 second moment v_t, 16-bit parameters; [ZF] "Execution Flow for
 * ZeRO-1", steps 3-4: the rank updates its own slice and emits 16-bit
 * parameters for the all-gather; [ZF] "ZeRO-Offload Mechanics": O(1) work per
 * parameter, so the update is bound by memory traffic (28 bytes per element).
 *
 * Per element, each operation one IEEE fp32 operation (no fused multiply-add),
 * in this order, with the scalars computed in fp64 on the host and rounded
 * once to fp32 (t = step):
 *   g = fp32(grad) * clip
 *   m = beta1*m + (1-beta1)*g
 *   v = beta2*v + (1-beta2)*(g*g)
 *   p = p * (1 - lr*weight_decay)
 *   p = p - (lr/(1-beta1^t)) * (m / (sqrt(v)/sqrt(1-beta2^t) + eps))
 *   param_out = bf16_rne(p)
 * master, exp_avg, exp_avg_sq  device [n] fp32, updated in place.
 * grad         device [n] bf16, read only.
 * param_out    device [n] bf16, written.
 *              The four written arrays must not overlap one another or grad
 *              (each element is read and written by one lane; arrays shifted
 *              against each other would race).
 * step         t >= 1 (1-based bias-correction step).
 * clip_scale   device float, nullable (NULL means 1). A non-finite value skips
 *              the update: nothing is read or written.
 * Errors: ZERO_EINVAL (null pointers with n > 0, n < 0, step < 1, beta1 or
 * beta2 outside [0, 1), eps <= 0, lr < 0, non-finite scalars, overlapping
 * arrays, named in zero_last_error()); ZERO_EHIP. */
zero_status zero_shard_adamw_step(float* master, float* exp_avg, float* exp_avg_sq,
                                  const uint16_t* grad, uint16_t* param_out, int64_t n,
                                  int64_t step, double lr, double beta1, double beta2, double eps,
                                  double weight_decay, const float* clip_scale,
                                  hipStream_t stream);

/* Step counted on the device, for a step captured in a HIP graph. [ZF] "Execution
 * Flow for ZeRO-1", step 3, repeated every iteration: zero_shard_adamw_step
 * takes t from the host and computes the step's scalars there, so a captured
 * launch would replay one step forever. A schedule holds, in device memory,
 * the number of updates applied and the scalars of the next step, and a table
 * of the scalars of steps 1..L (each as zero_shard_adamw_step computes them
 * on the host, so the results are the same bits). L is the step from which
 * both bias corrections are exactly 1 in fp64 (beta^t < 2^-56), or the length
 * of the learning-rate list if longer: every later step has step L's scalars.
 * For beta2 = 0.999, L = 38,797 (1.2 MB).
 *
 * zero_adamw_schedule_create: lr is a host array of n_lr >= 1 learning rates,
 * step t using lr[min(t, n_lr) - 1] (one value: a constant rate); betas, eps
 * and weight_decay as zero_shard_adamw_step; the first update applied is step
 * first_step >= 1 (a resumed run passes its next step). Allocates on the
 * current device. Errors: ZERO_EINVAL (bad hyperparameters, NULL lr or out,
 * n_lr < 1, first_step < 1); ZERO_ERANGE when L would pass 2^24 (a beta within
 * about 2.3e-6 of 1, or a longer list); ZERO_ENOMEM; ZERO_EHIP.
 * zero_shard_adamw_step_scheduled: zero_shard_adamw_step's update and
 * arguments, with the step's scalars read on the device from the schedule;
 * it does not move the schedule on, so a step may update any number of
 * arrays with it (buckets, tensors, ranks).
 * zero_adamw_schedule_advance: once per step, after the step's updates on the
 * same stream: counts the step as applied and loads the next step's scalars.
 * A non-finite clip coefficient (the updates skipped) leaves the schedule as it
 * is, so a skipped step is not counted. One lane; allocates nothing.
 * zero_adamw_schedule_applied: the number of updates applied, read back
 * synchronously (hipMemcpy; the caller first waits for the streams that
 * advanced the schedule). zero_adamw_schedule_length: L (-1 for NULL).
 * Calls that move one schedule on must be ordered by the caller (one stream).
 * Errors of the step and advance: ZERO_EINVAL (NULL schedule, the schedule on
 * another device, as zero_shard_adamw_step otherwise); ZERO_EHIP.
 *
 * zero_adamw_step_scalars: host only; the eight fp32 scalars every AdamW entry
 * point computes for step t, in order beta1, 1-beta1, beta2, 1-beta2, eps,
 * lr/(1-beta1^t), sqrt(1-beta2^t), 1-lr*weight_decay. Errors: as
 * zero_shard_adamw_step's hyperparameter checks; ZERO_EINVAL for a NULL out. */
typedef struct zero_adamw_schedule zero_adamw_schedule;
zero_status zero_adamw_schedule_create(const double* lr, int64_t n_lr, double beta1, double beta2,
                                       double eps, double weight_decay, int64_t first_step,
                                       zero_adamw_schedule** out);
void zero_adamw_schedule_free(zero_adamw_schedule* schedule);
int64_t zero_adamw_schedule_length(const zero_adamw_schedule* schedule);
zero_status zero_adamw_schedule_applied(const zero_adamw_schedule* schedule, int64_t* applied);
zero_status zero_adamw_schedule_advance(zero_adamw_schedule* schedule, const float* clip_scale,
                                        hipStream_t stream);
zero_status zero_shard_adamw_step_scheduled(float* master, float* exp_avg, float* exp_avg_sq,
                                            const uint16_t* grad, uint16_t* param_out, int64_t n,
                                            const zero_adamw_schedule* schedule,
                                            const float* clip_scale, hipStream_t stream);
zero_status zero_adamw_step_scalars(int64_t step, double lr, double beta1, double beta2, double eps,
                                    double weight_decay, float* out);
/* The scheduled forms of the multi-tensor table step and of the one-pass
 * reduce and update (declared with their plain forms below): the same
 * arguments and results, with the step's scalars read on the device from the
 * schedule, which they do not move on. Errors: as their plain forms (without
 * the hyperparameter checks); ZERO_EINVAL for a NULL schedule or one that
 * lives on another device than the current one (or, for the table, than the
 * table). */

/* Reduce and update in one pass. [ZF] "Execution Flow for ZeRO-1", steps 2-3:
 * the rank receives the averaged gradient of its slice and updates its master
 * weights and optimizer state from it. When the step needs no global norm
 * between the two (no clipping, or a clip coefficient the caller already
 * holds), they run as one pass over the rank's window: for every element of
 * [begin, begin + count) within the rank's shard, the averaged gradient is
 * zero_grad_reduce_shard's (fp32 sum in replica order, one fp32 division by
 * R, bf16 round-to-nearest-even) and the update zero_shard_adamw_step's on
 * it, bit for bit the two calls in sequence, without the gradient's round trip
 * through HBM (2R + 26 bytes per element instead of 2R + 30).
 * plan, rank, replicas, n_replicas, begin, count: as zero_grad_reduce_shard.
 * master, exp_avg, exp_avg_sq  device [S] fp32, the rank's shard state, in place.
 * param_out    device [S] bf16, the rank's parameter shard. Element i of
 *              these arrays is global element rank*S + i; only the window's
 *              part of the shard is read and written.
 * shard_grad   device [S] bf16, nullable: when given, also receives the
 *              averaged gradient, as zero_grad_reduce_shard writes it.
 *              Within the window, the written arrays (the three fp32 arrays,
 *              param_out, shard_grad) must not overlap one another or the
 *              replicas' slices the call reads.
 * step, lr, beta1, beta2, eps, weight_decay, clip_scale: as
 *              zero_shard_adamw_step; a non-finite coefficient skips the
 *              update (shard_grad, when given, is still written).
 * Errors: ZERO_EINVAL (null plan or replicas, a null replica or state array
 * for a non-empty window, R or rank out of range, bad window, bad
 * hyperparameters, overlapping arrays, named in zero_last_error());
 * ZERO_EHIP. */
zero_status zero_reduce_adamw_step(const zero_plan* plan, int32_t rank,
                                   const uint16_t* const* replicas, int32_t n_replicas,
                                   int64_t begin, int64_t count, float* master, float* exp_avg,
                                   float* exp_avg_sq, uint16_t* param_out, uint16_t* shard_grad,
                                   int64_t step, double lr, double beta1, double beta2, double eps,
                                   double weight_decay, const float* clip_scale,
                                   hipStream_t stream);
zero_status zero_reduce_adamw_step_scheduled(const zero_plan* plan, int32_t rank,
                                             const uint16_t* const* replicas, int32_t n_replicas,
                                             int64_t begin, int64_t count, float* master,
                                             float* exp_avg, float* exp_avg_sq, uint16_t* param_out,
                                             uint16_t* shard_grad, const zero_adamw_schedule* schedule,
                                             const float* clip_scale, hipStream_t stream);

/* Multi-tensor form. [ZF] "FSDP-2: Per-Parameter Sharding via DTensor
 * (fully_shard)": each parameter keeps its own local shard, so the rank's
 * optimizer step runs over a ragged list of per-parameter tensors rather than
 * one flat buffer. Tensor t has its own arrays masters[t], exp_avgs[t],
 * exp_avg_sqs[t] (device [numels[t]] fp32, in place), grads[t] (device bf16,
 * read only) and params_out[t] (device bf16, written); tensor t's four
 * written arrays must not overlap one another or grads[t], and different
 * tensors' written arrays must not overlap (that is the caller's to keep: the
 * call checks each tensor's arrays against each other only); the pointer arrays and numels are host arrays of
 * n_tensors entries. Every element gets zero_shard_adamw_step's arithmetic
 * (identical bits), with one step, one set of hyperparameters and one clip
 * coefficient for the whole list. Zero-sized tensors are skipped (their
 * pointers may be NULL). Any pointer alignment. The tensors are batched
 * largest first, 78 per launch (the order changes no result).
 * Errors: as zero_shard_adamw_step, per tensor (ZERO_EINVAL names it);
 * ZERO_ERANGE for a tensor of 2^39 elements or more; ZERO_ENOMEM; ZERO_EHIP. */
zero_status zero_multi_tensor_adamw_step(float* const* masters, float* const* exp_avgs,
                                         float* const* exp_avg_sqs, const uint16_t* const* grads,
                                         uint16_t* const* params_out, const int64_t* numels,
                                         int32_t n_tensors, int64_t step, double lr, double beta1,
                                         double beta2, double eps, double weight_decay,
                                         const float* clip_scale, hipStream_t stream);

/* The multi-tensor form for a fixed list, with its table in device memory.
 * [ZF] "FSDP-2: Per-Parameter Sharding via DTensor (fully_shard)": the same
 * per-parameter list is stepped every iteration, so its description can be
 * built once. zero_mt_table_create checks the list exactly as
 * zero_multi_tensor_adamw_step does and copies, to device memory that the
 * table owns, one 64-byte descriptor per non-empty tensor (its five device
 * pointers and its size) and one 4-byte tensor index per workgroup of 512
 * elements (about 0.8 bytes per 100 elements). zero_mt_table_adamw_step then
 * updates every tensor of the list in one launch (a list of 2^24 workgroups or
 * more, above 8.6e9 elements, in several), with zero_shard_adamw_step's
 * arithmetic: identical bits to both other AdamW entry points.
 * Create: the arguments as zero_multi_tensor_adamw_step's list; out receives
 * the table. It calls hipMalloc and a synchronous hipMemcpy on the current
 * device, once. The table keeps the device pointers (not the data): the
 * caller keeps those buffers alive and in place for the table's lifetime.
 * Errors: as zero_multi_tensor_adamw_step's list checks; ZERO_EINVAL for a
 * NULL out; ZERO_ERANGE for 2^31 workgroups or more; ZERO_ENOMEM; ZERO_EHIP
 * (allocation or copy failed).
 * Step: step, hyperparameters and clip_scale as zero_shard_adamw_step. It must
 * run with the table's device current (ZERO_EINVAL otherwise). An empty list
 * enqueues nothing.
 * Free: releases the device memory (hipFree, which waits for the device);
 * no step using the table may still be running. Accepts NULL.
 * Blocks: the workgroups of one step, or -1 for NULL. */
typedef struct zero_mt_table zero_mt_table;
zero_status zero_mt_table_create(float* const* masters, float* const* exp_avgs,
                                 float* const* exp_avg_sqs, const uint16_t* const* grads,
                                 uint16_t* const* params_out, const int64_t* numels,
                                 int32_t n_tensors, zero_mt_table** out);
void zero_mt_table_free(zero_mt_table* table);
int64_t zero_mt_table_blocks(const zero_mt_table* table);
zero_status zero_mt_table_adamw_step(const zero_mt_table* table, int64_t step, double lr,
                                     double beta1, double beta2, double eps, double weight_decay,
                                     const float* clip_scale, hipStream_t stream);
zero_status zero_mt_table_adamw_step_scheduled(const zero_mt_table* table,
                                               const zero_adamw_schedule* schedule,
                                               const float* clip_scale, hipStream_t stream);

/* ------------------------------------------------------------------ AdamW, moments in 8 bits
 *
 * [ZF] "Static Memory Allocation": the two fp32 moments are 8 of a parameter's
 * 16 bytes. These entry points hold them in 8 bits: an array of n moments is
 * cut into blocks of ZERO_STATE8_BLOCK consecutive elements (the last one may
 * be shorter), with one code byte per element and one scale byte per block
 * (ceil(n / ZERO_STATE8_BLOCK) of them), 2.02 bytes for both moments instead
 * of 8. The master weights stay fp32.
 *
 * Format. A code is an OCP 8-bit float e4m3 (bias 7, largest 448, no
 * infinity), a scale byte an e8m0 power of two: value = e4m3(code) *
 * 2^(byte - 127): 3 bits of mantissa down to 2^-13 of the block's largest, the
 * least code at 2^-17 to 2^-16 of it. Byte 255 stands for a block that held an
 * infinity or NaN: it reads as NaN throughout (its codes are written as 0).
 * All-zero bytes are zeros, so cleared arrays are the moments of a new run.
 * Encoding a block. E = the biased exponent field of the largest magnitude;
 * byte = 255 if E = 255, else max(E - 7, 0) (that magnitude then lies in
 * [2^7, 2^8) in code units and never saturates). In the steps, y = |x| *
 * 2^(7 - byte) as fp32, bits below its least subnormal dropped (every other y
 * is exact), and code = (bits(y) + r) >> 20 with 20 bits r of a random word,
 * and the sign in bit 7: stochastic rounding, so that a moment that moves by
 * less than a code's step still moves in the mean. zero_state8_quantize rounds
 * to the nearest code, ties to even. In the second moment a positive x has a
 * code of at least 1 (never rounded to zero): one below the block's least code
 * (2^-17 to 2^-16 of its largest) reads as that code, and its element takes
 * smaller steps than with fp32 moments; the mean is kept from that code on.
 * Random words. Element e of step t of a run with `seed` has a 32-bit word
 * that depends on (seed, t, e) only; elements are counted in windows of 2^28,
 * each with a key of its own. All arithmetic unsigned:
 *   w = e / 2^28, q = e % 2^28 / 8, j = e % 8;
 *   z = seed + t * 0x6A09E667F3BCC909 + w * 0xA54FF53A5F1D36F1;
 *   z = (z ^ z >> 32) * 0xBB67AE8584CAA73B;
 *   z = (z ^ z >> 29) * 0x3C6EF372FE94F82B;  z ^= z >> 32;          (64 bits)
 *   a = (q ^ low(z)) * 0xA54FF53B;           a ^= a >> 16;
 *   a = (a + high(z)) * 0x510E527F;          a ^= a >> 15;
 *   b = a * 0x9B05688D;  b = (b ^ b >> 16) | 1;  word = a + j * b   (32 bits)
 * The first moment's r is word >> 12, the second's word & 0xFFFFF.
 * first_element (a multiple of ZERO_STATE8_BLOCK, >= 0) is the number e of the
 * arrays' first element: a rank passes its shard's place in the flat buffer,
 * and a shard stepped window by window rounds as the whole shard does.
 *
 * The update per element is zero_shard_adamw_step's, in its order, on the
 * decoded m and v: the new fp32 m and v update p, and then are encoded.
 * Accesses: any pointer alignment; with master 16-byte, codes 4-byte, grad and
 * param_out 8-byte aligned (the usual case) a call is fastest; the results are
 * the same at any.
 *
 * zero_shard_adamw8_step
 * master       device [n] fp32, updated in place.
 * exp_avg, exp_avg_sq  device [n] codes, updated in place (exp_avg_sq's values
 *              are not negative).
 * exp_avg_scale, exp_avg_sq_scale  device [ceil(n / 128)] bytes, in place.
 * grad, param_out, n, step, lr, beta1, beta2, eps, weight_decay, clip_scale:
 *              as zero_shard_adamw_step (a non-finite coefficient skips the
 *              update). The six written arrays must not overlap one another
 *              or grad. A gradient that makes a moment infinite or NaN makes
 *              that moment's block NaN from the next step on.
 * Errors: as zero_shard_adamw_step; ZERO_EINVAL for a first_element that is
 * negative or no multiple of ZERO_STATE8_BLOCK; ZERO_ERANGE when first_element
 * + n overflows or n is past 2^48.
 * zero_shard_adamw8_step_scheduled: the step's scalars, and the step number of
 * the random words, read on the device from the schedule (which it does not
 * move on). Errors: as zero_shard_adamw_step_scheduled, and the above. */
#define ZERO_STATE8_BLOCK 128
zero_status zero_shard_adamw8_step(float* master, uint8_t* exp_avg, uint8_t* exp_avg_scale,
                                   uint8_t* exp_avg_sq, uint8_t* exp_avg_sq_scale,
                                   const uint16_t* grad, uint16_t* param_out, int64_t n,
                                   int64_t first_element, int64_t step, double lr, double beta1,
                                   double beta2, double eps, double weight_decay, uint64_t seed,
                                   const float* clip_scale, hipStream_t stream);
zero_status zero_shard_adamw8_step_scheduled(float* master, uint8_t* exp_avg, uint8_t* exp_avg_scale,
                                             uint8_t* exp_avg_sq, uint8_t* exp_avg_sq_scale,
                                             const uint16_t* grad, uint16_t* param_out, int64_t n,
                                             int64_t first_element,
                                             const zero_adamw_schedule* schedule, uint64_t seed,
                                             const float* clip_scale, hipStream_t stream);

/* Many tensors (zero_multi_tensor_adamw_step's and zero_mt_table_*'s
 * counterparts): each tensor has its own arrays, and its own blocks, counted
 * from its first element. Tensor t's elements are numbered from first_element
 * plus the lengths of the tensors before it, each rounded up to a multiple of
 * ZERO_STATE8_BLOCK; the results are zero_shard_adamw8_step's on each tensor.
 * The list form takes the arrays with every call, 48 tensors a launch (the
 * largest first, which changes no result). Errors: as
 * zero_multi_tensor_adamw_step (ZERO_ERANGE for a tensor of 1.7e10 elements or
 * more, which one launch does not hold), and zero_shard_adamw8_step's on
 * first_element.
 * The table form is for fixed buffers. Create, step, free, blocks and the
 * caller's duties as zero_mt_table_* (create: hipMalloc and a synchronous
 * hipMemcpy on the current device, once; 128 bytes per tensor and 4 per
 * workgroup of 512 elements; a longer list than one launch holds takes
 * several). Errors: as zero_mt_table_*, and zero_shard_adamw8_step's on first_element. */
zero_status zero_multi_tensor_adamw8_step(float* const* masters, uint8_t* const* exp_avgs,
                                          uint8_t* const* exp_avg_scales,
                                          uint8_t* const* exp_avg_sqs,
                                          uint8_t* const* exp_avg_sq_scales,
                                          const uint16_t* const* grads, uint16_t* const* params_out,
                                          const int64_t* numels, int32_t n_tensors,
                                          int64_t first_element, int64_t step, double lr,
                                          double beta1, double beta2, double eps,
                                          double weight_decay, uint64_t seed,
                                          const float* clip_scale, hipStream_t stream);
typedef struct zero_mt8_table zero_mt8_table;
zero_status zero_mt8_table_create(float* const* masters, uint8_t* const* exp_avgs,
                                  uint8_t* const* exp_avg_scales, uint8_t* const* exp_avg_sqs,
                                  uint8_t* const* exp_avg_sq_scales, const uint16_t* const* grads,
                                  uint16_t* const* params_out, const int64_t* numels,
                                  int32_t n_tensors, int64_t first_element, zero_mt8_table** out);
void zero_mt8_table_free(zero_mt8_table* table);
int64_t zero_mt8_table_blocks(const zero_mt8_table* table);
zero_status zero_mt8_table_adamw8_step(const zero_mt8_table* table, int64_t step, double lr,
                                       double beta1, double beta2, double eps, double weight_decay,
                                       uint64_t seed, const float* clip_scale, hipStream_t stream);
zero_status zero_mt8_table_adamw8_step_scheduled(const zero_mt8_table* table,
                                                 const zero_adamw_schedule* schedule, uint64_t seed,
                                                 const float* clip_scale, hipStream_t stream);

/* Reduce and update in one pass, moments in 8 bits (zero_reduce_adamw_step's
 * counterpart): the averaged gradient is zero_grad_reduce_shard's, the update
 * zero_shard_adamw8_step's on it, bit for bit the two calls in sequence;
 * 2R + 14 bytes per element. The state arrays are the rank's shard ([S] and
 * ceil(S / 128) scales), first_element the number of the shard's first
 * element. A block is encoded whole, so the window's part of the shard must
 * start at a multiple of ZERO_STATE8_BLOCK elements of the shard and end at
 * one or at the shard's end (ZERO_EINVAL otherwise).
 * Other arguments and errors: as zero_reduce_adamw_step and
 * zero_shard_adamw8_step. */
zero_status zero_reduce_adamw8_step(const zero_plan* plan, int32_t rank,
                                    const uint16_t* const* replicas, int32_t n_replicas,
                                    int64_t begin, int64_t count, float* master, uint8_t* exp_avg,
                                    uint8_t* exp_avg_scale, uint8_t* exp_avg_sq,
                                    uint8_t* exp_avg_sq_scale, uint16_t* param_out,
                                    uint16_t* shard_grad, int64_t first_element, int64_t step,
                                    double lr, double beta1, double beta2, double eps,
                                    double weight_decay, uint64_t seed, const float* clip_scale,
                                    hipStream_t stream);
zero_status zero_reduce_adamw8_step_scheduled(const zero_plan* plan, int32_t rank,
                                              const uint16_t* const* replicas, int32_t n_replicas,
                                              int64_t begin, int64_t count, float* master,
                                              uint8_t* exp_avg, uint8_t* exp_avg_scale,
                                              uint8_t* exp_avg_sq, uint8_t* exp_avg_sq_scale,
                                              uint16_t* param_out, uint16_t* shard_grad,
                                              int64_t first_element,
                                              const zero_adamw_schedule* schedule, uint64_t seed,
                                              const float* clip_scale, hipStream_t stream);

/* Moments between fp32 and 8 bits (a checkpoint read or written, a run moved
 * from or to 32-bit moments).
 * zero_state8_quantize: x device [n] fp32 into codes [n] and scales
 * [ceil(n / 128)], rounded to nearest, ties to even; second_moment != 0 keeps
 * a positive x at code 1 or more. The written arrays must not overlap one
 * another or x. zero_state8_dequantize: the values, out device [n] fp32 (exact
 * but for fp32 subnormals, which round to nearest); out must not overlap the
 * codes or the scales. Quantizing dequantized values need not give the same
 * bytes: a block whose largest is a power of two that stochastic rounding
 * reached gets the next scale, and codes below its normal ones lose a bit.
 * Errors: ZERO_EINVAL (n < 0; with n > 0, null pointers or overlapping arrays,
 * named in zero_last_error()); ZERO_ERANGE for n past 2^48; ZERO_EHIP. */
zero_status zero_state8_quantize(const float* x, int64_t n, int32_t second_moment, uint8_t* codes,
                                 uint8_t* scales, hipStream_t stream);
zero_status zero_state8_dequantize(const uint8_t* codes, const uint8_t* scales, int64_t n,
                                   float* out, hipStream_t stream);

/* ------------------------------------------------------------------ Muon: orthogonalised updates
 *
 * [ZF] "Execution Flow for ZeRO-1", steps 3-4 (the rank updates its fp32 master
 * weights and emits 16-bit parameters), with Muon's update in place of AdamW's:
 * a weight matrix moves along its orthogonalised momentum. The state is the fp32
 * master and one fp32 momentum. The other parameters of a model (vectors,
 * embeddings) keep AdamW.
 *
 * Orthogonalising. G is rows x cols, row-major; a tall one is taken transposed,
 * so that X has no more rows than columns:
 *   X = G / (|G| + eps), |G| the Frobenius norm (its squares summed in fp64; where
 *       values are held in two fp16 parts the trace of X X^T's fp32 sums, 5e-7
 *       off over 4 million values)
 *   for each step (a, b, c):  A = X X^T,  X <- a X + (b A + c A^2) X
 * Each step is an odd polynomial of the singular values; (3.4445, -4.7750,
 * 2.0315) five times takes those from 1/500 of the norm up to between 0.7 and
 * 1.2. A zero matrix gives zeros (with eps = 0 too); one that holds an infinity
 * or NaN gives NaN throughout, and no other matrix of the call is touched by it.
 * Precision: products of fp16 values (scaled by powers of two) summed in fp32,
 * with what rounding each X left carried along; after five usual steps about
 * 1.5e-3 of the result's Frobenius norm off the exact ones, less than rounding it
 * to bf16 (1.7e-3), and up to 7e-3 where few directions hold nearly all of the
 * norm or half of the singular values lie far below the rest. Singular values
 * below about 1e-5 of the norm, and directions that G does not have, come out as
 * noise of up to 0.02; elements below 3e-10 (a norm far below eps) as zeros or
 * noise of that size. Every step multiplies what lies in such directions by its a:
 * after nine usual ones the noise is up to 0.2, and a matrix whose singular
 * values lie above 1e-3 of the largest up to 4e-2 off. Where no matrix of a call
 * has a short side above 128 and the product of the squares of the steps' largest
 * factors (a, of the usual ones) but the last's is below 65,536, all values are held
 * in two fp16 parts, and five usual steps are about 3e-5 off.
 * Two steps are taken as one on the smaller side where that saves time and the
 * first's |a| is at most 4; this and the products' tiles follow the sizes and
 * number of a call's matrices.
 * The same call gives the same bits: no atomics.
 * Steps that contract to the very end of the interval that the one before leaves
 * and grow steeply past it (the published Polar Express coefficients, undivided)
 * would let fp16's roundings carry a singular value past that end. Where values are
 * held in one fp16 part, such a set is taken with (a, b, c) / (s, s^3, s^5) in all
 * steps but the last, s = 1 + 3 / 2048; divided by 1.003 or more those coefficients
 * are taken as they are.
 *
 * coefficients host [3 * n_steps] doubles, (a, b, c) of each step.
 * n_steps      1..32.
 * eps          >= 0.
 * workspace    device, 256-byte aligned, zero_muon_workspace_bytes(count, rows,
 *              cols) bytes or more (0 where the arguments are refused or there is nothing to do):
 *              about 8 bytes an element and 6 per element of the smaller side's
 *              square, both sides padded (to 64 or more). It needs no initialisation, its
 *              contents on return are unspecified, and calls that may run at the
 *              same time need separate ones.
 * Sides: the shorter up to 65,536, the longer up to 2^22.
 *
 * zero_orthogonalize: `count` matrices one after the other.
 * x            device [count * rows * cols], bf16 or fp32 by x_type.
 * out          device [count * rows * cols] bf16, rounded to nearest even once.
 *              Must not overlap x or the workspace.
 * Errors: ZERO_EINVAL (an unknown x_type, a negative count or side, bad steps
 * or eps, coefficients that let singular values, with what roundings add to
 * them, grow past 2^20 or a step multiply by more than 2^60; with something to do,
 * null pointers, a workspace not 256-byte aligned, overlapping arrays, named in
 * zero_last_error()); ZERO_ERANGE (a side past its limit, or more
 * workgroups than one launch holds); ZERO_ENOSPACE; ZERO_ENOMEM; ZERO_EHIP.
 *
 * zero_muon_step: the update of `count` matrices one after the other. Per
 * element, each operation one IEEE fp32 operation, in this order, the scalars
 * computed in fp64 and rounded once:
 *   g = fp32(grad) * clip
 *   momentum = mu * momentum + g
 *   u = nesterov ? g + mu * momentum : momentum
 *   o = the element of u's orthogonalised matrix, in bf16 as zero_orthogonalize
 *       returns it
 *   p = p * (1 - lr * weight_decay)
 *   p = p - (lr * scale) * o
 *   param_out = bf16_rne(p)
 * master, momentum  device fp32, updated in place.
 * grad         device bf16, read only.
 * param_out    device bf16, written. The written arrays and the workspace must
 *              not overlap one another or grad.
 * mu           in [0, 1).
 * scale        factor of the rate, usually a function of the sides: 0.2 *
 *              sqrt(max(rows, cols)) gives the update an AdamW step's root mean square.
 * clip_scale   device float, nullable (NULL means 1). A non-finite value skips
 *              the update: nothing of the caller's is written.
 * Errors: as zero_orthogonalize; ZERO_EINVAL (lr < 0, mu outside [0, 1),
 * non-finite scalars). */
#define ZERO_MATRIX_BF16 0
#define ZERO_MATRIX_F32 1
size_t zero_muon_workspace_bytes(int64_t count, int64_t rows, int64_t cols);
zero_status zero_orthogonalize(const void* x, int32_t x_type, uint16_t* out, int64_t count, int64_t rows,
                               int64_t cols, const double* coefficients, int32_t n_steps, double eps,
                               void* workspace, size_t workspace_bytes, hipStream_t stream);
zero_status zero_muon_step(float* master, float* momentum, const uint16_t* grad, uint16_t* param_out,
                           int64_t count, int64_t rows, int64_t cols, double lr, double mu,
                           int32_t nesterov, double weight_decay, double scale,
                           const double* coefficients, int32_t n_steps, double eps,
                           const float* clip_scale, void* workspace, size_t workspace_bytes,
                           hipStream_t stream);

/* zero_muon_step over a list of matrices of any shapes, described once in
 * device memory (as zero_mt_table_*): every product is one launch over all of
 * them. The results are zero_muon_step's on each matrix within its stated
 * precision: the form, the tiles and how the steps are grouped follow the whole
 * list, so one matrix with a short side above 128 takes those up to 128, which a
 * list of their own would leave 3e-5 off, to the precision of one fp16 part (where
 * few directions hold nearly all of the norm up to 1e-2 on short sides of 64, and
 * 5e-2 below 16).
 * Create: host arrays of n_matrices pointers, sides and scales; a matrix without
 * elements is left out. hipMalloc and a synchronous hipMemcpy on the current
 * device, once (128 bytes a matrix and 4 per workgroup). The table keeps the pointers,
 * not the data: the caller keeps the buffers alive and in place. The written
 * arrays must not overlap one another or a gradient.
 * Step: with the table's device current (ZERO_EINVAL otherwise); workspace of
 * zero_muon_table_workspace_bytes(table) bytes or more. An empty list enqueues nothing.
 * Free: releases the device memory (hipFree, which waits for the device); no
 * step using the table may still be running. Accepts NULL.
 * Matrices: those with elements, or -1 for NULL.
 * Errors: as zero_muon_step, the first overlap named in zero_last_error();
 * ZERO_EINVAL for a NULL out or a negative n_matrices; ZERO_ENOMEM; ZERO_EHIP. */
typedef struct zero_muon_table zero_muon_table;
zero_status zero_muon_table_create(float* const* masters, float* const* momenta,
                                   const uint16_t* const* grads, uint16_t* const* params_out,
                                   const int64_t* rows, const int64_t* cols, const double* scales,
                                   int32_t n_matrices, zero_muon_table** out);
void zero_muon_table_free(zero_muon_table* table);
size_t zero_muon_table_workspace_bytes(const zero_muon_table* table);
int32_t zero_muon_table_matrices(const zero_muon_table* table);
zero_status zero_muon_table_step(const zero_muon_table* table, double lr, double mu, int32_t nesterov,
                                 double weight_decay, const double* coefficients, int32_t n_steps,
                                 double eps, const float* clip_scale, void* workspace,
                                 size_t workspace_bytes, hipStream_t stream);

/* ------------------------------------------------------------------ gather
 *
 * [ZF] "Execution Flow for ZeRO-1", step 4 and "FSDP-1": the N_d bf16 shards,
 * concatenated in rank order, are the flat parameter buffer; tensor t is its
 * slice [offset_t, offset_t + numel_t). This copies every plan segment from
 * its shard into its tensor (padding is not copied). For a Shard(0) plan
 * ([ZF] "FSDP-2: Per-Parameter Sharding via DTensor"), tensor t is its ranks'
 * dim-0 chunks stacked in rank order, each read from its chunk's place in
 * that rank's coalesced buffer.
 * shards       host [N_d] of device pointers, each to S bf16 values. A NULL
 *              entry skips that rank's segments (their tensor elements are
 *              left as they are): ranks can be gathered in separate calls, for
 *              example the other ranks' while the own shard is being updated.
 * tensors      host [T] of device pointers, tensor t to numel_t bf16 values
 *              (may be NULL only for zero-sized tensors). Outputs must not
 *              overlap the shards or each other.
 * Errors: ZERO_EINVAL (null plan/arrays or a needed null pointer, a tensor
 * overlapping another tensor or a shard, named in zero_last_error());
 * ZERO_ENOMEM; ZERO_EHIP. */
zero_status zero_gather_params(const zero_plan* plan, const uint16_t* const* shards,
                               uint16_t* const* tensors, hipStream_t stream);

/* ------------------------------------------------------------------ flatten
 *
 * [ZF] "FSDP-1: FlatParameter and Module-Level Wrapping": a unit's tensors are
 * flattened into one contiguous 1-D buffer, padded to a length divisible by
 * the world size. This builds that buffer from per-tensor bf16 buffers: every
 * plan segment is copied from its tensor to its place in the flat buffer
 * (flat plans: tensor t at [offset_t, offset_t + numel_t); Shard(0) plans:
 * each rank's chunk into that rank's coalesced buffer) and every other
 * position is set to +0. It is the inverse of zero_gather_params and the step
 * before zero_grad_reduce_shard: each data-parallel replica flattens its
 * per-tensor gradients into the flat buffer that the reduce-scatter cuts into
 * N_d shards.
 * tensors      host [T] of device pointers, tensor t to numel_t bf16 values
 *              (may be NULL only for zero-sized tensors).
 * flat         device [P] bf16, written entirely; must not overlap the tensors.
 * Errors: ZERO_EINVAL (null plan/arrays or a needed null pointer, flat
 * overlapping a tensor, named in zero_last_error()); ZERO_ENOMEM; ZERO_EHIP. */
zero_status zero_flatten_params(const zero_plan* plan, const uint16_t* const* tensors,
                                uint16_t* flat, hipStream_t stream);

/* Gather and flatten for fixed buffers, with their tables in device memory.
 * A training loop gathers the same shards into the same tensors every step
 * (and flattens the same per-tensor gradients into the same flat buffer), so
 * the copy can be described once. zero_gather_table_create takes the
 * arguments of zero_gather_params, zero_flatten_table_create those of
 * zero_flatten_params, with the same checks. Each lists every plan segment
 * (for the flatten also every zero-filled gap) as a piece, and copies to
 * device memory that the table owns one 32-byte descriptor per piece (source,
 * destination, length) and one 4-byte piece index per workgroup of 2,048
 * elements (0.1% of the bytes copied). zero_copy_table_run then performs the
 * whole copy in one launch (several only past 2^24 workgroups, above 3.4e10
 * elements), for flat and Shard(0) plans alike, with the same result as the
 * call the table was made from: the same bits are copied, and the same
 * positions zero-filled.
 * Create: hipMalloc and a synchronous hipMemcpy on the current device, once.
 * The table keeps the device pointers, not the data: the caller keeps those
 * buffers alive and in place for the table's lifetime. A NULL shard skips its
 * rank, as in zero_gather_params. out receives the table.
 * Errors: as the call it mirrors; ZERO_EINVAL for a NULL out; ZERO_ERANGE for
 * 2^31 workgroups or more; ZERO_ENOMEM; ZERO_EHIP (allocation or copy).
 * Run: enqueued on stream; it must run with the table's device current
 * (ZERO_EINVAL otherwise). An empty table enqueues nothing.
 * Free: releases the device memory (hipFree, which waits for the device);
 * no run using the table may still be in flight. Accepts NULL.
 * Blocks: the workgroups of one run, or -1 for NULL. */
typedef struct zero_copy_table zero_copy_table;
zero_status zero_gather_table_create(const zero_plan* plan, const uint16_t* const* shards,
                                     uint16_t* const* tensors, zero_copy_table** out);
zero_status zero_flatten_table_create(const zero_plan* plan, const uint16_t* const* tensors,
                                      uint16_t* flat, zero_copy_table** out);
zero_status zero_copy_table_run(const zero_copy_table* table, hipStream_t stream);
int64_t zero_copy_table_blocks(const zero_copy_table* table);
void zero_copy_table_free(zero_copy_table* table);

/* Reduce from per-tensor replicas, for fixed buffers. [ZF] "FSDP-1:
 * FlatParameter and Module-Level Wrapping" (every tensor's place in the flat
 * padded buffer) with "Execution Flow for ZeRO-1", step 2 (the rank's slice
 * of the gradient averaged over the replicas). When the R replicas are still
 * per-tensor buffers, the rank's averaged gradient is reduced from them
 * directly, without first flattening each replica (zero_flatten_params): for
 * every segment of the rank's shard, tensor elements [tensor_offset,
 * tensor_offset + length) of each replica are reduced into shard elements
 * [shard_offset, shard_offset + length), and every other shard position
 * (padding) is set to +0. The bits are those of zero_flatten_params on each
 * replica followed by zero_grad_reduce_shard over the whole shard (fp32 sum in
 * replica order, one fp32 division by R, bf16 round-to-nearest-even); the
 * squared-norm partial, when asked for, is the same fp64 sum to within
 * rounding. Per shard element (2R + 2) bytes move, against 6R + 2 with the
 * flattens. Flat and Shard(0) plans alike.
 * plan, rank      the plan and this rank.
 * replica_tensors host [R * T] of device pointers: entry k * T + t is replica
 *                 k's tensor t, numel_t bf16 values; may be NULL only for
 *                 tensors with no segment in this rank's shard.
 * n_replicas      R, 1..ZERO_MAX_REPLICAS.
 * shard_grad      device [S] bf16, written entirely by each run; must not
 *                 overlap the replicas.
 * Create: lists the rank's segments and padding gaps as pieces and copies to
 * device memory that the table owns one 64-byte descriptor per piece, one
 * 4-byte piece index per workgroup of 2,048 shard elements, the R * T replica
 * pointers and room for one fp64 partial per workgroup (hipMalloc and a
 * synchronous hipMemcpy on the current device, once). The table keeps the
 * pointers, not the data: the caller keeps the buffers alive and in place.
 * Errors: ZERO_EINVAL (NULL out, plan, replica_tensors or shard_grad; rank or
 * R out of range; a NULL replica tensor the shard needs, or one that overlaps
 * shard_grad); ZERO_ERANGE (2^31
 * workgroups or more); ZERO_ENOMEM; ZERO_EHIP.
 * Run: enqueued on stream, with the table's device current (ZERO_EINVAL
 * otherwise); sqnorm_out (device double, nullable) receives the squared
 * norm of the written gradient. Runs of one table must not overlap (they
 * share its partials). Free: hipFree; accepts NULL. Blocks: the workgroups of
 * one run, or -1 for NULL. */
typedef struct zero_reduce_table zero_reduce_table;
zero_status zero_reduce_table_create(const zero_plan* plan, int32_t rank,
                                     const uint16_t* const* replica_tensors, int32_t n_replicas,
                                     uint16_t* shard_grad, zero_reduce_table** out);
zero_status zero_reduce_table_run(const zero_reduce_table* table, double* sqnorm_out,
                                  hipStream_t stream);
int64_t zero_reduce_table_blocks(const zero_reduce_table* table);
void zero_reduce_table_free(zero_reduce_table* table);

/* ------------------------------------------------------------------ ZeRO-Offload
 *
 * [ZF] "ZeRO-Offload Mechanics": the fp32 optimizer state lives in host DRAM;
 * the GPU's bf16 gradients travel to the host over PCIe / CXL, the host CPU
 * runs the fp32 Adam step and updates the fp32 weights, and the bf16
 * parameters travel back, the transfers overlapping the host work.
 *
 * zero_host_adamw_step: the host CPU update alone, on host arrays [n], with
 * zero_shard_adamw_step's exact per-element arithmetic (identical bits).
 * clip_scale is a host float (a non-finite value skips the step). The work is
 * split over a persistent pool of host threads: n_threads tasks, or one per
 * CPU in the calling process's affinity mask when n_threads <= 0. Calls from
 * several threads are safe; their parallel parts run one after another.
 * Errors: as zero_shard_adamw_step. */
zero_status zero_host_adamw_step(float* master, float* exp_avg, float* exp_avg_sq,
                                 const uint16_t* grad, uint16_t* param_out, int64_t n,
                                 int64_t step, double lr, double beta1, double beta2, double eps,
                                 double weight_decay, float clip_scale, int32_t n_threads);

/* zero_offload_adamw_step: one offloaded step. The bf16 gradient (device
 * d_grad [n]) is copied to the host chunk by chunk while the host updates the
 * previous chunk (h_master, h_exp_avg, h_exp_avg_sq: host [n] fp32, in place)
 * and the bf16 parameters of the chunk before go back to device
 * d_param_out [n]. h_staging: pinned host memory (hipHostMalloc or a pinned
 * torch tensor) of staging_elems bf16 values, split into two gradient and two
 * parameter buffers of staging_elems/4 elements each (the chunk size).
 * d_clip_scale: device float, nullable (1); a non-finite value skips the step
 * (nothing is written). n_threads: as zero_host_adamw_step. Work already
 * enqueued on `stream` happens before the gradient copies; work enqueued on
 * `stream` afterwards sees the new parameters. The copies run on two internal
 * streams of the current device (default priority). The call returns when the
 * host update is done and the staging buffers are free again, on errors too.
 * Calls from several host threads are safe: they share the worker pool and the
 * copy streams and so run one after another. The written ranges (the three
 * host state arrays, the staging in use, d_param_out) must not overlap one
 * another or d_grad.
 * Errors: as zero_host_adamw_step; ZERO_ENOSPACE if staging_elems < 4; ZERO_EHIP. */
zero_status zero_offload_adamw_step(float* h_master, float* h_exp_avg, float* h_exp_avg_sq,
                                    const uint16_t* d_grad, uint16_t* d_param_out,
                                    uint16_t* h_staging, int64_t staging_elems, int64_t n,
                                    int64_t step, double lr, double beta1, double beta2,
                                    double eps, double weight_decay, const float* d_clip_scale,
                                    int32_t n_threads, hipStream_t stream);

/* ------------------------------------------------------------------ diagnostics */
const char* zero_status_string(zero_status status);   /* static string */
const char* zero_last_error(void);                    /* thread-local; "" if none */

#ifdef __cplusplus
}
#endif

#endif /* ZERO_MI355X_H */
