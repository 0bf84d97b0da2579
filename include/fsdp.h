/*
 * fsdp.h - C ABI of the GB300 FSDP FlatParameter shard step.
 *
 * One GPU holds W virtual data-parallel ranks. For one FSDP unit the step is:
 * flatten the unit's tensors into one padded 1-D FlatParameter, reduce-scatter
 * the W bf16 full gradients (fp32 sum in fixed rank order, divided by W),
 * update each owned rank's fp32 master/exp_avg/exp_avg_sq shard with Adam in
 * place, cast the result to bf16, and all-gather the bf16 shards into the full
 * bf16 FlatParameter.
 *
 * The steps are labelled throughout the sources as follows:
 *   a1  flatten layout: tensor offsets, padding to a multiple of W, shard length
 *   a2  pack / unpack: tensors into the flat buffer (pad zeroed) and back
 *   a3  reduce-scatter: fp32 fold of the W bf16 rows in rank order, divided
 *       by W, at the rank's shard
 *   a4  Adam on a shard, in place (fp32 master, exp_avg, exp_avg_sq)
 *   a5  bf16 cast of the updated master shard
 *   a6  all-gather: the bf16 shards into the full FlatParameter
 *   a7  the fused step: a3 -> a4 -> a5 -> a6 in one pass
 *   a8  hybrid sharding (F | W): shard within groups of F, W / F replicas
 *   a9  closed-form memory and communication accountant
 *
 * Sources, cited by page title and section:
 *   [notes] "NOTE-003: PyTorch FSDP" (reading notes on the FSDP paper)
 *   [math]  "transformer math: FSDP"
 *   [gloss] glossary entry "fully sharded data parallel fsdp"
 *
 * Conventions for every call:
 *   - The caller owns all memory of the data. No call allocates, and the
 *     library keeps no state about the data between calls (it caches the SM
 *     count and kernel occupancy per device; fsdp_pipeline_step and
 *     fsdp_offload_step create and release CUDA events within a call; a
 *     per-device status word records a device wait that ran out, see
 *     fsdp_device_status). One fixed device array is part of the library's
 *     device code: the staging pool of fsdp_pipeline_step_noalloc, of
 *     FSDP_NOALLOC_STAGING_BYTES. The CUDA runtime reserves it on every GPU
 *     where it loads the library's device code, whether or not that entry
 *     point is ever called, and keeps it until the process exits.
 *   - Diagnostic calls that drive failure paths on purpose are declared in
 *     fsdp_test.h, not here.
 *   - "device" pointers point to CUDA global memory of the current device;
 *     pointer arrays themselves (const T* const*) are HOST arrays of device
 *     pointers and are read before the call returns.
 *   - Optimizer-state offload ([gloss] "CPU Offload"): the fp32 master,
 *     exp_avg and exp_avg_sq pointers of fsdp_shard_step(_grouped),
 *     fsdp_adam_shard_step and fsdp_pipeline_step may instead point to
 *     page-locked host memory mapped into the device's address space
 *     (cudaHostAlloc, or cudaHostRegister with cudaHostRegisterMapped, at an
 *     address the device can use as is). The kernels then read and write the
 *     state over the host link; nothing else changes. fsdp_offload_step
 *     instead copies the state between host memory and device slots.
 *   - bf16 values are passed as their uint16_t bit patterns; fp32 as float.
 *   - Every GPU call is asynchronous on `stream` (0 = legacy default stream).
 *     Inputs must stay unchanged, and outputs untouched, until the stream has
 *     passed the call.
 *   - Return value: FSDP_OK (0) or a negative status (below). All arguments
 *     are validated on the host before anything is launched; on a negative
 *     status nothing was launched (except FSDP_ECUDA from a failed launch).
 *     Kernels never trap.
 *   - Results are deterministic: the same inputs give bit-identical outputs.
 *   - Sizes are int64_t element counts; all device index arithmetic is 64-bit.
 */
#ifndef FSDP_GB300_H
#define FSDP_GB300_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* Same type as cudaStream_t; declared here so the header needs no CUDA headers. */
typedef struct CUstream_st *fsdp_stream_t;

#define FSDP_OK 0
#define FSDP_EINVAL (-1) /* null pointer, bad size, W outside [1,64], F not dividing W,
                            rank outside [0,W), inconsistent layout, step < 1,
                            weight_decay != 0, ... */
#define FSDP_EALIAS (-2) /* an output overlaps an input or another output */
#define FSDP_ECUDA (-3)  /* a CUDA call or launch failed (cudaGetLastError) */
#define FSDP_ENOSPACE (-4) /* the work does not fit the fixed staging capacity of
                              fsdp_pipeline_step_noalloc */
#define FSDP_EWORKSPACE (-5) /* the given workspace is smaller than the call needs */

#define FSDP_MAX_WORLD 64

#define FSDP_DTYPE_F32 0  /* 4-byte elements (fp32 master) */
#define FSDP_DTYPE_BF16 1 /* 2-byte elements (bf16 bits) */

/* Layout of one FlatParameter. [math] "The sharding unit: FlatParameter and the
 * wrapping policy": the unit's tensors are flattened into one 1-D buffer that is
 * split evenly over the ranks, each rank holding one contiguous slice.
 * [notes] "Key results": sharding factor F (F = W full shard, F = 1 DDP,
 * 1 < F < W hybrid). */
typedef struct {
  int64_t numel;        /* P: real elements (sum of tensor numels) */
  int64_t padded_numel; /* ceil(P / W) * W: zero padding at the end */
  int64_t shard_numel;  /* S = padded_numel / F: one rank's slice */
  int32_t world_size;   /* W, 1..64 */
  int32_t shard_factor; /* F, divides W; R = W / F replica groups */
  int32_t n_tensors;
} fsdp_layout_t;

/* Adam hyper-parameters (Kingma & Ba 2015, Algorithm 1; the pages name the
 * optimizer only: [math] "Why FSDP exists", [gloss] "Optimizer Step").
 * Each per-element fp32 scalar (lr, beta1, beta2, eps, 1-beta1, 1-beta2,
 * 1-beta1^step, 1-beta2^step) is formed in double and rounded once to fp32. */
typedef struct {
  double lr;
  double beta1;        /* in [0, 1) */
  double beta2;        /* in [0, 1) */
  double eps;          /* >= 0, added outside the square root */
  double weight_decay; /* must be 0 (the method uses none) */
  int64_t step;        /* t >= 1: the step being taken */
} fsdp_adam_t;

/* a1. Flatten layout (host only, no GPU).
 * [math] "The sharding unit: FlatParameter and the wrapping policy".
 * numels: n_tensors element counts (>= 0) in the order the tensors are packed
 * (row-major, concatenated, no padding between tensors).
 * offsets_out: caller-owned array of n_tensors + 1 entries; offsets_out[i] is
 * tensor i's first flat element, offsets_out[n_tensors] = P.
 * out: the layout. Padding is to a multiple of W for every F, so the layout is
 * the same for all sharding factors. EINVAL: n_tensors < 1, a negative numel,
 * W outside [1,64], F < 1 or F not dividing W, a null pointer. */
int fsdp_flatten_layout(const int64_t *numels, int32_t n_tensors, int32_t world_size,
                        int32_t shard_factor, int64_t *offsets_out, fsdp_layout_t *out);

/* a2. Pack tensors into the flat buffer (one launch), zero-filling the pad.
 * [math] "The sharding unit: FlatParameter and the wrapping policy": a unit's
 * parameters are flattened into one contiguous 1-D buffer (row-major, in the
 * listed order) that splits evenly over the ranks.
 * tensors: host array of n_tensors device pointers (contiguous tensors of the
 * element type `dtype`); offsets: the host array fsdp_flatten_layout wrote;
 * flat_out: device buffer of padded_numel elements. Pad elements become +0.0
 * (all-zero bits). EINVAL: a bad layout, dtype or offsets, a null pointer;
 * EALIAS if flat_out overlaps a tensor. */
int fsdp_pack_flat(const void *const *tensors, const fsdp_layout_t *layout,
                   const int64_t *offsets, int32_t dtype, void *flat_out, fsdp_stream_t stream);

/* a2. Unpack: copy each tensor's range of the flat buffer back out (pad dropped).
 * [math] "The sharding unit: FlatParameter and the wrapping policy": the
 * tensors are views of their ranges of the FlatParameter; this is the inverse
 * of fsdp_pack_flat. flat: device buffer of padded_numel elements of `dtype`;
 * tensors_out: host array of n_tensors device pointers, tensor i receives
 * elements [offsets[i], offsets[i+1]). EINVAL as for fsdp_pack_flat; EALIAS if
 * a tensor overlaps the flat buffer or another tensor. */
int fsdp_unpack_flat(const void *flat, const fsdp_layout_t *layout, const int64_t *offsets,
                     int32_t dtype, void *const *tensors_out, fsdp_stream_t stream);

/* a3. Reduce-scatter for one rank.
 * [math] "The backward cycle: all-gather, grads, reduce-scatter"; [gloss]
 * "Mixed Precision" (reduce_dtype fp32).
 * grads: host array of W device pointers, grads[k] = rank k's bf16 full
 * gradient, padded_numel elements (pad elements are expected to be zero).
 * rank: in [0, W); it keeps position p = rank mod F, i.e. elements [p*S, (p+1)*S).
 * grad_shard_out: device fp32 [S]:
 *   out[j] = ((((0 + g_0[pS+j]) + g_1[pS+j]) + ... ) + g_{W-1}[pS+j]) / W
 * a left fold in rank order over all W ranks, one fp32 rounding per add, IEEE
 * division. EALIAS if the output overlaps a gradient row. */
int fsdp_reduce_scatter(const uint16_t *const *grads, const fsdp_layout_t *layout,
                        int32_t rank, float *grad_shard_out, fsdp_stream_t stream);

/* a3 for the owned ranks [rank_begin, rank_end) in one launch (the same
 * definition and passages as fsdp_reduce_scatter; one GPU holding several
 * ranks reduces all of their slices at once).
 * grads: as in fsdp_reduce_scatter. grad_shards_out: rank_end - rank_begin
 * device pointers, fp32 [S] each, indexed by r - rank_begin; rank r's output
 * is fsdp_reduce_scatter of rank r bit for bit (ranks at the same position of
 * different groups get identical copies). EINVAL: a bad layout or rank range,
 * a null pointer; EALIAS: an output overlaps a gradient row or another
 * output. */
int fsdp_reduce_scatter_ranks(const uint16_t *const *grads, const fsdp_layout_t *layout,
                              int32_t rank_begin, int32_t rank_end, float *const *grad_shards_out,
                              fsdp_stream_t stream);

/* a4 + a5. Adam on one shard, in place, and its bf16 cast.
 * [math] "Why FSDP exists" (fp32 master, fp32 momentum and variance) and "The
 * backward cycle" (the optimizer updates the local slice in place).
 * master, exp_avg, exp_avg_sq: device fp32 [n], updated in place:
 *   m = b1 m + (1-b1) g;  v = b2 v + (1-b2) g*g;
 *   p = p - lr * ((m / (1-b1^t)) / (sqrt(v / (1-b2^t)) + eps))
 * every operation one fp32 rounding (no fused multiply-add).
 * grad_shard: device fp32 [n] (read only). bf16_shard_out: device bf16 [n],
 * round-to-nearest-even of the new master, or NULL for none. n >= 0. */
int fsdp_adam_shard_step(float *master, float *exp_avg, float *exp_avg_sq,
                         const float *grad_shard, int64_t n, const fsdp_adam_t *adam,
                         uint16_t *bf16_shard_out, fsdp_stream_t stream);

/* One shard of fsdp_adam_shard_step_grouped (same meaning as the arguments of
 * fsdp_adam_shard_step). */
typedef struct {
  float *master;            /* device fp32 [n], in place */
  float *exp_avg;           /* device fp32 [n], in place */
  float *exp_avg_sq;        /* device fp32 [n], in place */
  const float *grad_shard;  /* device fp32 [n], read only */
  uint16_t *bf16_shard_out; /* device bf16 [n], or NULL */
  int64_t n;                /* >= 0 */
} fsdp_adam_shard_t;

/* a4 + a5 over several shards (e.g. the shards of every rank a GPU holds, or
 * of several units) in one launch, with the same definition and passages as
 * fsdp_adam_shard_step and one set of hyper-parameters. Each shard's results
 * equal fsdp_adam_shard_step on it bit for bit. n_shards == 0 is a no-op.
 * EINVAL: n_shards < 0, a negative n, a null state or gradient pointer of a
 * non-empty shard, bad hyper-parameters; EALIAS: an output overlaps a
 * gradient or another output (of any shard). */
int fsdp_adam_shard_step_grouped(const fsdp_adam_shard_t *shards, int32_t n_shards,
                                 const fsdp_adam_t *adam, fsdp_stream_t stream);

/* a6. All-gather (unshard) one group.
 * [math] "The forward cycle: all-gather, compute, reshard".
 * shards: host array of F device pointers, shards[k] = bf16 [S] of position k;
 * full_out: device bf16 [padded_numel]; full_out[k*S + j] = shards[k][j].
 * A shard that already is the view full_out + k*S is left in place. */
int fsdp_all_gather(const uint16_t *const *shards, const fsdp_layout_t *layout,
                    uint16_t *full_out, fsdp_stream_t stream);

/* a7 / a8. Fused shard step of one unit for the owned ranks [rank_begin, rank_end):
 * reduce-scatter -> Adam -> bf16 cast -> all-gather in one launch, with no fp32
 * gradient written to memory.
 * Rank r belongs to group g = r / F (contiguous ranks form a group) at position
 * p = r mod F ([gloss] "Hybrid Sharding", "HSDP": shard within a group,
 * replicate across groups).
 *   grads:        W device pointers, bf16 [padded_numel] each (as in a3). For
 *                 every F all W ranks are summed in global rank order, so every
 *                 F gives bit-identical parameters.
 *   master, exp_avg, exp_avg_sq:
 *                 rank_end - rank_begin device pointers, fp32 [S] each, indexed
 *                 by r - rank_begin; updated in place (a4).
 *   other_shards: NULL when every group that contains an owned rank is fully
 *                 owned (all-ranks mode); otherwise W device pointers indexed by
 *                 rank, bf16 [S]: the already-updated shards of the non-owned
 *                 ranks in those groups (local-rank mode; entries of owned
 *                 ranks and of other groups are ignored and may be NULL).
 *   full_out:     R = W / F device pointers indexed by group, bf16 [padded_numel];
 *                 every group containing an owned rank is written completely:
 *                 owned positions with the new bf16 shard, the others copied
 *                 from other_shards (skipped when other_shards[r] already is
 *                 full_out[g] + p*S). Entries of other groups are ignored.
 * Positions owned by several replicas are reduced once and the result applied
 * to every replica. EALIAS: an output overlaps an input or another output.
 * padded_numel == 0 is a no-op. */
int fsdp_shard_step(const uint16_t *const *grads, const fsdp_layout_t *layout,
                    int32_t rank_begin, int32_t rank_end, float *const *master,
                    float *const *exp_avg, float *const *exp_avg_sq,
                    const uint16_t *const *other_shards, uint16_t *const *full_out,
                    const fsdp_adam_t *adam, fsdp_stream_t stream);

/* Arguments of one unit for fsdp_shard_step_grouped (same meaning as above). */
typedef struct {
  const fsdp_layout_t *layout;
  const uint16_t *const *grads;
  float *const *master;
  float *const *exp_avg;
  float *const *exp_avg_sq;
  const uint16_t *const *other_shards;
  uint16_t *const *full_out;
} fsdp_unit_args_t;

/* a7 over several units (e.g. one per transformer block, [math] "The sharding
 * unit": transformer_auto_wrap_policy makes each block a unit) in one launch
 * when they fit the launch's descriptor table, else in as few as needed.
 * The launch runs every unit's fused step first and then every unit's gather
 * of the other ranks' shards (the two touch disjoint memory, so the order
 * does not change any result). When many of the segments lie off 16-byte
 * alignment (shard lengths not a multiple of 8) and the aligned ones alone
 * fill the TMA form, the aligned segments go in a first launch and the
 * others in a second (again no result changes). All units share W, F, the owned rank range
 * and the hyper-parameters. Units must not share output memory.
 * n_units == 0 is a no-op. */
int fsdp_shard_step_grouped(const fsdp_unit_args_t *units, int32_t n_units, int32_t rank_begin,
                            int32_t rank_end, const fsdp_adam_t *adam, fsdp_stream_t stream);

/* Host only: the number of kernel launches fsdp_shard_step_grouped would make
 * for these arguments (validated exactly as the call validates them; nothing is
 * launched). *launches_out is written on FSDP_OK. */
int fsdp_shard_step_grouped_launches(const fsdp_unit_args_t *units, int32_t n_units,
                                     int32_t rank_begin, int32_t rank_end,
                                     int32_t *launches_out);

/* As fsdp_shard_step_grouped_launches, and *tma_launches_out (if not NULL)
 * receives how many of those launches use the TMA form of the kernel (bulk
 * copies into a shared-memory pipeline; chosen for W = 8 launches made of
 * one-replica step segments, and copies, for W = 16 ones whose gradient rows
 * do not all lie a multiple of 2 KB apart, and for launches of copies only, each with
 * enough chunks to fill every SM's pipeline and at most one eighth of its step
 * and of its copy chunks off 16-byte alignment), *tma_interleaved_out (if not
 * NULL) how many of the W = 8 TMA launches stage their step chunks in four
 * interleaved rounds of quarter-chunk copies (chosen when a launch's gradient
 * rows span 3 GiB or more of addresses).
 * Needs no GPU, but reads the SM count of the current device when one is
 * present. */
int fsdp_shard_step_grouped_plan(const fsdp_unit_args_t *units, int32_t n_units,
                                 int32_t rank_begin, int32_t rank_end, int32_t *launches_out,
                                 int32_t *tma_launches_out, int32_t *tma_interleaved_out);

/* The current device's sticky status word, read after all work of the
 * device, on every stream, has finished (the call synchronizes the device). Bit 0 is
 * set when a bounded wait of the TMA form (or of the norm's backward pass, the
 * orthogonalisation or the Muon step) ran out (2 s on one mbarrier): the
 * block that saw it stopped early, so the outputs of that launch are not
 * valid. This does not happen in a correct run. clear != 0 resets the word
 * after reading it. EINVAL: status_out NULL; ECUDA: the read failed. */
int fsdp_device_status(int32_t clear, uint32_t *status_out);

/* Pipelined step of one rank over many units (full sharding, F = W), with a
 * bounded pool of staging slots for the incoming gradients.
 * [notes] "Key results" (backward prefetching: issue the next unit's
 * collective before the current one finishes), [math] "Overlap: prefetching to
 * hide the collectives" and "Per-unit memory and communication, in numbers"
 * (transient = 2 U (1 + prefetch) bytes of bf16 per rank).
 * For unit u in order, slot s = u mod n_slots:
 *   on `copy`:    wait until the unit that last used slot s has been stepped,
 *                 then copy its W x S gradient slices into slot s;
 *   on `compute`: wait for that copy, run the fused local-rank step of `rank`
 *                 reading the gradients from slot s (reduce-scatter, Adam,
 *                 bf16 cast, all-gather of the other shards into full_out),
 *                 then copy the new bf16 shard to shard_out if given.
 * With n_slots = 1 (prefetch 0) copies and steps alternate; with n_slots = 2
 * (prefetch 1) the copy of unit u+1 overlaps the step of unit u.
 * The first and the last unit go through the same cycle in pieces of at most
 * 4,194,304 shard elements (whole 2048-element chunks; one 2D copy of the W
 * slices' ranges, one step and one shard_out copy per piece; each piece takes
 * the next slot), so that the first step starts before a whole unit has
 * arrived and little remains after the last copy in. Results do not depend on
 * the pieces.
 * staging: device bf16 buffer of n_slots x slot_numel elements, caller-owned,
 * slot_numel >= padded_numel of every unit (its W x S slices); n_slots in
 * [1, 8]; its contents are overwritten. The pool's size is the transient
 * gradient budget: 2 * n_slots * slot_numel bytes.
 * The call's copies start after the work queued on `compute` before the call
 * (so inputs written there, and a previous call's steps, come first); when the
 * call returns, `compute` is ordered after everything the call queued on both
 * streams, so later work on `compute` sees the results (order later work on
 * `copy` after `compute` yourself). The two streams may be the same stream (no
 * overlap). The call can be captured into a CUDA graph from `compute`.
 * Results are bit-identical to fsdp_shard_step_grouped on the same values.
 * EINVAL: F != W, a unit with
 * another W, bad rank, n_slots outside [1,8], a slot too small, null pointers;
 * EALIAS: outputs overlapping inputs, the staging pool or each other. */
typedef struct {
  const fsdp_layout_t *layout;
  const uint16_t *grad_slices;         /* W x S bf16 (row k = rank k's gradient at the
                                          owned slice), host (pinned) or device memory */
  float *master;                       /* device fp32 [S] of the owned rank, in place */
  float *exp_avg;                      /* device fp32 [S] */
  float *exp_avg_sq;                   /* device fp32 [S] */
  const uint16_t *const *other_shards; /* W device pointers by rank; the owned rank's entry
                                          is ignored */
  uint16_t *full_out;                  /* device bf16 [padded_numel] */
  uint16_t *shard_out;                 /* bf16 [S] (host or device) or NULL */
} fsdp_pipeline_unit_t;

int fsdp_pipeline_step(const fsdp_pipeline_unit_t *units, int32_t n_units, int32_t rank,
                       uint16_t *staging, int64_t slot_numel, int32_t n_slots,
                       const fsdp_adam_t *adam, fsdp_stream_t compute, fsdp_stream_t copy);

/* Staged optimizer-state offload: one rank's step over many units (full
 * sharding, F = W) with that rank's fp32 master, exp_avg and exp_avg_sq
 * shards in host memory.
 * [gloss] "CPU Offload" (optimizer state held in CPU memory and brought to the
 * GPU for the update); [math] "The backward cycle: all-gather, grads,
 * reduce-scatter" (the per-unit step it wraps).
 * For unit u in order, slot s = u mod n_slots of `staging`:
 *   on `h2d`:     wait until the unit that last used slot s is back in host
 *                 memory, then copy the unit's master, exp_avg, exp_avg_sq
 *                 (S fp32 each) into slot s;
 *   on `compute`: wait for those copies, run the fused local-rank step of
 *                 `rank` on the state in slot s (reduce-scatter of the rank's
 *                 slice of the W gradient rows, Adam, bf16 cast into full_out,
 *                 all-gather of the other ranks' shards into full_out);
 *   on `d2h`:     wait for the step, copy the three updated shards back to
 *                 host memory.
 * With n_slots >= 2 the copy in of unit u+1, the step of unit u and the copy
 * back of unit u-1 overlap, so both directions of the host link are busy at
 * once (the zero-copy form of the conventions above moves the same state by
 * kernel loads and stores instead).
 * staging: device fp32 buffer of n_slots x 3 x slot_numel, caller-owned,
 * contents overwritten; slot_numel >= shard_numel of every unit (a multiple
 * of 4 keeps every slot array 16-byte aligned, the vector path). n_slots in
 * [1, 8]. master/exp_avg/exp_avg_sq: host memory, page-locked for the copies
 * to overlap (pageable memory works but each copy then waits for the host);
 * device memory also works. The call's copies start after the work queued
 * on `compute` before the call; when the call returns, `compute` is ordered
 * after everything the call queued, the last copy back included, so later work
 * on `compute` sees the updated state. The streams may coincide (no overlap).
 * The call can be captured into a CUDA graph from `compute`. Results are
 * bit-identical to fsdp_shard_step_grouped with the same state in HBM.
 * EINVAL: F != W, a unit with another W, bad rank, n_slots outside [1,8], a
 * slot too small, null pointers; EALIAS: outputs (state, full_out, staging)
 * overlapping inputs or each other. */
typedef struct {
  const fsdp_layout_t *layout;
  const uint16_t *const *grads;        /* W device bf16 rows of padded_numel (rank k's
                                          gradient); the step reads the owned slice */
  float *master;                       /* fp32 [S] of the owned rank, host memory, in place */
  float *exp_avg;                      /* fp32 [S], host memory, in place */
  float *exp_avg_sq;                   /* fp32 [S], host memory, in place */
  const uint16_t *const *other_shards; /* W device pointers by rank; the owned rank's entry
                                          is ignored */
  uint16_t *full_out;                  /* device bf16 [padded_numel] */
} fsdp_offload_unit_t;

int fsdp_offload_step(const fsdp_offload_unit_t *units, int32_t n_units, int32_t rank, float *staging,
                      int64_t slot_numel, int32_t n_slots, const fsdp_adam_t *adam,
                      fsdp_stream_t compute, fsdp_stream_t h2d, fsdp_stream_t d2h);

/* Allocation-free form of fsdp_pipeline_step. (The FSDP pages have no
 * counterpart: this exists for callers, not for the method.)
 * For callers that cannot allocate device memory where they step the
 * optimizer: processes whose device memory is owned entirely by another
 * allocator (a framework's caching allocator, or a fixed arena carved out at
 * start-up), and loops that must not call cudaMalloc because it can
 * synchronize the device and stall the very streams the pipeline overlaps.
 * They pass only inputs and outputs; the staging pool is a fixed array of
 * FSDP_NOALLOC_STAGING_BYTES inside the library's device code, which the CUDA
 * runtime reserves on a GPU when it loads that code there and keeps until the
 * process exits. The call itself allocates nothing.
 * Same arguments and results as fsdp_pipeline_step, with slot_numel = the
 * largest padded_numel among the units rounded up to a multiple of 8 (so every
 * slot starts 16-byte aligned). FSDP_ENOSPACE (nothing launched) if
 * n_slots * slot_numel * 2 exceeds FSDP_NOALLOC_STAGING_BYTES.
 * The first call on a device looks up the array's device address (with that
 * device current); make that first call before any stream capture. Every
 * call on a device uses the same array: calls whose work overlaps on the GPU
 * (different streams without ordering between them) race on it and give
 * wrong results. Each unit's slot is filled completely before it is read, so
 * nothing needs clearing between calls. */
#define FSDP_NOALLOC_STAGING_BYTES (64ll << 20)

int fsdp_pipeline_step_noalloc(const fsdp_pipeline_unit_t *units, int32_t n_units, int32_t rank,
                               int32_t n_slots, const fsdp_adam_t *adam, fsdp_stream_t compute,
                               fsdp_stream_t copy);

/* Gather of any per-rank state into the full flat buffer of a group, for the
 * full state dict. [gloss] "Checkpoint/Resume": FULL_STATE_DICT gathers the
 * full model (on rank 0) instead of saving one piece per rank.
 * shards: F device pointers, shards[k] = S elements of position k, element
 * type `dtype` (FSDP_DTYPE_F32 for master / exp_avg / exp_avg_sq, FSDP_DTYPE_BF16
 * for parameters); full_out: padded_numel elements, full_out[k*S + j] =
 * shards[k][j]. A shard that already is the view full_out + k*S is left in
 * place. fsdp_unpack_flat then splits full_out into the unit's tensors. */
int fsdp_all_gather_state(const void *const *shards, const fsdp_layout_t *layout, int32_t dtype,
                          void *full_out, fsdp_stream_t stream);

/* ZeRO stage 1 step of one rank ([gloss] "ZeRO Stages": stage 1 shards only
 * the optimizer state; every rank keeps the full model and the full averaged
 * gradient; [notes] "Key results": F = 1 reduces to an all-reduce).
 * Two launches on `stream`: (1) the all-reduce average of the W bf16 gradients
 * over the whole padded buffer into avg_grad_out (fp32 [padded_numel], the
 * same fixed-order fold and division as the reduce-scatter); (2) Adam on the
 * rank's slice avg_grad_out[rank*S, (rank+1)*S) of its fp32 master/exp_avg/
 * exp_avg_sq [S] with the bf16 result written to full_out + rank*S, and the
 * other ranks' bf16 shards copied into full_out (other_shards by rank, the
 * owned entry ignored). Requires F = W. Results equal fsdp_shard_step of the
 * same rank bit for bit; avg_grad_out equals fsdp_reduce_scatter with F = 1. */
int fsdp_zero1_step(const uint16_t *const *grads, const fsdp_layout_t *layout, int32_t rank,
                    float *avg_grad_out, float *master, float *exp_avg, float *exp_avg_sq,
                    const uint16_t *const *other_shards, uint16_t *full_out, const fsdp_adam_t *adam,
                    fsdp_stream_t stream);

/* ZeRO-stage accountant (host only). Per-GPU persistent bytes with the 16
 * bytes per parameter of [math] "Why FSDP exists" split as 2 (bf16 weights)
 * + 2 (bf16 gradients) + 12 (fp32 master, m, v), and [gloss] "ZeRO Stages":
 *   stage 0 (DDP): 2P + 2P + 12P
 *   stage 1: 2P + 2P + 12P/N      (optimizer state sharded)
 *   stage 2: 2P + 2P/N + 12P/N    (+ gradients sharded)
 *   stage 3: 2P/N + 2P/N + 12P/N  (+ parameters sharded: FSDP full sharding)
 * comm_elems per rank per step (pages' rounded form, [math] "Per-unit memory
 * and communication"): 2P for stages 0-2 (an all-reduce, or reduce-scatter +
 * all-gather), 3P for stage 3. reduction_vs_ddp = 16P / total_bytes. */
typedef struct {
  double weights_bytes;
  double grads_bytes;
  double optimizer_bytes;
  double total_bytes;
  double reduction_vs_ddp;
  double comm_elems;
} fsdp_zero_account_t;

int fsdp_account_zero(double P, int32_t N, int32_t stage, fsdp_zero_account_t *out);

/* a9. Closed-form accountant (host only).
 * [math] "Why FSDP exists": ~16 bytes per parameter (bf16 weight + bf16 grad +
 * fp32 master + two fp32 Adam moments); DDP keeps 16P on every GPU.
 * [math] "Per-unit memory and communication, in numbers":
 *   persistent = 16 P / N, transient = 2 U (1 + prefetch); a ring all-gather or
 *   reduce-scatter moves ~P per rank, an all-reduce ~2P; FSDP pays
 *   AG(fwd) + AG(bwd) + RS(bwd) ~ 3P against DDP's ~2P; bf16 on the wire.
 * With sharding factor F over N ranks (R = N / F groups): persistent 16 P / F;
 * the three collectives run inside a group and the gradient slice P/F is
 * all-reduced across the R groups:
 *   comm_elems_ring = 3 (F-1)/F P + 2 (R-1)/R P/F
 *   comm_elems      = 3P [F > 1] + 2 P/F [R > 1]   (the pages' rounded form)
 * P, U: total parameters and parameters of the largest unit; prefetch >= 0
 * units gathered ahead. EINVAL: N < 1, F < 1, F not dividing N, negatives. */
typedef struct {
  double persistent_bytes;     /* 16 P / F */
  double ddp_persistent_bytes; /* 16 P */
  double transient_bytes;      /* 2 U (1 + prefetch) */
  double peak_bytes;           /* persistent + transient */
  double comm_elems;           /* per rank per step, rounded form */
  double comm_elems_ring;      /* per rank per step, exact ring form */
  double ddp_comm_elems;       /* 2P */
  double ddp_comm_elems_ring;  /* 2 (N-1)/N P */
  double comm_bytes;           /* 2 bytes per element */
  double ddp_comm_bytes;
} fsdp_account_t;

int fsdp_account(double P, double U, int32_t N, int32_t F, int32_t prefetch,
                 fsdp_account_t *out);

/* ------------------------------------------------------------------------
 * Operators of the training loop around the step.
 *
 * A unit's tensors are matrices (projections) and vectors (norm gains,
 * biases). The calls below are the norm that the gains belong to, forward and
 * backward, and an optimizer for the matrices: the Muon step, which
 * orthogonalises every matrix's update. (The FSDP pages have no counterpart.)
 *
 * Matrices are row-major with a row stride in elements (>= the row's length;
 * any value for a single row). Bytes beside a row in the 16-byte units that hold its ends may be
 * read, without effect; they are never written. A workspace is device memory of the caller, of
 * any alignment, at least as large as the call's ..._workspace function says
 * for the same arguments; it holds nothing between calls, and calls whose
 * work overlaps on the GPU need workspaces of their own. */

#define FSDP_DTYPE_E4M3 2 /* 1-byte elements (8-bit floats: 4 exponent, 3 mantissa bits) */

/* RMS norm of each row, with the residual's addition:
 *   h = x + residual                  (h = x without a residual)
 *   rstd = 1 / sqrt(mean_j h_j^2 + eps)
 *   y_j = h_j rstd gain_j
 * x, residual and h_out have type `dtype` (F32 or BF16), gain has gain_dtype,
 * y has y_dtype: `dtype`'s own, or E4M3 with scales. All sums are fp32, and
 * y comes from the unrounded h. residual and h_out are both null or both given;
 * rstd (fp32 [rows]) may be null.
 * E4M3: each row is cut into groups of `group` consecutive elements (32, 64, 128
 * or 256; 0: the whole row; the last group may be short), and
 *   scale = max(max|y| / 448, 2^-126),   y_out = round(y (1 / scale))
 * to the nearest even e4m3 value, at most 448, formed in fp32 (rstd and 1 / scale may be
 * multiplied first). A value on the boundary between two e4m3 values, or within a few
 * fp32 roundings of it, may go to either: with bf16 inputs about 0.04 % of the values lie
 * exactly on one. scales is fp32 [rows][ceil(cols / group)], contiguous. Other y types:
 * scales null and group 0. A row with an infinity or a NaN gives what the formulas give; the
 * maximum over a NaN is a NaN, so a group with one (an infinity times rstd = 0 included)
 * has the scale NaN and NaN for all its values.
 * In place: h_out may be x or residual, and y may be x (same address, stride
 * and type), as long as the outputs are distinct; column slices of one
 * buffer (equal strides, disjoint columns) may be mixed freely.
 * rows = 0 launches nothing. EINVAL: cols < 1 or > 2^30, rows < 0, a stride below cols, a
 * type, group or eps (finite, a float above 0) outside the above, a missing pointer, one not
 * aligned to its elements. EALIAS: other overlaps. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t x_stride;
  int64_t residual_stride;
  int64_t h_stride;
  int64_t y_stride;
  int32_t dtype;
  int32_t gain_dtype;
  int32_t y_dtype;
  int32_t group;
  double eps;
} fsdp_rmsnorm_t;

int fsdp_rmsnorm(const fsdp_rmsnorm_t *args, const void *x, const void *residual, const void *gain, void *h_out,
                 void *y, float *scales, float *rstd, fsdp_stream_t stream);

/* Gradients of fsdp_rmsnorm. dy: gradient of y; h, rstd: the forward's (h is x
 * where it had no residual); dh: gradient that reaches h by the residual path
 * (null: none). With u_j = dy_j gain_j and n_j = h_j rstd:
 *   dx_j = rstd (u_j - n_j mean_i(u_i n_i)) + dh_j   (also the residual's gradient)
 *   dgain_j = sum over the rows of dy_j n_j
 * dy, h, dh and dx have type `dtype`, gain and dgain gain_dtype. Sums are fp32
 * in an order fixed by the sizes; each output is rounded once. dgain may lie
 * anywhere in a rank's bf16 gradient row (2-byte alignment). dx may be dy or dh in place.
 * rows = 0 sets dgain to zero. EINVAL and EALIAS as above. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t dy_stride;
  int64_t h_stride;
  int64_t dh_stride;
  int64_t dx_stride;
  int32_t dtype;
  int32_t gain_dtype;
} fsdp_rmsnorm_backward_t;

int fsdp_rmsnorm_backward(const fsdp_rmsnorm_backward_t *args, const void *dy, const void *h, const void *gain,
                          const float *rstd, const void *dh, void *dx, void *dgain, void *workspace,
                          int64_t workspace_bytes, fsdp_stream_t stream);
int fsdp_rmsnorm_backward_workspace(int64_t rows, int64_t cols, int64_t *bytes_out);

/* Newton-Schulz orthogonalisation of matrices (Higham, "Functions of Matrices",
 * 2008, chapter 8, gives the iteration family; the default quintic is the one
 * that the Muon optimizer made common): with X_0 = G / (|G|_F + eps), each step
 * with its a, b, c
 *   A = X X^T,   X <- a X + (b A + c A^2) X
 * (for a matrix with more rows than columns, of its transpose). The result has
 * G's singular vectors and singular values near 1; a zero matrix stays zero.
 * terms: how the products take their operands. 1: rounded to 11 bits (fp16,
 * scaled by powers of two; the error is below 0.3 % of the result's norm,
 * typically 0.03 to 0.1 %); 3: as two such parts each, three products (about 1e-5); 0: 3 where the
 * short side is below 256 and 1 otherwise. Between steps X is held as two fp16
 * parts, 22 bits; accumulation is fp32, in segments of at most 16384 elements
 * along a long side (1e-4 at the longest). |G|^2 is an fp32 sum: |G| has to be below 1e19, and
 * with an eps below 1e-18 above that. */
typedef struct {
  int32_t steps;              /* 1 .. 32 */
  int32_t terms;              /* 0, 1 or 3 */
  const double *coefficients; /* host: a, b, c of each step (3 * steps values); null: 3.4445,
                                 -4.7750, 2.0315 for every step */
  double eps;                 /* finite, at least 2^-126 */
} fsdp_newton_schulz_t;

typedef struct {
  const void *source; /* rows x cols, type dtype */
  uint16_t *out;      /* rows x cols, bf16; may be source itself (same address, stride, BF16) */
  int64_t rows;
  int64_t cols;
  int64_t source_stride;
  int64_t out_stride;
  int32_t dtype; /* F32 or BF16 */
} fsdp_matrix_t;

/* Orthogonalises n matrices (host array), together in each launch. Empty
 * matrices are skipped. newton_schulz null: 5 steps, terms 0, eps 1e-7.
 * EINVAL: also coefficients whose iterates leave [-7, 7] or whose b s + c s^2
 * leaves [-30, 30] for some singular value in [0, 1] (the fp16 ranges); a side beyond
 * 2^30. EALIAS: an out that overlaps another out or a source but its own. */
int fsdp_newton_schulz(const fsdp_matrix_t *matrices, int32_t n, const fsdp_newton_schulz_t *newton_schulz,
                       void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);
int fsdp_newton_schulz_workspace(const fsdp_matrix_t *matrices, int32_t n, const fsdp_newton_schulz_t *newton_schulz,
                                 int64_t *bytes_out);

/* The Muon step of one unit, all W ranks (F = W): as fsdp_shard_step, with the
 * unit's matrices updated by
 *   g = fold of the W gradients / W                        (a3)
 *   m = momentum m + g                                     (exp_avg, in place)
 *   u = g + momentum m  (nesterov)  or  m
 *   p = p (1 - lr weight_decay) - lr scale O               (O: u orthogonalised)
 * and its other tensors (and the padding) by Adam, then cast and gathered into
 * full_out. A matrix's exp_avg_sq is left alone. `tensors` lists the unit's
 * tensors in flat order: layout->n_tensors entries whose sizes add up to
 * layout->numel. g, m, p are fp32 as in the step; O's precision is that of
 * fsdp_newton_schulz. EINVAL: F != W, sizes that do not add up, non-finite
 * hyper-parameters, momentum outside [0, 1). EALIAS, EWORKSPACE as above. */
typedef struct {
  int64_t rows; /* matrix: rows x cols; other tensor: rows elements, cols = 0 */
  int64_t cols;
  double scale; /* matrix: factor of its update */
} fsdp_muon_tensor_t;

typedef struct {
  double lr;
  double momentum;
  double weight_decay;
  int32_t nesterov;
  const fsdp_newton_schulz_t *newton_schulz; /* null: the defaults */
  fsdp_adam_t adam;                          /* for the other tensors; its own lr and step */
} fsdp_muon_t;

typedef struct {
  const fsdp_layout_t *layout;
  const fsdp_muon_tensor_t *tensors;
  const uint16_t *const *grads; /* W device rows of padded_numel bf16 */
  float *const *master;         /* W device shards of S fp32, in place */
  float *const *exp_avg;
  float *const *exp_avg_sq;
  uint16_t *full_out; /* device bf16 [padded_numel] */
} fsdp_muon_unit_t;

int fsdp_muon_step(const fsdp_muon_unit_t *unit, const fsdp_muon_t *muon, void *workspace, int64_t workspace_bytes,
                   fsdp_stream_t stream);
int fsdp_muon_workspace(const fsdp_muon_unit_t *unit, const fsdp_muon_t *muon, int64_t *bytes_out);

/* ------------------------------------------------------------------------
 * Operators at a model's two ends and between its blocks: what a root unit's
 * tensors (embedding tables, the head) are used with. Matrices, workspaces,
 * EINVAL, EALIAS and EWORKSPACE as above.
 *
 * Indexes (tokens, targets) are contiguous 32- or 64-bit integers in device memory,
 * which the host does not read. A negative one stands for "none"; one that is not below
 * `vocab` is a mistake of the caller, and what depends on it becomes NaN. */

#define FSDP_DTYPE_I32 3
#define FSDP_DTYPE_I64 4

/* Embedding lookup: out_r = scale table[token_r] + addend_r, formed in fp32 and rounded
 * once. table, addend (null: none) and out have type `dtype` (F32 or BF16). A token
 * below 0 takes a row of zeros (the addend is still added), one from vocab on a row of
 * NaN. out may be addend in place. rows = 0 launches nothing. EINVAL: cols, vocab < 1; rows < 0;
 * any of them > 2^30; a stride below cols; a type or a scale (not finite as a float) outside
 * the above; a missing pointer, one not aligned to its elements. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t vocab; /* rows of the table */
  int64_t table_stride;
  int64_t addend_stride;
  int64_t out_stride;
  int32_t dtype;
  int32_t token_dtype; /* I32 or I64 */
  double scale;
} fsdp_embedding_t;

int fsdp_embedding(const fsdp_embedding_t *args, const void *tokens, const void *table, const void *addend, void *out,
                   fsdp_stream_t stream);

/* Its gradient: dtable_v = scale times the sum of dout_r over the rows r with token_r = v;
 * accumulate: added to what dtable_v holds (a tied table's other gradient), and the
 * rows that no token names are left as they are, unread; else these are set to zero.
 * Rows whose token is below 0, or not below vocab, take no part. Sums are fp32, in an order
 * fixed by the tokens; each element is rounded once. dtable has table_dtype, dout `dtype` (F32 or
 * BF16 each), and dtable may lie anywhere in a rank's bf16 gradient row. rows = 0 sets dtable to
 * zero unless accumulate. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t vocab;
  int64_t dout_stride;
  int64_t dtable_stride;
  int32_t dtype;
  int32_t table_dtype;
  int32_t token_dtype;
  int32_t accumulate;
  double scale;
} fsdp_embedding_backward_t;

int fsdp_embedding_backward(const fsdp_embedding_backward_t *args, const void *tokens, const void *dout, void *dtable,
                            void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);
int fsdp_embedding_backward_workspace(int64_t rows, int64_t cols, int64_t vocab, int64_t *bytes_out);

/* Dropout with the residual's addition: out = residual + (kept ? x k : 0), formed in
 * fp32 and rounded once, with t = round(65536 p), k = 65536 / (65536 - t). Which elements are
 * kept follows from seed, offset and the element's place alone: element i = row cols + column
 * has draw i mod 8 of Philox4x32-10 (Salmon et al., 2011) with the 64-bit key `seed` and the
 * counter (i / 8, offset + *counter), its four words taken as eight 16-bit draws, low half
 * first, and is kept where its draw is at least t. No mask is stored: the gradient of x is the same
 * call on out's gradient without a residual. Give each use (layer, step) an offset of its own.
 * counter (device, may be null: 0) is read when the kernel runs, so that a captured graph can be
 * replayed with new draws. A dropped element's x has no effect, be it NaN. x, residual (null:
 * none) and out have type `dtype` (F32 or BF16); out may be x or residual in place. rows = 0
 * launches nothing. EINVAL: p outside [0, 1), or rounded to 1 in 16 bits; sides > 2^40; as above. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t x_stride;
  int64_t residual_stride;
  int64_t out_stride;
  uint64_t seed;
  uint64_t offset;
  int32_t dtype;
  double p;
} fsdp_dropout_t;

int fsdp_dropout(const fsdp_dropout_t *args, const void *x, const void *residual, const uint64_t *counter, void *out,
                 fsdp_stream_t stream);

/* Softmax cross entropy of a projection onto a vocabulary, with its gradients:
 *   x = hidden weight^T,  lse_r = log sum_v exp(x_rv),  loss_r = lse_r - x_r,target_r
 *   G_rv = g_r (exp(x_rv - lse_r) - [v = target_r]),  g_r = scale dloss_r  (dloss null: scale)
 *   dhidden = G weight,  dweight = G^T hidden
 * hidden, weight, dhidden and dweight are bf16; dloss, loss and lse (may be null) fp32 [rows].
 * A loss is never below 0. dhidden and dweight are both given or both null (losses alone; dloss is
 * null then). A row with a target below 0 has loss 0 and takes no part in the gradients, whatever
 * its hidden row holds (its dhidden row is zero); its lse is that of its logits. One with a target
 * from vocab on gives NaN. dweight may lie anywhere in a rank's bf16 gradient row; dhidden may be
 * hidden in place. The products take bf16 operands on the tensor cores and sum in fp32 (logits in
 * segments of 1024 columns, 256 up to 128 rows). The fp32 logits are not stored: losses alone keep
 * nothing of them, the gradients exp(x) rounded to bf16 in the workspace, of `piece` rows at a time
 * (0: as many as keep that below 1 GiB, at least 256; at most 2^20); dweight's sum over several
 * pieces is fp32 in the workspace. hidden's rows times their factors are rounded to bf16 for
 * dweight. Together with the results' own rounding the gradients are typically within 0.0023 of their norm.
 * Factors g_r are 0 or between 1e-18 and 1e18 (beyond, a row's gradients may be cut to zero or
 * infinite). The workspace always has room for a copy of the weight and of a piece's hidden rows (2
 * vocab cols bytes and more, with cols rounded up to 64, for losses alone too), made where one lies
 * off 16 bytes. Rows whose |lse|, or the largest logit of some 128 columns of the vocabulary, is
 * beyond 40 (all of them where the logits are not centred) take one more pass over what is kept,
 * which rounds nothing again: 8192 of them through a 50257 x 768 head take 1.5 ms in place of 1.2,
 * 4096 through 32000 x 4096 2.06 ms in place of 1.92, 64 through 50257 x 768 0.14 to 0.17 ms in
 * place of 0.06; losses alone take no longer. rows = 0 sets dweight to zero. EINVAL: cols > 2^24,
 * vocab > 2^30, rows > 2^40, piece < 0; a scale that is not finite as a float; as above. */
typedef struct {
  int64_t rows;
  int64_t cols;
  int64_t vocab; /* rows of the weight */
  int64_t hidden_stride;
  int64_t weight_stride;
  int64_t dhidden_stride;
  int64_t dweight_stride;
  int64_t piece;
  int32_t target_dtype; /* I32 or I64 */
  double scale;
} fsdp_cross_entropy_t;

int fsdp_cross_entropy(const fsdp_cross_entropy_t *args, const uint16_t *hidden, const uint16_t *weight,
                       const void *targets, const float *dloss, float *loss, float *lse, uint16_t *dhidden,
                       uint16_t *dweight, void *workspace, int64_t workspace_bytes, fsdp_stream_t stream);
/* Of the same args (their sizes and piece); gradients: whether dhidden and dweight will be given. */
int fsdp_cross_entropy_workspace(const fsdp_cross_entropy_t *args, int32_t gradients, int64_t *bytes_out);

/* Text of a status code (static storage). */
const char *fsdp_status_string(int status);

#ifdef __cplusplus
}
#endif

#endif /* FSDP_GB300_H */
