/*
 * zero_b200.h -- C ABI of libzero_b200: the ZeRO-DP sharded mixed-precision
 * optimizer step on one GPU (sm_103a), with Nd data-parallel ranks emulated in
 * that GPU's own memory.
 *
 * Pages cited (title as printed; section numbers are each page's own):
 *   [L18]  "第 18 讲 · Memory Optimization in Distributed Training: ZeRO"
 *   [Z026] "026｜ZeRO：数据并行中，没必要让每张卡保存全部训练状态"
 *   [L32]  "L3.2 显存优化与 ZeRO"
 *   [ZL8]  "图解分布式训练（八）—— ZeRO 学习"
 *   [PZ]   "ZeRO:" (ZeRO paper digest)
 *
 * One step, per element of the flat parameter vector ([L18] 2.2-2.4):
 *   (1) reduce-scatter: the Nd ranks' 16-bit local gradients are summed in
 *       fixed rank order (0..Nd-1, fp32, from 0.0f) and divided by Nd
 *       ([L18] 2.2, 2.5; [PZ] 5.2);
 *   (2) unscale by the loss scale; any inf/NaN sets the overflow flag, which
 *       under dynamic loss scaling skips the step and halves the scale
 *       ([L32] 4.3), and under a static scale skips it when the caller asks
 *       (zero_hparams_t.skip_on_overflow);
 *   (3) global gradient norm over every shard and clip-by-norm
 *       ([L32] 4.2 "gradient_clipping");
 *   (4) Adam / AdamW with bias correction on each shard's fp32 master, m, v
 *       ([L18] 2.1-2.2: Adam is elementwise, a rank needs only its slice);
 *   (5) cast to fp16/bf16 ([L18] 2.2);
 *   (6) all-gather of the 16-bit parameters: for ZeRO-1/2 every shard writes
 *       into one flat full-parameter buffer ([L18] 2.2; [L32] 2.3); for
 *       ZeRO-3 zero_gather_layer assembles one unit from its Nd slices
 *       ([L18] 2.4, 3.3; [ZL8] 8.4).
 *
 * Conventions for every entry point:
 *   - Errors: every call returns a zero_status_t and never aborts; arguments
 *     are validated before anything is launched.  CUDA failures return
 *     ZERO_ECUDA.  A skipped step is not an error.
 *   - Ownership: the caller allocates and owns every device buffer and the
 *     stream; the library borrows raw device pointers for the duration of a
 *     call.  A plan owns only its host bookkeeping and a small device block
 *     (optimizer scalars, step status, per-block partials: about 100 KB,
 *     allocated by zero_plan_create on the current device).
 *   - Device pointers must be 16-byte aligned.  Streams are cudaStream_t
 *     passed as void* (NULL = the legacy default stream).
 *   - Steps of one plan must be ordered (same stream, or ordered by events):
 *     they share the plan's device block.
 */
#ifndef ZERO_B200_H
#define ZERO_B200_H

#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef struct zero_plan* zero_plan_t;

/* Every entry point reports through its return value and never throws: a C++
 * exception inside the library (a host allocation or a worker thread that
 * cannot be had) comes back as ZERO_ENOMEM, or ZERO_EIO inside checkpoint IO. */
typedef enum {
    ZERO_OK       = 0,
    ZERO_EINVAL   = 1,   /* an argument is out of range, null or misaligned   */
    ZERO_ENOMEM   = 2,   /* host or device allocation failed                  */
    ZERO_ECUDA    = 3,   /* a CUDA call or kernel launch failed                */
    ZERO_ETIMEOUT = 4,   /* a bounded device-side wait gave up                 */
    ZERO_ENOENT   = 5,   /* a checkpoint file is missing or cannot be opened   */
    ZERO_ECORRUPT = 6,   /* a checkpoint file is truncated, fails a checksum,
                            or does not belong with the other files           */
    ZERO_EIO      = 7,   /* reading, writing or flushing a file failed         */
    ZERO_ESTATE   = 8    /* a failed checkpoint load left the plan's state
                            incomplete; steps are refused until a load succeeds */
} zero_status_t;

/* ZERO_FP32 is accepted only where an entry point says so. */
typedef enum { ZERO_FP16 = 0, ZERO_BF16 = 1, ZERO_FP32 = 2 } zero_dtype_t;

/* Optimizer and mixed-precision settings ([L32] 3.2 and 4.2 DeepSpeed config:
 * optimizer lr, fp16 loss scaling, gradient_clipping).
 *   lr, beta1, beta2, eps    Adam; bias-corrected with 1 - beta^t.
 *   weight_decay             0 = none.  decoupled_wd = 1: AdamW, the master is
 *                            multiplied by (1 - lr wd) before the update;
 *                            0: L2, wd * master is added to the gradient.
 *   clip_norm                clip by global norm; 0 = off.
 *   loss_scale               initial loss scale S (the gradients arrive
 *                            multiplied by S); 1 = none.
 *   dynamic_scale            1: an overflow skips the step (state untouched,
 *                            t unchanged) and multiplies S by backoff; after
 *                            growth_interval good steps in a row S doubles
 *                            (growth_interval <= 0: never).  Requires fp16.
 *                            0: static S (see skip_on_overflow).
 *   skip_on_overflow         with a static S: 1 = an overflow skips the step
 *                            (state untouched, t and S unchanged); 0 = the
 *                            flag is reported and the step goes ahead.
 *                            Ignored under dynamic_scale (which always skips).
 *
 * Overflow under a static scale (dynamic_scale 0, skip_on_overflow 0): the
 * skip belongs to loss scaling ([L32] 4.3 ties a NaN loss to the fp16
 * loss_scale setting), and a step that nothing global gates is what lets the
 * update run as one fused pass over the data.  The consequences of a non-finite
 * averaged gradient element i in such a step:
 *   - without clipping, only element i is affected: its master, m and v
 *     become NaN (or inf) and stay so; every other element is updated exactly
 *     as if element i's gradient had been finite;
 *   - with clipping, the norm is inf, the clip coefficient tau/inf = 0, so
 *     every finite element takes a zero-gradient step (m *= beta1,
 *     v *= beta2, the master moves by the remaining momentum) and element i
 *     becomes NaN (inf * 0).
 * A caller who wants such steps dropped sets skip_on_overflow = 1; the plan
 * then runs two passes (the flag must be known before any update), which
 * costs the fp32 gradient's write and read (8 bytes per element) on the
 * paths that would otherwise fuse. */
typedef struct {
    float lr, beta1, beta2, eps, weight_decay;
    int   decoupled_wd;
    float clip_norm;
    float loss_scale;
    int   dynamic_scale;
    float backoff;
    int   growth_interval;
    int   skip_on_overflow;
} zero_hparams_t;

/* ---- plans ------------------------------------------------------------ */

/* Largest psi a plan accepts (2^48 elements): far above any GPU's memory, and
 * small enough that every element index times nd fits the kernels' 64-bit
 * arithmetic. */
#define ZERO_MAX_PSI (1ull << 48)

/* Create a plan for a model of psi parameters made of ntensors tensors whose
 * shapes are given in list order: tensor i has ndims[i] dimensions, taken in
 * order from dims.  psi must equal the sum of the tensor sizes.
 * nd: emulated data-parallel ranks (1..1024).  stage: 0 = plain DP, 1, 2, 3.
 * dtype: format of the gradients and of the 16-bit parameters.
 * Layout ([L18] 3.2 flat partition; [ZL8] 8.4):
 *   stages 0-2: all tensors flattened into one vector and split into nd equal
 *     contiguous shards of S = ceil(psi/nd) rounded up to 64 elements; rank r
 *     owns [r S, (r+1) S); the flat length is nd S (the tail is padding).
 *   stage 3: each ZeRO-3 unit (here: one unit per tensor; see
 *     zero_plan_create_units) is flattened and split into nd slices of
 *     S_u = ceil(len_u/nd) rounded up to 64; a rank's shard is the
 *     concatenation of its slice of every unit in unit order.
 * The plan copies everything it needs; dims/ndims/hp may be freed afterwards.
 * Allocates the plan's device block on the current device.
 * Errors: ZERO_EINVAL (bad sizes, psi mismatch, psi > ZERO_MAX_PSI,
 * dynamic_scale with bf16, nd or stage out of range), ZERO_ENOMEM, ZERO_ECUDA. */
zero_status_t zero_plan_create(uint64_t psi, int nd, int stage, zero_dtype_t dtype,
                               const int64_t* dims, const int* ndims, int ntensors,
                               const zero_hparams_t* hp, zero_plan_t* out);

/* As zero_plan_create, with the ZeRO-3 unit of each tensor given explicitly:
 * unit_of_tensor[i] is tensor i's unit; units are numbered 0..U-1 in the
 * order their tensors appear and each unit's tensors are contiguous in the
 * list (e.g. embedding, one unit per transformer layer, final norm + head:
 * [L18] 3.3 the FSDP unit is usually one Transformer layer).  Ignored for
 * stages 0-2. */
zero_status_t zero_plan_create_units(uint64_t psi, int nd, int stage, zero_dtype_t dtype,
                                     const int64_t* dims, const int* ndims, int ntensors,
                                     const int* unit_of_tensor, const zero_hparams_t* hp,
                                     zero_plan_t* out);

/* Free the plan and its device block.  NULL is accepted. */
zero_status_t zero_plan_destroy(zero_plan_t plan);

/* Layout of the buffers zero_step expects (any output pointer may be NULL):
 *   shard_elems     S (stages 0-2), or the length of one rank's shard (stage 3)
 *   padded_elems    stages 0-2: nd * S, the flat parameter/state length;
 *                   stage 3: one rank's shard length (= shard_elems)
 *   nunits          ZeRO-3 units (stage 3), else 0
 *   workspace_bytes device scratch zero_step needs (0 when none). */
zero_status_t zero_plan_layout(zero_plan_t plan, uint64_t* shard_elems, uint64_t* padded_elems,
                               int* nunits, uint64_t* workspace_bytes);

/* Stage 3: unit u's length, slice length S_u and the slice's offset inside a
 * rank's shard. */
zero_status_t zero_plan_unit(zero_plan_t plan, int unit, uint64_t* len, uint64_t* slice_elems,
                             uint64_t* offset);

/* ---- the step ----------------------------------------------------------- */

/* One optimizer step, asynchronous on `stream` (no host synchronisation).
 * Stages 0-2 (every emulated rank's shard is updated):
 *   grads      [nd][nd*S] 16-bit: rank r's full local gradient at
 *              grads + r*nd*S; elements at flat index >= psi are ignored.
 *   master,m,v [nd*S] fp32, updated in place (elements >= psi untouched).
 *   params     [nd*S] 16-bit flat full-parameter buffer: every shard's updated
 *              parameters are written at their flat offset (the all-gather
 *              write-back); elements >= psi untouched.
 * Stage 3 (one rank's shard is resident):
 *   grads      [nd][L] 16-bit, L = that rank's shard length: the nd ranks'
 *              contributions to that shard;
 *   master,m,v,params [L] that rank's shard.  The overflow flag and the norm
 *              cover the resident shard (the scalar all-reduce over ranks has
 *              a single participant here).
 * workspace: zero_plan_layout's workspace_bytes of device scratch (NULL when 0).
 * grads may also lie in page-locked host memory that the device can address
 * (cudaHostAlloc, or cudaHostRegister; under unified addressing the host address
 * is the device address): the passes then read it in place over the host link,
 * with the same results; the caller must not rewrite it before the step is done
 * (zero_step_result waits for it).  Every other buffer is device memory.
 * On a skipped step nothing but the plan's loss scale changes.
 * Errors: ZERO_EINVAL (null or misaligned pointer), ZERO_ECUDA. */
zero_status_t zero_step(zero_plan_t plan, const void* grads, float* master, float* m, float* v,
                        void* params, void* workspace, void* stream);

/* Wait for the plan's last step and report it (any pointer may be NULL):
 * skipped (1 if the overflow skipped it), grad_norm (global L2 norm of the
 * unscaled averaged gradient, before clipping), clip_coef (the factor applied,
 * 1 when not clipped), loss_scale (the scale the next step uses), t (completed
 * steps).  Before any step: skipped 0, grad_norm 0, clip_coef 1, the initial
 * loss scale and t = 0.  Errors: ZERO_EINVAL (null plan), ZERO_ECUDA. */
zero_status_t zero_step_result(zero_plan_t plan, int* skipped, double* grad_norm,
                               float* clip_coef, float* loss_scale, int64_t* t);

/* The overflow flag of the plan's last step (1 if any gradient element was
 * inf/NaN after unscaling); waits like zero_step_result. */
zero_status_t zero_step_overflow(zero_plan_t plan, int* overflow);

/* ---- ZeRO-3 gather ------------------------------------------------------ */

/* Assemble unit `unit` of a stage-3 plan ([L18] 2.4: the owners send their
 * pieces before the unit is used; [ZL8] 8.4: one contiguous buffer per
 * module).  shard_ptrs[k] (k < nd, host array of device pointers) is rank k's
 * whole 16-bit parameter shard; out receives the unit's len elements:
 * out[k*S_u + j] = shard_k[off_u + j] for k*S_u + j < len.  Asynchronous.
 * Errors: ZERO_EINVAL (not stage 3, unit out of range, null or misaligned
 * pointer), ZERO_ECUDA. */
zero_status_t zero_gather_layer(zero_plan_t plan, int unit, const void* const* shard_ptrs,
                                void* out, void* stream);

/* ---- constant-size gradient buckets ------------------------------------------ */

/* [L18] 2.3 (ZeRO-2: as soon as the backward pass has a segment's gradients they
 * are reduced to the segment's owner and dropped, so each rank keeps only a
 * buffer for the segment in flight; the segment reduces together are one
 * reduce-scatter) and [L18] 4.3 / [PZ] 6.2 (a constant-size buffer worked
 * through piece by piece instead of one flat buffer that grows with the model).
 * A bucketed step takes the ranks' gradients bucket by bucket: bucket b covers
 * elements [b*B, min((b+1)*B, n)) of the flat vector (stage 3: of the resident
 * shard), B = bucket_elems (a multiple of 64).
 *   zero_plan_set_bucket   turns bucketed steps on (B > 0) or off (B = 0) and
 *                          reports the workspace they need: the fp32 reduced
 *                          gradient (n floats) plus one norm partial and one
 *                          flag per block of each bucket's reduce.  Waits for
 *                          the plan's last step.
 *   zero_step_bucket       reduces bucket b: bucket_grads is [nd][B] 16-bit
 *                          (rank stride B; a short last bucket uses its first
 *                          count columns); buckets may come in any order, each
 *                          exactly once per step (ZERO_EINVAL otherwise); the
 *                          bucket buffer may be reused once this call's work
 *                          on `stream` is done.
 *   zero_step_apply        after every bucket: the global norm from the bucket
 *                          reduces' block partials (summed in bucket, then
 *                          block, order), clip, skip decision, Adam, cast,
 *                          write-back; ZERO_EINVAL if a bucket is missing.
 *                          zero_step_result reports it.
 * Reduced gradients are bit-identical to zero_step's; the norm agrees to
 * 1e-5 (its partial sums are grouped by bucket).  Calls of one plan must be
 * ordered on one stream. */
zero_status_t zero_plan_set_bucket(zero_plan_t plan, uint64_t bucket_elems,
                                   uint64_t* workspace_bytes);
zero_status_t zero_step_bucket(zero_plan_t plan, uint64_t bucket, const void* bucket_grads,
                               void* workspace, void* stream);
zero_status_t zero_step_apply(zero_plan_t plan, float* master, float* m, float* v, void* params,
                              void* workspace, void* stream);

/* ---- ZeRO++ quantized weight gather (qwZ) ---------------------------------- */

/* [L18] 4.5 ZeRO++: the parameters a ZeRO-3 gather moves are quantized block
 * by block, one scale per block, so a few large weights coarsen only their own
 * block.  A rank's 16-bit shard of n elements is cut into blocks of 256
 * elements counted from the shard's start; for each block
 *   scale = max|x| / qmax  (qmax = 127 for bits = 8, 7 for bits = 4; binary32)
 *   code  = round_half_even(x / scale) clamped to [-qmax, qmax]; 0 if scale = 0.
 * codes: n bytes (bits 8, two's complement) or ceil(n/2) bytes (bits 4, two
 * codes per byte, the even element in the low nibble), 16-byte aligned;
 * scales: ceil(n/256) floats.  Asynchronous.  Errors: ZERO_EINVAL, ZERO_ECUDA. */
zero_status_t zero_quantize_shard(zero_dtype_t dtype, const void* shard, uint64_t n, int bits,
                                  void* codes, float* scales, void* stream);

/* The ZeRO-3 gather of unit `unit` from the nd ranks' quantized shards
 * (code_ptrs[k], scale_ptrs[k]: rank k's whole-shard codes and scales, as
 * zero_quantize_shard writes them): out[k*S_u + j] = 16-bit rounding of
 * code_k[off_u + j] * scale_k[(off_u + j) / 256] for k*S_u + j < len.  Moves
 * 1 (bits 8) or 0.5 (bits 4) bytes per element in instead of 2.  Errors:
 * ZERO_EINVAL (not stage 3, unit or bits out of range, null or misaligned
 * pointer), ZERO_ECUDA. */
zero_status_t zero_gather_layer_q(zero_plan_t plan, int unit, int bits,
                                  const void* const* code_ptrs, const float* const* scale_ptrs,
                                  void* out, void* stream);

/* One ZeRO-3 optimizer step (exactly zero_step's, same arguments) whose update
 * pass also quantizes the resident shard's updated 16-bit parameters for the
 * qwZ gather ([L18] 4.5): codes and scales receive what
 * zero_quantize_shard(dtype, params, L, bits, codes, scales) would write after
 * the step, L being the shard length, but the parameters are quantized from
 * the update's registers as they are written instead of being read back
 * (2 bytes per element and one launch saved).  On a skipped step the
 * unchanged parameters are quantized, so the codes are valid whatever the
 * buffers held.  codes: L bytes (bits 8) or L/2 bytes (bits 4), 16-byte
 * aligned; scales: ceil(L/256) floats.  Asynchronous.  Errors: ZERO_EINVAL
 * (not stage 3, bits not 4 or 8, null or misaligned pointer), ZERO_ESTATE,
 * ZERO_ECUDA. */
zero_status_t zero_step_qwz(zero_plan_t plan, const void* grads, float* master, float* m, float* v,
                            void* params, void* workspace, int bits, void* codes, float* scales,
                            void* stream);

/* ---- ping-pong step ------------------------------------------------------- */

/* One optimizer step as a single pass over the data even when an overflow may
 * skip it (dynamic loss scaling or skip_on_overflow, without a clip): the
 * caller keeps two sets of master, m, v; the step reads the current set and
 * writes the other, and only a step that is not skipped makes the other set
 * current, so a skipped step leaves the current state untouched without having
 * to know the overflow before the update.  The 16-bit parameters are written by
 * the pass; when the step is skipped, a small pass after it rewrites them from
 * the current set's master (4 + 2 bytes per element, on skipped steps only).
 * The arithmetic is zero_step's: the same state, parameters and report.
 *   set 0: master0, m0, v0; set 1: master1, m1, v1; each laid out as zero_step's
 *          master, m, v (stages 0-2: [nd*S]; stage 3: the resident shard).
 *   grads, params: as zero_step.
 * zero_plan_state_set reports which set is current after the plan's last step
 * (waiting for it): 0 after zero_plan_create and after zero_checkpoint_load
 * (load a checkpoint into set 0); checkpoint the current set.  A plan may mix
 * zero_step and zero_step_pingpong only if the caller passes the current set
 * to zero_step.  Asynchronous.  Errors: ZERO_EINVAL (clip_norm > 0, null or
 * misaligned pointer), ZERO_ESTATE, ZERO_ECUDA. */
zero_status_t zero_step_pingpong(zero_plan_t plan, const void* grads, float* master0, float* m0,
                                 float* v0, float* master1, float* m1, float* v1, void* params,
                                 void* stream);
zero_status_t zero_plan_state_set(zero_plan_t plan, int* set);

/* ---- gradient norm without allocating ------------------------------------ */

/* No counterpart on the pages: a convenience for callers that may not
 * allocate device memory (code running under another framework's memory pool
 * or allocator hooks, or code that only holds pre-allocated buffers and so
 * cannot create a plan, whose creation allocates).
 * Computes what zero_step's reduce pass reports: the global L2 norm of the
 * averaged, unscaled gradient g_i = (sum_r grads[r][i] / nd) / loss_scale (the
 * sum in rank order, fp32) and whether any g_i is inf/NaN.
 *   grads        [nd][rank_stride] 16-bit device array, 16-byte aligned; the
 *                first n elements of each rank's row are used.
 *   rank_stride  >= n, a multiple of 8.
 *   norm_out     device pointer to one double (8-byte aligned): the norm.
 *   overflow_out device pointer to one int: 1 if any g_i is inf/NaN, else 0.
 * Asynchronous on `stream`.  Allocates nothing: its scratch (one partial per
 * 2^17-element tile plus a counter, 196,864 bytes) is a fixed device array in
 * the library that every GPU loading the library keeps until process exit;
 * hence n is limited to 2^31 elements (ZERO_EINVAL beyond).  The first call on
 * a device looks up that array's device address (cudaGetSymbolAddress) and
 * keeps it per device context: after the device's primary context is reset
 * (cudaDeviceReset), the next call looks it up again.  Every call shares
 * the array, so calls whose executions overlap on the GPU (e.g. on two
 * concurrent streams) race and give wrong results; order them.  The norm
 * agrees with zero_step's within 1e-5 relative (the partial sums are grouped
 * differently); the flag is identical.
 * Errors: ZERO_EINVAL (sizes, alignment, null output), ZERO_ECUDA. */
zero_status_t zero_grad_norm_noalloc(const void* grads, int nd, uint64_t n, uint64_t rank_stride,
                                     zero_dtype_t dtype, float loss_scale, double* norm_out,
                                     int* overflow_out, void* stream);

/* ---- sharded checkpoint ------------------------------------------------------ */
/* [Z026] sec. 5: with the state sharded, each rank holds only its part of the
 * weights and optimizer state; a restore at another degree of parallelism
 * must regroup ownership while keeping the parameter order and each
 * element's moments together, and a rank's missing file must make the
 * restore fail explicitly rather than produce an incomplete model.
 * [L32] sec. 4.3: a resumable checkpoint holds the sharded optimizer state,
 * not the weights alone.
 *
 * A checkpoint is a directory holding manifest.zck and one file per rank of
 * the saving plan, shard_<rank>_of_<nd>.zck (5-digit decimal, zero-padded).
 * Each rank file holds, for the flat elements that rank owns (padding
 * excluded): master, m and v (fp32) and the 16-bit parameters.  The file
 * records those elements as segments [global_start, global_start + count) of
 * the flat parameter vector, so a checkpoint does not depend on the saving
 * plan's rank count or stage: a plan of any nd and stage over the same tensor
 * list can load it, each of its ranks taking the elements it owns.
 *
 * Format (all integers little-endian):
 *   manifest.zck, 88 bytes: "ZEROMAN1", u32 version (1), u32 size (88),
 *     u64 psi, i32 nd, i32 stage, i32 dtype, i32 0, u64 model_hash,
 *     scalars (32 bytes: f32 loss_scale, i32 good_steps, i64 t, f64 beta1^t,
 *     f64 beta2^t), u64 zck64 of bytes 0..79.
 *   shard file: a 4096-byte header: "ZEROSHD1", u32 version (1),
 *     u32 4096, u64 psi, i32 nd, i32 stage, i32 dtype, i32 rank,
 *     u64 model_hash, scalars (32 bytes, as above), u64 nseg, u64 n (elements
 *     held = sum of the segment counts), u64 block_elems (2^20), u64 nblocks
 *     (ceil(n / block_elems)), u64 table_offset (4096), u64 array_offset[4]
 *     (master, m, v, params), u64 file_bytes, u64 meta_hash; zeros up to 4096.
 *     At table_offset: nseg pairs {u64 global_start, u64 count} in shard
 *     order, then 4 x nblocks u64 block checksums (array a, block b at
 *     a * nblocks + b).  Each array holds its n values in segment order and
 *     starts on a 4096-byte boundary.  meta_hash = zck64 of header bytes
 *     0..159 plus zck64 of the table, mod 2^64.
 *   zck64 of a byte string whose first 8-byte word has index w0 within its
 *     array: the sum mod 2^64, over its 8-byte words x_i (the last one
 *     zero-padded), of mix(x_i + (w0 + i + 1) * 0x9E3779B97F4A7C15), where
 *     mix is the SplitMix64 finaliser (z ^= z >> 30; z *= 0xBF58476D1CE4E5B9;
 *     z ^= z >> 27; z *= 0x94D049BB133111EB; z ^= z >> 31).  Block b of an
 *     array covers elements [b * 2^20, min((b + 1) * 2^20, n)), w0 = its byte
 *     offset / 8.
 *   model_hash: FNV-1a 64 over the little-endian bytes of the int64 values
 *     ntensors, then for each tensor its ndims and its dims.
 */

/* flags of zero_checkpoint_save */
#define ZERO_CKPT_FSYNC      1   /* flush every file and the directory to storage  */
#define ZERO_CKPT_DROP_CACHE 2   /* with FSYNC: then drop the files' cached pages  */

/* Save rank `rank`'s state, or every rank's (rank = -1; stages 0-2 only).
 * Buffers: as zero_step.  Stages 0-2: the flat [nd*S] master, m, v, params;
 * stage 3: rank `rank`'s resident shard.  Writes shard_<rank>_of_<nd>.zck
 * (through a temporary name, renamed when complete) for each rank saved, and
 * manifest.zck when rank is 0 or -1, creating `dir` if it does not exist.
 * The scalars (loss scale, good steps, t, beta powers) are the plan's after
 * its last step.  Synchronous: waits for `stream` and the plan's last step,
 * returns when the files are written.  Host staging is pinned memory the plan
 * keeps until it is destroyed.
 * Errors: ZERO_EINVAL (null, misaligned or out-of-range argument), ZERO_EIO
 * (a file could not be created, written or flushed; no partial file is left
 * under the final name), ZERO_ENOMEM, ZERO_ECUDA. */
zero_status_t zero_checkpoint_save(zero_plan_t plan, const char* dir, int rank,
                                   const float* master, const float* m, const float* v,
                                   const void* params, int flags, void* stream);

/* Load rank `rank`'s state, or every rank's (rank = -1; stages 0-2 only), from
 * the checkpoint in `dir`, whatever rank count and stage saved it; the
 * elements of the plan's layout past each unit's or the model's end are set
 * to zero.  Buffers: as zero_checkpoint_save.  On success the plan's scalars
 * are the checkpoint's and its last-step report is reset.  Synchronous.
 * Checks, before any device memory is written: the manifest and every one of
 * the saving plan's rank files exist (ZERO_ENOENT), their headers are intact
 * and agree with each other, their segments cover the flat vector exactly once
 * (ZERO_ECORRUPT), and the model is the plan's: same psi, tensor shape list
 * and 16-bit type (ZERO_EINVAL); the buffers are then untouched.  Every data
 * block read is checked against its checksum; a mismatch or read error after
 * device writes began returns ZERO_ECORRUPT or ZERO_EIO and leaves the plan
 * refusing steps and gathers (ZERO_ESTATE) until a load succeeds.
 * Other errors: ZERO_ENOMEM, ZERO_ECUDA. */
zero_status_t zero_checkpoint_load(zero_plan_t plan, const char* dir, int rank, float* master,
                                   float* m, float* v, void* params, void* stream);

/* ---- ZeRO-Offload: the Adam update on the host ------------------------------- */
/* [L18] sec. 4.4: the device keeps the 16-bit parameters and gradients; the
 * host keeps the fp32 master, m and v and runs Adam, multithreaded and
 * vectorised; each step copies the 16-bit gradients to the host (2 psi bytes)
 * and the updated 16-bit parameters back (2 psi).  [ZL8] sec. 6.2, 7: the
 * device runs forward and backward, the host the parameter update. */

/* One offloaded step of a stages 0-2 plan.  On the device: the rank-order fp32
 * fold of the nd contributions divided by nd, rounded to the plan's 16-bit
 * type (the copied value; written to `workspace`), the overflow flag and the
 * global norm of that value divided by the loss scale, and the step's
 * scalars (skip, clip coefficient, loss-scale update, t, bias corrections), as
 * zero_step.  On the host, unless the step is skipped: g = copied value / S,
 * times the clip coefficient, then Adam/AdamW on master, m, v exactly as
 * zero_step's update, and the 16-bit parameters copied to `params`.
 *   grads      device [nd][nd*S] 16-bit, as zero_step.
 *   master,m,v HOST fp32 arrays of at least psi elements (elements >= psi
 *              untouched); pageable or pinned.
 *   params     device [nd*S] 16-bit flat parameters (elements >= psi untouched).
 *   workspace  device scratch of at least 2*psi bytes, 16-byte aligned.
 *   nthreads   host threads (<= 0: one per hardware thread).
 * The copies stream through the plan's pinned staging in 2^24-element chunks
 * overlapped with the host arithmetic.  Synchronous: returns when the
 * parameters are on the device.  zero_step_result reports the step.
 * Errors: ZERO_EINVAL (stage 3, null or misaligned pointer), ZERO_ESTATE,
 * ZERO_ENOMEM, ZERO_ECUDA. */
zero_status_t zero_offload_step(zero_plan_t plan, const void* grads, float* master, float* m,
                                float* v, void* params, void* workspace, int nthreads,
                                void* stream);

/* The host Adam alone, on host memory: for i < n, g = grads16[i] (the 16-bit
 * type `dtype`) / loss_scale * clip_coef, then Adam/AdamW with the bias
 * corrections bc1 = 1 - beta1^t and bc2 = 1 - beta2^t of this step, each
 * operation one binary32 rounding in the order of zero_step's update; master,
 * m, v updated in place, params16[i] = master[i] rounded to the 16-bit type.
 * nthreads <= 0: one thread per hardware thread.  Needs no GPU.
 * Errors: ZERO_EINVAL (null pointer, dtype, loss_scale/bc1/bc2 not > 0),
 * ZERO_ENOMEM. */
zero_status_t zero_cpu_adam(const void* grads16, zero_dtype_t dtype, uint64_t n, float loss_scale,
                            float clip_coef, float bc1, float bc2, const zero_hparams_t* hp,
                            float* master, float* m, float* v, void* params16, int nthreads);

/* ---- 8-bit activation checkpoints -------------------------------------------- */

/* [L18] part 4 and [PZ] part 6 name the activations kept for the backward pass as
 * the next memory after the sharded model state (checkpointing them, and
 * partitioning the checkpoints over ranks).  These calls keep an activation
 * matrix in 8 bits per element and use it in the backward pass without first
 * expanding it; the gradients they produce go straight into a rank's row of
 * zero_step's gradients.  The pages fix no format; this is the library's own:
 *
 *   A matrix of `cols` columns is stored row by row, zero_act_row_bytes(cols)
 *   bytes apart: with C = cols rounded up to 32, C code bytes (two's complement,
 *   |code| <= 127, 0 past cols), then C/32 exponent bytes, then zeros up to a
 *   multiple of 32 bytes.  Codes and exponent E of a block of 32 consecutive
 *   columns stand for code * 2^(E - 127).  E is the smallest exponent with
 *   max|x| <= 127 * 2^(E - 127), kept in [103, 136] for fp16 and [1, 248] for
 *   bf16 and fp32 inputs; code = round_half_even(x * 2^(127 - E)), clamped to
 *   +-127.  A block that holds an inf or a NaN has E = 255 and zero codes and
 *   reads back as NaN in all its columns (so the overflow flag of the step that
 *   receives the gradients is raised).
 * The scale is a power of two so that the value of a code is exact in the 16-bit
 * type: what a tensor core multiplies is the checkpoint's value itself.
 * Rows are independent: a range of rows of a checkpoint is a checkpoint. */

/* Most columns of a checkpointed matrix. */
#define ZERO_ACT_MAX_COLS (1ll << 24)

/* Bytes from one row of a checkpoint to the next (a matrix takes rows times
 * that); 0 if cols < 1 or cols > ZERO_ACT_MAX_COLS. */
uint64_t zero_act_row_bytes(int64_t cols);

/* Checkpoint x (dtype fp16, bf16 or fp32; rows ld elements apart, aligned to its
 * element; 16-byte aligned rows are read fastest).  Asynchronous.  rows = 0 is
 * accepted.  Errors: ZERO_EINVAL (dtype, sizes: rows in [0, 2^31), ld >= cols;
 * null or misaligned pointer), ZERO_ECUDA. */
zero_status_t zero_act_save(zero_dtype_t dtype, const void* x, int64_t rows, int64_t cols,
                            int64_t ld, void* ckpt, void* stream);

/* The values of a checkpoint, rounded to dtype (exact when dtype is the type that
 * was saved, or fp32), into out (rows ld elements apart, aligned to its element).
 * Asynchronous.  Errors: as zero_act_save. */
zero_status_t zero_act_load(zero_dtype_t dtype, const void* ckpt, int64_t rows, int64_t cols,
                            void* out, int64_t ld, void* stream);

/* The gradient of a linear layer's weight from the gradient of its output and
 * the checkpoint of its input.  With xh the checkpoint's values [tokens][k],
 *   dw[i][j] = sum_t dy[t][i] * (xh[t][j] * col_scale[j] + col_shift[j])
 *   db[i]    = sum_t dy[t][i]
 * summed in fp32: on the tensor cores, whose accumulators cut a sum off at each
 * step of 16 tokens, over at most 65536 tokens (fp32 gradients: 960), and by
 * rounded additions beyond.  col_scale and col_shift (dtype, [k]; NULL: 1 and 0) are the
 * weight and bias of a norm whose normalised rows were checkpointed, so one
 * checkpoint serves the norm's backward pass and every layer it feeds.
 *   dtype       fp16 or bf16: dy, col_scale, col_shift.  An fp16 dy needs a
 *               checkpoint saved as fp16 (block exponents outside fp16's range
 *               read as NaN).
 *   dy          [tokens] rows of n elements, ldy apart.
 *   grad_dtype  of dw and db: dtype, or fp32.
 *   dw          [n] rows of k elements, ldw apart (e.g. a tensor's place in a
 *               rank's gradient row); db [n], NULL: not wanted.
 *   accumulate  1: the sums are added to what dw and db hold (one rounding);
 *               0: overwritten.
 *   work        zero_act_wgrad_workspace(tokens, n, k) bytes, 16-byte aligned.
 *               The caller zeroes it once, before the first use (with any sizes);
 *               every call leaves it ready for the next.  Calls whose executions
 *               overlap need a workspace each.
 * Matrices need the alignment of their element; dy rows that are not 16-byte
 * aligned are first copied to the workspace (which always has room for that: 2
 * bytes a value of dy), 16-byte aligned dw rows are written in vectors.  tokens = 0
 * is accepted (the sums are zero).  Sums are taken in a fixed order: equal inputs
 * give equal bits.  Asynchronous.  A bounded device
 * wait that gives up (none should) sets the first int32 of `work` to
 * ZERO_ETIMEOUT and writes NaN where the sums are missing.
 * Errors: ZERO_EINVAL (types, sizes: tokens in [0, 2^31), n in [1, 2^24], k in
 * [1, ZERO_ACT_MAX_COLS], n k < 2^46, n <= ldy <= 2^31, k <= ldw <= 2^31; null or
 * misaligned pointer),
 * ZERO_ECUDA. */
zero_status_t zero_act_wgrad(zero_dtype_t dtype, const void* dy, int64_t tokens, int64_t n,
                             int64_t ldy, const void* ckpt, int64_t k, const void* col_scale,
                             const void* col_shift, zero_dtype_t grad_dtype, void* dw, int64_t ldw,
                             void* db, int accumulate, void* work, void* stream);

/* Workspace bytes of zero_act_wgrad; 0 on invalid sizes. */
uint64_t zero_act_wgrad_workspace(int64_t tokens, int64_t n, int64_t k);

/* ---- norms around a block, with its gate and residual scale ------------------- */

typedef enum { ZERO_NORM_NONE = 0, ZERO_NORM_RMS = 1, ZERO_NORM_LAYER = 2 } zero_norm_kind_t;

/* Most columns of a norm's rows. */
#define ZERO_NORM_MAX_COLS 16384

/* What stands between one block's output y and the next block's input x, on a
 * residual stream h (each row of `cols` elements on its own):
 *   yh = post-norm of y without weights        (ZERO_NORM_NONE: yh = y)
 *   z  = post_w yh + post_b
 *   h' = h + alpha * gate * z
 *   xh = pre-norm of h' without weights
 *   x  = pre_w xh + pre_b
 * where ZERO_NORM_RMS divides a row by sqrt(mean(v^2) + eps) and
 * ZERO_NORM_LAYER first subtracts the row's mean.  All in fp32, each output
 * rounded once; xh is taken of the unrounded h'.
 *   dtype       fp16 or bf16: y, x, weights, gate and their gradients' inputs.
 *   res_dtype   of the residual stream (h, h', their gradients): dtype or fp32.
 *   post, pre   zero_norm_kind_t; pre = ZERO_NORM_NONE: no x.
 *   alpha       residual scale (finite).  eps >= 0.
 *   group_rows  rows that share a row of the gate (e.g. a sequence's length): row
 *               i uses gate row i / group_rows; 0: one gate row for all.
 *   post_w, post_b, pre_w, pre_b   [cols]; NULL: 1 (weights), 0 (biases).  They
 *               belong to a norm: with ZERO_NORM_NONE they have to be NULL.
 *   gate        [ceil(rows / group_rows)][cols], contiguous; NULL: 1.
 * Pointers need the alignment of their element (16-byte aligned rows are
 * fastest); checkpoints and statistics 16 bytes. */
typedef struct {
    int32_t dtype, res_dtype, post, pre;
    int64_t rows, cols, group_rows;
    float   eps, alpha;
    const void *post_w, *post_b, *gate, *pre_w, *pre_b;
} zero_norm_t;

/* The forward pass.  h [rows] rows ldh apart, and y; y = NULL: no block yet, h' = h
 * (h_out may then be NULL, and post, gate, ckpt_y have to be none).  h_out may be
 * h itself.  x: NULL iff pre is ZERO_NORM_NONE.
 * For the backward pass (all may be NULL when there is none):
 *   ckpt_y   8-bit checkpoint of yh, ckpt_x of xh (the format above; the limits of
 *            dtype's exponents apply);
 *   stats    [rows][4] fp32: mean and 1/deviation of the post-norm, then of the
 *            pre-norm (0 and 1 where there is none).
 * Asynchronous.  rows = 0 is accepted.  Errors: ZERO_EINVAL (description, sizes:
 * rows in [0, 2^31), cols in [1, ZERO_NORM_MAX_COLS]; strides below cols; null or
 * misaligned pointer), ZERO_ECUDA. */
zero_status_t zero_norm_forward(const zero_norm_t* norm, const void* h, int64_t ldh, const void* y,
                                int64_t ldy, void* h_out, int64_t ldho, void* x, int64_t ldx,
                                void* ckpt_y, void* ckpt_x, float* stats, void* stream);

/* The backward pass, with yh and xh read from the checkpoints.  dh_out is the
 * gradient of h' from later use of the residual stream (NULL: zero), dx that of x
 * (NULL iff pre is none).  With r and the means from stats,
 *   D  = dh_out + r1 (pre_w dx - [mean(pre_w dx)] - xh mean(pre_w dx xh))
 *   dh = D
 *   dz = alpha gate D
 *   dy = r2 (post_w dz - [mean(post_w dz)] - yh mean(post_w dz yh))  (dz if none)
 * ([] for ZERO_NORM_LAYER), and summed over rows
 *   dpre_w = sum dx xh, dpre_b = sum dx, dpost_w = sum dz yh, dpost_b = sum dz,
 *   dgate[group] = sum over the group's rows of alpha D z.
 * dh may be dh_out itself, dy may be NULL (a stream without a block yet: ckpt_y,
 * post, gate none).  ckpt_y is needed if post is a norm or dgate is wanted.
 * dpost_w ... dpre_b [cols], dgate [groups][cols]: grad_dtype (dtype or fp32),
 * NULL where not wanted; accumulate as in zero_act_wgrad.  The gradients of a NULL
 * weight may be asked for too.  work: zero_norm_workspace(norm) bytes, 16-byte
 * aligned, contents ignored; calls whose executions overlap need one each.
 * Sums are taken in a fixed order: equal inputs give equal bits.  Asynchronous.
 * Errors: as zero_norm_forward. */
zero_status_t zero_norm_backward(const zero_norm_t* norm, const void* dh_out, int64_t lddho,
                                 const void* dx, int64_t lddx, const void* ckpt_y,
                                 const void* ckpt_x, const float* stats, void* dh, int64_t lddh,
                                 void* dy, int64_t lddy, zero_dtype_t grad_dtype, void* dpost_w,
                                 void* dpost_b, void* dgate, void* dpre_w, void* dpre_b,
                                 int accumulate, void* work, void* stream);

/* Workspace bytes of zero_norm_backward; 0 on an invalid description. */
uint64_t zero_norm_workspace(const zero_norm_t* norm);

/* ---- losses over the vocabulary ----------------------------------------------- */

/* Most rows, columns, vocabulary and teacher's entries a row of the head's losses. */
#define ZERO_HEAD_MAX_ROWS 65536
#define ZERO_HEAD_MAX_COLS 16384
#define ZERO_HEAD_MAX_VOCAB (1 << 24)
#define ZERO_HEAD_MAX_TOP 256

/* The end of a model: the last norm's rows x [rows][cols], the head's weights w
 * [vocab][cols], the logits z = x w^T and a loss of each row's softmax.  The logits
 * are computed tile by tile and never kept, neither by the forward pass nor by the
 * backward pass, which computes them once more, a piece of the vocabulary at a time;
 * its gradients go where they are wanted (dw: e.g. the tensor's place in a rank's
 * gradient row).
 *   dtype        fp16 or bf16: x, w, dx, dw.
 *   piece        columns of the vocabulary that the backward pass keeps the logits'
 *                gradient of at a time (2 rows piece bytes of workspace), rounded up
 *                to 256, at most 65536; 0: the library's choice (up to 1 GB, the fastest).
 *                The workspace also has room for a copy of unaligned rows of w (up to
 *                256 MB, less with a smaller piece): with few rows it is larger than their logits
 *                would be.
 *   z_loss       weight of the squared log-sum-exp (0: none).
 *   top, top_dtype, temperature, hard, soft   zero_distill_* only (others do not look at
 *                them, but top is counted in the workspace): the teacher's entries of a row,
 *                the type of its logits (fp16, bf16, fp32), the temperature (> 0) and the
 *                weights of the two parts of the loss. */
typedef struct {
    int32_t dtype, top, top_dtype;
    float   temperature, hard, soft, z_loss;
    int64_t rows, cols, vocab, piece;
} zero_head_t;

/* Softmax cross entropy.  With l = log sum_j exp(z_j) of row i and y its label,
 *   loss[i] = l - z_y + z_loss l^2,   lse[i] = l.
 * A row with a negative label takes no part: its x is not read, its loss and lse are
 * 0.  A label >= vocab gives NaN (loss and lse; the backward pass then gives NaN in
 * the row's dx and all of dw).
 *   labels   [rows] int32.     loss, lse   [rows] fp32.
 *   sums     two fp32 (NULL: not wanted): the sum of the losses, and the number of
 *            rows that take part.
 *   work     zero_head_workspace(head) bytes, 16-byte aligned, contents ignored; calls
 *            whose executions overlap need one each.
 * Rows of x and w lie ldx and ldw elements apart and need the alignment of their
 * element; rows of w that are not 16-byte aligned are first copied to the workspace,
 * a piece at a time.  The logits are fp32 sums of exact products, added by the tensor
 * cores in runs of at most 768 columns that are then added in fp32.  Sums are taken
 * in a fixed order: equal inputs give equal bits.  Asynchronous.  rows = 0 is accepted
 * (sums are 0).  A bounded device wait that gives up (none should) sets the first
 * int32 of `work` to ZERO_ETIMEOUT and gives NaN.
 * Errors: ZERO_EINVAL (description: type; rows in [0, ZERO_HEAD_MAX_ROWS], cols in [1,
 * ZERO_HEAD_MAX_COLS], vocab in [1, ZERO_HEAD_MAX_VOCAB], piece >= 0, top in [0,
 * ZERO_HEAD_MAX_TOP], z_loss not finite; strides below cols or above 2^31; null or
 * misaligned pointer), ZERO_ECUDA. */
zero_status_t zero_ce_forward(const zero_head_t* head, const void* x, int64_t ldx, const void* w,
                              int64_t ldw, const int32_t* labels, float* loss, float* lse,
                              float* sums, void* work, void* stream);

/* Its gradients: with g_i = scale * row_grad[i] / *divisor (row_grad [rows] fp32, NULL: 1;
 * divisor one fp32 on the device, e.g. sums + 1 for a mean, NULL: 1; g_i = 0 if it is 0),
 *   dz_ij = g_i (p_ij (1 + 2 z_loss l_i) - [j = y_i]),   p_ij = exp(z_ij - lse[i])
 *   dx_i  = sum_j dz_ij w_j,   dw_j = sum_i dz_ij x_i.
 * lse is what the forward pass wrote.  Rows that take no part, and rows with g_i = 0,
 * have dx = 0 and are not read, whatever their lse.  dz is rounded once to dtype, relative to its row's
 * own power of two (so neither a loss scale nor small weights cost bits), and dx gets back what that
 * cut off at the row's heaviest targets; all sums are fp32, and dx and dw are rounded once.
 * dw adds rows times their powers of two.  Where these differ (row_grad or z_loss), fp16's short exponent
 * moves a row's part of a dw by up to 2^-39 of the largest |g_i x_ik| of all rows (times hard + soft T and
 * 1 + 2 z_loss l): two of fp16's smallest numbers at most while that is within its range.  bf16 keeps rows whose
 * scale is 2^-100 of the largest.
 *   dx, dw      rows lddx, lddw apart, aligned to their element (16-byte aligned rows are
 *               written fastest); either may be NULL: not wanted.  dx may be x itself
 *               (lddx = ldx).
 *   accumulate  1: dw is added to what it holds (one rounding); 0: overwritten.
 * Results overlap no input but as said.  rows = 0 is accepted (dw is 0, or nothing is added).  The rest as zero_ce_forward. */
zero_status_t zero_ce_backward(const zero_head_t* head, const void* x, int64_t ldx, const void* w,
                               int64_t ldw, const int32_t* labels, const float* lse,
                               const float* row_grad, float scale, const float* divisor, void* dx,
                               int64_t lddx, void* dw, int64_t lddw, int accumulate, void* work,
                               void* stream);

/* Distillation from a teacher's top logits: a row has head->top entries (top_index[i][k],
 * top_logit[i][k]), rows ldt apart, in any order.  An entry with a negative index or a logit of
 * -inf is none (a teacher that kept fewer); entries of one index are added.  With T the
 * temperature, q = softmax of the row's logits / T over its entries and
 * l_T = log sum_j exp(z_j / T),
 *   loss[i] = soft T^2 sum_k q_k (log q_k - z_k / T + l_T) + hard (l - z_y + z_loss l^2)
 *   lse[i]  = {l_T, l}   ([rows][2]; l is 0 without labels)
 *   dz_ij   = g_i (soft T (exp(z_ij / T - l_T) - q_j) + hard (p_ij (1 + 2 z_loss l) - [j = y]))
 * labels may be NULL: no second part, and a row without an entry takes no part.  With
 * labels a row with a negative label takes no part, and one without an entry has no first
 * part.  An index >= vocab of an entry gives NaN as such a label does.  The rest as zero_ce_forward
 * and zero_ce_backward; also ZERO_EINVAL: head->top < 1, ldt < head->top, its type, weights
 * that are not finite, a temperature that is not > 0 (or whose inverse is not finite). */
zero_status_t zero_distill_forward(const zero_head_t* head, const void* x, int64_t ldx,
                                   const void* w, int64_t ldw, const int32_t* top_index,
                                   const void* top_logit, int64_t ldt, const int32_t* labels,
                                   float* loss, float* lse, float* sums, void* work, void* stream);
zero_status_t zero_distill_backward(const zero_head_t* head, const void* x, int64_t ldx,
                                    const void* w, int64_t ldw, const int32_t* top_index,
                                    const void* top_logit, int64_t ldt, const int32_t* labels,
                                    const float* lse, const float* row_grad, float scale,
                                    const float* divisor, void* dx, int64_t lddx, void* dw,
                                    int64_t lddw, int accumulate, void* work, void* stream);

/* Workspace bytes of the four calls above; 0 on an invalid description. */
uint64_t zero_head_workspace(const zero_head_t* head);

/* ---- memory ledger and communication volume ------------------------------- */

/* Bytes of model state one rank holds ([L18] 1.2, 2.1; [Z026] 2; [L32] 2.1,
 * 2.3): K bytes of optimizer state per parameter (12 for Adam; 16 in the
 * slides' count that keeps an fp32 gradient) plus 2 + 2 for the 16-bit
 * parameters and gradients:
 *   stage 0 (4+K) psi;  1: 4 psi + K psi/nd;  2: 2 psi + (2+K) psi/nd;
 *   stage 3 (4+K) psi/nd.  Divisions round up.  0 on invalid arguments. */
uint64_t zero_state_bytes(uint64_t psi, uint64_t nd, int stage, int K);

/* Elements each rank sends per step ([L18] 3.1; [L32] 2.3; [PZ] 0x07):
 * stages 0-2: 2 psi (reduce-scatter + all-gather); stage 3: 3 psi (the
 * parameters are gathered again for the backward pass).  exact = 1 keeps
 * only the (nd - 1)/nd share that is not already local (rounded up).
 * 0 on invalid arguments. */
uint64_t zero_comm_volume(uint64_t psi, uint64_t nd, int stage, int exact);

/* Largest psi whose model state fits in mem_bytes per rank ([L18] 2.6). */
uint64_t zero_max_params(uint64_t mem_bytes, uint64_t nd, int stage, int K);

/* ---- diagnostics ----------------------------------------------------------- */

/* Static string naming a status code. */
const char* zero_status_string(zero_status_t status);

/* Per-kernel timing: when enabled, zero_step records CUDA events around each
 * of its kernels on the step's stream; zero_plan_kernel_times waits for the
 * last step and returns the accumulated milliseconds of the reduce pass
 * (pass 1, or the fused pass), of the update pass (0 for the fused path), the
 * number of timed steps and the number of kernels the plan has launched.
 * enable = 0 turns timing off; enable = 1 also clears the accumulators. */
zero_status_t zero_plan_profile(zero_plan_t plan, int enable);
zero_status_t zero_plan_kernel_times(zero_plan_t plan, double* reduce_ms, double* update_ms,
                                     int64_t* steps, int64_t* launches);

/* Which kernel path the plan runs: 0 = fused single pass (no clip, no dynamic
 * scale, no skip_on_overflow), 1 = two passes through an fp32 gradient in the
 * workspace, 2 = two passes that re-read the 16-bit gradients (clip, dynamic
 * scale or skip_on_overflow, nd < 4). */
int zero_plan_path(zero_plan_t plan);

/* Which kernel runs the reduce pass of a two-pass plan: 0 = 128-bit loads of
 * the rank rows (the default, measured fastest at nd = 16), 1 = TMA bulk
 * staging (cp.async.bulk of each rank's 2 KB row slice into a ring of shared-
 * memory stages, a producer warp and eight consumer warps).  Both compute the
 * same reduced gradient bit for bit; the norm's partial sums are grouped
 * differently.  Kind 1 needs the two-pass path with the fp32 workspace and
 * 4 <= nd <= 48 (ZERO_EINVAL otherwise).  Waits for the plan's last step.
 * A bounded wait in kind 1 that gives up makes zero_step_result return
 * ZERO_ETIMEOUT from then on. */
zero_status_t zero_plan_set_reduce_kernel(zero_plan_t plan, int kind);

#ifdef __cplusplus
}
#endif
#endif
