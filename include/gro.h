/*
 * gro.h -- placement-aware gradient reduction, global L2 norm, clipping and
 * fused AdamW for one MI355X (gfx950).  C ABI.
 *
 * The operation is the per-step gradient-ownership path of data- and
 * tensor-parallel training described in NeMo Automodel issue #3857,
 * "refactor(distributed): establish shared native TP replica ownership":
 *
 *   section "Why this needs separate work" -- a replicated parameter's local
 *     gradient means one of four things: complete (redundant compute; averaged
 *     over the TP ranks), partial (head- or sequence-sharded compute; summed),
 *     a local shard (never synchronised as a replica), or already reduced by
 *     another owner (not reduced again);
 *   section "Preserved prototype and evidence" -- FP32 reduction, BF16
 *     gradients, gradient accumulation including partial windows, clipping,
 *     Adam updates;
 *   section "Proposed scope and acceptance criteria" -- explicit
 *     replica/partial/shard semantics, exactly one reduction owner per
 *     parameter, unsupported compositions rejected, global norms, clipping
 *     on/off, accumulation over 1, >1 and trailing windows.
 *
 * Mixle v0.8.1 "Distributed Transformer Training", section "Backend split":
 * a request that cannot be executed fails before fitting -- here every check
 * happens on the host before any device work, so a failed call has no side
 * effects.  Section "Optimizer and checkpoint semantics": the optimizer
 * addresses parameters by names that stay fixed across wrapping -- here a
 * caller-chosen 64-bit param_id.
 *
 * One GPU holds the R rank contributions of a replicated parameter as R
 * stacked slots in its own HBM; the kernels do that GPU's share of the work.
 *
 * Conventions
 *  - Memory: the caller allocates every device buffer (acc, master, m, v, the
 *    BF16 parameter copy, the per-bucket gradient buffers and the workspace).
 *    The library never allocates or frees device memory and never calls a
 *    collective.  A plan owns only host tables.
 *  - Device pointers must be 16-byte aligned (256-byte for the workspace); a
 *    group's and the layers' arrays only to their element.
 *  - Streams: `stream` is a hipStream_t passed as void* (NULL = the null
 *    stream).  All device work is enqueued on it, asynchronously.  Use one
 *    stream per plan, or per group, at a time.
 *  - Errors: functions return GRO_OK (0) or a negative GRO_E_* code and set
 *    a thread-local message (gro_last_error).  Validation precedes any device
 *    work.  Non-finite data is reported through gro_plan_get_norm's `finite`
 *    flag, not a return code, because device work is asynchronous.
 *  - Only gro_plan_bind, gro_plan_bind_static, gro_init_uniform,
 *    gro_plan_get_norm, gro_group_bind and gro_group_get_norm wait for the
 *    device.  The step's calls (gro_accumulate*, gro_reduce_norm,
 *    gro_clip_adamw, gro_clip_adamw_coded, gro_moments_encode,
 *    gro_moments_decode, gro_group_norm, gro_group_clip_adamw) and the layers'
 *    (gro_row_sort, gro_lookup*, gro_experts_*) only enqueue kernels
 *    -- no allocation, no synchronization, no memory fill -- so a step may be
 *    captured in a HIP graph after binding and replayed; the replay repeats
 *    the captured arguments, the AdamW step count included.
 *  - Not thread-safe per plan or group; distinct ones may be used from
 *    distinct threads.
 */
#ifndef GRO_H
#define GRO_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

/* ---- return codes ---- */
#define GRO_OK            0
#define GRO_E_INVALID    (-1)  /* null/misaligned pointer, bad size/shape/step/window, NaN max_norm */
#define GRO_E_PLACEMENT  (-2)  /* unknown placement, shard_index out of range, bad flags */
#define GRO_E_DUPLICATE  (-3)  /* a second owner for one param_id, or for memory of a group */
#define GRO_E_STATE      (-4)  /* unbound plan, window bookkeeping violated */
#define GRO_E_HIP        (-5)  /* HIP runtime or launch error */

/* ---- placements (what a rank-local gradient means) ---- */
#define GRO_REPLICATE 0  /* complete gradient on every rank: averaged over R */
#define GRO_PARTIAL   1  /* partial contribution per rank: summed over R */
#define GRO_SHARD     2  /* local shard owned by this rank: used as is */
#define GRO_REDUCED   3  /* already reduced by another owner: used as is */

/* ---- per-tensor flags ---- */
#define GRO_NO_DECAY  1u  /* no weight decay for this tensor */
#define GRO_FROZEN    2u  /* no gradient, not in the norm, not updated */
#define GRO_FP32_GRAD 4u  /* gradient contributions arrive in FP32 instead of BF16 */
#define GRO_CODED_MOMENTS 8u  /* groups only: this tensor's moments are held in 8 bits */

/* ---- gradient element types (gro_tensor_layout / gro_bucket_info) ---- */
#define GRO_GRAD_BF16 0
#define GRO_GRAD_FP32 1

/* ---- owner classes reported by gro_plan_tensor / gro_plan_bucket ---- */
#define GRO_OWNER_MEAN          0
#define GRO_OWNER_SUM           1
#define GRO_OWNER_LOCAL_SHARD   2
#define GRO_OWNER_LOCAL_REDUCED 3
#define GRO_OWNER_EXCLUDED      4

#define GRO_MAX_NDIM 8

/* One parameter as this GPU sees it.  `shape` (host memory, `ndim`
 * entries, each >= 0; may be NULL when ndim == 0, a scalar) is read only
 * during gro_plan_create.  `shard_index` is this rank's index in [0, R) for
 * GRO_SHARD and must be -1 for the other placements. */
typedef struct gro_tensor_desc {
  int64_t param_id;
  const int64_t* shape;
  int32_t ndim;
  int32_t placement;
  int32_t shard_index;
  uint32_t flags;
} gro_tensor_desc;

typedef struct gro_plan gro_plan;

typedef struct gro_plan_info {
  int32_t R;
  int32_t n_tensors;
  int32_t n_buckets;
  int32_t chunk_elems;      /* elements per chunk (norm partial granularity) */
  int64_t n_chunks;
  int64_t n_flat;           /* elements to allocate for acc, master, m, v, BF16 copy */
  int64_t n_owned;          /* elements inside buckets (reduced, in the norm, updated) */
  int64_t bucket_elems;     /* bucket capacity the plan was created with */
  uint64_t workspace_bytes; /* device workspace gro_plan_bind needs */
} gro_plan_info;

/* The ownership row of one tensor plus where it lives in the flat arrays.
 * A tensor is contiguous in the flat arrays: [flat_offset, flat_offset+numel).
 * It spans buckets first_bucket .. first_bucket+n_buckets-1 (more than one
 * only when it is larger than the bucket capacity). */
typedef struct gro_tensor_layout {
  int64_t param_id;
  int64_t numel;
  int64_t flat_offset;      /* -1 when excluded */
  int32_t owner;            /* GRO_OWNER_* */
  int32_t slots;            /* rank contributions read per microbatch (0 if excluded) */
  int32_t divisor;          /* R for MEAN, 1 for SUM/LOCAL, 0 if excluded */
  int32_t in_norm;
  int32_t updated;
  int32_t decayed;
  int32_t first_bucket;     /* -1 when the tensor has no elements in a bucket */
  int32_t n_buckets;
  int32_t grad_dtype;       /* GRO_GRAD_BF16 or GRO_GRAD_FP32 */
} gro_tensor_layout;

/* A bucket: flat range [flat_base, flat_base+len) of one owner class, one
 * decay setting and one gradient type.  Its gradient buffer is
 * [slots][slot_stride] elements of that type (BF16 or FP32): element
 * flat_base+i of slot r is at index r*slot_stride + i. */
typedef struct gro_bucket_info {
  int64_t flat_base;
  int64_t len;
  int64_t slot_stride;
  int64_t first_chunk;
  int64_t n_chunks;
  int32_t owner;
  int32_t slots;
  int32_t decayed;
  int32_t grad_dtype;       /* GRO_GRAD_BF16 or GRO_GRAD_FP32 */
} gro_bucket_info;

/* AdamW hyper-parameters as the user states them (FP64).  Per-step scalars
 * are derived from them in FP64 and rounded once to FP32. */
typedef struct gro_adamw_hparams {
  double lr;
  double beta1;
  double beta2;
  double eps;
  double weight_decay;
} gro_adamw_hparams;

/* Build a plan.  Passages: NeMo Automodel issue #3857, section "Why this
 * needs separate work" (what a local gradient of a replicated parameter
 * means, per placement) and section "Proposed scope and acceptance criteria"
 * (explicit replica/partial/shard semantics, exactly one reduction owner,
 * unsupported compositions rejected); NeMo AutoModel "Model Parallelizer
 * API", section "Choose the Extension Point" (sharding units may be drawn as
 * groups of one dtype -- here buckets hold one gradient type).
 * First the ownership of every tensor from its placement, one owner per
 * param_id: duplicates -> GRO_E_DUPLICATE; bad placement/shard_index/flags
 * -> GRO_E_PLACEMENT; R < 1, n_tensors < 0, ndim out of [0,8], negative
 * dims, bucket_elems < 64 -> GRO_E_INVALID.  Then the layout: tensors
 * grouped by (owner class, decay, gradient type) in the order MEAN, SUM,
 * LOCAL_SHARD, LOCAL_REDUCED (decayed first, BF16 first), descriptor order
 * within a group, packed into buckets of at most bucket_elems elements; only
 * a tensor larger than the capacity is split.  Host only, deterministic.  On
 * success *out owns the host tables. */
int gro_plan_create(const gro_tensor_desc* tensors, int32_t n_tensors, int32_t R,
                    int64_t bucket_elems, gro_plan** out);

/* Free a plan's host tables (NULL is ignored).  Device memory is the caller's. */
void gro_plan_destroy(gro_plan* plan);

int gro_plan_get_info(const gro_plan* plan, gro_plan_info* info);
int gro_plan_tensor(const gro_plan* plan, int32_t i, gro_tensor_layout* out);
int gro_plan_bucket(const gro_plan* plan, int32_t b, gro_bucket_info* out);

/* Upload the plan's bucket and chunk tables into the caller's device
 * workspace (>= workspace_bytes, 256-byte aligned) on `stream`, and wait for
 * the copy.  Must precede the calls below; may be repeated (rebinding). */
int gro_plan_bind(gro_plan* plan, void* d_workspace, uint64_t bytes, void* stream);

/* Bytes of the library's own device workspace, one per GPU, used by
 * gro_plan_bind_static (enough for about 700,000 chunks, i.e. plans of up to
 * about 2.8e9 elements). */
#define GRO_STATIC_WORKSPACE_BYTES 16777216ull

/* For callers that cannot allocate device memory (code under graph capture,
 * tight serving loops, harnesses that forbid hipMalloc): gro_plan_bind on a
 * workspace the library holds itself -- a static device array of
 * GRO_STATIC_WORKSPACE_BYTES per GPU, kept until the process ends -- instead
 * of one the caller allocates.  Every later call of the plan behaves as
 * after gro_plan_bind; the caller still passes the accumulator, the states
 * and the gradient buffers.  Allocates nothing, frees nothing.
 *  - A plan whose workspace_bytes exceeds GRO_STATIC_WORKSPACE_BYTES:
 *    GRO_E_INVALID, nothing done.
 *  - All plans bound this way on one GPU share that GPU's array.  Binding
 *    waits for all work on the current device to finish, then overwrites
 *    the array; from then on a plan bound to it earlier is rejected with
 *    GRO_E_STATE until it is bound again.  Device calls of two plans that
 *    overlap on one GPU would race on the array, which is why only the
 *    last plan bound may use it.
 *  - Binding clears what must start at zero -- the norm's completion
 *    counters (every bind does) -- and the norm scalars; every other byte
 *    of the array is written by a kernel before one reads it.
 *  - Waits for its own upload, like gro_plan_bind.  Not for use inside a
 *    graph capture (it synchronizes); bind first, then capture. */
int gro_plan_bind_static(gro_plan* plan, void* stream);

/* Reduce + cast + accumulate one microbatch for buckets [b0, b1) -- NeMo
 * Automodel issue #3857, section "Why this needs separate work" (Replicate
 * contributions averaged, Partial summed, Shard and already-reduced used as
 * they are) and section "Preserved prototype and evidence" (an FP32
 * reduction hook on BF16 gradients, gradient accumulation).
 * d_grad_buckets: host array of b1-b0 device pointers; entry j is bucket
 * b0+j's BF16 gradient buffer [slots][slot_stride].  d_acc: FP32 [n_flat].
 * Per element: the slots are widened and summed in FP32 in slot order; MEAN
 * divides by R; micro_index 0 starts the window (acc = reduced), later
 * microbatches add (acc += reduced).  micro_index must equal the number of
 * microbatches this bucket has accumulated in the current window (0 restarts).
 * window_size > 0 announces the window length: on its last microbatch the
 * kernel also writes the chunks' norm partials (saving gro_reduce_norm a read
 * of acc); 0 = not known.  Gradient buffers are only read.  All buckets of
 * one window accumulate into one d_acc: starting buckets on another
 * accumulator while other buckets of the window are in progress is
 * GRO_E_STATE (a window ends with gro_clip_adamw or a rebind). */
int gro_accumulate(gro_plan* plan, int32_t b0, int32_t b1, const void* const* d_grad_buckets,
                   float* d_acc, int32_t micro_index, int32_t window_size, void* stream);

/* The whole window of n microbatches for buckets [b0, b1) in one pass
 * (NeMo Automodel issue #3857, section "Proposed scope and acceptance
 * criteria": accumulation windows of one, several and a trailing number of
 * microbatches; the reduction itself as for gro_accumulate):
 * bit for bit what gro_accumulate with micro_index 0..n-1 and window_size n
 * computes (per element: acc = red_0, then acc = acc + red_k in microbatch
 * order; norm partials written at the end), but the accumulator is written
 * once instead of being read and written n times.  For callers that keep
 * every microbatch's gradient buckets resident until the window ends (on a
 * 288 GB MI355X this trades n * sum_b(slots_b * slot_stride_b) BF16
 * elements of memory for (8n - 4) bytes per element less traffic).
 * d_grad_buckets: host array of n*(b1-b0) device pointers, microbatch-major:
 * entry k*(b1-b0) + j is microbatch k's BF16 buffer [slots][slot_stride] of
 * bucket b0+j.  1 <= n <= 64.  Leaves these buckets with a complete window
 * of n (any earlier partial window of theirs is discarded).  The same
 * one-accumulator rule as gro_accumulate applies. */
int gro_accumulate_window(gro_plan* plan, int32_t b0, int32_t b1, const void* const* d_grad_buckets,
                          int32_t n, float* d_acc, void* stream);

/* Microbatches first_micro .. first_micro+n-1 of a window for buckets
 * [b0, b1) in one pass (NeMo Automodel issue #3857, section "Preserved
 * prototype and evidence": accumulation that includes partial windows):
 * bit for bit what gro_accumulate with those micro_index values computes (starting from the accumulator in memory when
 * first_micro > 0), with the accumulator read and written once for the
 * group.  For callers that can keep a few microbatches' gradient buckets
 * resident but not a whole window: n microbatches in g groups move
 * 8 * (n - g) bytes per element less accumulator traffic than one call per
 * microbatch (a window of 8 in groups of 4: 48 bytes per element).
 * d_grad_buckets: host array of n*(b1-b0) device pointers, microbatch-major,
 * as for gro_accumulate_window.  1 <= n <= 64, first_micro >= 0;
 * first_micro > 0 requires every bucket in the range to have accumulated
 * exactly first_micro microbatches of the current window into d_acc (else
 * GRO_E_STATE).  window_size as for gro_accumulate (0 = not known; when
 * first_micro + n == window_size the norm partials are written too;
 * first_micro + n > window_size is GRO_E_INVALID).  gro_accumulate_window is
 * this call with first_micro = 0 and window_size = n.  Calls of both kinds
 * and gro_accumulate may be mixed within a window. */
int gro_accumulate_microbatches(gro_plan* plan, int32_t b0, int32_t b1, const void* const* d_grad_buckets,
                                int32_t first_micro, int32_t n, int32_t window_size, float* d_acc,
                                void* stream);

/* Global L2 norm (NeMo Automodel issue #3857, section "Proposed scope and
 * acceptance criteria": global norms checked against explicit references, no
 * double reduction) of g = acc / window_size over every owned element, in
 * FP64, with no atomics: per-chunk partials summed in a fixed order, so the result
 * does not depend on launch shape and is bit-reproducible.  Every bucket must
 * have accumulated exactly window_size microbatches (else GRO_E_STATE).  The
 * result stays on the device (read it with gro_plan_get_norm). */
int gro_reduce_norm(gro_plan* plan, const float* d_acc, int32_t window_size, void* stream);

/* Wait for the plan's stream and read the last norm.  Any out pointer may be
 * NULL.  finite = 0 when the norm is NaN or infinite.  GRO_E_STATE before
 * the first gro_reduce_norm after binding.
 * Every device call (bind excepted) must run with the device the plan was
 * bound on current, else GRO_E_STATE. */
int gro_plan_get_norm(gro_plan* plan, double* norm, double* norm_sq, int32_t* finite);

/* Clip + fused AdamW on every updated element, after gro_reduce_norm of the
 * same window (NeMo Automodel issue #3857, section "Preserved prototype and
 * evidence": clipping and Adam updates on the owned state; section
 * "Proposed scope and acceptance criteria": clipping on and off; Mixle
 * "Distributed Transformer Training", section "Optimizer and checkpoint
 * semantics": AdamW over parameters addressed by stable names):
 *   g = acc / window_size;  coef = min(1, max_norm / (norm + 1e-6)) in FP64
 *   rounded to FP32 when 0 < max_norm < inf, else 1 (clipping off);
 *   g^ = g*coef; p = p*(1 - lr*wd) (1 when GRO_NO_DECAY); m = b1*m + (1-b1)*g^;
 *   v = b2*v + (1-b2)*g^*g^; p = p - (lr/(1-b1^step)) * m / (sqrt(v)/sqrt(1-b2^step) + eps);
 *   d_param_bf16 (nullable) = p rounded to BF16, nearest-even.
 * A non-finite norm skips the update: master, m, v and the BF16 copy stay
 * bit-unchanged.  step >= 1.  Ends the window. */
int gro_clip_adamw(gro_plan* plan, const float* d_acc, int32_t window_size, double max_norm,
                   const gro_adamw_hparams* hp, int64_t step, float* d_master, float* d_m,
                   float* d_v, uint16_t* d_param_bf16, void* stream);

/* Replica-consistent initialisation of the FP32 master shard (and the
 * optional BF16 copy) of every updated parameter, independent of the rank,
 * of the layout and of when it runs (NeMo Automodel issue #3857, section
 * "Why this needs separate work": parameters can be created after the
 * model is parallelised, and replicas must not rely on each rank's training
 * random stream to start alike -- this draws nothing from any other
 * generator).
 * Element i of parameter p gets offset_p + (2u - 1) * bound_p with u in
 * [0, 1) in steps of 2^-24, from Philox4x64-10 with key (seed, param_id)
 * and counter (g / 4, 0, 0, 0), word g % 4, top 24 bits, where g is the
 * element's index in the unsharded parameter: shard_index * numel + i for a
 * Shard tensor (equal dim-0 shards), i otherwise.  bounds[t] >= 0 and
 * offsets[t] (host, n_tensors entries in descriptor order, FP64 rounded to
 * FP32; NULL offsets = 0) -- e.g. offset 1, bound 0 for a norm weight.
 * Waits for its own upload before returning. */
int gro_init_uniform(gro_plan* plan, uint64_t seed, const double* bounds, const double* offsets,
                     float* d_master, uint16_t* d_param_bf16, void* stream);

/* ---- moments in 8 bits ----
 * Adam's moments as one code byte per element, with one FP32 scale per moment
 * and block of GRO_CODED_BLOCK consecutive elements: 2.125 bytes per element
 * instead of 8.
 *   m: scale s = max |m| over the block; code = the FP8 e4m3 value (no
 *      infinities, bias 7) nearest 256 * m / s.  Value: code * (s / 256).  A
 *      block whose s is below 2^-100 is held as zeros with scale 0.
 *   v: r = sqrt(v), scale s = max r; code = the unsigned 8-bit float of 4
 *      exponent bits (bias 15) and 4 mantissa bits, gradual underflow, nearest
 *      r / s -- the bits 6 to 13 of the FP16 of the same value; 240 is 1.0 and
 *      nothing above it occurs.  Value: (code * s)^2.  A v > 0 never gets the
 *      code 0.
 * Nearest means ties to even; the quotients are FP32, so a value within 2^-22
 * of the border between two codes may get either.  A block's largest element
 * is held exactly, and encoding what was decoded gives the same codes and
 * scales (unless a value leaves FP32's normal range on the way).  m comes back
 * within 2^-4 of itself or 2^-18 of its block's largest; sqrt(v) within 2^-5 of
 * itself or 2^-18 of its block's largest.  An infinite v is held as the largest
 * finite one; a NaN or negative v, or a NaN or infinite m, makes that moment
 * NaN in its whole block.
 * What rounding to the nearest code cannot follow: a step that changes a moment
 * by less than half a code leaves it as it is.  v with beta2 of 0.97 or more
 * and m with beta1 of 0.97 or more do not come down by decay alone: without a
 * gradient an element keeps its code, and its moment follows its block's
 * largest one only.  An element whose gradients become much smaller than its
 * block's largest for good keeps too large a v and takes steps that much too
 * small (after a tenfold fall 5 to 10 times, as long as the largest stays).
 * Meant for gradients whose sizes within 64 neighbours keep their order;
 * FP32 moments, which a group chooses by tensor, have no such limit.
 * In a plan a block is [64 k, 64 k + 64) of the flat arrays -- bucket bases
 * are multiples of 64, so no block spans two buckets; the part of a block past
 * the end of its bucket does not enter the scale and its bytes stay as they
 * are.  In a group's tensor blocks count from the tensor's first element. */
#define GRO_CODED_BLOCK 64

/* Device pointers of a plan's 8-bit moments: n_flat code bytes each and
 * n_flat / GRO_CODED_BLOCK scales each (all zeros = moments of zero).  16-byte
 * aligned; the four arrays, the other arrays of a call, the BF16 copy and the
 * workspace must not overlap. */
typedef struct gro_coded_moments {
  uint8_t* m;
  uint8_t* v;
  float* m_scale;
  float* v_scale;
} gro_coded_moments;

/* gro_clip_adamw with the moments in 8 bits: decode, the same update in FP32,
 * encode, in one pass.  The parameter is updated with the new moments before
 * they are rounded to codes.  Arguments, order of calls, clipping, the skipped
 * step of a non-finite norm (codes and scales stay bit-unchanged too) and
 * errors as gro_clip_adamw; overlapping arrays are GRO_E_INVALID. */
int gro_clip_adamw_coded(gro_plan* plan, const float* d_acc, int32_t window_size, double max_norm,
                         const gro_adamw_hparams* hp, int64_t step, float* d_master,
                         const gro_coded_moments* moments, uint16_t* d_param_bf16, void* stream);

/* FP32 moments of the plan's updated elements to 8 bits and back, for
 * example around a checkpoint or to change a running job over.  Elements
 * between buckets are neither read nor written.  No part of a window: may be
 * called at any time on a bound plan. */
int gro_moments_encode(gro_plan* plan, const float* d_m, const float* d_v, const gro_coded_moments* moments,
                       void* stream);
int gro_moments_decode(gro_plan* plan, const gro_coded_moments* moments, float* d_m, float* d_v, void* stream);

/* ---- groups: tensors that stay where they lie ----
 * A group steps many tensors at once whose gradients are complete (window
 * accumulation and reduction done elsewhere, for example by autograd and an
 * earlier owner) and which are not laid out by a plan: every master, moment,
 * BF16 copy and gradient is an allocation of its own or a contiguous view at
 * any element offset. */
typedef struct gro_group gro_group;

/* One tensor of a group: GRO_NO_DECAY, GRO_FP32_GRAD and GRO_CODED_MOMENTS
 * may be set. */
typedef struct gro_group_desc {
  int64_t numel;
  uint32_t flags;
  uint32_t reserved;        /* 0 */
} gro_group_desc;

/* Device pointers of one tensor, given when the group is bound.  m and v:
 * FP32, or with GRO_CODED_MOMENTS one code byte per element, and then
 * m_scale and v_scale hold ceil(numel / GRO_CODED_BLOCK) FP32 scales each
 * (else unused).  Each array aligned to its own element; a tensor is accessed
 * four elements at a time when its FP32 arrays are 16-byte, its BF16 ones
 * 8-byte and its codes 4-byte aligned, and one at a time otherwise. */
typedef struct gro_group_tensor {
  float* master;
  void* m;
  void* v;
  float* m_scale;
  float* v_scale;
  uint16_t* param_bf16;     /* may be NULL */
} gro_group_tensor;

typedef struct gro_group_info {
  int32_t n_tensors;
  int32_t chunk_elems;
  int64_t n_chunks;
  int64_t n_elems;
  uint64_t workspace_bytes; /* device workspace gro_group_bind needs */
} gro_group_info;

/* Host tables for n_tensors tensors (0 elements are allowed and do nothing).
 * GRO_E_INVALID for negative or too large sizes, GRO_E_PLACEMENT for unknown
 * flags or a nonzero reserved field. */
int gro_group_create(const gro_group_desc* tensors, int32_t n_tensors, gro_group** out);
void gro_group_destroy(gro_group* group);
int gro_group_get_info(const gro_group* group, gro_group_info* info);

/* Upload the tables into the caller's workspace (>= workspace_bytes, 256-byte
 * aligned) on `stream` and wait.  tensors: host array of n_tensors entries, read
 * only during the call.  An array that would be written twice -- a tensor given
 * twice, overlapping views, or one that overlaps the workspace -- is
 * GRO_E_DUPLICATE.  May be repeated, for example when a state has moved. */
int gro_group_bind(gro_group* group, const gro_group_tensor* tensors, void* d_workspace, uint64_t bytes,
                   void* stream);

/* Global L2 norm of g = gradient / window_size over the group's tensors, FP64,
 * no atomics, bit-reproducible, as gro_reduce_norm.  d_grads: host array of
 * n_tensors device pointers, BF16 or (GRO_FP32_GRAD) FP32, aligned to their
 * element; NULL leaves that tensor out of this step: not in the norm, not
 * decayed, not updated.  The gradients have to stay in place until
 * gro_group_clip_adamw, which reads the same ones; they must not overlap the
 * arrays the group writes. */
int gro_group_norm(gro_group* group, const void* const* d_grads, int32_t window_size, void* stream);

/* Clip + AdamW of the gradients given to the last gro_group_norm, per element
 * as gro_clip_adamw; a non-finite norm leaves everything bit-unchanged.  Needs a
 * gro_group_norm since the last call (else GRO_E_STATE), on the same stream or
 * ordered before this one.  GRO_E_HIP from one of the call's launches (one per
 * kind of tensor) may leave other kinds updated; the update is not repeated, the
 * next one needs a new norm.  After GRO_E_HIP from gro_group_norm there is no
 * norm, the last one's included. */
int gro_group_clip_adamw(gro_group* group, double max_norm, const gro_adamw_hparams* hp, int64_t step,
                         void* stream);

/* Wait for the stream of the last gro_group_norm and read its norm, as
 * gro_plan_get_norm. */
int gro_group_get_norm(gro_group* group, double* norm, double* norm_sq, int32_t* finite);

/* ---- layers: what makes the gradients of an embedding and of experts ----
 * A model's embedding and its experts' matrices are parameters like the others;
 * these calls are their forward passes, which read the BF16 copy that a step
 * leaves, and their gradients, written where gro_accumulate or gro_group_norm
 * reads them (a slot of a bucket, a gradient of a group).  Nothing is kept between
 * calls.  Sums are FP32 in an order that depends on the sizes, the rows' lengths
 * and the starts alone, never on timing: a call repeated gives the same bits.
 * Calls on different streams may overlap if each has a workspace of its own.  No
 * call waits, allocates or fills memory by a copy engine: all may be captured.
 * Arrays may lie at any address that is aligned to their element; outputs must not
 * overlap inputs or the workspace (columns side by side in one matrix do not). */
#define GRO_BF16 0
#define GRO_FP32 1
#define GRO_INT32 0
#define GRO_INT64 1

/* A matrix in device memory: element (i, j) is data[i * stride + j].  stride >=
 * cols where there is more than one row.  data may be NULL without elements. */
typedef struct gro_matrix {
  void* data;
  int64_t rows;
  int64_t cols;
  int64_t stride;
  int32_t type;             /* GRO_BF16 or GRO_FP32 */
  int32_t reserved;         /* 0 */
} gro_matrix;

/* Rows that a table of the calls below has at most (2^20). */
#define GRO_MAX_TABLE_ROWS 1048576

/* Positions by the row they name: the ids id[0..n) of a table shard that holds the
 * rows first_row .. first_row + n_rows - 1 of the whole table.  d_order[0..m): the m
 * positions whose id is one of them, by row and within a row ascending; what lies
 * behind stays as it was.  d_starts[r] (n_rows + 1 entries): where row r's positions
 * begin, d_starts[n_rows] = m.  Ids of other shards, negative ones and any other
 * values are left out.  Also gives experts' runs of rows: ids = a router's choices,
 * n_rows = the number of experts.
 * d_ids: GRO_INT32 or GRO_INT64 (id_type); n < 2^31 - 2^16.  The workspace (256-byte
 * aligned) has the bytes that gro_row_sort_workspace gives, 0 for short lists; shorter
 * lists need no more. */
int gro_row_sort_workspace(int64_t n, int64_t n_rows, uint64_t* bytes);
int gro_row_sort(const void* d_ids, int32_t id_type, int64_t n, int64_t first_row, int64_t n_rows,
                 int32_t* d_order, int32_t* d_starts, void* d_workspace, uint64_t bytes, void* stream);

/* out[i, :] = scale * table[id[i] - first_row, :], multiplied in FP32 and rounded
 * once; zeros where the id is none of the table's (another shard's: the shards'
 * results add up to the whole).  out->rows ids.  Table and out are BF16 or FP32
 * each.  The scale is rounded to FP32. */
int gro_lookup(const gro_matrix* table, int64_t first_row, const void* d_ids, int32_t id_type, double scale,
               const gro_matrix* out, void* stream);

/* The lookup's gradient from sorted positions (gro_row_sort of the same ids, with
 * n = dy->rows and n_rows = out->rows): out[r, :] = scale * sum of dy[i, :] over row
 * r's positions i.  Every row is written, zeros for rows without any; with
 * accumulate = 1 it is added to what is there, and rows without any are not touched
 * (a tied head's gradient, an FP32 gradient of several microbatches).  Sums are
 * FP32, rounded once.  dy and out are BF16 or FP32 each, of at most 2^24 columns.  Entries of d_order and
 * d_starts outside their range are never followed. */
int gro_lookup_grad_workspace(int64_t n, int64_t cols, uint64_t* bytes);
int gro_lookup_grad(const gro_matrix* dy, const int32_t* d_order, const int32_t* d_starts, double scale,
                    int32_t accumulate, const gro_matrix* out, void* d_workspace, uint64_t bytes, void* stream);

/* Experts' matrices W_e, [outer][inner] each: element (o, i) of expert e is
 * data[e * expert_stride + o * stride + i]. */
typedef struct gro_experts {
  void* data;
  int64_t outer;
  int64_t inner;
  int64_t stride;
  int64_t expert_stride;
  int32_t n_experts;        /* at most GRO_MAX_EXPERTS */
  int32_t type;             /* GRO_BF16, gradients GRO_BF16 or GRO_FP32 */
  int32_t reserved;         /* 0 */
} gro_experts;
#define GRO_MAX_EXPERTS 4096

/* Products of ragged runs of rows, each with its expert's matrix: rows d_starts[e]
 * .. d_starts[e + 1] - 1 are expert e's (n_experts + 1 entries, not descending;
 * entries are cut to 0 .. rows).  The runs' lengths are read on the device only.
 *   forward:      y = x W_e^T    x [rows][inner], y [rows][outer]
 *   input grad:   dx = dy W_e    dy [rows][outer], dx [rows][inner]
 *   weight grad:  dW_e = dy^T x  over the expert's rows; zeros for an expert without
 *                 rows; with accumulate = 1 added to what is there, and experts
 *                 without rows are not touched.
 * x, dy and W are BF16, results BF16 or FP32; products are summed in FP32 and rounded
 * once.  Rows in front of d_starts[0] and from d_starts[n_experts] on are neither
 * read nor written.  An expert's result depends on its own rows alone: infinities and
 * NaN of other rows do not reach it.  Few rows or small matrices leave few tiles for
 * the GPU; their sums are then taken in parts, whose workspace (256-byte aligned) has
 * the bytes that gro_experts_workspace gives, enough for any of the three and 0 for
 * most sizes. */
int gro_experts_workspace(int32_t n_experts, int64_t rows, int64_t inner, int64_t outer, uint64_t* bytes);
int gro_experts_forward(const gro_matrix* x, const gro_experts* weights, const int32_t* d_starts,
                        const gro_matrix* y, void* d_workspace, uint64_t bytes, void* stream);
int gro_experts_input_grad(const gro_matrix* dy, const gro_experts* weights, const int32_t* d_starts,
                           const gro_matrix* dx, void* d_workspace, uint64_t bytes, void* stream);
int gro_experts_weight_grad(const gro_matrix* dy, const gro_matrix* x, const int32_t* d_starts,
                            int32_t accumulate, const gro_experts* dw, void* d_workspace, uint64_t bytes,
                            void* stream);

/* Thread-local text of the last error ("" if none). */
const char* gro_last_error(void);

#ifdef __cplusplus
}
#endif

#endif /* GRO_H */
