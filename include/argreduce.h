/*
 * argreduce.h -- C ABI of the MI355X (gfx950) last-axis ArgMax / ArgMin library.
 *
 * One operation: for every row of a contiguous row-major [rows, cols] tensor, the int64
 * index of its maximum (ArgMax) or minimum (ArgMin). The result is defined by the
 * sequential one-thread-per-row scan described in "[CUDA] Parallelize ArgMax/ArgMin over
 * wide last axes" (ONNX Runtime pull request 32092), Description / Semantics:
 *   - the result equals, for every input, that of a scan that starts with element 0 as the
 *     running best and moves to a later element only when it compares strictly greater
 *     (ArgMax) or strictly less (ArgMin);
 *   - hence ties resolve to the lowest index (select_last_index == 0);
 *   - a NaN at index 0 yields 0, a NaN elsewhere is never selected (IEEE comparisons with
 *     NaN are false);
 *   - rows made only of -inf, +inf or NaN yield 0; -inf / +inf are ordinary values, which
 *     is why the parallel merge uses them, not the lowest / highest finite value, as the
 *     identity of an empty partial result.
 * Element formats are IEEE binary32 (f32), binary16 (f16), bfloat16 (bf16) and binary64
 * (f64); comparisons are exact (f16 and bf16 are widened exactly to binary32), subnormals
 * included.
 *
 * Threading, memory and streams (same page, Description / Approach and Testing):
 *   - every pointer argument is a DEVICE pointer owned by the caller; the library never
 *     allocates, frees or prints, and only argreduce_wait_timeouts (a diagnostic read of
 *     a device counter) synchronises;
 *   - all work is enqueued on the caller's HIP stream (`stream` is a hipStream_t, NULL for
 *     the default stream), so a call may be captured into a HIP graph and replayed;
 *   - functions are safe to call from several host threads; calls that share one scratch
 *     buffer must be ordered on one stream.
 *
 * Status codes: 0 on success, a negative ARGREDUCE_ERR_* value otherwise. On every error
 * except ARGREDUCE_ERR_HIP nothing has been enqueued and out_idx is untouched. One
 * device-side condition cannot be returned by the call, which returns before the kernels
 * run: should a workgroup of a split row never publish its result (not expected: those
 * workgroups wait on nothing), the row's finalizing workgroup gives up after a bounded
 * wait, stores -1 in out_idx[r] and adds one to the device's timeout count, which
 * argreduce_wait_timeouts reads.
 */
#ifndef ARGREDUCE_H
#define ARGREDUCE_H

#include <stddef.h>
#include <stdint.h>

#ifdef __cplusplus
extern "C" {
#endif

typedef enum {
    ARGREDUCE_F32 = 0,  /* IEEE binary32, 4-byte aligned */
    ARGREDUCE_F16 = 1,  /* IEEE binary16, 2-byte aligned */
    ARGREDUCE_BF16 = 2, /* bfloat16 (upper half of a binary32), 2-byte aligned */
    ARGREDUCE_F64 = 3,  /* IEEE binary64, 8-byte aligned */
    /* Integer formats: accepted by argreduce_scan_lastaxis only (the other entry points
     * return ARGREDUCE_ERR_UNSUPPORTED_DTYPE); compared exactly. */
    ARGREDUCE_I32 = 4,  /* int32, 4-byte aligned */
    ARGREDUCE_I64 = 5   /* int64, 8-byte aligned */
} argreduce_dtype_t;

typedef enum {
    ARGREDUCE_MAX = 0,      /* ArgMax, ties to the lowest index */
    ARGREDUCE_MIN = 1,      /* ArgMin, ties to the lowest index */
    /* Ties to the HIGHEST index: ONNX's select_last_index = 1, which the first page's
     * Semantics section names and leaves to the CPU. Defined here as the same sequential
     * scan with the non-strict comparison (>= / <=): a later equal element replaces the
     * running best, NaN is still never selected, a NaN at index 0 still yields 0, and a row
     * of all -inf (ArgMax) yields its last index. */
    ARGREDUCE_MAX_LAST = 2,
    ARGREDUCE_MIN_LAST = 3
} argreduce_op_t;

enum {
    ARGREDUCE_OK = 0,
    ARGREDUCE_ERR_INVALID_ARG = -1,      /* null pointer with rows > 0, rows < 0, cols < 1,
                                            bad op, misaligned x or out_idx */
    ARGREDUCE_ERR_UNSUPPORTED_DTYPE = -2,
    ARGREDUCE_ERR_TOO_WIDE = -3,         /* a reduced axis the entry point does not admit:
                                            len > INT32_MAX (argreduce_axis with inner > 1),
                                            cols > INT32_MAX (argreduce_scan_lastaxis), or
                                            more workgroups than a grid holds */
    ARGREDUCE_ERR_SCRATCH_TOO_SMALL = -4,/* scratch_bytes below argreduce_scratch_bytes() */
    ARGREDUCE_ERR_HIP = -5,              /* a HIP call or kernel launch failed */
    ARGREDUCE_ERR_NO_DEVICE = -6         /* no current HIP device to plan for */
};

/*
 * Bytes of scratch that argreduce_lastaxis needs for this shape on the CURRENT device
 * ("[CUDA] Parallelize ArgMax/ArgMin over wide last axes", Description / Approach: the
 * caller allocates the intermediate buffer; its size is bounded by the device's thread
 * capacity, so it stays in the low kilobytes for any shape).
 *
 * Returns 0 when the chosen launch needs no scratch, else 16 bytes (32 for F64) per
 * (row, workgroup) of a split row, or 16 bytes per (row, window) of a row wider than
 * INT32_MAX, plus 15 bytes of slack, so the buffer may start at any byte address. Returns
 * SIZE_MAX on an invalid argument (rows < 0, cols < 1, bad dtype) or when there is no
 * current device.
 */
size_t argreduce_scratch_bytes(int64_t rows, int64_t cols, argreduce_dtype_t dtype);

/*
 * out_idx[r] = ArgMax / ArgMin of row r of x, for r in [0, rows).
 *
 *   x             device pointer to rows * cols elements of `dtype`, row-major, rows
 *                 contiguous (row r starts at element r * cols); aligned to the element
 *                 size. Read only. rows * cols * element size must fit in int64.
 *   rows          >= 0; rows == 0 is a no-op that returns ARGREDUCE_OK.
 *   cols          >= 1 (an empty row has no index). rows * cols may exceed 2^31. Rows wider
 *                 than INT32_MAX are cut into windows of at most 2^30 elements (positions
 *                 stay 32-bit inside a window; "[CUDA] Parallelize ArgMax/ArgMin over wide
 *                 last axes", "Why not int64 positions"); each window's candidate carries
 *                 its 64-bit index to a merge kernel (ARGREDUCE_PATH_WIDE, two dispatches).
 *   out_idx       device pointer to `rows` int64 values, 8-byte aligned. Written only on
 *                 success; each value lies in [0, cols).
 *   scratch       device pointer to at least argreduce_scratch_bytes(rows, cols, dtype)
 *                 bytes, at any byte alignment, with any contents on entry: a row split
 *                 over several workgroups publishes two 8-byte words per workgroup (three
 *                 for F64), each tagged with a per-call nonce, and the call ignores words
 *                 that do not carry its own nonce and an in-range index (arbitrary
 *                 contents pass that filter with probability below 2^-32 per word). May be
 *                 NULL when that figure is 0. The call leaves the words it used zeroed.
 *                 Calls that can run at the same time (on different streams) need
 *                 separate scratch buffers.
 *   scratch_bytes size of the scratch buffer in bytes.
 *   stream        hipStream_t on which all work is enqueued (NULL = default stream).
 *
 * The call returns after enqueuing; results are ready when the stream reaches that point.
 */
int argreduce_lastaxis(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                       argreduce_op_t op, int64_t *out_idx, void *scratch,
                       size_t scratch_bytes, void *stream);

/* ----------------------------------------------------------------------------------------
 * For callers that cannot allocate device memory: code under HIP graph capture that must
 * not call hipMalloc, tight serving loops, harnesses that forbid allocation.
 *
 * argreduce_lastaxis without the scratch arguments: the scratch is a buffer the library
 * holds, a device array of ARGREDUCE_NOALLOC_SCRATCH_BYTES bytes, one copy per device,
 * located on the first call on that device and kept until the process ends. Same
 * arguments otherwise, same results, kernels and status codes; the call allocates and
 * frees nothing. Returns ARGREDUCE_ERR_SCRATCH_TOO_SMALL, before enqueuing anything, when
 * argreduce_scratch_bytes(rows, cols, dtype) exceeds ARGREDUCE_NOALLOC_SCRATCH_BYTES (on
 * MI355X no shape does: the split path needs at most 32 bytes per resident workgroup,
 * 65,551 bytes in all, and rows wider than INT32_MAX a few tens of KiB at any size that
 * fits in memory); ARGREDUCE_ERR_HIP when the buffer cannot be located.
 *
 * Every call on one device shares that device's buffer, which keeps the last call's
 * contents (the next call needs nothing cleared: its words carry a per-call nonce). Calls
 * that can overlap on one device (several streams, several host threads) race on the
 * buffer and may return wrong indices: the caller must order them, e.g. on one stream.
 */
#define ARGREDUCE_NOALLOC_SCRATCH_BYTES (128u * 1024u)
int argreduce_lastaxis_noalloc(const void *x, argreduce_dtype_t dtype, int64_t rows,
                               int64_t cols, argreduce_op_t op, int64_t *out_idx, void *stream);

/* ----------------------------------------------------------------------------------------
 * Launch plan and test hooks. The pages' tests force every dispatch path and simulate
 * devices of several thread capacities ("[CUDA] Parallelize ArgMax/ArgMin over wide last
 * axes", Description / Testing); these entry points expose the same controls.
 */

typedef enum {
    ARGREDUCE_PATH_AUTO = -1,
    ARGREDUCE_PATH_SUBWAVE = 0, /* a group of 1..64 lanes of one wavefront per row */
    ARGREDUCE_PATH_BLOCK = 1,   /* one workgroup per row, rows looped over the grid */
    ARGREDUCE_PATH_SPLIT = 2,   /* several workgroups per row; the highest-id one merges */
    ARGREDUCE_PATH_AXIS = 3,    /* middle-axis reduction: a tile of consecutive outputs per
                                   workgroup, thread rows along the axis (argreduce_axis) */
    ARGREDUCE_PATH_SCAN = 4,    /* cumulative scan: a tile of a row per workgroup, tiles of
                                   a row chained by look-back (argreduce_scan_lastaxis) */
    ARGREDUCE_PATH_WIDE = 5,    /* rows wider than INT32_MAX: windows of <= 2^30 elements,
                                   one workgroup each, merged by a second dispatch */
    ARGREDUCE_PATH_THREAD = 6   /* forced only, never chosen: one lane scans each row alone,
                                   the pages' serial thread-per-row kernel, for a "before"
                                   timing from the same library ("[CUDA] Parallelize
                                   ArgMax/ArgMin over wide last axes", Verification log);
                                   its plan reads as ARGREDUCE_PATH_SUBWAVE with one lane */
} argreduce_path_t;

typedef struct {
    int32_t path;             /* argreduce_path_t */
    int32_t lanes_per_row;    /* lanes that scan one row */
    int32_t blocks_per_row;   /* workgroups per row (1 unless SPLIT) */
    int32_t block_threads;    /* threads per workgroup */
    int64_t grid_blocks;      /* workgroups launched */
    int64_t grid_rows;        /* rows in flight at once (rows beyond are looped over) */
    int32_t unroll;           /* loads each lane keeps in flight per step */
    int32_t outputs_per_block;/* outputs one workgroup produces at a time */
    int64_t device_threads;   /* thread capacity the plan was made for */
    size_t scratch_bytes;     /* == argreduce_scratch_bytes() for the same arguments */
    int32_t load_bytes;       /* bytes of one lane load in the body of the scan: 16, or the
                                 element size for an AXIS plan whose `inner` row is not a
                                 multiple of 16 bytes */
    int32_t dispatches;       /* kernels one call launches: 1, or 2 for an AXIS or WIDE plan
                                 whose workgroups store partials that a second kernel merges */
    int64_t window;           /* WIDE: elements per window (one workgroup each); else 0 */
} argreduce_plan_t;

/* The plan argreduce_lastaxis would use for these arguments on the current device. */
int argreduce_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype, argreduce_plan_t *plan);

/* Plan as if the device held `threads` resident threads (0 = the real device). Process-wide.
 * Lets tests reach the row-loop and split paths of devices of other sizes, and lets
 * argreduce_plan / argreduce_scratch_bytes run without a GPU. */
int argreduce_debug_set_capacity(int64_t threads);

/* Force one path (ARGREDUCE_PATH_AUTO restores the automatic choice). Process-wide.
 * A forced path keeps its own geometry rules; a forced SPLIT uses at least two workgroups
 * per row, however short the row; a forced WIDE cuts every row into windows (of the size
 * set below, else the automatic one). SUBWAVE, BLOCK, SPLIT, WIDE and THREAD can be
 * forced (THREAD: 16-byte loads, one in flight per lane, so milliseconds per call on rows
 * of 10^5 elements). */
int argreduce_debug_force_path(int path);

/* Force the split path's geometry for every last-axis plan: blocks_per_row workgroups per
 * row (2 .. the plan's maximum, 1024) and unroll 16-byte loads per lane per step (1, 2, 4 or
 * 8); rows longer than one step take several. blocks_per_row = 0 restores the automatic
 * plans. Process-wide; for measuring plan alternatives (a forced grid may exceed what is
 * resident at once, and then relies on the in-order start of workgroups). Returns
 * ARGREDUCE_ERR_INVALID_ARG for other values. */
int argreduce_debug_force_split(int64_t blocks_per_row, int unroll);

/* Window size of the WIDE path in elements, 1 .. 2^30 (0 = automatic). Process-wide. Lets
 * tests run the windowed path on rows small enough for the CPU oracle. */
int argreduce_debug_set_window(int64_t elements);

/* ----------------------------------------------------------------------------------------
 * Reduction over a middle axis.
 *
 * out_idx[o * inner + i] = ArgMax / ArgMin over r in [0, len) of x[o][r][i], for a contiguous
 * row-major [outer, len, inner] tensor (flat position (o * len + r) * inner + i): ONNX's
 * ArgMax/ArgMin over any axis after collapsing the dimensions before it into `outer` and
 * those after it into `inner`. The first page (Semantics) notes that its CUDA provider
 * sends non-last axes to a fallback; the semantics here are exactly those of
 * argreduce_lastaxis applied to each (o, i) column, for every op. inner == 1 IS
 * argreduce_lastaxis (rows = outer, cols = len), with the same scratch and plan.
 *
 *   outer >= 0 (0 is a no-op), 1 <= len <= INT32_MAX, inner >= 1. Pointers, alignment,
 *   scratch, stream and status codes as for argreduce_lastaxis; out_idx holds
 *   outer * inner int64 values.
 *
 *   When few outputs leave the device idle, the axis is split over several workgroups per
 *   tile of outputs: each stores a (value, index) partial per output in scratch, and a
 *   second kernel, enqueued on the same stream, merges them (the plan's `dispatches` is
 *   then 2; nothing waits on another workgroup, so no output is ever -1). 16-byte loads
 *   are used when inner * element size is a multiple of 16 and x is 16-byte aligned; the
 *   scratch size returned covers both cases.
 */
size_t argreduce_axis_scratch_bytes(int64_t outer, int64_t len, int64_t inner,
                                    argreduce_dtype_t dtype);
int argreduce_axis(const void *x, argreduce_dtype_t dtype, int64_t outer, int64_t len,
                   int64_t inner, argreduce_op_t op, int64_t *out_idx, void *scratch,
                   size_t scratch_bytes, void *stream);
/* The plan argreduce_axis would use for a 16-byte aligned x (path ARGREDUCE_PATH_AXIS
 * unless inner == 1). */
int argreduce_axis_plan(int64_t outer, int64_t len, int64_t inner, argreduce_dtype_t dtype,
                        argreduce_plan_t *plan);

/* ----------------------------------------------------------------------------------------
 * Cumulative extremum with indices along the last axis: cummax / cummin.
 *
 * The PaddlePaddle issue on the cummax/cummin CUDA kernel (its reproduction scans the last
 * axis of [rows, cols] tensors; its fix proposals describe the operator as a (value,
 * index) reduce with ArgMax semantics, ties to the earlier index). For every row r and
 * position j:
 *   out_idx[r*cols + j]    = the index the ArgMax (op ARGREDUCE_MAX: cummax) / ArgMin
 *                            (ARGREDUCE_MIN: cummin) scan of x[r][0..j] returns, with the
 *                            semantics of argreduce_lastaxis: ties keep the earlier index,
 *                            a NaN after position 0 is never taken, a NaN at position 0
 *                            holds for the whole row (index 0);
 *   out_values[r*cols + j] = a copy of the element x[r][out_idx[r*cols + j]] (same format
 *                            and bits as x; a leading NaN keeps its own bit pattern).
 *
 *   Formats: F32, F16, BF16, F64, I32, I64 (integers compared exactly). Ops: ARGREDUCE_MAX
 *   and ARGREDUCE_MIN only. 1 <= cols <= INT32_MAX, rows >= 0 (0 is a no-op). x and
 *   out_values aligned to the element size, out_idx to 8 bytes; 16-byte aligned rows
 *   (x, out_values and out_idx 16-byte aligned and cols * element size a multiple of 16)
 *   move as 16-byte vectors. out_values and out_idx hold rows * cols elements each and must
 *   not overlap x.
 *
 *   Scratch: rows longer than one tile (argreduce_scan_plan's outputs_per_block elements)
 *   chain their tiles through per-tile state words in scratch (any contents on entry);
 *   argreduce_scan_scratch_bytes gives the size (0 when every row fits in one tile;
 *   SIZE_MAX for invalid arguments). One dispatch per call; when `stream` is being
 *   captured into a HIP graph, a small kernel that clears the state words is enqueued
 *   before it, so that graph replays stay correct. Calls that can run at the same time
 *   need separate scratch buffers. Status codes as argreduce_lastaxis;
 *   ARGREDUCE_ERR_TOO_WIDE also when rows * tiles per row exceeds 2^32 - 1.
 */
size_t argreduce_scan_scratch_bytes(int64_t rows, int64_t cols, argreduce_dtype_t dtype);
int argreduce_scan_lastaxis(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                            argreduce_op_t op, void *out_values, int64_t *out_idx,
                            void *scratch, size_t scratch_bytes, void *stream);
/* The plan argreduce_scan_lastaxis would use for 16-byte aligned buffers (path
 * ARGREDUCE_PATH_SCAN; blocks_per_row = tiles per row, outputs_per_block = elements per
 * tile). */
int argreduce_scan_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype,
                        argreduce_plan_t *plan);

/* ----------------------------------------------------------------------------------------
 * Logits operators: a softmax over the same last axis that ArgMax answers from. Logits are a
 * [rows, cols] tensor of f32, f16 or bf16 (other formats: ARGREDUCE_ERR_UNSUPPORTED_DTYPE), row
 * r starting at element r * row_stride (row_stride >= cols; ignored for rows <= 1), so a padded
 * vocabulary or a slice of a sequence needs no copy. With temperature T > 0:
 *
 *     p_j = exp(x_j / T) / sum_i exp(x_i / T)
 *
 * Statistics, sums and outputs are binary32 (a log probability below its range is -inf); a
 * gradient is computed in binary32 and rounded once, to the nearest even value of the logits'
 * format. Results do not depend on the order in which workgroups run: the same call gives the
 * same bits.
 *
 *   - A logit of -inf is masked: probability 0, never an alternative, and no gradient but by its
 *     own log probability, where it is the row's token (grad_logprob / T) or has a teacher's weight
 *     q (-grad_loss q / T). The lowest finite value is an ordinary value.
 *   - A row whose every logit is -inf has log probabilities -inf, entropy 0, no alternatives
 *     and gradient 0.
 *   - A row with a NaN or +inf has NaN log probabilities, entropy and gradient and no
 *     alternatives.
 *   - Rows are independent: a row's contents change no other row's results.
 *
 * rows >= 0 (0 is a no-op); 1 <= cols <= INT32_MAX, rows <= INT32_MAX, row_stride <= UINT32_MAX
 * (else ARGREDUCE_ERR_TOO_WIDE, also where the logits would span 2^48 bytes or more, or one of the
 * call's own launches would hold 2^32 threads or more); 2^-60 <= T <= 2^60. x is aligned to its elements, int64 arrays to 8 and float
 * arrays to 4 bytes. Inputs, outputs and scratch must not overlap. Scratch
 * (argreduce_*_scratch_bytes, which depends on the shape only) is as for argreduce_lastaxis: any
 * contents, any byte alignment, not shared by calls that can run at the same time. Token ids are
 * read on the device and cannot be refused by the call: no id makes a kernel read or write out
 * of range (what each gives is stated below). Everything else as for argreduce_lastaxis: the
 * caller's stream, status codes before anything is enqueued, calls may be captured.
 */
#define ARGREDUCE_TOP_MAX 64        /* alternatives per row */
#define ARGREDUCE_TEACHER_MAX 1024  /* teacher entries per row */
/* argreduce_logprobs: the entropy in a row of its own too (a value that no caller's "true" has) */
#define ARGREDUCE_ENTROPY_APART 0x61706172

/*
 * Log probabilities of given tokens, with entropy and the top alternatives.
 *
 *   tokens        [rows]: the token of each row. A negative one leaves the row out: its logits
 *                 do not matter, log probability and entropy are 0, and it has no alternatives.
 *                 One >= cols gives a NaN log probability (and a NaN gradient, unless every
 *                 logit of the row is -inf).
 *   entropy       non-zero: compute the entropy; 0: row 1 of stats is NaN. ARGREDUCE_ENTROPY_APART:
 *                 the entropy also goes to a fifth row of stats, which is [5, rows] then, for a
 *                 caller who hands that row out to be written over (argreduce_logprobs_grad reads
 *                 rows 1 to 3).
 *   top           alternatives per row, 0 .. ARGREDUCE_TOP_MAX.
 *   stats         [4, rows] out: ln p of the token; entropy -sum p ln p; and two rows for
 *                 argreduce_logprobs_grad (the row's maximum, and log2 sum exp((x - max) / T)).
 *   top_logprobs  [rows, top] out, top_tokens [rows, top] out (NULL if top is 0): the largest
 *                 logits' ln p and positions, largest first, equal logits by position (-0 and +0
 *                 are equal). Entries past the row's unmasked logits are -inf and -1 (NaN and
 *                 -1 in a row with NaN or +inf).
 */
size_t argreduce_logprobs_scratch_bytes(int64_t rows, int64_t cols, argreduce_dtype_t dtype);
int argreduce_logprobs(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                       int64_t row_stride, const int64_t *tokens, float temperature, int32_t entropy,
                       int32_t top, float *stats, float *top_logprobs, int64_t *top_tokens,
                       void *scratch, size_t scratch_bytes, void *stream);
/* The plan of argreduce_logprobs without alternatives, for contiguous rows in an aligned tensor:
 * SUBWAVE (a group of lanes or a wavefront per row), BLOCK (a workgroup per row) or SPLIT (several
 * workgroups per row, merged by a second dispatch; no workgroup waits on another). */
int argreduce_logprobs_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype,
                            argreduce_plan_t *plan);

/*
 * Gradient of sum_r (grad_logprob[r] * ln p of the token + grad_entropy[r] * entropy) with
 * respect to the logits, with t the row's token and H its entropy
 *
 *     grad_j = (grad_logprob (delta_jt - p_j) - grad_entropy p_j (ln p_j + H)) / T:
 *
 * [rows, cols], contiguous, in the logits' format, every element written; 0 in rows left out and in
 * rows of -inf. x, tokens and temperature are those of the
 * forward call, stats what it wrote (with entropy if grad_entropy is not NULL).
 */
int argreduce_logprobs_grad(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                            int64_t row_stride, const int64_t *tokens, float temperature,
                            const float *stats, const float *grad_logprob, const float *grad_entropy,
                            void *grad, void *stream);

/*
 * Distillation from a teacher's top logits: per row the divergence KL(q || p) of the student's
 * p (over all cols) from the teacher's q, the softmax at the same temperature over the row's k
 * teacher entries,
 *
 *     q_i = exp(v_i / T) / sum_l exp(v_l / T),   loss = sum_i q_i (ln q_i - ln p_{id_i}).
 *
 *   teacher_tokens  [rows, k]: ids. A negative one marks an absent entry (its value does not
 *                   matter). The same id twice: both entries count. An id >= cols with weight
 *                   makes the row's loss and gradient NaN, whatever its logits are.
 *   teacher_logits  [rows, k] f32: logits or log probabilities; -inf has no weight, and neither has
 *                   an entry whose q_i underflows in binary32 (below 2^-126). The outputs
 *                   of argreduce_logprobs (top_tokens, top_logprobs) can be passed as they are.
 *                   A NaN (or +inf) of a present entry makes loss and gradient NaN.
 *   k               1 .. ARGREDUCE_TEACHER_MAX.
 *   stats           [5, rows] out: the loss, and four rows for argreduce_distill_grad.
 *
 * A row without an entry of weight has loss 0 and gradient 0, its logits do not matter. A row
 * of -inf has loss +inf and gradient 0; a masked logit at an id with weight gives loss +inf.
 */
size_t argreduce_distill_scratch_bytes(int64_t rows, int64_t cols, argreduce_dtype_t dtype);
int argreduce_distill(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                      int64_t row_stride, int32_t k, const int64_t *teacher_tokens,
                      const float *teacher_logits, float temperature, float *stats, void *scratch,
                      size_t scratch_bytes, void *stream);
/* The plan of argreduce_distill with one entry, likewise. */
int argreduce_distill_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype,
                           argreduce_plan_t *plan);

/* Gradient of sum_r grad_loss[r] * loss[r]: grad[r][j] = grad_loss[r] (p_j - q_j) / T, [rows,
 * cols], contiguous, in the logits' format, every element written. Inputs as in the forward
 * call, stats what it wrote. */
int argreduce_distill_grad(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                           int64_t row_stride, int32_t k, const int64_t *teacher_tokens,
                           const float *teacher_logits, float temperature, const float *stats,
                           const float *grad_loss, void *grad, void *stream);

/* Both at once, for weights known before the loss: stats as argreduce_distill, grad as
 * argreduce_distill_grad with grad_loss = weights. The logits are read from HBM once. Scratch as
 * for argreduce_distill. */
int argreduce_distill_step(const void *x, argreduce_dtype_t dtype, int64_t rows, int64_t cols,
                           int64_t row_stride, int32_t k, const int64_t *teacher_tokens,
                           const float *teacher_logits, float temperature, const float *weights,
                           float *stats, void *grad, void *scratch, size_t scratch_bytes,
                           void *stream);

/* ----------------------------------------------------------------------------------------
 * Beam search: the step that chooses how a search goes on, and the reordering of what the model
 * keeps for every beam.
 *
 * Step. Row g * beams + b of the logits (format, stride, -inf, NaN and +inf as for the logits
 * operators) belongs to beam b of group g, whose score is a sum of log probabilities. A beam offers
 * for every unmasked token v the value
 *
 *     scores[g][b] + ln softmax(x / T)[v],
 *
 * and the step returns the `width` largest values of each group, largest first, equal ones by beam,
 * then by logit and by token, with their beams ("parents") and tokens. Logits of one row keep their order
 * (equal logits by token); values of different rows are compared in binary64 and rounded once, to binary32. Their
 * sums of exponentials are of binary32's precision, with a relative error of about 1e-7 (over rows of 64 to 202048
 * logits the root of its mean square was 0.3e-7 to 1.0e-7, the largest 1.0e-6), and the same in equal rows: values
 * of different rows that lie closer than that can come in either order, equal ones of equal rows come by beam.
 *
 *   scores       [groups, beams]. A beam whose score is -inf, +inf or NaN offers nothing, nor does a
 *                row with a NaN or +inf, or of -inf only. Rows that offer nothing by their score
 *                or because they have ended are not read.
 *   ended        [groups, beams] bytes or NULL: a non-zero one marks a beam that is finished: it offers
 *                one value, its score, with the token `end_token`.
 *   end_token    0 .. cols - 1, or negative: none (only without `ended`).
 *   temperature  2^-60 <= T <= 2^60.
 *   beams, width 1 .. ARGREDUCE_BEAM_MAX; groups * 256 <= INT32_MAX.
 *   out          argreduce_beam_out_bytes bytes, 8-byte aligned: parents int64 [groups, width], tokens
 *                int64 [groups, width], scores float [groups, width], ended bytes [groups, width] (1
 *                where the token is end_token), one after another. Where a group offers fewer values the
 *                rest is -1, -1, -inf and 0.
 *
 * Scratch, streams, captures and status codes as for the logits operators.
 */
#define ARGREDUCE_BEAM_MAX 64
size_t argreduce_beam_scratch_bytes(int64_t groups, int64_t beams, int64_t cols, argreduce_dtype_t dtype,
                                    int32_t width);
size_t argreduce_beam_out_bytes(int64_t groups, int32_t width);
int argreduce_beam_step(const void *x, argreduce_dtype_t dtype, int64_t groups, int64_t beams,
                        int64_t cols, int64_t row_stride, const float *scores, const uint8_t *ended,
                        int64_t end_token, double temperature, int32_t width, void *out, void *scratch,
                        size_t scratch_bytes, void *stream);
/* The plan of argreduce_beam_step: SUBWAVE (a wavefront per group of beams, four to a workgroup), BLOCK (a
 * workgroup per row, or with block_threads 64 a wavefront per row) or SPLIT (a workgroup per slice, blocks_per_row
 * slices to a row). */
int argreduce_beam_plan(int64_t groups, int64_t beams, int64_t cols, argreduce_dtype_t dtype, int32_t width,
                        argreduce_plan_t *plan);

/*
 * Reordering, in place: for every state, group g, beam b and position t in [first, last) of the group,
 *
 *     state[g][b][..., t, ...] = (state before the call)[g][parents[g][b]][..., t, ...],
 *
 * the other positions stay as they are. A state is a tensor of any element type, addressed in bytes:
 * element run (g, b, o, t) of `inner` contiguous bytes lies at base + g * group_stride + b * beam_stride
 * + o * outer_stride + t * position_stride. No two runs of a state may share a byte (else
 * ARGREDUCE_ERR_INVALID_ARG), nor may two states (not checked).
 *
 *   parents   [groups, beams]; one that is negative or >= beams leaves its beam as it is.
 *   first     [groups] int64, or NULL: first_value for all groups. Positions below 0 count as 0,
 *   last      likewise;               those past the state's as its last.
 *
 * argreduce_reorder_plan checks the states (in host memory) once; argreduce_reorder takes the plan, and
 * `table`, the same states in device memory. Beams that stay are neither read nor written; no scratch.
 */
#define ARGREDUCE_STATES_MAX 4096
typedef struct {
    void *base; /* device memory */
    int64_t group_stride, beam_stride;
    int64_t outer, outer_stride;
    int64_t positions, position_stride;
    int64_t inner;
} argreduce_state_t;
typedef struct {
    int32_t tensors, beams;
    int64_t groups;
    int64_t positions;      /* the most that a state has */
    int64_t position_bytes; /* of one beam and position: the most that a state has */
} argreduce_reorder_t;
int argreduce_reorder_plan(const argreduce_state_t *states, int32_t tensors, int64_t groups, int64_t beams,
                           argreduce_reorder_t *plan);
int argreduce_reorder(const argreduce_reorder_t *plan, const argreduce_state_t *table, const int64_t *parents,
                      const int64_t *first, const int64_t *last, int64_t first_value, int64_t last_value,
                      void *stream);

/* ----------------------------------------------------------------------------------------
 * Expert routing: the choice of `top` of the experts for every token from a router's logits, with
 * weights, per-expert counts and two losses, and the gradient.
 *
 * Row g * tokens + t of the logits [.., experts] (format, stride and -inf as for the logits operators)
 * belongs to token t of group g (a sequence, or all tokens of a batch). With p = softmax(x) of a token, c_e
 * the number of tokens of the group that chose expert e and n the number of its tokens:
 *
 *     chosen   the `top` largest logits, largest first, equal ones by expert
 *     weights  p of the chosen; with renormalize divided by their sum
 *     balance  experts / (top n^2) sum_e c_e sum_t p_te
 *     z        1 / n sum_t (ln sum_e exp x_te)^2
 *
 *   - A token that `live` marks with 0 is left out, and so is one whose every logit is -inf: chosen -1,
 *     weights 0, no part in counts, n and losses, and gradient 0. The logits of the former are not read.
 *   - Past the experts that are not masked: chosen -1, weights 0.
 *   - A live token with a NaN or +inf: chosen -2, weights NaN, no counts; the group's losses are NaN, and
 *     the token's own gradient.
 *   - A group without tokens has losses 0.
 *
 *   live      [groups, tokens] bytes or NULL.
 *   top       1 .. min(experts, ARGREDUCE_ROUTE_TOP_MAX); experts 1 .. ARGREDUCE_EXPERTS_MAX.
 *   weights   [groups, tokens, top] out; chosen [groups, tokens, top] out.
 *   totals    argreduce_route_totals_bytes bytes out, 8-byte aligned: counts int64 [groups, experts],
 *             tokens (n) int64 [groups], balance float [groups], z float [groups], one after another.
 *
 * Sums are in binary32 in a workgroup and in binary64 between them, in one order; z is +inf where a sum
 * leaves binary32.
 */
#define ARGREDUCE_EXPERTS_MAX 1024
#define ARGREDUCE_ROUTE_TOP_MAX 64
size_t argreduce_route_scratch_bytes(int64_t groups, int64_t tokens, int64_t experts, argreduce_dtype_t dtype);
size_t argreduce_route_totals_bytes(int64_t groups, int64_t experts);
int argreduce_route(const void *x, argreduce_dtype_t dtype, int64_t groups, int64_t tokens, int64_t experts,
                    int64_t row_stride, const uint8_t *live, int32_t top, int32_t renormalize, float *weights,
                    int64_t *chosen, void *totals, void *scratch, size_t scratch_bytes, void *stream);
/* The plan of argreduce_route (path SUBWAVE: lanes_per_row lanes of a wavefront per token). */
int argreduce_route_plan(int64_t groups, int64_t tokens, int64_t experts, argreduce_dtype_t dtype,
                         argreduce_plan_t *plan);

/* Gradient of sum (g_weights * weights) + sum_g (g_balance * balance + g_z * z) with respect to the
 * logits: [groups, tokens, experts], contiguous, in the logits' format, every element written. Choice and
 * counts are constants. x, top and renormalize are those of the forward call, chosen and totals what it
 * wrote (of totals the counts and n are read). g_weights [groups, tokens, top], g_balance [groups] and g_z
 * [groups] may be NULL: 0. An expert number beyond the row has no gradient. */
int argreduce_route_grad(const void *x, argreduce_dtype_t dtype, int64_t groups, int64_t tokens, int64_t experts,
                         int64_t row_stride, int32_t top, int32_t renormalize, const int64_t *chosen,
                         const void *totals, const float *g_weights, const float *g_balance, const float *g_z,
                         void *grad, void *stream);

/* Measurement hook: the launch floor. Enqueues one empty kernel (one workgroup of 64
 * threads) on `stream`, the same way argreduce_lastaxis enqueues its kernels, so that a
 * benchmark can time bare launch latency in the same harness ("[CUDA] Parallelize
 * ArgMax/ArgMin over wide last axes", Description / Results: per-call times include the
 * launch). Returns ARGREDUCE_OK or ARGREDUCE_ERR_HIP. */
int argreduce_debug_launch_empty(void *stream);

/* Measurement hook: the floor of a call that delivers a result. Enqueues one workgroup of
 * a kernel that takes one pointer argument and stores one int64 (0) at `out` (8-byte
 * aligned device memory) — the same launch and kernel-argument cost as every entry point,
 * with no data read. Returns ARGREDUCE_OK, ARGREDUCE_ERR_INVALID_ARG or ARGREDUCE_ERR_HIP. */
int argreduce_debug_launch_store(int64_t *out, void *stream);

/* Measurement hook: the practical read roofline. Enqueues on `stream` a plain streaming
 * read of `bytes` (a non-zero multiple of 16) at `x` (16-byte aligned device memory) by
 * `grid` workgroups of 256 threads (1 .. 65536): grid-stride 16-byte nontemporal loads, four
 * in flight per lane, folded with XOR. `out` (device memory of `grid` uint32 words, 4-byte
 * aligned) is written only when a workgroup's XOR equals one fixed 32-bit pattern, so in
 * practice nothing is written; the kernel does none of the reduction's work. Returns
 * ARGREDUCE_OK, ARGREDUCE_ERR_INVALID_ARG or ARGREDUCE_ERR_HIP. */
int argreduce_debug_launch_read(const void *x, size_t bytes, uint32_t *out, int64_t grid,
                                void *stream);

/* Test hook for the bounded waits (the split ArgMax path's finalizing workgroup, the scan's
 * look-back): polls of one published word before the wait gives up, the affected outputs
 * become -1 and argreduce_wait_timeouts counts it (0 restores the default, 2^20 polls). Process-wide. With a tiny limit
 * a wait can give up although nothing is wrong; this lets tests drive the time-out path
 * from the host while every kernel still ends normally. */
int argreduce_debug_set_spin_limit(uint32_t polls);

/* Bounded waits that gave up on the CURRENT device since the library was loaded. Two kinds
 * of workgroup wait for results that other workgroups of the same launch publish: the
 * finalizing workgroup of a split row (argreduce_lastaxis, "[CUDA] Parallelize ArgMax/ArgMin
 * over wide last axes", Description / Approach: the last block merges the partials) and a
 * tile of a long cumulative-scan row (argreduce_scan_lastaxis). Each stops after a bounded
 * number of polls (argreduce_debug_set_spin_limit); its outputs then hold -1 and the count
 * goes up by one per row (split) or per tile (scan). No wait is expected to give up unless a
 * test forces a tiny limit; a caller that must rule it out compares the count before and
 * after its calls. Copies the device's counter to *count synchronously, after the work
 * already enqueued on the default stream (call it off the hot path). Returns ARGREDUCE_OK,
 * ARGREDUCE_ERR_INVALID_ARG (count NULL), ARGREDUCE_ERR_NO_DEVICE or ARGREDUCE_ERR_HIP. */
int argreduce_wait_timeouts(uint64_t *count);

/* Measurement hook: when both are non-NULL, every later call launches its main kernel
 * (not a merge or clear kernel) with `start` recorded just before and
 * `stop` just after it on the same stream (hipEvent_t values created by the caller with
 * timing enabled); NULL, NULL turns this off. Process-wide; for benchmarks only. */
int argreduce_debug_set_kernel_events(void *start, void *stop);

#ifdef __cplusplus
}
#endif

#endif /* ARGREDUCE_H */
