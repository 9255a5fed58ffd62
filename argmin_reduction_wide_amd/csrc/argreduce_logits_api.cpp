// C ABI of the logits operators: argument checks, launch plans and scratch sizes. Declarations
// and the contract are in include/argreduce.h, the kernels in argreduce_logits.hip.
#include <hip/hip_runtime_api.h>

#include "argreduce_checks.hpp"

namespace argreduce {
namespace {

// Logits of up to this size are left in the 256 MiB Infinity Cache (struct Span). Log probabilities
// and their gradient of f32 rows of 32003, in us, logits left there and not: 4 MiB 9.5 and 11.6, 16
// MiB 15.0 and 17.7, 48 MiB 30.9 and 34.9, 64 MiB 46.4 and 46.0, 96 MiB 63.4 and 63.2, 128 MiB 85.6
// and 80.8, 256 MiB 164 and 151; the forward pass alone 4.6 and 5.5, 6.1 and 6.3, 11.9 and 11.7, 16.9
// and 15.9, 21.9 and 20.8, 27.7 and 26.2, 50.5 and 47.1. (bf16 within 3 us of these.)
constexpr int64_t kKeepBytes = int64_t{64} << 20;

// Checks of the arguments that every call takes; fills *a. Row stride: see the header.
int check_logits(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride,
                 float temperature, LogitsArgs* a) {
    const int rc = check_rows(x, dtype, rows, cols, stride);
    if (rc != ARGREDUCE_OK) return rc;
    // powers of two far inside the range of a float: log2(e) / T and its products stay normal
    if (!(temperature >= 0x1p-60f && temperature <= 0x1p60f)) return ARGREDUCE_ERR_INVALID_ARG;
    *a = LogitsArgs{x, dtype, rows, cols, rows > 1 ? stride : cols,
                    static_cast<float>(1.4426950408889634 / static_cast<double>(temperature)),
                    rows <= kKeepBytes / logits_elem_size(dtype) / cols};
    return ARGREDUCE_OK;
}

// Workgroups of the distillation step: as many as its registers (at most 128 per lane, 64 if it
// holds two vectors) and LDS let the CUs hold at once; each goes through several rows. The kernel
// takes the number in 16 bits.
int64_t step_blocks(int64_t cap, int team, int held, int k) {
    int64_t per_cu = team == 1024 ? 1 : team == 512 ? 2 : held > 2 ? 4 : 8;
    const size_t entries = entries_lds(team == 64 ? kBlock / 64 : 1, step_rows(team), k, true);
    const int64_t lds = static_cast<int64_t>(entries) + 1024;
    per_cu = std::min(per_cu, kLdsPerCu / lds);
    const int64_t cus = cap / kThreadsPerCu > 0 ? cap / kThreadsPerCu : 1;
    return per_cu * cus < 65535 ? per_cu * cus : 65535;
}

// Teacher entries, at most, of a row left to one wavefront: four rows' entries and tables then take
// 24 KiB of LDS. (A workgroup per row has a lane for each entry, and is slower: [21454,251] f16 with
// 130 entries, loss and gradient, 41 us by a wavefront, 153 by 256 lanes.)
constexpr int kWaveEntries = 256;

// What a plan is for.
enum Use { kLogprobs, kLogprobsTop, kDistill, kDistillStep };

// Rows of up to this many vectors (160 KiB, in a distillation step 256 KiB) are left to one
// workgroup each, however few they are: at about that length its kernel takes as long as the split
// ones and the gaps between them, with fewer launches. One bf16 row of 79000, statistics: 7.0 us,
// split 3.3 + 1.8; with 5 alternatives 10.7, split 3.3 + 5.9; step of 100 rows of 129000: 21.9 us,
// split 6.6 + 4.0 + 9.8.
constexpr int64_t kOneBlockVecs = 10240;
constexpr int64_t kOneBlockStepVecs = 16384;

// Scratch depends on the shape alone, so only the choices among plans without any go by
// `vec_rows` (every row starts on a 16-byte boundary).
// `k`: teacher entries (0: none).
int make_logits_plan(int dtype, int64_t rows, int64_t cols, Use use, int k, bool vec_rows,
                     LogitsPlan* p) {
    int rc = check_logits_shape(dtype, rows, cols);
    if (rc != ARGREDUCE_OK) return rc;
    int64_t cap = 0;
    rc = plan_device_threads(&cap);
    if (rc != ARGREDUCE_OK) return rc;
    const int64_t es = logits_elem_size(dtype);
    const int64_t rows1 = rows > 0 ? rows : 1;
    const int64_t vecs = span_vecs(cols, es);
    const int64_t cap_blocks = cap / kBlock > 0 ? cap / kBlock : 1;
    *p = LogitsPlan{};
    p->device_threads = cap;
    p->parts = 1;
    // Rows held by a group of lanes, a vector each, and at most four teacher entries per lane.
    // (Alternatives too, though they are taken one by one there: [65536,64] f16 16 us with 4 of
    // them, 39 with 30, and 61 and 70 with a wavefront per row and its selection.)
    const int64_t held = vec_rows ? ceil_div(cols * es, 16) : vecs;  // vectors a row lies in
    const int64_t lanes = next_pow2(std::max<int64_t>({held, ceil_div(k, 4), 4}));
    if (lanes <= 32) {
        p->path = ARGREDUCE_PATH_SUBWAVE;
        p->team = static_cast<int>(lanes);
        p->grid_blocks = ceil_div(rows1, kBlock / lanes);
        return grid_too_large(p->grid_blocks, kBlock) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
    }
    // a wavefront per row: up to four vectors per lane; in a distillation step up to the eight that
    // it holds ([19940,2312] f16, 291 vectors: 256 lanes 152 us, see the step's figures below).
    // Log probabilities of [49539,2032] bf16, 254 vectors: 37 us, 256 lanes 60; with 16 alternatives
    // 70 and 157. (Longer rows would gain too: of [31457,3200] 35 and 49, of [15728,6400] 35 and 39.)
    if (vecs <= (use == kDistillStep ? 512 : 256) && k <= kWaveEntries) {
        p->path = ARGREDUCE_PATH_SUBWAVE;
        p->team = 64;
        p->grid_blocks = ceil_div(rows1, kBlock / 64);
        if (use == kDistillStep) {
            p->held = vecs <= 128 ? 2 : 8;
            const int64_t most = step_blocks(cap, p->team, p->held, k);
            p->grid_blocks = p->grid_blocks < most ? p->grid_blocks : most;
        }
        return grid_too_large(p->grid_blocks, kBlock) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
    }
    // Long rows too few to give every second CU one: split, in one device wave.
    const int64_t one_block = use == kDistillStep ? kOneBlockStepVecs : kOneBlockVecs;
    if (vecs > one_block && rows1 <= cap / kThreadsPerCu / 2) {
        int64_t parts = ceil_div(vecs, kPartThreads * kPartUnroll);
        const int64_t most = cap_blocks / rows1;
        parts = parts < most ? parts : most;
        parts = parts < kMaxParts ? parts : kMaxParts;
        p->path = ARGREDUCE_PATH_SPLIT;
        p->team = kPartThreads;
        p->parts = static_cast<int>(parts);
        p->grid_blocks = rows1 * parts;
        p->scratch_bytes = 15 + static_cast<size_t>(rows1) * static_cast<size_t>(parts) * part_bytes();
        return ARGREDUCE_OK;
    }
    p->path = ARGREDUCE_PATH_BLOCK;
    if (use == kDistillStep)
        // One workgroup per CU where there are no more rows than CUs; else 8 vectors per lane of the
        // fewest lanes that hold the row, then 16. Measured with 64 entries, lanes x vectors: [4096,
        // 16000] bf16 256 x 8 59 us, 512 x 8 83; [8192,30000] 512 x 8 255, 256 x 16 264, 1024 x 8
        // 381; [4096,60000] 512 x 16 245, 1024 x 8 263; [4096,128256] 1024 x 16 477, 512 x 16 544.
        p->team = rows1 * kThreadsPerCu <= cap && vecs > 8 * 256 ? 1024
                  : vecs <= 8 * 256                             ? 256
                  : vecs <= 16 * 512                            ? 512
                                                                : 1024;
    // The figures below: bf16 rows, us by 256, 512 and 1024 lanes; after the semicolon with 16
    // alternatives.
    else if (vecs > 2048 && rows1 * 1024 <= cap)
        // The whole device in one wave of workgroups. [256,16320], 2040 vectors: 4.7, 4.9, 4.8; 9.2,
        // 8.2, 8.5. [256,32720]: 7.2, 6.6, 7.0; 14.1, 10.9, 10.2. [64,72000]: 9.0, 7.0, 6.8; 17.7, 11.9,
        // 11.1.
        p->team = 1024;
    else
        // [6168,16320], 2040 vectors: 33.9, 35.1, 42.2; 45.4, 55.7, 88.3. [3700,27200], 3400: 34.7, 32.5,
        // 39.5; 44.0, 47.0, 65.9. [2097,48000], 6000: 36.8, 34.2, 34.5; 48.2, 44.6, 50.0.
        p->team = vecs > (use == kLogprobsTop ? 4096 : 3000) ? 512 : 256;
    p->grid_blocks = rows1;
    if (use == kDistillStep) {
        p->held = vecs > 8 * p->team ? 16 : 8;
        const int64_t most = step_blocks(cap, p->team, p->held, k);
        p->grid_blocks = rows1 < most ? rows1 : most;
    }
    return grid_too_large(p->grid_blocks, p->team) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
}

// `k`: teacher entries (0: none).
int make_grad_plan(int dtype, int64_t rows, int64_t cols, int k, GradPlan* p) {
    const int64_t vecs = span_vecs(cols, logits_elem_size(dtype));
    const int64_t rows1 = rows > 0 ? rows : 1;
    int64_t team = next_pow2(vecs);
    if (k > 0) {
        // the team's LDS holds the entries: at most four to a lane, and beyond 32 lanes a wavefront
        // or a workgroup, by the forward pass's rules
        team = std::max<int64_t>(team, next_pow2(ceil_div(k, 4)));
        if (team > 32) team = vecs <= 256 && k <= kWaveEntries ? 64 : kBlock;
    }
    p->team = static_cast<int>(team < kBlock ? team : kBlock);
    p->slices = 1;
    if (p->team == kBlock) {
        // Four vectors to a thread, with many teacher entries more: every slice goes through them.
        // us by 2, 4, 8 and 16 vectors to a thread: [4096,32000] bf16 with 1024 random entries 323, 258,
        // 239, 265, with 64 of them 106, 114, 127, 130; [16,202048] f32 without any 7.2, 8.6, 12.6, 18.7.
        // (Two or three would gain where the entries are few: [4096,128256] bf16 with 64 371 and 366 us,
        // 421 with four.)
        const int64_t each = std::max(4, k / 64);
        p->slices = static_cast<int>(std::min<int64_t>(ceil_div(vecs, kBlock * each), 4095));
    }
    p->grid_blocks = ceil_div(rows1 * p->slices, kBlock / p->team);
    return grid_too_large(p->grid_blocks, kBlock) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
}

// Whether every row starts on a 16-byte boundary; of contiguous rows in an aligned tensor.
bool vec_rows(const LogitsArgs& a) {
    return aligned(a.x, 16) && a.row_stride * logits_elem_size(a.dtype) % 16 == 0;
}
bool vec_rows(int dtype, int64_t cols) { return cols * logits_elem_size(dtype) % 16 == 0; }

void fill_logits_plan(const LogitsPlan& p, int dispatches, argreduce_plan_t* out) {
    *out = argreduce_plan_t{};
    out->path = p.path;
    out->lanes_per_row = p.team * p.parts;
    out->blocks_per_row = p.parts;
    out->block_threads = p.path == ARGREDUCE_PATH_BLOCK ? p.team : static_cast<int32_t>(kBlock);
    out->grid_blocks = p.grid_blocks;
    out->grid_rows = p.path == ARGREDUCE_PATH_SUBWAVE ? p.grid_blocks * (kBlock / p.team)
                                                      : p.grid_blocks / p.parts;
    out->unroll = kPartUnroll;
    out->outputs_per_block = p.path == ARGREDUCE_PATH_SUBWAVE ? static_cast<int32_t>(kBlock / p.team) : 1;
    out->device_threads = p.device_threads;
    out->scratch_bytes = p.scratch_bytes;
    out->load_bytes = 16;
    out->dispatches = dispatches;
}

// Checks of the teacher's arguments.
int check_teacher(const LogitsArgs& a, int32_t k, const int64_t* ids, const float* values,
                  const float* stats) {
    if (k < 1 || k > kTeacherMax) return ARGREDUCE_ERR_INVALID_ARG;
    if (a.rows == 0) return ARGREDUCE_OK;
    if (!fits48(a.x) || !usable(ids, 8) || !usable(values, 4) || !usable(stats, 4))
        return ARGREDUCE_ERR_INVALID_ARG;
    return ARGREDUCE_OK;
}

int distill(const LogitsArgs& a, int32_t k, const int64_t* ids, const float* values, float* stats,
            const float* weights, void* grad, void* scratch, size_t scratch_bytes, void* stream) {
    LogitsPlan p;
    GradPlan g{};
    int rc = make_logits_plan(a.dtype, a.rows, a.cols, grad != nullptr ? kDistillStep : kDistill, k,
                              vec_rows(a), &p);
    if (rc != ARGREDUCE_OK) return rc;
    if (grad != nullptr && p.path == ARGREDUCE_PATH_SPLIT) {  // a launch of its own for the gradient
        rc = make_grad_plan(a.dtype, a.rows, a.cols, k, &g);
        if (rc != ARGREDUCE_OK) return rc;
    }
    uint8_t* scratch16 = nullptr;
    rc = scratch_of(p.scratch_bytes, scratch, scratch_bytes, &scratch16);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_distill(p, g, a, k, ids, values, stats, weights, grad, scratch16,
                                    static_cast<hipStream_t>(stream)));
}

}  // namespace
}  // namespace argreduce

using argreduce::GradPlan;
using argreduce::LogitsArgs;
using argreduce::LogitsPlan;

ARGREDUCE_EXPORT size_t argreduce_logprobs_scratch_bytes(int64_t rows, int64_t cols,
                                                         argreduce_dtype_t dtype) {
    LogitsPlan p;
    if (argreduce::make_logits_plan(dtype, rows, cols, argreduce::kLogprobs, 0,
                                    argreduce::vec_rows(dtype, cols), &p) != ARGREDUCE_OK)
        return std::numeric_limits<size_t>::max();
    return p.scratch_bytes;
}

ARGREDUCE_EXPORT int argreduce_logprobs_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype,
                                             argreduce_plan_t* out) {
    if (out == nullptr) return ARGREDUCE_ERR_INVALID_ARG;
    LogitsPlan p;
    const int rc = argreduce::make_logits_plan(dtype, rows, cols, argreduce::kLogprobs, 0,
                                               argreduce::vec_rows(dtype, cols), &p);
    if (rc != ARGREDUCE_OK) return rc;
    argreduce::fill_logits_plan(p, p.parts > 1 ? 2 : 1, out);
    return ARGREDUCE_OK;
}

ARGREDUCE_EXPORT int argreduce_logprobs(const void* x, argreduce_dtype_t dtype, int64_t rows,
                                        int64_t cols, int64_t row_stride, const int64_t* tokens,
                                        float temperature, int32_t entropy, int32_t top, float* stats,
                                        float* top_logprobs, int64_t* top_tokens, void* scratch,
                                        size_t scratch_bytes, void* stream) {
    using namespace argreduce;
    LogitsArgs a;
    int rc = check_logits(x, dtype, rows, cols, row_stride, temperature, &a);
    if (rc != ARGREDUCE_OK) return rc;
    if (top < 0 || top > kTopMax) return ARGREDUCE_ERR_INVALID_ARG;
    if (rows == 0) return ARGREDUCE_OK;
    if (!fits48(x) || !usable(tokens, 8) || !usable(stats, 4)) return ARGREDUCE_ERR_INVALID_ARG;
    if (top > 0 && (!usable(top_logprobs, 4) || !usable(top_tokens, 8))) return ARGREDUCE_ERR_INVALID_ARG;
    LogitsPlan p;
    rc = make_logits_plan(dtype, rows, cols, top > 0 ? kLogprobsTop : kLogprobs, 0, vec_rows(a), &p);
    if (rc != ARGREDUCE_OK) return rc;
    uint8_t* scratch16 = nullptr;
    rc = scratch_of(p.scratch_bytes, scratch, scratch_bytes, &scratch16);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_logprobs(p, a, tokens, entropy != 0, entropy == ARGREDUCE_ENTROPY_APART, top,
                                     stats, top > 0 ? top_logprobs : nullptr, top > 0 ? top_tokens : nullptr,
                                     scratch16, static_cast<hipStream_t>(stream)));
}

ARGREDUCE_EXPORT int argreduce_logprobs_grad(const void* x, argreduce_dtype_t dtype, int64_t rows,
                                             int64_t cols, int64_t row_stride, const int64_t* tokens,
                                             float temperature, const float* stats,
                                             const float* grad_logprob, const float* grad_entropy,
                                             void* grad, void* stream) {
    using namespace argreduce;
    LogitsArgs a;
    int rc = check_logits(x, dtype, rows, cols, row_stride, temperature, &a);
    if (rc != ARGREDUCE_OK) return rc;
    if (rows == 0) return ARGREDUCE_OK;
    if (!fits48(x) || !usable(tokens, 8) || !usable(stats, 4) || !usable(grad_logprob, 4) ||
        !usable(grad, static_cast<uintptr_t>(logits_elem_size(dtype))) ||
        (grad_entropy != nullptr && !usable(grad_entropy, 4)))
        return ARGREDUCE_ERR_INVALID_ARG;
    GradPlan g;
    rc = make_grad_plan(dtype, rows, cols, 0, &g);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_logprobs_grad(g, a, tokens, stats, grad_logprob, grad_entropy, grad,
                                          static_cast<hipStream_t>(stream)));
}

ARGREDUCE_EXPORT size_t argreduce_distill_scratch_bytes(int64_t rows, int64_t cols,
                                                        argreduce_dtype_t dtype) {
    LogitsPlan p;
    const bool vec = argreduce::vec_rows(dtype, cols);
    int rc = argreduce::make_logits_plan(dtype, rows, cols, argreduce::kDistill, 1, vec, &p);
    if (rc == ARGREDUCE_ERR_TOO_WIDE)  // rows that only a step's grid holds
        rc = argreduce::make_logits_plan(dtype, rows, cols, argreduce::kDistillStep, 1, vec, &p);
    return rc == ARGREDUCE_OK ? p.scratch_bytes : std::numeric_limits<size_t>::max();
}

ARGREDUCE_EXPORT int argreduce_distill_plan(int64_t rows, int64_t cols, argreduce_dtype_t dtype,
                                            argreduce_plan_t* out) {
    if (out == nullptr) return ARGREDUCE_ERR_INVALID_ARG;
    LogitsPlan p;
    const int rc = argreduce::make_logits_plan(dtype, rows, cols, argreduce::kDistill, 1,
                                               argreduce::vec_rows(dtype, cols), &p);
    if (rc != ARGREDUCE_OK) return rc;
    argreduce::fill_logits_plan(p, p.parts > 1 ? 2 : 1, out);
    return ARGREDUCE_OK;
}

ARGREDUCE_EXPORT int argreduce_distill(const void* x, argreduce_dtype_t dtype, int64_t rows,
                                       int64_t cols, int64_t row_stride, int32_t k,
                                       const int64_t* teacher_tokens, const float* teacher_logits,
                                       float temperature, float* stats, void* scratch,
                                       size_t scratch_bytes, void* stream) {
    using namespace argreduce;
    LogitsArgs a;
    int rc = check_logits(x, dtype, rows, cols, row_stride, temperature, &a);
    if (rc != ARGREDUCE_OK) return rc;
    rc = check_teacher(a, k, teacher_tokens, teacher_logits, stats);
    if (rc != ARGREDUCE_OK || rows == 0) return rc;
    return distill(a, k, teacher_tokens, teacher_logits, stats, nullptr, nullptr, scratch, scratch_bytes,
                   stream);
}

ARGREDUCE_EXPORT int argreduce_distill_grad(const void* x, argreduce_dtype_t dtype, int64_t rows,
                                            int64_t cols, int64_t row_stride, int32_t k,
                                            const int64_t* teacher_tokens, const float* teacher_logits,
                                            float temperature, const float* stats,
                                            const float* grad_loss, void* grad, void* stream) {
    using namespace argreduce;
    LogitsArgs a;
    int rc = check_logits(x, dtype, rows, cols, row_stride, temperature, &a);
    if (rc != ARGREDUCE_OK) return rc;
    rc = check_teacher(a, k, teacher_tokens, teacher_logits, stats);
    if (rc != ARGREDUCE_OK || rows == 0) return rc;
    if (!usable(grad_loss, 4) || !usable(grad, static_cast<uintptr_t>(logits_elem_size(dtype))))
        return ARGREDUCE_ERR_INVALID_ARG;
    GradPlan g;
    rc = make_grad_plan(dtype, rows, cols, k, &g);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_distill_grad(g, a, k, teacher_tokens, teacher_logits, stats, grad_loss, grad,
                                         static_cast<hipStream_t>(stream)));
}

ARGREDUCE_EXPORT int argreduce_distill_step(const void* x, argreduce_dtype_t dtype, int64_t rows,
                                            int64_t cols, int64_t row_stride, int32_t k,
                                            const int64_t* teacher_tokens, const float* teacher_logits,
                                            float temperature, const float* weights, float* stats,
                                            void* grad, void* scratch, size_t scratch_bytes,
                                            void* stream) {
    using namespace argreduce;
    LogitsArgs a;
    int rc = check_logits(x, dtype, rows, cols, row_stride, temperature, &a);
    if (rc != ARGREDUCE_OK) return rc;
    rc = check_teacher(a, k, teacher_tokens, teacher_logits, stats);
    if (rc != ARGREDUCE_OK || rows == 0) return rc;
    if (!usable(weights, 4) || !usable(grad, static_cast<uintptr_t>(logits_elem_size(dtype))))
        return ARGREDUCE_ERR_INVALID_ARG;
    return distill(a, k, teacher_tokens, teacher_logits, stats, weights, grad, scratch, scratch_bytes,
                   stream);
}
