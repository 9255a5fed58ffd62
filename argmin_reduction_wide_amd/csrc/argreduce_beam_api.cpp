// C ABI of beam search's step and reordering: argument checks, launch plans and scratch sizes.
// Declarations and the contract are in include/argreduce.h, the kernels in argreduce_beam.hip.
#include <hip/hip_runtime_api.h>

#include "argreduce_beam.hpp"
#include "argreduce_checks.hpp"

namespace argreduce {
namespace {

// Slices of at least this many vectors, two for each of 256 lanes, where rows are few ([8,4,32000] bf16 10.5 us, of
// twice as many 10.9), and of at least so many where they are more than the CUs.
constexpr int64_t kLeastSlice = 512, kLongSlice = 4000;

int check_beams(int64_t groups, int64_t beams, int64_t cols, int dtype) {
    if (logits_elem_size(dtype) == 0) return ARGREDUCE_ERR_UNSUPPORTED_DTYPE;
    if (groups < 0 || beams < 1 || beams > kBeamMax) return ARGREDUCE_ERR_INVALID_ARG;
    if (groups > std::numeric_limits<int32_t>::max() / kBeamLists) return ARGREDUCE_ERR_TOO_WIDE;
    return check_logits_shape(dtype, groups * beams, cols);
}

int make_beam_plan(int dtype, int64_t groups, int64_t beams, int64_t cols, int width, BeamPlan* p) {
    int rc = check_beams(groups, beams, cols, dtype);
    if (rc != ARGREDUCE_OK) return rc;
    if (width < 1 || width > kBeamMax) return ARGREDUCE_ERR_INVALID_ARG;
    int64_t cap = 0;
    rc = plan_device_threads(&cap);
    if (rc != ARGREDUCE_OK) return rc;
    *p = BeamPlan{};
    p->device_threads = cap;
    const int64_t rows = std::max<int64_t>(1, groups * beams);
    const int64_t cus = std::max<int64_t>(1, cap / kThreadsPerCu);
    const int64_t vecs = span_vecs(cols, logits_elem_size(dtype));
    // A wavefront per group, if its beams' rows are units of at most eight vectors per lane: [2048,4,64] f16 5.5 us, by
    // a wavefront per row and a join 18.3; [100,8,100] f32 8 and 10.8, [2000,8,500] f16 (eight vectors) 26.6 and 29.9.
    const int64_t whole = ceil_div(cols * logits_elem_size(dtype), 16);  // vectors of a row from its first element
    const int64_t lanes = std::max<int64_t>(4, next_pow2(whole));
    const int64_t units = next_pow2(lanes <= 64 ? ceil_div(beams, 64 / lanes) : beams * 2);
    if (lanes <= 128 && units <= 8) {
        p->path = ARGREDUCE_PATH_SUBWAVE;
        p->team = static_cast<int>(lanes);
        p->held = static_cast<int>(units);
        p->joins = true;
        p->parts = 1;
        p->grid_blocks = ceil_div(std::max<int64_t>(1, groups), kBlock / 64);
        return grid_too_large(p->grid_blocks, kBlock) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
    }
    // Slices of rows too few to give every CU one. More and longer rows are cut until the slices are six per CU:
    // [300,1,128256] f16 27.9 us in four slices, 41 in one, [400,2,260000] 97 and 110; but [256,8,128256] bf16 110 in
    // four and 103 in one.
    const int64_t parts =
        rows <= cus ? std::min({ceil_div(vecs, kLeastSlice), cus / rows, kBeamLists / beams})
                    : std::max<int64_t>(1, std::min({vecs / kLongSlice, ceil_div(6 * cus, rows), kBeamLists / beams}));
    const int64_t slice = parts > 1 ? ceil_div(vecs, parts) : whole;
    p->path = parts > 1 ? ARGREDUCE_PATH_SPLIT : ARGREDUCE_PATH_BLOCK;
    // Slices of at most 2048 vectors are held in registers where they are no more than the CUs, rows of at most 512 (256
    // where they are many) by a wavefront each where they are more: [2000,12,1000] f16 43 us instead of 116 in one pass
    // by 256 threads and 47 by a wavefront, [100,8,3500] 13.7 and 17.2 by a wavefront; but [2000,8,4000] bf16 66 and 54,
    // and held by 256 threads [1000,8,10000] 109 instead of 60.
    p->joins = rows <= cus && slice <= kSliceVecs * kSliceThreads;
    const bool many = rows >= 16 * cus;
    if (p->joins || slice <= (many ? 4 : kSliceVecs) * 64) {
        p->team = p->joins ? kSliceThreads : 64;
        p->held = static_cast<int>(next_pow2(ceil_div(slice, p->team)));
    } else {
        // One slice or less per CU: 1024 threads ([20,10,50000] f32 19.7 us, 25 with 256). Two, or six rows or more and
        // long ones: 512 ([30,12,25000] f16 22.0, 23.2 with 256; [256,8,128256] bf16 103 and 110; but [1000,8,10000]
        // 97 and 60, [200,5,32001] f16 31.8 and 27.0). Many short ones: a wavefront, few of whose steps wait for others
        // ([2000,8,6000] f16 58 us, 90 with 256, [1000,8,10000] bf16 51 and 60, [1000,8,20000] f16 81 and 87; but
        // [250,4,10000] 20.5 and 16.3).
        if (rows <= cus)
            p->team = 1024;
        else if (many && slice <= 2560)
            p->team = 64;
        else
            p->team = rows * parts <= 2 * cus || (rows >= 6 * cus && slice > kLongSlice) ? 512 : 256;
    }
    p->parts = static_cast<int>(parts);
    p->grid_blocks = rows * parts;
    p->scratch_bytes = 15 + beam_scratch(std::max<int64_t>(1, groups), beams * parts, width);
    return grid_too_large(p->grid_blocks, p->team) || grid_too_large(groups, kBlock) ? ARGREDUCE_ERR_TOO_WIDE
                                                                                     : ARGREDUCE_OK;
}

// One dimension of a state, in bytes.
struct Dim {
    int64_t n, stride;
};

// Whether no two elements of a state lie at the same place, and *span, the bytes it lies in.
bool apart(const argreduce_state_t& s, int64_t groups, int64_t beams, int64_t* span) {
    Dim d[4] = {{groups, s.group_stride}, {beams, s.beam_stride}, {s.outer, s.outer_stride},
                {s.positions, s.position_stride}};
    std::sort(d, d + 4, [](const Dim& a, const Dim& b) { return a.stride < b.stride; });
    int64_t bytes = s.inner;
    for (const Dim& e : d) {
        if (e.n <= 1) continue;
        if (e.stride < bytes || e.stride >= kMaxBytes / e.n) return false;
        bytes += e.stride * (e.n - 1);
    }
    *span = bytes;
    return true;
}

}  // namespace
}  // namespace argreduce

using namespace argreduce;

ARGREDUCE_EXPORT size_t argreduce_beam_scratch_bytes(int64_t groups, int64_t beams, int64_t cols,
                                                     argreduce_dtype_t dtype, int32_t width) {
    BeamPlan p;
    return make_beam_plan(dtype, groups, beams, cols, width, &p) == ARGREDUCE_OK
               ? p.scratch_bytes
               : std::numeric_limits<size_t>::max();
}

ARGREDUCE_EXPORT int argreduce_beam_plan(int64_t groups, int64_t beams, int64_t cols, argreduce_dtype_t dtype,
                                         int32_t width, argreduce_plan_t* out) {
    if (out == nullptr) return ARGREDUCE_ERR_INVALID_ARG;
    BeamPlan p;
    const int rc = make_beam_plan(dtype, groups, beams, cols, width, &p);
    if (rc != ARGREDUCE_OK) return rc;
    *out = argreduce_plan_t{};
    out->path = p.path;
    const bool wave = p.path == ARGREDUCE_PATH_SUBWAVE;
    out->lanes_per_row = p.team * p.parts;
    out->blocks_per_row = p.parts;
    out->block_threads = wave ? static_cast<int32_t>(kBlock) : p.team;
    out->grid_blocks = p.grid_blocks;
    out->outputs_per_block = wave ? static_cast<int32_t>(kBlock / 64 * beams) : 1;
    out->grid_rows = p.grid_blocks * out->outputs_per_block / p.parts;
    out->unroll = p.held > 0 ? p.held : logits_elem_size(dtype);  // 16 elements per lane and step
    out->device_threads = p.device_threads;
    out->scratch_bytes = p.scratch_bytes;
    out->load_bytes = 16;
    out->dispatches = p.joins ? 1 : 2;
    return ARGREDUCE_OK;
}

ARGREDUCE_EXPORT size_t argreduce_beam_out_bytes(int64_t groups, int32_t width) {
    if (groups < 0 || width < 1 || width > kBeamMax || groups > std::numeric_limits<int32_t>::max())
        return std::numeric_limits<size_t>::max();
    return static_cast<size_t>(groups) * static_cast<size_t>(width) * (8 + 8 + 4 + 1);
}

ARGREDUCE_EXPORT int argreduce_beam_step(const void* x, argreduce_dtype_t dtype, int64_t groups, int64_t beams,
                                         int64_t cols, int64_t row_stride, const float* scores,
                                         const uint8_t* ended, int64_t end_token, double temperature,
                                         int32_t width, void* out, void* scratch, size_t scratch_bytes,
                                         void* stream) {
    int rc = check_beams(groups, beams, cols, dtype);
    if (rc != ARGREDUCE_OK) return rc;
    const int64_t rows = groups * beams;
    rc = check_rows(x, dtype, rows, cols, row_stride);
    if (rc != ARGREDUCE_OK) return rc;
    if (!(temperature >= 0x1p-60 && temperature <= 0x1p60)) return ARGREDUCE_ERR_INVALID_ARG;
    if (width < 1 || width > kBeamMax || end_token >= cols || (ended != nullptr && end_token < 0))
        return ARGREDUCE_ERR_INVALID_ARG;
    if (rows == 0) return ARGREDUCE_OK;
    if (!fits48(x) || !usable(scores, 4) || !fits48(ended) || !usable(out, 8)) return ARGREDUCE_ERR_INVALID_ARG;
    BeamPlan p;
    rc = make_beam_plan(dtype, groups, beams, cols, width, &p);
    if (rc != ARGREDUCE_OK) return rc;
    uint8_t* scratch16 = nullptr;
    rc = scratch_of(p.scratch_bytes, scratch, scratch_bytes, &scratch16);
    if (rc != ARGREDUCE_OK) return rc;
    const BeamArgs a{x, dtype, groups, cols, rows > 1 ? row_stride : cols, static_cast<int>(beams), width,
                     scores, ended, end_token, temperature, static_cast<uint8_t*>(out)};
    return status_of(launch_beam_step(p, a, scratch16, static_cast<hipStream_t>(stream)));
}

ARGREDUCE_EXPORT int argreduce_reorder_plan(const argreduce_state_t* states, int32_t tensors, int64_t groups,
                                            int64_t beams, argreduce_reorder_t* plan) {
    if (plan == nullptr || states == nullptr || tensors < 1 || groups < 0 || beams < 1 || beams > kBeamMax)
        return ARGREDUCE_ERR_INVALID_ARG;
    if (tensors > ARGREDUCE_STATES_MAX || groups > std::numeric_limits<int32_t>::max() / tensors)
        return ARGREDUCE_ERR_TOO_WIDE;
    *plan = argreduce_reorder_t{tensors, static_cast<int32_t>(beams), groups, 0, 0};
    for (int32_t i = 0; i < tensors; ++i) {
        const argreduce_state_t& s = states[i];
        if (s.base == nullptr || !fits48(s.base) || s.outer < 1 || s.positions < 0 || s.inner < 1 ||
            s.group_stride < 0 || s.beam_stride < 0 || s.outer_stride < 0 || s.position_stride < 0)
            return ARGREDUCE_ERR_INVALID_ARG;
        int64_t span = 0;
        if (!apart(s, groups, beams, &span)) return ARGREDUCE_ERR_INVALID_ARG;
        // units (of 8 bytes at least, each run's last one perhaps less) are counted in 31 bits
        constexpr int64_t kMost = std::numeric_limits<int32_t>::max();
        const int64_t most = std::max<int64_t>(1, s.positions);
        if (span >= kMaxBytes || s.outer > kMost / most || s.inner / 8 + 1 > kMost / most / s.outer)
            return ARGREDUCE_ERR_TOO_WIDE;
        plan->positions = std::max(plan->positions, s.positions);
        plan->position_bytes = std::max(plan->position_bytes, s.outer * s.inner);
    }
    return ARGREDUCE_OK;
}

ARGREDUCE_EXPORT int argreduce_reorder(const argreduce_reorder_t* plan, const argreduce_state_t* table,
                                       const int64_t* parents, const int64_t* first, const int64_t* last,
                                       int64_t first_value, int64_t last_value, void* stream) {
    if (plan == nullptr || plan->tensors < 1 || plan->tensors > ARGREDUCE_STATES_MAX || plan->beams < 1 ||
        plan->beams > kBeamMax || plan->groups < 0 || plan->positions < 0 || plan->position_bytes < 1)
        return ARGREDUCE_ERR_INVALID_ARG;
    if (plan->groups == 0) return ARGREDUCE_OK;
    if (!usable(table, 8) || !usable(parents, 8)) return ARGREDUCE_ERR_INVALID_ARG;
    if ((first != nullptr && !usable(first, 8)) || (last != nullptr && !usable(last, 8)))
        return ARGREDUCE_ERR_INVALID_ARG;
    const int64_t from = first != nullptr ? 0 : std::min(std::max<int64_t>(first_value, 0), plan->positions);
    const int64_t to = last != nullptr ? plan->positions : std::min(std::max<int64_t>(last_value, 0), plan->positions);
    if (from >= to) return ARGREDUCE_OK;
    int64_t cap = 0;
    const int rc = plan_device_threads(&cap);
    if (rc != ARGREDUCE_OK) return rc;
    // Two device waves of workgroups; a lane goes through several units where there are more.
    const int64_t pairs = plan->tensors * plan->groups;
    const int64_t units = ceil_div((to - from) * plan->position_bytes, 16);
    const int64_t want = std::max<int64_t>(1, 2 * cap / kBlock / pairs);
    const int64_t blocks = std::min<int64_t>({ceil_div(units, kBlock), want, 65535});
    if (grid_too_large(pairs * blocks, kBlock)) return ARGREDUCE_ERR_TOO_WIDE;
    const ReorderArgs a{table, plan->tensors, plan->groups, plan->beams, parents, first, last, from, to,
                        static_cast<int>(blocks)};
    return status_of(launch_reorder(a, static_cast<hipStream_t>(stream)));
}
