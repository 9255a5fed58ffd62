// C ABI of expert routing: argument checks, launch plans and scratch sizes. Declarations and the
// contract are in include/argreduce.h, the kernels in argreduce_route.hip.
#include <hip/hip_runtime_api.h>

#include "argreduce_checks.hpp"
#include "argreduce_route.hpp"

namespace argreduce {

namespace {

int check_route(int dtype, int64_t groups, int64_t tokens, int64_t experts) {
    if (logits_elem_size(dtype) == 0) return ARGREDUCE_ERR_UNSUPPORTED_DTYPE;
    if (groups < 0 || tokens < 0 || experts < 1 || experts > kExpertsMax) return ARGREDUCE_ERR_INVALID_ARG;
    if (tokens > std::numeric_limits<int32_t>::max() ||
        (tokens > 0 && groups > std::numeric_limits<int32_t>::max() / tokens) ||
        groups > std::numeric_limits<int32_t>::max())
        return ARGREDUCE_ERR_TOO_WIDE;
    return ARGREDUCE_OK;
}

// Tokens up to this many (of all groups) take up to 16 lanes each, more of them up to 8, as long as a lane has no
// more than four vectors. Forward of [16,4096,256] bf16 with 8 experts per token, us: 8 lanes 27.3, 16 lanes 29.0, 32
// lanes 42.6; [16,4096,128] 18.6, 22.2; [16,4096,64] f16 with 2 (8 vectors) 12.0 by 8 lanes, 13.0 by 4, 15.9 by 2; but
// [1,300,256] 11.2 by 8, 9.6 by 16, and its gradient 8.1 and 5.6.
constexpr int64_t kFewTokens = 4096;
// Workgroups of 512 threads per CU, of all groups together: forward 1 ([16,4096,256] bf16 24.8 us, with 2 of them
// 32.5: more sums to join; with 2 of 256 threads 25.1, [8,4096,512] 25.2 and 31.0), gradient 2 ([16,4096,256] 17.8 us,
// with 4 of them 20.4).
constexpr int64_t kForwardPerCu = 1, kGradPerCu = 2;
// Tokens of a group that one workgroup goes through by itself, in rounds: nothing to join then ([1,32,256] bf16 in one
// round 5.4 us, over four workgroups 7.8).
constexpr int64_t kAloneRounds = 2;

int make_route_plan(int dtype, int64_t groups, int64_t tokens, int64_t experts, bool grad, RoutePlan* p) {
    int rc = check_route(dtype, groups, tokens, experts);
    if (rc != ARGREDUCE_OK) return rc;
    int64_t cap = 0;
    rc = plan_device_threads(&cap);
    if (rc != ARGREDUCE_OK) return rc;
    *p = RoutePlan{};
    p->device_threads = cap;
    const int64_t vecs = ceil_div(experts, 16 / logits_elem_size(dtype));
    const int64_t lanes = groups * tokens <= kFewTokens ? 16 : 8;
    p->vecs = static_cast<int>(std::min<int64_t>(4, next_pow2(ceil_div(vecs, lanes))));
    p->lanes = static_cast<int>(next_pow2(ceil_div(vecs, p->vecs)));
    const int64_t groups1 = std::max<int64_t>(1, groups), at_once = kRouteThreads / p->lanes;
    const int64_t per_cu = grad ? kGradPerCu : kForwardPerCu;
    const int64_t most = std::max<int64_t>(1, per_cu * (cap / kThreadsPerCu) / groups1);
    int64_t blocks = std::min({ceil_div(tokens, at_once), most, int64_t{kRouteSet * kRouteSet}});
    if (blocks < 1 || (!grad && tokens <= at_once * kAloneRounds)) blocks = 1;
    p->blocks = static_cast<int>(blocks);
    p->grid_blocks = groups1 * p->blocks;
    if (!grad)
        p->scratch_bytes = blocks == 1 ? 0 : 15 + static_cast<size_t>(groups1) * route_group_bytes(experts, p->blocks);
    return grid_too_large(p->grid_blocks, kRouteThreads) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
}

// The checks of both directions.
int check_routed(const void* x, int dtype, int64_t groups, int64_t tokens, int64_t experts, int64_t row_stride,
                 int32_t top, RouteArgs* a) {
    int rc = check_route(dtype, groups, tokens, experts);
    if (rc != ARGREDUCE_OK) return rc;
    const int64_t rows = groups * tokens;
    rc = check_rows(x, dtype, rows, experts, row_stride);
    if (rc != ARGREDUCE_OK) return rc;
    if (top < 1 || top > kRouteTopMax || top > experts || (rows > 0 && !fits48(x))) return ARGREDUCE_ERR_INVALID_ARG;
    *a = RouteArgs{x, dtype, groups, tokens, experts, rows > 1 ? row_stride : experts, top, false};
    return ARGREDUCE_OK;
}

}  // namespace
}  // namespace argreduce

using namespace argreduce;

ARGREDUCE_EXPORT size_t argreduce_route_scratch_bytes(int64_t groups, int64_t tokens, int64_t experts,
                                                      argreduce_dtype_t dtype) {
    RoutePlan p;
    return make_route_plan(dtype, groups, tokens, experts, false, &p) == ARGREDUCE_OK
               ? p.scratch_bytes
               : std::numeric_limits<size_t>::max();
}

ARGREDUCE_EXPORT int argreduce_route_plan(int64_t groups, int64_t tokens, int64_t experts, argreduce_dtype_t dtype,
                                          argreduce_plan_t* out) {
    if (out == nullptr) return ARGREDUCE_ERR_INVALID_ARG;
    RoutePlan p;
    const int rc = make_route_plan(dtype, groups, tokens, experts, false, &p);
    if (rc != ARGREDUCE_OK) return rc;
    *out = argreduce_plan_t{};
    out->path = ARGREDUCE_PATH_SUBWAVE;
    out->lanes_per_row = p.lanes;
    out->blocks_per_row = 1;
    out->block_threads = kRouteThreads;
    out->grid_blocks = p.grid_blocks;
    out->outputs_per_block = kRouteThreads / p.lanes;
    out->grid_rows = p.grid_blocks * out->outputs_per_block;
    out->unroll = p.vecs;
    out->device_threads = p.device_threads;
    out->scratch_bytes = p.scratch_bytes;
    out->load_bytes = 16;
    out->dispatches = 1;
    return ARGREDUCE_OK;
}

ARGREDUCE_EXPORT size_t argreduce_route_totals_bytes(int64_t groups, int64_t experts) {
    if (groups < 0 || groups > std::numeric_limits<int32_t>::max() || experts < 1 || experts > kExpertsMax)
        return std::numeric_limits<size_t>::max();
    return static_cast<size_t>(groups) * (8 * static_cast<size_t>(experts) + 8 + 4 + 4);
}

ARGREDUCE_EXPORT int argreduce_route(const void* x, argreduce_dtype_t dtype, int64_t groups, int64_t tokens,
                                     int64_t experts, int64_t row_stride, const uint8_t* live, int32_t top,
                                     int32_t renormalize, float* weights, int64_t* chosen, void* totals,
                                     void* scratch, size_t scratch_bytes, void* stream) {
    RouteArgs a;
    int rc = check_routed(x, dtype, groups, tokens, experts, row_stride, top, &a);
    if (rc != ARGREDUCE_OK) return rc;
    a.renormalize = renormalize != 0;
    if (groups == 0) return ARGREDUCE_OK;
    if (!usable(totals, 8) || !fits48(live)) return ARGREDUCE_ERR_INVALID_ARG;
    if (tokens > 0 && (!usable(weights, 4) || !usable(chosen, 8))) return ARGREDUCE_ERR_INVALID_ARG;
    RoutePlan p;
    rc = make_route_plan(dtype, groups, tokens, experts, false, &p);
    if (rc != ARGREDUCE_OK) return rc;
    uint8_t* scratch16 = nullptr;
    rc = scratch_of(p.scratch_bytes, scratch, scratch_bytes, &scratch16);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_route(p, a, live, weights, chosen, static_cast<uint8_t*>(totals), scratch16,
                                  static_cast<hipStream_t>(stream)));
}

ARGREDUCE_EXPORT int argreduce_route_grad(const void* x, argreduce_dtype_t dtype, int64_t groups, int64_t tokens,
                                          int64_t experts, int64_t row_stride, int32_t top, int32_t renormalize,
                                          const int64_t* chosen, const void* totals, const float* g_weights,
                                          const float* g_balance, const float* g_z, void* grad, void* stream) {
    RouteArgs a;
    int rc = check_routed(x, dtype, groups, tokens, experts, row_stride, top, &a);
    if (rc != ARGREDUCE_OK) return rc;
    a.renormalize = renormalize != 0;
    if (groups == 0 || tokens == 0) return ARGREDUCE_OK;
    const auto optional = [](const float* p) { return p == nullptr || usable(p, 4); };
    if (!usable(chosen, 8) || !usable(totals, 8) || !optional(g_weights) || !optional(g_balance) ||
        !optional(g_z) || !usable(grad, static_cast<uintptr_t>(logits_elem_size(dtype))))
        return ARGREDUCE_ERR_INVALID_ARG;
    RoutePlan p;
    rc = make_route_plan(dtype, groups, tokens, experts, true, &p);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_route_grad(p, a, chosen, static_cast<const uint8_t*>(totals), g_weights, g_balance,
                                       g_z, grad, static_cast<hipStream_t>(stream)));
}
