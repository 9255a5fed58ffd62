// C ABI of expert routing: argument checks, launch plans and scratch sizes. Declarations and the
// contract are in include/argreduce.h, the kernels in argreduce_route.hip.
#include <hip/hip_runtime_api.h>

#include "argreduce_checks.hpp"
#include "argreduce_route.hpp"

namespace argreduce {

size_t route_partial_bytes(int64_t experts);  // scratch of one workgroup

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

int make_route_plan(int dtype, int64_t groups, int64_t tokens, int64_t experts, RoutePlan* p) {
    int rc = check_route(dtype, groups, tokens, experts);
    if (rc != ARGREDUCE_OK) return rc;
    int64_t cap = 0;
    rc = plan_device_threads(&cap);
    if (rc != ARGREDUCE_OK) return rc;
    *p = RoutePlan{};
    p->device_threads = cap;
    const int64_t vw = 16 / logits_elem_size(dtype);
    const int64_t vecs = ceil_div(experts, vw);
    p->lanes = static_cast<int>(std::min<int64_t>(64, next_pow2(vecs)));
    p->vecs = static_cast<int>(next_pow2(ceil_div(vecs, 64)));
    // Two workgroups per CU, or as many as the tokens fill; several of one group's.
    const int64_t groups1 = std::max<int64_t>(1, groups), at_once = kBlock / p->lanes;
    const int64_t most = std::max<int64_t>(1, 2 * (cap / kThreadsPerCu) / groups1);
    p->blocks = static_cast<int>(std::max<int64_t>(1, std::min({ceil_div(tokens, at_once), most, int64_t{65535}})));
    p->grid_blocks = groups1 * p->blocks;
    p->scratch_bytes = 15 + static_cast<size_t>(p->grid_blocks) * route_partial_bytes(experts);
    return grid_too_large(p->grid_blocks, kBlock) ? ARGREDUCE_ERR_TOO_WIDE : ARGREDUCE_OK;
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
    return make_route_plan(dtype, groups, tokens, experts, &p) == ARGREDUCE_OK
               ? p.scratch_bytes
               : std::numeric_limits<size_t>::max();
}

ARGREDUCE_EXPORT int argreduce_route_plan(int64_t groups, int64_t tokens, int64_t experts, argreduce_dtype_t dtype,
                                          argreduce_plan_t* out) {
    if (out == nullptr) return ARGREDUCE_ERR_INVALID_ARG;
    RoutePlan p;
    const int rc = make_route_plan(dtype, groups, tokens, experts, &p);
    if (rc != ARGREDUCE_OK) return rc;
    *out = argreduce_plan_t{};
    out->path = ARGREDUCE_PATH_SUBWAVE;
    out->lanes_per_row = p.lanes;
    out->blocks_per_row = 1;
    out->block_threads = static_cast<int32_t>(kBlock);
    out->grid_blocks = p.grid_blocks;
    out->outputs_per_block = static_cast<int32_t>(kBlock) / p.lanes;
    out->grid_rows = p.grid_blocks * out->outputs_per_block;
    out->unroll = p.vecs;
    out->device_threads = p.device_threads;
    out->scratch_bytes = p.scratch_bytes;
    out->load_bytes = 16;
    out->dispatches = 2;
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
    rc = make_route_plan(dtype, groups, tokens, experts, &p);
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
    rc = make_route_plan(dtype, groups, tokens, experts, &p);
    if (rc != ARGREDUCE_OK) return rc;
    return status_of(launch_route_grad(p, a, chosen, static_cast<const uint8_t*>(totals), g_weights, g_balance,
                                       g_z, grad, static_cast<hipStream_t>(stream)));
}
