// Plans and launchers of expert routing (argreduce_route.hip), shared with its C ABI
// (argreduce_route_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "argreduce.h"

namespace argreduce {

constexpr int kExpertsMax = 1024;  // experts of a router (ARGREDUCE_EXPERTS_MAX)
constexpr int kRouteTopMax = 64;   // experts chosen per token (ARGREDUCE_ROUTE_TOP_MAX)

constexpr int kRouteThreads = 512;  // of a workgroup
constexpr uint32_t kRouteSet = 64;  // workgroups whose sums one of them adds up

// A token's logits lie in `lanes` lanes of a wavefront, `vecs` vectors of 16 bytes each.
struct RoutePlan {
    int lanes, vecs;
    int blocks;            // workgroups per group of tokens
    int64_t grid_blocks;
    int64_t device_threads;
    size_t scratch_bytes;  // including 15 bytes of alignment slack
};

struct RouteArgs {
    const void* x;
    int dtype;
    int64_t groups, tokens, experts, row_stride;
    int top;
    bool renormalize;
};

size_t route_group_bytes(int64_t experts, int blocks);  // scratch of one group

hipError_t launch_route(const RoutePlan& plan, const RouteArgs& a, const uint8_t* live, float* weights,
                        int64_t* chosen, uint8_t* totals, uint8_t* scratch16, hipStream_t stream);
hipError_t launch_route_grad(const RoutePlan& plan, const RouteArgs& a, const int64_t* chosen,
                             const uint8_t* totals, const float* g_weights, const float* g_balance,
                             const float* g_z, void* grad, hipStream_t stream);

// Thread capacity plans are made for (the simulated one if set); an ARGREDUCE_* status.
int plan_device_threads(int64_t* threads);

}  // namespace argreduce
