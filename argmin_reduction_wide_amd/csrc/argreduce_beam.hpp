// Plans and launchers of beam search's step and reordering (argreduce_beam.hip), shared with their
// C ABI (argreduce_beam_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "argreduce.h"

namespace argreduce {

constexpr int kBeamMax = 64;     // beams of a group, and candidates kept (ARGREDUCE_BEAM_MAX)
constexpr int kSliceThreads = 256;  // of a workgroup that holds a slice in registers
constexpr int kSliceVecs = 8;    // 16-byte vectors each of its lanes holds, at most
constexpr int kBeamLists = 256;  // lists of candidates that one group's join takes

// How one step is done.
struct BeamPlan {
    int path;             // argreduce_path_t: SUBWAVE (a wavefront per group), BLOCK or SPLIT
    int team;             // SUBWAVE: lanes per row, 4 to 128; else threads that scan one slice
    int parts;            // BLOCK, SPLIT: slices per row, each with a list of candidates of its own
    int held;             // 16-byte vectors per lane held in registers: 1, 2, 4, 8, or 0 (a slice in one pass)
    bool joins;           // whether the scanning kernel joins the lists, too
    int64_t grid_blocks;  // workgroups of the (scanning) kernel
    int64_t device_threads;
    size_t scratch_bytes; // including 15 bytes of alignment slack; 0 if none needed
};

struct BeamArgs {
    const void* x;
    int dtype;
    int64_t groups, cols, row_stride;
    int beams, width;
    const float* scores;
    const uint8_t* ended;  // or null
    int64_t end_token;
    double temperature;
    uint8_t* out;          // parents, tokens, scores, ended
};

size_t beam_scratch(int64_t groups, int64_t lists, int width);  // scratch of a step with so many lists per group
hipError_t launch_beam_step(const BeamPlan& plan, const BeamArgs& a, uint8_t* scratch16, hipStream_t stream);

// Positions [first, last) of every group's beams: values, or arrays of one per group.
struct ReorderArgs {
    const argreduce_state_t* table;  // on the device
    int tensors;
    int64_t groups;
    int beams;
    const int64_t* parents;
    const int64_t* first;  // or null: first_value
    const int64_t* last;
    int64_t first_value, last_value;
    int blocks;            // workgroups per tensor and group
};
hipError_t launch_reorder(const ReorderArgs& a, hipStream_t stream);

// Thread capacity plans are made for (the simulated one if set); an ARGREDUCE_* status.
int plan_device_threads(int64_t* threads);

}  // namespace argreduce
