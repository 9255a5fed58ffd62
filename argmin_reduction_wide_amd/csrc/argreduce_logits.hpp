// Plans and launchers of the logits operators (argreduce_logits.hip), shared with their C ABI
// (argreduce_logits_api.cpp).
#pragma once

#include <hip/hip_runtime.h>
#include <stddef.h>
#include <stdint.h>

#include "argreduce.h"

namespace argreduce {

constexpr int kTopMax = 64;            // alternatives per row (ARGREDUCE_TOP_MAX)
constexpr int kTeacherMax = 1024;      // teacher entries per row (ARGREDUCE_TEACHER_MAX)
constexpr int kPartThreads = 256;      // threads of a workgroup that scans a slice of a row
constexpr int kPartUnroll = 4;         // 16-byte loads each of its lanes keeps in flight
constexpr int kMaxParts = 256;         // slices of a row
constexpr size_t kEntryBytes = 16;     // LDS of one teacher entry
// More teacher entries than this get a hash table in LDS. The gradient of [20000,700] f16, us with the
// table and with every entry compared with every other: 17 entries 26.7 and 34.5, 32 29.5 and 43.6, 64
// 26.8 and 64.5; loss and gradient 31.2 and 33.8, 35.0 and 37.9, 31.0 and 46.8. (Fewer would gain
// little: 8 entries 26.7 and 29.4, loss and gradient 31.1 and 31.8.)
constexpr int kTeacherCompared = 16;
inline int teacher_places(int k) {
    int n = 2;
    while (n < 2 * k) n *= 2;
    return k <= kTeacherCompared ? 0 : n;
}
// LDS of a workgroup for the entries of `rows` teacher rows of each of its teams, and for a table
// of each team.
inline size_t entries_lds(int teams, int rows, int k, bool tables) {
    return teams * (rows * k * kEntryBytes + (tables ? teacher_places(k) * sizeof(uint32_t) : 0));
}

// Teacher rows that a team of the distillation step has in LDS: wavefronts of one team may work on
// two rows at a time.
constexpr int step_rows(int team) { return team == 64 ? 1 : 2; }

// How the rows of one forward call are scanned.
struct LogitsPlan {
    int path;             // argreduce_path_t: SUBWAVE, BLOCK or SPLIT
    int team;             // lanes that scan one row (SUBWAVE, BLOCK), else kPartThreads
    int parts;            // SPLIT: workgroups per row
    int held;             // distillation step: vectors per lane kept in registers, 2, 8 or 16
    int64_t grid_blocks;  // workgroups of the scanning kernel
    int64_t device_threads;
    size_t scratch_bytes; // including 15 bytes of alignment slack; 0 if none needed
};

// How the rows of one gradient call are cut: `team` lanes per slice of a row.
struct GradPlan {
    int team;             // 1 .. 256, a power of two
    int slices;           // slices per row (1 unless team == 256)
    int64_t grid_blocks;
};

// Logits of one call. `scale` is log2(e) / temperature; `keep`: read them so that they stay in the
// Infinity Cache.
struct LogitsArgs {
    const void* x;
    int dtype;
    int64_t rows, cols, row_stride;
    float scale;
    bool keep;
};

size_t part_bytes();  // scratch of one slice of a split row

// `apart`: the entropy also goes to a fifth row of stats.
hipError_t launch_logprobs(const LogitsPlan& plan, const LogitsArgs& a, const int64_t* tokens,
                           bool entropy, bool apart, int top, float* stats, float* top_logprobs,
                           int64_t* top_tokens, uint8_t* scratch16, hipStream_t stream);
hipError_t launch_logprobs_grad(const GradPlan& plan, const LogitsArgs& a, const int64_t* tokens,
                                const float* stats, const float* g_logprob, const float* g_entropy,
                                void* grad, hipStream_t stream);
// With `weights` and `grad` the gradient too (argreduce_distill_step), by `gplan` where the
// plan splits rows (else it is not read).
hipError_t launch_distill(const LogitsPlan& plan, const GradPlan& gplan, const LogitsArgs& a, int k,
                          const int64_t* ids, const float* values, float* stats,
                          const float* weights, void* grad, uint8_t* scratch16, hipStream_t stream);
hipError_t launch_distill_grad(const GradPlan& plan, const LogitsArgs& a, int k, const int64_t* ids,
                               const float* values, const float* stats, const float* g_loss,
                               void* grad, hipStream_t stream);

// Thread capacity plans are made for (the simulated one if set); an ARGREDUCE_* status.
int plan_device_threads(int64_t* threads);

}  // namespace argreduce
