// Checks and arithmetic that the host sides of the operators on logits share.
#pragma once

#include <algorithm>
#include <limits>

#include "argreduce.h"
#include "argreduce_logits.hpp"

#define ARGREDUCE_EXPORT extern "C" __attribute__((visibility("default")))

namespace argreduce {

constexpr int64_t kBlock = 256;
constexpr int64_t kThreadsPerCu = 2048;
constexpr int64_t kLdsPerCu = 160 * 1024;
constexpr int64_t kMaxGridThreads = int64_t{1} << 32;  // a launch's grid holds fewer threads
constexpr int64_t kMaxBytes = int64_t{1} << 48;        // a device address is below it

inline int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }
inline int64_t next_pow2(int64_t v) {
    int64_t p = 1;
    while (p < v) p <<= 1;
    return p;
}

inline int64_t logits_elem_size(int dtype) {
    switch (dtype) {
        case ARGREDUCE_F32: return 4;
        case ARGREDUCE_F16: return 2;
        case ARGREDUCE_BF16: return 2;
        default: return 0;
    }
}

// 16-byte vectors that a row's bytes lie in, for the worst aligned row.
inline int64_t span_vecs(int64_t cols, int64_t es) { return cols * es / 16 + 2; }

inline int check_logits_shape(int dtype, int64_t rows, int64_t cols) {
    if (logits_elem_size(dtype) == 0) return ARGREDUCE_ERR_UNSUPPORTED_DTYPE;
    if (rows < 0 || cols < 1) return ARGREDUCE_ERR_INVALID_ARG;
    if (cols > std::numeric_limits<int32_t>::max() || rows > std::numeric_limits<int32_t>::max())
        return ARGREDUCE_ERR_TOO_WIDE;
    return ARGREDUCE_OK;
}

// The logits of a call: [rows, cols] with rows `stride` elements apart.
inline int check_rows(const void* x, int dtype, int64_t rows, int64_t cols, int64_t stride) {
    const int rc = check_logits_shape(dtype, rows, cols);
    if (rc != ARGREDUCE_OK) return rc;
    if (rows > 1 && stride > std::numeric_limits<uint32_t>::max()) return ARGREDUCE_ERR_TOO_WIDE;
    if (rows > 1 && stride < cols) return ARGREDUCE_ERR_INVALID_ARG;
    if (rows > 0 && (x == nullptr || reinterpret_cast<uintptr_t>(x) % logits_elem_size(dtype) != 0))
        return ARGREDUCE_ERR_INVALID_ARG;
    if (rows > 1 && stride >= kMaxBytes / logits_elem_size(dtype) / rows) return ARGREDUCE_ERR_TOO_WIDE;
    return ARGREDUCE_OK;
}

// Device addresses carry 16 bits of other arguments in their upper bits (tagged()).
inline bool fits48(const void* p) { return (reinterpret_cast<uintptr_t>(p) >> 48) == 0; }
inline bool aligned(const void* p, uintptr_t n) { return reinterpret_cast<uintptr_t>(p) % n == 0; }
// A device array of `n`-byte elements that a call with rows > 0 needs.
inline bool usable(const void* p, uintptr_t n) { return p != nullptr && aligned(p, n) && fits48(p); }

inline bool grid_too_large(int64_t blocks, int64_t threads) { return blocks >= kMaxGridThreads / threads; }

// The caller's scratch aligned up to 16 bytes in *out; an ARGREDUCE_* status.
inline int scratch_of(size_t need, void* scratch, size_t bytes, uint8_t** out) {
    *out = nullptr;
    if (need == 0) return ARGREDUCE_OK;
    if (scratch == nullptr || bytes < need) return ARGREDUCE_ERR_SCRATCH_TOO_SMALL;
    if (!fits48(scratch)) return ARGREDUCE_ERR_INVALID_ARG;
    *out = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(scratch) + 15u) &
                                      ~static_cast<uintptr_t>(15u));
    return ARGREDUCE_OK;
}

inline int status_of(hipError_t e) { return e == hipSuccess ? ARGREDUCE_OK : ARGREDUCE_ERR_HIP; }

}  // namespace argreduce
