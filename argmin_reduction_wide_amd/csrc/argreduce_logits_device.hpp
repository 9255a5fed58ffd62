// Device-side building blocks of the kernels that read logits: a row as its aligned vectors, the
// online softmax over it, and the selection of its best elements. (Helpers have internal linkage:
// each translation unit compiles its own.)
//
// Products and sums are fused where the source says so and nowhere else, so that two kernels that
// compute the same quantity from the same inputs get the same bits: an including file says
// "#pragma clang fp contract(off)" too, for its own part.
#pragma once

#include <hip/hip_runtime.h>
#include <stdint.h>

#include "argreduce_device.hpp"
#include "argreduce_logits.hpp"

#pragma clang fp contract(off)

namespace argreduce {
namespace {

constexpr float kLowest = -3.402823466e+38f;
constexpr float kLn2 = 0.69314718055994530942f;
constexpr float kZFloor = -16384.0f;
constexpr uint32_t kNoVec = 0xffffffffu;

// ---------------------------------------------------------------------------------------
// Kernel arguments. All of a kernel's arguments have to fit the 14 dwords that the hardware
// preloads into SGPRs at wave launch; the kernels with six pointers get there by carrying
// 16-bit values in the unused upper bits of 48-bit device addresses.

constexpr int kAddrBits = 48;
// (Through a pointer to global memory, so that the accesses are global ones, not flat ones.)
template <typename T>
__device__ inline T* addr(uint64_t a) {
    typedef __attribute__((address_space(1))) uint8_t Global;
    return (T*)(Global*)(a & ((uint64_t{1} << kAddrBits) - 1));
}
__device__ inline uint32_t tag(uint64_t a) { return static_cast<uint32_t>(a >> kAddrBits); }
__device__ inline uint32_t tags(uint64_t lo, uint64_t hi) { return tag(lo) | (tag(hi) << 16); }

inline uint64_t tagged(const void* p, uint32_t t) {
    return reinterpret_cast<uintptr_t>(p) | (static_cast<uint64_t>(t & 0xffffu) << kAddrBits);
}
inline uint32_t bits_of(float f) { return __builtin_bit_cast(uint32_t, f); }

// ---------------------------------------------------------------------------------------
// Arithmetic and lanes

__device__ inline float exp2_f(float v) { return __builtin_amdgcn_exp2f(v); }
__device__ inline float log2_f(float v) { return __builtin_amdgcn_logf(v); }
// One instruction each; the C functions add a canonicalisation of every operand.
__device__ inline float max_f(float a, float b) {
    float r;
    asm("v_max_f32 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
    return r;
}
__device__ inline float max3_f(float a, float b, float c) {
    float r;
    asm("v_max3_f32 %0, %1, %2, %3" : "=v"(r) : "v"(a), "v"(b), "v"(c));
    return r;
}

// Reduction over aligned groups of G lanes; every lane gets the result, and the same one:
// each step combines two values that all lanes of a half share.
template <int G, typename Op>
__device__ inline float lanes_all(float v, Op op) {
    if constexpr (G >= 2) v = op(v, dpp_val<0xB1, 0xf>(v));
    if constexpr (G >= 4) v = op(v, dpp_val<0x4E, 0xf>(v));
    if constexpr (G >= 8) v = op(v, dpp_val<0x141, 0xf>(v));
    if constexpr (G >= 16) v = op(v, dpp_val<0x140, 0xf>(v));
    if constexpr (G >= 32) v = op(v, __shfl_xor(v, 16));
    if constexpr (G >= 64) v = op(v, __shfl_xor(v, 32));
    return v;
}
template <int G>
__device__ inline float lanes_max(float v) {
    return lanes_all<G>(v, [](float a, float b) { return max_f(a, b); });
}
template <int G>
__device__ inline float lanes_sum(float v) {
    return lanes_all<G>(v, [](float a, float b) { return a + b; });
}

// The sum of G lanes' values in binary64, in every lane (by DPP and lane swaps: six shuffles through LDS
// took 900 cycles).
template <int CTRL>
__device__ inline double dpp64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    const uint32_t lo = dpp_u32<CTRL, 0xf>(static_cast<uint32_t>(u));
    const uint32_t hi = dpp_u32<CTRL, 0xf>(static_cast<uint32_t>(u >> 32));
    return __builtin_bit_cast(double, static_cast<uint64_t>(hi) << 32 | lo);
}
// v of each lane's own half of 32 (HALF 16) or 64 (HALF 32) lanes and of the other one: the same two in both.
template <int HALF>
__device__ inline void halves(uint32_t v, uint32_t& a, uint32_t& b) {
    const auto r = HALF == 16 ? __builtin_amdgcn_permlane16_swap(v, v, false, false)
                              : __builtin_amdgcn_permlane32_swap(v, v, false, false);
    a = r[0];
    b = r[1];
}
template <int HALF>
__device__ inline void halves64(double v, double& a, double& b) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v);
    uint32_t l[2], h[2];
    halves<HALF>(static_cast<uint32_t>(u), l[0], l[1]);
    halves<HALF>(static_cast<uint32_t>(u >> 32), h[0], h[1]);
    a = __builtin_bit_cast(double, static_cast<uint64_t>(h[0]) << 32 | l[0]);
    b = __builtin_bit_cast(double, static_cast<uint64_t>(h[1]) << 32 | l[1]);
}
template <int G = kWave>
__device__ inline double lanes_sum64(double v) {
    static_assert(G >= 16, "whole rows of lanes");
    v += dpp64<0xB1>(v);
    v += dpp64<0x4E>(v);
    v += dpp64<0x141>(v);
    v += dpp64<0x140>(v);
    double a, b;
    if constexpr (G >= 32) {
        halves64<16>(v, a, b);
        v = a + b;
    }
    if constexpr (G >= 64) {
        halves64<32>(v, a, b);
        v = a + b;
    }
    return v;
}

// A team is one wavefront (T == 64, four teams to a workgroup) or one workgroup of T threads.
// The barrier orders LDS accesses only: __syncthreads() would also wait for every load and store
// to global memory under way, which no team exchanges anything through.
template <int T>
__device__ inline void team_sync() {
    if constexpr (T == kWave) {
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        __builtin_amdgcn_wave_barrier();
    } else {
        __builtin_amdgcn_fence(__ATOMIC_RELEASE, "workgroup", "local");
        __builtin_amdgcn_s_barrier();
        __builtin_amdgcn_fence(__ATOMIC_ACQUIRE, "workgroup", "local");
    }
}

// A thread's team in its workgroup and its lane in the team; the team as a wave-uniform value, so
// that row addresses stay in scalar registers.
template <int T>
__device__ inline uint32_t team_of() {
    if constexpr (T == kWave)
        return __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    else
        return 0;
}
template <int T>
__device__ inline int lane_of() {
    return T == kWave ? threadIdx.x % kWave : threadIdx.x;
}

template <int T>
constexpr int kTeamsPerBlock = T == kWave ? kBlockThreads / kWave : 1;
template <int T>
constexpr int kTeamBlock = T == kWave ? kBlockThreads : T;

// ln p of a logit v in a row of maximum m: in units of e, not of 2, since (v - m) k can leave
// binary32's range where (v - m) / T does not (v the lowest finite value, as some masks have it).
__device__ inline float ln_p(float v, float m, float l2, float scale) {
    return fmaf(v - m, scale * kLn2, -l2 * kLn2);
}

struct Stat {
    float m, s, h;
    __device__ void init() {
        m = kLowest;
        s = 0.0f;
        h = 0.0f;
    }
    // Expresses the part relative to the maximum `to` >= m.
    template <bool ENT>
    __device__ void move(float to, float k) {
        const float d = (to - m) * k;
        const float r = exp2_f(-d);
        if constexpr (ENT) h = r * fmaf(-fminf(d, -kZFloor), s, h);
        s *= r;
        m = to;
    }
};

// A team's LDS words per wavefront: three for team_merge, and one for each reduction of a row.
enum Slot { kSlotMax = 3, kSlotSum, kSlotEntropy, kSlotLoss, kShared = 8 };

// A value that every lane of the wavefront holds, as a scalar.
__device__ inline float uniform(float v) {
    return __uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(v)));
}

// Merges the lanes' parts; every thread of the team gets the row's. The wavefronts' parts go
// through LDS; each wavefront then merges them all, one per lane of each group of T / 64 lanes.
template <bool ENT, int T>
__device__ inline void team_merge(Stat& a, float k, int lane, float (*sh)[kShared]) {
    a.move<ENT>(lanes_max<kWave>(a.m), k);
    a.s = lanes_sum<kWave>(a.s);
    if constexpr (ENT) a.h = lanes_sum<kWave>(a.h);
    if constexpr (T > kWave) {
        constexpr int kWaves = T / kWave;
        if (lane % kWave == 0) {
            sh[lane / kWave][0] = a.m;
            sh[lane / kWave][1] = a.s;
            sh[lane / kWave][2] = a.h;
        }
        team_sync<T>();
        const float* w = sh[lane % kWaves];
        a = {w[0], w[1], ENT ? w[2] : 0.0f};
        a.move<ENT>(lanes_max<kWaves>(a.m), k);
        a.s = lanes_sum<kWaves>(a.s);
        if constexpr (ENT) a.h = lanes_sum<kWaves>(a.h);
        team_sync<T>();
    }
    a = {uniform(a.m), uniform(a.s), uniform(a.h)};
}

// One barrier: a slot is written again only for the team's next row, and other barriers lie between.
template <int T, bool MAX>
__device__ inline float team_reduce(float v, int lane, float (*sh)[kShared], Slot slot) {
    v = MAX ? lanes_max<kWave>(v) : lanes_sum<kWave>(v);
    if constexpr (T > kWave) {
        if (lane % kWave == 0) sh[lane / kWave][slot] = v;
        team_sync<T>();
        v = sh[lane % (T / kWave)][slot];
        v = MAX ? lanes_max<T / kWave>(v) : lanes_sum<T / kWave>(v);
    }
    return uniform(v);
}

// ---------------------------------------------------------------------------------------
// A row as the aligned 16-byte vectors that its bytes lie in. Vector v holds the elements
// v * VW - off .. + VW - 1; vectors [va, vb) lie wholly in the row, the first and the last may
// not ("edges", lanes 0 and 1). An edge vector is read whole: it holds a byte of the row, so
// it lies in a mapped page.

// KEEP: ordinary loads, which leave the logits in the Infinity Cache for a gradient call to read;
// else nontemporal ones, for logits too large for it (kKeepBytes has the figures of both).
template <typename Fmt, bool KEEP = false>
struct Span {
    const uint8_t* base;
    uint32_t off, cols, vs, va, vb;
    __device__ Span(const uint8_t* row, uint32_t n) {
        const uintptr_t a = reinterpret_cast<uintptr_t>(row);
        base = row - (a & 15);
        off = static_cast<uint32_t>(a & 15) / Fmt::kSize;
        cols = n;
        const uint32_t end = off + n;  // n <= INT32_MAX
        vs = (end + Fmt::VW - 1) / Fmt::VW;
        va = off ? 1 : 0;
        vb = end % Fmt::VW ? vs - 1 : vs;
        vb = vb < va ? va : vb;
    }
    // The edge vector of lane 0 or 1, or kNoVec.
    __device__ uint32_t edge(int lane) const {
        if (lane == 0) return off ? 0u : kNoVec;
        return (lane == 1 && (off + cols) % Fmt::VW && (vs > 1 || !off)) ? vs - 1 : kNoVec;
    }
    __device__ const uint8_t* at(uint32_t v) const { return base + static_cast<size_t>(v) * 16; }
    __device__ typename Fmt::Vec load(uint32_t v) const {
        const auto* p = reinterpret_cast<const typename Fmt::Vec*>(at(v));
        if constexpr (KEEP)
            return *p;
        else
            return __builtin_nontemporal_load(p);
    }
    // A vector that lies wholly in the row.
    __device__ typename Fmt::Vec load_whole(uint32_t v) const { return load(v); }
    // Position of element 0 of vector v (wraps for elements before the row).
    __device__ uint32_t pos(uint32_t v) const { return v * Fmt::VW - off; }
};

// A vector of -inf.
template <typename Fmt>
__device__ inline typename Fmt::Vec masked16() {
    constexpr uint32_t w = std::is_same<Fmt, F32>::value   ? 0xff800000u
                           : std::is_same<Fmt, F16>::value ? 0xfc00fc00u
                                                           : 0xff80ff80u;
    return __builtin_bit_cast(typename Fmt::Vec, u32x4{w, w, w, w});
}
template <typename Fmt>
__device__ inline typename Fmt::Vec masked_unless(bool in, const typename Fmt::Vec& v) {
    const u32x4 a = __builtin_bit_cast(u32x4, v), b = __builtin_bit_cast(u32x4, masked16<Fmt>());
    return __builtin_bit_cast(typename Fmt::Vec,
                              u32x4{in ? a.x : b.x, in ? a.y : b.y, in ? a.z : b.z, in ? a.w : b.w});
}

// The same of a row counted from its first element, wherever that lies (the hardware reads a vector at
// any element's address): lanes and sums do not depend on the row's address, so equal rows have equal
// statistics. Vectors [0, vb) lie wholly in the row; what is left past them is the one edge, read element
// by element.
template <typename Fmt>
struct RowSpan {
    const uint8_t* base;
    uint32_t cols, va, vb;
    __device__ RowSpan(const uint8_t* row, uint32_t n) : base(row), cols(n), va(0), vb(n / Fmt::VW) {}
    __device__ uint32_t edge(int lane) const { return lane == 0 && cols % Fmt::VW ? vb : kNoVec; }
    __device__ typename Fmt::Vec load_whole(uint32_t v) const {
        typedef typename Fmt::Vec __attribute__((aligned(2))) Anywhere;
        return __builtin_nontemporal_load(reinterpret_cast<const Anywhere*>(base + static_cast<size_t>(v) * 16));
    }
    // The edge, -inf past the row's end.
    __device__ typename Fmt::Vec load_tail() const {
        struct Bits {
            typename Fmt::Bits b[Fmt::VW];
        };
        const auto* p = reinterpret_cast<const typename Fmt::Bits*>(base + static_cast<size_t>(vb) * 16);
        Bits t = __builtin_bit_cast(Bits, masked16<Fmt>());
#pragma unroll
        for (uint32_t i = 0; i < Fmt::VW; ++i)
            if (i < cols % Fmt::VW) t.b[i] = p[i];
        return __builtin_bit_cast(typename Fmt::Vec, t);
    }
    __device__ typename Fmt::Vec load(uint32_t v) const { return v < vb ? load_whole(v) : load_tail(); }
    __device__ uint32_t pos(uint32_t v) const { return v * Fmt::VW; }
};

// Vectors a lane reads per step of a scan: four, or 16 elements where the alternatives' segments
// take registers too ([2048,128256] bf16, T = 512, four and two vectors: 87 and 93 us without
// alternatives, 107 and 98 with 64 of them).
template <typename Fmt, bool TOP>
constexpr int kUnroll = TOP ? 16 / Fmt::VW : 4;

// Takes N (even) elements into the running part; returns the larger of `m` and their maximum.
template <bool ENT, int N>
__device__ inline float take(const float (&e)[N], float k, Stat& a, float m = kLowest) {
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max3_f(m, e[i], e[i + 1]);
    a.move<ENT>(max_f(a.m, m), k);
#pragma unroll
    for (int i = 0; i < N; ++i) {
        const float z = (e[i] - a.m) * k;
        const float p = exp2_f(z);
        a.s += p;
        if constexpr (ENT) a.h = fmaf(p, max_f(z, kZFloor), a.h);
    }
    return m;
}

template <typename Fmt, int U>
__device__ inline void unpack_all(const typename Fmt::Vec (&q)[U], float (&e)[U * Fmt::VW]) {
#pragma unroll
    for (int u = 0; u < U; ++u) {
        float f[Fmt::VW];
        Fmt::unpack(q[u], f);
#pragma unroll
        for (int i = 0; i < Fmt::VW; ++i) e[u * Fmt::VW + i] = f[i];
    }
}
template <int N>
__device__ inline float max_of(const float (&e)[N]) {
    float m = e[0];
#pragma unroll
    for (int i = 1; i + 1 < N; i += 2) m = max3_f(m, e[i], e[i + 1]);
    return N % 2 ? m : max_f(m, e[N - 1]);
}

// The edge vector of lane 0 or 1.
template <typename Fmt, bool ENT, typename Sp>
__device__ inline void scan_edge(const Sp& sp, int lane, float k, Stat& a) {
    const uint32_t v = sp.edge(lane);
    if (v == kNoVec) return;
    float e[Fmt::VW];
    Fmt::unpack(sp.load(v), e);
    const uint32_t p0 = sp.pos(v);
#pragma unroll
    for (int i = 0; i < Fmt::VW; ++i) e[i] = p0 + i < sp.cols ? e[i] : -__builtin_huge_valf();
    take<ENT>(e, k, a);
}

// The segments of vectors [first, last) whose maxima a scan by T lanes in steps of U vectors per
// lane leaves for top_select, at most `most` of them: single vectors, or eight neighbouring ones
// (whole 128-byte lines), or eight lanes' vectors of `group` steps.
struct Segments {
    uint32_t first, last, lg_vecs, group, row;  // row: vectors between two of a lane's
    int oct;
    template <int T, int U>
    __device__ static Segments cut(uint32_t first, uint32_t last, uint32_t most) {
        const uint32_t n = last - first, steps = (n + U * T - 1) / (U * T);
        Segments g{first, last, 0, 0, T, T / 8};
        if (n > most) {
            g.lg_vecs = 3;
            if (n > 8 * most) {
                g.group = (steps * g.oct + most - 1) / most;
                g.lg_vecs = 32 - __clz(8 * U * g.group - 1);
            }
        }
        g.group *= U;
        return g;
    }
    __device__ uint32_t count() const {
        const uint32_t n = last - first;
        return group == 0 ? (n + (1u << lg_vecs) - 1) >> lg_vecs : (n + group * row - 1) / (group * row) * oct;
    }
    // Vector i (of 2^lg_vecs) of segment s, or kNoVec.
    __device__ uint32_t vec(uint32_t s, uint32_t i) const {
        uint32_t v;
        if (group == 0) {
            v = first + (s << lg_vecs) + i;
        } else {
            if (i / 8 >= group) return kNoVec;
            v = first + (s / oct * group + i / 8) * row + s % oct * 8 + i % 8;
        }
        return v < last ? v : kNoVec;
    }
};

// One lane's share of a row: its edge vector (scan_span), then vectors first + lane, + T, ... below
// last: in steps of U vectors, and the last, incomplete step one by one, lanes past the end with
// -inf. With SEG the maxima of g's segments go to seg[].
template <typename Fmt, bool ENT, int T, int U, bool SEG = false, typename Sp>
__device__ inline void scan_on(const Sp& sp, uint32_t first, uint32_t last, int lane, float k, Stat& a,
                               const Segments& g = Segments{}, float* seg = nullptr) {
    constexpr int VW = Fmt::VW;
    using Vec = typename Fmt::Vec;
    float m = kLowest;  // of the running group of segments
    uint32_t left = g.group, at = lane / 8;
    const auto vector_max = [&](const float(&f)[VW], uint32_t i) {  // segments of one or eight vectors
        float v = max_of(f);
        if (g.lg_vecs) v = lanes_max<8>(v);
        if (i < last - first && (i & ((1u << g.lg_vecs) - 1)) == 0) seg[i >> g.lg_vecs] = v;
    };
    const auto group_max = [&] {
        m = lanes_max<8>(m);
        if (lane % 8 == 0) seg[at] = m;
        m = kLowest;
        left = g.group;
        at += T / 8;
    };
    uint32_t base = first;
    for (; last - base >= U * T; base += U * T) {
        Vec q[U];
        float e[U * VW];
#pragma unroll
        for (int u = 0; u < U; ++u) q[u] = sp.load_whole(base + lane + u * T);
        unpack_all<Fmt, U>(q, e);
        if constexpr (SEG) {
            if (g.group == 0) {
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    float f[VW];
                    Fmt::unpack(q[u], f);
                    vector_max(f, base - first + lane + u * T);
                }
                take<ENT>(e, k, a);
            } else {
                m = take<ENT>(e, k, a, m);
                left -= U;
                if (left == 0) group_max();
            }
        } else {
            take<ENT>(e, k, a);
        }
    }
    if (base < last) {
        Vec q[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            const uint32_t v = base + lane + u * T;
            if (base + u * T < last) q[u] = sp.load_whole(v < last ? v : last - 1);
        }
#pragma unroll
        for (int u = 0; u < U; ++u) {
            if (base + u * T < last) {
                float f[VW];
                Fmt::unpack(masked_unless<Fmt>(base + lane + u * T < last, q[u]), f);
                if constexpr (SEG) {
                    if (g.group == 0) vector_max(f, base - first + lane + u * T);
                    m = take<ENT>(f, k, a, g.group ? m : kLowest);
                } else {
                    take<ENT>(f, k, a);
                }
            }
        }
        if constexpr (SEG) left = 0;
    }
    if constexpr (SEG)
        if (g.group != 0 && left != g.group) group_max();
}
template <typename Fmt, bool ENT, int T, int U, bool SEG = false, typename Sp>
__device__ inline void scan_span(const Sp& sp, bool edges, uint32_t first, uint32_t last, int lane,
                                 float k, Stat& a, const Segments& g = Segments{}, float* seg = nullptr) {
    a.init();
    if (edges && lane < 2) scan_edge<Fmt, ENT>(sp, lane, k, a);
    scan_on<Fmt, ENT, T, U, SEG>(sp, first, last, lane, k, a, g, seg);
}

// ---------------------------------------------------------------------------------------
// The k best elements of a row, by (value descending, position ascending).
//
// A pass over the row leaves the maximum of each of S segments (struct Segments). For a tau that at
// least k of these maxima reach, the k best elements are all >= tau and lie in segments whose
// maximum is >= tau: only these are read again, from the caches, and their elements >= tau collected
// in LDS as 64-bit keys (value above complemented position). Ranking the keys by counting gives the
// sorted result. tau comes from a bisection that stops when few more than k maxima reach it. Ties
// may put more keys into the buffer than it holds; the collection then starts again in steps that
// cannot overflow it, the buffer cut to its k best in between.

__device__ inline uint64_t key_of(float v, uint32_t pos) { return Key32<kMax>::make(v, pos); }
// Unsigned integers in the order of the floats, and back.
__device__ inline uint32_t order_of(float v) {
    const uint32_t u = __float_as_uint(v);
    return (u >> 31) ? ~u : (u | 0x80000000u);
}
__device__ inline float value_of(uint32_t o) {
    return __uint_as_float((o >> 31) ? (o & 0x7fffffffu) : ~o);
}

template <int T, int S>
struct TopLds {
    static constexpr int kStep = T / 4;  // vectors per step of the bounded collection
    static constexpr int kCap = 8 * kStep + kTopMax;
    uint64_t buf[kCap];
    uint64_t best[T];
    float seg[S];
    uint16_t list[S];
    uint32_t count, listed;
    float tau;
    uint64_t least;  // keys at or below it cannot be among the k best
};

// Cuts the buffer to its k best keys, sorted. Called by the whole team after a team_sync.
template <int T, int S>
__device__ inline void top_cut(TopLds<T, S>& L, int lane, uint32_t k) {
    constexpr int kPer = (TopLds<T, S>::kCap + T - 1) / T;
    uint32_t n = L.count;
    if (n > 2 * kTopMax + 64) {
        // the k-th largest of the threads' own maxima bounds the k-th best key from below
        uint64_t mine[kPer], top = 0;
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const uint32_t i = lane + j * T;
            mine[j] = i < n ? L.buf[i] : 0;
            top = mine[j] > top ? mine[j] : top;
        }
        L.best[lane] = top;
        if (lane == 0) L.least = 0;
        team_sync<T>();
        uint32_t above = 0;
        for (int j = 0; j < T; ++j) above += L.best[j] > top ? 1 : 0;
        if (top != 0 && above == k - 1) L.least = top;
        if (lane == 0) L.count = 0;
        team_sync<T>();
        const uint64_t least = L.least;
#pragma unroll
        for (int j = 0; j < kPer; ++j)
            if (mine[j] != 0 && mine[j] >= least) L.buf[atomicAdd(&L.count, 1u)] = mine[j];
        team_sync<T>();
        n = L.count;
    }
    // ranks: kShare lanes count for a key, each over every kShare-th of the others
    constexpr int kShare = T >= 512 ? 4 : (T >= 256 ? 2 : 1);
    for (uint32_t i = lane / kShare; i < n; i += T / kShare) {
        const uint64_t key = L.buf[i];
        uint32_t above = 0;
#pragma unroll 4
        for (uint32_t j = lane % kShare; j < n; j += kShare) above += L.buf[j] > key ? 1 : 0;
        if constexpr (kShare >= 2) above += dpp_u32<0xB1, 0xf>(above);
        if constexpr (kShare >= 4) above += dpp_u32<0x4E, 0xf>(above);
        if (above < k) L.best[above] = key;
    }
    team_sync<T>();
    const uint32_t kept = n < k ? n : k;
    if (static_cast<uint32_t>(lane) < kept) L.buf[lane] = L.best[lane];
    if (lane == 0) {
        L.count = kept;
        L.least = kept == k ? L.best[k - 1] : 0;
    }
    team_sync<T>();
}

// The low bits that every value of a format, as an ordered integer, has alike.
template <typename Fmt>
constexpr int kLowBits = std::is_same<Fmt, F32>::value ? 0 : std::is_same<Fmt, F16>::value ? 13 : 16;

// Bisection for kth_bound over N maxima per lane: N comparisons a step, the counts from lane masks. Stops
// when at most `enough` maxima reach the bound.
template <int N>
__device__ inline uint32_t bisect(const uint32_t (&o)[N], uint32_t k, uint32_t enough) {
    uint32_t hi = 0, lo = 0;
#pragma unroll
    for (int j = 0; j < N; ++j) {
        hi = o[j] > hi ? o[j] : hi;
        lo = o[j] != 0 && ~o[j] > lo ? ~o[j] : lo;
    }
    hi = wave_max_u32(hi) + 1;
    lo = ~wave_max_u32(lo);
    while (hi - lo > 1) {
        const uint32_t mid = lo + (hi - lo) / 2;
        uint32_t n = 0;
#pragma unroll
        for (int j = 0; j < N; ++j) n += __popcll(__ballot(o[j] >= mid));
        if (n >= k) {
            lo = mid;
            if (n <= enough) break;
        } else {
            hi = mid;
        }
    }
    return lo;
}

template <int N>
__device__ inline uint32_t bisect(const uint32_t (&o)[N], uint32_t k) {
    return bisect(o, k, k + k / 8 + 2);
}

// A value that at least k, and if the values allow few more, of the `segs` maxima reach (the
// lowest finite value if there are fewer than k). One wavefront computes it, from the maxima of
// 64 N groups of segments: with k / (64 N) = 1/4 groups above it, about 11% more segments than
// groups are. N = 4, or 1 for few alternatives; all 16 or 32 maxima of a lane in each step
// measured 2.5 to 5.9 us here, a third of the time that the alternatives cost.
template <typename Fmt, int S>
__device__ inline float kth_bound(const float* seg, uint32_t segs, uint32_t k, int lane) {
    constexpr int kPer = (S + kWave - 1) / kWave, N = kPer < 4 ? kPer : 4;
    if (segs < k) return kLowest;
    float m[N];
#pragma unroll
    for (int j = 0; j < N; ++j) m[j] = -__builtin_huge_valf();
#pragma unroll
    for (int j = 0; j < kPer; ++j) {
        const uint32_t s = lane + j * kWave;
        if (s < segs) m[j % N] = max_f(m[j % N], seg[s]);
    }
    uint32_t o[N], bound;
#pragma unroll
    for (int j = 0; j < N; ++j)
        o[j] = lane + static_cast<uint32_t>(j) * kWave < segs ? order_of(m[j]) >> kLowBits<Fmt> : 0;
    if (k <= kWave / 4) {
        uint32_t top[1] = {o[0]};
#pragma unroll
        for (int j = 1; j < N; ++j) top[0] = o[j] > top[0] ? o[j] : top[0];
        bound = bisect(top, k);
    } else {
        bound = bisect(o, k);
    }
    bound <<= kLowBits<Fmt>;  // below the lowest finite value: segments of masked elements alone
    return bound > order_of(kLowest) ? value_of(bound) : kLowest;
}

// `segs` maxima are in L.seg. `vec(seg, i)` names vector i (of 2^lg_seg) of a segment, or kNoVec;
// `edges`: the row's edge vectors are looked at too. Leaves the k best (fewer if there are fewer) in
// L.buf, their number in L.count.
template <typename Fmt, int T, int S, typename Sp, typename VecOf>
__device__ inline void top_select(TopLds<T, S>& L, const Sp& sp, uint32_t segs,
                                  uint32_t lg_seg, uint32_t k, int lane, VecOf vec,
                                  bool edges = true) {
    constexpr int VW = Fmt::VW;
    constexpr int U = 4;  // vectors a thread reads at once
    if (lane == 0) {
        L.count = 0;
        L.listed = 0;
        L.least = 0;
    }
    team_sync<T>();
    if (lane < kWave) {
        const float t = kth_bound<Fmt, S>(L.seg, segs, k, lane);
        if (lane == 0) L.tau = t;
    }
    team_sync<T>();
    const float tau = L.tau;
    for (uint32_t s = lane; s < segs; s += T)
        if (L.seg[s] >= tau) L.list[atomicAdd(&L.listed, 1u)] = static_cast<uint16_t>(s);
    team_sync<T>();
    const uint32_t main_items = L.listed << lg_seg;
    const uint32_t items = main_items + (edges ? 2 : 0);
    const auto item_vec = [&](uint32_t it) {
        if (it < main_items) return vec(L.list[it >> lg_seg], it & ((1u << lg_seg) - 1));
        return it < items ? sp.edge(static_cast<int>(it - main_items)) : kNoVec;
    };
    const auto visit = [&](const typename Fmt::Vec& q, uint32_t v, uint64_t least, bool bounded) {
        float e[VW];
        Fmt::unpack(q, e);
        if (v == kNoVec || !(max_of(e) >= tau)) return;
        const uint32_t p0 = sp.pos(v);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            if (e[i] >= tau && p0 + i < sp.cols) {
                const uint64_t key = key_of(e[i], p0 + i);
                if (key > least) {
                    const uint32_t at = atomicAdd(&L.count, 1u);
                    if (!bounded || at < TopLds<T, S>::kCap) L.buf[at] = key;
                }
            }
        }
    };
    for (uint32_t it = lane; it < items; it += U * T) {
        typename Fmt::Vec q[U];
        uint32_t v[U];
#pragma unroll
        for (int u = 0; u < U; ++u) {
            v[u] = item_vec(it + u * T);
            q[u] = sp.load(v[u] == kNoVec ? 0 : v[u]);  // vector 0 can always be read
        }
#pragma unroll
        for (int u = 0; u < U; ++u)
            if (it + u * T < items) visit(q[u], v[u], 0, true);
    }
    team_sync<T>();
    if (L.count > TopLds<T, S>::kCap) {
        constexpr uint32_t kStep = TopLds<T, S>::kStep;
        team_sync<T>();
        if (lane == 0) L.count = 0;
        for (uint32_t base = 0; base < items; base += kStep) {
            team_sync<T>();
            if (L.count > kTopMax) top_cut(L, lane, k);  // then 8 kStep more keys fit
            const uint64_t least = L.least;
            team_sync<T>();
            if (static_cast<uint32_t>(lane) < kStep) {
                const uint32_t v = item_vec(base + lane);
                visit(sp.load(v == kNoVec ? 0 : v), v, least, false);
            }
        }
        team_sync<T>();
    }
    top_cut(L, lane, k);
}

// ---------------------------------------------------------------------------------------
// Rows, slices of a row, and vectors at any address.

template <typename Fmt>
__device__ inline float load_at(const uint8_t* row, int64_t t, uint32_t cols) {
    return t < static_cast<int64_t>(cols) ? Fmt::load1(row + t * Fmt::kSize) : __builtin_nanf("");
}
__device__ inline uint32_t ceil_log2(uint32_t v) { return v <= 1 ? 0 : 32 - __clz(v - 1); }
template <typename Fmt>
__device__ inline const uint8_t* row_ptr(const void* x, uint32_t r, uint32_t stride) {
    return static_cast<const uint8_t*>(x) + static_cast<size_t>(r) * stride * Fmt::kSize;
}

// Segments of a row with alternatives, at most.
template <int T>
constexpr int kSegs = T == kWave ? 256 : 1024;

// Slice b of a row split over `parts` workgroups: vectors [first, last).
__device__ inline uint32_t part_vecs(uint32_t span_max, uint32_t parts) {
    return (span_max + parts - 1) / parts;
}
template <typename Fmt>
__device__ inline uint32_t span_max(uint32_t cols) {  // vectors of the worst aligned row
    return cols / Fmt::VW + 2;
}
template <typename Fmt>
struct Unaligned {
    typename Fmt::Vec v;
} __attribute__((packed, aligned(2)));

template <typename Fmt>
__device__ inline typename Fmt::Vec load16_any(const uint8_t* p) {
    return reinterpret_cast<const Unaligned<Fmt>*>(p)->v;
}

template <typename Fmt>
__device__ inline void store16_any(uint8_t* p, const typename Fmt::Vec& v) {
    reinterpret_cast<Unaligned<Fmt>*>(p)->v = v;
}

// Rounds to nearest even. binary16 by the instruction: the compiler may join the conversion with
// the product before it, in one kernel and not in another.
template <typename Fmt>
__device__ inline typename Fmt::Bits round_to(float v) {
    if constexpr (Fmt::kSize == 4) {
        return __float_as_uint(v);
    } else if constexpr (std::is_same<Fmt, F16>::value) {
        uint32_t h;
        asm("v_cvt_f16_f32 %0, %1" : "=v"(h) : "v"(v));
        return static_cast<uint16_t>(h);
    } else {
        return __builtin_bit_cast(uint16_t, static_cast<__bf16>(v));
    }
}
template <typename Fmt>
__device__ inline typename Fmt::Vec pack(const float (&g)[Fmt::VW]) {
    typename Fmt::Bits b[Fmt::VW];
#pragma unroll
    for (int i = 0; i < Fmt::VW; ++i) b[i] = round_to<Fmt>(g[i]);
    return __builtin_bit_cast(typename Fmt::Vec, b);
}

// ---------------------------------------------------------------------------------------
// Which workgroup of a launch is the last of several to be done with its part, so that it can join the
// parts: nothing waits, and the words in scratch may hold anything before. Every workgroup stores its part
// with store_part, then the launch's tag into its own slot, and then reads all slots: who finds the tag in
// all of them comes after all parts. Several can find it, and the first of them to put the tag's complement into
// the owner's word is the one. The parts are read with load_part.
//
// The tag is made from the call's nonce, and the replays of a captured call have one nonce, so no word may hold
// the tag before its launch puts it there: the last workgroup clears the slots when it is done (leave), so that
// no launch leaves the tag in any word, and the first one clears the owner before its slot can be seen, and with
// it all slots. What other kernels leave in this memory between two replays then does not matter, nor what of it
// they leave as it was or copy from elsewhere: none of it is the tag.
//
// Parts and slots are agent-scope accesses, which pass the L2 caches of the XCDs; a store is done when its
// wavefront's count of memory operations says so (vmcnt), so that no cache has to be written back.

template <typename T>
__device__ inline void store_part(T* p, T v) {
    __hip_atomic_store(p, v, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
template <typename T>
__device__ inline T load_part(const T* p) {
    return __hip_atomic_load(p, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT);
}
__device__ inline void stores_done() { asm volatile("s_waitcnt vmcnt(0)" ::: "memory"); }

// A nonce as one of 2^64 words (never 0).
__device__ inline uint64_t arrival_tag(uint32_t nonce) {
    uint64_t v = 0x9e3779b97f4a7c15ull * (nonce | uint64_t{1} << 32);
    v = (v ^ (v >> 30)) * 0xbf58476d1ce4e5b9ull;
    v = (v ^ (v >> 27)) * 0x94d049bb133111ebull;
    return v ^ (v >> 31);
}

// Called by the whole workgroup after its last store_part; `found` is in LDS. Whether it is the last of n.
__device__ inline bool arrive(uint64_t* slots, uint64_t* owner, uint32_t mine, uint32_t n, uint64_t tag,
                              uint32_t* found) {
    if (mine == 0 && threadIdx.x == 0) store_part(owner, uint64_t{0});
    stores_done();
    __syncthreads();
    if (threadIdx.x < kWave) {
        if (threadIdx.x == 0) store_part(slots + mine, tag);
        stores_done();
        bool there = true;
        for (uint32_t i = threadIdx.x; i < n; i += kWave) there &= load_part(slots + i) == tag;
        bool one = __ballot(!there) == 0;
        if (threadIdx.x == 0) {
            if (one) one = __hip_atomic_exchange(owner, ~tag, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_AGENT) != ~tag;
            *found = one ? 1 : 0;
        }
    }
    __syncthreads();
    return *found != 0;
}
// Called by the T threads of the last workgroup, once all n slots hold the tag.
template <int T>
__device__ inline void leave(uint64_t* slots, uint32_t n) {
    for (uint32_t i = threadIdx.x; i < n; i += T) store_part(slots + i, uint64_t{0});
}

// ---------------------------------------------------------------------------------------
// Launches.

template <typename F>
inline void with_format(int dtype, F f) {
    switch (dtype) {
        case ARGREDUCE_F32: f(F32{}); break;
        case ARGREDUCE_F16: f(F16{}); break;
        default: f(BF16{}); break;
    }
}
template <int N>
struct Int {
    static constexpr int value = N;
};
template <typename F>
inline void with_bool(bool b, F f) {
    if (b)
        f(Int<1>{});
    else
        f(Int<0>{});
}

inline uint32_t log2_of(int v) { return static_cast<uint32_t>(__builtin_ctz(static_cast<unsigned>(v))); }

template <typename... KArgs, typename... Args>
inline void launch(void (*kernel)(KArgs...), uint32_t grid, int block, hipStream_t s, Args... args) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), 0, s, args...);
}

}  // namespace
}  // namespace argreduce
