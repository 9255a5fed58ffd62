// Expert routing on gfx950: the choice of `top` experts per token from a router's logits, their
// weights, how often every expert is chosen, and two losses that train the router, with the gradient.
//
// For the tokens t of a group and its experts e, with p_t = softmax(x_t), c_e the number of choices of
// expert e, n the number of tokens, k = top and E the number of experts:
//   weights  w_ti = p_t(e_i), or divided by their sum over the token's choices;
//   balance  L = E / (k n^2) sum_e c_e sum_t p_te  (1 where choices or probabilities are even);
//   z        Z = 1 / n sum_t (ln sum_e exp x_te)^2.
// The choice and c are constants of the gradient. With gw, gL, gZ those of weights and losses,
//   dx_tj = p_tj (gL E / (k n^2) (c_j - sum_e c_e p_te) + gZ 2/n ln sum exp x_t) + (weights' part),
//   weights' part  w_ti (gw_ti - sum_l gw_tl w_tl) at j = e_i if they are divided by their sum, else
//                  (gw_ti p_tj at j = e_i) - p_tj sum_l gw_tl p_tl.
//
// A token's logits lie in the registers of a group of G lanes, and a lane's columns are the same for
// all tokens, so that it sums p of its own columns in registers; choices are counted in LDS. A workgroup
// leaves one word of sums per expert in scratch, and the last one of a group adds them up. No atomics on
// floats: results do not depend on the order in which workgroups run.
#include <hip/hip_runtime.h>

#include "argreduce_launch.hpp"
#include "argreduce_logits_device.hpp"
#include "argreduce_route.hpp"

#pragma clang fp contract(off)

namespace argreduce {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr uint32_t kColBits = 10;  // of an expert's number in a key
static_assert(kExpertsMax == 1 << kColBits, "numbers of experts in a key");

// ---------------------------------------------------------------------------------------
// Keys of logits: larger for a larger logit and among equals for the lower expert, so that two keys are
// never equal and a maximum takes one instruction. A logit's bits count as sign and magnitude, which
// makes -0 and +0 alike. Keys below kSome are those of -inf and of nothing.

template <typename Fmt>
struct Key;

// 16-bit formats: the signed value of the bits above 16 bits for the expert.
struct Key16 {
    using T = int32_t;
    static constexpr T kNone = INT32_MIN;
    __device__ static T max(T a, T b) { return a > b ? a : b; }
    __device__ static T min(T a, T b) { return a < b ? a : b; }
    template <int CTRL>
    __device__ static T dpp(T v) {
        return static_cast<T>(dpp_u32<CTRL, 0xf>(static_cast<uint32_t>(v)));
    }
    template <int HALF>
    __device__ static void both(T v, T& a, T& b) {
        uint32_t x, y;
        halves<HALF>(static_cast<uint32_t>(v), x, y);
        a = static_cast<T>(x);
        b = static_cast<T>(y);
    }
    // The keys of a vector's eight elements; the first is expert `col`.
    __device__ static void make(const u32x4 q, uint32_t col, T (&k)[8]) {
        const uint32_t c = kExpertsMax - 1 - col;
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            typedef short s16x2 __attribute__((ext_vector_type(2)));
            const uint32_t two = q[i];  // (a bit cast of q[i] itself would read q[0])
            const s16x2 sign = __builtin_bit_cast(s16x2, two) >> 15;
            const s16x2 magnitude = __builtin_bit_cast(s16x2, two & 0x7fff7fffu);
            const uint32_t v = __builtin_bit_cast(uint32_t, (magnitude ^ sign) - sign);
            k[2 * i] = static_cast<T>(v << 16 | (c - 2 * i));
            k[2 * i + 1] = static_cast<T>((v & 0xffff0000u) | (c - 2 * i - 1));
        }
    }
    __device__ static uint32_t bits(T k) {
        const int32_t v = k >> 16;
        return v < 0 ? 0x8000u | static_cast<uint32_t>(-v) : static_cast<uint32_t>(v);
    }
    __device__ static uint32_t col(T k) { return kExpertsMax - 1 - (static_cast<uint32_t>(k) & (kExpertsMax - 1)); }
};
template <>
struct Key<F16> : Key16 {
    static constexpr T kSome = -0x7bff * 0x10000;  // the lowest finite value's, of the last expert
    __device__ static float value(T k) { return static_cast<float>(__builtin_bit_cast(_Float16, static_cast<uint16_t>(bits(k)))); }
};
template <>
struct Key<BF16> : Key16 {
    static constexpr T kSome = -0x7f7f * 0x10000;
    __device__ static float value(T k) { return __uint_as_float(bits(k) << 16); }
};
// binary32: 32 bits for the value and 10 for the expert, as the mantissa of a binary64 in [1, 2), which has a
// maximum and a minimum in one instruction.
template <>
struct Key<F32> {
    using T = double;
    static constexpr T kNone = 1.0;
    __device__ static T from(uint32_t o, uint32_t low) {
        return __builtin_bit_cast(double, static_cast<uint64_t>(0x3ff00000u | o >> 12) << 32 | (o << 20 | low));
    }
    static constexpr T kSome = 1.0 + 0x00800001 * 0x1p-32;
    __device__ static T max(T a, T b) {
        T r;
        asm("v_max_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    __device__ static T min(T a, T b) {
        T r;
        asm("v_min_f64 %0, %1, %2" : "=v"(r) : "v"(a), "v"(b));
        return r;
    }
    template <int CTRL>
    __device__ static T dpp(T v) {
        return dpp64<CTRL>(v);
    }
    template <int HALF>
    __device__ static void both(T v, T& a, T& b) {
        halves64<HALF>(v, a, b);
    }
    __device__ static void make(const u32x4 q, uint32_t col, T (&k)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const int32_t sign = static_cast<int32_t>(q[i]) >> 31;
            const int32_t v = (static_cast<int32_t>(q[i] & 0x7fffffffu) ^ sign) - sign;
            k[i] = from(static_cast<uint32_t>(v) ^ 0x80000000u, kExpertsMax - 1 - col - i);
        }
    }
    __device__ static float value(T k) {
        const uint64_t u = __builtin_bit_cast(uint64_t, k);
        const int32_t v = static_cast<int32_t>(static_cast<uint32_t>(u >> 20) ^ 0x80000000u);
        return __uint_as_float(v < 0 ? 0x80000000u | static_cast<uint32_t>(-v) : static_cast<uint32_t>(v));
    }
    __device__ static uint32_t col(T k) {
        return kExpertsMax - 1 - (static_cast<uint32_t>(__builtin_bit_cast(uint64_t, k)) & (kExpertsMax - 1));
    }
};

// Sorting networks, descending. A list of L keys in registers is merged with another one by taking the
// larger of each two that stand opposite, which leaves the L largest of both, and sorting those.
template <typename K>
__device__ inline void exchange(typename K::T& a, typename K::T& b) {
    const typename K::T hi = K::max(a, b);
    b = K::min(a, b);
    a = hi;
}
template <typename K, int L>
__device__ inline void sort_merged(typename K::T (&a)[L]) {
#pragma unroll
    for (int d = L / 2; d > 0; d /= 2)
#pragma unroll
        for (int i = 0; i < L; ++i)
            if ((i & d) == 0) exchange<K>(a[i], a[i + d]);
}
template <typename K, int L>
__device__ inline void merge(typename K::T (&a)[L], const typename K::T (&b)[L]) {
#pragma unroll
    for (int i = 0; i < L; ++i) a[i] = K::max(a[i], b[L - 1 - i]);
    sort_merged<K, L>(a);
}
template <typename K>
__device__ inline void sort8(typename K::T* a) {
    constexpr int8_t kPairs[19][2] = {{0, 1}, {2, 3}, {4, 5}, {6, 7}, {0, 2}, {1, 3}, {4, 6}, {5, 7}, {1, 2}, {5, 6},
                                      {0, 4}, {1, 5}, {2, 6}, {3, 7}, {2, 4}, {3, 5}, {1, 2}, {3, 4}, {5, 6}};
#pragma unroll
    for (int i = 0; i < 19; ++i) exchange<K>(a[kPairs[i][0]], a[kPairs[i][1]]);
}

template <typename K, int L>
__device__ inline void sort(typename K::T (&a)[L]) {
    static_assert(L == 8 || L == 16, "lists of eight or sixteen");
    sort8<K>(a);
    if constexpr (L == 16) {
        sort8<K>(a + 8);
        typename K::T hi[8], lo[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            hi[i] = K::max(a[i], a[15 - i]);
            lo[i] = K::min(a[i], a[15 - i]);
        }
        sort_merged<K, 8>(hi);
        sort_merged<K, 8>(lo);
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            a[i] = hi[i];
            a[8 + i] = lo[i];
        }
    }
}

// The L largest of a lane's N keys, sorted.
template <typename K, int L, int N>
__device__ inline void best_of_lane(const typename K::T (&key)[N], typename K::T (&best)[L]) {
    if constexpr (L == 2) {
        best[0] = key[0];
        best[1] = K::kNone;
#pragma unroll
        for (int i = 1; i < N; ++i) {
            best[1] = K::max(best[1], K::min(best[0], key[i]));
            best[0] = K::max(best[0], key[i]);
        }
    } else {
#pragma unroll
        for (int j = 0; j < N; j += L) {
            typename K::T part[L];
#pragma unroll
            for (int i = 0; i < L; ++i) part[i] = j + i < N ? key[j + i] : K::kNone;
            sort<K, L>(part);
            if (j == 0) {
#pragma unroll
                for (int i = 0; i < L; ++i) best[i] = part[i];
            } else {
                merge<K, L>(best, part);
            }
        }
    }
}
// The L largest of G lanes' lists, in every lane.
template <typename K, int G, int L>
__device__ inline void best_of_lanes(typename K::T (&a)[L]) {
    const auto with = [&](auto ctrl) {
        typename K::T b[L];
#pragma unroll
        for (int i = 0; i < L; ++i) b[i] = K::template dpp<decltype(ctrl)::value>(a[i]);
        merge<K, L>(a, b);
    };
    const auto across = [&](auto half) {
        typename K::T b[L];
#pragma unroll
        for (int i = 0; i < L; ++i) K::template both<decltype(half)::value>(a[i], a[i], b[i]);
        merge<K, L>(a, b);
    };
    if constexpr (G >= 2) with(Int<0xB1>{});
    if constexpr (G >= 4) with(Int<0x4E>{});
    if constexpr (G >= 8) with(Int<0x141>{});
    if constexpr (G >= 16) with(Int<0x140>{});
    if constexpr (G >= 32) across(Int<16>{});
    if constexpr (G >= 64) across(Int<32>{});
}
template <typename K, int G>
__device__ inline typename K::T lanes_best(typename K::T v) {
    if constexpr (G >= 2) v = K::max(v, K::template dpp<0xB1>(v));
    if constexpr (G >= 4) v = K::max(v, K::template dpp<0x4E>(v));
    if constexpr (G >= 8) v = K::max(v, K::template dpp<0x141>(v));
    if constexpr (G >= 16) v = K::max(v, K::template dpp<0x140>(v));
    typename K::T a = v, b = v;
    if constexpr (G >= 32) {
        K::template both<16>(v, a, b);
        v = K::max(a, b);
    }
    if constexpr (G >= 64) {
        K::template both<32>(v, a, b);
        v = K::max(a, b);
    }
    return v;
}

// The sum of the lanes i, i + G, i + 2 G ... of a wavefront, in lane i < G (and the others, in other orders). By DPP
// and lane swaps: with three shuffles through LDS for each of 32 columns [16,4096,256] bf16 took 27.3 us instead of 25.5.
template <int G>
__device__ inline float teams_sum(float v) {
    if constexpr (G <= 1) v += dpp_val<0x121, 0xf>(v);
    if constexpr (G <= 2) v += dpp_val<0x122, 0xf>(v);
    if constexpr (G <= 4) v += dpp_val<0x124, 0xf>(v);
    if constexpr (G <= 8) v += dpp_val<0x128, 0xf>(v);
    uint32_t a, b;
    if constexpr (G <= 16) {
        halves<16>(__float_as_uint(v), a, b);
        v = __uint_as_float(a) + __uint_as_float(b);
    }
    if constexpr (G <= 32) {
        halves<32>(__float_as_uint(v), a, b);
        v = __uint_as_float(a) + __uint_as_float(b);
    }
    return v;
}

// A vector of one token's logits from column c on; -inf past the last expert.
template <typename Fmt>
__device__ inline typename Fmt::Vec load_cols(const uint8_t* row, uint32_t c, uint32_t experts) {
    if (c + Fmt::VW <= experts) return load16_any<Fmt>(row + static_cast<size_t>(c) * Fmt::kSize);
    struct Bits {
        typename Fmt::Bits b[Fmt::VW];
    };
    Bits t = __builtin_bit_cast(Bits, masked16<Fmt>());
    const auto* p = reinterpret_cast<const typename Fmt::Bits*>(row) + c;
#pragma unroll
    for (uint32_t i = 0; i < Fmt::VW; ++i)
        if (c + i < experts) t.b[i] = p[i];
    return __builtin_bit_cast(typename Fmt::Vec, t);
}

// A token's maximum and sum of exponentials; e becomes exp(x - m).
template <int G, int N>
__device__ inline void softmax(float (&e)[N], float& m, float& s) {
    m = kLowest;
#pragma unroll
    for (int i = 0; i < N; i += 2) m = max3_f(m, e[i], e[i + 1]);
    m = lanes_max<G>(m);
    s = 0.0f;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        e[i] = exp2_f((e[i] - m) * kLog2e);
        s += e[i];
    }
    s = lanes_sum<G>(s);
}

// ---------------------------------------------------------------------------------------
// Sums over the tokens of a group: one partial per workgroup, joined by the last of up to kRouteSet
// workgroups; of more than that, the sets' partials by the last set's.

// A partial: per expert the sum of its probabilities and how often it was chosen, and one more column for the sum of
// z and the number of tokens. A workgroup's has a word per column, the sum in binary32 below the number; a set's, of
// sums that more than binary32 holds, two. kBatch: columns that a thread loads at once, 16 words (32 would take
// registers from the tokens' part: 157 instead of 72).
struct BlockPart {
    static constexpr uint32_t kWords = 1, kBatch = 16;
    uint64_t w;
    __device__ static BlockPart load(const uint64_t* p) { return {load_part(p)}; }
    __device__ static void store(uint64_t* p, float sum, uint32_t count) {
        store_part(p, static_cast<uint64_t>(count) << 32 | __float_as_uint(sum));
    }
    __device__ double sum() const { return static_cast<double>(__uint_as_float(static_cast<uint32_t>(w))); }
    __device__ uint32_t count() const { return static_cast<uint32_t>(w >> 32); }
};
struct SetPart {
    static constexpr uint32_t kWords = 2, kBatch = 8;
    uint64_t s, n;
    __device__ static SetPart load(const uint64_t* p) { return {load_part(p), load_part(p + 1)}; }
    __device__ static void store(uint64_t* p, double sum, uint32_t count) {
        store_part(p, __builtin_bit_cast(uint64_t, sum));
        store_part(p + 1, static_cast<uint64_t>(count));
    }
    __device__ double sum() const { return __builtin_bit_cast(double, s); }
    __device__ uint32_t count() const { return static_cast<uint32_t>(n); }
};

// A group's words in scratch: owners and slots of its sets, and an owner and slots of the group where there are
// several sets (arrive); partials of workgroups and of sets.
struct Group {
    uint64_t *owners, *slots, *last, *set_slots, *partials, *set_partials;
    __host__ __device__ static uint32_t sets(uint32_t blocks) { return (blocks + kRouteSet - 1) / kRouteSet; }
    __host__ __device__ static size_t words(uint32_t experts, uint32_t blocks) {
        const uint32_t n = sets(blocks);
        const size_t columns = static_cast<size_t>(experts) + 1;
        return 1 + n + (blocks + n) + (BlockPart::kWords * blocks + SetPart::kWords * n) * columns;
    }
    __device__ Group(uint8_t* scratch, uint32_t g, uint32_t experts, uint32_t blocks) {
        const uint32_t n = sets(blocks);
        owners = reinterpret_cast<uint64_t*>(scratch) + g * words(experts, blocks);
        slots = owners + n;
        last = slots + blocks;
        set_slots = last + 1;
        partials = set_slots + n;
        set_partials = partials + static_cast<size_t>(blocks) * (experts + 1);
    }
};

struct JoinLds {
    double share[kRouteThreads];
    uint32_t times[kRouteThreads];
    double red[kRouteThreads / kWave];
};

// Adds up n <= kRouteSet partials: each(expert, sum, count) by the threads of the workgroup in turn, in teams that
// take a share of the partials each where there are fewer experts than threads. Returns the sums of z and of the
// tokens, in the first wavefront.
struct Tail {
    double z;
    uint32_t tokens;
};
template <typename Part, typename Each>
__device__ inline Tail add_up(JoinLds& L, const uint64_t* partials, uint32_t n, uint32_t experts, Each each) {
    constexpr uint32_t kBatch = Part::kBatch;
    static_assert(kRouteSet <= kWave, "a lane for each partial's last column");
    const auto part = [&](uint32_t b, uint32_t c) {
        return Part::load(partials + Part::kWords * (static_cast<size_t>(b) * (experts + 1) + c));
    };
    Part tail{};
    if (threadIdx.x < n) tail = part(threadIdx.x, experts);
    uint32_t wide = kRouteThreads / 8;
    while (wide < kRouteThreads && wide < experts) wide *= 2;
    const uint32_t teams = kRouteThreads / wide, team = threadIdx.x / wide;
    for (uint32_t c0 = 0; c0 < experts; c0 += wide) {
        const uint32_t c = c0 + threadIdx.x % wide;
        double share = 0.0;
        uint32_t times = 0;
        if (c < experts) {
#pragma unroll 1
            for (uint32_t b0 = team; b0 < n; b0 += kBatch * teams) {
                Part w[kBatch];
#pragma unroll
                for (uint32_t i = 0; i < kBatch; ++i) {
                    const uint32_t b = b0 + i * teams;
                    w[i] = b < n ? part(b, c) : Part{};
                }
#pragma unroll
                for (uint32_t i = 0; i < kBatch; ++i) {
                    share += w[i].sum();
                    times += w[i].count();
                }
            }
        }
        if (teams > 1) {
            __syncthreads();
            L.share[threadIdx.x] = share;
            L.times[threadIdx.x] = times;
            __syncthreads();
            if (team == 0)
                for (uint32_t t = 1; t < teams; ++t) {
                    share += L.share[t * wide + threadIdx.x];
                    times += L.times[t * wide + threadIdx.x];
                }
        }
        if (team == 0 && c < experts) each(c, share, times);
    }
    return {lanes_sum64(tail.sum()), static_cast<uint32_t>(lanes_sum64(static_cast<double>(tail.count())))};
}

// Totals of all groups, one after another: counts (int64 [groups, experts]), tokens (int64 [groups]),
// balance and z (float [groups] each).
struct Totals {
    int64_t *counts, *tokens;
    float *balance, *z;
    __device__ Totals(uint8_t* p, uint32_t groups, uint32_t experts) {
        counts = reinterpret_cast<int64_t*>(p);
        tokens = counts + static_cast<size_t>(groups) * experts;
        balance = reinterpret_cast<float*>(tokens + groups);
        z = balance + groups;
    }
};

// A group's balance, z and tokens: `both` is the thread's share of sum_e c_e sum_t p_te, tail that of thread 0.
__device__ inline void finish(JoinLds& L, const Totals& out, double both, Tail tail, uint32_t g, uint32_t experts,
                              uint32_t top) {
    both = lanes_sum64(both);
    if (threadIdx.x % kWave == 0) L.red[threadIdx.x / kWave] = both;
    __syncthreads();
    if (threadIdx.x == 0) {
        both = 0.0;
        for (int i = 0; i < kRouteThreads / kWave; ++i) both += L.red[i];
        const double n = tail.tokens;
        out.tokens[g] = tail.tokens;
        out.balance[g] = n > 0.0 ? static_cast<float>(both * experts / (top * n * n)) : 0.0f;
        out.z[g] = n > 0.0 ? static_cast<float>(tail.z / n) : 0.0f;
    }
}

// One pass over the logits; 24.8 us for [16,4096,256] bf16 with 8 experts per token (40 MB read and written: 1.6 TB/s),
// 14.5 more for each further 65536 tokens. What bounds it is arithmetic, some 1000 vector instructions per eight
// tokens, half of them the lists' exchanges, and 10 us of launch, first loads, sums and the last workgroup's join.
// G lanes per token, NV vectors each: vector v of the token in lane v % G. L: the length of the lists that
// are merged (2, 8 or 16), or 0 for more choices than that, which are taken one by one (16 of [16,4096,256] bf16:
// 43 us, by lists 28.5).
// Tags: experts in x, top (and 0x8000: renormalize) in live, workgroups per group in weights, nonce in
// (chosen, scratch).
template <typename Fmt, int G, int NV, int L>
__global__ __launch_bounds__(kRouteThreads) void k_route(uint64_t x, uint64_t live_, uint64_t weights,
                                                         uint64_t chosen, uint64_t scratch, uint64_t totals,
                                                         uint32_t stride, uint32_t tokens) {
    constexpr int VW = Fmt::VW, N = NV * VW, kTeams = kRouteThreads / G, kWaves = kRouteThreads / kWave;
    using K = Key<Fmt>;
    using T = typename K::T;
    __shared__ float s_sum[kWaves][G * N];
    __shared__ uint32_t s_cnt[G * N];
    __shared__ float s_z[kWaves];
    __shared__ uint32_t s_n[kWaves];
    __shared__ uint32_t s_found;
    __shared__ JoinLds s_join;
    const uint32_t experts = tag(x), top = tag(live_) & 0x7fffu, blocks = tag(weights);
    const bool renormalize = (tag(live_) & 0x8000u) != 0;
    const uint32_t g = blockIdx.x / blocks, b = blockIdx.x - g * blocks;
    const uint32_t per = (tokens + blocks - 1) / blocks;
    const uint32_t t0 = b * per < tokens ? b * per : tokens;
    const uint32_t t1 = tokens - t0 < per ? tokens : t0 + per;
    const uint32_t team = threadIdx.x / G;
    const int lane = threadIdx.x % G;
    const uint8_t* live = addr<const uint8_t>(live_);
    const Group group(addr<uint8_t>(scratch), g, experts, blocks);
    for (int i = threadIdx.x; i < G * N; i += kRouteThreads) s_cnt[i] = 0;
    __syncthreads();
    float sum[N], z = 0.0f;
    uint32_t n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) sum[i] = 0.0f;
    // the next token's logits and the one after's `live` are on their way while a token is worked on
    const auto is_live = [&](uint32_t t) {
        return t < t1 && (live == nullptr || live[static_cast<size_t>(g) * tokens + t] != 0);
    };
    const auto load = [&](uint32_t t, bool on, typename Fmt::Vec(&to)[NV]) {
        const uint8_t* row = addr<const uint8_t>(x) + (static_cast<size_t>(g) * tokens + t) * stride * Fmt::kSize;
#pragma unroll
        for (int v = 0; v < NV; ++v) to[v] = masked16<Fmt>();
        if (on) {
#pragma unroll
            for (int v = 0; v < NV; ++v) to[v] = load_cols<Fmt>(row, (v * G + lane) * VW, experts);
        }
    };
    typename Fmt::Vec next[NV];
    load(t0 + team, is_live(t0 + team), next);
    bool next_on = is_live(t0 + team + kTeams);
    for (uint32_t base = t0; base < t1; base += kTeams) {
        const uint32_t t = base + team;
        const size_t r = static_cast<size_t>(g) * tokens + t;
        const bool there = t < t1;
        typename Fmt::Vec q[NV];
#pragma unroll
        for (int v = 0; v < NV; ++v) q[v] = next[v];
        load(t + kTeams, next_on, next);
        next_on = is_live(t + 2 * kTeams);
        float e[N];
        T key[N];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VW];
            T k[VW];
            Fmt::unpack(q[v], f);
            K::make(__builtin_bit_cast(u32x4, q[v]), (v * G + lane) * VW, k);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                e[v * VW + i] = f[i];
                key[v * VW + i] = k[i];
            }
        }
        float m, s;
        softmax<G, N>(e, m, s);
        const bool ok = s > 0.0f && s < __builtin_huge_valf();
        const bool bad = !(s < __builtin_huge_valf());  // NaN or +inf
        const float inv = 1.0f / s;
        if (s != 0.0f) {  // else left out, or every logit is -inf
            const float lse = fmaf(log2_f(s), kLn2, m);
            if (lane == 0) {
                z = fmaf(lse, lse, z);
                ++n;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) sum[i] = fmaf(e[i], inv, sum[i]);
        }
        float* wt = addr<float>(weights) + r * top;
        int64_t* ch = addr<int64_t>(chosen) + r * top;
        // lane j % G stores choice j
        const auto store = [&](uint32_t j, T k, float w, bool some) {
            ch[j] = some ? static_cast<int64_t>(K::col(k)) : bad ? -2 : -1;
            wt[j] = bad ? __builtin_nanf("") : w;
            if (some) atomicAdd(&s_cnt[K::col(k)], 1u);
        };
        if constexpr (L > 0) {
            constexpr int kRounds = (L + G - 1) / G;
            T best[L];
            best_of_lane<K, L, N>(key, best);
            best_of_lanes<K, G, L>(best);
            T mine[kRounds];
            float w[kRounds], kept = 0.0f;
#pragma unroll
            for (int c = 0; c < kRounds; ++c) {
                mine[c] = K::kNone;
#pragma unroll
                for (int i = c * G; i < L && i < (c + 1) * G; ++i) mine[c] = lane == i - c * G ? best[i] : mine[c];
                const bool some = ok && mine[c] >= K::kSome && static_cast<uint32_t>(c * G + lane) < top;
                w[c] = some ? exp2_f((K::value(mine[c]) - m) * kLog2e) : 0.0f;
                kept += w[c];
            }
            const float scale = renormalize ? 1.0f / lanes_sum<G>(kept) : inv;
#pragma unroll
            for (int c = 0; c < kRounds; ++c) {
                const uint32_t j = c * G + lane;
                if (there && j < top) store(j, mine[c], ok ? w[c] * scale : 0.0f, ok && mine[c] >= K::kSome);
            }
        } else {
            float kept = 0.0f;
            for (uint32_t j0 = 0; j0 < top; j0 += G) {
                T mine = K::kNone;
                const uint32_t j1 = top - j0 < G ? top - j0 : G;
                for (uint32_t j = 0; j < j1; ++j) {
                    T best = key[0];
#pragma unroll
                    for (int i = 1; i < N; ++i) best = K::max(best, key[i]);
                    best = lanes_best<K, G>(best);
                    if (static_cast<uint32_t>(lane) == j) mine = best;
#pragma unroll
                    for (int i = 0; i < N; ++i) key[i] = key[i] == best ? K::kNone : key[i];
                }
                const bool some = ok && mine >= K::kSome;
                const float w = some ? exp2_f((K::value(mine) - m) * kLog2e) : 0.0f;
                kept += w;
                if (there && static_cast<uint32_t>(lane) < j1) store(j0 + lane, mine, some ? w * (renormalize ? 1.0f : inv) : 0.0f, some);
            }
            kept = lanes_sum<G>(kept);
            if (renormalize && there && ok)
                for (uint32_t j = lane; j < top; j += G) wt[j] = wt[j] / kept;
        }
    }
    // the workgroup's sums: of a wavefront's teams by lanes, then of the wavefronts
    const int wave = threadIdx.x / kWave;
    z = lanes_sum<kWave>(z);
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) n += __shfl_xor(n, o);
    if (threadIdx.x % kWave == 0) {
        s_z[wave] = z;
        s_n[wave] = n;
    }
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const float t = teams_sum<G>(sum[v * VW + i]);
            if (threadIdx.x % kWave < G) s_sum[wave][(v * G + lane) * VW + i] = t;
        }
    __syncthreads();
    const Totals out(addr<uint8_t>(totals), gridDim.x / blocks, experts);
    uint64_t* part = group.partials + static_cast<size_t>(b) * (experts + 1);
    int64_t* counts = out.counts + static_cast<size_t>(g) * experts;
    double both = 0.0;
    for (uint32_t c = threadIdx.x; c < experts; c += kRouteThreads) {
        float total = 0.0f;
#pragma unroll
        for (int i = 0; i < kWaves; ++i) total += s_sum[i][c];
        const uint32_t times = s_cnt[c];
        if (blocks == 1) {  // nothing to join
            counts[c] = times;
            both += static_cast<double>(times) * static_cast<double>(total);
        } else {
            BlockPart::store(part + c, total, times);
        }
    }
    float zs = 0.0f;
    uint32_t ns = 0;
#pragma unroll
    for (int i = 0; i < kWaves; ++i) {
        zs += s_z[i];
        ns += s_n[i];
    }
    if (blocks == 1) return finish(s_join, out, both, {zs, ns}, g, experts, top);
    if (threadIdx.x == 0) BlockPart::store(part + experts, zs, ns);
    const uint64_t launch_tag = arrival_tag(tags(chosen, scratch));
    const uint32_t set = b / kRouteSet, sets = Group::sets(blocks), from = set * kRouteSet;
    const uint32_t many = blocks - from < kRouteSet ? blocks - from : kRouteSet;
    if (!arrive(group.slots + from, group.owners + set, b - from, many, launch_tag, &s_found)) return;
    const uint64_t* ours = group.partials + static_cast<size_t>(from) * (experts + 1);
    const auto total = [&](uint32_t c, double share, uint32_t times) {
        counts[c] = times;
        both += static_cast<double>(times) * share;
    };
    Tail tail;
    if (sets == 1) {
        tail = add_up<BlockPart>(s_join, ours, many, experts, total);
    } else {
        uint64_t* to = group.set_partials + SetPart::kWords * (static_cast<size_t>(set) * (experts + 1));
        tail = add_up<BlockPart>(s_join, ours, many, experts, [&](uint32_t c, double share, uint32_t times) {
            SetPart::store(to + SetPart::kWords * c, share, times);
        });
        if (threadIdx.x == 0) SetPart::store(to + SetPart::kWords * experts, tail.z, tail.tokens);
        if (!arrive(group.set_slots, group.last, set, sets, launch_tag, &s_found)) return;
        tail = add_up<SetPart>(s_join, group.set_partials, sets, experts, total);
    }
    finish(s_join, out, both, tail, g, experts, top);
    leave<kRouteThreads>(group.slots, blocks);
    if (sets > 1) leave<kRouteThreads>(group.set_slots, sets);
}

// A row is read once and kept. In LDS lies, per team and expert, per_balance c_j, and while a token is worked on also
// add_j of its chosen ones: dx_j = p_j (per_balance c_j + add_j + each). [16,4096,256] bf16 with 8 experts per token:
// 17.5 us, 73 MB read and written at 4.2 TB/s; without the next token's loads under way, and with the counts loaded by
// every lane for itself, 23.6. Four wavefronts per SIMD (with three, for 8 more registers, 28).
// Tags: experts in x, top (and 0x8000: renormalize) in chosen, blocks per group in totals, tokens in
// (g_weights, g_balance), row stride in (g_z, grad). g_weights, g_balance and g_z may be null.
template <typename Fmt, int G, int NV>
__global__ __launch_bounds__(kRouteThreads, 4) void k_route_grad(uint64_t x, uint64_t chosen, uint64_t totals,
                                                              uint64_t g_weights, uint64_t g_balance,
                                                              uint64_t g_z, uint64_t grad) {
    constexpr int VW = Fmt::VW, N = NV * VW, kTeams = kRouteThreads / G;
    __shared__ float s_add[kTeams][G * N + 4];  // (4: teams begin in other banks)
    const uint32_t experts = tag(x), top = tag(chosen) & 0x7fffu, blocks = tag(totals);
    const bool renormalize = (tag(chosen) & 0x8000u) != 0;
    const uint32_t tokens = tags(g_weights, g_balance), stride = tags(g_z, grad);
    const uint32_t groups = gridDim.x / blocks;
    const uint32_t g = blockIdx.x / blocks, b = blockIdx.x - g * blocks;
    const uint32_t per = (tokens + blocks - 1) / blocks;
    const uint32_t t0 = b * per < tokens ? b * per : tokens;
    const uint32_t t1 = tokens - t0 < per ? tokens : t0 + per;
    const uint32_t team = threadIdx.x / G;
    const int lane = threadIdx.x % G;
    const Totals tot(addr<uint8_t>(totals), groups, experts);
    const double n = static_cast<double>(tot.tokens[g]);
    const float* gb = addr<const float>(g_balance);
    const float* gz = addr<const float>(g_z);
    const float* gw = addr<const float>(g_weights);
    const float per_balance =
        gb != nullptr && n > 0.0 ? static_cast<float>(gb[g] * static_cast<double>(experts) / (top * n * n)) : 0.0f;
    const float per_z = gz != nullptr && n > 0.0 ? static_cast<float>(2.0 * gz[g] / n) : 0.0f;
    // per_balance times the counts of every expert, and the same per team: with what the choices of its token add
    __shared__ float s_even[G * N];
    for (uint32_t c = threadIdx.x; c < G * N; c += kRouteThreads)
        s_even[c] = c < experts ? per_balance * static_cast<float>(tot.counts[static_cast<size_t>(g) * experts + c]) : 0.0f;
    __syncthreads();
    float* mine = s_add[team];
#pragma unroll
    for (int v = 0; v < NV; ++v)
#pragma unroll
        for (int i = 0; i < VW; ++i) mine[(v * G + lane) * VW + i] = s_even[(v * G + lane) * VW + i];
    team_sync<kWave>();
    // The next token's logits and its choice `lane`, and the one after's choice, are on their way while a token
    // is worked on.
    struct Choice {
        bool on;  // else left out, or every logit is -inf
        uint64_t at;
        float gw;
    };
    const auto choice = [&](uint32_t t) {
        Choice k{false, ~uint64_t{0}, 0.0f};
        if (t >= t1) return k;
        const size_t i = (static_cast<size_t>(g) * tokens + t) * top;
        const int64_t* ch = addr<const int64_t>(chosen) + i;
        k.on = ch[0] != -1;
        if (gw != nullptr && static_cast<uint32_t>(lane) < top) {
            k.at = static_cast<uint64_t>(ch[lane]);
            k.gw = gw[i + lane];
        }
        return k;
    };
    const auto row_of = [&](uint32_t t) {
        return addr<const uint8_t>(x) + (static_cast<size_t>(g) * tokens + t) * stride * Fmt::kSize;
    };
    typename Fmt::Vec next[NV];
    float next_x = 0.0f;
    const auto load = [&](uint32_t t, const Choice& k) {
#pragma unroll
        for (int v = 0; v < NV; ++v) next[v] = masked16<Fmt>();
        if (!k.on) return;
        const uint8_t* row = row_of(t);
#pragma unroll
        for (int v = 0; v < NV; ++v) next[v] = load_cols<Fmt>(row, (v * G + lane) * VW, experts);
        if (k.at < experts) next_x = Fmt::load1(row + k.at * Fmt::kSize);
    };
    Choice next_k = choice(t0 + team);
    load(t0 + team, next_k);
    Choice after = choice(t0 + team + kTeams);
    for (uint32_t base = t0; base < t1; base += kTeams) {
        const uint32_t t = base + team;
        const size_t r = static_cast<size_t>(g) * tokens + t;
        const bool there = t < t1;
        const Choice k = next_k;
        const bool on = k.on;
        const float x_k = next_x;
        float e[N];
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            float f[VW];
            Fmt::unpack(next[v], f);
#pragma unroll
            for (int i = 0; i < VW; ++i) e[v * VW + i] = f[i];
        }
        next_k = after;
        load(t + kTeams, next_k);
        after = choice(t + 2 * kTeams);
        float m, s;
        softmax<G, N>(e, m, s);
        const float inv = 1.0f / s, lse = fmaf(log2_f(s), kLn2, m);
        float even = 0.0f;  // per_balance sum_e c_e p_te
#pragma unroll
        for (int v = 0; v < NV; ++v)
#pragma unroll
            for (int i = 0; i < VW; ++i) even = fmaf(mine[(v * G + lane) * VW + i], e[v * VW + i], even);
        even = lanes_sum<G>(even) * inv;
        // the chosen: lane j % G has choice j
        float inside = 0.0f, by = 1.0f, less = 0.0f;
        const auto others = [&](auto each) {  // choices G and on
            for (uint32_t j = G + lane; on && j < top; j += G) {
                const uint64_t at = static_cast<uint64_t>(addr<const int64_t>(chosen)[r * top + j]);
                if (at < experts) each(at, gw[r * top + j]);
            }
        };
        const bool has = on && k.at < experts;
        float was = 0.0f;
        if (gw != nullptr) {
            float kept = 0.0f;
            const auto add = [&](float logit, float grad_weight) {
                const float p = exp2_f((logit - m) * kLog2e) * inv;
                kept += p;
                inside = fmaf(grad_weight, p, inside);
            };
            if (has) add(x_k, k.gw);
            others([&](uint64_t at, float grad_weight) { add(Fmt::load1(row_of(t) + at * Fmt::kSize), grad_weight); });
            inside = lanes_sum<G>(inside);
            if (renormalize) {
                by = 1.0f / lanes_sum<G>(kept);
                less = inside * by;
                inside = 0.0f;
            }
            if (has) {
                was = mine[k.at];
                mine[k.at] = was + (k.gw - less) * by;
            }
            others([&](uint64_t at, float grad_weight) { mine[at] += (grad_weight - less) * by; });
            team_sync<kWave>();
        }
        const float each = fmaf(per_z, lse, -even) - inside;
        uint8_t* out = addr<uint8_t>(grad) + r * experts * Fmt::kSize;
#pragma unroll
        for (int v = 0; v < NV; ++v) {
            const uint32_t col = (v * G + lane) * VW;
            float f[VW];
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const int o = v * VW + i;
                const float d = e[o] * inv * (mine[col + i] + each);
                f[i] = on ? d : 0.0f;
            }
            if (!there) continue;
            if (col + VW <= experts) {
                store16_any<Fmt>(out + static_cast<size_t>(col) * Fmt::kSize, pack<Fmt>(f));
            } else {
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    if (col + i < experts) reinterpret_cast<typename Fmt::Bits*>(out)[col + i] = round_to<Fmt>(f[i]);
            }
        }
        if (gw != nullptr) {
            team_sync<kWave>();
            if (has) mine[k.at] = was;
            others([&](uint64_t at, float) { mine[at] = s_even[at]; });
            team_sync<kWave>();
        }
    }
}

// f(lanes, vectors per lane) of a plan.
template <typename Fmt, typename F>
void with_lanes(const RoutePlan& p, F f) {
    switch (p.lanes * 8 + p.vecs) {
        case 1 * 8 + 1: return f(Int<1>{}, Int<1>{});
        case 2 * 8 + 1: return f(Int<2>{}, Int<1>{});
        case 4 * 8 + 1: return f(Int<4>{}, Int<1>{});
        case 8 * 8 + 1: return f(Int<8>{}, Int<1>{});
        case 16 * 8 + 1: return f(Int<16>{}, Int<1>{});
        case 8 * 8 + 2: return f(Int<8>{}, Int<2>{});
        case 16 * 8 + 2: return f(Int<16>{}, Int<2>{});
        case 8 * 8 + 4: return f(Int<8>{}, Int<4>{});
        case 16 * 8 + 4: return f(Int<16>{}, Int<4>{});
        case 32 * 8 + 4: return f(Int<32>{}, Int<4>{});
        case 64 * 8 + 4:
            if constexpr (Fmt::VW == 4) return f(Int<64>{}, Int<4>{});
    }
}

}  // namespace

size_t route_group_bytes(int64_t experts, int blocks) {
    return 8 * Group::words(static_cast<uint32_t>(experts), static_cast<uint32_t>(blocks));
}

hipError_t launch_route(const RoutePlan& plan, const RouteArgs& a, const uint8_t* live, float* weights,
                        int64_t* chosen, uint8_t* totals, uint8_t* scratch16, hipStream_t s) {
    const uint32_t nonce = next_nonce();
    with_format(a.dtype, [&](auto fmt) {
        with_lanes<decltype(fmt)>(plan, [&](auto lanes, auto vecs) {
            const auto go = [&](auto list) {
                launch(k_route<decltype(fmt), decltype(lanes)::value, decltype(vecs)::value, decltype(list)::value>,
                       static_cast<uint32_t>(plan.grid_blocks), kRouteThreads, s, tagged(a.x, a.experts),
                       tagged(live, a.top | (a.renormalize ? 0x8000 : 0)), tagged(weights, plan.blocks),
                       tagged(chosen, nonce), tagged(scratch16, nonce >> 16), tagged(totals, 0),
                       static_cast<uint32_t>(a.row_stride), static_cast<uint32_t>(a.tokens));
            };
            if (a.top <= 2)
                go(Int<2>{});
            else if (a.top <= 8)
                go(Int<8>{});
            else if (a.top <= 16)
                go(Int<16>{});
            else
                go(Int<0>{});
        });
    });
    return hipGetLastError();
}

hipError_t launch_route_grad(const RoutePlan& plan, const RouteArgs& a, const int64_t* chosen,
                             const uint8_t* totals, const float* g_weights, const float* g_balance,
                             const float* g_z, void* grad, hipStream_t s) {
    const uint32_t tokens = static_cast<uint32_t>(a.tokens), stride = static_cast<uint32_t>(a.row_stride);
    with_format(a.dtype, [&](auto fmt) {
        with_lanes<decltype(fmt)>(plan, [&](auto lanes, auto vecs) {
            launch(k_route_grad<decltype(fmt), decltype(lanes)::value, decltype(vecs)::value>,
                   static_cast<uint32_t>(plan.grid_blocks), kRouteThreads, s, tagged(a.x, a.experts),
                   tagged(chosen, a.top | (a.renormalize ? 0x8000 : 0)), tagged(totals, plan.blocks),
                   tagged(g_weights, tokens), tagged(g_balance, tokens >> 16), tagged(g_z, stride),
                   tagged(grad, stride >> 16));
        });
    });
    return hipGetLastError();
}

}  // namespace argreduce
