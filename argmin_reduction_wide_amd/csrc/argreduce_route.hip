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
// all tokens, so that it sums p and counts choices of its own columns in registers; a workgroup leaves
// one sum per expert in scratch. No atomics on floats: results do not depend on the order in which
// workgroups run.
#include <hip/hip_runtime.h>

#include "argreduce_logits_device.hpp"
#include "argreduce_route.hpp"

#pragma clang fp contract(off)

namespace argreduce {
namespace {

constexpr float kLog2e = 1.44269504088896340736f;
constexpr int kRouteThreads = 256;
constexpr uint32_t kColBits = 10;  // of an expert's number in a key
static_assert(kExpertsMax == 1 << kColBits, "numbers of experts in a key");

// Keys of logits, larger for a larger logit and among equals for the lower expert; 0: none. 16-bit
// formats have at most 19 bits that differ between values (kLowBits), so 32 bits hold both.
template <typename Fmt>
struct Key {
    using T = uint32_t;
    __device__ static T make(float v, uint32_t col) {
        return (order_of(v + 0.0f) >> kLowBits<Fmt>) << kColBits | ((1u << kColBits) - 1 - col);
    }
    __device__ static float value(T k) {
        const uint32_t o = k >> kColBits << kLowBits<Fmt>;  // the low bits are ones in a negative value's order
        return value_of((o >> 31) ? o : o | ((1u << kLowBits<Fmt>) - 1));
    }
    __device__ static uint32_t col(T k) { return (1u << kColBits) - 1 - (k & ((1u << kColBits) - 1)); }
};
template <>
struct Key<F32> {
    using T = uint64_t;
    __device__ static T make(float v, uint32_t col) { return key_of(v, col); }
    __device__ static float value(T k) { return value_of(static_cast<uint32_t>(k >> 32)); }
    __device__ static uint32_t col(T k) { return ~static_cast<uint32_t>(k); }
};

template <int G>
__device__ inline uint32_t lanes_best(uint32_t v) {
    const auto up = [&](uint32_t o) { v = o > v ? o : v; };
    if constexpr (G >= 2) up(dpp_u32<0xB1, 0xf>(v));
    if constexpr (G >= 4) up(dpp_u32<0x4E, 0xf>(v));
    if constexpr (G >= 8) up(dpp_u32<0x141, 0xf>(v));
    if constexpr (G >= 16) up(dpp_u32<0x140, 0xf>(v));
    if constexpr (G >= 32) up(__shfl_xor(v, 16));
    if constexpr (G >= 64) up(__shfl_xor(v, 32));
    return v;
}
template <int G>
__device__ inline uint64_t lanes_best(uint64_t v) {
    const auto up = [&](uint64_t o) { v = o > v ? o : v; };
    if constexpr (G >= 2) v = dpp_max_key<0xB1, 0xf>(v);
    if constexpr (G >= 4) v = dpp_max_key<0x4E, 0xf>(v);
    if constexpr (G >= 8) v = dpp_max_key<0x141, 0xf>(v);
    if constexpr (G >= 16) v = dpp_max_key<0x140, 0xf>(v);
    if constexpr (G >= 32) up(__shfl_xor(static_cast<unsigned long long>(v), 16));
    if constexpr (G >= 64) up(__shfl_xor(static_cast<unsigned long long>(v), 32));
    return v;
}

// A lane's columns of one token: NV vectors from column `col` on; -inf past the last expert.
template <typename Fmt, int NV>
__device__ inline void load_cols(const uint8_t* row, uint32_t col, uint32_t experts, float (&e)[NV * Fmt::VW]) {
    constexpr int VW = Fmt::VW;
#pragma unroll
    for (int n = 0; n < NV; ++n) {
        const uint32_t c = col + n * VW;
        float f[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) f[i] = -__builtin_huge_valf();
        if (c + VW <= experts) {
            Fmt::unpack(load16_any<Fmt>(row + static_cast<size_t>(c) * Fmt::kSize), f);
        } else {
#pragma unroll
            for (int i = 0; i < VW; ++i)
                if (c + i < experts) f[i] = Fmt::load1(row + static_cast<size_t>(c + i) * Fmt::kSize);
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) e[n * VW + i] = f[i];
    }
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

// Partial sums of a workgroup in scratch: [experts] float, [experts] uint32, and these.
struct Tail {
    float z;
    uint32_t tokens;
};
__host__ __device__ inline size_t partial_bytes(uint32_t experts) { return 8 * static_cast<size_t>(experts) + sizeof(Tail); }

// Tags: experts in x, top in live, blocks per group in weights, whether to renormalize in chosen.
template <typename Fmt, int G, int NV>
__global__ __launch_bounds__(kRouteThreads) void k_route(uint64_t x, uint64_t live_, uint64_t weights,
                                                         uint64_t chosen, uint64_t scratch, uint32_t stride,
                                                         uint32_t tokens) {
    constexpr int N = NV * Fmt::VW, kTeams = kRouteThreads / G;
    using K = Key<Fmt>;
    __shared__ float s_sum[kTeams * G * N];
    __shared__ uint32_t s_cnt[kTeams * G * N];
    __shared__ float s_z[kRouteThreads / kWave];
    __shared__ uint32_t s_n[kRouteThreads / kWave];
    const uint32_t experts = tag(x), top = tag(live_), blocks = tag(weights);
    const bool renormalize = tag(chosen) != 0;
    const uint32_t g = blockIdx.x / blocks, b = blockIdx.x - g * blocks;
    const uint32_t per = (tokens + blocks - 1) / blocks;
    const uint32_t t0 = b * per < tokens ? b * per : tokens;
    const uint32_t t1 = tokens - t0 < per ? tokens : t0 + per;
    const uint32_t team = threadIdx.x / G;
    const int lane = threadIdx.x % G;
    const uint32_t col = lane * N;
    const uint8_t* live = addr<const uint8_t>(live_);
    float sum[N], z = 0.0f;
    uint32_t cnt[N], n = 0;
#pragma unroll
    for (int i = 0; i < N; ++i) {
        sum[i] = 0.0f;
        cnt[i] = 0;
    }
    for (uint32_t base = t0; base < t1; base += kTeams) {
        const uint32_t t = base + team;
        const size_t r = static_cast<size_t>(g) * tokens + t;
        const bool there = t < t1;
        const bool on = there && (live == nullptr || live[r] != 0);
        float e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = -__builtin_huge_valf();
        if (on) load_cols<Fmt, NV>(addr<const uint8_t>(x) + r * stride * Fmt::kSize, col, experts, e);
        typename K::T key[N];
#pragma unroll
        for (int i = 0; i < N; ++i) key[i] = e[i] >= kLowest ? K::make(e[i], col + i) : 0;
        float m, s;
        softmax<G, N>(e, m, s);
        const bool counts = on && s != 0.0f;  // a token whose every logit is -inf is left out
        const bool ok = s > 0.0f && s < __builtin_huge_valf();
        const float inv = 1.0f / s;
        if (counts) {
            const float lse = fmaf(log2_f(s), kLn2, m);
            if (lane == 0) {
                z = fmaf(lse, lse, z);
                ++n;
            }
#pragma unroll
            for (int i = 0; i < N; ++i) sum[i] = fmaf(e[i], inv, sum[i]);
        }
        // the best key left, `top` times: lane j % G keeps the j-th
        float kept_sum = 0.0f;
        float* wt = addr<float>(weights) + r * top;
        int64_t* ch = addr<int64_t>(chosen) + r * top;
        for (uint32_t j0 = 0; j0 < top; j0 += G) {
            typename K::T mine = 0;
            const uint32_t j1 = top - j0 < G ? top - j0 : G;
            for (uint32_t j = 0; j < j1; ++j) {
                typename K::T best = 0;
#pragma unroll
                for (int i = 0; i < N; ++i) best = key[i] > best ? key[i] : best;
                best = lanes_best<G>(best);
                if (static_cast<uint32_t>(lane) == j) mine = best;
                if (!ok) best = 0;
                const typename K::T gone = best == 0 ? ~typename K::T{0} : best;
#pragma unroll
                for (int i = 0; i < N; ++i) {
                    const bool taken = key[i] == gone;
                    key[i] = taken ? 0 : key[i];
                    cnt[i] += taken ? 1u : 0u;
                }
            }
            const bool some = ok && mine != 0;
            const float w = some ? exp2_f((K::value(mine) - m) * kLog2e) : 0.0f;
            kept_sum += lanes_sum<G>(w);
            if (there && static_cast<uint32_t>(lane) < j1) {
                const bool bad = on && !(s < __builtin_huge_valf());  // NaN or +inf
                ch[j0 + lane] = some ? static_cast<int64_t>(K::col(mine)) : bad ? -2 : -1;
                wt[j0 + lane] = bad ? __builtin_nanf("") : renormalize ? w : w * inv;
                if (!bad && !some) wt[j0 + lane] = 0.0f;
            }
        }
        if (renormalize && there && ok) {
            for (uint32_t j = lane; j < top; j += G) wt[j] = wt[j] / kept_sum;
        }
    }
    // the workgroup's sums
    z = lanes_sum<kWave>(z);
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) n += __shfl_xor(n, o);
    if (threadIdx.x % kWave == 0) {
        s_z[threadIdx.x / kWave] = z;
        s_n[threadIdx.x / kWave] = n;
    }
#pragma unroll
    for (int i = 0; i < N; ++i) {
        s_sum[team * G * N + col + i] = sum[i];
        s_cnt[team * G * N + col + i] = cnt[i];
    }
    __syncthreads();
    uint8_t* out = addr<uint8_t>(scratch) + blockIdx.x * partial_bytes(experts);
    for (uint32_t c = threadIdx.x; c < experts; c += kRouteThreads) {
        float total = 0.0f;
        uint32_t times = 0;
        for (int i = 0; i < kTeams; ++i) {
            total += s_sum[i * G * N + c];
            times += s_cnt[i * G * N + c];
        }
        reinterpret_cast<float*>(out)[c] = total;
        reinterpret_cast<uint32_t*>(out)[experts + c] = times;
    }
    if (threadIdx.x == 0) {
        float zs = 0.0f;
        uint32_t ns = 0;
        for (int i = 0; i < kRouteThreads / kWave; ++i) {
            zs += s_z[i];
            ns += s_n[i];
        }
        *reinterpret_cast<Tail*>(out + 8 * static_cast<size_t>(experts)) = Tail{zs, ns};
    }
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

__device__ inline double lanes_sum64(double v) {
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) v += __shfl_xor(v, o);
    return v;
}

// One workgroup per group adds its partial sums up, in binary64. Tags: experts in scratch, top in totals.
__global__ __launch_bounds__(kRouteThreads) void k_route_join(uint64_t scratch, uint64_t totals, uint32_t blocks,
                                                              uint32_t groups) {
    __shared__ double s_red[3][kRouteThreads / kWave];
    const uint32_t experts = tag(scratch), top = tag(totals), g = blockIdx.x;
    const Totals out(addr<uint8_t>(totals), groups, experts);
    const size_t step = partial_bytes(experts);
    const uint8_t* part = addr<const uint8_t>(scratch) + static_cast<size_t>(g) * blocks * step;
    double both = 0.0, z = 0.0, n = 0.0;
    for (uint32_t c = threadIdx.x; c < experts; c += kRouteThreads) {
        double share = 0.0;
        int64_t times = 0;
        for (uint32_t b = 0; b < blocks; ++b) {
            share += static_cast<double>(reinterpret_cast<const float*>(part + b * step)[c]);
            times += reinterpret_cast<const uint32_t*>(part + b * step)[experts + c];
        }
        out.counts[static_cast<size_t>(g) * experts + c] = times;
        both += static_cast<double>(times) * share;
    }
    for (uint32_t b = threadIdx.x; b < blocks; b += kRouteThreads) {
        const Tail t = *reinterpret_cast<const Tail*>(part + b * step + 8 * static_cast<size_t>(experts));
        z += static_cast<double>(t.z);
        n += static_cast<double>(t.tokens);
    }
    both = lanes_sum64(both);
    z = lanes_sum64(z);
    n = lanes_sum64(n);
    if (threadIdx.x % kWave == 0) {
        s_red[0][threadIdx.x / kWave] = both;
        s_red[1][threadIdx.x / kWave] = z;
        s_red[2][threadIdx.x / kWave] = n;
    }
    __syncthreads();
    if (threadIdx.x == 0) {
        both = z = n = 0.0;
        for (int i = 0; i < kRouteThreads / kWave; ++i) {
            both += s_red[0][i];
            z += s_red[1][i];
            n += s_red[2][i];
        }
        out.tokens[g] = static_cast<int64_t>(n);
        out.balance[g] = n > 0.0 ? static_cast<float>(both * experts / (top * n * n)) : 0.0f;
        out.z[g] = n > 0.0 ? static_cast<float>(z / n) : 0.0f;
    }
}

// Marks an expert that the token has not chosen, among the gradients of weights (a NaN that no
// arithmetic gives; a gradient of these very bits is read as the ordinary NaN).
constexpr uint32_t kNotChosen = 0xffffffffu;

// Tags: experts in x, top (and 0x8000: renormalize) in chosen, blocks per group in totals, tokens in
// (g_weights, g_balance), row stride in (g_z, grad). g_weights, g_balance and g_z may be null.
template <typename Fmt, int G, int NV>
__global__ __launch_bounds__(kRouteThreads) void k_route_grad(uint64_t x, uint64_t chosen, uint64_t totals,
                                                              uint64_t g_weights, uint64_t g_balance,
                                                              uint64_t g_z, uint64_t grad) {
    constexpr int VW = Fmt::VW, N = NV * VW, kTeams = kRouteThreads / G;
    __shared__ uint32_t s_gw[kTeams * G * N];
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
    const uint32_t col = lane * N;
    const Totals tot(addr<uint8_t>(totals), groups, experts);
    const double n = static_cast<double>(tot.tokens[g]);
    const float* gb = addr<const float>(g_balance);
    const float* gz = addr<const float>(g_z);
    const float* gw = addr<const float>(g_weights);
    const float per_balance =
        gb != nullptr && n > 0.0 ? static_cast<float>(gb[g] * static_cast<double>(experts) / (top * n * n)) : 0.0f;
    const float per_z = gz != nullptr && n > 0.0 ? static_cast<float>(2.0 * gz[g] / n) : 0.0f;
    float c[N];
#pragma unroll
    for (int i = 0; i < N; ++i) {
        c[i] = col + i < experts ? static_cast<float>(tot.counts[static_cast<size_t>(g) * experts + col + i]) : 0.0f;
        s_gw[team * G * N + col + i] = kNotChosen;
    }
    uint32_t* mine = s_gw + team * G * N;
    for (uint32_t base = t0; base < t1; base += kTeams) {
        const uint32_t t = base + team;
        const size_t r = static_cast<size_t>(g) * tokens + t;
        const bool there = t < t1;
        const int64_t* ch = addr<const int64_t>(chosen) + r * top;
        const bool on = there && ch[0] != -1;  // left out, or every logit -inf
        float e[N];
#pragma unroll
        for (int i = 0; i < N; ++i) e[i] = -__builtin_huge_valf();
        if (on) load_cols<Fmt, NV>(addr<const uint8_t>(x) + r * stride * Fmt::kSize, col, experts, e);
        if (on && gw != nullptr) {
            for (uint32_t j = lane; j < top; j += G) {
                const uint64_t at = static_cast<uint64_t>(ch[j]);
                const uint32_t v = __float_as_uint(gw[r * top + j]);
                if (at < experts) mine[at] = v == kNotChosen ? 0x7fc00000u : v;
            }
        }
        float m, s;
        softmax<G, N>(e, m, s);
        const float inv = 1.0f / s, lse = fmaf(log2_f(s), kLn2, m);
        team_sync<kWave>();
        float even = 0.0f, inside = 0.0f, kept = 0.0f, w[N];
        bool of[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            e[i] *= inv;
            even = fmaf(c[i], e[i], even);
            const uint32_t v = mine[col + i];
            of[i] = v != kNotChosen;
            w[i] = of[i] ? __uint_as_float(v) : 0.0f;
            if (of[i]) {
                inside = fmaf(w[i], e[i], inside);
                kept += e[i];
            }
        }
        even = lanes_sum<G>(even);
        inside = lanes_sum<G>(inside);
        kept = lanes_sum<G>(kept);
        team_sync<kWave>();
        if (on && gw != nullptr) {
            for (uint32_t j = lane; j < top; j += G) {
                const uint64_t at = static_cast<uint64_t>(ch[j]);
                if (at < experts) mine[at] = kNotChosen;
            }
        }
        const float each = fmaf(per_z, lse, -per_balance * even) - (renormalize ? 0.0f : inside);
        const float by = renormalize ? 1.0f / kept : 1.0f, less = renormalize ? inside * by : 0.0f;
        float d[N];
#pragma unroll
        for (int i = 0; i < N; ++i) {
            d[i] = e[i] * fmaf(per_balance, c[i], each);
            if (of[i]) d[i] = fmaf(e[i] * by, w[i] - less, d[i]);
            if (!on) d[i] = 0.0f;
        }
        if (there) {
            uint8_t* out = addr<uint8_t>(grad) + r * experts * Fmt::kSize;
#pragma unroll
            for (int v = 0; v < NV; ++v) {
                const uint32_t at = col + v * VW;
                float f[VW];
#pragma unroll
                for (int i = 0; i < VW; ++i) f[i] = d[v * VW + i];
                if (at + VW <= experts) {
                    store16_any<Fmt>(out + static_cast<size_t>(at) * Fmt::kSize, pack<Fmt>(f));
                } else {
#pragma unroll
                    for (int i = 0; i < VW; ++i)
                        if (at + i < experts)
                            reinterpret_cast<typename Fmt::Bits*>(out)[at + i] = round_to<Fmt>(f[i]);
                }
            }
        }
    }
}

// f(lanes, vectors per lane) of a plan: 16-bit formats have at most two vectors per lane.
template <typename Fmt, typename F>
void with_lanes(const RoutePlan& p, F f) {
    if constexpr (Fmt::VW == 4)
        if (p.vecs == 4) return f(Int<64>{}, Int<4>{});
    if (p.vecs == 2) return f(Int<64>{}, Int<2>{});
    switch (p.lanes) {
        case 1: return f(Int<1>{}, Int<1>{});
        case 2: return f(Int<2>{}, Int<1>{});
        case 4: return f(Int<4>{}, Int<1>{});
        case 8: return f(Int<8>{}, Int<1>{});
        case 16: return f(Int<16>{}, Int<1>{});
        case 32: return f(Int<32>{}, Int<1>{});
        default: return f(Int<64>{}, Int<1>{});
    }
}

}  // namespace

size_t route_partial_bytes(int64_t experts) { return partial_bytes(static_cast<uint32_t>(experts)); }

hipError_t launch_route(const RoutePlan& plan, const RouteArgs& a, const uint8_t* live, float* weights,
                        int64_t* chosen, uint8_t* totals, uint8_t* scratch16, hipStream_t s) {
    const uint32_t groups = static_cast<uint32_t>(a.groups);
    with_format(a.dtype, [&](auto fmt) {
        with_lanes<decltype(fmt)>(plan, [&](auto lanes, auto vecs) {
            launch(k_route<decltype(fmt), decltype(lanes)::value, decltype(vecs)::value>,
                   static_cast<uint32_t>(plan.grid_blocks), kRouteThreads, s, tagged(a.x, a.experts),
                   tagged(live, a.top), tagged(weights, plan.blocks), tagged(chosen, a.renormalize),
                   tagged(scratch16, 0), static_cast<uint32_t>(a.row_stride), static_cast<uint32_t>(a.tokens));
        });
    });
    launch(k_route_join, groups, kRouteThreads, s, tagged(scratch16, a.experts), tagged(totals, a.top),
           static_cast<uint32_t>(plan.blocks), groups);
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
