// Logits operators for gfx950: log probabilities of given tokens with entropy and top
// alternatives, and distillation from a teacher's top logits, each with its gradient.
//
// Mathematics. For a row x of logits, m = max x, k = log2(e) / T:
//   z_j = (x_j - m) k        (base-2 exponents, <= 0)
//   s   = sum 2^z_j,  h = sum 2^z_j z_j,  p_j = 2^(z_j - log2 s)
//   logprob of t  = ln 2 (z_t - log2 s)
//   entropy       = ln 2 (log2 s - h / s)
// (m, s, h) of two parts of a row merge exactly as in an online softmax: moving a part from
// its own maximum m' to m = m' + d / k turns s into 2^-d s and h into 2^-d (h - d s). Every
// statistic is held in binary32; the one rounding to the logits' type is a gradient's store.
//
// What bounds the forward kernels is the read of the logits: per element one subtraction, one
// multiplication, one exponential and one addition (two more operations with the entropy),
// which the vector units do about as fast as HBM delivers 16-bit elements.
//
// Masked logits are -inf: 2^-inf = 0 and the h term is cut off at z = -16384, where 2^z is 0
// already, so that 0 * inf does not arise. A running maximum starts at the lowest finite
// number, never at -inf, so that x - m is never inf - inf; a row whose every element is -inf
// ends with s = 0. NaN and +inf make s NaN.
#include <hip/hip_runtime.h>

#include "argreduce_launch.hpp"
#include "argreduce_logits.hpp"
#include "argreduce_logits_device.hpp"

// Products and sums are fused where the source says so and nowhere else, so that two kernels
// that compute the same quantity from the same inputs get the same bits.
#pragma clang fp contract(off)

namespace argreduce {
namespace {

// Writes a row's alternatives from L.buf, or k empty ones.
template <int T, int S>
__device__ inline void top_store(const TopLds<T, S>& L, uint32_t k, int lane, const Stat& a,
                                 float scale, float l2, float* lp, int64_t* tok) {
    if (static_cast<uint32_t>(lane) < k) {
        if (static_cast<uint32_t>(lane) < L.count) {
            float v;
            uint32_t i;
            Key32<kMax>::split(L.buf[lane], v, i);
            lp[lane] = ln_p(v, a.m, l2, scale);
            tok[lane] = i;
        } else {
            lp[lane] = -__builtin_huge_valf();
            tok[lane] = -1;
        }
    }
}
__device__ inline void top_none(uint32_t k, int lane, int step, float v, float* lp, int64_t* tok) {
    for (uint32_t i = lane; i < k; i += step) {
        lp[i] = v;
        tok[i] = -1;
    }
}

// ---------------------------------------------------------------------------------------
// Log probabilities: outputs of one row.

struct RowOut {
    float logprob, entropy, m, l2;
};
// A row's alternatives, and whether the entropy goes to a row of its own too, in 16 bits.
constexpr uint32_t kApart = 0x8000u;
__device__ inline uint32_t alternatives(uint32_t outputs) { return outputs & ~kApart; }
// stats is [4, rows]: log probability, entropy, maximum, log2 of the sum; [5, rows]: the entropy again.
template <bool ENT>
__device__ inline void store_stats(float* stats, uint32_t rows, uint32_t r, const RowOut& o,
                                   uint32_t outputs) {
    stats[r] = o.logprob;
    stats[static_cast<size_t>(rows) + r] = o.entropy;
    stats[2 * static_cast<size_t>(rows) + r] = o.m;
    stats[3 * static_cast<size_t>(rows) + r] = o.l2;
    if (ENT && (outputs & kApart)) stats[4 * static_cast<size_t>(rows) + r] = o.entropy;
}
template <bool ENT>
__device__ inline RowOut row_out(const Stat& a, float xt, float scale) {
    RowOut o;
    o.m = a.m;
    o.l2 = log2_f(a.s);
    o.logprob = ln_p(xt, a.m, o.l2, scale);
    o.entropy = ENT ? (o.l2 - a.h / a.s) * kLn2 : __builtin_nanf("");
    if (a.s == 0.0f) {  // every logit is -inf, and xt too unless its token is none of the row's
        o.logprob = xt != xt ? xt : -__builtin_huge_valf();
        if (ENT) o.entropy = 0.0f;
    }
    return o;
}
template <bool ENT>
__device__ inline RowOut row_left_out() {
    return {0.0f, ENT ? 0.0f : __builtin_nanf(""), 0.0f, 0.0f};
}

// Rows of at most G vectors, G lanes each, the row held in registers: maximum first, then the
// exponentials. Alternatives are taken one by one, as the largest key left. [65536,64] f16 with
// entropy and 2 alternatives: 8.3 us (8 lanes; 12 MB, 1.4 TB/s), bound by the latency of one load and
// the chain of reductions after it: a wavefront has eight rows and no work beside them. With 30
// alternatives and no entropy 38 us, bound by their rounds.
template <typename Fmt, bool KEEP, bool ENT, int G>
__global__ __launch_bounds__(kBlockThreads) void k_lp_group(const void* x, uint32_t cols,
                                                            uint32_t stride, float scale,
                                                            uint32_t rows, const int64_t* tokens,
                                                            float* stats, uint64_t top_lp,
                                                            int64_t* top_tok) {
    constexpr int VW = Fmt::VW;
    const uint32_t outputs = tag(top_lp), k = alternatives(outputs);
    const uint32_t want = blockIdx.x * (kBlockThreads / G) + threadIdx.x / G;
    const uint32_t r = want < rows ? want : rows - 1;  // lanes past the end repeat the last row
    const int lane = threadIdx.x % G;
    const uint8_t* row = row_ptr<Fmt>(x, r, stride);
    const int64_t t = tokens[r];
    const bool live = t >= 0;
    const Span<Fmt, KEEP> sp(row, cols);
    float e[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) e[i] = -__builtin_huge_valf();
    if (live && static_cast<uint32_t>(lane) < sp.vs) {
        Fmt::unpack(sp.load(lane), e);
        const uint32_t p0 = sp.pos(lane);
#pragma unroll
        for (int i = 0; i < VW; ++i) e[i] = p0 + i < cols ? e[i] : -__builtin_huge_valf();
    }
    const float xt = live ? load_at<Fmt>(row, t, cols) : 0.0f;
    Stat a;
    a.init();
    float m = a.m;
#pragma unroll
    for (int i = 0; i < VW; i += 2) m = max3_f(m, e[i], e[i + 1]);
    a.m = lanes_max<G>(m);
    take<ENT>(e, scale, a);
    a.s = lanes_sum<G>(a.s);
    if constexpr (ENT) a.h = lanes_sum<G>(a.h);
    const RowOut o = live ? row_out<ENT>(a, xt, scale) : row_left_out<ENT>();
    if (lane == 0 && want < rows) store_stats<ENT>(stats, rows, r, o, outputs);
    if (k == 0) return;
    float* lp = addr<float>(top_lp) + static_cast<size_t>(r) * k;
    int64_t* tok = top_tok + static_cast<size_t>(r) * k;
    uint64_t key[VW];
    const uint32_t p0 = sp.pos(lane);
    const bool ok = a.s == a.s;  // a row with NaN or +inf has no alternatives
#pragma unroll
    for (int i = 0; i < VW; ++i) key[i] = (ok && e[i] >= kLowest) ? key_of(e[i], p0 + i) : 0;
    for (uint32_t j = 0; j < k; ++j) {
        uint64_t b = 0;
#pragma unroll
        for (int i = 0; i < VW; ++i) b = key[i] > b ? key[i] : b;
        if constexpr (G >= 2) b = dpp_max_key<0xB1, 0xf>(b);
        if constexpr (G >= 4) b = dpp_max_key<0x4E, 0xf>(b);
        if constexpr (G >= 8) b = dpp_max_key<0x141, 0xf>(b);
        if constexpr (G >= 16) b = dpp_max_key<0x140, 0xf>(b);
        if constexpr (G >= 32) {
            const uint64_t other = __shfl_xor(static_cast<unsigned long long>(b), 16);
            b = other > b ? other : b;
        }
#pragma unroll
        for (int i = 0; i < VW; ++i) key[i] = key[i] == b ? 0 : key[i];
        if (lane == 0 && want < rows) {
            float v;
            uint32_t i;
            Key32<kMax>::split(b, v, i);
            lp[j] = b != 0 ? ln_p(v, a.m, o.l2, scale)
                           : (ok ? -__builtin_huge_valf() : __builtin_nanf(""));
            tok[j] = b != 0 ? static_cast<int64_t>(i) : -1;
        }
    }
}

// A team of T lanes per row, in one pass. [4001,32001] f16 with a tenth of the rows left out: 37.6 us,
// 6.1 TB/s, bound by the read; [2048,128256] bf16 with entropy 95 us, 5.5 TB/s, with 64 alternatives and
// no entropy 96 us, 5.5 TB/s: the read, and the alternatives' selection (about 10 us a row) as far as
// the CU's other rows do not hide it. [49539,2032] bf16 by wavefronts 36 us, 5.6 TB/s. [1,32000] f32
// with entropy and 5 alternatives: 8.1 us, the latency of the read and of the selection's barriers
// (split over 8 workgroups: 10, and a second launch).
template <typename Fmt, bool KEEP, bool ENT, bool TOP, int T>
__global__ __launch_bounds__(kTeamBlock<T>) void k_lp_team(const void* x, uint32_t cols,
                                                           uint32_t stride, float scale,
                                                           uint32_t rows, const int64_t* tokens,
                                                           float* stats, uint64_t top_lp,
                                                           int64_t* top_tok) {
    constexpr int kTeams = kTeamsPerBlock<T>;
    constexpr int U = kUnroll<Fmt, TOP>;
    __shared__ float sh[T / kWave][kShared];
    __shared__ TopLds<TOP ? T : 64, TOP ? kSegs<T> : 1> lds[TOP ? kTeams : 1];
    const uint32_t team = team_of<T>();
    const uint32_t r = blockIdx.x * kTeams + team;
    const int lane = lane_of<T>();
    if (r >= rows) return;  // whole teams, and never one of several wavefronts
    const int64_t t = tokens[r];
    const uint32_t outputs = tag(top_lp), k = alternatives(outputs);
    float* lp = addr<float>(top_lp) + static_cast<size_t>(r) * k;
    int64_t* tok = top_tok + static_cast<size_t>(r) * k;
    if (t < 0) {
        if (lane == 0) store_stats<ENT>(stats, rows, r, row_left_out<ENT>(), outputs);
        if constexpr (TOP) top_none(k, lane, T, -__builtin_huge_valf(), lp, tok);
        return;
    }
    const uint8_t* row = row_ptr<Fmt>(x, r, stride);
    const float xt = load_at<Fmt>(row, t, cols);
    const Span<Fmt, KEEP> sp(row, cols);
    Stat a;
    auto& L = lds[TOP ? team : 0];
    const Segments g = Segments::cut<T, U>(sp.va, sp.vb, kSegs<T>);
    scan_span<Fmt, ENT, T, U, TOP>(sp, true, sp.va, sp.vb, lane, scale, a, g, L.seg);
    team_merge<ENT, T>(a, scale, lane, sh);
    const RowOut o = row_out<ENT>(a, xt, scale);
    if (lane == 0) store_stats<ENT>(stats, rows, r, o, outputs);
    if constexpr (TOP) {
        if (!(a.s > 0.0f)) {
            top_none(k, lane, T, a.s == 0.0f ? -__builtin_huge_valf() : __builtin_nanf(""), lp, tok);
            return;
        }
        top_select<Fmt, T, kSegs<T>>(L, sp, g.count(), g.lg_vecs, k, lane,
                                     [&](uint32_t s, uint32_t i) { return g.vec(s, i); });
        top_store(L, k, lane, a, scale, o.l2, lp, tok);
    }
}

struct Part {  // what a slice leaves in scratch
    float m, s, h, pad;
    float oct_max[kPartThreads / 8];  // of every eight lanes
};

// A slice per workgroup. [32,202048] bf16 with entropy: 6.4 us (12.9 MB, 2 TB/s), [1,202048] f32 3.3 us:
// a launch and the latency of four loads per lane.
template <typename Fmt, bool KEEP, bool ENT>
__global__ __launch_bounds__(kPartThreads) void k_part(const void* x, uint32_t cols, uint32_t stride,
                                                       float scale, uint32_t parts,
                                                       const int64_t* tokens, Part* out) {
    __shared__ float sh[kPartThreads / kWave][kShared];
    const uint32_t r = blockIdx.x / parts;
    const uint32_t b = blockIdx.x - r * parts;
    if (tokens != nullptr && tokens[r] < 0) return;
    const Span<Fmt, KEEP> sp(row_ptr<Fmt>(x, r, stride), cols);
    const uint32_t n = part_vecs(span_max<Fmt>(cols), parts);
    uint32_t first = sp.va + b * n;
    first = first < sp.vb ? first : sp.vb;
    const uint32_t last = sp.vb - first < n ? sp.vb : first + n;
    const int lane = threadIdx.x;
    Stat a;
    scan_span<Fmt, ENT, kPartThreads, kPartUnroll>(sp, b == 0, first, last, lane, scale, a);
    const float oct_max = lanes_max<8>(a.m);  // with the edges': a bound is all that is needed
    team_merge<ENT, kPartThreads>(a, scale, lane, sh);
    if (lane % 8 == 0) out[blockIdx.x].oct_max[lane / 8] = oct_max;
    if (lane == 0) {
        out[blockIdx.x].m = a.m;
        out[blockIdx.x].s = a.s;
        out[blockIdx.x].h = a.h;
    }
}

constexpr int kMergeThreads = 256;
constexpr int kMergeTopThreads = 1024;  // with alternatives: vectors to read again in one step
constexpr int kMergeSegs = 2048;

// The merged statistics of a split row, in every thread.
template <bool ENT, int T>
__device__ inline Stat merge_parts(const Part* p, uint32_t parts, float scale, int lane,
                                   float (*sh)[kShared]) {
    Stat a;
    a.init();
    for (uint32_t b = lane; b < parts; b += T) {
        Stat o{p[b].m, p[b].s, ENT ? p[b].h : 0.0f};
        const float m = max_f(a.m, o.m);
        a.move<ENT>(m, scale);
        o.move<ENT>(m, scale);
        a.s += o.s;
        a.h += o.h;
    }
    team_merge<ENT, T>(a, scale, lane, sh);
    return a;
}

// One workgroup per split row; with 20 alternatives 6.8 us ([1,202048] f32), with 8 7.5 us
// ([32,202048] bf16): chained latencies, of the slices' statistics, the bisection, and the segments'
// second read, all of them after k_part has ended. (One launch for both, through words tagged with a
// nonce as k_split joins its slices by, has not been built.) Tags: columns in (x, tokens), slices,
// outputs, scale.
template <typename Fmt, bool ENT, bool TOP, int T = TOP ? kMergeTopThreads : kMergeThreads>
__global__ __launch_bounds__(T) void k_lp_merge(uint64_t x, uint64_t tokens,
                                                            uint64_t part, uint64_t stats_,
                                                            uint64_t top_lp, uint64_t top_tok,
                                                            uint32_t stride, uint32_t rows) {
    __shared__ float sh[T / kWave][kShared];
    __shared__ TopLds<TOP ? T : 64, TOP ? kMergeSegs : 1> L;
    const uint32_t cols = tags(x, tokens);
    const uint32_t parts = tag(part), outputs = tag(stats_), k = alternatives(outputs);
    const float scale = __uint_as_float(tags(top_lp, top_tok));
    float* stats = addr<float>(stats_);
    const uint32_t r = blockIdx.x;
    const int lane = threadIdx.x;
    const int64_t t = addr<const int64_t>(tokens)[r];
    float* lp = addr<float>(top_lp) + static_cast<size_t>(r) * k;
    int64_t* tok = addr<int64_t>(top_tok) + static_cast<size_t>(r) * k;
    if (t < 0) {
        if (lane == 0) store_stats<ENT>(stats, rows, r, row_left_out<ENT>(), outputs);
        if constexpr (TOP) top_none(k, lane, T, -__builtin_huge_valf(), lp, tok);
        return;
    }
    const uint8_t* row = row_ptr<Fmt>(addr<const void>(x), r, stride);
    const float xt = load_at<Fmt>(row, t, cols);
    const Part* p = addr<const Part>(part) + static_cast<size_t>(r) * parts;
    const Stat a = merge_parts<ENT, T>(p, parts, scale, lane, sh);
    const RowOut o = row_out<ENT>(a, xt, scale);
    if (lane == 0) store_stats<ENT>(stats, rows, r, o, outputs);
    if constexpr (TOP) {
        if (!(a.s > 0.0f)) {
            top_none(k, lane, T, a.s == 0.0f ? -__builtin_huge_valf() : __builtin_nanf(""), lp, tok);
            return;
        }
        // a slice's 32 maxima as they are, or two, four, ... together so that kMergeSegs hold them
        constexpr uint32_t kOct = kPartThreads / 8;
        const uint32_t lg = ceil_log2((parts * kOct + kMergeSegs - 1) / kMergeSegs);
        const uint32_t per = kOct >> lg, segs = parts * per, lanes = 8u << lg;
        for (uint32_t s = lane; s < segs; s += T) {
            const float* o = p[s / per].oct_max + (s % per << lg);
            float m = o[0];
            for (uint32_t i = 1; i < 1u << lg; ++i) m = max_f(m, o[i]);
            L.seg[s] = m;
        }
        const Span<Fmt> sp(row, cols);
        const uint32_t n = part_vecs(span_max<Fmt>(cols), parts);
        const uint32_t steps = (n + kPartThreads - 1) / kPartThreads;
        top_select<Fmt, T, kMergeSegs>(
            L, sp, segs, ceil_log2(steps * lanes), k, lane, [&](uint32_t s, uint32_t i) {
                const uint32_t in = i / lanes * kPartThreads + s % per * lanes + i % lanes;
                const uint32_t v = sp.va + s / per * n + in;
                return in < n && v < sp.vb ? v : kNoVec;
            });
        top_store(L, k, lane, a, scale, o.l2, lp, tok);
    }
}

// ---------------------------------------------------------------------------------------
// Gradients. A slice of a row is written as the aligned vectors of the gradient's row; the
// logits are read at the same positions, aligned or not (the hardware reads a vector at any
// element's address). f(element, position) gives the gradient of one element.

template <typename Fmt>
struct GradSlice {
    const uint8_t* x;  // the row's logits
    uint8_t* g;        // the row's gradient
    Span<Fmt> sp;      // of the gradient's row
    uint32_t first, last;
    __device__ GradSlice(const uint8_t* xr, uint8_t* gr, uint32_t cols, uint32_t slice, uint32_t slices)
        : x(xr), g(gr), sp(gr, cols) {
        const uint32_t n = part_vecs(span_max<Fmt>(cols), slices);
        first = slice * n < sp.vs ? slice * n : sp.vs;
        last = sp.vs - first < n ? sp.vs : first + n;
    }
    __device__ bool holds(int64_t i) const {
        const int64_t v = (i + sp.off) / Fmt::VW;
        return v >= first && v < last;
    }
    // take(values, position of the first, out): the gradients of VW elements.
    template <typename Take>
    __device__ void write(int lane, int team, bool zero, Take take) const {
        constexpr int VW = Fmt::VW;
        for (uint32_t v = first + lane; v < last; v += team) {
            const uint32_t p0 = sp.pos(v);
            float e[VW], d[VW];
            if (v >= sp.va && v < sp.vb) {
#pragma unroll
                for (int i = 0; i < VW; ++i) d[i] = 0.0f;
                if (!zero) {
                    Fmt::unpack(load16_any<Fmt>(x + static_cast<size_t>(p0) * Fmt::kSize), e);
                    take(e, p0, d);
                }
                *reinterpret_cast<typename Fmt::Vec*>(g + static_cast<size_t>(p0) * Fmt::kSize) =
                    pack<Fmt>(d);
            } else {
#pragma unroll
                for (int i = 0; i < VW; ++i) {
                    d[i] = 0.0f;
                    e[i] = (!zero && p0 + i < sp.cols)
                               ? Fmt::load1(x + static_cast<size_t>(p0 + i) * Fmt::kSize)
                               : 0.0f;
                }
                if (!zero) take(e, p0, d);
#pragma unroll
                for (int i = 0; i < VW; ++i)
                    if (p0 + i < sp.cols)
                        reinterpret_cast<typename Fmt::Bits*>(g)[p0 + i] = round_to<Fmt>(d[i]);
            }
        }
    }
};

// d logprob and d entropy: dx_j = [ g (delta_jt - p_j) - e p_j (ln p_j + H) ] / T.
// One exponential per element: bound by the read and the store. [2048,128256] bf16 with the entropy's
// gradient 195 us, 5.4 TB/s read and written; [257,32003] f32 with a quarter of the rows left out 10.6
// us, 5.4 TB/s, the logits from the Infinity Cache. Slices of 1024 vectors (make_grad_plan has other
// lengths' figures), so that few rows occupy every CU and a workgroup's loads are all under way at
// once. Tags: columns in (x, tokens), scale in (stats, g_lp), slices in g_ent,
// log2 of the team's lanes in grad.
template <typename Fmt, bool ENT, bool WIDE>
__global__ __launch_bounds__(kBlockThreads) void k_lp_grad(uint64_t x, uint64_t tokens,
                                                           uint64_t stats_, uint64_t g_lp,
                                                           uint64_t g_ent, uint64_t grad,
                                                           uint32_t stride, uint32_t rows) {
    constexpr int VW = Fmt::VW;
    const uint32_t cols = tags(x, tokens), slices = tag(g_ent);
    const uint32_t lg = WIDE ? 8 : tag(grad);  // WIDE: a slice per workgroup, wave-uniform addresses
    const float scale = __uint_as_float(tags(stats_, g_lp));
    const uint32_t unit = WIDE ? blockIdx.x : (blockIdx.x << (8 - lg)) + (threadIdx.x >> lg);
    const uint32_t r = WIDE ? unit / slices : unit;
    if (r >= rows) return;
    const int lane = threadIdx.x & ((1u << lg) - 1);
    const float* stats = addr<const float>(stats_);
    const int64_t t = addr<const int64_t>(tokens)[r];
    const float h = ENT ? stats[static_cast<size_t>(rows) + r] : 0.0f;
    const float m = stats[2 * static_cast<size_t>(rows) + r];
    const float l2 = stats[3 * static_cast<size_t>(rows) + r];
    const float inv_t = scale * kLn2;
    float a = addr<const float>(g_lp)[r] * inv_t;
    if (t >= static_cast<int64_t>(cols)) a = __builtin_nanf("");
    const float b = ENT ? addr<const float>(g_ent)[r] * inv_t * kLn2 : 0.0f;
    const float h2 = h * (1.0f / kLn2);
    const bool zero = t < 0 || l2 == -__builtin_huge_valf();
    const GradSlice<Fmt> gs(row_ptr<Fmt>(addr<const void>(x), r, stride),
                            const_cast<uint8_t*>(row_ptr<Fmt>(addr<void>(grad), r, cols)), cols,
                            WIDE ? unit - r * slices : 0, slices);
    gs.write(lane, 1 << lg, zero, [&](const float (&e)[VW], uint32_t p0, float (&d)[VW]) {
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const float z = fmaf(e[i] - m, scale, -l2);
            const float p = exp2_f(z);
            d[i] = ENT ? -p * fmaf(b, max_f(z, kZFloor) + h2, a) : -p * a;
        }
        const uint32_t at = static_cast<uint32_t>(t) - p0;
        if (at < VW) {
#pragma unroll
            for (int i = 0; i < VW; ++i) d[i] += at == static_cast<uint32_t>(i) ? a : 0.0f;
        }
    });
}

// ---------------------------------------------------------------------------------------
// Distillation. The teacher's distribution q is the softmax of its k values over the entries
// with an id >= 0; loss = sum q_i (ln q_i - ln p_i), the first part known before the student's.
// stats is [5, rows]: loss, maximum, log2 of the sum, and the same two of the teacher's row.

struct Teacher {
    float m, l2;    // log2 q_i = (v_i - m) scale - l2
    float entropy;  // -sum q_i ln q_i
    __device__ float log_weight(float v, float scale) const { return fmaf(v - m, scale, -l2); }
    __device__ float weight(float v, float scale) const { return exp2_f(log_weight(v, scale)); }
};
// An entry of the teacher's row in LDS: id (-1: absent, cols: beyond the row), weight (first the
// value), the weight of all entries with this id, and the student's logit there. Entry i belongs to
// the lanes i mod T.
struct Entry {
    int32_t id;
    float w, total, x;
};
extern __shared__ Entry s_entries[];

template <typename Fmt>
__device__ inline float student_at(const uint8_t* row, int32_t id, uint32_t cols) {
    return id >= 0 && static_cast<uint32_t>(id) < cols
               ? Fmt::load1(row + static_cast<size_t>(id) * Fmt::kSize)
               : __builtin_nanf("");
}
__device__ inline Entry entry_of(int64_t id, float value, uint32_t cols) {
    return {static_cast<int32_t>(id < 0 ? -1 : id < static_cast<int64_t>(cols) ? id : cols),
            id >= 0 ? value : -__builtin_huge_valf(), 0.0f, __builtin_nanf("")};
}
__device__ inline Entry entry_at(const int64_t* ids, const float* values, uint32_t i, uint32_t cols) {
    return entry_of(ids[i], values[i], cols);
}
// A lane's entry where there are no more entries than lanes, read ahead of its use: up to 64 of them
// every wavefront has its own copy (the student's logits in the team's first alone), beyond that
// the team has one.
template <int T>
__device__ inline Entry own_entry(const int64_t* ids, const float* values, uint32_t k, int lane,
                                  uint32_t cols) {
    const uint32_t i = k <= kWave ? lane % kWave : lane;
    if (k <= T && i < k) return entry_at(ids, values, i, cols);
    return {-1, -__builtin_huge_valf(), 0.0f, __builtin_nanf("")};
}
template <typename Fmt>
__device__ inline void own_student(Entry& mine, const uint8_t* row, uint32_t k, int lane, uint32_t cols) {
    if (k > kWave || lane < kWave) mine.x = student_at<Fmt>(row, mine.id, cols);
}

// Which ids of a row of more than kTeacherCompared entries occur more than once: an open hash table
// in LDS of at least twice as many places. [21454,251] f16 with 251 different ids, loss and gradient:
// 229 us with every entry compared with every other, 129 with the table instead. A place holds an id,
// its top bit set once the id has come again. (No id has all 31 bits set: ids are below cols <=
// INT32_MAX, and cols itself, for ids beyond the row, is not entered.)
struct IdTable {
    uint32_t* place;
    uint32_t mask;
    int32_t cols;
    static constexpr uint32_t kFree = 0xffffffffu, kAgain = 0x80000000u;
    __device__ static uint32_t size(uint32_t k) {
        return k <= kTeacherCompared ? 0 : 2u << (32 - __clz(k - 1));  // as teacher_places
    }
    __device__ void clear(int lane, int team) const {
        for (uint32_t i = lane; i <= mask; i += team) place[i] = kFree;
    }
    __device__ bool entered(int32_t id) const { return id >= 0 && id < cols; }
    __device__ uint32_t first(int32_t id) const {
        return (static_cast<uint32_t>(id) * 0x9e3779b1u) >> 8 & mask;
    }
    __device__ void add(int32_t id) const {
        if (!entered(id)) return;
        for (uint32_t i = first(id);; i = (i + 1) & mask) {  // ends: there are more places than ids
            const uint32_t old = atomicCAS(&place[i], kFree, static_cast<uint32_t>(id));
            if (old == kFree) return;
            if ((old & ~kAgain) == static_cast<uint32_t>(id)) {
                atomicOr(&place[i], kAgain);
                return;
            }
        }
    }
    __device__ bool once(int32_t id) const {
        if (!entered(id)) return true;
        uint32_t i = first(id);
        while ((place[i] & ~kAgain) != static_cast<uint32_t>(id)) i = (i + 1) & mask;
        return place[i] < kAgain;
    }
};

// The totals of a row's entries in LDS, each the sum in the entries' order. A top-k list has no id
// twice: where one is, a wavefront takes such ids of its entries one after the other and looks the row
// through for them, 64 entries at a time. ([4096,32000] bf16 with 1024 random ids, about 16 of them
// there already, loss and gradient: 307 us so, 1036 with a lane per entry adding its row up; 164 with
// different ids. Where most ids are there several times this bounds the kernel: [21454,251] f16 with
// 251 random ids 397 us, 57 with different ones.)
template <int T>
__device__ inline void entry_totals(Entry* ent, const IdTable& table, uint32_t k, int lane) {
    const uint32_t l = lane % kWave;
    for (uint32_t base = lane - l; base < k; base += T) {
        const uint32_t i = base + l;
        const int32_t id = i < k ? ent[i].id : -1;
        float total = i < k ? ent[i].w : 0.0f;
        uint64_t todo = __ballot(table.entered(id) && (k <= kTeacherCompared || !table.once(id)));
        while (todo != 0) {
            const int32_t one = __builtin_amdgcn_readlane(id, __builtin_ctzll(todo));
            float sum = 0.0f;
            for (uint32_t c = 0; c < k; c += kWave) {
                const uint32_t j = c + l < k ? c + l : k - 1;
                const float w = ent[j].w;
                uint64_t hits = __ballot(c + l < k && ent[j].id == one);
                for (; hits != 0; hits &= hits - 1)
                    sum += __uint_as_float(
                        __builtin_amdgcn_readlane(__float_as_uint(w), __builtin_ctzll(hits)));
            }
            if (id == one) total = sum;
            todo &= ~__ballot(id == one);
        }
        if (i < k) ent[i].total = total;
    }
}

// The teacher's row: its entries into `ent`, the distribution's numbers to every thread. *bad: the
// whole gradient is NaN (a weight is NaN, or an id with weight lies beyond the row). With TOTALS the
// totals too: each the sum of the weights with its id, in the entries' order. Up to 64 entries take
// no barrier, up to T (`mine`) three; more are read here and worked off in turns.
template <typename Fmt, int T, bool TOTALS>
__device__ inline Teacher teacher_row(Entry* ent, const IdTable& table, Entry mine, const uint8_t* row,
                                      uint32_t cols, const int64_t* ids, const float* values, uint32_t k,
                                      float scale, int lane, float (*sh)[kShared], bool* bad) {
    // an entry's part of the entropy; NaN for an id with weight beyond the row
    const auto spread = [&](int32_t id, float w, float lw) {
        if (id == static_cast<int32_t>(cols) && w != 0.0f) return __builtin_nanf("");
        return id >= 0 && w > 0.0f ? -w * (lw * kLn2) : 0.0f;
    };
    const auto numbers = [&](float m, float s) {
        return Teacher{s == s ? m : __builtin_nanf(""), log2_f(s), 0.0f};
    };
    // a value's part of the sum; NaN for NaN, which a maximum passes over
    const auto part = [&](float v, float m) {
        return v != v ? v : (m > -__builtin_huge_valf() ? exp2_f((v - m) * scale) : 0.0f);
    };
    float m = -__builtin_huge_valf(), s = 0.0f, h = 0.0f;
    Teacher q;
    if (k <= kWave) {
        m = lanes_max<kWave>(max_f(mine.w, m));
        q = numbers(m, s = lanes_sum<kWave>(part(mine.w, m)));
        const float lw = q.log_weight(mine.w, scale);
        mine.w = exp2_f(lw);
        q.entropy = lanes_sum<kWave>(spread(mine.id, mine.w, lw));
        if (TOTALS && lane < kWave) {
            bool alone = false;
            if (k > kTeacherCompared) {
                table.clear(lane, kWave);
                team_sync<kWave>();
                table.add(mine.id);
                team_sync<kWave>();
                alone = table.once(mine.id);
            }
            mine.total = mine.w;
            if (__any(!alone)) {
                mine.total = 0.0f;
#pragma unroll 8
                for (uint32_t j = 0; j < k; ++j) {
                    const int32_t id = __builtin_amdgcn_readlane(mine.id, static_cast<int>(j));
                    const float w = __uint_as_float(
                        __builtin_amdgcn_readlane(__float_as_uint(mine.w), static_cast<int>(j)));
                    mine.total += id == mine.id ? w : 0.0f;
                }
            }
        }
        if (static_cast<uint32_t>(lane) < k) ent[lane] = mine;
        team_sync<kWave>();
    } else if (k <= T) {
        if constexpr (TOTALS) table.clear(lane, T);
        m = team_reduce<T, true>(max_f(mine.w, m), lane, sh, kSlotMax);
        if constexpr (TOTALS) table.add(mine.id);
        q = numbers(m, s = team_reduce<T, false>(part(mine.w, m), lane, sh, kSlotSum));
        const float lw = q.log_weight(mine.w, scale);
        mine.w = exp2_f(lw);
        if (static_cast<uint32_t>(lane) < k) ent[lane] = mine;
        q.entropy = team_reduce<T, false>(spread(mine.id, mine.w, lw), lane, sh, kSlotEntropy);
    } else {
        if constexpr (TOTALS) table.clear(lane, T);
        constexpr uint32_t N = 4;  // entries a lane loads at once
        for (uint32_t base = lane; base < k; base += N * T) {
            int64_t id[N];
            float v[N];
            Entry e[N];
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                const uint32_t i = base + j * T < k ? base + j * T : base;
                id[j] = ids[i];
                v[j] = values[i];
            }
#pragma unroll
            for (uint32_t j = 0; j < N; ++j) {
                e[j] = entry_of(id[j], v[j], cols);
                if constexpr (TOTALS) e[j].x = student_at<Fmt>(row, e[j].id, cols);
                m = max_f(m, e[j].w);
            }
#pragma unroll
            for (uint32_t j = 0; j < N; ++j)
                if (base + j * T < k) ent[base + j * T] = e[j];
        }
        m = team_reduce<T, true>(m, lane, sh, kSlotMax);
        if constexpr (T == kWave) team_sync<T>();
        for (uint32_t i = lane; i < k; i += T) {
            s += part(ent[i].w, m);
            if constexpr (TOTALS) table.add(ent[i].id);
        }
        q = numbers(m, s = team_reduce<T, false>(s, lane, sh, kSlotSum));
        for (uint32_t i = lane; i < k; i += T) {
            const int32_t id = ent[i].id;
            const float lw = q.log_weight(ent[i].w, scale);
            const float w = exp2_f(lw);
            ent[i].w = w;
            h += spread(id, w, lw);
            // (the loss alone: [4096,32000] bf16 with 1024 entries 72 us, 86 with them above; the step
            // [8192,16000] f16 with 1000 the other way round, 216 and 188)
            if constexpr (!TOTALS) ent[i].x = student_at<Fmt>(row, id, cols);
        }
        q.entropy = team_reduce<T, false>(h, lane, sh, kSlotEntropy);
    }
    if constexpr (TOTALS) {
        if (k > kWave) {  // (the last reduction's barrier has made the table and the weights visible)
            if constexpr (T == kWave) team_sync<T>();
            entry_totals<T>(ent, table, k, lane);
        }
    }
    *bad = s != s || q.entropy != q.entropy;
    return q;
}

__device__ inline void store_distill(float* stats, uint32_t rows, uint32_t r, float loss, float m,
                                     float l2, const Teacher& q) {
    const size_t n = rows;
    stats[r] = loss;
    stats[n + r] = m;
    stats[2 * n + r] = l2;
    stats[3 * n + r] = q.m;
    stats[4 * n + r] = q.l2;
}

// sum q ln p is added up in units of 2^8: weights that add up to a little more than 1 would take a
// row whose every weight lies on logits of the lowest finite value (a mask) out of range. Infinite
// is only the loss of a row with a logit of -inf at a weight.
constexpr float kLossUnit = 0x1p-8f;
__device__ inline float loss_of(const Teacher& q, float sum) {
    const float v = sum * (1.0f / kLossUnit);
    return -q.entropy - (sum > -__builtin_huge_valf() ? max_f(v, kLowest) : v);
}

// The loss of a row from its merged statistics and log2 of their sum (in lane 0 of the team).
template <int T>
__device__ inline float distill_loss(const Entry* ent, uint32_t k, float scale, const Teacher& q,
                                     const Stat& a, float l2, int lane, float (*sh)[kShared]) {
    float sum = 0.0f;
    for (uint32_t i = lane; i < k; i += T) {
        const Entry e = ent[i];
        if (e.id < 0 || e.w == 0.0f) continue;
        const float lp = a.s == 0.0f ? -__builtin_huge_valf() : ln_p(e.x, a.m, l2, scale);
        sum = fmaf(e.w, lp * kLossUnit, sum);
    }
    sum = k <= kWave ? lanes_sum<kWave>(sum) : team_reduce<T, false>(sum, lane, sh, kSlotLoss);
    return loss_of(q, sum);
}

// The loss alone, a team of T lanes per row. [512,128256] f16 with 32 entries: 23.7 us, 5.5 TB/s, bound
// by the read of two rows per CU one after the other, with the tail of each exposed.
template <typename Fmt, bool KEEP, int T>
__global__ __launch_bounds__(kTeamBlock<T>) void k_ds_team(const void* x, uint32_t cols,
                                                           uint32_t stride, float scale,
                                                           uint32_t rows, uint32_t k,
                                                           const int64_t* ids_, const float* values_,
                                                           float* stats) {
    __shared__ float sh[T / kWave][kShared];
    const uint32_t r = blockIdx.x * kTeamsPerBlock<T> + team_of<T>();
    const int lane = lane_of<T>();
    if (r >= rows) return;
    const int64_t* ids = ids_ + static_cast<size_t>(r) * k;
    const float* values = values_ + static_cast<size_t>(r) * k;
    const uint8_t* row = row_ptr<Fmt>(x, r, stride);
    Entry* ent = s_entries + team_of<T>() * k;
    bool bad;
    Entry mine = own_entry<T>(ids, values, k, lane, cols);
    own_student<Fmt>(mine, row, k, lane, cols);
    const Teacher q = teacher_row<Fmt, T, false>(ent, IdTable{}, mine, row, cols, ids, values, k, scale,
                                                 lane, sh, &bad);
    if (q.m == -__builtin_huge_valf()) {
        if (lane == 0) store_distill(stats, rows, r, 0.0f, 0.0f, 0.0f, q);
        return;
    }
    const Span<Fmt, KEEP> sp(row, cols);
    Stat a;
    scan_span<Fmt, false, T, kUnroll<Fmt, false>>(sp, true, sp.va, sp.vb, lane, scale, a);
    team_merge<false, T>(a, scale, lane, sh);
    const float l2 = bad ? __builtin_nanf("") : log2_f(a.s);
    const float loss = distill_loss<T>(ent, k, scale, q, a, l2, lane, sh);
    if (lane == 0) store_distill(stats, rows, r, loss, a.m, l2, q);
}

// Rows of at most G vectors, G lanes each, the row held in registers; with GRAD the gradient too.
// [52618,63] bf16 with 16 entries: 8.0 us for the loss, 13.8 for both (24 MB, 1.8 TB/s, bound by a
// row's chain of loads and reductions); 29.8 and 95.8 with a wavefront per row. Tags as for k_ds_grad
// (none in grad).
template <typename Fmt, bool GRAD, int G>
__global__ __launch_bounds__(kBlockThreads) void k_ds_group(uint64_t x, uint64_t ids_, uint64_t values_,
                                                            uint64_t stats_, uint64_t w, uint64_t grad,
                                                            uint32_t stride, uint32_t rows) {
    constexpr int VW = Fmt::VW;
    const uint32_t cols = tags(x, ids_), k = tag(values_);
    const float scale = __uint_as_float(tags(stats_, w));
    const uint32_t want = blockIdx.x * (kBlockThreads / G) + threadIdx.x / G;
    const bool extra = want >= rows;  // lanes past the end repeat the last row and store nothing
    const uint32_t r = extra ? rows - 1 : want;
    const int lane = threadIdx.x % G;
    const int64_t* ids = addr<const int64_t>(ids_) + static_cast<size_t>(r) * k;
    const float* values = addr<const float>(values_) + static_cast<size_t>(r) * k;
    const uint8_t* row = row_ptr<Fmt>(addr<const void>(x), r, stride);
    Entry* ent = s_entries + threadIdx.x / G * k;
    const Span<Fmt, true> sp(row, cols);
    const uint32_t p0 = sp.pos(lane);
    float e[VW];
#pragma unroll
    for (int i = 0; i < VW; ++i) e[i] = -__builtin_huge_valf();
    if (static_cast<uint32_t>(lane) < sp.vs) {
        Fmt::unpack(sp.load(lane), e);
#pragma unroll
        for (int i = 0; i < VW; ++i) e[i] = p0 + i < cols ? e[i] : -__builtin_huge_valf();
    }
    // the teacher's row
    float m = -__builtin_huge_valf(), s = 0.0f, h = 0.0f;
    for (uint32_t i = lane; i < k; i += G) {
        Entry t = entry_at(ids, values, i, cols);
        t.x = student_at<Fmt>(row, t.id, cols);
        m = max_f(m, t.w);
        if (t.w != t.w) s = t.w;
        ent[i] = t;
    }
    m = lanes_max<G>(m);
    if (m > -__builtin_huge_valf())
        for (uint32_t i = lane; i < k; i += G) s += exp2_f((ent[i].w - m) * scale);
    s = lanes_sum<G>(s);
    Teacher q{s == s ? m : __builtin_nanf(""), log2_f(s), 0.0f};
    for (uint32_t i = lane; i < k; i += G) {
        const float lw = q.log_weight(ent[i].w, scale), wt = exp2_f(lw);
        // NaN for an id with weight beyond the row, so that the loss is NaN whatever the logits are
        if (ent[i].id == static_cast<int32_t>(cols) && wt != 0.0f) h = __builtin_nanf("");
        if (ent[i].id >= 0 && wt > 0.0f) h -= wt * (lw * kLn2);
        ent[i].w = wt;
    }
    q.entropy = lanes_sum<G>(h);
    const bool bad = s != s || q.entropy != q.entropy;
    team_sync<kWave>();
    if constexpr (GRAD) {
        for (uint32_t i = lane; i < k; i += G) {
            const int32_t id = ent[i].id;
            float total = 0.0f;
#pragma unroll 4
            for (uint32_t j = 0; j < k; ++j) total += ent[j].id == id ? ent[j].w : 0.0f;
            ent[i].total = total;
        }
    }
    // the student's row
    const bool absent = q.m == -__builtin_huge_valf();
    Stat a;
    a.init();
    a.m = lanes_max<G>(max_f(a.m, max_of(e)));
    take<false>(e, scale, a);
    a.s = lanes_sum<G>(a.s);
    const float l2 = bad ? __builtin_nanf("") : log2_f(a.s);
    float sum = 0.0f;
    for (uint32_t i = lane; i < k; i += G) {
        const Entry t = ent[i];
        if (t.id < 0 || t.w == 0.0f) continue;
        const float lp = a.s == 0.0f ? -__builtin_huge_valf() : ln_p(t.x, a.m, l2, scale);
        sum = fmaf(t.w, lp * kLossUnit, sum);
    }
    sum = lanes_sum<G>(sum);
    if (lane == 0 && !extra)
        store_distill(addr<float>(stats_), rows, r, absent ? 0.0f : loss_of(q, sum), absent ? 0.0f : a.m,
                      absent ? 0.0f : l2, q);
    if constexpr (GRAD) {
        if (extra) return;
        uint8_t* out = const_cast<uint8_t*>(row_ptr<Fmt>(addr<void>(grad), r, cols));
        const bool zero = absent || l2 == -__builtin_huge_valf();
        const float coef = addr<const float>(w)[r] * scale * kLn2;
        float d[VW];
#pragma unroll
        for (int i = 0; i < VW; ++i) d[i] = coef * exp2_f(fmaf(e[i] - a.m, scale, -l2));
        if (zero) {
#pragma unroll
            for (int i = 0; i < VW; ++i) d[i] = 0.0f;
        }
        const uint32_t v = lane;
        if (v >= sp.va && v < sp.vb) {
            store16_any<Fmt>(out + static_cast<size_t>(p0) * Fmt::kSize, pack<Fmt>(d));
        } else if (v < sp.vs) {
#pragma unroll
            for (int i = 0; i < VW; ++i)
                if (p0 + i < cols) reinterpret_cast<typename Fmt::Bits*>(out)[p0 + i] = round_to<Fmt>(d[i]);
        }
        // (the wavefront's own stores to an address keep their order)
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (zero) return;
        for (uint32_t i = lane; i < k; i += G) {
            const Entry t = ent[i];
            if (t.id < 0 || static_cast<uint32_t>(t.id) >= cols) continue;
            const float p = exp2_f(fmaf(t.x - a.m, scale, -l2));
            reinterpret_cast<typename Fmt::Bits*>(out)[t.id] = round_to<Fmt>(coef * (p - t.total));
        }
    }
}

// One workgroup per split row: 2.5 us for one row, 3.9 for 100, a launch and the latencies of the
// entries and the slices' statistics. Tags: teacher entries in ids, slices of the row in values.
template <typename Fmt>
__global__ __launch_bounds__(kMergeThreads) void k_ds_merge(const void* x, uint32_t cols,
                                                            uint32_t stride, float scale,
                                                            uint32_t rows, uint64_t ids_,
                                                            uint64_t values_, const Part* part,
                                                            float* stats) {
    constexpr int T = kMergeThreads;
    __shared__ float sh[T / kWave][kShared];
    const uint32_t k = tag(ids_), parts = tag(values_);
    const uint32_t r = blockIdx.x;
    const int lane = threadIdx.x;
    const int64_t* ids = addr<const int64_t>(ids_) + static_cast<size_t>(r) * k;
    const float* values = addr<const float>(values_) + static_cast<size_t>(r) * k;
    const uint8_t* row = row_ptr<Fmt>(x, r, stride);
    bool bad;
    Entry mine = own_entry<T>(ids, values, k, lane, cols);
    own_student<Fmt>(mine, row, k, lane, cols);
    const Teacher q = teacher_row<Fmt, T, false>(s_entries, IdTable{}, mine, row, cols, ids, values, k, scale,
                                                 lane, sh, &bad);
    if (q.m == -__builtin_huge_valf()) {
        if (lane == 0) store_distill(stats, rows, r, 0.0f, 0.0f, 0.0f, q);
        return;
    }
    const Stat a = merge_parts<false, T>(part + static_cast<size_t>(r) * parts, parts, scale, lane, sh);
    const float l2 = bad ? __builtin_nanf("") : log2_f(a.s);
    const float loss = distill_loss<T>(s_entries, k, scale, q, a, l2, lane, sh);
    if (lane == 0) store_distill(stats, rows, r, loss, a.m, l2, q);
}

// The gradient of a row: g (p_j - q_j) / T. The dense part g p_j / T is stored first; after it each
// teacher entry's element is stored again with its weight taken off: the sum of the weights of equal
// ids, which every one of them stores. A team of T lanes (32: of 2^lg, up to 32) for a slice of a
// row has the slice's entries in LDS. [4096,128256] bf16 with 64 entries: 416 us, 5.1 TB/s read and
// written, bound by that; [4096,32000] with 1024 random ones 265 us, bound by the entries (553 and 7958
// us with each entry compared with all others from global memory). A row by a wavefront: [21454,251]
// f16 with 251 different ids 42 us; by a group of lanes: [52618,63] bf16 with 16 12.2 us. Tags: columns
// in (x, ids), teacher entries in values, scale in (stats, g), lg and the slices (12 bits above 4) in
// grad.
template <typename Fmt, int T>
__global__ __launch_bounds__(kBlockThreads) void k_ds_grad(uint64_t x, uint64_t ids_, uint64_t values_,
                                                           uint64_t stats_, uint64_t g, uint64_t grad,
                                                           uint32_t stride, uint32_t rows) {
    constexpr int VW = Fmt::VW;
    constexpr bool kWide = T == kBlockThreads;
    const uint32_t cols = tags(x, ids_), k = tag(values_);
    const float scale = __uint_as_float(tags(stats_, g));
    const uint32_t lg = kWide ? 8 : T == kWave ? 6 : tag(grad) & 15, slices = kWide ? tag(grad) >> 4 : 1;
    const uint32_t team = kWide ? 0 : T == kWave ? team_of<kWave>() : threadIdx.x >> lg;
    const uint32_t unit = kWide ? blockIdx.x : (blockIdx.x << (8 - lg)) + team;
    const uint32_t r = kWide ? unit / slices : unit;
    if (r >= rows) return;  // whole teams, and never one of several wavefronts
    const uint32_t lanes = 1u << lg;
    const int lane = threadIdx.x & (lanes - 1);
    const float* stats = addr<const float>(stats_);
    const size_t n = rows;
    const float m = stats[n + r], l2 = stats[2 * n + r];
    const Teacher q{stats[3 * n + r], stats[4 * n + r], 0.0f};
    const float coef = addr<const float>(g)[r] * scale * kLn2;
    const GradSlice<Fmt> gs(row_ptr<Fmt>(addr<const void>(x), r, stride),
                            const_cast<uint8_t*>(row_ptr<Fmt>(addr<void>(grad), r, cols)), cols,
                            kWide ? unit - r * slices : 0, slices);
    const bool zero = q.m == -__builtin_huge_valf() || l2 == -__builtin_huge_valf();
    Entry* ent = s_entries + team * k;
    const uint32_t places = T == 32 ? 0 : IdTable::size(k);  // the tables lie behind all teams' entries
    const IdTable table{reinterpret_cast<uint32_t*>(s_entries + (kBlockThreads >> lg) * k) + team * places,
                        places - 1, static_cast<int32_t>(cols)};
    if (!zero) {
        const int64_t* ids = addr<const int64_t>(ids_) + static_cast<size_t>(r) * k;
        const float* values = addr<const float>(values_) + static_cast<size_t>(r) * k;
        if (places != 0) {
            table.clear(lane, lanes);
            if constexpr (T > 32) team_sync<T>();
        }
        for (uint32_t i = lane; i < k; i += lanes) {
            const int64_t id = ids[i];
            const bool in = id >= 0 && id < static_cast<int64_t>(cols) && gs.holds(id);
            Entry t{in ? static_cast<int32_t>(id) : -1, 0.0f, 0.0f, 0.0f};
            if (in) {
                t.w = q.weight(values[i], scale);
                t.x = Fmt::load1(gs.x + id * Fmt::kSize);
            }
            ent[i] = t;
            if (places != 0) table.add(t.id);
        }
    }
    gs.write(lane, lanes, zero, [&](const float (&e)[VW], uint32_t, float (&d)[VW]) {
#pragma unroll
        for (int i = 0; i < VW; ++i) d[i] = coef * exp2_f(fmaf(e[i] - m, scale, -l2));
    });
    // the dense stores before those of the entries: a wavefront's own keep their order
    if constexpr (kWide)
        __syncthreads();
    else
        team_sync<kWave>();
    if (zero) return;
    if constexpr (T > 32) entry_totals<T>(ent, table, k, lane);
    for (uint32_t i = lane; i < k; i += lanes) {
        Entry t = ent[i];
        if (t.id < 0) continue;
        if constexpr (T == 32) {
#pragma unroll 4
            for (uint32_t j = 0; j < k; ++j) t.total += ent[j].id == t.id ? ent[j].w : 0.0f;
        }
        const float p = exp2_f(fmaf(t.x - m, scale, -l2));
        reinterpret_cast<typename Fmt::Bits*>(gs.g)[t.id] = round_to<Fmt>(coef * (p - t.total));
    }
}

// Loss and gradient of a row in one kernel. A lane keeps its first NV vectors in registers from
// the pass that takes the maximum and the sum to the pass that writes the gradient, so that the
// logits are read from memory once; vectors beyond them are read again, mostly from the caches.
// The registers of a CU hold few rows, so a team goes through several, and as soon as a vector's
// gradient is stored, the vector of the team's next row is loaded in its place: the loads run
// beside the second pass's arithmetic and stores. [4096,128256] bf16 with 64 entries: 439 us, 4.8 TB/s
// read and written (535 with all vectors read again, 597 held without that overlap); [1003,50001] f16
// 43 us, 4.6 TB/s; [16,32000] f32 8.5 us, a row's latency from end to end. Rows of up to 128 vectors
// hold two per lane, in half the registers, so that twice the wavefronts hide their latency:
// [21454,251] f16 with 251 different entries 57 us, 100 with eight. A row without a teacher is read
// like any other, since its loads are under way before its entries are known: with three rows in four
// of [4096,128256] so, 430 us. Tags as for k_ds_grad, but the workgroups of the grid in grad.
template <int T>
constexpr int kStepRows = step_rows(T);
template <typename Fmt, int T, int NV>
__global__ __launch_bounds__(kTeamBlock<T>, NV > 2 ? 4 : 8) void k_ds_step(uint64_t x, uint64_t ids_, uint64_t values_,
                                                           uint64_t stats_, uint64_t w, uint64_t grad_,
                                                           uint32_t stride, uint32_t rows) {
    constexpr int VW = Fmt::VW;
    // 128 registers suffice, 64 for two vectors
    constexpr int U = NV == 8 ? kUnroll<Fmt, false> : kUnroll<Fmt, false> / 2;
    static_assert(NV % U == 0, "whole steps");
    __shared__ float sh[T / kWave][kShared];
    const uint32_t cols = tags(x, ids_), k = tag(values_), teams = tag(grad_) * kTeamsPerBlock<T>;
    const float scale = __uint_as_float(tags(stats_, w));
    const int lane = lane_of<T>();
    uint32_t r = blockIdx.x * kTeamsPerBlock<T> + team_of<T>();
    if (r >= rows) return;
    // the entries of two rows if a wavefront may be one row ahead of another
    constexpr uint32_t kBuffers = kStepRows<T>;
    Entry* ent = s_entries + team_of<T>() * kBuffers * k;
    Entry* other = ent + (kBuffers - 1) * k;
    const uint32_t places = IdTable::size(k);  // the tables lie behind all teams' entries
    const IdTable table{reinterpret_cast<uint32_t*>(s_entries + kTeamsPerBlock<T> * kBuffers * k) +
                            team_of<T>() * places,
                        places - 1, static_cast<int32_t>(cols)};
    const auto ids_at = [&](uint32_t n) { return addr<const int64_t>(ids_) + static_cast<size_t>(n) * k; };
    const auto values_at = [&](uint32_t n) { return addr<const float>(values_) + static_cast<size_t>(n) * k; };
    const auto row_at = [&](uint32_t n) { return row_ptr<Fmt>(addr<const void>(x), n, stride); };
    typename Fmt::Vec held[NV];
    const auto load = [&](const Span<Fmt>& sp, int i) {
        const uint32_t v = sp.va + lane + i * T;
        if (sp.va + i * T < sp.vb) held[i] = sp.load(v < sp.vb ? v : sp.vb - 1);
    };
    Entry mine = own_entry<T>(ids_at(r), values_at(r), k, lane, cols);
    {
        const Span<Fmt> sp(row_at(r), cols);
#pragma unroll
        for (int i = 0; i < NV; ++i) load(sp, i);
    }
    while (true) {
        const uint8_t* row = row_at(r);
        own_student<Fmt>(mine, row, k, lane, cols);
        uint8_t* out = const_cast<uint8_t*>(row_ptr<Fmt>(addr<void>(grad_), r, cols));
        const Span<Fmt> sp(row, cols);
        bool bad;
        const Teacher q = teacher_row<Fmt, T, true>(ent, table, mine, row, cols, ids_at(r), values_at(r), k,
                                                    scale, lane, sh, &bad);
        const bool absent = q.m == -__builtin_huge_valf();
        float loss = 0.0f, l2 = 0.0f;
        Stat a{0.0f, 0.0f, 0.0f};
        const uint32_t rest = sp.vb - sp.va > NV * T ? sp.va + NV * T : sp.vb;  // first vector not held
        if (!absent) {
            // the steps of scan_span, the first of them from registers
            a.init();
            if (lane < 2) scan_edge<Fmt, false>(sp, lane, scale, a);
#pragma unroll
            for (int i = 0; i < NV; i += U) {
                if (sp.vb - sp.va >= (i + U) * T) {
                    typename Fmt::Vec h[U];
                    float e[U * VW];
#pragma unroll
                    for (int u = 0; u < U; ++u) h[u] = held[i + u];
                    unpack_all<Fmt, U>(h, e);
                    take<false>(e, scale, a);
                } else {
#pragma unroll
                    for (int u = 0; u < U; ++u) {
                        if (sp.va + (i + u) * T < sp.vb) {
                            float f[VW];
                            Fmt::unpack(masked_unless<Fmt>(sp.va + lane + (i + u) * T < sp.vb, held[i + u]), f);
                            take<false>(f, scale, a);
                        }
                    }
                }
            }
            if (rest < sp.vb) scan_on<Fmt, false, T, U>(sp, rest, sp.vb, lane, scale, a);
            team_merge<false, T>(a, scale, lane, sh);
            l2 = bad ? __builtin_nanf("") : log2_f(a.s);
            loss = distill_loss<T>(ent, k, scale, q, a, l2, lane, sh);
        } else {
            team_sync<T>();  // every row has a barrier: none gets two rows ahead of another
        }
        if (lane == 0) store_distill(addr<float>(stats_), rows, r, loss, a.m, l2, q);
        const bool zero = absent || l2 == -__builtin_huge_valf();
        const float coef = addr<const float>(w)[r] * scale * kLn2;
        const auto write = [&](const typename Fmt::Vec& v16, uint32_t v) {
            float e[VW], d[VW];
            Fmt::unpack(v16, e);
#pragma unroll
            for (int j = 0; j < VW; ++j) d[j] = coef * exp2_f(fmaf(e[j] - a.m, scale, -l2));
            typename Fmt::Vec g = pack<Fmt>(d);
            if (zero) g = __builtin_bit_cast(typename Fmt::Vec, u32x4{0, 0, 0, 0});
            store16_any<Fmt>(out + static_cast<size_t>(sp.pos(v)) * Fmt::kSize, g);
        };
        const uint32_t next = r + teams;
        const uint32_t nr = next < rows ? next : r;
        const Span<Fmt> np(row_at(nr), cols);
        mine = own_entry<T>(ids_at(nr), values_at(nr), k, lane, cols);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const uint32_t v = sp.va + lane + i * T;
            if (v < sp.vb) write(held[i], v);
            if (next < rows) load(np, i);
        }
        for (uint32_t v = rest + lane; v < sp.vb; v += T) write(sp.load(v), v);
        const uint32_t ev = sp.edge(lane);
        if (ev != kNoVec) {
            const uint32_t p0 = sp.pos(ev);
            for (uint32_t p = p0; p != p0 + VW; ++p) {
                if (p >= cols) continue;
                const float e = Fmt::load1(row + static_cast<size_t>(p) * Fmt::kSize);
                reinterpret_cast<typename Fmt::Bits*>(out)[p] =
                    round_to<Fmt>(zero ? 0.0f : coef * exp2_f(fmaf(e - a.m, scale, -l2)));
            }
        }
        // Each wavefront stores again the elements at the teacher's ids that it has just stored: its
        // own stores to an address keep their order, so no barrier is needed.
        __builtin_amdgcn_fence(__ATOMIC_ACQ_REL, "wavefront");
        if (!zero) {
            for (uint32_t i = lane % kWave; i < k; i += kWave) {
                const Entry e = ent[i];
                if (e.id < 0 || static_cast<uint32_t>(e.id) >= cols) continue;
                const uint32_t v = (static_cast<uint32_t>(e.id) + sp.off) / VW;
                const uint32_t owner = v >= sp.va && v < sp.vb ? (v - sp.va) % T / kWave : 0;
                if (owner != static_cast<uint32_t>(lane) / kWave) continue;
                const float p = exp2_f(fmaf(e.x - a.m, scale, -l2));
                reinterpret_cast<typename Fmt::Bits*>(out)[e.id] = round_to<Fmt>(coef * (p - e.total));
            }
        }
        if (next >= rows) return;
        Entry* const t = ent;
        ent = other;
        other = t;
        r = next;
    }
}

// ---------------------------------------------------------------------------------------
// Launch

template <typename F>
void with_team(int team, F f) {
    switch (team) {
        case 64: f(Int<64>{}); break;
        case 256: f(Int<256>{}); break;
        case 512: f(Int<512>{}); break;
        default: f(Int<1024>{}); break;
    }
}
template <typename F>
void with_group(int lanes, F f) {
    switch (lanes) {
        case 4: f(Int<4>{}); break;
        case 8: f(Int<8>{}); break;
        case 16: f(Int<16>{}); break;
        default: f(Int<32>{}); break;
    }
}
template <typename F>
void with_format_and_keep(const LogitsArgs& a, F f) {
    with_format(a.dtype, [&](auto fmt) { with_bool(a.keep, [&](auto keep) { f(fmt, keep); }); });
}

// With LDS for the teacher's entries of the workgroup's rows, and a hash table for each.
static_assert(sizeof(Entry) == kEntryBytes, "the plans count with it");
template <typename... KArgs, typename... Args>
void launch_entries(void (*kernel)(KArgs...), uint32_t grid, int block, size_t lds, hipStream_t s,
                    Args... args) {
    hipLaunchKernelGGL(kernel, dim3(grid), dim3(block), lds, s, args...);
}

}  // namespace

size_t part_bytes() { return sizeof(Part); }

hipError_t launch_logprobs(const LogitsPlan& plan, const LogitsArgs& a, const int64_t* tokens,
                           bool entropy, bool apart, int top, float* stats, float* top_logprobs,
                           int64_t* top_tokens, uint8_t* scratch16, hipStream_t s) {
    const uint32_t outputs = static_cast<uint32_t>(top) | (apart ? kApart : 0);
    const uint32_t cols = static_cast<uint32_t>(a.cols), stride = static_cast<uint32_t>(a.row_stride);
    const uint32_t rows = static_cast<uint32_t>(a.rows);
    const uint32_t grid = static_cast<uint32_t>(plan.grid_blocks);
    with_format_and_keep(a, [&](auto fmt, auto keep) {
        using Fmt = decltype(fmt);
        constexpr bool KEEP = decltype(keep)::value;
        with_bool(entropy, [&](auto ent) {
            constexpr bool ENT = decltype(ent)::value;
            if (plan.path == ARGREDUCE_PATH_SUBWAVE && plan.team < kWave) {
                const auto go = [&](auto g) {
                    launch(k_lp_group<Fmt, KEEP, ENT, decltype(g)::value>, grid, kBlockThreads, s, a.x, cols,
                           stride, a.scale, rows, tokens, stats, tagged(top_logprobs, outputs), top_tokens);
                };
                with_group(plan.team, go);
                return;
            }
            with_bool(top > 0, [&](auto tp) {
                constexpr bool TOP = decltype(tp)::value;
                if (plan.path == ARGREDUCE_PATH_SPLIT) {
                    Part* part = reinterpret_cast<Part*>(scratch16);
                    launch(k_part<Fmt, KEEP, ENT>, grid, kPartThreads, s, a.x, cols, stride, a.scale,
                           static_cast<uint32_t>(plan.parts), tokens, part);
                    const uint32_t sc = bits_of(a.scale);
                    launch(k_lp_merge<Fmt, ENT, TOP>, rows, TOP ? kMergeTopThreads : kMergeThreads, s,
                           tagged(a.x, cols), tagged(tokens, cols >> 16), tagged(part, plan.parts),
                           tagged(stats, outputs), tagged(top_logprobs, sc), tagged(top_tokens, sc >> 16), stride, rows);
                    return;
                }
                with_team(plan.team, [&](auto team) {
                    constexpr int T = decltype(team)::value;
                    launch(k_lp_team<Fmt, KEEP, ENT, TOP, T>, grid, kTeamBlock<T>, s, a.x, cols, stride,
                           a.scale, rows, tokens, stats, tagged(top_logprobs, outputs), top_tokens);
                });
            });
        });
    });
    return hipGetLastError();
}

hipError_t launch_logprobs_grad(const GradPlan& plan, const LogitsArgs& a, const int64_t* tokens,
                                const float* stats, const float* g_logprob, const float* g_entropy,
                                void* grad, hipStream_t s) {
    const uint32_t cols = static_cast<uint32_t>(a.cols), sc = bits_of(a.scale);
    with_format(a.dtype, [&](auto fmt) {
        using Fmt = decltype(fmt);
        with_bool(g_entropy != nullptr, [&](auto ent) {
            with_bool(plan.team == kBlockThreads, [&](auto wide) {
                launch(k_lp_grad<Fmt, decltype(ent)::value, decltype(wide)::value>,
                       static_cast<uint32_t>(plan.grid_blocks), kBlockThreads, s, tagged(a.x, cols),
                       tagged(tokens, cols >> 16), tagged(stats, sc), tagged(g_logprob, sc >> 16),
                       tagged(g_entropy, plan.slices), tagged(grad, log2_of(plan.team)),
                       static_cast<uint32_t>(a.row_stride), static_cast<uint32_t>(a.rows));
            });
        });
    });
    return hipGetLastError();
}

hipError_t launch_distill_grad(const GradPlan& plan, const LogitsArgs& a, int k, const int64_t* ids,
                               const float* values, const float* stats, const float* g_loss,
                               void* grad, hipStream_t s) {
    const uint32_t cols = static_cast<uint32_t>(a.cols), sc = bits_of(a.scale);
    with_format(a.dtype, [&](auto fmt) {
        using Fmt = decltype(fmt);
        const auto go = [&](auto team) {
            constexpr int T = decltype(team)::value;
            const int teams = kBlockThreads / plan.team;
            launch_entries(k_ds_grad<Fmt, T>, static_cast<uint32_t>(plan.grid_blocks), kBlockThreads,
                           entries_lds(teams, 1, k, T > 32), s, tagged(a.x, cols), tagged(ids, cols >> 16),
                           tagged(values, k), tagged(stats, sc), tagged(g_loss, sc >> 16),
                           tagged(grad, log2_of(plan.team) | (plan.slices << 4)),
                           static_cast<uint32_t>(a.row_stride), static_cast<uint32_t>(a.rows));
        };
        if (plan.team == kBlockThreads)
            go(Int<kBlockThreads>{});
        else if (plan.team == kWave)
            go(Int<kWave>{});
        else
            go(Int<32>{});
    });
    return hipGetLastError();
}

hipError_t launch_distill(const LogitsPlan& plan, const GradPlan& gplan, const LogitsArgs& a, int k,
                          const int64_t* ids, const float* values, float* stats,
                          const float* weights, void* grad, uint8_t* scratch16, hipStream_t s) {
    const uint32_t cols = static_cast<uint32_t>(a.cols), stride = static_cast<uint32_t>(a.row_stride);
    const uint32_t rows = static_cast<uint32_t>(a.rows), sc = bits_of(a.scale);
    const uint32_t grid = static_cast<uint32_t>(plan.grid_blocks);
    with_format_and_keep(a, [&](auto fmt, auto keep) {
        using Fmt = decltype(fmt);
        constexpr bool KEEP = decltype(keep)::value;
        if (plan.path == ARGREDUCE_PATH_SPLIT) {
            Part* part = reinterpret_cast<Part*>(scratch16);
            launch(k_part<Fmt, KEEP, false>, grid, kPartThreads, s, a.x, cols, stride, a.scale,
                   static_cast<uint32_t>(plan.parts), static_cast<const int64_t*>(nullptr), part);
            launch_entries(k_ds_merge<Fmt>, rows, kMergeThreads, k * kEntryBytes, s, a.x, cols, stride, a.scale,
                           rows, tagged(ids, k), tagged(values, plan.parts), static_cast<const Part*>(part), stats);
            return;
        }
        if (plan.team < kWave) {
            with_bool(grad != nullptr, [&](auto gr) {
                const auto go = [&](auto g) {
                    constexpr int G = decltype(g)::value;
                    launch_entries(k_ds_group<Fmt, decltype(gr)::value, G>, grid, kBlockThreads,
                                   entries_lds(kBlockThreads / G, 1, k, false), s, tagged(a.x, cols),
                                   tagged(ids, cols >> 16), tagged(values, k), tagged(stats, sc), tagged(weights, sc >> 16),
                                   tagged(grad, 0), stride, rows);
                };
                with_group(plan.team, go);
            });
            return;
        }
        with_team(plan.team, [&](auto team) {
            constexpr int T = decltype(team)::value;
            const auto step = [&](auto held) {
                launch_entries(k_ds_step<Fmt, T, decltype(held)::value>, grid, kTeamBlock<T>,
                               entries_lds(kTeamsPerBlock<T>, kStepRows<T>, k, true), s, tagged(a.x, cols),
                               tagged(ids, cols >> 16), tagged(values, k), tagged(stats, sc),
                               tagged(weights, sc >> 16), tagged(grad, grid), stride, rows);
            };
            if (grad != nullptr && T >= 512 && plan.held > 8)
                step(Int<T >= 512 ? 16 : 8>{});
            else if (grad != nullptr && T == kWave && plan.held < 8)
                step(Int<T == kWave ? 2 : 8>{});
            else if (grad != nullptr)
                step(Int<8>{});
            else
                launch_entries(k_ds_team<Fmt, KEEP, T>, grid, kTeamBlock<T>,
                               entries_lds(kTeamsPerBlock<T>, 1, k, false), s, a.x, cols, stride, a.scale, rows,
                               static_cast<uint32_t>(k), ids, values, stats);
        });
    });
    if (plan.path == ARGREDUCE_PATH_SPLIT && grad != nullptr)
        return launch_distill_grad(gplan, a, k, ids, values, stats, weights, grad, s);
    return hipGetLastError();
}

}  // namespace argreduce
