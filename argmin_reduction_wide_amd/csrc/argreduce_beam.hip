// Beam search on gfx950: the step that chooses the best continuations of a group of beams from their
// logits, and the reordering of the beams' states that follows it.
//
// Step. Row b of a group holds the logits x of beam b, whose score (sum of log probabilities) is S_b.
// With k = log2(e) / T,
//   value(b, v) = S_b + ln p_bv = S_b + (x_bv - m_b) / T - ln s_b,
//   m_b = max_v x_bv,  s_b = sum_v 2^((x_bv - m_b) k),
// and the step keeps the `width` largest values over all beams and tokens. Inside a row the order is
// that of the logits, whatever the statistics are: a slice of a row leaves its `width` largest logits
// and its part of (m, s) in scratch, and one workgroup per group joins the lists. There the order
// between rows depends on ln s, and two continuations of different beams can lie as close to each
// other as they like: everything after the slices' sums is in binary64, and two error terms that are
// alike for a whole row are taken out of the sums:
//   * 2^(d k) with k rounded to binary32 (k_hi) lacks the factor 2^(d k_lo) = 1 + ln 2 d k_lo:
//     with h = sum 2^z z, z = d k_hi, the sum is s + ln 2 (k_lo / k_hi) h;
//   * the logarithm is binary64's.
// What is left is the rounding of the single terms and of a lane's running sum, which is random: about
// 1e-8 of s. Equal rows have equal sums wherever they lie (RowSpan), so that equal continuations of
// different beams tie.
#include <hip/hip_runtime.h>

#include "argreduce_beam.hpp"
#include "argreduce_logits_device.hpp"

#pragma clang fp contract(off)

namespace argreduce {
namespace {

constexpr double kLn2d = 0.693147180559945309417;

// What a slice leaves in scratch, before its list of candidates (keys of key_of, best first).
struct Slice {
    float m, s, h;
    uint32_t count;
};

__device__ inline bool alive(float score) { return score > -__builtin_huge_valf() && score < __builtin_huge_valf(); }

// One slice of a row per team. [2048,128256] bf16: bound by the read, like the log probabilities
// with alternatives.
// Tags: columns in (x, scores), slices per row in ended, width in scratch.
template <typename Fmt, int T>
__global__ __launch_bounds__(kTeamBlock<T>) void k_beam_scan(uint64_t x, uint64_t scores_, uint64_t ended_,
                                                             uint64_t scratch, uint32_t stride,
                                                             uint32_t slices, float scale) {
    constexpr int kTeams = kTeamsPerBlock<T>;
    constexpr int U = kUnroll<Fmt, true>;
    __shared__ float sh[T / kWave][kShared];
    __shared__ TopLds<T, kSegs<T>> lds[kTeams];
    const uint32_t cols = tags(x, scores_), parts = tag(ended_), k = tag(scratch);
    const uint32_t team = team_of<T>();
    const uint32_t at = blockIdx.x * kTeams + team;
    const int lane = lane_of<T>();
    if (at >= slices) return;  // whole teams, and never one of several wavefronts
    const uint32_t r = at / parts, b = at - r * parts;
    const uint8_t* ended = addr<const uint8_t>(ended_);
    if (!alive(addr<const float>(scores_)[r]) || (ended != nullptr && ended[r] != 0)) return;
    const RowSpan<Fmt> sp(row_ptr<Fmt>(addr<const void>(x), r, stride), cols);
    const uint32_t n = part_vecs(span_max<Fmt>(cols), parts);
    uint32_t first = sp.va + b * n;
    first = first < sp.vb ? first : sp.vb;
    const uint32_t last = sp.vb - first < n ? sp.vb : first + n;
    auto& L = lds[team];
    const Segments g = Segments::cut<T, U>(first, last, kSegs<T>);
    Stat a;
    scan_span<Fmt, true, T, U, true>(sp, b == 0, first, last, lane, scale, a, g, L.seg);
    team_merge<true, T>(a, scale, lane, sh);
    Slice* slice = addr<Slice>(scratch) + at;
    uint64_t* list = reinterpret_cast<uint64_t*>(addr<Slice>(scratch) + slices) + static_cast<size_t>(at) * k;
    uint32_t count = 0;
    if (a.s > 0.0f) {  // not only masked logits, and neither NaN nor +inf
        top_select<Fmt, T, kSegs<T>>(L, sp, g.count(), g.lg_vecs, k, lane,
                                     [&](uint32_t s, uint32_t i) { return g.vec(s, i); }, b == 0);
        count = L.count;
        if (static_cast<uint32_t>(lane) < count) list[lane] = L.buf[lane];
    }
    if (lane == 0) *slice = Slice{a.m, a.s, a.h, count};
}

// ---------------------------------------------------------------------------------------
// A slice that its workgroup holds in registers: the best of each wavefront by itself, then of the four.

constexpr int kSliceWaves = kSliceThreads / kWave;
constexpr int kWaveCap = 256;  // keys that a wavefront collects
static_assert(kWaveCap >= kBeamMax, "the k best fit");

// Lanes before this one in a mask.
__device__ inline uint32_t below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// Keys of a wavefront's elements, the k best among them, in buf; returns their number. q: vectors of
// one lane, element 0 of vector u at position pos + u * step; lane_max: the lane's maximum.
//
// A bound that k to 2 k of the 64 lanes' maxima reach (bisection by lane masks) bounds the k-th best
// element from below; what reaches it is collected, each lane's at an offset of its own (a ballot and a
// branch per element took 3600 cycles for 32 of them, this 1100). Where ties or a mask put more there than
// buf holds, the k best are taken one by one.
template <typename Fmt, int NV>
__device__ inline uint32_t wave_best(const typename Fmt::Vec (&q)[NV], uint32_t pos, uint32_t step,
                                     float lane_max, uint32_t k, uint64_t* buf, int lane) {
    constexpr int VW = Fmt::VW;
    const uint32_t o[1] = {lane_max >= kLowest ? order_of(lane_max) >> kLowBits<Fmt> : 0};
    float tau = kLowest;
    if (static_cast<uint32_t>(__popcll(__ballot(o[0] != 0))) >= k) {
        const uint32_t bound = bisect(o, k, 2 * k) << kLowBits<Fmt>;
        tau = bound > order_of(kLowest) ? value_of(bound) : kLowest;
    }
    uint32_t hits = 0;
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float e[VW];
        Fmt::unpack(q[u], e);
#pragma unroll
        for (int i = 0; i < VW; ++i) hits += e[i] >= tau ? 1 : 0;
    }
    uint32_t at = hits;  // those of this lane and the lanes before it
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const uint32_t other = __shfl_up(at, off);
        at += lane >= off ? other : 0;
    }
    const uint32_t n = __builtin_amdgcn_readlane(at, kWave - 1);
    if (n <= kWaveCap) {
        at -= hits;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float e[VW];
            Fmt::unpack(q[u], e);
#pragma unroll
            for (int i = 0; i < VW; ++i)
                if (e[i] >= tau) buf[at++] = key_of(e[i], pos + u * step + i);
        }
        return n;
    }
    uint64_t last = ~uint64_t{0};
    uint32_t taken = 0;
    for (; taken < k; ++taken) {
        uint64_t best = 0;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float e[VW];
            Fmt::unpack(q[u], e);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const uint64_t key = e[i] >= kLowest ? key_of(e[i], pos + u * step + i) : 0;
                best = key < last && key > best ? key : best;
            }
        }
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const uint64_t other = __shfl_xor(static_cast<unsigned long long>(best), off);
            best = other > best ? other : best;
        }
        if (best == 0) break;
        if (lane == 0) buf[taken] = best;
        last = best;
    }
    return taken;
}

// One slice of up to NV vectors per lane. Tags as k_beam_scan's.
template <typename Fmt, int NV>
__global__ __launch_bounds__(kSliceThreads) void k_beam_slice(uint64_t x, uint64_t scores_, uint64_t ended_,
                                                              uint64_t scratch, uint32_t stride,
                                                              uint32_t slices, float scale) {
    constexpr int VW = Fmt::VW;
    __shared__ uint64_t s_buf[kSliceWaves][kWaveCap];
    __shared__ Stat s_stat[kSliceWaves];
    __shared__ uint32_t s_count[kSliceWaves];
    const uint32_t cols = tags(x, scores_), parts = tag(ended_), k = tag(scratch);
    const uint32_t at = blockIdx.x;
    const int tid = threadIdx.x, lane = tid % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const uint32_t r = at / parts, b = at - r * parts;
    const uint8_t* ended = addr<const uint8_t>(ended_);
    if (!alive(addr<const float>(scores_)[r]) || (ended != nullptr && ended[r] != 0)) return;
    const RowSpan<Fmt> sp(row_ptr<Fmt>(addr<const void>(x), r, stride), cols);
    const uint32_t n = part_vecs(span_max<Fmt>(cols), parts);  // the row's last vector is in the last slices
    const uint32_t first = b * n, vecs = sp.vb + (cols % VW ? 1 : 0);
    const uint32_t last = first < vecs ? (vecs - first < n ? vecs : first + n) : first;
    typename Fmt::Vec q[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const uint32_t v = first + tid + u * kSliceThreads;
        q[u] = masked16<Fmt>();
        if (v < last) {
            if (v < sp.vb) {
                q[u] = sp.load_whole(v);
            } else {
                q[u] = sp.load_tail();
            }
        }
    }
    Stat a;
    a.init();
    float most = -__builtin_huge_valf();  // the lane's maximum
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float e[VW];
        Fmt::unpack(q[u], e);
        most = max_f(most, max_of(e));
    }
    a.m = lanes_max<kWave>(max_f(most, kLowest));
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        float e[VW];
        Fmt::unpack(q[u], e);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const float z = (e[i] - a.m) * scale;
            const float p = exp2_f(z);
            a.s += p;
            a.h = fmaf(p, max_f(z, kZFloor), a.h);
        }
    }
    a.s = lanes_sum<kWave>(a.s);
    a.h = lanes_sum<kWave>(a.h);
    uint32_t count = 0;
    if (a.s > 0.0f)
        count = wave_best<Fmt, NV>(q, (first + tid) * VW, kSliceThreads * VW, most, k, s_buf[wave], lane);
    if (lane == 0) {
        s_stat[wave] = a;
        s_count[wave] = count;
    }
    __syncthreads();
    // every thread merges the four statistics; the keys' ranks among all of them
    Stat all = s_stat[0];
    uint32_t total = s_count[0];
#pragma unroll
    for (int w = 1; w < kSliceWaves; ++w) {
        Stat o = s_stat[w];
        const float to = max_f(all.m, o.m);
        all.move<true>(to, scale);
        o.move<true>(to, scale);
        all.s += o.s;
        all.h += o.h;
        total += s_count[w];
    }
    Slice* slice = addr<Slice>(scratch) + at;
    uint64_t* list = reinterpret_cast<uint64_t*>(addr<Slice>(scratch) + slices) + static_cast<size_t>(at) * k;
    const bool ok = all.s > 0.0f;
    for (uint32_t i = tid; ok && i < total; i += kSliceThreads) {
        uint32_t in = i, w = 0;
#pragma unroll
        for (int x = 0; x < kSliceWaves - 1; ++x)
            if (w == static_cast<uint32_t>(x) && in >= s_count[x]) {
                in -= s_count[x];
                ++w;
            }
        const uint64_t key = s_buf[w][in];
        uint32_t rank = 0;
#pragma unroll
        for (int x = 0; x < kSliceWaves; ++x) {
            const uint32_t many = s_count[x];
#pragma unroll 8
            for (uint32_t j = 0; j < many; ++j) rank += s_buf[x][j] > key ? 1 : 0;
        }
        if (rank < k) list[rank] = key;
    }
    if (tid == 0) *slice = Slice{all.m, all.s, all.h, ok ? (total < k ? total : k) : 0};
}

// ---------------------------------------------------------------------------------------
// The join of one group's lists, at most kBeamLists of them, one per thread.

constexpr int kJoinThreads = 256;
static_assert(kJoinThreads >= kBeamLists, "a thread for each list");

// Values in the order of unsigned integers, and back.
__device__ inline uint64_t order64(double v) {
    const uint64_t u = __builtin_bit_cast(uint64_t, v + 0.0);  // -0 -> +0
    return (u >> 63) ? ~u : (u | (uint64_t{1} << 63));
}
__device__ inline double value64(uint64_t o) {
    return __builtin_bit_cast(double, (o >> 63) ? (o & ~(uint64_t{1} << 63)) : ~o);
}

// A candidate: its value, its beam, and its logit and token as a key of key_of. Of equal values the lower
// beam's comes first, and of one beam's that of the larger key: two logits whose difference is lost in
// their values keep their order.
struct Cand {
    uint64_t value, key;  // value 0: none
    uint32_t beam;
    __device__ bool above(const Cand& o) const {  // without branches
        const bool before = (beam < o.beam) | ((beam == o.beam) & (key > o.key));
        return (value > o.value) | ((value == o.value) & before);
    }
};

// Candidates in LDS.
template <int N>
struct CandLds {
    uint64_t value[N], key[N];
    uint8_t beam[N];
    __device__ Cand get(uint32_t i) const { return {value[i], key[i], beam[i]}; }
    __device__ void put(uint32_t i, const Cand& c) {
        value[i] = c.value;
        key[i] = c.key;
        beam[i] = static_cast<uint8_t>(c.beam);
    }
};

constexpr uint16_t kNoList = 0xffff;
constexpr int kCands = kBeamMax * (kBeamMax + 1) / 2;
struct JoinLds {
    double base[kBeamMax];  // S_b - ln s_b, of a row that can be continued
    float m[kBeamMax];
    CandLds<kBeamLists> head;
    uint16_t near[kBeamLists];  // lists whose heads can be among the width best
    uint16_t entries[kBeamLists];
    uint16_t list[kBeamMax];    // of the r-th best head
    uint32_t close;
    // What can be among the width best: entry j of the list whose head is the r-th best where r + j < width.
    CandLds<kCands> cand;
    uint32_t count;
};

__device__ inline double lanes_sum64(double v) {
#pragma unroll
    for (int o = 1; o < kWave; o *= 2) v += __shfl_xor(v, o);
    return v;
}

struct JoinArgs {
    const float* scores;   // of the group
    const uint8_t* ended;  // or null
    const Slice* slices;
    const uint64_t* lists;
    uint32_t beams, parts, width, end_token;
    double k, lo;          // log2(e) / T, and ln 2 k_lo / k_hi
};

// Statistics of the rows, a wavefront each; the heads of the lists, one per thread, and their ranks; the
// entries that can be among the best, all at once. Leaves them in L.cand, their number in L.count.
__device__ inline void join(JoinLds& L, const JoinArgs& a) {
    const int tid = threadIdx.x, lane = tid % kWave;
    const double invt = a.k * kLn2d;
    const uint32_t lists = a.beams * a.parts, width = a.width;
    // this thread's list: loaded ahead of the statistics it is judged by
    const bool mine = static_cast<uint32_t>(tid) < lists;
    const uint32_t b_mine = mine ? tid / a.parts : 0;
    const float score_mine = a.scores[b_mine];
    const bool done_mine = a.ended != nullptr && a.ended[b_mine] != 0;
    const bool on = mine && alive(score_mine) && !done_mine;
    uint64_t key = 0;
    uint32_t entries = 0;
    if (on) {
        entries = a.slices[tid].count;
        key = a.lists[static_cast<size_t>(tid) * width];
    }
    for (uint32_t b = tid / kWave; b < a.beams; b += kJoinThreads / kWave) {
        const float score = a.scores[b];
        double base = -__builtin_huge_val();
        float m = kLowest;
        if (alive(score) && !(a.ended != nullptr && a.ended[b] != 0)) {
            const Slice* p = a.slices + b * a.parts;
            Slice s[kBeamLists / kWave];
#pragma unroll
            for (int i = 0; i < kBeamLists / kWave; ++i) {
                s[i] = Slice{kLowest, 0.0f, 0.0f, 0};
                if (lane + i * kWave < a.parts) s[i] = p[lane + i * kWave];
                m = max_f(m, s[i].m);
            }
            m = lanes_max<kWave>(m);
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < kBeamLists / kWave; ++i)
                if (static_cast<uint32_t>(i) * kWave < a.parts)
                    sum += (static_cast<double>(s[i].s) + a.lo * static_cast<double>(s[i].h)) *
                           exp2((static_cast<double>(s[i].m) - static_cast<double>(m)) * a.k);
            sum = lanes_sum64(sum);
            if (sum > 0.0) base = static_cast<double>(score) - log(sum);
        }
        if (lane == 0) {
            L.base[b] = base;
            L.m[b] = m;
        }
    }
    if (tid == 0) L.count = 0;
    if (tid < kBeamMax) L.list[tid] = kNoList;
    __syncthreads();
    const auto candidate = [&](uint32_t b, uint64_t k) {
        float v;
        uint32_t i;
        Key32<kMax>::split(k, v, i);
        const double value = L.base[b] + (static_cast<double>(v) - static_cast<double>(L.m[b])) * invt;
        return Cand{order64(value), k, b};
    };
    Cand head{0, 0, 0};
    if (on) {
        if (L.base[b_mine] > -__builtin_huge_val() && entries > 0) head = candidate(b_mine, key);
    } else if (mine && done_mine && alive(score_mine) && tid % a.parts == 0) {  // goes on as it is
        head = Cand{order64(static_cast<double>(score_mine)), key_of(0.0f, a.end_token), b_mine};
        entries = 1;
    }
    if (tid < kBeamLists) {
        L.head.put(tid, head);
        L.entries[tid] = static_cast<uint16_t>(entries);
    }
    __syncthreads();
    // One wavefront finds a bound that the width best heads reach, and few more (by the upper words of the
    // values); the others wait. Ranks among all heads took 25 us with 256 of them.
    if (tid < kWave) {
        constexpr int kPer = kBeamLists / kWave;
        uint32_t o[kPer], some = 0, bound = 0, n = 0;
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            o[i] = static_cast<uint32_t>(L.head.value[tid + i * kWave] >> 32);
            some += __popcll(__ballot(o[i] != 0));
        }
        if (some > width) bound = bisect(o, width);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool in = o[i] != 0 && o[i] >= bound;
            const uint64_t mask = __ballot(in);
            if (in) L.near[n + below(mask)] = static_cast<uint16_t>(tid + i * kWave);
            n += __popcll(mask);
        }
        if (tid == 0) L.close = n;
    }
    __syncthreads();
    const uint32_t close = L.close;
    if (static_cast<uint32_t>(tid) < close) {
        const uint32_t list = L.near[tid];
        const Cand c = L.head.get(list);
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t i = 0; i < close; ++i) rank += L.head.get(L.near[i]).above(c) ? 1 : 0;
        if (rank < width) L.list[rank] = static_cast<uint16_t>(list);
    }
    __syncthreads();
    const uint64_t least = L.list[width - 1] != kNoList ? L.head.value[L.list[width - 1]] : 0;
    for (uint32_t i = tid; i < width * width; i += kJoinThreads) {
        const uint32_t r = i / width, j = i - r * width, list = L.list[r];
        if (r + j >= width || list == kNoList || j >= L.entries[list]) continue;
        Cand c = L.head.get(list);
        if (j > 0) c = candidate(c.beam, a.lists[static_cast<size_t>(list) * width + j]);
        if (c.value >= least) L.cand.put(atomicAdd(&L.count, 1u), c);
    }
    __syncthreads();
}

// Outputs of all groups, one after another: parents, tokens (int64), scores (float), ended (bytes).
struct BeamOut {
    int64_t *parents, *tokens;
    float* scores;
    uint8_t* ended;
    __device__ BeamOut(uint8_t* out, uint32_t groups, uint32_t width) {
        const size_t n = static_cast<size_t>(groups) * width;
        parents = reinterpret_cast<int64_t*>(out);
        tokens = parents + n;
        scores = reinterpret_cast<float*>(tokens + n);
        ended = reinterpret_cast<uint8_t*>(scores + n);
    }
    __device__ void put(size_t at, int64_t parent, int64_t token, float score, bool end) const {
        parents[at] = parent;
        tokens[at] = token;
        scores[at] = score;
        ended[at] = end ? 1 : 0;
    }
};

constexpr uint32_t kNoEnd = 0xffffffffu;

// Tags: beams in scores, slices per row in ended, width in scratch, the low part of k (bf16) in out.
__global__ __launch_bounds__(kJoinThreads) void k_beam_join(uint64_t scores, uint64_t ended, uint64_t scratch,
                                                            uint64_t out, uint32_t end_token, float k_hi,
                                                            uint32_t groups) {
    __shared__ JoinLds L;
    const uint32_t g = blockIdx.x, width = tag(scratch);
    const int tid = threadIdx.x;
    JoinArgs a;
    a.beams = tag(scores);
    a.parts = tag(ended);
    a.width = width;
    a.end_token = end_token;
    const size_t lists = static_cast<size_t>(a.beams) * a.parts;
    a.scores = addr<const float>(scores) + static_cast<size_t>(g) * a.beams;
    a.ended = addr<const uint8_t>(ended);
    if (a.ended != nullptr) a.ended += static_cast<size_t>(g) * a.beams;
    a.slices = addr<const Slice>(scratch) + g * lists;
    a.lists = reinterpret_cast<const uint64_t*>(addr<const Slice>(scratch) + groups * lists) + g * lists * width;
    const double hi = k_hi, lo = __uint_as_float(tag(out) << 16);
    a.k = hi + lo;
    a.lo = kLn2d * lo / hi;
    join(L, a);
    const BeamOut o(addr<uint8_t>(out), groups, width);
    const uint32_t n = L.count;
    for (uint32_t i = tid; i < n; i += kJoinThreads) {
        const Cand c = L.cand.get(i);
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t j = 0; j < n; ++j) rank += L.cand.get(j).above(c) ? 1 : 0;
        if (rank < width) {
            const uint32_t token = ~static_cast<uint32_t>(c.key);
            o.put(static_cast<size_t>(g) * width + rank, c.beam, token, static_cast<float>(value64(c.value)),
                  end_token != kNoEnd && token == end_token);
        }
    }
    if (static_cast<uint32_t>(tid) < width && static_cast<uint32_t>(tid) >= n)
        o.put(static_cast<size_t>(g) * width + tid, -1, -1, -__builtin_huge_valf(), false);
}

// ---------------------------------------------------------------------------------------
// Reordering, in place. A lane owns the same 16 bytes of all beams of a group: it loads them from
// the parents of the beams that move, all of them before it stores the first, and no other lane
// touches them, so nothing has to be set aside. Beams that stay are neither read nor written.

template <typename V>
struct __attribute__((packed, aligned(1))) Anywhere {
    V v;
};
template <typename V>
__device__ inline V load_any(const uint8_t* p) {
    return reinterpret_cast<const Anywhere<V>*>(p)->v;
}
template <typename V>
__device__ inline void store_any(uint8_t* p, V v) {
    reinterpret_cast<Anywhere<V>*>(p)->v = v;
}

// Moves one unit of up to NB beams. move[j]: source beam, and destination << 16; scalars.
template <typename V, int NB>
__device__ inline void move_unit(uint8_t* at, const uint32_t (&move)[NB], int n, int64_t beam_stride) {
    V v[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        if (j < n) v[j] = load_any<V>(at + (move[j] & 0xffffu) * beam_stride);
#pragma unroll
    for (int j = 0; j < NB; ++j)
        if (j < n) store_any<V>(at + (move[j] >> 16) * beam_stride, v[j]);
}

// Tags: beams in parents, workgroups per tensor and group in last.
template <typename V, int NB>
__global__ __launch_bounds__(kBlockThreads) void k_reorder(uint64_t table, uint64_t parents_, uint64_t first_,
                                                           uint64_t last_, uint32_t first_value,
                                                           uint32_t last_value, uint32_t groups) {
    __shared__ uint32_t s_move[NB];
    __shared__ int s_n;
    const uint32_t beams = tag(parents_), blocks = tag(last_);
    const uint32_t pair = blockIdx.x / blocks, block = blockIdx.x - pair * blocks;
    const uint32_t t = pair / groups, g = pair - t * groups;
    const argreduce_state_t s = addr<const argreduce_state_t>(table)[t];
    const int64_t* firsts = addr<const int64_t>(first_);
    const int64_t* lasts = addr<const int64_t>(last_);
    int64_t first = firsts != nullptr ? firsts[g] : first_value;
    int64_t last = lasts != nullptr ? lasts[g] : last_value;
    first = first < 0 ? 0 : first;
    last = last > s.positions ? s.positions : last;
    if (first >= last) return;
    if (threadIdx.x < kWave) {  // the beams that move, in order
        const uint32_t b = threadIdx.x;
        int64_t p = b < beams ? addr<const int64_t>(parents_)[static_cast<size_t>(g) * beams + b] : -1;
        const bool moves = p >= 0 && p < static_cast<int64_t>(beams) && p != static_cast<int64_t>(b);
        const uint64_t mask = __ballot(moves);
        if (moves) {
            const int at = __popcll(mask & ((uint64_t{1} << b) - 1));
            s_move[at] = static_cast<uint32_t>(p) | b << 16;
        }
        if (b == 0) s_n = __popcll(mask);
    }
    __syncthreads();
    const int n = __builtin_amdgcn_readfirstlane(s_n);
    if (n == 0) return;
    uint32_t move[NB];
#pragma unroll
    for (int j = 0; j < NB; ++j) move[j] = __builtin_amdgcn_readfirstlane(j < n ? s_move[j] : 0);
    // The widest access that every address of the state allows, for what a run has past its last unit.
    const uint64_t all = reinterpret_cast<uint64_t>(s.base) | s.group_stride | s.beam_stride |
                         s.outer_stride | s.position_stride | s.inner;
    const int grain = all & 1 ? 1 : all & 2 ? 2 : all & 4 ? 4 : 8;
    // The group's positions as `segments` runs of `bytes` contiguous bytes.
    uint8_t* base = reinterpret_cast<uint8_t*>(s.base) + g * s.group_stride + first * s.position_stride;
    uint32_t per = static_cast<uint32_t>(last - first);  // segments of one `outer`
    int64_t bytes = s.inner;
    if (s.position_stride == s.inner) {
        bytes *= per;
        per = 1;
    }
    const uint32_t segments = static_cast<uint32_t>(s.outer) * per;
    constexpr uint32_t kUnit = sizeof(V);
    const uint32_t units = static_cast<uint32_t>((bytes + kUnit - 1) / kUnit), total = segments * units;
    for (uint32_t i = block * kBlockThreads + threadIdx.x; i < total; i += blocks * kBlockThreads) {
        const uint32_t seg = i / units, u = i - seg * units;
        const uint32_t o = seg / per, pos = seg - o * per;
        uint8_t* at = base + o * s.outer_stride + pos * s.position_stride + static_cast<int64_t>(u) * kUnit;
        const int64_t left = bytes - static_cast<int64_t>(u) * kUnit;
        if (left >= kUnit) {
            move_unit<V, NB>(at, move, n, s.beam_stride);
        } else {
            for (int64_t e = 0; e < left; e += grain) {
                if (grain == 1)
                    move_unit<uint8_t, NB>(at + e, move, n, s.beam_stride);
                else if (grain == 2)
                    move_unit<uint16_t, NB>(at + e, move, n, s.beam_stride);
                else if (grain == 4)
                    move_unit<uint32_t, NB>(at + e, move, n, s.beam_stride);
                else
                    move_unit<uint64_t, NB>(at + e, move, n, s.beam_stride);
            }
        }
    }
}

}  // namespace

size_t beam_list_bytes(int width) { return sizeof(Slice) + static_cast<size_t>(width) * sizeof(uint64_t); }

hipError_t launch_beam_step(const BeamPlan& plan, const BeamArgs& a, uint8_t* scratch16, hipStream_t s) {
    const uint32_t cols = static_cast<uint32_t>(a.cols), groups = static_cast<uint32_t>(a.groups);
    const uint32_t slices = groups * static_cast<uint32_t>(a.beams * plan.parts);
    const double k = 1.4426950408889634074 / a.temperature;
    const float hi = static_cast<float>(k);
    // the rest of k to 8 bits: k is then good to 2^-33 of itself
    const float rest = static_cast<float>(k - static_cast<double>(hi));
    const uint32_t low = (bits_of(rest) + 0x8000u) >> 16;
    const auto scan = [&](auto fmt, auto team) {
        constexpr int T = decltype(team)::value;
        launch(k_beam_scan<decltype(fmt), T>, static_cast<uint32_t>(plan.grid_blocks), kTeamBlock<T>, s,
               tagged(a.x, cols), tagged(a.scores, cols >> 16), tagged(a.ended, plan.parts),
               tagged(scratch16, a.width), static_cast<uint32_t>(a.row_stride), slices, hi);
    };
    const auto slice = [&](auto fmt, auto held) {
        launch(k_beam_slice<decltype(fmt), decltype(held)::value>, slices, kSliceThreads, s, tagged(a.x, cols),
               tagged(a.scores, cols >> 16), tagged(a.ended, plan.parts), tagged(scratch16, a.width),
               static_cast<uint32_t>(a.row_stride), slices, hi);
    };
    with_format(a.dtype, [&](auto fmt) {
        switch (plan.held) {
            case 1: return slice(fmt, Int<1>{});
            case 2: return slice(fmt, Int<2>{});
            case 4: return slice(fmt, Int<4>{});
            case 8: return slice(fmt, Int<8>{});
        }
        switch (plan.team) {
            case 64: scan(fmt, Int<64>{}); break;
            case 256: scan(fmt, Int<256>{}); break;
            case 512: scan(fmt, Int<512>{}); break;
            default: scan(fmt, Int<1024>{}); break;
        }
    });
    const uint32_t end = a.end_token < 0 ? kNoEnd : static_cast<uint32_t>(a.end_token);
    launch(k_beam_join, groups, kJoinThreads, s, tagged(a.scores, a.beams), tagged(a.ended, plan.parts),
           tagged(scratch16, a.width), tagged(a.out, low), end, hi, groups);
    return hipGetLastError();
}

hipError_t launch_reorder(const ReorderArgs& a, hipStream_t s) {
    const uint32_t groups = static_cast<uint32_t>(a.groups);
    const uint32_t grid = static_cast<uint32_t>(a.tensors) * groups * static_cast<uint32_t>(a.blocks);
    const auto go = [&](auto kernel) {
        launch(kernel, grid, kBlockThreads, s, tagged(a.table, 0), tagged(a.parents, a.beams),
               tagged(a.first, 0), tagged(a.last, a.blocks), static_cast<uint32_t>(a.first_value),
               static_cast<uint32_t>(a.last_value), groups);
    };
    if (a.beams <= 4)
        go(k_reorder<u32x4, 4>);
    else if (a.beams <= 8)
        go(k_reorder<u32x4, 8>);
    else if (a.beams <= 16)
        go(k_reorder<u32x4, 16>);
    else if (a.beams <= 32)
        go(k_reorder<u32x4, 32>);
    else
        go(k_reorder<uint64_t, 64>);
    return hipGetLastError();
}

}  // namespace argreduce
