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
// other as they like: everything after the slices' sums is in binary64, and what would be off alike for
// all terms of a row, and so does not average out, is taken out of the sums:
//   * 2^(d k) with k rounded to binary32 (k_hi) lacks the factor 2^(d k_lo) = 1 + ln 2 d k_lo:
//     with h = sum 2^z z, z = d k_hi, the sum is s + ln 2 (k_lo / k_hi) h;
//   * the logarithm is binary64's.
// What is left is the rounding of the terms and of the sums, binary32's, of lanes, of wavefronts and of a slice: about
// 1e-7 of s (N(0, 2.5^2) logits: root of the mean square 0.3e-7 to 0.6e-7 where slices are held in registers, 0.8e-7 to
// 1.0e-7 in one pass, the largest of 10000 rows 1.0e-6). Equal rows have equal sums wherever they lie (RowSpan), so that
// equal continuations of different beams tie.
#include <hip/hip_runtime.h>

#include "argreduce_beam.hpp"
#include "argreduce_launch.hpp"
#include "argreduce_logits_device.hpp"

#pragma clang fp contract(off)

namespace argreduce {
namespace {

constexpr double kLn2d = 0.693147180559945309417;

__device__ inline bool alive(float score) { return score > -__builtin_huge_valf() && score < __builtin_huge_valf(); }

// The sum over groups of 2^lg lanes, lg <= 4 and the same in all lanes.
__device__ inline uint32_t lanes_sum_u32(uint32_t v, uint32_t lg) {
    if (lg >= 1) v += dpp_u32<0xB1, 0xf>(v);
    if (lg >= 2) v += dpp_u32<0x4E, 0xf>(v);
    if (lg >= 3) v += dpp_u32<0x141, 0xf>(v);
    if (lg >= 4) v += dpp_u32<0x140, 0xf>(v);
    return v;
}

// Lanes before this one in a mask.
__device__ inline uint32_t below(uint64_t mask) {
    return __builtin_amdgcn_mbcnt_hi(static_cast<uint32_t>(mask >> 32),
                                     __builtin_amdgcn_mbcnt_lo(static_cast<uint32_t>(mask), 0));
}

// ---------------------------------------------------------------------------------------
// The join of one group's lists, at most kBeamLists of them.

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
struct JoinLds {
    double base[kBeamMax];  // S_b - ln s_b, of a row that can be continued
    float m[kBeamMax];
    CandLds<kBeamLists> head;
    uint16_t near[kBeamLists];  // lists whose heads can be among the width best
    uint16_t entries[kBeamLists];
    uint16_t list[kBeamMax];    // of the r-th best head
    uint32_t least[kSliceThreads / kWave];  // of each wavefront's candidates
    uint32_t close, bound, count, picked;
};
// What can be among the width best, at most entry j of the list whose head is the r-th best where r + j < width: in LDS
// that the launch sizes (beam_cands).
__host__ __device__ inline uint32_t beam_room(uint32_t width) {
    const uint32_t most = width * (width + 1) / 2;
    return most < 64 ? 64 : most;
}
struct Cands {
    uint64_t *value, *key;
    uint16_t* picked;  // numbers of those that are ranked
    uint8_t* beam;
    __device__ Cands(uint64_t* lds, uint32_t width) {
        const uint32_t n = beam_room(width);
        value = lds;
        key = lds + n;
        picked = reinterpret_cast<uint16_t*>(lds + 2 * n);
        beam = reinterpret_cast<uint8_t*>(picked + n);
    }
    __device__ Cand get(uint32_t i) const { return {value[i], key[i], beam[i]}; }
    __device__ void put(uint32_t i, const Cand& c) const {
        value[i] = c.value;
        key[i] = c.key;
        beam[i] = static_cast<uint8_t>(c.beam);
    }
};
inline size_t beam_cands(uint32_t width) { return static_cast<size_t>(beam_room(width)) * 19; }

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
    __device__ void put(size_t at, const Cand& c, uint32_t end_token) const {
        const uint32_t token = ~static_cast<uint32_t>(c.key);
        put(at, c.beam, token, static_cast<float>(value64(c.value)), token == end_token);
    }
    __device__ void none(size_t at) const { put(at, -1, -1, -__builtin_huge_valf(), false); }
};
constexpr uint32_t kNoEnd = 0xffffffffu;  // no token's number

// What is alike for all rows: k = log2(e) / T in two parts, and what follows from it.
struct Scale {
    double k, lo, invt;  // k, ln 2 k_lo / k_hi, 1 / T
    __device__ Scale(float hi, uint32_t low) {  // low: the upper half of the low part's bits
        const double l = __uint_as_float(low << 16);
        k = static_cast<double>(hi) + l;
        lo = kLn2d * l / static_cast<double>(hi);
        invt = k * kLn2d;
    }
    // S_b - ln s_b of a row whose sums are s and h; -inf if the row has nothing to offer (s 0 or NaN).
    __device__ double base(float score, double s) const {
        return s > 0.0 ? static_cast<double>(score) - log(s) : -__builtin_huge_val();
    }
    __device__ Cand candidate(double base, float m, uint32_t b, uint64_t key) const {
        float v;
        uint32_t i;
        Key32<kMax>::split(key, v, i);
        return {order64(base + (static_cast<double>(v) - static_cast<double>(m)) * invt), key, b};
    }
};
__device__ inline Cand finished(float score, uint32_t b, uint32_t end_token) {
    return {order64(static_cast<double>(score)), key_of(0.0f, end_token), b};
}

// Scratch: an owner for every group (in 16 bytes), a slot for every slice (arrive), slices, lists.
struct Scratch {
    uint64_t *owner, *slots;   // of the group
    uint64_t *slices, *lists;  // of the group: two words, and width words each
    static size_t bytes(int64_t groups, int64_t lists, int width) {
        return 8 * static_cast<size_t>(groups) * (2 + static_cast<size_t>(lists) * (3 + width));
    }
    __device__ Scratch(uint8_t* p, uint32_t groups, uint32_t g, uint32_t lists_, uint32_t width) {
        uint64_t* w = reinterpret_cast<uint64_t*>(p);
        const size_t all = static_cast<size_t>(groups) * lists_, mine = static_cast<size_t>(g) * lists_;
        owner = w + 2 * static_cast<size_t>(g);
        slots = w + 2 * static_cast<size_t>(groups) + mine;
        slices = w + 2 * static_cast<size_t>(groups) + all + 2 * mine;
        lists = w + 2 * static_cast<size_t>(groups) + 3 * all + mine * width;
    }
};
__device__ inline uint64_t two(float a, uint32_t b) { return static_cast<uint64_t>(b) << 32 | __float_as_uint(a); }
__device__ inline float low_of(uint64_t w) { return __uint_as_float(static_cast<uint32_t>(w)); }
__device__ inline uint32_t high_of(uint64_t w) { return static_cast<uint32_t>(w >> 32); }

struct Step {
    const float* scores;   // of the group
    const uint8_t* ended;  // or null
    uint32_t g, beams, parts, width, end_token;
    __device__ bool done(uint32_t b) const { return ended != nullptr && ended[b] != 0; }
};

// The best of the group's lists, by a workgroup of T threads: statistics of the rows, a wavefront each; the heads
// of the lists, one per thread, and those that can be among the best; their entries, all at once; ranks.
template <int T>
__device__ inline void join(JoinLds& L, const Cands& cands, const Step& a, const Scratch& w, const Scale& k,
                            const BeamOut& out) {
    const int tid = threadIdx.x;
    const uint32_t lists = a.beams * a.parts, width = a.width;
    // this thread's list: loaded ahead of the statistics it is judged by
    const bool mine = static_cast<uint32_t>(tid) < lists;
    const uint32_t b_mine = mine ? tid / a.parts : 0;
    const float score_mine = a.scores[b_mine];
    const bool done_mine = a.done(b_mine);
    const bool on = mine && alive(score_mine) && !done_mine;
    uint64_t key = 0;
    uint32_t entries = 0;
    if (on) {
        entries = high_of(load_part(w.slices + 2 * tid + 1));
        key = load_part(w.lists + static_cast<size_t>(tid) * width);
    }
    // a row's slices by 16, 32 or 64 lanes, so that few rounds do
    const auto rows = [&](auto lanes) {
        constexpr int G = decltype(lanes)::value, kPer = G == kWave ? kBeamLists / kWave : 1;
        const int at = tid % G;
        for (uint32_t b = tid / G; b < a.beams; b += T / G) {
            const float score = a.scores[b];
            const bool live = alive(score) && !a.done(b);
            const uint64_t* p = w.slices + 2 * static_cast<size_t>(b) * a.parts;
            uint64_t one[kPer];
            float h[kPer], m = kLowest;
#pragma unroll
            for (int i = 0; i < kPer; ++i) {
                one[i] = two(kLowest, 0);
                h[i] = 0.0f;
                if (live && at + i * G < static_cast<int>(a.parts)) {
                    one[i] = load_part(p + 2 * (at + i * G));
                    h[i] = low_of(load_part(p + 2 * (at + i * G) + 1));
                }
            }
#pragma unroll
            for (int i = 0; i < kPer; ++i) m = max_f(m, low_of(one[i]));
            m = lanes_max<G>(m);
            double sum = 0.0;
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                if (i == 0 || static_cast<uint32_t>(i) * G < a.parts)
                    sum += (static_cast<double>(__uint_as_float(high_of(one[i]))) + k.lo * static_cast<double>(h[i])) *
                           exp2((static_cast<double>(low_of(one[i])) - static_cast<double>(m)) * k.k);
            const double base = k.base(score, lanes_sum64<G>(sum));
            if (at == 0) {
                L.base[b] = live ? base : -__builtin_huge_val();
                L.m[b] = m;
            }
        }
    };
    if (a.parts <= 16)
        rows(Int<16>{});
    else if (a.parts <= 32)
        rows(Int<32>{});
    else
        rows(Int<64>{});
    if (tid == 0) L.count = L.picked = 0;
    if (tid < kBeamMax) L.list[tid] = kNoList;
    __syncthreads();
    Cand head{0, 0, 0};
    if (on) {
        if (L.base[b_mine] > -__builtin_huge_val() && entries > 0)
            head = k.candidate(L.base[b_mine], L.m[b_mine], b_mine, key);
    } else if (mine && done_mine && alive(score_mine) && tid % a.parts == 0) {  // goes on as it is
        head = finished(score_mine, b_mine, a.end_token);
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
            o[i] = high_of(L.head.value[tid + i * kWave]);
            some += __popcll(__ballot(o[i] != 0));
        }
        if (some > width) bound = bisect(o, width, width + width / 4 + 1);
#pragma unroll
        for (int i = 0; i < kPer; ++i) {
            const bool in = o[i] != 0 && o[i] >= bound;
            const uint64_t mask = __ballot(in);
            if (in) L.near[n + below(mask)] = static_cast<uint16_t>(tid + i * kWave);
            n += __popcll(mask);
        }
        if (tid == 0) {
            L.close = n;
            L.bound = bound;
        }
    }
    __syncthreads();
    // All entries of those lists that reach the bound; where ties make them too many, those alone that can be among
    // the best by the ranks of the heads: entry j of the list of the r-th best head where r + j < width.
    const uint32_t close = L.close, room = beam_room(width);
    const uint64_t bound = static_cast<uint64_t>(L.bound) << 32;
    const auto entry = [&](uint32_t list, uint32_t j) {
        const Cand c = L.head.get(list);
        return j == 0 ? c : k.candidate(L.base[c.beam], L.m[c.beam], c.beam,
                                        load_part(w.lists + static_cast<size_t>(list) * width + j));
    };
    for (uint32_t i = tid; i < close * width; i += T) {
        const uint32_t r = i / width, j = i - r * width, list = L.near[r];
        if (j >= L.entries[list]) continue;
        const Cand c = entry(list, j);
        if (c.value < bound) continue;
        const uint32_t at = atomicAdd(&L.count, 1u);
        if (at < room) cands.put(at, c);
    }
    __syncthreads();
    if (L.count > room) {
        __syncthreads();
        if (tid == 0) L.count = 0;
        for (uint32_t i = tid; i < close; i += T) {
            const uint32_t list = L.near[i];
            const Cand c = L.head.get(list);
            uint32_t rank = 0;
            for (uint32_t x = 0; x < close; ++x) rank += L.head.get(L.near[x]).above(c) ? 1 : 0;
            if (rank < width) L.list[rank] = static_cast<uint16_t>(list);
        }
        __syncthreads();
        for (uint32_t i = tid; i < width * width; i += T) {
            const uint32_t r = i / width, j = i - r * width, list = L.list[r];
            if (r + j < width && list != kNoList && j < L.entries[list]) cands.put(atomicAdd(&L.count, 1u), entry(list, j));
        }
        __syncthreads();
    }
    // Of many, those are ranked that reach the smallest of the bounds that an even share of the width best reaches
    // among each wavefront's (200 ranked candidates took 20 us).
    const uint32_t all = L.count;
    uint32_t n = all;
    if (all > kWave) {
        constexpr uint32_t kWaves = T / kWave;
        const uint32_t each = (width + kWaves - 1) / kWaves, wave = tid / kWave;
        const auto least = [&](auto words) {
            constexpr int P = decltype(words)::value;
            uint32_t o[P], some = 0;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const uint32_t at = tid % kWave * kWaves + wave + i * T;
                o[i] = at < all ? high_of(cands.value[at]) : 0;
                some += __popcll(__ballot(o[i] != 0));
            }
            return some < each ? 0 : bisect(o, each, each + each / 4 + 1);
        };
        constexpr uint32_t kMost = kBeamMax * (kBeamMax + 1) / 2;
        const uint32_t mine = all <= T ? least(Int<1>{}) : least(Int<(kMost + T - 1) / T>{});
        if (tid % kWave == 0) L.least[wave] = mine;
        __syncthreads();
        uint32_t enough = L.least[0];
#pragma unroll
        for (uint32_t i = 1; i < kWaves; ++i) enough = L.least[i] < enough ? L.least[i] : enough;
        for (uint32_t i = tid; i < all; i += T)
            if (high_of(cands.value[i]) >= enough) cands.picked[atomicAdd(&L.picked, 1u)] = static_cast<uint16_t>(i);
        __syncthreads();
        n = L.picked;
    }
    const auto ranked = [&](uint32_t i) { return cands.get(all > kWave ? cands.picked[i] : i); };
    // ranks: several lanes count for a candidate, each over its share of the others
    const size_t first = static_cast<size_t>(a.g) * width;
    const uint32_t lg = n <= T / 16 ? 4 : n <= T / 8 ? 3 : n <= T / 4 ? 2 : n <= T / 2 ? 1 : 0;
    for (uint32_t i = tid >> lg; i < n; i += T >> lg) {
        const Cand c = ranked(i);
        uint32_t rank = 0;
#pragma unroll 2
        for (uint32_t j = tid & ((1u << lg) - 1); j < n; j += 1u << lg) rank += ranked(j).above(c) ? 1 : 0;
        rank = lanes_sum_u32(rank, lg);
        if ((tid & ((1u << lg) - 1)) == 0 && rank < width) out.put(first + rank, c, a.end_token);
    }
    if (static_cast<uint32_t>(tid) < width && static_cast<uint32_t>(tid) >= n) out.none(first + tid);
}

// What the kernels over slices have in common. Tags: columns in (x, scores), beams - 1 and slices per row - 1 (8 bits
// each) in ended, width in scratch, the low part of k in out.
struct SliceJob {
    uint32_t cols, parts, width, row, part, at, beams, groups;
    Step step;
    __device__ SliceJob(uint64_t x, uint64_t scores, uint64_t ended, uint64_t scratch, uint32_t end_token) {
        cols = tags(x, scores);
        beams = (tag(ended) >> 8) + 1;
        parts = (tag(ended) & 0xffu) + 1;
        width = tag(scratch);
        at = blockIdx.x;
        row = at / parts;
        part = at - row * parts;
        groups = gridDim.x / (beams * parts);
        const uint32_t g = row / beams;
        const uint8_t* e = addr<const uint8_t>(ended);
        step = {addr<const float>(scores) + static_cast<size_t>(g) * beams,
                e == nullptr ? e : e + static_cast<size_t>(g) * beams, g, beams, parts, width, end_token};
    }
    __device__ uint32_t beam() const { return row - step.g * beams; }
    __device__ bool on() const { return alive(step.scores[beam()]) && !step.done(beam()); }
    // This slice's number in its group.
    __device__ uint32_t list() const { return at - step.g * beams * parts; }
};

// After a slice's words are stored: the group's last workgroup joins its lists.
template <int T>
__device__ inline void join_if_last(JoinLds& L, uint64_t* cands, uint32_t* found, const SliceJob& j, const Scratch& w,
                                    uint32_t nonce, float k_hi, uint64_t out) {
    if (!arrive(w.slots, w.owner, j.list(), j.beams * j.parts, arrival_tag(nonce), found)) return;
    join<T>(L, Cands(cands, j.width), j.step, w, Scale(k_hi, tag(out)), BeamOut(addr<uint8_t>(out), j.groups, j.width));
    leave<T>(w.slots, j.beams * j.parts);
}

// One slice of a row per workgroup, in one pass; the join is a launch of its own (its registers would halve the
// wavefronts of a CU: [256,8,128256] bf16 131 us with it, 92 and 6 apart, 5.7 TB/s). Arithmetic bounds it as much as
// the read: 14 vector instructions' time per logit, four of them the exponential's.
template <typename Fmt, int T>
__global__ __launch_bounds__(T) void k_beam_scan(uint64_t x, uint64_t scores, uint64_t ended, uint64_t scratch,
                                                 uint32_t stride, float k_hi) {
    constexpr int U = kUnroll<Fmt, true>;
    __shared__ float sh[T / kWave][kShared];
    __shared__ TopLds<T, kSegs<T>> L;
    const SliceJob j(x, scores, ended, scratch, kNoEnd);
    const Scratch w(addr<uint8_t>(scratch), j.groups, j.step.g, j.beams * j.parts, j.width);
    const int lane = threadIdx.x;
    if (!j.on()) return;
    const RowSpan<Fmt> sp(row_ptr<Fmt>(addr<const void>(x), j.row, stride), j.cols);
    const uint32_t n = part_vecs(span_max<Fmt>(j.cols), j.parts);
    uint32_t first = sp.va + j.part * n;
    first = first < sp.vb ? first : sp.vb;
    const uint32_t last = sp.vb - first < n ? sp.vb : first + n;
    const Segments g = Segments::cut<T, U>(first, last, kSegs<T>);
    Stat a;
    scan_span<Fmt, true, T, U, true>(sp, j.part == 0, first, last, lane, k_hi, a, g, L.seg);
    team_merge<true, T>(a, k_hi, lane, sh);
    uint32_t count = 0;
    if (a.s > 0.0f) {  // not only masked logits, and neither NaN nor +inf
        top_select<Fmt, T, kSegs<T>>(L, sp, g.count(), g.lg_vecs, j.width, lane,
                                     [&](uint32_t s, uint32_t i) { return g.vec(s, i); }, j.part == 0);
        count = L.count;
        if (static_cast<uint32_t>(lane) < count)
            store_part(w.lists + static_cast<size_t>(j.list()) * j.width + lane, L.buf[lane]);
    }
    if (lane == 0) {
        store_part(w.slices + 2 * j.list(), two(a.m, __float_as_uint(a.s)));
        store_part(w.slices + 2 * j.list() + 1, two(a.h, count));
    }
}

// One workgroup per group; 6 us for 256 groups of 8 lists, 15 for 2000 of 12. Tags as SliceJob's, without the columns.
__global__ __launch_bounds__(kSliceThreads) void k_beam_join(uint64_t scores, uint64_t ended, uint64_t scratch,
                                                             uint64_t out, uint32_t end_token, float k_hi) {
    __shared__ JoinLds L;
    extern __shared__ uint64_t s_cands[];
    const uint32_t g = blockIdx.x, beams = (tag(ended) >> 8) + 1, parts = (tag(ended) & 0xffu) + 1, width = tag(scratch);
    const uint8_t* e = addr<const uint8_t>(ended);
    const Step step{addr<const float>(scores) + static_cast<size_t>(g) * beams,
                    e == nullptr ? e : e + static_cast<size_t>(g) * beams, g, beams, parts, width, end_token};
    join<kSliceThreads>(L, Cands(s_cands, width), step, Scratch(addr<uint8_t>(scratch), gridDim.x, g, beams * parts, width),
                        Scale(k_hi, tag(out)), BeamOut(addr<uint8_t>(out), gridDim.x, width));
}

// ---------------------------------------------------------------------------------------
// A slice that its workgroup holds in registers. Its k best elements are at least the smallest of four bounds
// that k / 4 lanes of each wavefront reach; what reaches that, less than 2 k as a rule, is collected and ranked by
// counting. (By a bound for k of each wavefront alone, 16 best of 6300 elements took 9000 cycles more.)

template <int W>
struct SliceLds {
    static constexpr uint32_t kCap = 256;  // keys that a wavefront collects
    static_assert(kCap >= kBeamMax, "the k best of each wavefront fit");
    Stat stat[W];
    uint32_t bound[W], total;
    uint64_t best[W][kBeamMax];
    uint64_t buf[W * kCap];
};

// A vector as the compiler does not know it: what was made of it before is not kept in registers.
template <typename Vec>
__device__ inline Vec anew(Vec v) {
    asm volatile("" : "+v"(v));
    return v;
}

// A bound that at least k (and few more) of the wavefront's 64 lane maxima reach, by bisection; -inf if there
// are fewer than k. As an ordered integer: 0 for -inf.
template <typename Fmt>
__device__ inline uint32_t wave_bound(float lane_max, uint32_t k) {
    const uint32_t o[1] = {lane_max >= kLowest ? order_of(lane_max) >> kLowBits<Fmt> : 0};
    if (static_cast<uint32_t>(__popcll(__ballot(o[0] != 0))) < k) return 0;
    return bisect(o, k, k + k / 4 + 1);
}

// Word i of N (a power of two) in registers.
template <int N>
__device__ __forceinline__ uint32_t pick(const uint32_t (&w)[N], uint32_t i) {
    if constexpr (N == 1) {
        return w[0];
    } else {
        uint32_t half[N / 2];
        const uint32_t upper = 0u - (i / (N / 2) & 1u);  // (a choice by ?: would put w into memory)
#pragma unroll
        for (int j = 0; j < N / 2; ++j) half[j] = (w[j + N / 2] & upper) | (w[j] & ~upper);
        return pick(half, i);
    }
}

// Which of a lane's elements are at least tau, as masks of 32; and their keys, one per lane and round (a ballot and
// a branch per element took 3600 cycles for 32 of them).
template <typename Fmt, int NV>
struct Hits {
    static constexpr int kElems = NV * Fmt::VW, kMasks = (kElems + 31) / 32;
    uint32_t mask[kMasks];
    uint32_t count;
    __device__ Hits(const typename Fmt::Vec (&q)[NV], float tau) {
        count = 0;
#pragma unroll
        for (int m = 0; m < kMasks; ++m) mask[m] = 0;
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float e[Fmt::VW];
            Fmt::unpack(anew(q[u]), e);
#pragma unroll
            for (int i = 0; i < Fmt::VW; ++i) {
                const int at = u * Fmt::VW + i;
                mask[at / 32] |= e[i] >= tau ? 1u << (at % 32) : 0;
            }
        }
#pragma unroll
        for (int m = 0; m < kMasks; ++m) count += __popc(mask[m]);
    }
    // put(key); element 0 of vector u is at position pos + u * step.
    template <typename Put>
    __device__ void each(const typename Fmt::Vec (&q)[NV], uint32_t pos, uint32_t step, Put put) {
        constexpr int kVecs = kElems < 32 ? NV : 32 / Fmt::VW, kWords = 4 * kVecs;  // of a mask's elements
#pragma unroll
        for (int m = 0; m < kMasks; ++m) {
            uint32_t w[kWords];
#pragma unroll
            for (int i = 0; i < kVecs; ++i) {
                const u32x4 v = __builtin_bit_cast(u32x4, q[m * kVecs + i]);
                w[4 * i] = v.x;
                w[4 * i + 1] = v.y;
                w[4 * i + 2] = v.z;
                w[4 * i + 3] = v.w;
            }
            while (__ballot(mask[m] != 0) != 0) {
                const bool some = mask[m] != 0;
                const uint32_t i = some ? __builtin_ctz(mask[m]) : 0;
                mask[m] &= mask[m] - 1;
                constexpr uint32_t kPerWord = 4 / Fmt::kSize;
                const uint32_t word = pick(w, i / kPerWord);
                const float e = Fmt::from_bits(static_cast<typename Fmt::Bits>(word >> (i % kPerWord * 16)));
                const uint32_t at = m * 32 + i;
                if (some) put(key_of(e, pos + at / Fmt::VW * step + at % Fmt::VW));
            }
        }
    }
};

// The k best keys of a wavefront's elements, one by one, best first; returns their number.
template <typename Fmt, int NV>
__device__ inline uint32_t wave_best(const typename Fmt::Vec (&q)[NV], uint32_t pos, uint32_t step, uint32_t k,
                                     uint64_t* buf, int lane) {
    constexpr int VW = Fmt::VW;
    uint64_t last = ~uint64_t{0};
    uint32_t taken = 0;
    for (; taken < k; ++taken) {
        uint64_t best = 0;
        uint32_t from = pos;  // (the keys, too, are made anew in every round)
        asm volatile("" : "+v"(from));
#pragma unroll
        for (int u = 0; u < NV; ++u) {
            float e[VW];
            Fmt::unpack(q[u], e);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const uint64_t key = e[i] >= kLowest ? key_of(e[i], from + u * step + i) : 0;
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

// One slice of up to NV vectors per lane, by W wavefronts.
template <typename Fmt, int NV, int W>
__device__ inline void hold_slice(SliceLds<W>& L, const SliceJob& j, const Scratch& w, uint64_t x, uint32_t stride,
                                  float k_hi) {
    constexpr int VW = Fmt::VW, T = W * kWave;
    const int tid = threadIdx.x, lane = tid % kWave;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const RowSpan<Fmt> sp(row_ptr<Fmt>(addr<const void>(x), j.row, stride), j.cols);
    const uint32_t n = part_vecs(span_max<Fmt>(j.cols), j.parts);  // the row's last vector is in the last slices
    const uint32_t first = j.part * n, vecs = sp.vb + (j.cols % VW ? 1 : 0);
    const uint32_t last = first < vecs ? (vecs - first < n ? vecs : first + n) : first;
    typename Fmt::Vec q[NV];
#pragma unroll
    for (int u = 0; u < NV; ++u) {
        const uint32_t v = first + tid + u * T;
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
        Fmt::unpack(anew(q[u]), e);
#pragma unroll
        for (int i = 0; i < VW; ++i) {
            const float z = (e[i] - a.m) * k_hi;
            const float p = exp2_f(z);
            a.s += p;
            a.h = fmaf(p, max_f(z, kZFloor), a.h);
        }
    }
    a.s = lanes_sum<kWave>(a.s);
    a.h = lanes_sum<kWave>(a.h);
    const uint32_t enough = a.s > 0.0f ? wave_bound<Fmt>(most, (j.width + W - 1) / W) : 0;
    if (lane == 0) {
        L.stat[wave] = a;
        L.bound[wave] = enough;
    }
    if (tid == 0) L.total = 0;
    __syncthreads();
    uint32_t bound = L.bound[0];
#pragma unroll
    for (int w = 1; w < W; ++w) bound = L.bound[w] < bound ? L.bound[w] : bound;
    if (bound == 0) bound = wave_bound<Fmt>(most, j.width);  // a wavefront with next to nothing
    bound <<= kLowBits<Fmt>;
    const float tau = bound > order_of(kLowest) ? value_of(bound) : kLowest;
    const uint32_t pos = (first + tid) * VW;
    // the lanes' hits, and those of the lanes before each
    Hits<Fmt, NV> hits(q, a.s > 0.0f ? tau : __builtin_nanf(""));
    uint32_t at = hits.count;
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const uint32_t other = __shfl_up(at, off);
        at += lane >= off ? other : 0;
    }
    const uint32_t many = __builtin_amdgcn_readlane(at, kWave - 1);
    at -= hits.count;
    uint32_t place = 0;
    if (many <= L.kCap) {
        if (lane == 0) place = atomicAdd(&L.total, many);
        at += __builtin_amdgcn_readfirstlane(place);
        hits.each(q, pos, T * VW, [&](uint64_t key) { L.buf[at++] = key; });
    } else {  // ties
        const uint32_t n = wave_best<Fmt, NV>(q, pos, T * VW, j.width, L.best[wave], lane);
        team_sync<kWave>();
        if (lane == 0) place = atomicAdd(&L.total, n);
        place = __builtin_amdgcn_readfirstlane(place);
        if (static_cast<uint32_t>(lane) < n) L.buf[place + lane] = L.best[wave][lane];
    }
    __syncthreads();
    // every thread merges the four statistics
    Stat all = L.stat[0];
#pragma unroll
    for (int x = 1; x < W; ++x) {
        Stat o = L.stat[x];
        const float to = max_f(all.m, o.m);
        all.move<true>(to, k_hi);
        o.move<true>(to, k_hi);
        all.s += o.s;
        all.h += o.h;
    }
    // ranks: several lanes count for a key, each over its share of the others
    const uint32_t total = L.total;
    const bool ok = all.s > 0.0f;
    const uint32_t lg = total <= 16 ? 4 : total <= 32 ? 3 : total <= 64 ? 2 : total <= 128 ? 1 : 0;
    for (uint32_t i = tid >> lg; ok && i < total; i += T >> lg) {
        const uint64_t key = L.buf[i];
        uint32_t rank = 0;
#pragma unroll 4
        for (uint32_t y = tid & ((1u << lg) - 1); y < total; y += 1u << lg) rank += L.buf[y] > key ? 1 : 0;
        rank = lanes_sum_u32(rank, lg);
        if ((tid & ((1u << lg) - 1)) == 0 && rank < j.width)
            store_part(w.lists + static_cast<size_t>(j.list()) * j.width + rank, key);
    }
    if (tid == 0) {
        store_part(w.slices + 2 * j.list(), two(all.m, __float_as_uint(all.s)));
        store_part(w.slices + 2 * j.list() + 1, two(all.h, ok ? (total < j.width ? total : j.width) : 0));
    }
}

// Few slices: the last one joins. Latencies bound it: [1,4,32000] f32 10.2 us captured (kernel trace 10.3), [1,8,202048]
// bf16 13.2 (13.6), [16,5,32001] f16 12.8 (13.1), where the launch takes 2.8, the arrival about 3 and the join 3; with the
// join as a launch of its own 15 to 17.
template <typename Fmt, int NV>
__global__ __launch_bounds__(kSliceThreads) void k_beam_slice(uint64_t x, uint64_t scores, uint64_t ended,
                                                              uint64_t scratch, uint64_t out, uint32_t stride,
                                                              uint32_t end_token, float k_hi, uint32_t nonce) {
    __shared__ uint32_t s_found;
    __shared__ union Lds {
        SliceLds<kSliceThreads / kWave> slice;
        JoinLds join;
        __device__ Lds() {}
    } lds;
    extern __shared__ uint64_t s_cands[];
    const SliceJob j(x, scores, ended, scratch, end_token);
    const Scratch w(addr<uint8_t>(scratch), j.groups, j.step.g, j.beams * j.parts, j.width);
    if (j.on()) hold_slice<Fmt, NV>(lds.slice, j, w, x, stride, k_hi);
    join_if_last<kSliceThreads>(lds.join, s_cands, &s_found, j, w, nonce, k_hi, out);
}

// Many rows of up to 512 vectors: a wavefront each, and the join is a launch of its own. [2000,12,1000] f16 28 us and 14
// for the join; arithmetic bounds it, 33 vector instructions' time per logit.
template <typename Fmt, int NV>
__global__ __launch_bounds__(kWave) void k_beam_rows(uint64_t x, uint64_t scores, uint64_t ended, uint64_t scratch,
                                                         uint32_t stride, float k_hi) {
    __shared__ SliceLds<1> s_slice;
    const SliceJob j(x, scores, ended, scratch, kNoEnd);
    const Scratch w(addr<uint8_t>(scratch), j.groups, j.step.g, j.beams * j.parts, j.width);
    if (j.on()) hold_slice<Fmt, NV>(s_slice, j, w, x, stride, k_hi);
}

// ---------------------------------------------------------------------------------------
// Groups of short rows: one wavefront per group holds all of its beams' logits and needs no scratch.

constexpr int kGroupCap = 256;  // candidates that a wavefront collects

// G lanes per row, 64 / G rows to a unit (C == 1), or a row of C units of 64 vectors; I units of a vector per lane.
// Every lane judges its elements by the row's base in binary64; a bound that `width` lanes' best reach leaves few
// more to collect and rank. [2048,4,64] f16 5.2 us (1.1 MB: the launch and one chain of loads, reductions and ranks);
// by a workgroup per row and a join 24.6.
// Tags: columns in (x, scores), beams - 1 and width (8 bits each) in ended, the low part of k in out.
template <typename Fmt, int G, int C, int I>
__global__ __launch_bounds__(kBlockThreads) void k_beam_group(uint64_t x, uint64_t scores_, uint64_t ended_, uint64_t out_,
                                                              uint32_t stride, uint32_t end_token, float k_hi,
                                                              uint32_t groups) {
    constexpr int VW = Fmt::VW, kRows = kWave / G;  // rows of a unit
    static_assert(C == 1 || G == kWave, "long rows take whole units");
    __shared__ CandLds<kGroupCap> s_cand[kBlockThreads / kWave];
    const uint32_t cols = tags(x, scores_), beams = (tag(ended_) >> 8) + 1, width = tag(ended_) & 0xffu;
    const uint32_t wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const uint32_t g = blockIdx.x * (kBlockThreads / kWave) + wave;
    if (g >= groups) return;  // whole wavefronts, and no barriers
    const int lane = threadIdx.x % kWave;
    auto& cand = s_cand[wave];
    const Scale k(k_hi, tag(out_));
    const float* scores = addr<const float>(scores_) + static_cast<size_t>(g) * beams;
    const uint8_t* ended = addr<const uint8_t>(ended_);
    const auto beam = [&](int u) { return C > 1 ? static_cast<uint32_t>(u / C) : static_cast<uint32_t>(u * kRows + lane / G); };
    const auto vec = [&](int u) { return C > 1 ? static_cast<uint32_t>(u % C * kWave + lane) : static_cast<uint32_t>(lane % G); };
    typename Fmt::Vec q[I];
    float score[I];
    bool on[I], done[I];
#pragma unroll
    for (int u = 0; u < I; ++u) {
        const uint32_t b = beam(u), v = vec(u);
        score[u] = b < beams ? scores[b] : -__builtin_huge_valf();
        done[u] = b < beams && ended != nullptr && ended[static_cast<size_t>(g) * beams + b] != 0;
        on[u] = alive(score[u]) && !done[u];
        done[u] = done[u] && alive(score[u]) && v == 0;  // offers its score, from the row's first lane
        q[u] = masked16<Fmt>();
        if (on[u]) {
            const RowSpan<Fmt> sp(row_ptr<Fmt>(addr<const void>(x), g * beams + b, stride), cols);
            if (v < sp.vb)
                q[u] = sp.load_whole(v);
            else if (v == sp.vb && cols % VW != 0)
                q[u] = sp.load_tail();
        }
    }
    // statistics of the rows
    float most[I], m[I];
    double base[I];
#pragma unroll
    for (int u = 0; u < I; ++u) {
        float e[VW];
        Fmt::unpack(q[u], e);
        most[u] = max_of(e);
    }
#pragma unroll
    for (int r = 0; r < I; r += C) {
        float top = kLowest, s = 0.0f, h = 0.0f;
#pragma unroll
        for (int c = 0; c < C; ++c) top = max_f(top, most[r + c]);
        top = lanes_max<G>(top);
#pragma unroll
        for (int c = 0; c < C; ++c) {
            float e[VW];
            Fmt::unpack(anew(q[r + c]), e);
#pragma unroll
            for (int i = 0; i < VW; ++i) {
                const float z = (e[i] - top) * k_hi, p = exp2_f(z);
                s += p;
                h = fmaf(p, max_f(z, kZFloor), h);
            }
        }
        s = lanes_sum<G>(s);
        h = lanes_sum<G>(h);
        const double b = k.base(score[r], static_cast<double>(s) + k.lo * static_cast<double>(h));
#pragma unroll
        for (int c = 0; c < C; ++c) {
            m[r + c] = top;
            base[r + c] = on[r + c] ? b : -__builtin_huge_val();
        }
    }
    const auto valid = [&](int u) { return base[u] > -__builtin_huge_val(); };
    // the lane's best value, and a bound that `width` of them reach
    uint64_t best = 0;
#pragma unroll
    for (int u = 0; u < I; ++u) {
        uint64_t o = 0;
        if (valid(u) && most[u] >= kLowest)
            o = order64(base[u] + (static_cast<double>(most[u]) - static_cast<double>(m[u])) * k.invt);
        if (done[u]) o = order64(static_cast<double>(score[u]));
        best = o > best ? o : best;
    }
    const uint32_t o[1] = {high_of(best)};
    uint32_t bound = 0;
    if (static_cast<uint32_t>(__popcll(__ballot(o[0] != 0))) > width) bound = bisect(o, width, width + width / 4 + 1);
    // what a logit must be at least, row by row: the bound's, less what the rounding of this can be off by
    const double least = value64(static_cast<uint64_t>(bound) << 32), t = 1.0 / k.invt;
    uint32_t count = 0;
    float tau[I];
#pragma unroll
    for (int u = 0; u < I; ++u) {
        tau[u] = __builtin_nanf("");  // nothing reaches it, not +inf either
        if (valid(u)) {
            const double v = static_cast<double>(m[u]) + (least - base[u]) * t;
            const double off = (fabs(least) + fabs(base[u])) * 0x1p-48 * t + fabs(v) * 0x1p-20 + 0x1p-120;
            const float f = static_cast<float>(v - off);
            tau[u] = bound != 0 && f > kLowest ? f : kLowest;
        }
        const typename Fmt::Vec one[1] = {q[u]};
        count += Hits<Fmt, 1>(one, tau[u]).count + (done[u] ? 1 : 0);
    }
    uint32_t at = count;
#pragma unroll
    for (int off = 1; off < kWave; off *= 2) {
        const uint32_t other = __shfl_up(at, off);
        at += lane >= off ? other : 0;
    }
    const uint32_t n = __builtin_amdgcn_readlane(at, kWave - 1);
    at -= count;
    const BeamOut out(addr<uint8_t>(out_), groups, width);
    const size_t first = static_cast<size_t>(g) * width;
    if (n <= kGroupCap) {
#pragma unroll
        for (int u = 0; u < I; ++u) {
            const typename Fmt::Vec one[1] = {q[u]};
            Hits<Fmt, 1> hits(one, tau[u]);
            hits.each(one, vec(u) * VW, 0, [&](uint64_t key) { cand.put(at++, k.candidate(base[u], m[u], beam(u), key)); });
            if (done[u]) cand.put(at++, finished(score[u], beam(u), end_token));
        }
        team_sync<kWave>();
        // ranks: several lanes count for a candidate, each over its share of the others
        const uint32_t lg = n <= 4 ? 4 : n <= 8 ? 3 : n <= 16 ? 2 : n <= 32 ? 1 : 0;
        for (uint32_t i = lane >> lg; i < n; i += kWave >> lg) {
            const Cand c = cand.get(i);
            uint32_t rank = 0;
#pragma unroll 2
            for (uint32_t j = lane & ((1u << lg) - 1); j < n; j += 1u << lg) rank += cand.get(j).above(c) ? 1 : 0;
            rank = lanes_sum_u32(rank, lg);
            if ((lane & ((1u << lg) - 1)) == 0 && rank < width) out.put(first + rank, c, end_token);
        }
        if (static_cast<uint32_t>(lane) < width && static_cast<uint32_t>(lane) >= n) out.none(first + lane);
        return;
    }
    // ties: the best are taken one by one
    Cand last{~uint64_t{0}, ~uint64_t{0}, 0};
    for (uint32_t r = 0; r < width; ++r) {
        Cand top{0, 0, 0};
        const auto offer = [&](const Cand& c) {
            if (last.above(c) && c.above(top)) top = c;
        };
#pragma unroll
        for (int u = 0; u < I; ++u) {
            float e[VW];
            Fmt::unpack(anew(q[u]), e);
#pragma unroll
            for (int i = 0; i < VW; ++i)
                if (valid(u) && e[i] >= kLowest) offer(k.candidate(base[u], m[u], beam(u), key_of(e[i], vec(u) * VW + i)));
            if (done[u]) offer(finished(score[u], beam(u), end_token));
        }
#pragma unroll
        for (int off = 1; off < kWave; off *= 2) {
            const Cand c{__shfl_xor(static_cast<unsigned long long>(top.value), off),
                         __shfl_xor(static_cast<unsigned long long>(top.key), off), __shfl_xor(top.beam, off)};
            if (c.above(top)) top = c;
        }
        if (lane == 0) {
            if (top.value != 0)
                out.put(first + r, top, end_token);
            else
                out.none(first + r);
        }
        last = top;
    }
}

// ---------------------------------------------------------------------------------------
// Reordering, in place. A lane owns the same 16 bytes of all beams of a group: it loads them from
// the parents of the beams that move, all of them before it stores the first, and no other lane
// touches them, so nothing has to be set aside. Beams that stay are neither read nor written. [16,8,8,512,128]
// bf16, 16 tensors, 5 of 8 beams moved (2.1 GB read and written): 420 us, 5.1 TB/s, the rate of a plain copy.

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
    typedef V __attribute__((aligned(1))) U;  // nontemporal: 438 us, plain ones 441; 64.7 and 75 for [33,5,600,3,65] f32
    __builtin_nontemporal_store(v, reinterpret_cast<U*>(p));
}

// Moves U units of up to NB beams. move[j]: source beam, and destination << 16; scalars.
template <typename V, int NB, int U>
__device__ inline void move_units(uint8_t* const (&at)[U], const uint32_t (&move)[NB], int n, int64_t beam_stride) {
    V v[NB][U];
#pragma unroll
    for (int j = 0; j < NB; ++j)
        if (j < n) {
            const int64_t off = (move[j] & 0xffffu) * beam_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) v[j][u] = load_any<V>(at[u] + off);
        }
#pragma unroll
    for (int j = 0; j < NB; ++j)
        if (j < n) {
            const int64_t off = (move[j] >> 16) * beam_stride;
#pragma unroll
            for (int u = 0; u < U; ++u) store_any<V>(at[u] + off, v[j][u]);
        }
}
template <typename V, int NB>
__device__ inline void move_unit(uint8_t* at, const uint32_t (&move)[NB], int n, int64_t beam_stride) {
    uint8_t* const one[1] = {at};
    move_units<V, NB, 1>(one, move, n, beam_stride);
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
    const auto place = [&](uint32_t i) {  // of unit i
        const uint32_t seg = i / units, u = i - seg * units;
        const uint32_t o = seg / per, pos = seg - o * per;
        return base + o * s.outer_stride + pos * s.position_stride + static_cast<int64_t>(u) * kUnit;
    };
    // Two units at once where their registers leave room: 420 us instead of 438 for [16,8,8,512,128] bf16 in 16 tensors.
    constexpr uint32_t U = NB <= 8 ? 2 : 1, kStep = kBlockThreads * U;
    if (bytes % kUnit == 0) {
        uint32_t i = block * kStep + threadIdx.x;
        for (; i + (U - 1) * kBlockThreads < total; i += blocks * kStep) {
            uint8_t* at[U];
#pragma unroll
            for (uint32_t k = 0; k < U; ++k) at[k] = place(i + k * kBlockThreads);
            move_units<V, NB, U>(at, move, n, s.beam_stride);
        }
        if (i < total) move_unit<V, NB>(place(i), move, n, s.beam_stride);
        return;
    }
    for (uint32_t i = block * kBlockThreads + threadIdx.x; i < total; i += blocks * kBlockThreads) {
        uint8_t* at = place(i);
        const uint32_t u = i % units;
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

size_t beam_scratch(int64_t groups, int64_t lists, int width) { return Scratch::bytes(groups, lists, width); }

hipError_t launch_beam_step(const BeamPlan& plan, const BeamArgs& a, uint8_t* scratch16, hipStream_t s) {
    const uint32_t cols = static_cast<uint32_t>(a.cols), stride = static_cast<uint32_t>(a.row_stride);
    const double k = 1.4426950408889634074 / a.temperature;
    const float hi = static_cast<float>(k);
    // the rest of k to 8 bits: k is then good to 2^-33 of itself
    const float rest = static_cast<float>(k - static_cast<double>(hi));
    const uint32_t low = (bits_of(rest) + 0x8000u) >> 16;
    const uint32_t end = a.end_token < 0 ? kNoEnd : static_cast<uint32_t>(a.end_token);
    const uint32_t shape = static_cast<uint32_t>(a.beams - 1) << 8 | static_cast<uint32_t>(plan.parts - 1);
    const uint32_t grid = static_cast<uint32_t>(plan.grid_blocks);
    const auto x = tagged(a.x, cols), scores = tagged(a.scores, cols >> 16), ended = tagged(a.ended, shape),
               scratch = tagged(scratch16, a.width), out = tagged(a.out, low);
    const auto slice = [&](auto kernel) {
        hipLaunchKernelGGL(kernel, dim3(grid), dim3(kSliceThreads), beam_cands(a.width), s, x, scores, ended, scratch, out,
                           stride, end, hi, next_nonce());
    };
    const auto scan = [&](auto kernel) {
        launch(kernel, grid, plan.team, s, x, scores, ended, scratch, stride, hi);
        hipLaunchKernelGGL(k_beam_join, dim3(static_cast<uint32_t>(a.groups)), dim3(kSliceThreads), beam_cands(a.width), s,
                           scores, ended, scratch, out, end, hi);
    };
    const auto group = [&](auto kernel) {
        const uint32_t sizes = static_cast<uint32_t>(a.beams - 1) << 8 | static_cast<uint32_t>(a.width);
        launch(kernel, grid, kBlockThreads, s, x, scores, tagged(a.ended, sizes), out, stride, end, hi,
               static_cast<uint32_t>(a.groups));
    };
    with_format(a.dtype, [&](auto fmt) {
        using Fmt = decltype(fmt);
        if (plan.path == ARGREDUCE_PATH_SUBWAVE) {
            const auto units = [&](auto lanes, auto chunks) {
                constexpr int G = decltype(lanes)::value, C = decltype(chunks)::value;
                switch (plan.held) {
                    case 1:
                        if constexpr (C == 1) return group(k_beam_group<Fmt, G, C, 1>);
                    case 2: return group(k_beam_group<Fmt, G, C, 2>);
                    case 4: return group(k_beam_group<Fmt, G, C, 4>);
                    default: return group(k_beam_group<Fmt, G, C, 8>);
                }
            };
            switch (plan.team) {
                case 4: return units(Int<4>{}, Int<1>{});
                case 8: return units(Int<8>{}, Int<1>{});
                case 16: return units(Int<16>{}, Int<1>{});
                case 32: return units(Int<32>{}, Int<1>{});
                case 64: return units(Int<64>{}, Int<1>{});
                default: return units(Int<64>{}, Int<2>{});
            }
        }
        if (plan.held > 0) {
            const auto held = [&](auto vecs) {
                constexpr int NV = decltype(vecs)::value;
                if (plan.joins)
                    slice(k_beam_slice<Fmt, NV>);
                else
                    scan(k_beam_rows<Fmt, NV>);
            };
            switch (plan.held) {
                case 1: return held(Int<1>{});
                case 2: return held(Int<2>{});
                case 4: return held(Int<4>{});
                default: return held(Int<8>{});
            }
        }
        switch (plan.team) {
            case 64: return scan(k_beam_scan<Fmt, 64>);
            case 256: return scan(k_beam_scan<Fmt, 256>);
            case 512: return scan(k_beam_scan<Fmt, 512>);
            default: return scan(k_beam_scan<Fmt, 1024>);
        }
    });
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
