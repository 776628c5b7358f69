// Beam search's selection over beams and vocabulary, for gfx950.
//
// For a group of beams with scores s_b and rows of logits x_b, the k largest of
//   s_b + x_b[v] - lse_b,   lse_b = log sum_v exp x_b[v]
// in two launches, or one.
//
// 1. The four waves of a workgroup stream a row (or a piece of one), each every
//    fourth group of 4 KB, with a running maximum and sum of the softmax.  A
//    row's order is that of its logits whatever lse_b is, so its k best are
//    collected beside it: at least j elements of a wave reach the j-th largest of its 64
//    lanes' maxima, so the k best reach the least of the four waves' with
//    j = k / 4.  Few elements reach this bound once some groups have passed (k / n
//    of the n-th element's kind).  The 16-byte words that they lie in are kept in
//    LDS as they are, three instructions and two stores a word; only at the end, when the bound is
//    what the whole piece gave, are their elements looked at, a lane an element.
//    What is left (some 20 for k = 8) is ranked by counting the larger ones.
// 2. A workgroup a group joins its rows' pieces and ranks the rows' candidates
//    against each other by their values in 64 bits.
// Where rows are short and beams few, one workgroup does both.
//
// Bound by the reads.  Measured, the scan and the join: 256 x 102400 bf16, k = 8:
// 15.9 + 5.0 us (3.3 TB/s); 1024 x 131072 bf16 and k = 32, the whole call: 62 us
// (4.3 TB/s); 1024 x 131071 f32, k = 32: 94 to 99 + 7 us (5.4 to 5.7 TB/s).  On short rows it is
// bound by the chain of steps that a piece is: 2000 clocks to the first group, 850 its
// sum, 900 a bound, 2500 the end.  Elements appended one at a time as a row passes
// took the first case 17.3 us.
#include <type_traits>

#include "rts_device.hpp"
#include "rts_internal.h"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kBeamWaves = 4;
constexpr int kBeamBlock = kBeamWaves * kWave;
constexpr int kWords = 4;         // of 16 bytes that a lane loads at a time: a group of 4 KB a wave
template <typename T>
constexpr int group_elements() { return kWords * kWave * 16 / (int)sizeof(T); }
template <typename T>
__host__ __device__ __forceinline__ int64_t row_groups(int64_t vocab) {
    return (vocab + group_elements<T>() - 1) / group_elements<T>();
}
constexpr int kStaged = 384;      // words with candidates that a wave holds
constexpr int kListed = 2 * kWave;  // candidates
constexpr int kAtOnce = 8;
constexpr int kMaxJoinWaves = 16;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -3.402823466e38f;  // the lowest finite number

// A wave's part of a row's sum: sum e^ref.
struct PieceStat {
    double ref, sum;
};

template <typename Op>
__device__ __forceinline__ double wave_reduce(double x, Op op) {
    const uint64_t r = wave_reduce64((uint64_t)__double_as_longlong(x), [&](uint64_t a, uint64_t b) {
        return (uint64_t)__double_as_longlong(op(__longlong_as_double((long long)a), __longlong_as_double((long long)b)));
    });
    return __longlong_as_double((long long)r);
}

__device__ __forceinline__ float wave_max(float x) {
    auto step = [](float a, uint32_t b) { return fmaxf(a, __uint_as_float(b)); };
    x = step(x, dpp32<kDppQuadXor1>(__float_as_uint(x), __float_as_uint(x)));
    x = step(x, dpp32<kDppQuadXor2>(__float_as_uint(x), __float_as_uint(x)));
    x = step(x, dpp32<kDppRowHalfMirror>(__float_as_uint(x), __float_as_uint(x)));
    x = step(x, dpp32<kDppRowMirror>(__float_as_uint(x), __float_as_uint(x)));
    x = step(x, dpp32<kDppRowBcast15, 0xA>(__float_as_uint(x), __float_as_uint(x)));
    x = step(x, dpp32<kDppRowBcast31, 0xC>(__float_as_uint(x), __float_as_uint(x)));
    return __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(x), kWave - 1));
}

// An element of a 16-byte word.
template <typename T>
__device__ __forceinline__ float element_of(const uint4& w, int e) {
    const uint32_t x[4] = {w.x, w.y, w.z, w.w};
    if constexpr (sizeof(T) == 4) return __uint_as_float(x[e]);
    else return __uint_as_float(e & 1 ? x[e >> 1] & 0xFFFF0000u : x[e >> 1] << 16);
}

// 16 bytes at any multiple of 4, or of 2.
typedef uint32_t words_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t words_at2 __attribute__((ext_vector_type(4), aligned(2)));

// Word w of a row is its elements kEach w .. + kEach, whatever the row's alignment
// is (loads of 16 bytes take any address), so that equal rows give equal sums.
// Word j of group g is the lanes' (g kWords + j) * 64 + lane.
template <typename T>
struct RowReader {
    static constexpr int kEach = 16 / sizeof(T);
    using words = std::conditional_t<sizeof(T) == 4, words_at4, words_at2>;
    const T* row;
    int64_t vocab;
    __device__ __forceinline__ int64_t word_of(int64_t g, int j) const { return (g * kWords + j) * kWave + lane_id(); }
    __device__ __forceinline__ bool inside(int64_t g) const { return (g + 1) * group_elements<T>() <= vocab; }
    __device__ __forceinline__ uint4 load(int64_t g, int j) const {  // a group inside of the row
        const words w = *reinterpret_cast<const words*>(row + word_of(g, j) * kEach);
        return uint4{w[0], w[1], w[2], w[3]};
    }
    // The last group: what lies behind the row is -inf.
    __device__ __forceinline__ uint4 load_edge(int64_t g, int j) const {
        uint32_t x[4] = {0, 0, 0, 0};
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int64_t at = word_of(g, j) * kEach + e;
            const T t = row[at < vocab ? at : vocab - 1];
            if constexpr (sizeof(T) == 4) x[e] = at < vocab ? __float_as_uint(t) : 0xFF800000u;
            else x[e / 2] |= (uint32_t)(at < vocab ? t : 0xFF80) << 16 * (e % 2);
        }
        return uint4{x[0], x[1], x[2], x[3]};
    }
};

// Merges the sorted (descending) list `more` into `best`, the 64 largest stay.
__device__ __forceinline__ void merge_sorted(uint64_t& best, uint64_t more) {
    const int lane = lane_id();
    const uint32_t lo = __shfl((uint32_t)more, kWave - 1 - lane), hi = __shfl((uint32_t)(more >> 32), kWave - 1 - lane);
    uint64_t v[1] = {umax64(best, (uint64_t)hi << 32 | lo)};
    wave_bitonic_merge<1, true>(v);
    best = v[0];
}

template <int WAVES>
struct ScanLds {
    uint4 words[WAVES][kStaged];     // with candidates
    uint64_t listed[WAVES][kListed];
    float published[WAVES];          // a bound that enough of the wave's elements reach
    uint32_t at[WAVES][kStaged];
    int kept[WAVES], places[WAVES * kWave];
};
static_assert(kStaged >= kWords * kWave && kListed >= kWave + kAtOnce, "a group; a full list and what follows it");

// The scan of `count` groups from g0 on of a row by EACH waves of a workgroup, whose other waves scan
// other rows (or none: 0 groups): stat(part of the sum) by lane 0 of each, put(place, entry) for places 0..k-1
// by any thread of theirs.
template <typename T, int WAVES, int EACH, typename Stat, typename Put>
__device__ __forceinline__ void scan_row(const BeamArgs& a, ScanLds<WAVES>& lds, const RowReader<T>& in, int64_t g0,
                                         int64_t groups, Stat&& stat, Put&& put) {
    constexpr int kEach = RowReader<T>::kEach;
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int side = EACH == WAVES ? wave : wave % EACH;  // the wave's number in its row
    const int team = EACH == WAVES ? 0 : wave - side;     // the first of them
    uint4* const staged_words = lds.words[wave];
    uint32_t* const staged_at = lds.at[wave];
    uint64_t* const listed = lds.listed[wave];
    float* const published = lds.published + team;
    // Waves that have a whole group (the row's last one may have too few elements for a bound of use).
    const int64_t whole = groups > 1 && !in.inside(g0 + groups - 1) ? groups - 1 : groups;
    const int busy = whole < EACH ? (int)whole : EACH;
    const int64_t n = (groups - side + EACH - 1) / EACH;  // this wave's

    // The next group is on its way while one is looked at.
    uint4 next[kWords];
    auto group_of = [&](int64_t i) { return g0 + side + i * EACH; };
    auto load = [&](int64_t i) __attribute__((always_inline)) {
        if (i < n && in.inside(group_of(i)))
#pragma unroll
            for (int j = 0; j < kWords; ++j) next[j] = in.load(group_of(i), j);
    };
    load(0);

    // One more than k where the end token may be among them.
    const int need = a.k + (a.eos >= 0 ? 1 : 0), share = (need + busy - 1) / (busy > 0 ? busy : 1);
    if (lane == 0) published[side] = side < busy ? -INFINITY : INFINITY;
    __syncthreads();

    float m = kLeast, lane_most = -INFINITY;
    // Terms are 2^(x log2(e) - c2) in 32 bits, c2 the whole number next to m log2(e), so
    // that sums go over to a new maximum without a rounding.  The sum is taken relative to the
    // maximum's own term, what is computed for x = m: a row whose weight is all on one logit has
    // its logarithm to the last bit, and none is below its largest logit.  A group's terms are added in
    // 32 bits, groups in 64: ten roundings of a row's sum are left at most, some 1e-7 of it.
    // Past 1e6 the difference would come near the range of an exponential, and they are e^(x - m).
    double sum = 0.;
    float c2;
    bool huge;
    auto set_reference = [&] {
        huge = fabsf(m) > 1e6f;
        c2 = huge ? 0.f : rintf(m * kLog2e);
    };
    set_reference();
    float bound = kLeast;  // elements from here on are candidates; -inf is none
    uint64_t best = 0;     // what was sorted, where the stage ran over
    int held = 0, in_list = 0;
    bool best_any = false;
    // Sorts the last 64 (or fewer) of the list into the best.
    auto flush = [&] {
        const int count = in_list < kWave ? in_list : kWave;
        in_list -= count;
        wave_lds_sync();
        uint64_t v[1] = {lane < count ? listed[in_list + lane] : 0};
        wave_lds_sync();
        wave_bitonic_sort<1, true>(v);
        merge_sorted(best, v[0]);
        best_any = true;
    };
    auto raise = [&](float to) { bound = to > bound ? to : bound; };
    // A bound that n of the lanes' maxima reach, and few more: their keys' common
    // bits, then two bits a step.
    auto reached_by = [&](int n) {
        const uint32_t key = key32_of_bits(__float_as_uint(lane_most));
        const uint32_t least = wave_min32(key), most = key32_of_bits(__float_as_uint(m));
        if (n == kWave || least >= most) return float_of_key32(least);
        int bit = 31 - __builtin_clz(least ^ most) & ~1;
        const int last = bit > 24 ? 16 : bit > 8 ? bit - 8 : 0;
        uint32_t to = most & ~3u << bit;
        for (; bit >= last; bit -= 2) {
            uint32_t with[3];
            int count[3], chosen = 0;
#pragma unroll
            for (int d = 0; d < 3; ++d) {
                with[d] = to | (uint32_t)(d + 1) << bit;
                count[d] = __popcll(__ballot(key >= with[d]));
            }
#pragma unroll
            for (int d = 0; d < 3; ++d)
                if (count[d] >= n) to = with[d], chosen = count[d];
            if (chosen == n) break;
        }
        return float_of_key32(to > least ? to : least);
    };
    auto refresh = [&] {
        if (side >= busy || share > kWave) return;
        const float x = reached_by(share);
        if (lane == 0) __hip_atomic_store(&published[side], x, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    };
    auto heed = [&] {  // the other waves
        typedef float bounds __attribute__((ext_vector_type(EACH)));
        // Through a plain pointer the read waits for the group under way as well,
        // and that is faster: 1024 x 131072 bf16 65 us, read as LDS without that wait 74.
        const bounds p = *reinterpret_cast<volatile bounds*>(published);
        float least = p[0];
#pragma unroll
        for (int w = 1; w < EACH; ++w) least = fminf(least, p[w]);
        raise(__uint_as_float(__builtin_amdgcn_readfirstlane(__float_as_uint(least))));
    };
    // The maximum and the sum of a group.
    auto add = [&](const uint4 (&x)[kWords], const float (&top)[kWords]) __attribute__((always_inline)) {
        float most = fmaxf(fmaxf(top[0], top[1]), fmaxf(top[2], top[3]));
        lane_most = fmaxf(lane_most, most);
        most = wave_max(most);
        if (most > m) {
            const float was = m, from = c2;
            const bool was_huge = huge;
            m = most;
            set_reference();
            if (!huge && !was_huge) {
                sum = ldexp(sum, (int)(from - c2));
            } else {
                const float lower = !huge      ? fmaf(was, kLog2e, -c2)
                                    : was_huge ? (was - m) * kLog2e
                                               : -fmaf(m, kLog2e, -from);
                sum *= __builtin_amdgcn_exp2f(lower);
            }
        }
        auto terms = [&](auto term) __attribute__((always_inline)) {
            float all = 0.f;
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                float part = 0.f;
#pragma unroll
                for (int e = 0; e < kEach; ++e) part += __builtin_amdgcn_exp2f(term(element_of<T>(x[j], e)));
                all += part;
            }
            sum += all;
        };
        if (huge) terms([&](float v) { return (v - m) * kLog2e; });
        else terms([&](float v) { return fmaf(v, kLog2e, -c2); });
    };
    // Stages the words of a group in which something reaches the bound.
    auto collect = [&](int64_t g, const uint4 (&x)[kWords], const float (&top)[kWords]) __attribute__((always_inline)) {
#pragma unroll
        for (int j = 0; j < kWords; ++j) {
            const uint64_t mask = __ballot(top[j] >= bound);
            if (!mask) continue;
            if (top[j] >= bound) {
                const int at = held + mbcnt64(mask);
                staged_words[at] = x[j];
                staged_at[at] = (uint32_t)in.word_of(g, j);
            }
            held += __popcll(mask);
        }
    };
    // Lists the elements of the staged words that reach the bound, a lane an element.
    auto expand = [&] {
        // More than there should be: the other waves hold the bound down (their elements
        // are masked, or rise), and this wave's own may be higher.  256 x 102400 bf16, the whole
        // call: all but 2048 masked 24.5 us without it, 20.9 with it; rows in order 153 and 53.
        if (held > kWave && need <= kWave) raise(reached_by(need));
        wave_lds_sync();
        for (int i = 0; i < held; i += kWave / kEach) {
            const int from = i + lane / kEach;
            const uint32_t at = from < held ? staged_at[from] * kEach + lane % kEach : 0;
            const T t = reinterpret_cast<const T*>(&staged_words[from < held ? from : 0])[lane % kEach];
            float v;
            if constexpr (sizeof(T) == 4) v = t;
            else v = __uint_as_float((uint32_t)t << 16);
            const bool hit = from < held && v >= bound && at != (uint32_t)a.eos;
            const uint64_t mask = __ballot(hit);
            // -0 and 0 are one logit: the sum is 0 for both.
            if (hit) listed[in_list + mbcnt64(mask)] = composite(key32_of_bits(__float_as_uint(v + 0.f)), at);
            in_list += __popcll(mask);
            if (in_list > kWave) {
                flush();
                // Later elements of this wave lie behind what it has sorted: they
                // count if they are larger than the k-th of that.
                const uint64_t kth = readlane64(best, a.k - 1);
                if (kth) raise(float_of_key32((uint32_t)(kth >> 32) + 1));
            }
        }
        held = 0;
    };

    for (int64_t i = 0;; ++i) {
        if (i < n) {
            const int64_t g = group_of(i);
            if (!in.inside(g))
#pragma unroll
                for (int j = 0; j < kWords; ++j) next[j] = in.load_edge(g, j);
            uint4 x[kWords];
            float top[kWords];
#pragma unroll
            for (int j = 0; j < kWords; ++j) {
                x[j] = next[j];
                top[j] = element_of<T>(x[j], 0);
#pragma unroll
                for (int e = 1; e < kEach; ++e) top[j] = fmaxf(top[j], element_of<T>(x[j], e));
            }
            load(i + 1);
            add(x, top);
            if ((i & (i + 1)) == 0) refresh();  // groups 0, 1, 3, 7, ..
            if (i == 0) __syncthreads();        // little is known of the first: all waves' together
            heed();
            collect(g, x, top);
        } else {
            if (n == 0) __syncthreads();
            if ((n & (n - 1)) != 0) refresh();  // else it was after the last
            __syncthreads();
            heed();
        }
        if (held > kStaged - kWords * kWave || i >= n) expand();
        if (i >= n) break;
    }

    if (best_any) {
        while (in_list > 0) flush();
        wave_lds_sync();
        const uint64_t mask = __ballot(best != 0);  // the first lanes
        listed[lane] = best;
        in_list = __popcll(mask);
    }
    if (lane < kAtOnce) listed[in_list + lane] = 0;
    if (lane == 0) lds.kept[wave] = in_list;
    lds.places[threadIdx.x] = 0;
    __syncthreads();
    // All of the row's waves' together.
    int* const places = lds.places + team * kWave;
    int upto[EACH], count = 0;
#pragma unroll
    for (int w = 0; w < EACH; ++w) upto[w] = count += lds.kept[team + w];
    auto entry_at = [&](int at) {
        int w = 0, before = 0;
#pragma unroll
        for (int u = 0; u + 1 < EACH; ++u)
            if (at >= upto[u]) w = u + 1, before = upto[u];
        return at < count ? lds.listed[team + w][at - before] : 0;
    };
    const int thread = side * kWave + lane;
    const uint64_t mine = entry_at(thread);
    {
        const double total = wave_reduce(sum, [](double x, double y) { return x + y; });
        const float own = __builtin_amdgcn_exp2f(huge ? (m - m) * kLog2e : fmaf(m, kLog2e, -c2));
        if (lane == 0) stat(PieceStat{(double)m, total / own});
    }
    // An entry's place is the number of larger ones: a wave counts those of its own.
    for (int at = lane; at - lane < count; at += kWave) {
        const uint64_t v = entry_at(at);
        int larger = 0;
        for (int i = 0; i < in_list; i += kAtOnce) {
            uint64_t other[kAtOnce];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) other[u] = listed[i + u];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) larger += other[u] > v;
        }
        if (at < count && larger) __hip_atomic_fetch_add(&places[at], larger, __ATOMIC_RELAXED, __HIP_MEMORY_SCOPE_WORKGROUP);
    }
    __syncthreads();
    const int place = thread < count ? places[thread] : thread;
    if (place < a.k) put(place, mine);
}

template <typename T>
__global__ __launch_bounds__(kBeamBlock) void beam_scan_kernel(BeamArgs a, int64_t piece_groups,
                                                               uint64_t* __restrict__ lists,
                                                               PieceStat* __restrict__ stats) {
    __shared__ __align__(16) ScanLds<kBeamWaves> lds;
    const int64_t r = blockIdx.x, unit = r * gridDim.y + blockIdx.y;
    const int64_t g0 = blockIdx.y * piece_groups, all = row_groups<T>(a.vocab);
    scan_row<T, kBeamWaves, kBeamWaves>(
        a, lds, RowReader<T>{static_cast<const T*>(a.logits) + r * a.ld, a.vocab}, g0,
        all - g0 < piece_groups ? all - g0 : piece_groups,
        [&](PieceStat x) { stats[unit * kBeamWaves + threadIdx.x / kWave] = x; },
        [&](int place, uint64_t x) { lists[unit * a.k + place] = x; });
}

// A candidate among those of other beams: the upper 52 bits of its value's
// key, so that values closer than 2^-40 of their size count as equal (a row's sum, of 32-bit terms,
// puts all of its values some 1e-7 off), and below them its beam and its rank there, ascending.  0 is below all.
static_assert(kMaxBeams <= 64 && kMaxBeamK <= 64, "12 bits");
__device__ __forceinline__ uint64_t entry(double v, int beam, int rank) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return ((u >> 63 ? ~u : u | 1ull << 63) | 0xFFF) - (uint32_t)(beam * 64 + rank);
}

template <typename T>
__device__ __forceinline__ float end_logit_of(const BeamArgs& a, int64_t r) {
    const T x = static_cast<const T*>(a.logits)[r * a.ld + a.eos];
    if constexpr (sizeof(T) == 4) return x;
    else return __uint_as_float((uint32_t)x << 16);
}

// What joins a group: `waves` waves (others of the workgroup only keep step) that take a beam each in turn.
struct JoinLds {
    uint64_t* merged;  // [waves][64]
    float* values;     // [beams][64] by rank in their beam
    uint32_t* cols;
};
// list(r, u), of piece u of row r, this lane's entry; stat(r, p) of its part p.
template <typename T, typename List, typename Stat, typename Score>
__device__ __forceinline__ void join_group(const BeamArgs& a, int64_t group, int waves, const JoinLds& lds, int pieces,
                                           int parts, List&& list, Stat&& stat, Score&& score_of) {
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    uint64_t mine = 0;
    for (int b = wave; b < a.beams; b += waves) {
        const int64_t r = group * a.beams + b;
        constexpr int kAhead = 4;
        uint64_t some[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) some[u] = lane < a.k && u < pieces ? list(r, u) : 0;
        const PieceStat first = lane < parts ? stat(r, lane) : PieceStat{-1e300, 0.};
        float end_logit;
        const float score = score_of(r, end_logit);
        uint64_t best = some[0];
        for (int p0 = 0; p0 < pieces; p0 += kAhead) {
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                if (p0 + u >= pieces) break;
                if (p0 + u > 0) merge_sorted(best, some[u]);
                some[u] = lane < a.k && p0 + u + kAhead < pieces ? list(r, p0 + u + kAhead) : 0;
            }
        }
        // The row's sum: a wave's part of a piece a lane.
        auto sums = [](double x, double y) { return x + y; };
        double m = first.ref;
        for (int p = lane + kWave; p < parts; p += kWave) m = fmax(m, stat(r, p).ref);
        m = wave_reduce(m, [](double x, double y) { return fmax(x, y); });
        double sum = first.sum * exp(first.ref - m);
        for (int p = lane + kWave; p < parts; p += kWave) sum += stat(r, p).sum * exp(stat(r, p).ref - m);
        sum = wave_reduce(sum, sums);
        // A row without a finite sum (NaN or +inf in it, or -inf only) and a beam
        // without a finite score have no candidates.
        const bool takes_part = sum > 0 && sum <= 1e300 && fabs(m) <= 1e300 && fabsf(score) <= 3.402823466e38f;
        const double shift = (double)score - log(sum);
        // The difference first: logits of any size keep what lies behind their last place.
        auto value = [&](float x) { return ((double)x - m) + shift; };
        const double v = value(float_of_key32((uint32_t)(best >> 32)));
        lds.values[b * 64 + lane] = (float)v;
        lds.cols[b * 64 + lane] = composite_id(best);
        const uint64_t here = takes_part && best != 0 && lane < a.k ? entry(v, b, lane) : 0;
        if (b == wave) mine = here;
        else merge_sorted(mine, here);
        if (a.ended && lane == 0) a.ended[r] = takes_part ? (float)value(end_logit) : -INFINITY;
    }
    // The waves' lists, two by two.
    for (int step = 1; step < waves; step <<= 1) {
        if ((wave & (2 * step - 1)) == step) lds.merged[wave * kWave + lane] = mine;
        __syncthreads();
        if ((wave & (2 * step - 1)) == 0 && wave + step < waves) merge_sorted(mine, lds.merged[(wave + step) * kWave + lane]);
    }
    if (wave > 0 || lane >= a.k) return;
    const int64_t at = group * a.k + lane;
    const int from = 0xFFF - (int)(mine & 0xFFF);
    a.out_scores[at] = mine ? lds.values[from] : -INFINITY;
    a.parents[at] = mine ? (int32_t)(group * a.beams + from / 64) : -1;
    a.tokens[at] = mine ? (int32_t)lds.cols[from] : -1;
}

template <typename T>
__global__ __launch_bounds__(kMaxJoinWaves * kWave) void beam_join_kernel(BeamArgs a, int pieces,
                                                                         const uint64_t* __restrict__ lists,
                                                                         const PieceStat* __restrict__ stats) {
    extern __shared__ uint64_t memory[];
    const int waves = blockDim.x / kWave, parts = pieces * kBeamWaves, lane = lane_id();
    float* const values = reinterpret_cast<float*>(memory + waves * kWave);
    join_group<T>(a, blockIdx.x, waves, JoinLds{memory, values, reinterpret_cast<uint32_t*>(values + a.beams * 64)}, pieces, parts,
                  [&](int64_t r, int u) { return lists[(r * pieces + u) * a.k + lane]; },
                  [&](int64_t r, int p) { return stats[r * parts + p]; },
                  [&](int64_t r, float& end_logit) {
                      end_logit = a.ended ? end_logit_of<T>(a, r) : 0.f;
                      return a.scores[r];
                  });
}

// Both at once, a workgroup a group: EACH waves a row.
template <typename T, int EACH>
__global__ __launch_bounds__(kMaxJoinWaves * kWave) void beam_group_kernel(BeamArgs a) {
    constexpr int kWaves = kMaxJoinWaves, kRows = kWaves / EACH;
    __shared__ __align__(16) ScanLds<kWaves> lds;
    __shared__ PieceStat stats[kWaves];
    // What the scan's waves have staged is gone when their lists are ranked.
    static_assert(sizeof(lds.words) >= 3 * kWaves * kWave * sizeof(uint64_t), "lists, merged lists, values and tokens");
    uint64_t* const lists = reinterpret_cast<uint64_t*>(lds.words);  // [beams][64]
    uint64_t* const merged = lists + kRows * kWave;
    float* const values = reinterpret_cast<float*>(merged + kWaves * kWave);
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave), beam = wave / EACH;
    const int64_t group = blockIdx.x, r = group * a.beams + (beam < a.beams ? beam : 0);
    // Of the row that this wave joins.
    const int64_t own = group * a.beams + (wave < a.beams ? wave : 0);
    const float own_score = a.scores[own], own_end = a.ended ? end_logit_of<T>(a, own) : 0.f;
    scan_row<T, kWaves, EACH>(
        a, lds, RowReader<T>{static_cast<const T*>(a.logits) + r * a.ld, a.vocab}, 0, beam < a.beams ? row_groups<T>(a.vocab) : 0,
        [&](PieceStat x) { stats[wave] = x; }, [&](int place, uint64_t x) { lists[beam * kWave + place] = x; });
    __syncthreads();
    join_group<T>(a, group, a.beams, JoinLds{merged, values, reinterpret_cast<uint32_t*>(values + kRows * kWave)}, 1, EACH,
                  [&](int64_t row, int) { return lists[(row - group * a.beams) * kWave + lane]; },
                  [&](int64_t row, int p) { return stats[(row - group * a.beams) * EACH + p]; },
                  [&](int64_t, float& end_logit) {
                      end_logit = own_end;
                      return own_score;
                  });
}

// Short rows of few beams are scanned and joined in one launch, a CU a group, as far as
// that saves more than a second launch costs.  Calls, us, in one launch and in two: 16 x 4 beams fp32,
// 4096 tokens 12.2 and 16.4, 16384 14.5 and 16.4, 32768 20.4 and 16.5; 16 x 8 beams bf16, 8192
// tokens 13.0 and 16.4, 16384 18.1 and 16.4; 600 x 4 beams fp32, 8192 tokens 32 and 25.
constexpr int64_t kWholeElements = 4096;  // of a wave
constexpr int64_t kWholeGroups = 256;
BeamPlan plan_beam_select(int dtype, int64_t groups, int32_t beams, int64_t vocab, int32_t k) {
    const int64_t each = dtype == RTS_F32 ? group_elements<float>() : group_elements<uint16_t>();
    const int64_t rows = groups * beams, all = (vocab + each - 1) / each;
    BeamPlan p;
    p.each = beams <= 4 ? 4 : beams <= 8 ? 2 : beams <= 16 ? 1 : 0;
    if (p.each && groups <= kWholeGroups && vocab <= kWholeElements * p.each) return BeamPlan{all, 1, 0, p.each};
    p.each = 0;
    // Three workgroups a CU: 256 x 102400 bf16 takes 19.7 us with 768 of them, 20.5 with 512, 21.3 with
    // 1024 and 24 with 1536; 512 x 102400 fp32 45.8, 44.5, 45.9 and 48.
    int64_t pieces = (768 + rows - 1) / rows;
    const int64_t most = (all + kBeamWaves - 1) / kBeamWaves;
    pieces = pieces < most ? pieces : most;
    p.piece_groups = (all + pieces - 1) / pieces;
    p.pieces = (int)((all + p.piece_groups - 1) / p.piece_groups);
    p.ws_bytes = (size_t)(rows * p.pieces) * ((size_t)k * sizeof(uint64_t) + kBeamWaves * sizeof(PieceStat));
    return p;
}

template <typename T>
static int launch_beam(const BeamArgs& a, const BeamPlan& plan, void* workspace, hipStream_t s) {
    if (plan.each) {
        const dim3 grid((unsigned)a.groups), block(kMaxJoinWaves * kWave);
        if (plan.each == 4) hipLaunchKernelGGL((beam_group_kernel<T, 4>), grid, block, 0, s, a);
        else if (plan.each == 2) hipLaunchKernelGGL((beam_group_kernel<T, 2>), grid, block, 0, s, a);
        else hipLaunchKernelGGL((beam_group_kernel<T, 1>), grid, block, 0, s, a);
        return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
    }
    const int64_t units = a.groups * a.beams * plan.pieces;
    uint64_t* lists = static_cast<uint64_t*>(workspace);
    PieceStat* stats = reinterpret_cast<PieceStat*>(lists + units * a.k);
    hipLaunchKernelGGL(beam_scan_kernel<T>, dim3((unsigned)(a.groups * a.beams), plan.pieces),
                       dim3(kBeamBlock), 0, s, a, plan.piece_groups, lists, stats);
    if (hipGetLastError() != hipSuccess) return RTS_EHIP;
    const int waves = a.beams < kMaxJoinWaves ? a.beams : kMaxJoinWaves;
    hipLaunchKernelGGL(beam_join_kernel<T>, dim3((unsigned)a.groups), dim3(waves * kWave), (size_t)(waves + a.beams) * 64 * 8, s,
                       a, plan.pieces, lists, stats);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

int launch_beam_select(const BeamArgs& a, const BeamPlan& plan, void* workspace, hipStream_t s) {
    return a.dtype == RTS_F32 ? launch_beam<float>(a, plan, workspace, s)
                              : launch_beam<uint16_t>(a, plan, workspace, s);
}

}  // namespace rts
