// Beam search's selection over beams and vocabulary, for gfx950.
//
// For a group of beams with scores s_b and rows of logits x_b, the k largest of
//   s_b + x_b[v] - lse_b,   lse_b = log sum_v exp x_b[v]
// in two launches.
//
// 1. A wave streams a piece of a row once, in chunks of 512 elements, with the
//    running maximum and sum of the softmax.  A row's order is that of its logits
//    whatever lse_b is, so the piece's k best are found beside it without it: the
//    wave keeps every lane's and every chunk's maximum.  At least k elements reach
//    the k-th largest of the 64 lanes' maxima, so only chunks whose maximum reaches it can
//    hold one of the k best: they are read once more (a few, from the caches)
//    and what reaches the bound is sorted, 64 at a time, into a list of k.
// 2. A workgroup a group joins its rows' pieces and ranks the rows' candidates
//    against each other by their values in 64 bits.
#include <type_traits>

#include "rts_device.hpp"
#include "rts_internal.h"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kBeamBlock = 256;
constexpr int kBeamWaves = kBeamBlock / kWave;
constexpr int kChunk = 512;       // elements: 8 a lane
constexpr int kMaxChunks = 64;    // of a piece: a lane keeps one's maximum
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLeast = -3.402823466e38f;  // the lowest finite number

struct PieceStat {
    float m, sum;
};

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

// A lane's 8 elements of a chunk, as they lie in memory.
template <typename T>
struct Chunk8;
template <>
struct Chunk8<uint16_t> {
    uint4 w[1];
    __device__ __forceinline__ float get(int e) const {
        const uint32_t x[4] = {w[0].x, w[0].y, w[0].z, w[0].w};
        return __uint_as_float(e & 1 ? x[e >> 1] & 0xFFFF0000u : x[e >> 1] << 16);
    }
};
template <>
struct Chunk8<float> {
    uint4 w[2];
    __device__ __forceinline__ float get(int e) const {
        const uint32_t x[8] = {w[0].x, w[0].y, w[0].z, w[0].w, w[1].x, w[1].y, w[1].z, w[1].w};
        return __uint_as_float(x[e]);
    }
};

// 16 bytes at any multiple of 4, or of 2.
typedef uint32_t words_at4 __attribute__((ext_vector_type(4), aligned(4)));
typedef uint32_t words_at2 __attribute__((ext_vector_type(4), aligned(2)));

// Chunk c of a row holds its elements 512 c .. + 512 whatever the row's alignment
// is (loads of 16 bytes take any address), so that equal rows give equal sums.
// Load j of a lane is elements (j * 64 + lane) * kEach .. + kEach of the chunk.
template <typename T>
struct RowReader {
    static constexpr int kEach = 16 / sizeof(T), G = kChunk / kWave / kEach;
    using words = std::conditional_t<sizeof(T) == 4, words_at4, words_at2>;
    const T* row;
    int64_t vocab;
    // The element that a lane's e-th of chunk c is (it may lie behind the row).
    __device__ __forceinline__ int64_t element(int64_t c, int e) const {
        return c * kChunk + (e / kEach * kWave + lane_id()) * kEach + e % kEach;
    }
    __device__ __forceinline__ bool inside(int64_t c) const { return (c + 1) * kChunk <= vocab; }
    __device__ __forceinline__ Chunk8<T> load(int64_t c) const {  // a chunk inside of the row
        Chunk8<T> r;
#pragma unroll
        for (int j = 0; j < G; ++j) {
            const words w = *reinterpret_cast<const words*>(row + element(c, j * kEach));
            r.w[j] = uint4{w[0], w[1], w[2], w[3]};
        }
        return r;
    }
    // The last chunk: what lies behind the row is -inf.
    __device__ __forceinline__ void load_edge(int64_t c, float (&v)[8]) const {
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = element(c, e);
            v[e] = -INFINITY;
            if (at < vocab) {
                if constexpr (sizeof(T) == 4) v[e] = row[at];
                else v[e] = __uint_as_float((uint32_t)row[at] << 16);
            }
        }
    }
    __device__ __forceinline__ void load_any(int64_t c, float (&v)[8]) const {
        if (!inside(c)) return load_edge(c, v);
        const Chunk8<T> x = load(c);
#pragma unroll
        for (int e = 0; e < 8; ++e) v[e] = x.get(e);
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

template <typename T>
__global__ __launch_bounds__(kBeamBlock) void beam_scan_kernel(BeamArgs a, int64_t pieces, int chunks,
                                                               uint64_t* __restrict__ lists,
                                                               PieceStat* __restrict__ stats) {
    __shared__ uint64_t stage_memory[kBeamWaves][2 * kWave];
    const int lane = lane_id();
    const int wave = __builtin_amdgcn_readfirstlane(threadIdx.x / kWave);
    const int64_t unit = (int64_t)blockIdx.x * kBeamWaves + wave;
    const int64_t rows = a.groups * a.beams;
    if (unit >= rows * pieces) return;
    const int64_t r = unit / pieces, piece = unit - r * pieces;
    const RowReader<T> in{static_cast<const T*>(a.logits) + r * a.ld, a.vocab};
    const int64_t c0 = piece * chunks, all = (a.vocab + kChunk - 1) / kChunk;
    const int n = (int)(all - c0 < chunks ? all - c0 : chunks);

    float m = kLeast, sum = 0.f, lane_most = -INFINITY, chunk_most = -INFINITY;
    auto take = [&](const float (&v)[8], int i) {
        float top = v[0];
#pragma unroll
        for (int e = 1; e < 8; ++e) top = fmaxf(top, v[e]);
        lane_most = fmaxf(lane_most, top);
        const float most = wave_max(top);
        if (lane == i) chunk_most = most;
        if (most > m) {
            sum *= __builtin_amdgcn_exp2f((m - most) * kLog2e);
            m = most;
        }
        // The differences are taken first: a rounded m log2(e) would be the same
        // error in every term of a row.
        float part = 0.f;
#pragma unroll
        for (int e = 0; e < 8; ++e) part += __builtin_amdgcn_exp2f((v[e] - m) * kLog2e);
        sum += part;
    };
    constexpr int kAhead = 4;
    for (int i = 0; i < n; i += kAhead) {
        if (i + kAhead <= n && in.inside(c0 + i + kAhead - 1)) {
            Chunk8<T> x[kAhead];
#pragma unroll
            for (int u = 0; u < kAhead; ++u) x[u] = in.load(c0 + i + u);
#pragma unroll
            for (int u = 0; u < kAhead; ++u) {
                float v[8];
#pragma unroll
                for (int e = 0; e < 8; ++e) v[e] = x[u].get(e);
                take(v, i + u);
            }
        } else {
            for (int u = i; u < n && u < i + kAhead; ++u) {
                float v[8];
                in.load_any(c0 + u, v);
                take(v, u);
            }
        }
    }
    {
        double total = sum;
        for (int d = 1; d < kWave; d <<= 1) total += __shfl_xor(total, d);
        if (lane == 0) stats[unit] = PieceStat{m, (float)total};
    }

    // One more than k where the end token may be among them.
    const int need = a.k + (a.eos >= 0 ? 1 : 0);
    uint32_t key[1] = {key32_of_bits(__float_as_uint(lane_most))};
    wave_bitonic_sort<1, true>(key);
    // -inf is no candidate.
    float bound = kLeast;
    if (need <= kWave)
        bound = fmaxf(bound, float_of_key32(__builtin_amdgcn_readlane(key[0], need <= kWave ? need - 1 : 0)));
    uint64_t best = 0;
    uint64_t* const stage = stage_memory[wave];
    int held = 0;
    bool ties = true;  // elements equal to the bound count (they lie before all that set it, or it is no element's)
    auto flush = [&](int count) {  // the first `count` staged entries, 64 at most
        wave_lds_sync();
        uint64_t v[1] = {lane < count ? stage[lane] : 0};
        const uint64_t rest = stage[kWave + lane];
        wave_lds_sync();
        stage[lane] = rest;
        wave_bitonic_sort<1, true>(v);
        merge_sorted(best, v[0]);
        held -= count;
    };
    for (uint64_t left = __ballot(lane < n && chunk_most >= bound); left; left &= left - 1) {
        const int i = __builtin_ctzll(left);
        const float most = __uint_as_float(__builtin_amdgcn_readlane(__float_as_uint(chunk_most), i));
        if (ties ? most < bound : most <= bound) continue;
        float v[8];
        in.load_any(c0 + i, v);
#pragma unroll
        for (int e = 0; e < 8; ++e) {
            const int64_t at = in.element(c0 + i, e);
            const bool in_list = (ties ? v[e] >= bound : v[e] > bound) && at != a.eos;
            const uint64_t mask = __ballot(in_list);
            if (!mask) continue;
            if (in_list) stage[held + mbcnt64(mask)] = composite(key32_of_bits(__float_as_uint(v[e])), (uint32_t)at);
            held += __popcll(mask);
            if (held >= kWave) flush(kWave);
        }
        // Later chunks' elements come after all of this one's: they count if they
        // are larger than the k-th so far.
        const uint64_t kth = readlane64(best, a.k - 1);
        if (kth) {
            const float v_kth = float_of_key32((uint32_t)(kth >> 32));
            if (v_kth >= bound) bound = v_kth, ties = false;
        }
    }
    if (held > 0) flush(held);
    if (lane < a.k) lists[unit * a.k + lane] = best;
}

// The key of a 64-bit value that orders like it; 0 is below all.
__device__ __forceinline__ uint64_t key64(double v) {
    const uint64_t u = (uint64_t)__double_as_longlong(v);
    return u >> 63 ? ~u : u | 1ull << 63;
}

template <typename T>
__global__ __launch_bounds__(kBeamBlock) void beam_join_kernel(BeamArgs a, int64_t pieces,
                                                               const uint64_t* __restrict__ lists,
                                                               const PieceStat* __restrict__ stats) {
    extern __shared__ uint64_t keys[];  // [beams][k] values by rank in their beam, 0: none
    uint32_t* const cols = reinterpret_cast<uint32_t*>(keys + a.beams * a.k);
    float* const values = reinterpret_cast<float*>(cols + a.beams * a.k);
    __shared__ int total;
    const int lane = lane_id(), wave = threadIdx.x / kWave;
    const int64_t group = blockIdx.x;
    if (threadIdx.x == 0) total = 0;
    for (int b = wave; b < a.beams; b += kBeamWaves) {
        const int64_t r = group * a.beams + b;
        // The row's sum: a piece a lane.
        float m = kLeast;
        bool bad = false;
        for (int64_t p = lane; p < pieces; p += kWave) m = fmaxf(m, stats[r * pieces + p].m);
        m = wave_max(m);
        double sum = 0;
        for (int64_t p = lane; p < pieces; p += kWave) {
            const PieceStat s = stats[r * pieces + p];
            sum += (double)s.sum * exp((double)s.m - (double)m);
            bad |= !(s.sum <= 3e38f);
        }
        for (int d = 1; d < kWave; d <<= 1) sum += __shfl_xor(sum, d);
        const float score = a.scores[r];
        // A row without a finite sum (NaN or +inf in it, or -inf only) and a beam
        // without a finite score have no candidates.
        const bool takes_part = !__any(bad) && sum > 0 && fabsf(score) <= 3.402823466e38f;
        const double shift = (double)score - ((double)m + log(sum));
        uint64_t best = lane < a.k ? lists[r * pieces * a.k + lane] : 0;
        for (int64_t p = 1; p < pieces; ++p)
            merge_sorted(best, lane < a.k ? lists[(r * pieces + p) * a.k + lane] : 0);
        const bool there = takes_part && best != 0;
        if (lane < a.k) {
            const double v = shift + (double)float_of_key32((uint32_t)(best >> 32));
            keys[b * a.k + lane] = there ? key64(v) : 0;
            cols[b * a.k + lane] = composite_id(best);
            values[b * a.k + lane] = (float)v;
        }
        if (a.ended && lane == 0) {
            const T* row = static_cast<const T*>(a.logits) + r * a.ld;
            float x;
            if constexpr (sizeof(T) == 4) x = row[a.eos];
            else x = __uint_as_float((uint32_t)row[a.eos] << 16);
            a.ended[r] = takes_part ? (float)(shift + (double)x) : -INFINITY;
        }
        const int n = __popcll(__ballot(there && lane < a.k));
        if (lane == 0) atomicAdd(&total, n);
    }
    __syncthreads();
    // An entry's place: its own rank and, in every other beam, the entries ahead of it.
    for (int e = threadIdx.x; e < a.beams * a.k; e += kBeamBlock) {
        const int b = e / a.k;
        const uint64_t mine = keys[e];
        if (mine == 0) continue;
        int place = e - b * a.k;
        for (int o = 0; o < a.beams && place < a.k; ++o) {
            if (o == b) continue;
            const uint64_t* list = keys + o * a.k;
            const uint64_t ahead = o < b ? mine : mine + 1;  // equal values by ascending beam
            int lo = 0, hi = a.k;  // entries >= ahead
            while (lo < hi) {
                const int mid = (lo + hi) >> 1;
                if (list[mid] >= ahead) lo = mid + 1; else hi = mid;
            }
            place += lo;
        }
        if (place < a.k) {
            const int64_t at = group * a.k + place;
            a.out_scores[at] = values[e];
            a.parents[at] = (int32_t)(group * a.beams + b);
            a.tokens[at] = (int32_t)cols[e];
        }
    }
    for (int i = threadIdx.x; i < a.k; i += kBeamBlock)
        if (i >= total) {
            const int64_t at = group * a.k + i;
            a.out_scores[at] = -INFINITY;
            a.parents[at] = -1;
            a.tokens[at] = -1;
        }
}

BeamPlan plan_beam_select(int dtype, int64_t groups, int32_t beams, int64_t vocab, int32_t k) {
    const int64_t rows = groups * beams, all = (vocab + kChunk - 1) / kChunk;
    int64_t pieces = (2048 + rows - 1) / rows;
    const int64_t most = (all + 3) / 4, least = (all + kMaxChunks - 1) / kMaxChunks;
    pieces = pieces < most ? pieces : most;
    pieces = pieces > least ? pieces : least;
    BeamPlan p;
    p.chunks = (int)((all + pieces - 1) / pieces);
    p.pieces = (all + p.chunks - 1) / p.chunks;
    p.ws_bytes = (size_t)(rows * p.pieces) * ((size_t)k * sizeof(uint64_t) + sizeof(PieceStat));
    return p;
}

template <typename T>
static int launch_beam(const BeamArgs& a, const BeamPlan& plan, void* workspace, hipStream_t s) {
    const int64_t units = a.groups * a.beams * plan.pieces;
    uint64_t* lists = static_cast<uint64_t*>(workspace);
    PieceStat* stats = reinterpret_cast<PieceStat*>(lists + units * a.k);
    hipLaunchKernelGGL(beam_scan_kernel<T>, dim3((unsigned)((units + kBeamWaves - 1) / kBeamWaves)), dim3(kBeamBlock), 0,
                       s, a, plan.pieces, plan.chunks, lists, stats);
    if (hipGetLastError() != hipSuccess) return RTS_EHIP;
    hipLaunchKernelGGL(beam_join_kernel<T>, dim3((unsigned)a.groups), dim3(kBeamBlock), (size_t)a.beams * a.k * 16, s, a,
                       plan.pieces, lists, stats);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

int launch_beam_select(const BeamArgs& a, const BeamPlan& plan, void* workspace, hipStream_t s) {
    return a.dtype == RTS_F32 ? launch_beam<float>(a, plan, workspace, s)
                              : launch_beam<uint16_t>(a, plan, workspace, s);
}

}  // namespace rts
