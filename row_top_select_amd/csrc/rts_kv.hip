// Attention of new tokens over a paged cache of keys and values, for gfx950.
//
// For a token's 16 query heads of one key head, over the positions that it
// sees, 32 at a time:
//   S^T = K Q^T,  P^T = exp2((S^T - m) c),  O^T += V^T P^T
// in 16x16x32 matrix products, formed transposed: a lane owns one query head (shared
// with the lanes 16, 32 and 48 further on), so its maximum, sum and rescaling
// factor are plain registers, and the weights come out of the first product in
// the registers that the second one reads them from.  A contraction may take
// its terms in any order, so lane group g has keys 4 g + 0..3 and 16 + 4 g + 0..3,
// which the transposing LDS reads deliver of V in the same order.
//
// A wave has keys of its own, every second (or fourth, or eighth) tile of the workgroup's piece, and a
// ring of two tiles in LDS, loaded straight from memory by whole rows; nothing
// passes between waves until the end, where they join their sums through LDS.
// Rows that a token does not see score -inf and their values are cleared in LDS,
// so that nothing of theirs reaches a result.
//
// Weights go into the second product as two bf16 terms, the rounded one and what it
// lost: with one alone the weights' rounding is the larger part of a result's error (2.3e-3
// for 1.7e-3 of its size, which is the rounding of the output itself).
//
// Bound by the reads: 64 requests of up to 16384 positions, 8 key heads of 128, bf16, 567 us
// (5.7 TB/s); three of 131072, 4 key heads, e4m3, 66 us (4.6 TB/s) and the join 6.6.
// Pieces are of one size over all rows, so that the last workgroups end together
// however ragged the contexts are (a number of pieces a row, and offsets in 64 bits,
// took 605 and 88 us with the joins, for 573 and 70).
#include <type_traits>

#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x2 __attribute__((ext_vector_type(2)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kKvTile = 32;     // keys of a stage
constexpr int kKvStages = 2;
constexpr int kKvWaves = 2;     // (1: 64 requests of 16384 positions 584 us for 567, 4 of 2000 11.1 for 11.2)
constexpr int kKvHeads = 16;    // query heads of a workgroup
// Tiles of a piece at least: one a wave.  Kernels, us, with 2, 4 and 8: 4 requests of 2000 positions 11.2, 11.8
// and 12.0; of 3800, 64 elements, 10.2, 10.3 and 10.7.
constexpr int kKvLeast = kKvLeastKeys / kKvTile;
// Tiles of a piece of long contexts.  3 requests of 131072 positions, e4m3, 63 us (24: 74, 96: 62); 64 of
// 16384, bf16, 569 us (24: 570, 96: 572, whose last pieces end later).
constexpr int kKvGoal = 48;
constexpr int kKvRounds = 8;    // pieces a place at most
constexpr int kKvWhole = 9 << 14;
constexpr int kKvEntries = 4;   // tiles of block-table entries that a wave holds
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A maximum before the first score: no finite score is below it, and x - kNoMax is -inf for x = -inf.
constexpr float kNoMax = -3.402823466e38f;
// The next number: a maximum of scores that are all -inf (weights 0, but 0 times what is not finite is NaN).
constexpr float kLeastMax = -3.402823264e38f;
constexpr float kLazy = 8.f;    // how far (log2) a score may pass the maximum before O is rescaled

template <int D, bool E4M3>
struct KvShape {
    static constexpr int kRowB = D * (E4M3 ? 1 : 2);
    static constexpr int kChunks = kRowB / 16;           // of a row, 16 bytes each: lanes that load it
    static constexpr int kRowsEach = kWave / kChunks;    // rows of a load
    static constexpr int kLoads = kKvTile / kRowsEach;   // of a tile's keys, and as many of its values
    static constexpr int kHalfB = kKvTile * kRowB;       // keys or values of a stage
    static constexpr int kStageB = 2 * kHalfB;
    static constexpr int kWaveB = kKvStages * kStageB + kKvEntries * 256;
    // The pattern that a key's chunks are XOR-ed with, so that 16 keys' chunks of the
    // same number lie in different banks.
    static __device__ __forceinline__ int swizzle(int key) {
        return kChunks >= 16 ? key & 15 : kChunks == 8 ? (key >> 1) & 7 : (key >> 2) & 3;
    }
};

// The pieces' results: [part][heads][D], [part][heads] maxima and sums of the softmax, and each row's
// first part and number of pieces.  (Not the sum's logarithm: scores past 3.4e38 have none in 32 bits.)
struct KvParts {
    float* out;
    float2* stat;
    int2* rows;
};

// What turns a product of q and k into a score, and into an exponent of 2.
struct KvFactor {
    float factor, c;
};
__device__ __forceinline__ KvFactor factor_of(float scale, const float* k_scales, int kvh) {
    const float f = scale * (k_scales ? k_scales[kvh] : 1.f);
    return {f, f == 0.f ? 1.f : fabsf(f) * kLog2e};
}
__device__ __forceinline__ float lse_of(const KvFactor& f, float most, float total) {
    return total == 0.f ? -INFINITY : most * fabsf(f.factor) + __builtin_amdgcn_logf(total) * kLn2;
}

__device__ __forceinline__ float wave_sum(float x) {
    return __uint_as_float(wave_reduce32(__float_as_uint(x), [](uint32_t a, uint32_t b) {
        return __float_as_uint(__uint_as_float(a) + __uint_as_float(b));
    }));
}

__device__ const uint4 g_no_row[512 / 16] = {};  // stands in for a cache without rows

// 16 bytes a lane from base + offset to LDS at `to` + 16 * lane; as load_to_lds
// otherwise.  BIG: the offset counts 16 bytes.
template <bool BIG>
__device__ __forceinline__ void load_row(const char* base, uint32_t offset, uint32_t to) {
    if constexpr (BIG) {
        load_to_lds<16, 0>(base + ((uint64_t)offset << 4), to);
    } else {
        asm volatile("s_nop 0\n\tglobal_load_lds_dwordx4 %1, %2" ::"{m0}"(to), "v"(offset), "s"(base) : "memory");
    }
}

__device__ __forceinline__ int kv_widen2(int w, bool hi) {
    return hi ? __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, true))
              : __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, false));
}
// 8 e4m3 as bf16 (exact).
__device__ __forceinline__ bf16x8 kv_widen8(i32x2 w) {
    return __builtin_bit_cast(bf16x8, i32x4{kv_widen2(w[0], false), kv_widen2(w[0], true), kv_widen2(w[1], false),
                                            kv_widen2(w[1], true)});
}

// The largest, and the sum, of what lanes l, l ^ 16, l ^ 32 and l ^ 48 hold.
template <typename Op>
__device__ __forceinline__ float over_groups(float x, Op op) {
    const auto a = __builtin_amdgcn_permlane32_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    x = op(__uint_as_float(a[0]), __uint_as_float(a[1]));
    const auto b = __builtin_amdgcn_permlane16_swap(__float_as_uint(x), __float_as_uint(x), false, false);
    return op(__uint_as_float(b[0]), __uint_as_float(b[1]));
}

__device__ __forceinline__ void lds_write(uint32_t at, i32x4 v) {
    *(__attribute__((address_space(3))) i32x4*)(uintptr_t)at = v;
}

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}

template <int D, bool E4M3, bool BIG, int WAVES>
__global__ __launch_bounds__(WAVES * kWave) void kv_attend_kernel(KvArgs a, int target, int rounds, KvParts parts) {
    using S = KvShape<D, E4M3>;
    constexpr int NK = D / 32, NT = D / 16;  // steps of the first product, tiles of the second
    extern __shared__ __align__(1024) char lds_memory[];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t ring = lds_address(lds_memory) + wave * S::kWaveB, entries = ring + kKvStages * S::kStageB;

    // blockIdx: key heads, then blocks of 16 query heads, then pieces of tokens.
    const int group = a.heads / a.kv_heads, blocks = (group + kKvHeads - 1) / kKvHeads;
    uint32_t rest = blockIdx.x;
    const int kvh = rest % a.kv_heads;
    rest /= a.kv_heads;
    const int block = rest % blocks;
    const int64_t unit = rest / blocks;

    // What a token sees.
    struct Row { int req, begin, end; };
    auto row = [&](int64_t t) {
        Row r{-1, 0, 0};
        if (t >= a.rows) return r;
        const int req = a.req_id[t];
        int end = a.row_ends[t];
        const int64_t held = (int64_t)a.pages.cols * a.pages.block_size;
        if (end < 0 || req < 0 || req >= a.pages.table_rows) end = 0;
        // A window counts back from the row's end, which may lie past its table.
        if (a.window > 0 && end > a.window) r.begin = end - (int)a.window;
        if (end > held) end = (int)held;
        if (r.begin > end) r.begin = end;
        r.req = req;
        r.end = end;
        return r;
    };
    int64_t token = unit;
    Row seen;
    int piece = 0, pieces = 1, part = 0;  // of the token's; its first part's place
    int p0, p1;
    if (target == 0) {
        seen = row(unit);
        p0 = seen.begin, p1 = seen.end;
    } else {
        // Lengths differ and are known here only, so the pieces are of one size for
        // all tokens: one that gives the chip's places (`target` units) a piece each,
        // or more of kKvGoal tiles each, up to `rounds` a place.  A running sum of
        // the tokens' pieces, 64 tokens at a time, says which one this workgroup has.
        const Row of_lane = row(lane);  // the first 64 are read once
        auto rows = [&](int64_t t0) { return t0 == 0 ? of_lane : row(t0 + lane); };
        auto tiles_of = [](const Row& r) { return (r.end - r.begin) / kKvTile + ((r.end - r.begin) % kKvTile != 0); };
        auto count_of = [](int tiles, int chunk) {
            return tiles > chunk ? (int)((uint32_t)(tiles + chunk - 1) / (uint32_t)chunk) : 1;
        };
        float total = 0.f;
        for (int64_t t0 = 0; t0 < a.rows; t0 += kWave) total += wave_sum((float)tiles_of(rows(t0)));
        const float most = total * 1.0001f / (float)(target * rounds);  // more pieces have no room
        float size = total / (float)target;
        size = fmaxf(fminf(size, (float)kKvGoal), fmaxf(most, (float)kKvLeast));
        int chunk = __builtin_amdgcn_readfirstlane((int)fminf(size, 1e9f) + 1);
        // Where a place has one piece, rounding must not leave a few for another round.
        if (size * (float)target > total * 0.75f)
            for (int tries = 0; tries < 4; ++tries) {
                float sum = 0.f;
                for (int64_t t0 = 0; t0 < a.rows; t0 += kWave) {
                    const int tiles = tiles_of(rows(t0));
                    sum += wave_sum(t0 + lane < a.rows ? (float)count_of(tiles, chunk) : 0.f);
                }
                if (sum <= (float)target) break;
                chunk += chunk / 16 + 1;
            }
        uint32_t before = 0, part_before = 0;
        token = -1;
        for (int64_t t0 = 0; t0 < a.rows; t0 += kWave) {
            const Row r = rows(t0);
            const int tiles = tiles_of(r);
            const uint32_t n = t0 + lane >= a.rows ? 0 : count_of(tiles, chunk);
            const uint32_t several = n > 1 ? n : 0;
            const uint32_t upto = wave_incl_scan32(n), part_upto = wave_incl_scan32(several);
            const uint64_t past = __ballot(before + upto > unit);
            if (past) {
                const int at = __builtin_ctzll(past);
                token = t0 + at;
                seen = Row{__builtin_amdgcn_readlane(r.req, at), __builtin_amdgcn_readlane(r.begin, at),
                           __builtin_amdgcn_readlane(r.end, at)};
                pieces = __builtin_amdgcn_readlane(n, at);
                piece = (int)(unit - before - __builtin_amdgcn_readlane(upto - n, at));
                part = part_before + __builtin_amdgcn_readlane(part_upto - several, at);
                break;
            }
            before += __builtin_amdgcn_readlane(upto, kWave - 1);
            part_before += __builtin_amdgcn_readlane(part_upto, kWave - 1);
        }
        if (token < 0) return;
        // Even pieces, in whole tiles.
        const int64_t each = (int64_t)((uint32_t)(tiles_of(seen) + pieces - 1) / (uint32_t)pieces) * kKvTile;
        const int64_t from = seen.begin + piece * each, to = from + each;
        p0 = (int)(from < seen.end ? from : seen.end);
        p1 = (int)(to < seen.end ? to : seen.end);
        if (piece == 0 && kvh == 0 && block == 0 && tid == 0) parts.rows[token] = int2{part, pieces};
    }
    const int head = kvh * group + block * kKvHeads + col;
    const bool head_ok = block * kKvHeads + col < group;
    i32x4 raw_q[NK];  // under way beside what leads to the first tile
    {
        const uint16_t* qp = a.q + token * a.ld_q + (int64_t)(head_ok ? head : kvh * group) * a.ld_qhead + g * 8;
#pragma unroll
        for (int i = 0; i < NK; ++i) raw_q[i] = *reinterpret_cast<const i32x4*>(qp + i * 32);
    }
    const int32_t* const table = a.pages.table + (int64_t)(seen.req < 0 ? 0 : seen.req) * a.pages.ld;
    const int tiles = (p1 - p0) / kKvTile + ((p1 - p0) % kKvTile != 0);
    const int count = __builtin_amdgcn_readfirstlane((tiles - wave + WAVES - 1) / WAVES);  // of this wave

    const KvFactor of = factor_of(a.scale, a.k_scales, kvh);
    const float factor = of.factor, c = of.c;
    const float lazy = kLazy / c;

    // The first position of the wave's tile n.  Past the piece's end they may pass 2^31.
    auto tile_at = [&](int n) { return (uint32_t)p0 + ((uint32_t)n * WAVES + wave) * kKvTile; };
    auto look = [&](int n) {
        uint32_t e = tile_at(n) + (lane & 31);
        e = e < (uint32_t)p1 ? e : (uint32_t)(p1 - 1);
        load_to_lds<4, 0>(reinterpret_cast<const char*>(table) + (uint64_t)block_of(a.pages, e) * 4,
                          entries + (n & (kKvEntries - 1)) * 256);
    };
    // The physical row of key lane % 32 of tile n, negative where there is none.
    auto row_of = [&](int n) {
        const int entry = lds_read<int>(entries + (n & (kKvEntries - 1)) * 256 + (lane & 31) * 4);
        const uint32_t e = tile_at(n) + (lane & 31);
        return n < count && e < (uint32_t)p1 ? phys_row(a.pages, entry, e) : -1;
    };
    constexpr int kEsz = E4M3 ? 1 : 2;
    const bool no_rows = a.pages.cache_rows == 0;
    const char* const keys = no_rows ? reinterpret_cast<const char*>(g_no_row) : static_cast<const char*>(a.k) + kvh * a.ld_head * kEsz;
    const char* const values = no_rows ? reinterpret_cast<const char*>(g_no_row) : static_cast<const char*>(a.v) + kvh * a.ld_head * kEsz;
    const uint32_t row_step = (uint32_t)(a.ld_cache * kEsz / (BIG ? 16 : 1));
    // Loads tile n into its stage; row: what row_of(n) gives.  In place of a row
    // that is not seen comes the cache's first.
    auto fetch = [&](int n, int row) {
        const uint32_t to = ring + (n & (kKvStages - 1)) * S::kStageB, mine = row < 0 ? 0 : (uint32_t)row * row_step;
        uint32_t at[S::kLoads];
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int key = i * S::kRowsEach + lane / S::kChunks;
            const uint32_t chunk = (lane % S::kChunks) ^ S::swizzle(key);
            at[i] = (uint32_t)__builtin_amdgcn_ds_bpermute(key * 4, mine) + chunk * (BIG ? 1 : 16);
        }
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) load_row<BIG>(keys, at[i], to + i * 1024);
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) load_row<BIG>(values, at[i], to + S::kHalfB + i * 1024);
    };
    auto exists = [&](int row) { return (uint32_t)__ballot(row >= 0); };

    // Behind tile n are under way, as long as there is a tile n + 1, the entries of
    // tile n + 2 and the tile n + 1, in this order; behind the last tile nothing that matters.
    uint32_t exist = 0, exist_next = 0;  // which keys of tiles n and n + 1 are seen
    if (count > 0) {
        look(0);
        look(1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const int first = row_of(0), second = row_of(1);
        fetch(0, first);
        if (count > 1) {
            look(2);
            fetch(1, second);
        }
        exist = exists(first);
        exist_next = exists(second);
    }

    // Lane group g holds elements 32 i + 8 g .. + 8 of its query head.
    bf16x8 q[NK];
    {
        const uint32_t flip = factor < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            i32x4 v = head_ok ? raw_q[i] : i32x4{};
            if (factor == 0.f) {  // 0, or NaN for what is not finite
#pragma unroll
                for (int e = 0; e < 4; ++e)
                    v[e] = ((v[e] & 0x7F80) == 0x7F80 ? 0x7FC0 : 0) |
                           ((v[e] & 0x7F800000) == 0x7F800000 ? 0x7FC00000 : 0);
            }
            q[i] = __builtin_bit_cast(bf16x8, v ^ (int)flip);
        }
    }

    f32x4 o[NT] = {};
    float m = kNoMax, l = 0.f;
    for (int n = 0; n < count; ++n) {
        // Tile n has arrived once only what was issued behind it is under way.
        if (n + 1 < count)
            asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * S::kLoads + 1) : "memory");
        else
            asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const uint32_t at = ring + (n & (kKvStages - 1)) * S::kStageB;
        f32x4 s[2] = {};
#pragma unroll
        for (int i = 0; i < NK; ++i)
#pragma unroll
            for (int sub = 0; sub < 2; ++sub) {
                const int key = sub * 16 + col;
                bf16x8 k;
                if constexpr (E4M3) {
                    const int chunk = (2 * i + (g >> 1)) ^ S::swizzle(key);
                    k = kv_widen8(lds_read<i32x2>(at + key * S::kRowB + chunk * 16 + (g & 1) * 8));
                } else {
                    const int chunk = (4 * i + g) ^ S::swizzle(key);
                    k = lds_read<bf16x8>(at + key * S::kRowB + chunk * 16);
                }
                s[sub] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(k, q[i], s[sub], 0, 0, 0);
            }
        const uint32_t see = exist;
        if (see != ~0u) {
            // What is not seen scores -inf, and its values, whatever they are, become 0.
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (!(see >> ((r >> 2) * 16 + 4 * g + (r & 3)) & 1)) s[r >> 2][r & 3] = -INFINITY;
#pragma unroll
            for (int i = 0; i < S::kLoads; ++i)
                if (!(see >> (i * S::kRowsEach + lane / S::kChunks) & 1))
                    lds_write(at + S::kHalfB + i * 1024 + lane * 16, i32x4{0, 0, 0, 0});
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
        }
        float top = s[0][0];
#pragma unroll
        for (int r = 1; r < 8; ++r) top = fmaxf(top, s[r >> 2][r & 3]);
        top = over_groups(top, [](float x, float y) { return fmaxf(x, y); });
        if (see) m = fmaxf(m, kLeastMax);
        if (__any(top > m + lazy)) {
            const float to = fmaxf(m, top);
            const float f = __builtin_amdgcn_exp2f((m - to) * c);
            l *= f;
#pragma unroll
            for (int t = 0; t < NT; ++t) o[t] *= f;
            m = to;
        }
        bf16x8 p, low;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float x = __builtin_amdgcn_exp2f((s[r >> 2][r & 3] - m) * c);
            l += x;
            p[r] = (__bf16)x;
            low[r] = (__bf16)(x - (float)p[r]);
        }
        const uint32_t v_at = at + S::kHalfB;
#pragma unroll
        for (int t = 0; t < NT; ++t) {
            bf16x8 v;
            if constexpr (E4M3) {
                // Each 16 lanes read 8 keys x 16 values and get a value's 8 keys a lane.
                const int i = col >> 1, key = (i >> 2) * 16 + 4 * g + (i & 3);
                const int chunk = t ^ S::swizzle(key);
                typedef __attribute__((address_space(3))) i32x2* lds_i2;
                v = kv_widen8(__builtin_amdgcn_ds_read_tr8_b64_v2i32(
                    (lds_i2)(uintptr_t)(v_at + key * S::kRowB + chunk * 16 + (col & 1) * 8)));
            } else {
                // Each 16 lanes read 4 keys x 16 values and get a value's 4 keys a lane.
                typedef __attribute__((address_space(3))) bf16x4* lds_b4;
                bf16x4 part[2];
#pragma unroll
                for (int sub = 0; sub < 2; ++sub) {
                    const int key = sub * 16 + 4 * g + (col >> 2);
                    const int chunk = (2 * t + ((col & 3) >> 1)) ^ S::swizzle(key);
                    part[sub] = __builtin_amdgcn_ds_read_tr16_b64_v4bf16(
                        (lds_b4)(uintptr_t)(v_at + key * S::kRowB + chunk * 16 + (col & 1) * 8));
                }
                v = __builtin_shufflevector(part[0], part[1], 0, 1, 2, 3, 4, 5, 6, 7);
            }
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, p, o[t], 0, 0, 0);
            o[t] = __builtin_amdgcn_mfma_f32_16x16x32_bf16(v, low, o[t], 0, 0, 0);
        }
        exist = exist_next;
        if (n + 2 >= count) continue;
        // The stage is read, and tile n + 2's entries have arrived.
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * S::kLoads) : "memory");
        const int next = row_of(n + 2);
        exist_next = exists(next);
        look(n + 3);
        fetch(n + 2, next);
    }
    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is loaded into LDS behind this
    l = over_groups(l, [](float x, float y) { return x + y; });

    // The waves join: each leaves its sums in its own ring, 4 values a group,
    // groups XOR-ed with the head.
    float* const mine = reinterpret_cast<float*>(lds_memory + wave * S::kWaveB);
#pragma unroll
    for (int t = 0; t < NT; ++t) *reinterpret_cast<f32x4*>(mine + col * D + ((t * 4 + g) ^ col) * 4) = o[t];
    if (g == 0) {
        float* const stat = reinterpret_cast<float*>(lds_memory + wave * S::kWaveB + kKvStages * S::kStageB);
        stat[col] = m;
        stat[16 + col] = l;
    }
    __syncthreads();
    const float v_scale = a.v_scales ? a.v_scales[kvh] : 1.f;
    for (int i = tid; i < kKvHeads * D / 8; i += WAVES * kWave) {
        const int h = i / (D / 8), d8 = i % (D / 8);
        if (block * kKvHeads + h >= group) break;
        float wm[WAVES], wl[WAVES], most = kNoMax, total = 0.f;
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float* stat = reinterpret_cast<const float*>(lds_memory + w * S::kWaveB + kKvStages * S::kStageB);
            wm[w] = stat[h];
            wl[w] = stat[16 + h];
            most = fmaxf(most, wm[w]);
        }
        f32x4 sum[2] = {};
#pragma unroll
        for (int w = 0; w < WAVES; ++w) {
            const float f = __builtin_amdgcn_exp2f((wm[w] - most) * c);
            total += wl[w] * f;
            const float* from = reinterpret_cast<const float*>(lds_memory + w * S::kWaveB) + h * D;
#pragma unroll
            for (int u = 0; u < 2; ++u) sum[u] += *reinterpret_cast<const f32x4*>(from + ((2 * d8 + u) ^ h) * 4) * f;
        }
        const float inv = total == 0.f ? 0.f : v_scale / total;
        const int64_t rh = token * a.heads + kvh * group + block * kKvHeads + h;
        if (pieces == 1) {
            if (d8 == 0 && a.lse) a.lse[rh] = lse_of(of, most, total);
            *reinterpret_cast<uint4*>(a.out + rh * D + d8 * 8) =
                uint4{bf16_pair(sum[0][0] * inv, sum[0][1] * inv), bf16_pair(sum[0][2] * inv, sum[0][3] * inv),
                      bf16_pair(sum[1][0] * inv, sum[1][1] * inv), bf16_pair(sum[1][2] * inv, sum[1][3] * inv)};
            continue;
        }
        const int64_t at = (int64_t)(part + piece) * a.heads + kvh * group + block * kKvHeads + h;
        if (d8 == 0) parts.stat[at] = float2{most, total};
        if (most == kNoMax) continue;  // nothing was seen: the join reads no values of such a part
        float* const to = parts.out + at * D + d8 * 8;
        reinterpret_cast<f32x4*>(to)[0] = sum[0] * inv;
        reinterpret_cast<f32x4*>(to)[1] = sum[1] * inv;
    }
}

// The join of a row and head's pieces: with maxima m_s and sums l_s of products, and their largest
// maximum m, out = sum_s w_s part_s / sum_s w_s, w_s = 2^((m_s - m) c) l_s.  A
// workgroup takes W elements of one, its threads 4 of them each of every n-th piece,
// with a running maximum: what they read does not wait for anything.  (64 pieces
// of 192 (row, head) pairs, one after the other, took 15 us.)
constexpr int kJoinBlock = 256;

template <int D, int W>
__global__ __launch_bounds__(kJoinBlock) void kv_join_kernel(KvParts parts, int heads, int group, float scale,
                                                             const float* __restrict__ k_scales,
                                                             uint16_t* __restrict__ out, float* __restrict__ lse) {
    constexpr int kColumns = W / 4, kSide = kJoinBlock / kColumns;  // pieces side by side
    __shared__ f32x4 sums[kSide][kColumns];
    __shared__ float totals[kSide], tops[kSide];
    const int64_t rh = blockIdx.x, row = rh / heads;
    const int head = (int)(rh - row * heads);
    const int col = threadIdx.x % kColumns, side = threadIdx.x / kColumns, d = blockIdx.y * W + col * 4;
    const int2 of_row = parts.rows[row];
    const int splits = of_row.y;
    if (splits == 1) return;  // written by its one workgroup
    const KvFactor of = factor_of(scale, k_scales, head / group);
    const int64_t first = (int64_t)of_row.x * heads + head;
    const float2* const stat = parts.stat + first;
    const float* const from = parts.out + first * D + d;
    float m = kNoMax, total = 0.f;  // a piece that saw something has a greater maximum
    f32x4 acc = {};
    constexpr int kAhead = 4;
    for (int s0 = side; s0 < splits; s0 += kSide * kAhead) {
        float2 x[kAhead];
        f32x4 v[kAhead];
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            const int64_t s = s0 + u * kSide < splits ? s0 + u * kSide : side;
            x[u] = stat[s * heads];
            v[u] = *reinterpret_cast<const f32x4*>(from + s * heads * D);
            if (s0 + u * kSide >= splits) x[u].x = kNoMax;
        }
        float top = m;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) top = fmaxf(top, x[u].x);
        if (top == kNoMax) continue;
        const float f = __builtin_amdgcn_exp2f((m - top) * of.c);
        total *= f;
        acc *= f;
        m = top;
#pragma unroll
        for (int u = 0; u < kAhead; ++u) {
            if (x[u].x == kNoMax) continue;  // an empty piece has no values
            const float w = __builtin_amdgcn_exp2f((x[u].x - m) * of.c) * x[u].y;
            total += w;
            acc += v[u] * w;
        }
    }
    sums[side][col] = acc;
    if (col == 0) totals[side] = total, tops[side] = m;
    __syncthreads();
    if (side > 0) return;
    float most = m;
#pragma unroll
    for (int i = 1; i < kSide; ++i) most = fmaxf(most, tops[i]);
    acc = f32x4{};
    total = 0.f;
#pragma unroll
    for (int i = 0; i < kSide; ++i) {
        if (tops[i] == kNoMax) continue;
        const float f = __builtin_amdgcn_exp2f((tops[i] - most) * of.c);
        acc += sums[i][col] * f;
        total += totals[i] * f;
    }
    const float inv = total == 0.f ? 0.f : 1.f / total;
    *reinterpret_cast<uint2*>(out + rh * D + d) =
        uint2{bf16_pair(acc[0] * inv, acc[1] * inv), bf16_pair(acc[2] * inv, acc[3] * inv)};
    if (lse && d == 0) lse[rh] = lse_of(of, most, total);
}

// Workgroups of a token.
static int64_t kv_blocks(int32_t heads, int32_t kv_heads) {
    return kv_heads * ((heads / kv_heads + kKvHeads - 1) / kKvHeads);
}
// Waves of a workgroup that has whole rows: as many as have room in a CU where there
// are no more workgroups than CUs.
constexpr int kKvWideMost = 256;
static constexpr int wide_waves(int row_bytes) { return row_bytes <= 128 ? 8 : row_bytes <= 256 ? 4 : kKvWaves; }
static int kv_waves(int64_t workgroups, int row_bytes) {
    return workgroups <= kKvWideMost ? wide_waves(row_bytes) : kKvWaves;
}
// Workgroups of a split call that a CU has room for.
static int kv_places(int32_t dim, int dtype) {
    const int wave_bytes = kKvStages * 2 * kKvTile * dim * (dtype == RTS_E4M3 ? 1 : 2) + kKvEntries * 256;
    return 160 * 1024 / (kKvWaves * wave_bytes);  // by the LDS: 1 to 8
}

bool kv_attend_fits(int64_t rows, int32_t heads, int32_t kv_heads) {
    return rows * kv_blocks(heads, kv_heads) <= kMaxThreads / (kKvWaves * kWave);
}

KvPlan plan_kv_attend(int64_t rows, int32_t heads, int32_t kv_heads, int32_t dim, int dtype, int64_t max_len,
                      bool allow_split) {
    const int64_t blocks = kv_blocks(heads, kv_heads);
    // Rows that a workgroup each has done in the time of the second launch are not split: a step
    // of 64 keys takes two waves 0.7, 1.0 and 1.85 us for 64, 128 and 256 elements, and more waves less.
    // The border is that of eager calls, which wait some 4 us more for the host's second launch; replayed from a
    // graph, calls of few rows gain by a split from about half of it on.  Calls of 4 rows of 32 heads on 8, us,
    // split and whole, eager, then replayed: 128 elements, bf16, four waves 18.5 and 14.2, 10.6 and 11.7 for 768
    // keys, 19.9 and 17.3, 13.2 and 16.3 for 1256, 18.4 and 23.5, 14.5 and 22.5 for 2000; e4m3, eight waves 19.1 and
    // 17.0, 13.0 and 16.1 for 2000; 64 elements, eight waves 18.7 and 18.7, 13.7 and 17.6 for 3000; 256
    // elements, two waves 18.8 and 16.8, 12.7 and 15.4 for 384.  Of 16 rows: 128 elements 20.6 and 18.6, 19.1 and
    // 17.8 for 1256, 27 and 31, 26 and 30 for 2000.
    // Every workgroup of a split call sums up the rows, so calls of very many are not split, either.  Up to some
    // 2048 rows that pays where one is much longer than the others, and costs where they are alike (a caller
    // who knows that gives no workspace).  Replayed, us, split and whole, 1 key head of 128, bf16: one row of
    // 30000 keys among others of 500: of 64 rows 24 and 257, 1024 297 and 539, 2048 300 and 561, 4096 719 and 602;
    // 1000 to 2000 keys: 64 rows 18 and 23, 256 61 and 48, 1024 187 and 152, 4096 981 and 564; 3000 to 6000 keys:
    // 256 rows 123 and 114, 4096 1827 and 1655; 8 key heads, 1000 to 2000: 64 rows 88 and 84, 512 599 and 570.
    const int64_t waves = kv_waves(rows * blocks, dim * (dtype == RTS_E4M3 ? 1 : 2));
    if (!allow_split || max_len <= kKvWhole * (waves + 2) / 4 / (dim + 48) || rows > 4096) return KvPlan{0, 0, 0};
    // The grid has room for what max_len may need: workgroups without a piece take
    // a place for 2 us each.  With 131072 for a bound, 4 rows of 4000 keys take 22 us in place of 17; of 1000, which
    // are split by it, 16.7 in place of 14.1, and 64 of them 56 in place of 48 split and 45 whole (replayed).
    const int64_t tiles = max_len < (1ll << 31) ? (max_len + kKvTile - 1) / kKvTile : 1ll << 26, all = rows * tiles;
    const int64_t places = (256 * kv_places(dim, dtype) + blocks - 1) / blocks, least = (all + kKvLeast - 1) / kKvLeast;
    KvPlan p;
    p.target = (int)(places < least ? places : least);
    const int64_t rounds = (all + kKvGoal * p.target - 1) / (kKvGoal * p.target);
    p.rounds = (int)(rounds < kKvRounds ? rounds : kKvRounds);
    // Rows of several pieces have no more than twice the most of them.
    p.ws_bytes = (size_t)(2 * p.rounds * p.target) * heads * (dim + 2) * 4 + (size_t)rows * 8;
    p.ws_bytes = (p.ws_bytes + 15) & ~size_t(15);
    return p;
}

template <int D, bool E4M3, bool BIG, int WAVES>
static int launch_kv_waves(const KvArgs& a, int64_t grid, const KvPlan& plan, const KvParts& parts, hipStream_t s) {
    if (grid > kMaxThreads / (WAVES * kWave)) return RTS_EUNSUPPORTED;  // never: kv_attend_fits, and fewer rows where split
    hipLaunchKernelGGL((kv_attend_kernel<D, E4M3, BIG, WAVES>), dim3((unsigned)grid), dim3(WAVES * kWave),
                       WAVES * (KvShape<D, E4M3>::kWaveB), s, a, plan.target, plan.rounds, parts);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

template <int D, bool E4M3, bool BIG>
static int launch_kv_of(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t s) {
    const int64_t blocks = kv_blocks(a.heads, a.kv_heads);
    if (plan.target == 0) {
        constexpr int kWide = wide_waves(KvShape<D, E4M3>::kRowB);
        return a.rows * blocks <= kKvWideMost ? launch_kv_waves<D, E4M3, BIG, kWide>(a, a.rows * blocks, plan, KvParts{}, s)
                                            : launch_kv_waves<D, E4M3, BIG, kKvWaves>(a, a.rows * blocks, plan, KvParts{}, s);
    }
    const int64_t most = (int64_t)plan.target * plan.rounds;
    KvParts parts;
    parts.out = static_cast<float*>(workspace);
    parts.stat = reinterpret_cast<float2*>(parts.out + 2 * most * a.heads * D);
    parts.rows = reinterpret_cast<int2*>(parts.stat + 2 * most * a.heads);
    const int rc = launch_kv_waves<D, E4M3, BIG, kKvWaves>(a, (a.rows + most + 1) * blocks, plan, parts, s);
    if (rc != RTS_OK) return rc;
    // Few of them are cut finer, to have more of the chip read the pieces: 8 heads of one
    // request of 131072 positions 7.3 us, 15.8 whole; 32 heads 5.6 both; 128 (4 requests of 2000) 5.0 and 3.9.
    const dim3 pairs((unsigned)(a.rows * a.heads)), block(kJoinBlock);  // split calls: 2^22 pairs at most
    const int group = a.heads / a.kv_heads;
    if (a.rows * a.heads <= 32)
        hipLaunchKernelGGL((kv_join_kernel<D, 32>), dim3(pairs.x, D / 32), block, 0, s, parts, a.heads, group, a.scale,
                           a.k_scales, a.out, a.lse);
    else
        hipLaunchKernelGGL((kv_join_kernel<D, D>), pairs, block, 0, s, parts, a.heads, group, a.scale, a.k_scales, a.out, a.lse);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// Offsets into a cache are held in 32 bits: of bytes, or of 16 bytes where it is
// larger than 4 GB (two more vector instructions a load: 4 requests of 1000 positions 14.0
// and 14.2 us, 64 of 16384 567 and 569).
template <int D, bool E4M3>
static int launch_kv(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t s) {
    const int64_t bytes = a.cache_rows * a.ld_cache * (E4M3 ? 1 : 2);
    if (bytes >> 4 > 0xFFFFFF00ll) return RTS_EUNSUPPORTED;
    return bytes > 0xFFFFF000ll ? launch_kv_of<D, E4M3, true>(a, plan, workspace, s)
                                : launch_kv_of<D, E4M3, false>(a, plan, workspace, s);
}

int launch_kv_attend(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t s) {
    const bool e4m3 = a.dtype == RTS_E4M3;
    if (a.dim == 64) return e4m3 ? launch_kv<64, true>(a, plan, workspace, s) : launch_kv<64, false>(a, plan, workspace, s);
    if (a.dim == 128)
        return e4m3 ? launch_kv<128, true>(a, plan, workspace, s) : launch_kv<128, false>(a, plan, workspace, s);
    return e4m3 ? launch_kv<256, true>(a, plan, workspace, s) : launch_kv<256, false>(a, plan, workspace, s);
}

}  // namespace rts
