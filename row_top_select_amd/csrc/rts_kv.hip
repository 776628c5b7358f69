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
// A wave has keys of its own, every kKvWaves-th tile of the workgroup's piece, and a
// ring of two tiles in LDS, loaded straight from memory by whole rows; nothing
// passes between waves until the end, where they join their sums through LDS.
// Rows that a token does not see are read from a row of zeros, so that nothing of
// theirs reaches a result.
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
constexpr int kKvWaves = 2;
constexpr int kKvBlock = kKvWaves * kWave;
constexpr int kKvHeads = 16;    // query heads of a workgroup
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

__device__ const uint4 g_zero_kv[512 / 16] = {};  // where rows that are not seen are read from

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

__device__ __forceinline__ uint32_t bf16_pair(float lo, float hi) {
    return (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)lo) | (uint32_t)__builtin_bit_cast(uint16_t, (__bf16)hi) << 16;
}

template <int D, bool E4M3>
__global__ __launch_bounds__(kKvBlock) void kv_attend_kernel(KvArgs a, int splits, int64_t piece_keys,
                                                             float* __restrict__ part_out,
                                                             float* __restrict__ part_lse) {
    using S = KvShape<D, E4M3>;
    constexpr int NK = D / 32, NT = D / 16;  // steps of the first product, tiles of the second
    extern __shared__ __align__(1024) char lds_memory[];
    const int tid = threadIdx.x, lane = tid & 63, g = lane >> 4, col = lane & 15;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const uint32_t ring = lds_address(lds_memory) + wave * S::kWaveB, entries = ring + kKvStages * S::kStageB;

    // blockIdx: key heads, then blocks of 16 query heads, tokens, pieces.
    const int group = a.heads / a.kv_heads, blocks = (group + kKvHeads - 1) / kKvHeads;
    uint32_t rest = blockIdx.x;
    const int kvh = rest % a.kv_heads;
    rest /= a.kv_heads;
    const int block = rest % blocks;
    rest /= blocks;
    const int64_t token = rest % (uint32_t)a.rows;
    const int split = rest / (uint32_t)a.rows;

    const int req = a.req_id[token];
    int end = a.row_ends[token], begin = 0;
    {
        const int64_t held = (int64_t)a.pages.cols * a.pages.block_size;
        if (end > held) end = (int)held;
        if (end < 0 || req < 0 || req >= a.pages.table_rows) end = 0;
        if (a.window > 0 && end > a.window) begin = end - (int)a.window;
    }
    const int64_t seen = end - begin;
    int pieces = 1;
    if (splits > 1 && seen > piece_keys) {
        const int64_t n = (seen + piece_keys - 1) / piece_keys;
        pieces = n < splits ? (int)n : splits;
    }
    if (split >= pieces) return;
    const int p0 = begin + (int)(split * piece_keys);
    const int p1 = split == pieces - 1 ? end : p0 + (int)piece_keys;  // the last has what is left, however much
    const int32_t* const table = a.pages.table + (int64_t)(req < 0 ? 0 : req) * a.pages.ld;
    const int tiles = (p1 - p0) / kKvTile + ((p1 - p0) % kKvTile != 0);
    const int count = (tiles - wave + kKvWaves - 1) / kKvWaves;  // of this wave

    const float factor = a.scale * (a.k_scales ? a.k_scales[kvh] : 1.f);
    const float c = factor == 0.f ? 1.f : fabsf(factor) * kLog2e;
    const float lazy = kLazy / c;

    // The first position of the wave's tile n.  Past the piece's end they may pass 2^31.
    auto tile_at = [&](int n) { return (uint32_t)p0 + ((uint32_t)n * kKvWaves + wave) * kKvTile; };
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
    const int64_t esz = E4M3 ? 1 : 2, ldb = a.ld_cache * esz;
    const char* const keys = static_cast<const char*>(a.k) + kvh * a.ld_head * esz;
    const char* const values = static_cast<const char*>(a.v) + kvh * a.ld_head * esz;
    // Loads tile n into its stage; row: what row_of(n) gives.
    auto fetch = [&](int n, int row) {
        const uint32_t to = ring + (n & (kKvStages - 1)) * S::kStageB;
        const char* from[2][S::kLoads];
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) {
            const int key = i * S::kRowsEach + lane / S::kChunks;
            const int r = __builtin_amdgcn_ds_bpermute(key * 4, row);
            const int chunk = ((lane % S::kChunks) ^ S::swizzle(key)) * 16;
            from[0][i] = (r < 0 ? reinterpret_cast<const char*>(g_zero_kv) : keys + r * ldb) + chunk;
            from[1][i] = (r < 0 ? reinterpret_cast<const char*>(g_zero_kv) : values + r * ldb) + chunk;
        }
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) load_to_lds<16, 0>(from[0][i], to + i * 1024);
#pragma unroll
        for (int i = 0; i < S::kLoads; ++i) load_to_lds<16, 0>(from[1][i], to + S::kHalfB + i * 1024);
    };
    auto exists = [&](int row) { return (uint32_t)__ballot(row >= 0); };

    // The ring is always filled (behind the last tile with zeros), so that the
    // number of loads under way is the same at every tile.
    uint32_t exist = 0, exist_next = 0;  // which keys of tiles n and n + 1 are seen
    if (count > 0) {
        look(0);
        look(1);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        const int first = row_of(0), second = row_of(1);
        fetch(0, first);
        look(2);
        fetch(1, second);
        exist = exists(first);
        exist_next = exists(second);
    }

    // Lane group g holds elements 32 i + 8 g .. + 8 of its query head.
    const int head = kvh * group + block * kKvHeads + col;
    const bool head_ok = block * kKvHeads + col < group;
    bf16x8 q[NK];
    {
        const uint16_t* qp = a.q + token * a.ld_q + (int64_t)head * a.ld_qhead + g * 8;
        const uint32_t flip = factor < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < NK; ++i) {
            i32x4 v = {};
            if (head_ok) v = *reinterpret_cast<const i32x4*>(qp + i * 32);
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
        asm volatile("s_waitcnt vmcnt(%0)" ::"n"(2 * S::kLoads + 1) : "memory");
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
#pragma unroll
            for (int r = 0; r < 8; ++r)
                if (!(see >> ((r >> 2) * 16 + 4 * g + (r & 3)) & 1)) s[r >> 2][r & 3] = -INFINITY;
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
        bf16x8 p;
#pragma unroll
        for (int r = 0; r < 8; ++r) {
            const float x = __builtin_amdgcn_exp2f((s[r >> 2][r & 3] - m) * c);
            l += x;
            p[r] = (__bf16)x;
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
        }
        // The stage is read, and tile n + 2's entries have arrived.
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(2 * S::kLoads) : "memory");
        const int next = row_of(n + 2);
        exist = exist_next;
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
    for (int i = tid; i < kKvHeads * D / 8; i += kKvBlock) {
        const int h = i / (D / 8), d8 = i % (D / 8);
        if (block * kKvHeads + h >= group) break;
        float wm[kKvWaves], wl[kKvWaves], most = kNoMax, total = 0.f;
#pragma unroll
        for (int w = 0; w < kKvWaves; ++w) {
            const float* stat = reinterpret_cast<const float*>(lds_memory + w * S::kWaveB + kKvStages * S::kStageB);
            wm[w] = stat[h];
            wl[w] = stat[16 + h];
            most = fmaxf(most, wm[w]);
        }
        f32x4 sum[2] = {};
#pragma unroll
        for (int w = 0; w < kKvWaves; ++w) {
            const float f = __builtin_amdgcn_exp2f((wm[w] - most) * c);
            total += wl[w] * f;
            const float* from = reinterpret_cast<const float*>(lds_memory + w * S::kWaveB) + h * D;
#pragma unroll
            for (int u = 0; u < 2; ++u) sum[u] += *reinterpret_cast<const f32x4*>(from + ((2 * d8 + u) ^ h) * 4) * f;
        }
        const float inv = total == 0.f ? 0.f : v_scale / total;
        const float lse = total == 0.f ? -INFINITY : most * fabsf(factor) + __builtin_amdgcn_logf(total) * kLn2;
        const int64_t rh = token * a.heads + kvh * group + block * kKvHeads + h;
        if (splits == 1) {
            if (d8 == 0 && a.lse) a.lse[rh] = lse;
            *reinterpret_cast<uint4*>(a.out + rh * D + d8 * 8) =
                uint4{bf16_pair(sum[0][0] * inv, sum[0][1] * inv), bf16_pair(sum[0][2] * inv, sum[0][3] * inv),
                      bf16_pair(sum[1][0] * inv, sum[1][1] * inv), bf16_pair(sum[1][2] * inv, sum[1][3] * inv)};
            continue;
        }
        const int64_t n = a.rows * a.heads, part = split * n + rh;
        const bool empty = total == 0.f && most == kNoMax;  // nothing was seen
        if (d8 == 0) {
            part_lse[part] = total == 0.f && !empty ? kNoMax : lse;  // the join reads its zeros and NaN
            if (split == 0)  // the join sees `splits` parts of every row
                for (int p = pieces; p < splits; ++p) part_lse[p * n + rh] = -INFINITY;
        }
        if (empty) continue;  // the join reads no values of an empty part
        float* const to = part_out + part * D + d8 * 8;
        reinterpret_cast<f32x4*>(to)[0] = sum[0] * inv;
        reinterpret_cast<f32x4*>(to)[1] = sum[1] * inv;
    }
}

KvPlan plan_kv_attend(int64_t rows, int32_t heads, int32_t kv_heads, int32_t dim, int dtype, int64_t max_len,
                      bool allow_split) {
    const int group = heads / kv_heads;
    const int64_t blocks = rows * kv_heads * ((group + kKvHeads - 1) / kKvHeads);
    const int64_t longest = max_len < 0x7FFFFFFF ? max_len : 0x7FFFFFFF;
    KvPlan p{1, longest, 0};
    if (!allow_split) return p;
    // Pieces of about 1024 keys, or as many as it takes to have 1024 workgroups, of 128 keys at least.
    int64_t n = (longest + 1023) / 1024;
    const int64_t fill = (1024 + blocks - 1) / blocks, most = (longest + 127) / 128;
    n = n > fill ? n : fill;
    n = n < most ? n : most;
    n = n < 64 ? n : 64;
    if (n <= 1) return p;
    p.piece = ((longest + n - 1) / n + 63) & ~63ll;
    p.splits = (int)((longest + p.piece - 1) / p.piece);
    if (p.splits <= 1) return KvPlan{1, longest, 0};
    p.ws_bytes = ((size_t)p.splits * rows * heads * (dim + 1) * 4 + 15) & ~size_t(15);
    return p;
}

template <int D, bool E4M3>
static int launch_kv(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t s) {
    const int64_t group = a.heads / a.kv_heads;
    const int64_t grid = a.rows * a.kv_heads * ((group + kKvHeads - 1) / kKvHeads) * plan.splits;
    if (grid > kMaxThreads / kKvBlock) return RTS_EUNSUPPORTED;
    const int64_t n = a.rows * a.heads;
    float* part_out = static_cast<float*>(workspace);
    float* part_lse = part_out ? part_out + (int64_t)plan.splits * n * D : nullptr;
    hipLaunchKernelGGL((kv_attend_kernel<D, E4M3>), dim3((unsigned)grid), dim3(kKvBlock),
                       kKvWaves * (KvShape<D, E4M3>::kWaveB), s, a, plan.splits, plan.piece, part_out, part_lse);
    if (hipGetLastError() != hipSuccess) return RTS_EHIP;
    if (plan.splits == 1) return RTS_OK;
    return launch_merge_attend(part_out, RTS_F32, part_lse, plan.splits, a.rows, a.heads, D, a.out, RTS_BF16, a.lse,
                               nullptr, true, s);
}

int launch_kv_attend(const KvArgs& a, const KvPlan& plan, void* workspace, hipStream_t s) {
    const bool e4m3 = a.dtype == RTS_E4M3;
    if (a.dim == 64) return e4m3 ? launch_kv<64, true>(a, plan, workspace, s) : launch_kv<64, false>(a, plan, workspace, s);
    if (a.dim == 128)
        return e4m3 ? launch_kv<128, true>(a, plan, workspace, s) : launch_kv<128, false>(a, plan, workspace, s);
    return e4m3 ? launch_kv<256, true>(a, plan, workspace, s) : launch_kv<256, false>(a, plan, workspace, s);
}

}  // namespace rts
