// Indexer logits: logits[t, s] = ks[s] * sum_h w[t, h] * max(0, q[t, h] . k[s]),
// over contiguous or paged keys, for gfx950.
//
// A score is a matrix product (heads x dim by dim x keys) with a reduction
// over the heads behind it, 2 * heads * dim operations for 4 bytes written, so
// prompts are bound by the matrix cores and decodes (one token a request) lie
// near the ridge.  The product is formed with the heads as rows and the keys
// as columns of a 32x32 matrix tile: a lane then holds 16 heads of one key, so
// the weighted relu sum runs down the lane's own registers and one swap of the
// wave's halves finishes it; keys never mix, so a key that does not count
// costs no masking.
//
// A workgroup keeps the queries of a few tokens in LDS, in the order in which
// lanes read them (16 bytes a lane, no bank conflicts).  Each of its waves
// streams 64 keys at a time through a ring of its own in LDS into registers,
// where they serve all those tokens.  The ring is loaded straight from memory,
// whole rows next to each other: read into registers at once, as the product
// wants them (16 bytes of 32 rows), the same keys came at 3.4 TB/s whatever the
// number of heads.  16-byte chunks are XOR-ed by the key's number so that the
// reads do not meet in a bank.  Waves wait for their own loads only.
//
// What bounds it: 1024 x 16384 x 64 heads x 128 take 206 us, 1300
// TFLOP/s, more than a large library product reaches; decode of 64 requests
// with 16384 to 32768 e4m3 keys takes 52 us, 4.1 TB/s.
//
// e4m3 queries and keys are widened to bf16, which holds every e4m3 value, and
// take the bf16 product: the 8-bit matrix instructions of this chip align the
// products of a step before they add them and lose what lies 2^-16 below the
// largest (1.4e-5 of the result on N(0, 1) data in 64- and 16-element steps
// alike, against 1e-7 here), too much for a select by score.  The queries are
// widened once a workgroup, the keys once for all its tokens.
#include <type_traits>

#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kKeyTile = 64;  // keys of a wave's step: two 32-column tiles
constexpr int kRingInts = 2;  // steps of block-table entries and of key scales that a wave holds

// Two of the four e4m3 in `w` as bf16 (exact).
template <bool HI>
__device__ __forceinline__ int widen2(int w) {
    return __builtin_bit_cast(int, __builtin_amdgcn_cvt_scalef32_pk_bf16_fp8(w, 1.0f, HI));
}

// 16 e4m3 as the bf16 operands of two product steps.
__device__ __forceinline__ void widen16(i32x4 w, i32x4& lo, i32x4& hi) {
    lo = i32x4{widen2<false>(w[0]), widen2<true>(w[0]), widen2<false>(w[1]), widen2<true>(w[1])};
    hi = i32x4{widen2<false>(w[2]), widen2<true>(w[2]), widen2<false>(w[3]), widen2<true>(w[3])};
}

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}

// What stands in for the keys of an empty cache; the factors of keys without
// scales and of keys that do not exist.
__device__ const uint4 g_no_key[256 / 16] = {};
__device__ const float g_key_factor[2] = {1.f, __builtin_nanf("")};

// Sizes of one kernel.
template <int D, bool E4M3>
struct LogitsShape {
    static constexpr int kEsz = E4M3 ? 1 : 2;
    static constexpr int kRowB = D * kEsz;         // bytes of a key
    static constexpr int NI = D / 16;              // product steps
    static constexpr int NC = kRowB / 32;          // 16-byte chunk pairs of a key
    static constexpr int kStageB = kKeyTile * kRowB;
    static constexpr int kLoads = kStageB / 1024 + 1;  // of a stage: rows and scales
    // 64 keys of 256 bytes in a ring and 64 registers of them: half the waves.
    static constexpr int kWaves = kRowB == 256 ? 4 : 8;
    static constexpr int kStep = kWaves * kKeyTile;
    static constexpr int ring_bytes(int stages) {
        return kWaves * (stages * kStageB + 2 * kRingInts * kKeyTile * 4);
    }
};

// D elements a row; tb tokens a workgroup, head_tiles tiles of 32 heads, `span`
// columns a workgroup, `stages` (1 or 2) of the waves' rings.
//
// The heads that fill up the last tile are copies of the last head with 2^-64
// of its weight (never 0 unless the weight is): their 31 parts at most are lost
// in the first rounding of the last head's, and a key's infinity stays one,
// which zeros in the queries or in the weights would turn into NaN.
//
// Both operands of product step i cover the same 16 elements of a row in the
// same order, which is all that the sum needs: bf16 step i, half h has chunk
// 2 i + h; e4m3 steps 2 c and 2 c + 1, half h have the halves of chunk 2 c + h.
template <int D, bool E4M3, bool PAGED, typename Out>
__global__ __launch_bounds__((LogitsShape<D, E4M3>::kWaves * kWave), 1) void indexer_logits_kernel(
    LogitsArgs a, int tb, int head_tiles, int64_t span, int stages) {
    using S = LogitsShape<D, E4M3>;
    constexpr int NI = S::NI, NC = S::NC, kEsz = S::kEsz, kBlock = S::kWaves * kWave;
    constexpr int NCH = S::kRowB / 16;               // chunks of a row
    constexpr int kPairRows = 16 / NCH;              // rows in 256 bytes of LDS
    extern __shared__ __align__(1024) char lds_memory[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int n_tok = (int)(a.rows - t0 < tb ? a.rows - t0 : tb);
    const int hp = head_tiles * 32;
    char* ring_memory = lds_memory + wave * (S::ring_bytes(stages) / S::kWaves);
    const uint32_t ring = lds_address(ring_memory);                    // [stages][64 keys]
    const uint32_t entries = ring + stages * S::kStageB;               // [kRingInts][64]
    const uint32_t scales = entries + kRingInts * kKeyTile * 4;        // [kRingInts][64]
    i32x4* lq = reinterpret_cast<i32x4*>(lds_memory + S::ring_bytes(stages));  // [tb][head_tiles][NI][64]
    float* lw = reinterpret_cast<float*>(lq + tb * head_tiles * NI * kWave);   // [tb][hp]
    int32_t* le = reinterpret_cast<int32_t*>(lw + tb * hp);                    // [tb] row ends
    int32_t* lr = le + tb;                                                     // [tb] requests

    for (int th = wave; th < n_tok * head_tiles; th += S::kWaves) {
        const int tok = th / head_tiles, row = (th - tok * head_tiles) * 32 + (lane & 31);
        const int head = row < a.heads ? row : a.heads - 1;
        const char* src = static_cast<const char*>(a.q) + ((t0 + tok) * a.ld_q + (int64_t)head * D) * kEsz + half * 16;
        i32x4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) raw[c] = *reinterpret_cast<const i32x4*>(src + c * 32);
        i32x4* dst = lq + th * NI * kWave + lane;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (E4M3)
                widen16(raw[c], dst[2 * c * kWave], dst[(2 * c + 1) * kWave]);
            else
                dst[c * kWave] = raw[c];
        }
    }
    for (int i = tid; i < n_tok * hp; i += kBlock) {
        const int t = i / hp, h = i - t * hp, last = a.heads - 1;
        const float w = a.weights[(t0 + t) * a.ld_weights + (h < last ? h : last)];
        const float part = ldexpf(w, -64);
        lw[i] = h <= last ? w : part != 0.f || w == 0.f ? part : copysignf(1e-45f, w);
    }
    if (tid < n_tok) {
        const int64_t e = a.row_ends ? a.row_ends[t0 + tid] : a.cols;
        int32_t end = (int32_t)(e < 0 ? 0 : e < a.cols ? e : a.cols);
        if constexpr (PAGED) {
            const int32_t r = a.req_id[t0 + tid];
            lr[tid] = r;
            if (r < 0 || r >= a.pages.table_rows) end = 0;
        }
        le[tid] = end;
    }
    __syncthreads();

    const int ends = le[lane < n_tok ? lane : 0];  // lane t: of token t
    // An empty cache is never read: its keys do not exist, and row 0 is zeros.
    const bool no_keys = PAGED && a.pages.cache_rows == 0;
    const char* keys = no_keys ? reinterpret_cast<const char*>(g_no_key) : static_cast<const char*>(a.keys);
    const uint32_t ld_bytes = (uint32_t)(a.ld_keys * kEsz);
    const int64_t c0 = (int64_t)blockIdx.y * span;
    // Runs of tokens that share their keys: all of them, or one request's.
    for (int ta = 0, tz; ta < n_tok; ta = tz) {
        int32_t end = le[ta];
        tz = ta + 1;
        while (tz < n_tok && (!PAGED || lr[tz] == lr[ta])) {
            end = le[tz] > end ? le[tz] : end;
            ++tz;
        }
        end = __builtin_amdgcn_readfirstlane(end);
        tz = __builtin_amdgcn_readfirstlane(tz);
        const int64_t cend = c0 + span < end ? c0 + span : end;
        const int64_t first = c0 + wave * kKeyTile;  // this wave's first column
        if (first >= cend) continue;
        const int steps = (int)((cend - first + S::kStep - 1) / S::kStep);
        const int32_t* page = reinterpret_cast<const int32_t*>(g_no_key);
        uint32_t last_block = 0;
        if constexpr (PAGED) {
            if (a.pages.cols > 0) {
                page = a.pages.table + (int64_t)lr[ta] * a.pages.ld;
                last_block = (uint32_t)(a.pages.cols - 1);
            }
        }

        // Reads the block-table entries of step n's keys, one a lane.
        auto look = [&](int n) {
            if constexpr (PAGED) {
                const int64_t key = first + (int64_t)n * S::kStep + lane;
                uint32_t at = block_of(a.pages, (uint32_t)(key < cend ? key : cend - 1));
                at = at < last_block ? at : last_block;
                load_to_lds<4, 0>(reinterpret_cast<const char*>(page) + (uint64_t)at * 4,
                                  entries + (n & (kRingInts - 1)) * (kKeyTile * 4));
            }
        };
        // Starts the loads of step n's keys and their factors.  A key that does
        // not exist has row 0 in its place and the factor NaN; behind the last
        // column the last key, whose scores are not stored.
        auto fetch = [&](int n) {
            int lane = tid & (kWave - 1);
            asm volatile("" : "+v"(lane));  // offsets are formed here and not kept in registers
            const int64_t key = first + (int64_t)n * S::kStep + lane;
            int row = (int)(key < cend ? key : cend - 1);
            const char* factor = reinterpret_cast<const char*>(g_key_factor);
            if constexpr (PAGED) {
                const int entry = lds_read<int>(entries + (n & (kRingInts - 1)) * (kKeyTile * 4) + lane * 4);
                row = phys_row(a.pages, entry, (uint32_t)row);
                if (row < 0) factor = reinterpret_cast<const char*>(g_key_factor + 1);
            }
            if (a.key_scales && row >= 0) factor = reinterpret_cast<const char*>(a.key_scales + row);
            row = row < 0 ? 0 : row;
            // This lane loads a chunk of key i * (64 / NCH) + lane / NCH.
            int rows[S::kStageB / 1024];
#pragma unroll
            for (int i = 0; i < S::kStageB / 1024; ++i) {
                if constexpr (PAGED) {
                    rows[i] = __shfl(row, i * (64 / NCH) + lane / NCH);
                } else {
                    const int64_t k = first + (int64_t)n * S::kStep + i * (64 / NCH) + lane / NCH;
                    rows[i] = (int)(k < cend ? k : cend - 1);
                }
            }
            load_to_lds<4, 0>(factor, scales + (n & (kRingInts - 1)) * (kKeyTile * 4));
            const uint32_t stage = ring + (stages == 2 ? (n & 1) * S::kStageB : 0);
#pragma unroll
            for (int i = 0; i < S::kStageB / 1024; ++i) {
                const int k = i * (64 / NCH) + lane / NCH;
                const int chunk = (lane % NCH) ^ ((k / kPairRows) & (NCH - 1));
                load_to_lds<16, 0>(keys + (uint64_t)(uint32_t)rows[i] * ld_bytes + chunk * 16, stage + i * 1024);
            }
        };
        // Step n's keys have arrived; those of a later step may be under way.
        auto arrive = [&](bool later) {
            if (later)
                asm volatile("s_waitcnt vmcnt(%0)" ::"n"(S::kLoads) : "memory");
            else
                asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
        };
        // Chunk 2 c + half of key u * 32 + lane % 32.
        auto read_key = [&](int n, int u, int c) {
            const int k = lane & 31;
            const uint32_t at = ring + (stages == 2 ? (n & 1) * S::kStageB : 0) + u * 32 * S::kRowB + k * S::kRowB;
            return lds_read<i32x4>(at + (((2 * c + half) ^ ((k / kPairRows) & (NCH - 1))) * 16));
        };

        // Entries are two steps deep: those of a step are asked for when the
        // step before has used its place, and before the keys that may still be
        // under way when they are needed.
        look(0);
        look(1);
        if constexpr (PAGED) arrive(false);
        fetch(0);
        if (stages == 2) {
            look(2);
            if (steps > 1) fetch(1);
        }

        // The items of a wave's work are (step, token, head tile), in that order.
        // A turn forms the products of one item while the weighted sum of the
        // item before it is taken, so that the matrix unit and the vector unit
        // both have work in one wave.  Queries and weights are re-read for the
        // item after as soon as their registers are used.
        const int item0 = ta * head_tiles, items = (tz - ta) * head_tiles;
        i32x4 x[NI];
        f32x4 w[4];
        f32x16 even[2] = {}, odd[2] = {};  // the scores of every other item
        float sum[2] = {0.f, 0.f};
        auto read_x = [&](int item, int i) { x[i] = lq[((item0 + item) * NI + i) * kWave + lane]; };
        auto read_w = [&](int item, int g) {  // heads 8 g + 4 half + (0..3) of the item's tile
            w[g] = *(reinterpret_cast<const f32x4*>(lw + (item0 + item) * 32) + half + 2 * g);
        };
#pragma unroll
        for (int i = 0; i < NI; ++i) read_x(0, i);
#pragma unroll
        for (int g = 0; g < 4; ++g) read_w(0, g);

        int item = 0, next_item = items > 1 ? 1 : 0;  // whose products are formed; the one after
        int tile = head_tiles - 1, token = tz - 1;    // what is summed: before the first item, nothing
        const int64_t ld_out = a.ld_logits * (int64_t)sizeof(Out);
        char* const out_row = static_cast<char*>(a.logits) + (t0 + ta) * ld_out;
        char* out = out_row;                          // where the wave's 64 columns of the summed token start
        const int limits = ends < (int)cend ? ends : (int)cend;
        int step_c = 0, sum_c = 0x7FFFFFFF;           // first columns: of the step, of what is summed (not stored)
        float step_scale = 0.f, sum_scale = 0.f;
        auto turn = [&](const i32x4 (&k)[2][NI], const f32x16 (&s)[2], f32x16 (&next)[2], auto products) {
            constexpr bool kProducts = decltype(products)::value;
            next[0] = next[1] = f32x16{};
#pragma unroll
            for (int i = 0; i < NI; ++i) {
                if constexpr (kProducts) {
                    const bf16x8 q = __builtin_bit_cast(bf16x8, x[i]);
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        next[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(q, __builtin_bit_cast(bf16x8, k[u][i]),
                                                                          next[u], 0, 0, 0);
                    read_x(next_item, i);
                }
#pragma unroll
                for (int r = i * 16 / NI; r < (i + 1) * 16 / NI; ++r) {
#pragma unroll
                    for (int u = 0; u < 2; ++u)
                        sum[u] = fmaf(w[r >> 2][r & 3], __builtin_elementwise_maximum(s[u][r], 0.f), sum[u]);
                    if (kProducts && (r & 3) == 3) read_w(item, r >> 2);
                }
                __builtin_amdgcn_sched_barrier(0);
            }
            if (++tile < head_tiles) return;
            tile = 0;
            // Both halves' sums of the key tile that this half stores.
            const auto z = __builtin_amdgcn_permlane32_swap(__float_as_uint(sum[0]), __float_as_uint(sum[1]), false,
                                                            false);
            const float v = (__uint_as_float(z[0]) + __uint_as_float(z[1])) * sum_scale;
            if (lane < __builtin_amdgcn_readlane(limits, token) - sum_c)
                store_logit(reinterpret_cast<Out*>(out) + lane, v);
            out += ld_out;
            sum[0] = sum[1] = 0.f;
            if (++token == tz) {  // from here on the items of the step under way are summed
                token = ta;
                sum_c = step_c;
                sum_scale = step_scale;
                out = out_row + step_c * (int64_t)sizeof(Out);
            }
        };
        // All items of the step at column c, two a pass so that no score is copied.
        bool in_odd = false;  // where the scores of the item before are
        auto step = [&](int c, const i32x4 (&k)[2][NI], float scale) {
            step_c = c;
            step_scale = scale;
            auto done = [&] {
                item = next_item;
                next_item = next_item + 1 < items ? next_item + 1 : 0;
            };
            int n = 0;
            if (in_odd) {
                turn(k, odd, even, std::true_type{});
                done();
                ++n;
            }
            for (; n + 1 < items; n += 2) {
                turn(k, even, odd, std::true_type{});
                done();
                turn(k, odd, even, std::true_type{});
                done();
            }
            in_odd = n < items;
            if (in_odd) {
                turn(k, even, odd, std::true_type{});
                done();
            }
        };

        i32x4 k[2][NI];
        for (int n = 0; n < steps; ++n) {
            arrive(stages == 2 && n + 1 < steps);
            const float scale = lds_read<float>(scales + (n & (kRingInts - 1)) * (kKeyTile * 4) + lane * 4);
#pragma unroll
            for (int u = 0; u < 2; ++u)
#pragma unroll
                for (int c = 0; c < NC; ++c) {
                    const i32x4 raw = read_key(n, u, c);
                    if constexpr (E4M3)
                        widen16(raw, k[u][2 * c], k[u][2 * c + 1]);
                    else
                        k[u][c] = raw;
                }
            // The keys are in registers: their place takes those of `stages` steps on.
            asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
            look(n + stages + 1);
            if (n + stages < steps) fetch(n + stages);
            step((int)(first + (int64_t)n * S::kStep), k, scale);
        }
        if (in_odd)
            turn(k, odd, even, std::false_type{});
        else
            turn(k, even, odd, std::false_type{});
        arrive(false);  // entries behind the last step
    }
}

// `reqs`: requests of the paged form, or -1.
template <int D, bool E4M3>
static LogitsPlan plan_logits(int64_t rows, int64_t cols, int32_t heads, int64_t reqs) {
    using S = LogitsShape<D, E4M3>;
    constexpr int kLds = 160 << 10;
    const int head_tiles = (heads + 31) / 32;
    const int per_token = head_tiles * D * 64 + head_tiles * 32 * 4 + 8;
    // Tokens that share keys: all, or about those of one request.
    int64_t want = rows;
    if (reqs >= 0) {
        reqs = reqs < rows ? reqs : rows;
        want = reqs > 0 ? (rows + reqs - 1) / reqs : 1;
    }
    // Two stages of keys where few tokens leave little time for the next one
    // (decode of 64 x 32768 e4m3 keys: 51.9 us, 52.5 us with one).
    const int stages = S::ring_bytes(2) + per_token * want <= kLds ? 2 : 1;
    const int64_t fit = (kLds - S::ring_bytes(stages)) / per_token;
    const int64_t most = want < 16 ? (want < fit ? want : fit) : (fit < 16 ? fit : 16);
    const int64_t steps = (cols + S::kStep - 1) / S::kStep;
    // Tokens a workgroup and columns a workgroup by estimated time: a workgroup
    // takes a CU, 6 us around its steps, 0.5 us a step and kItemUs a head tile
    // of a token in a step (64 keys a wave through the matrix unit).  What
    // matters is that the last round of the 256 CUs is full: 333 x 8191 x 32
    // bf16 takes 28.8 us with 11 tokens a workgroup (248 workgroups), 50.0 us
    // with 5 (268 workgroups); 1024 x 16384 x 64 e4m3 209 us with 4 (256
    // workgroups), 229 us with 2 (512).
    constexpr double kItemUs = (D / 128.0) * (S::kWaves / 4) * 0.25;
    int64_t tb = 1, per = steps;
    double best = 1e300;
    for (int64_t t = 1; t <= most; ++t) {
        const int64_t bx = (rows + t - 1) / t;
        for (int round = 1; round <= 4; ++round) {
            int64_t parts = 256 * round / bx;
            parts = parts < 1 ? 1 : parts > steps ? steps : parts;
            const int64_t p = (steps + parts - 1) / parts;
            const double us = (double)((bx * ((steps + p - 1) / p) + 255) / 256) *
                              (6.0 + p * (0.5 + t * head_tiles * kItemUs));
            if (us < best) best = us, tb = t, per = p;
        }
    }
    return LogitsPlan{(int)tb, stages, S::kStep, per, S::ring_bytes(stages) + per_token * tb};
}

LogitsPlan plan_indexer_logits(int dtype, int64_t rows, int64_t cols, int32_t heads, int32_t dim, int64_t reqs) {
    if (dtype == RTS_BF16)
        return dim == 128 ? plan_logits<128, false>(rows, cols, heads, reqs) : plan_logits<64, false>(rows, cols, heads, reqs);
    return dim == 128 ? plan_logits<128, true>(rows, cols, heads, reqs) : plan_logits<64, true>(rows, cols, heads, reqs);
}

template <int D, bool E4M3, bool PAGED, typename Out>
static int launch_logits(const LogitsArgs& a, hipStream_t s) {
    using S = LogitsShape<D, E4M3>;
    const LogitsPlan p = plan_logits<D, E4M3>(a.rows, a.cols, a.heads, PAGED ? a.pages.table_rows : -1);
    const int64_t span = p.steps * S::kStep;
    const int64_t blocks_x = (a.rows + p.tokens - 1) / p.tokens, parts = (a.cols + span - 1) / span;
    if (blocks_x > kMaxThreads / (S::kWaves * kWave)) return RTS_EUNSUPPORTED;
    hipLaunchKernelGGL((indexer_logits_kernel<D, E4M3, PAGED, Out>),
                       dim3((unsigned)blocks_x, (unsigned)parts), dim3(S::kWaves * kWave), (size_t)p.lds, s, a, p.tokens,
                       (a.heads + 31) / 32, span, p.stages);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

template <int D, bool E4M3>
static int launch_logits_as(const LogitsArgs& a, hipStream_t s) {
    if (a.req_id)
        return a.logits_dtype == RTS_F32 ? launch_logits<D, E4M3, true, float>(a, s)
                                         : launch_logits<D, E4M3, true, uint16_t>(a, s);
    return a.logits_dtype == RTS_F32 ? launch_logits<D, E4M3, false, float>(a, s)
                                     : launch_logits<D, E4M3, false, uint16_t>(a, s);
}

int launch_indexer_logits(const LogitsArgs& a, hipStream_t s) {
    if (a.dtype == RTS_BF16)
        return a.dim == 128 ? launch_logits_as<128, false>(a, s) : launch_logits_as<64, false>(a, s);
    return a.dim == 128 ? launch_logits_as<128, true>(a, s) : launch_logits_as<64, true>(a, s);
}

}  // namespace rts
