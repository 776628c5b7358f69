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
// lanes read them (16 bytes a lane, no bank conflicts), and each of its waves
// streams 64 keys at a time straight into registers, where they serve all
// those tokens while the next 64 are on their way.
//
// e4m3 queries and keys are widened to bf16, which holds every e4m3 value, and
// take the bf16 product: the 8-bit matrix instructions of this chip align the
// products of a step before they add them and lose what lies 2^-16 below the
// largest (1.4e-5 of the result on N(0, 1) data in 64- and 16-element steps
// alike, against 1e-7 here), too much for a select by score.  The queries are
// widened once a workgroup, the keys once for all its tokens.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x2 __attribute__((ext_vector_type(2)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kLogitsWaves = 4;
constexpr int kLogitsBlock = kLogitsWaves * kWave;
constexpr int kKeyTile = 64;  // keys of a wave's step: two 32-column tiles
constexpr int64_t kLogitsStep = kLogitsWaves * kKeyTile;

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

// What a wave holds of its 64 keys: row chunks as they lie in memory (lane
// half h has the 16-byte chunks 2 c + h of its two keys), and the factor of
// the column that this lane stores (NaN: the key does not exist).
template <int NC>
struct Keys {
    i32x4 raw[2][NC];
    float scale;
};

// D elements a row; tb tokens a workgroup, head_tiles tiles of 32 heads
// (padded with zeros), `span` columns a workgroup.
//
// Both operands of product step i cover the same 16 elements of a row in the
// same order, which is all that the sum needs: bf16 step i, half h has chunk
// 2 i + h; e4m3 steps 2 c and 2 c + 1, half h have the halves of chunk 2 c + h.
template <int D, bool E4M3, bool PAGED, typename Out>
__global__ __launch_bounds__(kLogitsBlock, 2) void indexer_logits_kernel(LogitsArgs a, int tb, int head_tiles,
                                                                         int64_t span) {
    constexpr int NI = D / 16;                // product steps
    constexpr int kEsz = E4M3 ? 1 : 2;
    constexpr int NC = D * kEsz / 32;         // chunk pairs of a row
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), half = lane >> 5;
    const int wave = __builtin_amdgcn_readfirstlane(tid / kWave);
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int n_tok = (int)(a.rows - t0 < tb ? a.rows - t0 : tb);
    const int hp = head_tiles * 32;
    i32x4* lq = reinterpret_cast<i32x4*>(lds);                                // [tb][head_tiles][NI][64]
    float* lw = reinterpret_cast<float*>(lq + tb * head_tiles * NI * kWave);  // [tb][hp]
    int32_t* le = reinterpret_cast<int32_t*>(lw + tb * hp);                   // [tb] row ends
    int32_t* lr = le + tb;                                                    // [tb] requests

    for (int th = wave; th < n_tok * head_tiles; th += kLogitsWaves) {
        const int tok = th / head_tiles, head = (th - tok * head_tiles) * 32 + (lane & 31);
        const char* src = static_cast<const char*>(a.q) + ((t0 + tok) * a.ld_q + (int64_t)head * D) * kEsz + half * 16;
        i32x4 raw[NC];
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            raw[c] = i32x4{};
            if (head < a.heads) raw[c] = *reinterpret_cast<const i32x4*>(src + c * 32);
        }
        i32x4* dst = lq + th * NI * kWave + lane;
#pragma unroll
        for (int c = 0; c < NC; ++c) {
            if constexpr (E4M3)
                widen16(raw[c], dst[2 * c * kWave], dst[(2 * c + 1) * kWave]);
            else
                dst[c * kWave] = raw[c];
        }
    }
    for (int i = tid; i < n_tok * hp; i += kLogitsBlock) {
        const int t = i / hp, h = i - t * hp;
        lw[i] = h < a.heads ? a.weights[(t0 + t) * a.ld_weights + h] : 0.f;
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

    const int64_t c0 = (int64_t)blockIdx.y * span;
    // Runs of tokens that share their keys: all of them, or one request's.
    for (int ta = 0, tz; ta < n_tok; ta = tz) {
        int32_t end = le[ta];
        tz = ta + 1;
        while (tz < n_tok && (!PAGED || lr[tz] == lr[ta])) {
            end = le[tz] > end ? le[tz] : end;
            ++tz;
        }
        const int64_t cend = c0 + span < end ? c0 + span : end;
        const int32_t* page = nullptr;
        if constexpr (PAGED) {
            if (end > 0) page = a.pages.table + (int64_t)lr[ta] * a.pages.ld;
        }

        auto load = [&](int64_t c, Keys<NC>& k) {
            int64_t phys[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t key = c + u * 32 + (lane & 31);
                phys[u] = -1;
                if (key < cend) {
                    if constexpr (PAGED)
                        phys[u] = phys_row(a.pages, page, (int32_t)key);
                    else
                        phys[u] = key;
                }
            }
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const char* kp = static_cast<const char*>(a.keys) + phys[u] * a.ld_keys * kEsz + half * 16;
#pragma unroll
                for (int i = 0; i < NC; ++i) {
                    k.raw[u][i] = i32x4{};
                    if (phys[u] >= 0) k.raw[u][i] = *reinterpret_cast<const i32x4*>(kp + i * 32);
                }
            }
            const int64_t mine = half ? phys[1] : phys[0];  // this lane stores column c + lane
            k.scale = mine < 0 ? __builtin_nanf("") : 1.f;
            if (a.key_scales && mine >= 0) k.scale = a.key_scales[mine];
        };

        auto score = [&](int64_t c, const i32x4 (&k)[2][NI], float scale) {
            for (int t = ta; t < tz; ++t) {
                float sum[2] = {0.f, 0.f};
                for (int tile = 0; tile < head_tiles; ++tile) {
                    const i32x4* qa = lq + (t * head_tiles + tile) * NI * kWave + lane;
                    f32x16 s[2] = {};
#pragma unroll
                    for (int i = 0; i < NI; ++i) {
                        const bf16x8 x = __builtin_bit_cast(bf16x8, qa[i * kWave]);
#pragma unroll
                        for (int u = 0; u < 2; ++u)
                            s[u] = __builtin_amdgcn_mfma_f32_32x32x16_bf16(
                                x, __builtin_bit_cast(bf16x8, k[u][i]), s[u], 0, 0, 0);
                    }
                    const f32x4* w4 = reinterpret_cast<const f32x4*>(lw + t * hp + tile * 32) + half;
#pragma unroll
                    for (int g = 0; g < 4; ++g) {
                        const f32x4 w = w4[2 * g];  // heads 8 g + 4 half + (0..3)
#pragma unroll
                        for (int u = 0; u < 2; ++u)
#pragma unroll
                            for (int r = 0; r < 4; ++r)
                                sum[u] = fmaf(w[r], __builtin_elementwise_maximum(s[u][4 * g + r], 0.f), sum[u]);
                    }
                }
                // Both halves' sums of the key tile that this half stores.
                const float other = __shfl_xor(half ? sum[0] : sum[1], 32);
                const float v = ((half ? sum[1] : sum[0]) + other) * scale;
                if (c + lane < le[t] && c + lane < cend)
                    store_logit(static_cast<Out*>(a.logits) + (t0 + t) * a.ld_logits + c + lane, v);
            }
        };

        constexpr int64_t stride = kLogitsStep;
        int64_t c = c0 + wave * kKeyTile;
        if (c >= cend) continue;
        Keys<NC> k0;
        load(c, k0);
        if constexpr (E4M3) {
            for (; c < cend; c += stride) {
                i32x4 k[2][NI];
#pragma unroll
                for (int u = 0; u < 2; ++u)
#pragma unroll
                    for (int i = 0; i < NC; ++i) widen16(k0.raw[u][i], k[u][2 * i], k[u][2 * i + 1]);
                const float scale = k0.scale;
                if (c + stride < cend) load(c + stride, k0);
                score(c, k, scale);
            }
        } else {
            Keys<NC> k1;  // the two take turns, so that no register is copied
            for (;;) {
                if (c + stride < cend) load(c + stride, k1);
                score(c, k0.raw, k0.scale);
                c += stride;
                if (c >= cend) break;
                if (c + stride < cend) load(c + stride, k0);
                score(c, k1.raw, k1.scale);
                c += stride;
                if (c >= cend) break;
            }
        }
    }
}

template <int D, bool E4M3, bool PAGED, typename Out>
static int launch_logits(const LogitsArgs& a, hipStream_t s) {
    const int head_tiles = (a.heads + 31) / 32;
    const size_t per_token = (size_t)head_tiles * D * 64 + head_tiles * 32 * 4 + 8;
    int tb = (int)((72 << 10) / per_token);  // two workgroups a CU
    if (tb > 16) tb = 16;
    if (PAGED) {  // about the tokens that one request has
        const int64_t each = a.pages.table_rows > 0 ? (a.rows + a.pages.table_rows - 1) / a.pages.table_rows : 1;
        if (tb > each) tb = (int)each;
    }
    if (tb > a.rows) tb = (int)a.rows;
    if (tb < 1) tb = 1;
    const int64_t blocks_x = (a.rows + tb - 1) / tb;
    const int64_t steps = (a.cols + kLogitsStep - 1) / kLogitsStep;
    int64_t parts = (512 + blocks_x - 1) / blocks_x;
    if (parts < (steps + 7) / 8) parts = (steps + 7) / 8;
    if (parts > steps) parts = steps;
    if (parts > 65535) parts = 65535;
    const int64_t per = (steps + parts - 1) / parts;
    parts = (steps + per - 1) / per;
    hipLaunchKernelGGL((indexer_logits_kernel<D, E4M3, PAGED, Out>),
                       dim3((unsigned)blocks_x, (unsigned)parts), dim3(kLogitsBlock), per_token * tb, s, a, tb,
                       head_tiles, per * kLogitsStep);
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
