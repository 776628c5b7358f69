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
// those tokens.  Both operands are cut into 16-byte chunks by the same rule,
// chunk 2 i + (lane >> 5) of a row being step i's: the order of a row's
// elements within the product does not matter as long as both sides share it.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));
typedef int i32x8 __attribute__((ext_vector_type(8)));

constexpr int kLogitsWaves = 4;
constexpr int kLogitsBlock = kLogitsWaves * kWave;
constexpr int kKeyTile = 64;  // keys of a wave's step: two 32-column tiles

// acc += the product over step i's chunks of a 32-head tile and a 32-key tile.
// e4m3 takes two chunks a lane, bf16 one.
template <bool E4M3, int NI>
__device__ __forceinline__ f32x16 tile_product(const i32x4 (&a)[NI], const i32x4 (&k)[NI]) {
    f32x16 acc = {};
    if constexpr (E4M3) {
#pragma unroll
        for (int i = 0; i < NI; i += 2) {
            const i32x8 x = __builtin_shufflevector(a[i], a[i + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            const i32x8 y = __builtin_shufflevector(k[i], k[i + 1], 0, 1, 2, 3, 4, 5, 6, 7);
            acc = __builtin_amdgcn_mfma_scale_f32_32x32x64_f8f6f4(x, y, acc, 0, 0, 0, 0, 0, 0);
        }
    } else {
#pragma unroll
        for (int i = 0; i < NI; ++i)
            acc = __builtin_amdgcn_mfma_f32_32x32x16_bf16(__builtin_bit_cast(bf16x8, a[i]),
                                                          __builtin_bit_cast(bf16x8, k[i]), acc, 0, 0, 0);
    }
    return acc;
}

__device__ __forceinline__ void store_logit(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_logit(uint16_t* p, float v) {
    *p = __builtin_bit_cast(uint16_t, (__bf16)v);  // round to nearest even
}

// NI: 16-byte chunk pairs of a row.  tb tokens a workgroup, head_tiles tiles of
// 32 heads (padded with zeros), `span` columns a workgroup.
template <int NI, bool E4M3, bool PAGED, typename Out>
__global__ __launch_bounds__(kLogitsBlock, 2) void indexer_logits_kernel(LogitsArgs a, int tb, int head_tiles,
                                                                         int64_t span) {
    extern __shared__ __align__(16) char lds[];
    const int tid = threadIdx.x, lane = tid & (kWave - 1), wave = tid / kWave, half = lane >> 5;
    const int64_t t0 = (int64_t)blockIdx.x * tb;
    const int n_tok = (int)(a.rows - t0 < tb ? a.rows - t0 : tb);
    const int hp = head_tiles * 32;
    i32x4* lq = reinterpret_cast<i32x4*>(lds);                       // [tb][head_tiles][NI][64]
    float* lw = reinterpret_cast<float*>(lq + tb * head_tiles * NI * kWave);  // [tb][hp]
    int32_t* le = reinterpret_cast<int32_t*>(lw + tb * hp);          // [tb] row ends
    int32_t* lr = le + tb;                                           // [tb] requests
    constexpr int kRowBytes = NI * 32;
    constexpr int kEsz = E4M3 ? 1 : 2;

    for (int i = tid; i < n_tok * head_tiles * NI * kWave; i += kLogitsBlock) {
        const int l = i & 63, step = (i >> 6) % NI, th = (i >> 6) / NI;
        const int tile = th % head_tiles, tok = th / head_tiles;
        const int head = tile * 32 + (l & 31);
        i32x4 v = {};
        if (head < a.heads)
            v = *reinterpret_cast<const i32x4*>(static_cast<const char*>(a.q) + (t0 + tok) * a.ld_q * kEsz +
                                                (int64_t)head * kRowBytes + (2 * step + (l >> 5)) * 16);
        lq[i] = v;
    }
    for (int i = tid; i < n_tok * hp; i += kLogitsBlock) {
        const int h = i % hp;
        lw[i] = h < a.heads ? a.weights[(t0 + i / hp) * a.ld_weights + h] : 0.f;
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
        for (int64_t c = c0 + wave * kKeyTile; c < cend; c += kLogitsWaves * kKeyTile) {
            i32x4 k[2][NI];
            int64_t phys[2];
#pragma unroll
            for (int u = 0; u < 2; ++u) {
                const int64_t key = c + u * 32 + (lane & 31);
                if constexpr (PAGED)
                    phys[u] = key < cend ? phys_row(a.pages, page, (int32_t)key) : -1;
                else
                    phys[u] = key < cend ? key : -1;
                const char* kp = static_cast<const char*>(a.keys) + phys[u] * a.ld_keys * kEsz + half * 16;
#pragma unroll
                for (int i = 0; i < NI; ++i) {
                    k[u][i] = i32x4{};
                    if (phys[u] >= 0) k[u][i] = *reinterpret_cast<const i32x4*>(kp + i * 32);
                }
            }
            const int64_t mine = half ? phys[1] : phys[0];  // this lane stores column c + lane
            float ks = 1.f;
            if (a.key_scales && mine >= 0) ks = a.key_scales[mine];
            if (mine < 0) ks = __builtin_nanf("");
            for (int t = ta; t < tz; ++t) {
                float sum[2] = {0.f, 0.f};
                for (int tile = 0; tile < head_tiles; ++tile) {
                    const i32x4* qa = lq + (t * head_tiles + tile) * NI * kWave + lane;
                    i32x4 x[NI];
#pragma unroll
                    for (int i = 0; i < NI; ++i) x[i] = qa[i * kWave];
                    const f32x4* w4 = reinterpret_cast<const f32x4*>(lw + t * hp + tile * 32) + half;
                    f32x4 w[4];
#pragma unroll
                    for (int g = 0; g < 4; ++g) w[g] = w4[2 * g];  // heads 8 g + 4 half + (0..3)
#pragma unroll
                    for (int u = 0; u < 2; ++u) {
                        const f32x16 s = tile_product<E4M3, NI>(x, k[u]);
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            sum[u] = fmaf(w[r >> 2][r & 3], __builtin_elementwise_maximum(s[r], 0.f), sum[u]);
                    }
                }
                const float other = __shfl_xor(half ? sum[0] : sum[1], 32);
                const float v = ((half ? sum[1] : sum[0]) + other) * ks;
                if (c + lane < le[t] && c + lane < cend)
                    store_logit(static_cast<Out*>(a.logits) + (t0 + t) * a.ld_logits + c + lane, v);
            }
        }
    }
}

template <int NI, bool E4M3, bool PAGED, typename Out>
static int launch_logits(const LogitsArgs& a, hipStream_t s) {
    const int head_tiles = (a.heads + 31) / 32;
    const size_t per_token = (size_t)head_tiles * NI * kWave * 16 + head_tiles * 32 * 4 + 8;
    int tb = (int)((72 << 10) / per_token);
    if (tb > 16) tb = 16;
    if (PAGED) {  // about the tokens that one request has
        const int64_t each = a.pages.table_rows > 0 ? (a.rows + a.pages.table_rows - 1) / a.pages.table_rows : 1;
        if (tb > each) tb = (int)each;
    }
    if (tb > a.rows) tb = (int)a.rows;
    if (tb < 1) tb = 1;
    const int64_t blocks_x = (a.rows + tb - 1) / tb;
    constexpr int64_t kStep = kLogitsWaves * kKeyTile;
    int64_t parts = (2048 + blocks_x - 1) / blocks_x;
    const int64_t most = (a.cols + kStep - 1) / kStep;
    if (parts > most) parts = most;
    const int64_t span = ((a.cols + parts - 1) / parts + kStep - 1) / kStep * kStep;
    parts = (a.cols + span - 1) / span;
    hipLaunchKernelGGL((indexer_logits_kernel<NI, E4M3, PAGED, Out>),
                       dim3((unsigned)blocks_x, (unsigned)parts), dim3(kLogitsBlock), per_token * tb, s, a, tb,
                       head_tiles, span);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

template <int NI, bool E4M3>
static int launch_logits_as(const LogitsArgs& a, hipStream_t s) {
    if (a.req_id)
        return a.logits_dtype == RTS_F32 ? launch_logits<NI, E4M3, true, float>(a, s)
                                         : launch_logits<NI, E4M3, true, uint16_t>(a, s);
    return a.logits_dtype == RTS_F32 ? launch_logits<NI, E4M3, false, float>(a, s)
                                     : launch_logits<NI, E4M3, false, uint16_t>(a, s);
}

int launch_indexer_logits(const LogitsArgs& a, hipStream_t s) {
    if (a.dtype == RTS_BF16)
        return a.dim == 128 ? launch_logits_as<8, false>(a, s) : launch_logits_as<4, false>(a, s);
    return a.dim == 128 ? launch_logits_as<4, true>(a, s) : launch_logits_as<2, true>(a, s);
}

}  // namespace rts
