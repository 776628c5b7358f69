// Attention over a latent cache (one vector a token is every head's key, its
// leading part every head's value), over selected rows or whole paged
// prefixes, and the join of partial results, for gfx950.
#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

constexpr int kRope = 64;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;

__device__ __forceinline__ float bf16_f32(uint16_t b) { return __uint_as_float((uint32_t)b << 16); }
__device__ __forceinline__ uint16_t f32_bf16(float f) {
    const __bf16 b = (__bf16)f;  // round to nearest even
    return __builtin_bit_cast(uint16_t, b);
}

// The request of token t: the last i with starts[i] <= t (reqs if t is behind
// the last token).
__device__ __forceinline__ int64_t request_of(const int32_t* starts, int64_t reqs, int64_t t) {
    if (t >= starts[reqs]) return reqs;
    int64_t lo = 0, hi = reqs;
    while (hi - lo > 1) {
        const int64_t mid = (lo + hi) >> 1;
        if (starts[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

// One wave per (row, head): lane l holds elements l + 64 i of the query and of
// the sum, and the running maximum and sum of the softmax.
template <int DL>
__global__ __launch_bounds__(64) void latent_attend_simple_kernel(AttendArgs a) {
    constexpr int NQ = (DL + kRope) / 64, NV = DL / 64;
    const int64_t row = blockIdx.x / a.heads;
    const int head = blockIdx.x % a.heads, lane = threadIdx.x;
    int64_t n, ctx = 0, idx = 0, req = 0, news = 0;
    if (!a.paged) {
        n = a.k;
        if (a.counts) n = a.counts[row] < 0 ? 0 : a.counts[row] < n ? a.counts[row] : n;
    } else {
        req = request_of(a.query_starts, a.reqs, row);
        if (req >= a.reqs) return;
        ctx = a.ctx_lens[req] > 0 ? a.ctx_lens[req] : 0;
        idx = row - a.query_starts[req];
        news = a.query_starts[req + 1] - a.query_starts[req];
        n = ctx + news;
    }
    float q[NQ], o[NV], m = -INFINITY, l = 0.f;
    for (int i = 0; i < NQ; ++i) q[i] = bf16_f32(a.q[row * a.ld_q + head * a.ld_head + lane + 64 * i]);
    for (int i = 0; i < NV; ++i) o[i] = 0.f;
    for (int64_t j = 0; j < n; ++j) {
        int64_t r;
        if (!a.paged) {
            r = a.ids[row * a.ld_ids + j];
            if (r >= a.cache_rows) r = -1;
        } else {
            const int64_t d = j - ctx;
            if (d >= 0 && (a.tree ? d >= 64 || !((a.tree[row] >> d) & 1) : d > idx)) continue;
            r = phys_row(a.pages, a.pages.table + req * a.pages.ld, (int32_t)j);
        }
        if (r < 0) continue;
        const uint16_t* c = a.cache + r * a.ld_cache;
        float x[NQ], z = 0.f;
        for (int i = 0; i < NQ; ++i) {
            x[i] = bf16_f32(c[lane + 64 * i]);
            z += q[i] * x[i];
        }
        for (int s = 32; s > 0; s >>= 1) z += __shfl_xor(z, s);
        z *= a.scale * kLog2e;
        const float mn = fmaxf(m, z), f = m == -INFINITY ? 0.f : exp2f(m - mn), p = exp2f(z - mn);
        l = l * f + p;
        for (int i = 0; i < NV; ++i) o[i] = o[i] * f + p * x[i];
        m = mn;
    }
    const int64_t at = row * a.heads + head;
    for (int i = 0; i < NV; ++i)
        a.out[at * DL + lane + 64 * i] = f32_bf16(l == 0.f ? 0.f : o[i] / l);
    if (a.lse && lane == 0) a.lse[at] = l == 0.f ? -INFINITY : (m + log2f(l)) * kLn2;
}

AttendPlan plan_attend_rows(int64_t rows, int32_t heads, int32_t d_latent, int32_t k, bool allow_split) {
    return AttendPlan{1, 0};
}

AttendPlan plan_attend_paged(int64_t tokens, int64_t reqs, int32_t heads, int32_t d_latent,
                             int64_t max_len, bool allow_split) {
    return AttendPlan{1, 0};
}

int launch_latent_attend(const AttendArgs& a, const AttendPlan& plan, void* workspace, hipStream_t s) {
    const dim3 g((unsigned)(a.rows * a.heads)), b(64);
    if (a.d_latent == 512)
        hipLaunchKernelGGL(latent_attend_simple_kernel<512>, g, b, 0, s, a);
    else
        hipLaunchKernelGGL(latent_attend_simple_kernel<256>, g, b, 0, s, a);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

// --------------------------------------------------------------- rank merge

typedef float f32x8 __attribute__((ext_vector_type(8)));

__device__ __forceinline__ f32x8 load8(const float* p) {
    const float4 x = reinterpret_cast<const float4*>(p)[0], y = reinterpret_cast<const float4*>(p)[1];
    return f32x8{x.x, x.y, x.z, x.w, y.x, y.y, y.z, y.w};
}
__device__ __forceinline__ f32x8 load8(const uint16_t* p) {
    const uint4 x = *reinterpret_cast<const uint4*>(p);
    f32x8 r;
    const uint32_t w[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        r[2 * i] = __uint_as_float(w[i] << 16);
        r[2 * i + 1] = __uint_as_float(w[i] & 0xFFFF0000u);
    }
    return r;
}
__device__ __forceinline__ void store8(float* p, f32x8 v) {
    reinterpret_cast<float4*>(p)[0] = float4{v[0], v[1], v[2], v[3]};
    reinterpret_cast<float4*>(p)[1] = float4{v[4], v[5], v[6], v[7]};
}
__device__ __forceinline__ void store8(uint16_t* p, f32x8 v) {
    uint32_t w[4];
#pragma unroll
    for (int i = 0; i < 4; ++i)
        w[i] = (uint32_t)f32_bf16(v[2 * i]) | ((uint32_t)f32_bf16(v[2 * i + 1]) << 16);
    *reinterpret_cast<uint4*>(p) = uint4{w[0], w[1], w[2], w[3]};
}

// out = sum_r e^(lse_r - lse) parts_r.  One thread per 8 elements of one
// (row, head), so each part is read once in 16-byte loads and nothing passes
// between threads; the world statistics are re-read by the dim / 8 threads of
// a (row, head) from the caches.
template <typename In, typename Out>
__global__ __launch_bounds__(256) void merge_attend_kernel(
    const In* __restrict__ parts, const float* __restrict__ part_lse, int world, int64_t n, int dim8,
    int heads, const int32_t* __restrict__ row_limit, Out* __restrict__ out, float* __restrict__ lse) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * dim8) return;
    const int64_t rh = i / dim8;
    const int d = (int)(i - rh * dim8) * 8;
    if (row_limit && rh / heads >= *row_limit) return;
    float m = -INFINITY;
    for (int r = 0; r < world; ++r) m = fmaxf(m, part_lse[r * n + rh]);
    f32x8 acc = {};
    float total = 0.f;
    if (m > -INFINITY) {
        for (int r = 0; r < world; ++r) {
            const float x = part_lse[r * n + rh];
            if (x == -INFINITY) continue;
            const float w = __builtin_amdgcn_exp2f((x - m) * kLog2e);
            total += w;
            const f32x8 v = load8(parts + (r * n + rh) * dim8 * 8 + d);
#pragma unroll
            for (int e = 0; e < 8; ++e) acc[e] = fmaf(w, v[e], acc[e]);
        }
        const float inv = 1.f / total;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= inv;
    }
    store8(out + rh * dim8 * 8 + d, acc);
    if (lse && d == 0) lse[rh] = m > -INFINITY ? m + __builtin_amdgcn_logf(total) * kLn2 : m;
}

int launch_merge_attend(const void* parts, int dtype, const float* part_lse, int32_t world, int64_t rows,
                        int32_t heads, int32_t dim, void* out, int out_dtype, float* lse,
                        const int32_t* row_limit, hipStream_t s) {
    const int64_t n = rows * heads, blocks = (n * (dim / 8) + 255) / 256;
    if (blocks > 0x7FFFFFFFll) return RTS_EUNSUPPORTED;
    const dim3 g((unsigned)blocks), b(256);
    const int d8 = dim / 8;
    const float* pf = static_cast<const float*>(parts);
    const uint16_t* ph = static_cast<const uint16_t*>(parts);
    float* of = static_cast<float*>(out);
    uint16_t* oh = static_cast<uint16_t*>(out);
    if (dtype == RTS_F32 && out_dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<float, float>), g, b, 0, s, pf, part_lse, world, n, d8, heads, row_limit, of, lse);
    else if (dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<float, uint16_t>), g, b, 0, s, pf, part_lse, world, n, d8, heads, row_limit, oh, lse);
    else if (out_dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<uint16_t, float>), g, b, 0, s, ph, part_lse, world, n, d8, heads, row_limit, of, lse);
    else
        hipLaunchKernelGGL((merge_attend_kernel<uint16_t, uint16_t>), g, b, 0, s, ph, part_lse, world, n, d8, heads, row_limit, oh, lse);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

}  // namespace rts
