// Attention over a latent cache (one vector a token is every head's key, its
// leading part every head's value), over selected rows or whole paged
// prefixes, and the join of partial results, for gfx950.
//
// For a block of query rows (heads of a token, or (token, head) pairs of a
// request) over a list of keys, 32 keys at a time:
//   S^T = K Q^T,  P^T = exp2((S^T - m) c),  O^T += V^T P^T
// with K [32, L + 64] in LDS and V its first L columns.  Both products are
// formed transposed, so that a query row is a column of every 32x32 matrix
// tile: a lane owns one query row (shared with the lane 32 further on), its
// maximum, sum and rescaling factor are plain registers, and the weights come
// out of the first product in the very registers that the second one reads
// them from.  A contraction may take its terms in any order, so the second
// product's 16 keys a step are those that the lane half holds (4 h + 0..3 and
// 8 + 4 h + 0..3), and the transposing LDS reads deliver V in the same order.
//
// Q (144 registers) and O (64 to 256 registers) stay in registers; a wave has
// a SIMD's registers for itself.  A workgroup is four waves of 32 query rows x
// all values (HG = 4), 64 rows x half of the values (HG = 2) or 32 rows x a
// quarter (HG = 1): with fewer rows than 128 the scores are formed more than
// once, which costs matrix time where the rows' bytes bound the call.
//
// Key rows come through a ring of four 32-key stages, loaded straight into LDS
// three stages ahead; where a row lies (its id, or its block-table entry) comes
// the same way another two stages ahead.  Waits are counted by hand, one barrier
// a stage.  A stage is stored by 64-element
// columns, [column][key][128 bytes]: a load of 8 keys x 128 bytes is then 64
// lanes in a row, and a lane's nine loads differ by constants only.  A wave has
// eight issue slots a matrix instruction and needs most of them for LDS reads
// and the softmax, so the loads must cost few (with 1024-byte rows and scalar
// address arithmetic they made the loop issue-bound: 33% matrix busy).
// 16-byte chunks of a 128-byte row are XOR-ed by the key's number, so that
// neither the row reads of the first product nor the transposed reads of the
// second meet in a bank.
//
// What bounds it: 1024 tokens x 128 heads x 2048 rows take 565 us, 1040 TFLOP/s
// with the matrix units 52% busy (a large library product reaches 1200 to 1250);
// deeper read-ahead of either operand changes nothing.  A stage takes a CU that
// has the chip for itself 1.12, 1.25 or 1.50 us with one, two or four row groups,
// wherever its rows lie (one row over and over: 1.13 us with one group), and
// 1.44, 1.62 or 1.95 us beside 255 busy CUs (one row over and over: 1.18 us).
// So with few rows three quarters of a stage are the CU's own: every wave reads
// all keys and forms the same scores, 36 of its 44 matrix instructions.  Prompts
// pay that for every token: 1024 x 16 heads x 2048 rows take 406 us.
//
// The maximum m is one of products, before the scale: the difference is taken
// first, so that the greatest weight is 1 for scores of any size (S c - m with
// m = round(max S c) is off by 2^-25 of the score: 2^128 and more past 2^31).
// The running maximum is only moved when a score exceeds it by 2^8: then, and
// not at every step, O is rescaled.  Any reference gives the same quotient; a
// weight of up to 2^8 costs neither the 32-bit sums nor bf16 precision.
#include <type_traits>

#include "rts_device.hpp"
#include "rts_internal.h"
#include "rts_paged.hpp"
#include "../../include/row_top_select.h"

namespace rts {

typedef float f32x16 __attribute__((ext_vector_type(16)));
typedef float f32x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x4 __attribute__((ext_vector_type(4)));
typedef __bf16 bf16x8 __attribute__((ext_vector_type(8)));
typedef int i32x4 __attribute__((ext_vector_type(4)));

constexpr int kRope = 64;
constexpr int kTile = 32;    // keys of a stage, query rows of a wave
constexpr int kStages = 4;
constexpr int kEntryStages = 8;  // of list entries, read two stages further ahead
constexpr int kLeastPiece = 4;   // stages: what lies around a piece takes as long as 5 to 8
constexpr int kAttendWaves = 4;
constexpr int kAttendBlock = kAttendWaves * kWave;
constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
// A maximum before the first score: no finite score is below it, and x - kNoMax is -inf for x = -inf.
constexpr float kNoMax = -3.402823466e38f;
// The next number: a maximum of scores that are all -inf (weights 0, but 0 times what is not finite is NaN).
constexpr float kLeastMax = -3.402823264e38f;
constexpr float kLazy = 8.f;       // how far (log2) a score may pass the maximum before O is rescaled

template <int DL>
constexpr int stage_bytes() { return kTile * (DL + kRope) * 2; }
// Paged form: which values of a stage's keys are not finite, a bit each, and which keys have any.
template <int DL>
constexpr int flaw_bytes() { return kTile * DL / 8 + 16; }

// 0 times 8 bf16: 0, or NaN for what is not finite.
__device__ __forceinline__ i32x4 times_zero(i32x4 v) {
#pragma unroll
    for (int e = 0; e < 4; ++e)
        v[e] = ((v[e] & 0x7F80) == 0x7F80 ? 0x7FC0 : 0) | ((v[e] & 0x7F800000) == 0x7F800000 ? 0x7FC00000 : 0);
    return v;
}

__device__ __forceinline__ uint16_t f32_bf16(float f) {
    return __builtin_bit_cast(uint16_t, (__bf16)f);  // round to nearest even
}

// Where rows that do not exist are read from.
__device__ const uint4 g_zero_row[(512 + kRope) * 2 / 16] = {};

// o += v p with the sums in accumulation registers, where the compiler would
// put them only under pressure and with copies.  It does not see the product,
// so the wait states are here: two after a vector instruction that wrote an
// operand (s_nop 1, in the shadow of the product before), and sums_ready()
// before other code reads the sums.
__device__ __forceinline__ void add_product(f32x16& o, bf16x8 v, bf16x8 p) {
    asm volatile("s_nop 1\n\tv_mfma_f32_32x32x16_bf16 %0, %1, %2, %0" : "+a"(o) : "v"(v), "v"(p));
}
// Keeps a sum in accumulation registers at this point.
__device__ __forceinline__ void pin(f32x16& o) { asm volatile("" : "+a"(o)); }
template <int N>
__device__ __forceinline__ void sums_ready(f32x16 (&o)[N]) {
    asm volatile("s_nop 15\n\ts_nop 7" ::: "memory");
#pragma unroll
    for (int t = 0; t < N; ++t) pin(o[t]);
}

// The 3-bit pattern that a key's chunks are XOR-ed with.  A pair of keys fills
// the banks, so the 8 pairs among 16 keys have patterns of their own (row
// reads), and of any 4 neighbouring pairs two take the upper half of their 128
// bytes (transposed reads of 8 keys x 64 bytes).
__device__ __forceinline__ int chunk_xor(int key) {
    return ((key >> 1) & 1) << 2 | ((key >> 2) & 1) << 1 | ((key >> 3) & 1);
}

// f(integral_constant 0), ..., f(integral_constant N - 1).
template <int N, typename F>
__device__ __forceinline__ void each(F&& f) {
    if constexpr (N > 0) {
        each<N - 1>(f);
        f(std::integral_constant<int, N - 1>{});
    }
}

// Query rows and keys of one workgroup.
struct Work {
    int64_t q0;       // first token
    int32_t head0;    // rows form: first head
    int32_t flat0;    // paged form: first (token, head) pair of the request
    int32_t tokens;   // paged form: the request's tokens
    int32_t ctx;      // paged form: cached tokens
    int32_t n;        // keys
    int32_t masked;   // keys from here on need the rows' own limits
    const int32_t* list;  // ids of the row, or the request's block-table row
};

// x of the lane that CTRL names within rows of 16 lanes or of the rows before
// (0x111.. row shifts by 1.., 0x142 and 0x143 the last lane of the row or half
// before); `none` where there is no such lane.
template <int CTRL, int ROWS>
__device__ __forceinline__ int from_lane(int none, int x) {
    return __builtin_amdgcn_update_dpp(none, x, CTRL, ROWS, 0xF, false);
}
// Inclusive sums over the wave's lanes: a few cycles a step, where a shuffle
// through LDS takes a hundred.
__device__ __forceinline__ int wave_sums(int x) {
    x += from_lane<0x111, 0xF>(0, x);
    x += from_lane<0x112, 0xF>(0, x);
    x += from_lane<0x114, 0xF>(0, x);
    x += from_lane<0x118, 0xF>(0, x);
    x += from_lane<0x142, 0xA>(0, x);
    x += from_lane<0x143, 0xC>(0, x);
    return x;
}
__device__ __forceinline__ float wave_total(float x) {
    auto get = [](int v) { return __int_as_float(v); };
    x += get(from_lane<0x111, 0xF>(0, __float_as_int(x)));
    x += get(from_lane<0x112, 0xF>(0, __float_as_int(x)));
    x += get(from_lane<0x114, 0xF>(0, __float_as_int(x)));
    x += get(from_lane<0x118, 0xF>(0, __float_as_int(x)));
    x += get(from_lane<0x142, 0xA>(0, __float_as_int(x)));
    x += get(from_lane<0x143, 0xC>(0, __float_as_int(x)));
    return get(__builtin_amdgcn_readlane(__float_as_int(x), 63));
}
__device__ __forceinline__ int wave_most(int x) {  // of numbers >= 0
    auto most = [](int p, int q) { return p > q ? p : q; };
    x = most(x, from_lane<0x111, 0xF>(0, x));
    x = most(x, from_lane<0x112, 0xF>(0, x));
    x = most(x, from_lane<0x114, 0xF>(0, x));
    x = most(x, from_lane<0x118, 0xF>(0, x));
    x = most(x, from_lane<0x142, 0xA>(0, x));
    x = most(x, from_lane<0x143, 0xC>(0, x));
    return __builtin_amdgcn_readlane(x, 63);
}

// Paged form: how many keys of its request a token's rows may see, `upto` being
// the tokens of the request up to it.
__device__ __forceinline__ int keys_seen(const AttendArgs& a, int ctx, int tokens, int upto) {
    int64_t n = (int64_t)ctx + (a.tree ? (tokens < 64 ? tokens : 64) : upto);
    const int64_t held = (int64_t)a.pages.cols * a.pages.block_size;
    n = n < held ? n : held;
    return (int)(n < 0x7FFFFFC0 ? n : 0x7FFFFFC0);
}

// The pieces of `stages` at `chunk` a piece; a row block without keys is one.
__device__ __forceinline__ int pieces_of(int stages, int chunk) {
    return stages > chunk ? (stages + chunk - 1) / chunk : 1;
}

template <int DL, int HG, bool PAGED>
__global__ __launch_bounds__(kAttendBlock, 1) void latent_attend_kernel(AttendArgs a, int splits, int target,
                                                                        float* __restrict__ part_out,
                                                                        float* __restrict__ part_lse) {
    constexpr int DP = kAttendWaves / HG;      // parts of the values
    constexpr int NT = DL / 32 / DP;           // output tiles of a wave
    constexpr int NQ = (DL + kRope) / 16;      // steps of the first product
    constexpr int kStageB = stage_bytes<DL>();
    constexpr int kColumnB = kTile * 128;      // a column of a stage
    constexpr int MB = 32 * HG;                // query rows of a workgroup
    constexpr int kLoads = DL / 64 + 1;        // columns: loads of a wave and stage
    extern __shared__ __align__(1024) char lds_memory[];
    const uint32_t lds = lds_address(lds_memory);
    const uint32_t entries = lds + kStages * kStageB;  // [wave][stage % 8][64]: ids or block ids of 32 keys, twice

    char* const flaws = lds_memory + kStages * kStageB + kAttendWaves * kEntryStages * 256;  // [key][DL bits]
    int* const flawed_keys = reinterpret_cast<int*>(flaws + kTile * DL / 8);

    const int tid = threadIdx.x, lane = tid & 63, half = lane >> 5, col = lane & 31;
    const int wave = __builtin_amdgcn_readfirstlane(tid >> 6);
    const int hg = wave % HG, dp = wave / HG;

    int split;       // which piece of the block's keys, of how many
    int pieces = splits;
    Work w{};
    if constexpr (!PAGED) {
        const int blocks = (a.heads + MB - 1) / MB;
        const int64_t block = blockIdx.x / (uint32_t)splits;
        split = (int)(blockIdx.x - (uint32_t)block * (uint32_t)splits);
        w.q0 = block / blocks;
        w.head0 = (int)(block - w.q0 * blocks) * MB;
        int n = a.k;
        if (a.counts) n = a.counts[w.q0] < 0 ? 0 : a.counts[w.q0] < n ? a.counts[w.q0] : n;
        w.n = __builtin_amdgcn_readfirstlane(n);
        w.masked = w.n;
        w.list = a.ids + w.q0 * a.ld_ids;
    } else {
        // A request's tokens, row blocks and stages (of its last block).
        struct Request { int64_t st; int tokens, ctx, blocks, stages; };
        auto request = [&](int64_t i) {
            Request r{};
            if (i >= a.reqs) return r;
            int64_t st = a.query_starts[i], en = a.query_starts[i + 1];
            st = st < 0 ? 0 : st < a.rows ? st : a.rows;
            en = en < st ? st : en < a.rows ? en : a.rows;
            r.st = st;
            r.tokens = (int)(en - st);
            r.ctx = a.ctx_lens[i] < 0 ? 0 : a.ctx_lens[i];
            r.blocks = (int)(((en - st) * a.heads + MB - 1) / MB);
            r.stages = (keys_seen(a, r.ctx, r.tokens, r.tokens) + kTile - 1) / kTile;
            return r;
        };
        // Lengths differ, so the pieces are of about one size, not of one
        // number a request: the smallest size tried, upwards in steps of 1/16,
        // with which all requests' pieces are no more than `target` workgroups.
        // The grid has room for `target` and one piece a block, which is
        // enough for any size tried (all are at least total / target).
        const Request of_lane = request(lane);  // the first 64 are read once
        auto requests = [&](int64_t i0) { return i0 == 0 ? of_lane : request(i0 + lane); };
        int chunk = 0x7FFFFFFF;
        if (splits > 1) {
            float total = 0.f, blocks = 0.f;
            int longest = 0;
            for (int64_t i0 = 0; i0 < a.reqs; i0 += 64) {
                const Request r = requests(i0);
                total += wave_total((float)r.blocks * (float)r.stages);
                blocks += wave_total((float)r.blocks);
                const int most = wave_most(r.blocks > 0 ? r.stages : 0);
                longest = most > longest ? most : longest;
            }
            // Rounding up costs about half a piece a block.
            const float room = (float)target - 0.5f * blocks;
            const float least = total * 1.0001f / (room > 0.5f * (float)target ? room : 0.5f * (float)target) + 1.f;
            chunk = (longest + splits - 1) / splits;
            chunk = chunk > (int)least ? chunk : (int)least;
            chunk = chunk > kLeastPiece ? chunk : kLeastPiece;
            for (int tries = 0; tries < 8; ++tries) {
                float sum = 0.f;
                for (int64_t i0 = 0; i0 < a.reqs; i0 += 64) {
                    const Request r = requests(i0);
                    sum += wave_total((float)r.blocks * (float)pieces_of(r.stages, chunk));
                }
                if (sum <= (float)target) break;
                chunk += chunk / 16 + 1;
            }
            chunk = __builtin_amdgcn_readfirstlane(chunk);
        }
        // This workgroup's request, row block and piece: a running sum of the
        // requests' workgroups, 64 requests at a time.  They follow each other
        // without gaps (idle ones among them would leave shader engines
        // without work, since workgroups go around them in turn).
        int64_t before = 0, req = -1;
        int flat = 0;
        for (int64_t i0 = 0; i0 < a.reqs; i0 += 64) {
            const Request r = requests(i0);
            const int mine = pieces_of(r.stages, chunk), own = r.blocks * mine;
            const int sum = wave_sums(own);
            const uint64_t past = __ballot(before + sum > (int64_t)blockIdx.x);
            if (past) {
                const int at = __ffsll((unsigned long long)past) - 1;
                req = i0 + at;
                w.q0 = __builtin_amdgcn_readlane((int)r.st, at);
                w.tokens = __builtin_amdgcn_readlane(r.tokens, at);
                w.ctx = __builtin_amdgcn_readlane(r.ctx, at);
                pieces = __builtin_amdgcn_readlane(mine, at);
                const int in = (int)((int64_t)blockIdx.x - before) - __builtin_amdgcn_readlane(sum - own, at);
                flat = in / pieces * MB;
                split = in % pieces;
                break;
            }
            before += __builtin_amdgcn_readlane(sum, 63);
        }
        if (req < 0) return;
        req = __builtin_amdgcn_readfirstlane((int)req);
        if (flat < 0 || flat >= (int64_t)w.tokens * a.heads) return;
        w.flat0 = flat;
        const int first = flat / a.heads, last_row = first + (flat - first * a.heads + MB - 1) / a.heads;
        const int last = last_row < w.tokens ? last_row : w.tokens - 1;
        const int n = keys_seen(a, w.ctx, w.tokens, last + 1);
        w.n = __builtin_amdgcn_readfirstlane(n);
        const int64_t masked = (int64_t)w.ctx + (a.tree ? 0 : first + 1);
        w.masked = __builtin_amdgcn_readfirstlane((int)(masked < w.n ? masked : w.n));
        w.list = a.pages.table + req * a.pages.ld;
    }

    const int all = w.n / kTile + (w.n % kTile != 0);   // stages
    const int per = (all + pieces - 1) / pieces;
    const int s0 = split * per;
    const int s1 = s0 + per < all ? s0 + per : all;

    // This lane's query row.
    int64_t token;
    int head;
    bool row_ok;
    int idx = 0;                // paged: the token's place in its request
    if constexpr (!PAGED) {
        token = w.q0;
        head = w.head0 + hg * 32 + col;
        row_ok = head < a.heads;
    } else {
        const int f = w.flat0 + hg * 32 + col;
        idx = f / a.heads;
        head = f - idx * a.heads;
        row_ok = idx < w.tokens;
        token = w.q0 + idx;
    }
    const float c = a.scale == 0.f ? 1.f : fabsf(a.scale) * kLog2e;
    const float lazy = kLazy / c;
    uint64_t tree = 0;
    if constexpr (PAGED) {
        if (a.tree && row_ok) tree = a.tree[token];
    }

    // Reads the list's entries of stage j's 32 keys into the wave's own copy.
    const uint32_t my_entries = entries + wave * (kEntryStages * 256);
    auto look = [&](int j) {
        const uint32_t e = (uint32_t)j * kTile + col;
        uint32_t at = e < (uint32_t)w.n ? e : (uint32_t)(w.n - 1);
        if constexpr (PAGED) at = block_of(a.pages, at);
        load_to_lds<4, 0>(reinterpret_cast<const char*>(w.list) + (uint64_t)at * 4,
                          my_entries + (j & (kEntryStages - 1)) * 256);
    };
    // The physical row of key `i` of stage j, negative where there is none.
    auto row_of = [&](int j, int i) {
        const int entry = lds_read<int>(my_entries + (j & (kEntryStages - 1)) * 256 + i * 4);
        const uint32_t e = (uint32_t)j * kTile + i;
        int r;
        if constexpr (PAGED)
            r = phys_row(a.pages, entry, e);
        else
            r = entry < a.cache_rows ? entry : -1;
        return e < (uint32_t)w.n && j < s1 ? r : -1;
    };
    // The loads of the wave's 8 keys of stage j into the ring, a column each;
    // lane l brings chunk l % 8 of key l / 8.
    const int64_t ldb = a.ld_cache * 2;
    auto source = [&](int j) {
        const int i = wave * 8 + (lane >> 3);
        const int r = row_of(j, i);
        const char* row = r < 0 ? reinterpret_cast<const char*>(g_zero_row)
                                : reinterpret_cast<const char*>(a.cache) + r * ldb;
        return row + (((lane & 7) ^ chunk_xor(i)) * 16);
    };
    auto fetch = [&](int j, const char* src, auto column) {
        constexpr int i = decltype(column)::value;
        load_to_lds<16, i * 128>(src, lds + (j & (kStages - 1)) * kStageB + i * (kColumnB - 128) + wave * 1024);
    };

    if constexpr (PAGED) {  // read behind the barriers of a stage
        for (int i = tid; i < flaw_bytes<DL>() / 4; i += kAttendBlock) reinterpret_cast<int*>(flaws)[i] = 0;
    }
    // The ring is always filled (behind the last stage with the zero row), so
    // that the number of loads under way is the same at every stage.
    if (s0 < s1) {
#pragma unroll
        for (int p = 0; p < kStages + 1; ++p) look(s0 + p);
        asm volatile("s_waitcnt vmcnt(0)" ::: "memory");
#pragma unroll
        for (int p = 0; p < kStages - 1; ++p) {
            const char* src = source(s0 + p);
            each<kLoads>([&](auto i) { fetch(s0 + p, src, i); });
        }
    }

    bf16x8 q[NQ];
    {
        const uint16_t* qp = a.q + token * a.ld_q + (int64_t)head * a.ld_head + half * 8;
        const uint32_t flip = a.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
        for (int i = 0; i < NQ; ++i) {
            i32x4 v = {};
            if (row_ok) v = *reinterpret_cast<const i32x4*>(qp + i * 16);
            if (a.scale == 0.f) v = times_zero(v);
            q[i] = __builtin_bit_cast(bf16x8, v ^ (int)flip);
        }
    }

    // First product: chunk 2 i + half of key col; the XOR of two steps' chunks
    // and a column's offset are constants.
    const uint32_t ka = lds + col * 128 + ((half ^ chunk_xor(col)) * 16);
    // Second product: each 16 lanes read 4 keys x 16 values and get a value's
    // 4 keys a lane.
    const int vkey = 4 * half + ((lane & 15) >> 2);
    const uint32_t va = lds + (dp * NT / 2) * kColumnB + vkey * 128 +
                        (((dp * NT & 1) * 4 + ((lane >> 4) & 1) * 2 + ((lane & 3) >> 1)) ^ chunk_xor(vkey)) * 16 +
                        (lane & 1) * 8;

    f32x16 o[NT] = {};
#pragma unroll
    for (int t = 0; t < NT; ++t) pin(o[t]);  // sums of their own, not copies of one zero
    float m = kNoMax, l = 0.f;

    // Waits until a stage has arrived, AFTER later ones being under way, and
    // every wave is done with what it read before.
    auto arrive = [&](auto after) {
        asm volatile("s_waitcnt vmcnt(%0) lgkmcnt(0)" ::"n"(decltype(after)::value * kLoads) : "memory");
        __builtin_amdgcn_s_barrier();
        asm volatile("" ::: "memory");
    };
    constexpr int KB = 2, VB = 3;         // groups of keys and tiles of values in registers
    constexpr int GQ = 4, NG = NQ / GQ;  // the first product in groups, each read one group ahead
    static_assert(NG == kLoads, "one piece of the next loads a group");
    auto read_k = [&](const uint32_t (&at)[4], int g, bf16x8 (&k)[GQ]) {
#pragma unroll
        for (int i = 0; i < GQ; ++i) k[i] = lds_read<bf16x8>(at[i] + g * kColumnB);
    };
    auto k_addresses = [&](int j, uint32_t (&at)[4]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at[i] = (ka + (j & (kStages - 1)) * kStageB) ^ (i * 32);
            asm("" : "+v"(at[i]));  // four registers, and the columns in the reads' offsets
        }
    };
    typedef __attribute__((address_space(3))) bf16x4* lds_b4;
    // The values of output tile t, in the two steps' order; at: [t & 1][lower, upper 8 keys].
    auto read_v = [&](const uint32_t (&at)[2][2], int t, bf16x8 (&v)[2]) {
#pragma unroll
        for (int k = 0; k < 2; ++k) {
            const int off = (t >> 1) * kColumnB + k * 16 * 128;
            const bf16x4 lo = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_b4)(uintptr_t)(at[t & 1][0] + off));
            const bf16x4 hi = __builtin_amdgcn_ds_read_tr16_b64_v4bf16((lds_b4)(uintptr_t)(at[t & 1][1] + off + 1024));
            v[k] = __builtin_shufflevector(lo, hi, 0, 1, 2, 3, 4, 5, 6, 7);
        }
    };
    auto v_addresses = [&](int j, uint32_t (&at)[2][2]) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            at[i >> 1][i & 1] = (va + (j & (kStages - 1)) * kStageB) ^ ((i >> 1) * 64 + (i & 1) * 16);
            asm("" : "+v"(at[i >> 1][i & 1]));
        }
    };

    f32x16 s = {};
    if (s0 < s1) {
        arrive(std::integral_constant<int, kStages - 2>{});
        uint32_t at[4];
        k_addresses(s0, at);
#pragma unroll
        for (int g = 0; g < NG; ++g) {
            bf16x8 k[GQ];
            read_k(at, g, k);
#pragma unroll
            for (int i = 0; i < GQ; ++i)
                s = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[i], q[g * GQ + i], s, 0, 0, 0);
        }
    }

    // Stage j's scores are in s, with their maximum, the keys that exist and the
    // next rows to load.  A pass forms the scores of stage j + 1 while the
    // weights of stage j are computed, then adds stage j's values while what
    // the next pass begins with is made ready.
    float top = s[0];
    uint32_t exist = 0;
    const char* src = nullptr;
    if (s0 < s1) {
#pragma unroll
        for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
        exist = (uint32_t)__ballot(row_of(s0, col) >= 0);
        src = source(s0 + kStages - 1);
    }
    for (int j = s0; j < s1; ++j) {
#pragma unroll
        for (int t = 0; t < NT; ++t) pin(o[t]);  // they stay there from pass to pass
        // Which of the 32 keys this lane's row sees.
        uint32_t see = exist;
        const bool rows_differ = PAGED && j * kTile + kTile > w.masked;
        if constexpr (PAGED) {
            if (rows_differ) {
                const int d0 = j * kTile - w.ctx;  // draft number of the stage's first key
                uint32_t mine;
                if (!a.tree) {
                    const int upto = idx + 1 - d0;  // keys of the stage that are seen
                    mine = upto >= 32 ? ~0u : upto <= 0 ? 0u : (1u << upto) - 1;
                } else {
                    const uint64_t live = w.tokens >= 64 ? ~0ull : (1ull << w.tokens) - 1;
                    const uint64_t bits = tree & live;
                    if (d0 >= 64)
                        mine = 0;
                    else if (d0 >= 0)
                        mine = (uint32_t)(bits >> d0);
                    else if (d0 > -32)
                        mine = (uint32_t)(bits << -d0) | ((1u << -d0) - 1);
                    else
                        mine = ~0u;
                }
                see &= mine;
            }
        }
        if (rows_differ || see != ~0u) {
            const uint32_t bits = see >> (4 * half);
#pragma unroll
            for (int r = 0; r < 16; ++r)
                if (!((bits >> ((r & 3) + 8 * (r >> 2))) & 1)) s[r] = -INFINITY;
            top = s[0];
#pragma unroll
            for (int r = 1; r < 16; ++r) top = fmaxf(top, s[r]);
        }
        {
            const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(top), __float_as_uint(top), false, false);
            top = fmaxf(__uint_as_float(x[0]), __uint_as_float(x[1]));
        }
        if (see) m = fmaxf(m, kLeastMax);
        if (__any(top > m + lazy)) {
            const float to = fmaxf(m, top);
            if (j != s0) {
                const float f = __builtin_amdgcn_exp2f((m - to) * c);
                l *= f;
                sums_ready(o);
#pragma unroll
                for (int t = 0; t < NT; ++t) {
#pragma unroll
                    for (int r = 0; r < 16; ++r) o[t][r] *= f;
                    pin(o[t]);  // one tile at a time in vector registers
                }
            }
            m = to;
        }

        bf16x8 p[2];
        float sum = 0.f;
        // The weights are rounded to bf16 because the matrix instructions take both
        // operands in one 16-bit type, and the values' range is bf16's; their sum
        // keeps 32 bits.  A result is then 1.8e-3 to 2.1e-3 from 64 bits (relative,
        // over all elements), of which 1.65e-3 is its own rounding to bf16.  Weights in
        // two terms, the rounded one and its remainder, gave 1.65e-3 and cost a second
        // product: 64 tokens x 16 heads x 2048 rows 42.4 us for 40.2, 1024 x 128 heads
        // 731 for 567, dense decode 207 for 152, a causal chunk of 1024 tokens x 128
        // heads 1457 for 1021.
        auto weigh = [&](int r) {
            const float x = __builtin_amdgcn_exp2f((s[r] - m) * c);
            sum += x;
            p[r >> 3][r & 7] = (__bf16)x;
        };
        bf16x8 v[VB][2];
        uint32_t v_at[2][2];
        v_addresses(j, v_at);
        auto first_v = [&] {
#pragma unroll
            for (int t = 0; t < VB - 1 && t < NT; ++t) read_v(v_at, t, v[t]);
        };
        f32x16 next = {};
        if (j + 1 < s1) {
            // After this the place of stage j - 1 is free for stage j + 3.
            arrive(std::integral_constant<int, kStages - 3>{});
            uint32_t at[4];
            k_addresses(j + 1, at);
            bf16x8 k[KB][GQ];
#pragma unroll
            for (int g = 0; g < KB - 1; ++g) read_k(at, g, k[g]);
            look(j + kStages + 1);
            each<NG>([&](auto group) {
                constexpr int g = decltype(group)::value;
                if constexpr (g + KB - 1 < NG) read_k(at, g + KB - 1, k[(g + KB - 1) % KB]);
                if constexpr (g + 1 == NG) first_v();
                fetch(j + kStages - 1, src, group);
#pragma unroll
                for (int i = 0; i < GQ; ++i)
                    next = __builtin_amdgcn_mfma_f32_32x32x16_bf16(k[g % KB][i], q[g * GQ + i], next, 0, 0, 0);
#pragma unroll
                for (int r = g * 16 / NG; r < (g + 1) * 16 / NG; ++r) weigh(r);
                __builtin_amdgcn_sched_barrier(0);
            });
        } else {
#pragma unroll
            for (int r = 0; r < 16; ++r) weigh(r);
            if (!PAGED || !rows_differ) first_v();
        }
        l += sum;

        if constexpr (PAGED) {
            if (rows_differ) {
                // A key that only some rows see must not reach the others as
                // 0 * NaN or 0 * inf: what is not finite is noted and taken as
                // 0 in the product, and the rows that see it get their NaN
                // (a score of -inf, the weight 0) by the notes.
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                constexpr int kEach = kTile * DL * 2 / 16 / kAttendBlock;
                static_assert(kEach == DL / 64, "a thread has its key's chunk of every column");
                const int key = tid >> 3;
                char* const note = flaws + key * (DL / 8) + ((tid & 7) ^ chunk_xor(key));
                i32x4* x16 = reinterpret_cast<i32x4*>(lds_memory + (j & (kStages - 1)) * kStageB) + tid;
                i32x4 x[kEach];
#pragma unroll
                for (int i = 0; i < kEach; ++i) x[i] = x16[i * kAttendBlock];
                bool noted = false;
#pragma unroll
                for (int i = 0; i < kEach; ++i) {
                    int bad = 0;
#pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        const bool lo = (x[i][e] & 0x7F80) == 0x7F80, hi = (x[i][e] & 0x7F800000) == 0x7F800000;
                        x[i][e] &= (lo ? 0xFFFF0000 : ~0u) & (hi ? 0xFFFF : ~0u);
                        bad |= (int)lo << (2 * e) | (int)hi << (2 * e + 1);
                    }
                    if (bad) {
                        x16[i * kAttendBlock] = x[i];
                        note[i * 8] = (char)bad;
                        noted = true;
                    }
                }
                if (noted) atomicOr(flawed_keys, (int)(1u << key));
                asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                __builtin_amdgcn_s_barrier();
                asm volatile("" ::: "memory");
                const uint32_t flawed = __builtin_amdgcn_readfirstlane(*flawed_keys);
                if (flawed) {
                    uint32_t nan_at[NT] = {};
                    for (uint32_t keys = flawed; keys; keys &= keys - 1) {
                        const int k = __builtin_ctz(keys);
                        const uint32_t* bits = reinterpret_cast<const uint32_t*>(flaws + k * (DL / 8)) + dp * NT;
                        const uint32_t mine = see >> k & 1 ? ~0u : 0u;
#pragma unroll
                        for (int t = 0; t < NT; ++t) nan_at[t] |= bits[t] & mine;
                    }
                    sums_ready(o);
#pragma unroll
                    for (int t = 0; t < NT; ++t) {
                        const uint32_t at = nan_at[t] >> (4 * half);
#pragma unroll
                        for (int r = 0; r < 16; ++r)
                            if (at >> ((r & 3) + 8 * (r >> 2)) & 1) o[t][r] = __builtin_nanf("");
                        pin(o[t]);
                        __builtin_amdgcn_sched_barrier(0);
                    }
                    asm volatile("s_waitcnt lgkmcnt(0)" ::: "memory");
                    __builtin_amdgcn_s_barrier();
                    asm volatile("" ::: "memory");
                    // Cleared before the next stage's first barrier.
                    if (noted)
                        for (int i = 0; i < kEach; ++i) note[i * 8] = 0;
                    if (tid == 0) *flawed_keys = 0;
                }
                first_v();
            }
        }

#pragma unroll
        for (int t = 0; t < NT; ++t) {
            if (t + VB - 1 < NT) read_v(v_at, t + VB - 1, v[(t + VB - 1) % VB]);
#pragma unroll
            for (int k = 0; k < 2; ++k) add_product(o[t], v[t % VB][k], p[k]);
            if (t == 0) {
                exist = (uint32_t)__ballot(row_of(j + 1, col) >= 0);
                src = source(j + kStages);
            }
            if (t == NT / 2) top = next[0];
            if (t >= NT / 2)
#pragma unroll
                for (int r = (t - NT / 2) * 32 / NT; r < (t - NT / 2 + 1) * 32 / NT; ++r) top = fmaxf(top, next[r]);
            __builtin_amdgcn_sched_barrier(0);
        }
        s = next;
    }

    asm volatile("s_waitcnt vmcnt(0)" ::: "memory");  // nothing is loaded into LDS behind the workgroup's end
    {
        const auto x = __builtin_amdgcn_permlane32_swap(__float_as_uint(l), __float_as_uint(l), false, false);
        l = __uint_as_float(x[0]) + __uint_as_float(x[1]);
    }
    const float inv = l == 0.f ? 0.f : 1.f / l;
    sums_ready(o);
    if (!row_ok) return;
    const int64_t rh = token * a.heads + head;
    const float lse = l == 0.f ? -INFINITY : m * fabsf(a.scale) + __builtin_amdgcn_logf(l) * kLn2;
    const int64_t part = (int64_t)split * a.rows * a.heads + rh;
    const bool empty = l == 0.f && m == kNoMax;  // nothing was seen
    if (dp == 0 && half == 0) {
        if (splits > 1) {
            part_lse[part] = l == 0.f && !empty ? kNoMax : lse;  // the join reads its zeros and NaN
            if (split == 0)  // the join sees `splits` parts of every row
                for (int p = pieces; p < splits; ++p) part_lse[(int64_t)p * a.rows * a.heads + rh] = -INFINITY;
        } else if (a.lse)
            a.lse[rh] = lse;
    }
    if (splits > 1) {
        if (empty) return;  // the join reads no values of an empty part
        float* dst = part_out + part * DL + dp * NT * 32 + 4 * half;
#pragma unroll
        for (int t = 0; t < NT; ++t)
#pragma unroll
            for (int g = 0; g < 4; ++g)
                *reinterpret_cast<f32x4*>(dst + t * 32 + g * 8) =
                    f32x4{o[t][4 * g] * inv, o[t][4 * g + 1] * inv, o[t][4 * g + 2] * inv, o[t][4 * g + 3] * inv};
        return;
    }
    // The halves trade 4 values each, so that a lane stores 8 (16 bytes) of one
    // group: the lower half those of group g, the upper those of g + 1.
    uint16_t* dst = a.out + rh * DL + dp * NT * 32 + 8 * half;
#pragma unroll
    for (int t = 0; t < NT; ++t)
#pragma unroll
        for (int g = 0; g < 4; g += 2) {
            uint32_t lo[2], hi[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                lo[i] = f32_bf16(o[t][4 * g + 2 * i] * inv) | (uint32_t)f32_bf16(o[t][4 * g + 2 * i + 1] * inv) << 16;
                hi[i] = f32_bf16(o[t][4 * g + 4 + 2 * i] * inv) | (uint32_t)f32_bf16(o[t][4 * g + 5 + 2 * i] * inv) << 16;
            }
            const auto x = __builtin_amdgcn_permlane32_swap(lo[0], hi[0], false, false);
            const auto y = __builtin_amdgcn_permlane32_swap(lo[1], hi[1], false, false);
            *reinterpret_cast<uint4*>(dst + t * 32 + g * 8) = uint4{x[0], y[0], x[1], y[1]};
        }
}

constexpr int kCus = 256;

// How a call is cut: the row groups of a workgroup (1, 2 or 4 of 32 query
// rows) and the pieces of the keys that take the least estimated time.  A
// workgroup has a CU for itself.  On 256 busy CUs a stage takes 1.44, 1.62 or
// 1.95 us with 1, 2 or 4 groups and what lies around the stages, the launch
// included, 9, 12 or 17 us; the rule has 5% more for a stage and 1 to 2 us less
// around.  Pieces cost a second launch and the way of their 32-bit results out
// and back at 4 TB/s.  Measured (groups/pieces: us), the rule's choice first: 64
// tokens x 128 heads x 2048 keys 4/4: 65, 2/2: 77, 2/1: 93, 1/1: 101; 8 tokens
// 1/7: 31, 1/8: 30, 4/8: 38, 4/4: 46; 64 tokens x 16 heads 1/4: 36, 1/8: 46, 1/2:
// 49; 1024 tokens x 128 heads x 512 keys 4/1: 195, 2/1: 294, 4/2: 429.
static AttendPlan plan_pieces(int64_t units, int64_t rows_each, int64_t stages, int64_t out_rows,
                              int32_t d_latent, bool allow) {
    constexpr float kStageUs[3] = {1.5f, 1.75f, 2.05f}, kAroundUs[3] = {7.f, 11.f, 16.f};
    const float piece = (float)out_rows * d_latent * 8 / 4e6f;
    const uint32_t n = (uint32_t)(stages < 1 ? 1 : stages < 0x7FFFFFFF ? stages : 0x7FFFFFFF);
    const uint32_t most = !allow ? 1 : n < 64 ? n : 64;
    AttendPlan best{1, 4, 1, 0};
    float best_us = 3e38f;
    for (int g = 0; g < 3; ++g) {
        const int hg = 1 << g;
        const int64_t blocks = units * ((rows_each + 32 * hg - 1) / (32 * hg));
        for (uint32_t s = 1; s <= most; ++s) {
            const uint32_t per = (n + s - 1) / s;
            const float us = (float)((blocks * s + kCus - 1) / kCus) * (per * kStageUs[g] + kAroundUs[g]) +
                             (s > 1 ? 4.f + s * piece : 0.f);
            if (us < best_us) best_us = us, best.splits = s, best.groups = hg, best.target = (int)(blocks * s);
        }
    }
    return best;
}

static AttendPlan with_workspace(AttendPlan p, int64_t out_rows, int32_t d_latent) {
    if (p.splits > 1) p.ws_bytes = ((size_t)p.splits * out_rows * (d_latent + 1) * 4 + 15) & ~size_t(15);
    return p;
}

AttendPlan plan_attend_rows(int64_t rows, int32_t heads, int32_t d_latent, int32_t k, bool allow_split) {
    return with_workspace(plan_pieces(rows, heads, ((int64_t)k + kTile - 1) / kTile, rows * heads, d_latent,
                                      allow_split), rows * heads, d_latent);
}

// Goes by the mean number of tokens a request.  Pieces are of one size there,
// so a long request may have twice the mean number of them.
AttendPlan plan_attend_paged(int64_t tokens, int64_t reqs, int32_t heads, int32_t d_latent,
                             int64_t max_len, bool allow_split) {
    const int64_t active = reqs < tokens ? reqs : tokens;
    AttendPlan p = plan_pieces(active, (tokens + active - 1) / active * heads,
                               max_len / kTile + (max_len % kTile != 0), tokens * heads, d_latent, allow_split);
    if (p.splits > 1) p.splits = p.splits < 32 ? 2 * p.splits : 64;
    return with_workspace(p, tokens * heads, d_latent);
}

template <int DL, int HG, bool PAGED>
static int launch_attend(const AttendArgs& a, const AttendPlan& plan, void* workspace, hipStream_t s) {
    constexpr int kRows = 32 * HG;
    // Paged: no more row blocks than this, whatever the requests' lengths are,
    // and one piece a block more than `target` at most.
    const int64_t blocks = PAGED ? a.rows * a.heads / kRows + (a.reqs < a.rows ? a.reqs : a.rows)
                                 : a.rows * ((a.heads + kRows - 1) / kRows);
    const int64_t grid = plan.splits == 1 ? blocks : PAGED ? blocks + plan.target : blocks * plan.splits;
    if (grid > kMaxThreads / kAttendBlock) return RTS_EUNSUPPORTED;
    const int64_t n = a.rows * a.heads;
    float* part_out = static_cast<float*>(workspace);
    float* part_lse = part_out ? part_out + (int64_t)plan.splits * n * DL : nullptr;
    constexpr size_t lds = kStages * stage_bytes<DL>() + kAttendWaves * kEntryStages * 256 +
                           (PAGED ? flaw_bytes<DL>() : 0);
    hipLaunchKernelGGL((latent_attend_kernel<DL, HG, PAGED>), dim3((unsigned)grid), dim3(kAttendBlock), lds, s, a,
                       plan.splits, plan.target, part_out, part_lse);
    if (hipGetLastError() != hipSuccess) return RTS_EHIP;
    if (plan.splits == 1) return RTS_OK;
    return launch_merge_attend(part_out, RTS_F32, part_lse, plan.splits, a.rows, a.heads, DL, a.out, RTS_BF16, a.lse,
                               PAGED ? a.query_starts + a.reqs : nullptr, true, s);
}

template <int DL, bool PAGED>
static int launch_attend_of(const AttendArgs& a, const AttendPlan& plan, void* workspace, hipStream_t s) {
    if (plan.groups == 1) return launch_attend<DL, 1, PAGED>(a, plan, workspace, s);
    if (plan.groups == 2) return launch_attend<DL, 2, PAGED>(a, plan, workspace, s);
    return launch_attend<DL, 4, PAGED>(a, plan, workspace, s);
}

int launch_latent_attend(const AttendArgs& a, const AttendPlan& plan, void* workspace, hipStream_t s) {
    if (a.paged)
        return a.d_latent == 512 ? launch_attend_of<512, true>(a, plan, workspace, s)
                                 : launch_attend_of<256, true>(a, plan, workspace, s);
    return a.d_latent == 512 ? launch_attend_of<512, false>(a, plan, workspace, s)
                             : launch_attend_of<256, false>(a, plan, workspace, s);
}

// --------------------------------------------------------------- rank merge

typedef float f32x8 __attribute__((ext_vector_type(8)));

// 8 elements as they lie in memory.
template <typename T>
struct Raw8;
template <>
struct Raw8<uint16_t> {
    uint4 w;
    __device__ __forceinline__ f32x8 widen() const {
        f32x8 r;
        const uint32_t x[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            r[2 * i] = __uint_as_float(x[i] << 16);
            r[2 * i + 1] = __uint_as_float(x[i] & 0xFFFF0000u);
        }
        return r;
    }
};
template <>
struct Raw8<float> {
    float4 lo, hi;
    __device__ __forceinline__ f32x8 widen() const {
        return f32x8{lo.x, lo.y, lo.z, lo.w, hi.x, hi.y, hi.z, hi.w};
    }
};
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
// a (row, head) from the caches.  kMergeAhead parts are on their way while as
// many are added, the first also while the maximum is still being found.  Bound
// by the bytes: 8 ranks x 1000 x 128 x 512 in bf16 take 207 us, 5.7 TB/s.
// Where no part's lse is above `none` the lse is -inf.
constexpr int kMergeAhead = 4;

template <typename In, typename Out>
__global__ __launch_bounds__(256) void merge_attend_kernel(
    const In* __restrict__ parts, const float* __restrict__ part_lse, int world, int64_t n, int dim8,
    int heads, const int32_t* __restrict__ row_limit, float none, Out* __restrict__ out, float* __restrict__ lse) {
    const int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x;
    if (i >= n * dim8) return;
    const int64_t rh = i / dim8;
    const int d = (int)(i - rh * dim8) * 8;
    if (row_limit && rh / heads >= *row_limit) return;
    const In* mine = parts + rh * dim8 * 8 + d;
    const int64_t step = n * dim8 * 8;
    const float* stat = part_lse + rh;

    struct Group { float x[kMergeAhead]; Raw8<In> v[kMergeAhead]; };
    // Parts r0.. of the world; one that is empty or does not exist is not read.
    auto load = [&](int r0, Group& g) {
#pragma unroll
        for (int u = 0; u < kMergeAhead; ++u) g.x[u] = r0 + u < world ? stat[(r0 + u) * n] : -INFINITY;
#pragma unroll
        for (int u = 0; u < kMergeAhead; ++u) {
            g.v[u] = Raw8<In>{};
            if (g.x[u] != -INFINITY) g.v[u] = *reinterpret_cast<const Raw8<In>*>(mine + (r0 + u) * step);
        }
    };
    Group even, odd;
    load(0, even);
    float m = even.x[0];  // NaN if any part's is
#pragma unroll
    for (int u = 1; u < kMergeAhead; ++u) m = __builtin_elementwise_maximum(m, even.x[u]);
#pragma unroll 8
    for (int r = kMergeAhead; r < world; ++r) m = __builtin_elementwise_maximum(m, stat[r * n]);
    f32x8 acc = {};
    float total = 0.f;
    auto add = [&](const Group& g) {
#pragma unroll
        for (int u = 0; u < kMergeAhead; ++u) {
            const float w = __builtin_amdgcn_exp2f((g.x[u] - m) * kLog2e);
            total += w;
            const f32x8 e = g.v[u].widen();
#pragma unroll
            for (int k = 0; k < 8; ++k) acc[k] = fmaf(w, e[k], acc[k]);
        }
    };
    if (m != -INFINITY) {
        for (int r0 = 0;;) {
            if ((r0 += kMergeAhead) < world) load(r0, odd);
            add(even);
            if (r0 >= world) break;
            if ((r0 += kMergeAhead) < world) load(r0, even);
            add(odd);
            if (r0 >= world) break;
        }
        const float inv = 1.f / total;
#pragma unroll
        for (int e = 0; e < 8; ++e) acc[e] *= inv;
    }
    store8(out + rh * dim8 * 8 + d, acc);
    if (lse && d == 0) lse[rh] = m <= none ? -INFINITY : m + __builtin_amdgcn_logf(total) * kLn2;
}

int launch_merge_attend(const void* parts, int dtype, const float* part_lse, int32_t world, int64_t rows,
                        int32_t heads, int32_t dim, void* out, int out_dtype, float* lse,
                        const int32_t* row_limit, bool pieces, hipStream_t s) {
    const float none = pieces ? kNoMax : -INFINITY;
    const int64_t n = rows * heads, blocks = (n * (dim / 8) + 255) / 256;
    if (blocks > kMaxThreads / 256) return RTS_EUNSUPPORTED;
    const dim3 g((unsigned)blocks), b(256);
    const int d8 = dim / 8;
    const float* pf = static_cast<const float*>(parts);
    const uint16_t* ph = static_cast<const uint16_t*>(parts);
    float* of = static_cast<float*>(out);
    uint16_t* oh = static_cast<uint16_t*>(out);
    if (dtype == RTS_F32 && out_dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<float, float>), g, b, 0, s, pf, part_lse, world, n, d8, heads, row_limit, none, of, lse);
    else if (dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<float, uint16_t>), g, b, 0, s, pf, part_lse, world, n, d8, heads, row_limit, none, oh, lse);
    else if (out_dtype == RTS_F32)
        hipLaunchKernelGGL((merge_attend_kernel<uint16_t, float>), g, b, 0, s, ph, part_lse, world, n, d8, heads, row_limit, none, of, lse);
    else
        hipLaunchKernelGGL((merge_attend_kernel<uint16_t, uint16_t>), g, b, 0, s, ph, part_lse, world, n, d8, heads, row_limit, none, oh, lse);
    return hipGetLastError() == hipSuccess ? RTS_OK : RTS_EHIP;
}

}  // namespace rts
