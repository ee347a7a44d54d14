// Choice of the cache blocks that a query attends to, by bounds on their keys.
//
// A block is one page.  Its bounds are the per-channel minimum and maximum of its keys, and
//     s_j = max over the G heads of a kv head of  sum_d max(q_d, 0) kmax_jd + min(q_d, 0) kmin_jd
// is an upper bound on every q.k of block j.  The highest n blocks are wanted, ties to the lower index, and
// exactly: two blocks at the border may differ by less than fp32 sums hold.
//
// attn_score_kernel computes all scores on mma.sync (bf16 products are exact in fp32; the sums are not) and is
// bound by reading the bounds, 4 d bytes per block: every warp streams an equal, contiguous share of all groups
// of 16 blocks through its own ring of cp.async stages, whatever the lengths are.  attn_choose_kernel then needs
// only fp32's word on most blocks: with e a bound on the error of any score and t the n-th highest fp32 score,
// blocks above t + 2 e are in and blocks below t - 2 e are out; the few between are scored again exactly and
// ranked.
// Measured (CUDA graph, pages of 64, 32 query heads on 8 kv heads of 128, 64 blocks chosen): one sequence of 131001
// tokens 10.9 us, latency; 32 sequences x 2 tokens, 20000 to 90000 tokens, 30.2 us, of which the scores take about 19 (5.9
// TB/s) and the choice the rest: dependent steps (scores in, counts, border, output) of about 1 us each.
#include "paged.cuh"

namespace hla {
namespace {

constexpr int kGroupBlocks = 16;      // blocks scored together by a warp
constexpr int kScoreThreads = 128;
constexpr int kScoreStages = 2;       // groups in flight or in use per warp
constexpr int kScoreCtas = 3;         // CTAs per SM
constexpr int kMaxBlocks = 65536;     // blocks per sequence (a bit each in shared memory)
constexpr int kStaged = 6144;         // most scores of a row in shared memory; longer rows are read through L2
constexpr int kListed = 1024;         // blocks near the border kept in shared memory
constexpr int kFewInBin = 64;         // a bin with no more scores is not split again

struct SelectParams {
    const uint16_t *q, *k_min, *k_max;
    const int32_t *table, *past;
    int32_t *sel;
    float *score;                 // [B, T, Hkv, stride]
    unsigned long long *exact;    // [B, T, Hkv, stride]: exact scores, as ordered integers, of the blocks near the border when too many to list
    float *absmax;                // [B, Hkv, groups]: largest magnitude among the bounds of each group of 16 blocks
    int B, T, H, Hkv, G, d;
    int max_blocks, n_pages, pshift;
    int n_select, n_first, n_last;
    int stride, groups;
    int staged;                   // scores of a row that attn_choose_kernel keeps in shared memory
    uint32_t by_G, by_Hkv, by_T;  // for divided()
};

// Blocks that token t of a sequence sees.
__device__ __forceinline__ int visible_blocks(const SelectParams &p, int b, int t) {
    const int past = p.past[b];
    if (past < 0) return 0;
    const long n = (((long)past + t) >> p.pshift) + 1;
    return n < p.max_blocks ? (int)n : p.max_blocks;
}

__device__ __forceinline__ uint32_t relu2(uint32_t x) {  // max(x, 0) of two bf16, NaN kept
    const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&x), z);
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t neg2(uint32_t x) {  // min(x, 0) of two bf16, NaN kept
    const __nv_bfloat162 z = __float2bfloat162_rn(0.f);
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&x), z);
    return *reinterpret_cast<const uint32_t *>(&r);
}

__device__ __forceinline__ float max_keep_nan(float a, float b) {
    float r;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(r) : "f"(a), "f"(b));
    return r;
}
__device__ __forceinline__ uint4 lds_v4(uint32_t at) {
    uint4 w;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(w.x), "=r"(w.y), "=r"(w.z), "=r"(w.w) : "r"(at) : "memory");
    return w;
}

// Prefix sums of the sequences' groups per kv head into pre[0..B]; ends with a block barrier.
__device__ __forceinline__ void group_prefix(const SelectParams &p, int *pre) {
    const int lane = threadIdx.x;
    auto groups = [&](int b) { return (visible_blocks(p, b, p.T - 1) + kGroupBlocks - 1) / kGroupBlocks; };
    if (p.B <= 32) {
        if (lane < 32) {
            const int x = warp_prefix(lane < p.B ? groups(lane) : 0, lane);
            if (lane < p.B) pre[lane + 1] = x;
            if (lane == 0) pre[0] = 0;
        }
    } else {
        for (int b = threadIdx.x; b < p.B; b += blockDim.x) pre[b + 1] = groups(b);
        block_prefix(pre, p.B);
    }
    __syncthreads();
}

template <int D>
__host__ __device__ constexpr int score_ring() {  // shared memory of one warp's stages
    return kScoreStages * 2 * kGroupBlocks * 2 * D;
}

// Scores of groups of 16 blocks of one (sequence, kv head) for all T x G queries.  The blocks are the products' 16 rows
// and the queries their 8 columns, NQ times: a tile of 8 NQ queries holds whole groups of G heads (or a part of one).
// The order of channels within a sum is free, so lane (i, j) takes channels 32 c + 8 j .. + 7 of rows i and i + 8 and of
// query i, four of them for each of two products: 16 bytes to a load of q or of shared memory.
// NQ = 1, for at most 8 queries, against 2 there: 32 sequences x 2 tokens of 4 heads 2.6 us less.  The operands loaded from
// global memory into registers ahead of their use, without shared memory, are no faster (32.1 us with either) and slower
// for one sequence (14.1 against 12.1).
template <int D, int NQ>
__global__ void __launch_bounds__(kScoreThreads, kScoreCtas) attn_score_kernel(const SelectParams p) {
    constexpr int ROWS = 8 * NQ, RB = 2 * D, CPR = RB / 16, KS = D / 16, GB = kGroupBlocks * RB, NS = kScoreStages;
    constexpr unsigned ALL = 0xffffffffu;
    extern __shared__ __align__(128) uint8_t smem[];
    int *const s_pre = reinterpret_cast<int *>(smem + 4 * score_ring<D>());  // [B + 1]
    __shared__ float s_tile[4][ROWS][17];
    __shared__ unsigned s_has[4][NS];  // blocks of each staged group that have a page
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = lane >> 2, j = lane & 3;
    pdl_wait_trigger();
    group_prefix(p, s_pre);
    const int total = s_pre[p.B] * p.Hkv, warps = gridDim.x * 4;
    const int share = (total + warps - 1) / warps, w = blockIdx.x * 4 + warp;
    const int begin = (long)share * w < total ? share * w : total, n = share < total - begin ? share : total - begin;
    const uint32_t ring = smem_u32(smem) + warp * score_ring<D>();

    // place of group x of all: sequence, kv head, group of the sequence.  cur: where the copies are; use: the products
    struct Place {
        int b, hk, g, groups, nb;
    };
    auto place = [&](int x) {
        int lo = 0, hi = p.B;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (s_pre[mid] * p.Hkv <= x) lo = mid;
            else hi = mid;
        }
        Place a;
        a.b = lo;
        a.groups = s_pre[lo + 1] - s_pre[lo];
        const int rem = x - s_pre[lo] * p.Hkv;
        a.g = divided(rem, p.by_Hkv);  // the heads of a group one after another: their bounds are neighbours in memory
        a.hk = rem - a.g * p.Hkv;
        a.nb = visible_blocks(p, lo, p.T - 1);
        return a;
    };
    auto page_of = [&](const Place &a) -> int {  // lane l: page of the group's block l (16 lanes)
        const int blk = a.g * kGroupBlocks + (lane & 15);
        const int pg = blk < a.nb ? p.table[(size_t)a.b * p.max_blocks + blk] : -1;
        return pg < p.n_pages ? pg : -1;
    };
    // The place and pages of the group that is copied next are looked up one step ahead.
    Place ahead = n > 0 ? place(begin) : Place{};
    int pg = n > 0 ? page_of(ahead) : -1;
    // This lane's 16-byte chunks of a group: row y ROWS_IN + lane / CPR, chunk lane % CPR, for every y
    constexpr int ROWS_IN = 32 / CPR;
    const uint8_t *const from_max = reinterpret_cast<const uint8_t *>(p.k_max) + lane % CPR * 16;
    const uint8_t *const from_min = reinterpret_cast<const uint8_t *>(p.k_min) + lane % CPR * 16;
    const uint32_t to = ring + lane / CPR * RB + ((lane % CPR ^ (lane / CPR & 1) << 2) << 4);
    auto issue = [&](int x, int stage) {
        const uint32_t dst = to + stage * 2 * GB;
        const uint32_t row = pg * p.Hkv + ahead.hk;
        if (__all_sync(ALL, pg >= 0)) {
#pragma unroll
            for (int y = 0; y < GB / 512; ++y) {
                const size_t o = (size_t)__shfl_sync(ALL, row, y * ROWS_IN + lane / CPR) * RB;
                cp_async16_s(dst + y * 512, from_max + o);
                cp_async16_s(dst + y * 512 + GB, from_min + o);
            }
        } else {
#pragma unroll
            for (int y = 0; y < GB / 512; ++y) {
                const bool in = __shfl_sync(ALL, pg, y * ROWS_IN + lane / CPR) >= 0;
                const uint32_t r = __shfl_sync(ALL, row, y * ROWS_IN + lane / CPR);
                const size_t o = in ? (size_t)r * RB : 0;
                cp_async16_or_zero(dst + y * 512, from_max + o, in);
                cp_async16_or_zero(dst + y * 512 + GB, from_min + o, in);
            }
        }
        const unsigned has = __ballot_sync(ALL, pg >= 0);
        if (lane == 0) s_has[warp][stage] = has;
        if (x + 1 < n && ++ahead.hk == p.Hkv) {
            ahead.hk = 0;
            if (++ahead.g == ahead.groups) ahead = place(begin + x + 1);
            pg = page_of(ahead);
        }
    };
#pragma unroll
    for (int x = 0; x < NS - 1; ++x) {
        if (x < n) issue(x, x);
        cp_async_commit();
    }

    const int per = NQ == 1 ? p.T : p.G <= ROWS ? ROWS / p.G : 1;  // tokens per query tile
    const int parts = NQ == 1 ? 1 : (p.G + ROWS - 1) / ROWS;       // query tiles per token
    const bool one_tile = NQ == 1 || (parts == 1 && per >= p.T);
    Place use = n > 0 ? place(begin) : Place{};
    uint4 qf[KS / 2][NQ];
    // fragments of the query tile of tokens t0.. and part `part` of the heads
    auto load_q = [&](int t0, int part) {
#pragma unroll
        for (int y = 0; y < NQ; ++y) {
            const int r = i + 8 * y;
            const int tl = divided(r, p.by_G);
            const int t = t0 + (parts == 1 ? tl : 0), g = parts == 1 ? r - tl * p.G : part * ROWS + r;
            const bool on = t < p.T && g < p.G && (parts > 1 || r < per * p.G);
            const uint16_t *src = p.q + (on ? ((size_t)(use.b * p.T + t) * p.H + use.hk * p.G + g) * D + 8 * j : 0);
#pragma unroll
            for (int c = 0; c < KS / 2; ++c)
                qf[c][y] = on ? *reinterpret_cast<const uint4 *>(src + 32 * c) : make_uint4(0u, 0u, 0u, 0u);
        }
    };
    // chunk 4 c + j of row i sits at 4 (c ^ (i & 1)) + j, so that two rows' four chunks are in different banks
    const uint32_t at0 = ring + i * RB + j * 16 + (i & 1) * 64, at1 = ring + i * RB + j * 16 + (~i & 1) * 64;
    if (one_tile && n > 0) load_q(0, 0);
    for (int x = 0, stage = 0, next = NS - 1; x < n; ++x) {
        cp_async_wait<NS - 2>();
        __syncwarp();
        if (x + NS - 1 < n) issue(x + NS - 1, next);
        cp_async_commit();
        const uint32_t stage_off = stage * 2 * GB;
        const int j0 = use.g * kGroupBlocks;
        const unsigned has = s_has[warp][stage];
        uint32_t top = 0, low = 0;  // largest k_max and smallest k_min of the group, or 0

        for (int t0 = 0; t0 < p.T; t0 += per) {
            const int tokens = p.T - t0 < per ? p.T - t0 : per;
            float keep[ROWS / 2];                 // of (token t0 + y / 16, block y % 16) for outputs y of this lane
#pragma unroll
            for (int y = 0; y < ROWS / 2; ++y) keep[y] = -INFINITY;
            for (int part = 0; part < parts; ++part) {
                if (!one_tile) load_q(t0, part);
                // four chains of sums per tile (even and odd steps of both halves): a chain's products wait for one another
                float s[4][NQ][4] = {};
#pragma unroll
                for (int c = 0; c < KS / 2; ++c) {  // 32 channels: lane j has 8 j .. 8 j + 7, four of them for each product
                    const uint32_t at = (c & 1 ? at1 : at0) + (c >> 1) * 128;
                    uint4 f[2], g[2];  // of rows i and i + 8
#pragma unroll
                    for (int h = 0; h < 2; ++h) {
                        f[h] = lds_v4(at + stage_off + h * 8 * RB);
                        g[h] = lds_v4(at + stage_off + GB + h * 8 * RB);
                    }
#pragma unroll
                    for (int y = 0; y < NQ; ++y) {
                        const uint4 w = qf[c][y];
                        mma_bf16_16816(s[0][y], f[0].x, f[1].x, f[0].y, f[1].y, relu2(w.x), relu2(w.y));
                        mma_bf16_16816(s[1][y], g[0].x, g[1].x, g[0].y, g[1].y, neg2(w.x), neg2(w.y));
                        mma_bf16_16816(s[2][y], f[0].z, f[1].z, f[0].w, f[1].w, relu2(w.z), relu2(w.w));
                        mma_bf16_16816(s[3][y], g[0].z, g[1].z, g[0].w, g[1].w, neg2(w.z), neg2(w.w));
                    }
                    if (t0 == 0 && part == 0)
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            top = max2(max2(max2(max2(top, f[h].x), f[h].y), f[h].z), f[h].w);
                            low = min2(min2(min2(min2(low, g[h].x), g[h].y), g[h].z), g[h].w);
                        }
                }
                __syncwarp();
#pragma unroll
                for (int y = 0; y < NQ; ++y)
#pragma unroll
                    for (int e = 0; e < 4; ++e) s_tile[warp][8 * y + 2 * j + (e & 1)][i + 8 * (e >> 1)] = (s[0][y][e] + s[2][y][e]) + (s[1][y][e] + s[3][y][e]);
                __syncwarp();
                // maximum over the heads (a NaN stays)
                const int rows = parts == 1 ? p.G : (p.G - part * ROWS < ROWS ? p.G - part * ROWS : ROWS);
#pragma unroll
                for (int y = 0; y < ROWS / 2; ++y) {
                    const int o = y * 32 + lane, tl = o >> 4, bl = o & 15;
                    if (2 * y >= tokens) break;  // (the whole warp)
                    for (int g = 0; g < rows && tl < tokens; ++g) {
                        const float v = s_tile[warp][(parts == 1 ? tl * p.G : 0) + g][bl];
                        keep[y] = max_keep_nan(v, keep[y]);
                    }
                }
            }
#pragma unroll
            for (int y = 0; y < ROWS / 2; ++y) {
                const int o = y * 32 + lane, tl = o >> 4, bl = o & 15, t = t0 + tl;
                if (2 * y >= tokens) break;
                if (tl < tokens && j0 + bl < use.nb)
                    p.score[((size_t)(use.b * p.T + t) * p.Hkv + use.hk) * p.stride + j0 + bl] = has >> bl & 1 ? keep[y] : -INFINITY;
            }
        }
        // the largest magnitude (k_min <= k_max, so no other is larger), as the bits of a bf16 (a NaN's are the largest)
        uint32_t big = max2(top, low ^ 0x80008000u) & 0x7fff7fffu;
        big = __reduce_max_sync(ALL, big >> 16 > (big & 0xffffu) ? big >> 16 : big & 0xffffu);
        if (lane == 0) p.absmax[((size_t)use.b * p.Hkv + use.hk) * p.groups + use.g] = bf16_bits_to_float((uint16_t)big);
        if (x + 1 < n) {
            if (++use.hk == p.Hkv) {
                use.hk = 0;
                if (++use.g == use.groups) use = place(begin + x + 1);
            }
            if (one_tile) load_q(0, 0);  // (on its way while the copies are waited for)
        }
        stage = stage + 1 == NS ? 0 : stage + 1;
        next = next + 1 == NS ? 0 : next + 1;
    }
}

// Unsigned integers in the order of the values (-0 and +0 alike, NaN above all; never 0).
__device__ __forceinline__ unsigned long long ordered(double x) {
    if (x != x) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}
__device__ __forceinline__ float max_nan(float a, float b) { return a > b || a != a ? a : b; }  // a NaN stays

template <int WARPS>
__device__ __forceinline__ int block_sum(int x, int *s_red) {
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < WARPS; ++w) all += s_red[w];
    return all;
}
// One CTA per (sequence, token, kv head).  The steps are short and latency-bound (5 to 6 us for 1000 to 2000 blocks): few
// barriers, loads of a step all on their way before the first is used, and loops kept rolled otherwise, since code that
// runs once is fetched once.  At 80 registers a thread, three CTAs of 256 to an SM, 512 rows take two waves (3.5 us more).
// 256 threads while all rows run at once, 128, with less work in all, behind that: against 256 there, 1024 rows 36.0 us
// (scores and choice) for 39.6 and 2048 rows 59.3 for 67.0; against 128, 8 rows 11.0 for 12.8 and 512 rows 30.3 for 31.8.
template <int D, int THREADS>
__global__ void __launch_bounds__(THREADS, 1024 / THREADS) attn_choose_kernel(const SelectParams p) {
    extern __shared__ float s_score[];                 // as many as a row may have, kStaged at most
    uint32_t *const s_bits = reinterpret_cast<uint32_t *>(s_score) + p.staged;  // the choice, a bit per block
    constexpr int WARPS = THREADS / 32, BINS = 8 * THREADS;  // bins of a row's scores, to find the n-th highest
    __shared__ __align__(16) unsigned long long s_key[kListed];
    __shared__ int s_blk[kListed];
    __shared__ int s_red[WARPS];
    __shared__ float s_f[4][WARPS];
    __shared__ int s_near, s_sure, s_bin, s_count;
    int *const s_hist = reinterpret_cast<int *>(s_key);  // [BINS], before the keys
    static_assert(BINS * sizeof(int) <= sizeof(s_key), "the bins lie in the keys' place");
    constexpr int CPL = D / 32;                          // channels per lane
    constexpr unsigned ALL = 0xffffffffu;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int row = blockIdx.x, bt = divided(row, p.by_Hkv), b = divided(bt, p.by_T), hk = row - bt * p.Hkv, t = bt - b * p.T;
    int32_t *sel = p.sel + (size_t)row * p.n_select;

    // what the score kernel does not write, before waiting for it: lengths and the query's size
    const int nb = visible_blocks(p, b, t);
    const int words = (nb + 31) >> 5;
    const bool choose = nb > p.n_select;
    // the first and last blocks are in; k of those between, [e0, e1), are to be chosen
    const int e0 = p.n_first, e1 = nb - p.n_last, k = p.n_select - p.n_first - p.n_last;
    const uint16_t *qrow = p.q + ((size_t)(b * p.T + t) * p.H + hk * p.G) * D + lane * CPL;
    const int32_t *table = p.table + (size_t)b * p.max_blocks;
    // this lane's channels of a row of D bf16
    auto channels = [](const uint16_t *at, float (&f)[CPL]) {
#pragma unroll
        for (int c = 0; c < CPL; c += 2) {
            const uint32_t u = *reinterpret_cast<const uint32_t *>(at + c);
            f[c] = bf16_lo(u);
            f[c + 1] = bf16_hi(u);
        }
    };
    float absq = 0.f, absb = 0.f;
    if (choose) {
#pragma unroll 1
        for (int g = warp; g < p.G; g += WARPS) {
            float f[CPL], a = 0.f;
            channels(qrow + (size_t)g * D, f);
#pragma unroll
            for (int c = 0; c < CPL; ++c) a += fabsf(f[c]);
#pragma unroll
            for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(ALL, a, m);
            absq = max_nan(a, absq);
        }
        for (int x = tid; x < words; x += THREADS) {  // bits e0.. e1 - 1 open, the others in
            const int f = e0 - 32 * x, l = e1 - 32 * x, last = nb - 32 * x;
            auto below = [](int n) -> uint32_t { return n <= 0 ? 0u : n >= 32 ? ALL : (1u << n) - 1u; };
            s_bits[x] = below(f) | (below(last) & ~below(l));
        }
        for (int x = tid; x < BINS; x += THREADS) s_hist[x] = 0;
        if (tid == 0) s_near = s_sure = 0;
    }
    pdl_wait_trigger();
    if (!choose) {
        for (int x = tid; x < p.n_select; x += THREADS) sel[x] = x < nb ? x : -1;
        return;
    }

    // the scores; a block without a page below every other, but finite
    const float *row_score = p.score + (size_t)row * p.stride;
    const bool staged = nb <= p.staged;
    const int groups = (visible_blocks(p, b, p.T - 1) + kGroupBlocks - 1) / kGroupBlocks;
    const float *row_abs = p.absmax + ((size_t)b * p.Hkv + hk) * p.groups;
    if (tid < groups) absb = row_abs[tid];  // in flight together with the scores
    float lo = INFINITY, hi = -INFINITY;
#pragma unroll 1
    for (int x0 = tid; x0 < nb; x0 += 8 * THREADS) {
        float r[8];  // all on their way before the first is stored
#pragma unroll
        for (int y = 0; y < 8; ++y) r[y] = x0 + y * THREADS < nb ? row_score[x0 + y * THREADS] : 0.f;
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int x = x0 + y * THREADS;
            const float v = fmaxf(r[y], -3e38f);
            if (staged && x < nb) s_score[x] = v;
            if (x >= e0 && x < e1) {
                lo = fminf(lo, v);
                hi = fmaxf(hi, v);
            }
        }
    }
    for (int c = tid + THREADS; c < groups; c += THREADS) absb = max_nan(row_abs[c], absb);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        absb = max_nan(__shfl_xor_sync(ALL, absb, m), absb);
        lo = fminf(lo, __shfl_xor_sync(ALL, lo, m));
        hi = fmaxf(hi, __shfl_xor_sync(ALL, hi, m));
    }
    if (lane == 0) {
        s_f[0][warp] = absq;
        s_f[1][warp] = absb;
        s_f[2][warp] = lo;
        s_f[3][warp] = hi;
    }
    __syncthreads();
#pragma unroll
    for (int w = 0; w < WARPS; ++w) {
        absq = max_nan(s_f[0][w], absq);
        absb = max_nan(s_f[1][w], absb);
        lo = fminf(lo, s_f[2][w]);
        hi = fmaxf(hi, s_f[3][w]);
    }
    auto score = [&](int x) -> float { return staged ? s_score[x] : fmaxf(row_score[x], -3e38f); };

    // Bound on any score's error: 2^-16 sum |q| max |bound|.  A score is four chains of at most 4 products of 16 terms,
    // added up; a sum of 17 values that keeps 23 bits of the largest errs by at most 17 2^-23 of it, 4 times over in each
    // chain, and the chains' sizes add up to the score's: 68 2^-23, and 3 2^-24 for the last additions.
    const float size = absq * absb, err = size * 1.52587890625e-05f;

    // [low, high]: the band in which fp32 does not decide.  The k-th highest score is in the bin of scores in which the
    // count from above reaches k; a bin with many scores is split again until it is as narrow as the error.
    // Infinities, NaN and sums near the ends of fp32's range decide nothing.
    float low = -INFINITY, high = INFINITY;
    const bool usable = size > 1e-20f && size < 1e37f;
    if (k > 0 && usable) {
        int need = k;  // rank wanted among the scores in [lo, hi]
        while (hi - lo > err) {
            // (infinite for a range of zero to fp32: then NaN and infinity all go to the last bin)
            const float inv = (BINS - 1) / (hi - lo);
            for (int x = e0 + tid; x < e1; x += THREADS) {
                const float v = score(x);
                if (v >= lo && v <= hi) atomicAdd(&s_hist[(int)fminf((v - lo) * inv, BINS - 1)], 1);
            }
            __syncthreads();
            // counts from the highest bin down: thread tid has bins BINS - 8 - 8 tid .. BINS - 1 - 8 tid
            int4 *const mine = reinterpret_cast<int4 *>(s_hist) + BINS / 4 - 2 - 2 * tid;
            const int4 c = mine[1], d = mine[0];
            const int sum = (c.x + c.y + c.z + c.w) + (d.x + d.y + d.z + d.w);
            int before = sum;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_up_sync(ALL, before, m);
                if (lane >= m) before += y;
            }
            if (lane == 31) s_red[warp] = before;
            __syncthreads();
#pragma unroll
            for (int w = 0; w < WARPS; ++w) before += w < warp ? s_red[w] : 0;
            before -= sum;
            if (before < need && need <= before + sum) {  // one thread's
                const int each[8] = {c.w, c.z, c.y, c.x, d.w, d.z, d.y, d.x};
                int at = BINS - 1 - 8 * tid, n = each[0];
#pragma unroll
                for (int y = 1; y < 8; ++y)
                    if (need > before + n) {
                        before += n;
                        --at;
                        n = each[y];
                    }
                s_bin = at;
                s_count = n;
            }
            mine[0] = mine[1] = make_int4(0, 0, 0, 0);
            __syncthreads();
            // The bin's ends, wider by more than the rounding of a bin number, at most 2048 2^-22.  (That of lo itself, 2^-23 of
            // a score, is far below the error.)
            const float l = fmaxf(lo, lo + (s_bin - 0.01f) / inv), h = fminf(hi, lo + (s_bin + 1.01f) / inv);
            if (!(l > lo || h < hi)) break;
            lo = l;
            hi = h;
            if (s_count <= kFewInBin) break;
            int above = 0;  // (the widened end may take in scores of the bin above)
            for (int x = e0 + tid; x < e1; x += THREADS) above += score(x) > hi;
            need = k - block_sum<WARPS>(above, s_red);
        }
        low = lo - 2.f * err;
        high = hi + 2.f * err;
    }
    auto in_band = [&](float v) -> bool { return !usable || (v >= low && v <= high); };
    if (k > 0) {
        int sure = 0;
        for (int x = e0 + tid; x < e1; x += THREADS) {
            const float v = score(x);
            if (in_band(v)) {
                const int at = atomicAdd(&s_near, 1);  // any order: they are ranked by score and index below
                if (at < kListed) s_blk[at] = x;
            } else if (v > high) {
                ++sure;
                atomicOr(&s_bits[x >> 5], 1u << (x & 31));
            }
        }
        sure = __reduce_add_sync(ALL, sure);
        if (lane == 0 && sure) atomicAdd(&s_sure, sure);
    }
    __syncthreads();
    const int near = s_near, want = k - s_sure;
    if (want > 0 && near > want) {
        // Exact scores of the blocks in the band as integers in their order, a warp to a block.  A product of two
        // bf16 is exact in fp32 and, times a power of two that holds the sum below 2^62, in 64-bit fixed point down to
        // 2^-37 of the largest: integer sums, so equal scores are equal whatever the order.  Where the size is out of
        // fp32's comfort (infinities and NaN too) the sum is fp64's.
        const int shift = usable ? 61 - ilogbf(size) : 0;  // 2^shift size < 2^62
        const float s1 = exp2f((float)(shift / 2)), s2 = exp2f((float)(shift - shift / 2));
        // The highest of the heads' scores of block x, four heads at a time.
        auto exact = [&](int x) -> unsigned long long {
            float q[4][CPL], up[CPL], dn[CPL];
            unsigned long long best = 0;
            const int pg = table[x];
            const bool has = pg >= 0 && pg < p.n_pages;
            const size_t row = ((size_t)(has ? pg : 0) * p.Hkv + hk) * D + lane * CPL;
#pragma unroll 1
            for (int g = 0; g < p.G; g += 4) {
#pragma unroll
                for (int y = 0; y < 4; ++y) channels(qrow + (size_t)(g + y < p.G ? g + y : g) * D, q[y]);
                if (g == 0) {
                    channels(p.k_max + row, up);
                    channels(p.k_min + row, dn);
                }
                if (usable) {
                    long long s[4] = {};
#pragma unroll
                    for (int y = 0; y < 4; ++y)
#pragma unroll
                        for (int c = 0; c < CPL; ++c)
                            s[y] += __float2ll_rn(__fmul_rn(__fmul_rn(__fmul_rn(q[y][c], q[y][c] > 0.f ? up[c] : dn[c]), s1), s2));
#pragma unroll
                    for (int m = 16; m > 0; m >>= 1)
#pragma unroll
                        for (int y = 0; y < 4; ++y) s[y] += __shfl_xor_sync(ALL, s[y], m);
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        const unsigned long long o = (unsigned long long)s[y] ^ 1ull << 63;
                        best = o > best ? o : best;
                    }
                } else {
#pragma unroll 1
                    for (int y = 0; y < 4; ++y) {
                        double s = 0.0;
#pragma unroll
                        for (int c = 0; c < CPL; ++c) {
                            const float w = y == 0 ? q[0][c] : y == 1 ? q[1][c] : y == 2 ? q[2][c] : q[3][c];
                            s += (double)(w < 0.f ? 0.f : w) * (double)up[c] + (double)(w > 0.f ? 0.f : w) * (double)dn[c];
                        }
#pragma unroll
                        for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(ALL, s, m);
                        const unsigned long long o = ordered(s);
                        best = o > best ? o : best;
                    }
                }
            }
            return has ? best : usable ? 1 : ordered(-INFINITY);  // (below every finite score; among others -infinity is a score)
        };
        if (near <= kListed) {  // ranked one against another
#pragma unroll 1
            for (int c = warp; c < near; c += WARPS) {
                const unsigned long long o = exact(s_blk[c]);
                if (lane == 0) s_key[c] = o;
            }
            __syncthreads();
            for (int c = tid; c < near; c += THREADS) {
                const unsigned long long o = s_key[c];
                const int x = s_blk[c];
                int rank = 0;
                for (int y = 0; y < near; ++y) rank += s_key[y] > o || (s_key[y] == o && s_blk[y] < x);
                if (rank < want) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
            }
        } else {  // many equals (keys never written, say): by block in the workspace, 0 for those outside the band
            unsigned long long *key = p.exact + (size_t)row * p.stride;
#pragma unroll 1
            for (int x = e0 + warp; x < e1; x += WARPS) {
                const unsigned long long o = in_band(score(x)) ? exact(x) : 0;
                if (lane == 0) key[x] = o;
            }
            __syncthreads();
            // the want-th highest key: the largest klo with count(key >= klo) >= want
            unsigned long long klo = 1, khi = ~0ull;
            while (klo < khi) {
                const unsigned long long mid = khi - (khi - klo) / 2;
                int n = 0;
                for (int x = e0 + tid; x < e1; x += THREADS) n += key[x] >= mid;
                if (block_sum<WARPS>(n, s_red) >= want) klo = mid;
                else khi = mid - 1;
            }
            int above = 0;
            for (int x = e0 + tid; x < e1; x += THREADS) {
                if (key[x] > klo) {
                    ++above;
                    atomicOr(&s_bits[x >> 5], 1u << (x & 31));
                }
            }
            // and the lowest indexes among its equals: those below the largest cut that takes `equal` of them
            const int equal = want - block_sum<WARPS>(above, s_red);
            int clo = e0, chi = e1;
            while (clo < chi) {
                const int mid = chi - (chi - clo) / 2;
                int n = 0;
                for (int x = e0 + tid; x < mid; x += THREADS) n += key[x] == klo;
                if (block_sum<WARPS>(n, s_red) <= equal) clo = mid;
                else chi = mid - 1;
            }
            for (int x = e0 + tid; x < clo; x += THREADS)
                if (key[x] == klo) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
        }
    } else if (want > 0) {  // the whole band
        for (int x = e0 + tid; x < e1; x += THREADS)
            if (in_band(score(x))) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
    }
    __syncthreads();

    // the chosen indexes in ascending order
    int base = 0;
#pragma unroll 1
    for (int w0 = 0; w0 < words; w0 += THREADS) {
        const uint32_t m = w0 + tid < words ? s_bits[w0 + tid] : 0u;
        int n = __popc(m);
        const int mine = n;
#pragma unroll
        for (int y = 1; y < 32; y <<= 1) {
            const int z = __shfl_up_sync(ALL, n, y);
            if (lane >= y) n += z;
        }
        if (w0) __syncthreads();
        if (lane == 31) s_red[warp] = n;
        __syncthreads();
        int at = base + n - mine;
#pragma unroll
        for (int w = 0; w < WARPS; ++w) {
            at += w < warp ? s_red[w] : 0;
            base += s_red[w];
        }
        for (uint32_t x = m; x; x &= x - 1) {
            if (at < p.n_select) sel[at] = 32 * (w0 + tid) + __ffs(x) - 1;
            ++at;
        }
    }
}

template <int D, int NQ>
cudaError_t launch_score(const SelectParams &p, cudaStream_t st) {
    constexpr size_t ring = 4 * (size_t)score_ring<D>();
    // the shared-memory limit is a per-device attribute: raise it once on every device used
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(attn_score_kernel<D, NQ>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)(ring + (kMaxBatch + 1) * sizeof(int)));
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    const long most = ((long)p.B * p.Hkv * p.groups + 3) / 4;  // a group per warp
    const int slots = kScoreCtas * sm_count();
    return launch_kernel(attn_score_kernel<D, NQ>, dim3((unsigned)(most < slots ? most : slots)), dim3(kScoreThreads),
                         ring + (p.B + 1) * sizeof(int), st, p);
}

size_t row_stride(int max_blocks) { return round_up((size_t)max_blocks, 4); }

size_t select_ws(const hla_kv_cache *C, int B, int T, int H, int max_blocks) {
    if (check_cache(C, false, false) != HLA_OK || check_window(C, B, T, H, max_blocks) != HLA_OK || max_blocks > kMaxBlocks)
        return 0;
    const size_t rows = (size_t)B * T * C->kv_heads, groups = (max_blocks + kGroupBlocks - 1) / kGroupBlocks;
    return rows * row_stride(max_blocks) * (sizeof(unsigned long long) + sizeof(float)) + round_up((size_t)B * C->kv_heads * groups * sizeof(float), 16);
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" size_t attn_select_blocks_workspace_size(const hla_kv_cache *C, int B, int T, int H, int max_blocks) {
    return select_ws(C, B, T, H, max_blocks);
}

extern "C" int attn_select_blocks(const hla_kv_cache *C, int B, int T, int H, int max_blocks, const int32_t *block_table,
                                  const int32_t *past_len, int n_select, int n_first, int n_last, const hla_bf16 *q,
                                  int32_t *sel, void *ws, size_t ws_bytes, hla_stream stream) {
    int e = check_cache(C, false, true);
    if (e != HLA_OK) return e;
    e = check_window(C, B, T, H, max_blocks);
    if (e != HLA_OK) return e;
    HLA_REQUIRE(max_blocks <= kMaxBlocks, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(block_table && past_len && q && sel, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(n_select >= 1 && n_first >= 0 && n_last >= 0 && n_first <= n_select && n_last <= n_select - n_first, HLA_ERR_INVALID_ARG);
    // rows and groups are counted in 32 bits
    HLA_REQUIRE((long)C->n_pages * C->kv_heads < (1L << 31) && (long)B * T * C->kv_heads < (1L << 31) &&
                    (long)B * C->kv_heads * ((max_blocks + kGroupBlocks - 1) / kGroupBlocks) < (1L << 31), HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(aligned16(block_table) && aligned16(past_len) && aligned16(q) && aligned16(sel), HLA_ERR_MISALIGNED);
    HLA_REQUIRE(ws && ws_bytes >= select_ws(C, B, T, H, max_blocks), HLA_ERR_WORKSPACE);
    HLA_REQUIRE(aligned16(ws), HLA_ERR_MISALIGNED);
    SelectParams p = {};
    p.q = q; p.k_min = C->k_min; p.k_max = C->k_max; p.table = block_table; p.past = past_len; p.sel = sel;
    p.B = B; p.T = T; p.H = H; p.Hkv = C->kv_heads; p.G = H / C->kv_heads; p.d = C->head_dim;
    p.max_blocks = max_blocks; p.n_pages = C->n_pages; p.pshift = page_shift(C->page_size);
    p.n_select = n_select; p.n_first = n_first; p.n_last = n_last;
    p.stride = (int)row_stride(max_blocks);
    p.by_G = divisor(p.G); p.by_Hkv = divisor(p.Hkv); p.by_T = divisor(T);
    p.groups = (max_blocks + kGroupBlocks - 1) / kGroupBlocks;
    p.staged = max_blocks < kStaged ? max_blocks : kStaged;
    const size_t rows = (size_t)B * T * p.Hkv;
    p.exact = static_cast<unsigned long long *>(ws);
    p.score = reinterpret_cast<float *>(p.exact + rows * p.stride);
    p.absmax = p.score + rows * p.stride;
    const cudaStream_t st = (cudaStream_t)stream;
    set_variant("attn_select<d%d>", p.d);
    // the choice always follows the scores programmatically (HLA_PDL=0 turns that off as everywhere)
    PdlChain chain(st, pdl_default(1));
    e = launched(p.T * p.G <= 8 ? p.d == 128 ? launch_score<128, 1>(p, st) : launch_score<64, 1>(p, st)
                               : p.d == 128 ? launch_score<128, 2>(p, st) : launch_score<64, 2>(p, st));
    if (e != HLA_OK) return e;
    const size_t smem = p.staged * sizeof(float) + (max_blocks + 31) / 32 * sizeof(uint32_t);
    auto choose = [&](auto kernel, int threads) { return launched(launch_kernel(kernel, dim3((unsigned)rows), dim3(threads), smem, st, p)); };
    if (rows <= 4u * sm_count()) return p.d == 128 ? choose(attn_choose_kernel<128, 256>, 256) : choose(attn_choose_kernel<64, 256>, 256);
    return p.d == 128 ? choose(attn_choose_kernel<128, 128>, 128) : choose(attn_choose_kernel<64, 128>, 128);
}
