// Attention of the newest tokens of each sequence over a paged key-value cache.
//
// For a query row (sequence b, window token t, head h) over its keys c
//     s_c = scale k_scale q.k_c,   o = v_scale sum_c exp(s_c - m) v_c / sum_c exp(s_c - m),   m = max_c s_c,
// in one pass: a running maximum m, sum l and accumulator o, both rescaled when m grows; partial
// (m, l, o) of two key ranges join as m = max, l = sum l_i 2^(m_i - m), o likewise.
//
// Every cached row is needed once by the T x G query rows that share its kv head (G = H / Hkv), so the
// step is bound by reading the cache: 2 d elements per key against 4 d T G operations.  The products
// run on mma.sync (one pass of 16 rows costs 256 tensor cycles per 64 keys of d = 128, against about
// 1400 cycles of an SM's share of HBM for their 32 KB), which takes the rows in tiles of 16, 32 or 64.
//
// Work split.  A tile is 64 keys of one unit; a unit is (sequence, kv head, row tile), and for the
// sparse form (sequence, token, kv head, row tile).  The lengths live on the device, so the grid is
// fixed and every CTA takes an equal, contiguous share of all tiles, whatever the lengths are: it may
// finish one unit, run others whole and begin a last one.  A unit that one CTA holds whole is written
// out by it; the pieces of the others go to the workspace and attn_join_kernel adds them in order.
//
// Within a CTA the four warps take 16 keys of each tile each.  With 16 or 32 rows a warp runs its own
// keys against all rows, from its own ring of cp.async stages, and meets the other warps only at the
// end of a unit; with 64 rows the warps share the tile and take 16 rows each.
#include "paged.cuh"

namespace hla {
namespace {

constexpr int kTile = 64;       // keys per tile
constexpr int kGroup = 16;      // keys of a tile that one warp copies: never more than one page
constexpr int kAttnThreads = 128;
constexpr int kNoKeys = 1 << 30;  // token index of a group without keys: behind every row's last key
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnParams {
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const uint16_t *q;
    void *o;
    const int32_t *table, *past, *sel;  // sel: null for the dense form
    float *part_o, *part_ml;
    float scale;
    int B, T, H, Hkv, G;
    int max_blocks, n_pages, pshift, n_select;
    int row_tiles;    // row tiles of a unit's rows
    int units_per_b;  // units of one sequence
    int min_share;    // least tiles per CTA
    int o_bf16;
};

// Cached tokens of sequence b; negative: an idle slot.  Held below 2^30 so that token indexes stay in 32 bits
// (the table covers fewer).
__device__ __forceinline__ int cached(const AttnParams &p, int b) {
    const int x = p.past[b];
    return x < kNoKeys - 16 ? x : kNoKeys - 16;
}

// Tiles of one unit of a sequence with `past` cached tokens.
__device__ __forceinline__ int unit_tiles(const AttnParams &p, int past) {
    if (past < 0) return 0;
    if (p.sel) return (int)((((long)p.n_select << p.pshift) + kTile - 1) / kTile);
    const long cap = (long)p.max_blocks << p.pshift;
    const long len = (long)past + p.T < cap ? (long)past + p.T : cap;
    return (int)((len + kTile - 1) / kTile);
}

// Prefix sums of the sequences' tiles per unit into pre[0..B]; all threads of the block take part.
__device__ __forceinline__ void tile_prefix(const AttnParams &p, long long *pre) {
    __shared__ long long s_warp[kAttnThreads / 32];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long base = 0;
    if (tid == 0) pre[0] = 0;
    for (int b0 = 0; b0 < p.B; b0 += kAttnThreads) {
        const int b = b0 + tid;
        long long x = b < p.B ? unit_tiles(p, cached(p, b)) : 0;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const long long y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m) x += y;
        }
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        long long add = base, all = 0;
        for (int w = 0; w < kAttnThreads / 32; ++w) {
            if (w < warp) add += s_warp[w];
            all += s_warp[w];
        }
        if (b < p.B) pre[b + 1] = add + x;
        base += all;
        __syncthreads();
    }
    __syncthreads();
}

// Tiles that each CTA of the attention grid takes.
__device__ __forceinline__ long long cta_share(const AttnParams &p, long long total, int grid) {
    const long long s = (total + grid - 1) / grid;
    return s < p.min_share ? p.min_share : s;
}

// The sequence whose units hold tile t: pre[b] * units <= t < pre[b + 1] * units.
__device__ __forceinline__ int find_sequence(const long long *pre, int B, int units, long long t) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] * units <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void store_out(const AttnParams &p, size_t at, float x, float y) {
    if (p.o_bf16)
        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(p.o) + at) = pack_bf16x2(x, y);
    else
        *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.o) + at) = make_float2(x, y);
}

// Stages of the copy ring: about 96 KB per CTA, two CTAs per SM.
template <int D, bool FP8>
__host__ __device__ constexpr int ring_stages() {
    constexpr int tile_bytes = 2 * kTile * D * (FP8 ? 1 : 2);
    return 96 * 1024 / tile_bytes < 6 ? 96 * 1024 / tile_bytes : 6;
}
template <int D, bool FP8>
__host__ __device__ constexpr int warp_region() {  // shared memory of one warp's groups over all stages
    return ring_stages<D, FP8>() * 2 * kGroup * D * (FP8 ? 1 : 2);
}

// B fragments (16 keys x 8 channels) of accumulator tiles t and t + 1 (t even) from a group's V rows: f[0], f[1]
// for t and f[2], f[3] for t + 1.  bf16: tile t holds channels 8 t + n of column n.  e4m3: a transposed 8x8 of
// byte pairs gives lane (i, j) channels 8 t + 2 i, + 1 of keys 2 j, 2 j + 1, so the tiles hold the even and the
// odd channels of the 16-byte chunk t / 2.
template <int D, bool FP8>
__device__ __forceinline__ void v_fragments(uint32_t (&f)[4], uint32_t vb, int t, int lane) {
    constexpr int RB = D * (FP8 ? 1 : 2);
    if constexpr (!FP8) {
        ldmatrix_x4_trans(f, vb + swizzled<RB>(lane & 15, t + (lane >> 4)));
    } else {
        uint32_t a, b;
        ldmatrix_x2_trans(a, b, vb + swizzled<RB>(lane & 15, t >> 1));
        f[0] = e4m3x2_to_f16x2(__byte_perm(a, 0, 0x4420));
        f[1] = e4m3x2_to_f16x2(__byte_perm(b, 0, 0x4420));
        f[2] = e4m3x2_to_f16x2(__byte_perm(a, 0, 0x4431));
        f[3] = e4m3x2_to_f16x2(__byte_perm(b, 0, 0x4431));
    }
}

template <bool FP8>
__device__ __forceinline__ void mma_pv(float (&d)[4], const uint32_t (&a)[4], uint32_t b0, uint32_t b1) {
    if constexpr (FP8) mma_f16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
    else mma_bf16_16816(d, a[0], a[1], a[2], a[3], b0, b1);
}

// Whether the V rows [r0, r1] of a group hold an infinity or a NaN (the same answer in every lane).
template <int D, bool FP8>
__device__ __noinline__ bool strange_value(const uint8_t *v, int r0, int r1, int lane) {
    constexpr int RB = D * (FP8 ? 1 : 2), CPR = RB / 16;
    bool odd = false;
    r0 = r0 > 0 ? r0 : 0;
    r1 = r1 < kGroup - 1 ? r1 : kGroup - 1;
    for (int x = r0 * CPR + lane; x < (r1 + 1) * CPR; x += 32) {
        const uint4 w = *reinterpret_cast<const uint4 *>(v + swizzled<RB>(x / CPR, x % CPR));
        const uint32_t a[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int y = 0; y < 4; ++y)
            odd |= FP8 ? __vcmpeq4(a[y] & 0x7f7f7f7fu, 0x7f7f7f7fu) != 0 : __vcmpeq2(a[y] & 0x7f807f80u, 0x7f807f80u) != 0;
    }
    return __any_sync(0xffffffffu, odd);
}

// RT: 16-row tiles per warp; WR: warps that divide the rows (1: every warp has all rows and its own keys;
// 4: every warp has its own rows and all keys of the tile).
template <int D, bool FP8, int RT, int WR>
__global__ void __launch_bounds__(kAttnThreads, 2) attn_kernel(const AttnParams p) {
    constexpr int ES = FP8 ? 1 : 2, RB = D * ES, CPR = RB / 16;
    constexpr int NS = ring_stages<D, FP8>();
    constexpr int GB = kGroup * RB;           // bytes of one group's K (or V) rows
    constexpr int REGION = warp_region<D, FP8>();
    constexpr int M = 16 * RT * WR;
    constexpr int KS = D / 16, NT = D / 8;
    constexpr int PITCH = D + 8;              // fp32 row pitch of the merge buffer
    static_assert(WR == 4 || 16 * RT * PITCH * 4 <= REGION, "a warp merges its rows in its own stages");
    extern __shared__ __align__(128) uint8_t smem[];
    __shared__ long long s_pre[kMaxBatch + 1];
    __shared__ int s_tok[4][NS];              // first token of each staged group
    __shared__ float s_m[4][16 * RT], s_l[4][16 * RT];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = lane & 3, i = lane >> 2;    // fragment column pair and row
    pdl_wait_trigger();
    tile_prefix(p, s_pre);
    const long long total = s_pre[p.B] * p.units_per_b;
    const long long share = cta_share(p, total, gridDim.x);
    long long at = share * blockIdx.x;
    const long long end = at + share < total ? at + share : total;
    const uint32_t region = smem_u32(smem) + warp * REGION;

    while (at < end) {
        // ---- the piece of a unit that this CTA runs: tiles [k0, k1) of nt
        const int b = find_sequence(s_pre, p.B, p.units_per_b, at);
        const int nt = (int)(s_pre[b + 1] - s_pre[b]);
        const long long rem = at - s_pre[b] * p.units_per_b;
        int u = (int)(rem / nt);
        const int k0 = (int)(rem - (long long)u * nt);
        const int k1 = (long long)(nt - k0) < end - at ? nt : k0 + (int)(end - at);
        at += k1 - k0;
        const int rt = u % p.row_tiles;
        u /= p.row_tiles;
        const int hk = u % p.Hkv;
        const int tq = u / p.Hkv;             // sparse form: the window token
        const int past = cached(p, b);
        const int rows = p.sel ? p.G : p.T * p.G;
        // last visible token of any row of the unit, and of the row with the fewest
        const int lim_hi = p.sel ? past + tq : past + p.T - 1, lim_lo = p.sel ? past + tq : past;
        const int32_t *list = p.sel ? p.sel + ((size_t)(b * p.T + tq) * p.Hkv + hk) * p.n_select : nullptr;
        const int32_t *table = p.table + (size_t)b * p.max_blocks;

        // row r of the unit: token t, head h of q and o
        auto row_at = [&](int r) -> size_t {
            const int t = p.sel ? tq : r / p.G, g = p.sel ? r : r % p.G;
            return ((size_t)(b * p.T + t) * p.H + hk * p.G + g) * D;
        };
        const int row0 = rt * M + (WR == 4 ? warp * 16 * RT : 0);

        // ---- query fragments.  bf16: element pairs (8 c + 2 j) of chunk c.  e4m3 keys come out of ldmatrix
        // four bytes to a lane, so lane j takes elements 16 c + 4 j .. + 3 of k-step c, and the rows go to
        // fp16 scaled by a power of two that puts their largest element in [2^14, 2^15): exact down to 2^-28
        // of it; the factor comes back in the row's score scale.
        uint32_t qf[RT][KS][4];
        float sc[RT][2];
        int lim[RT][2];
        const float kscale = FP8 ? p.k_scale[hk] : 1.f;
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int r = row0 + 16 * x + 8 * hrow + i;
                const bool on = r < rows;
                const uint16_t *src = p.q + (on ? row_at(r) : 0);
                lim[x][hrow] = !on ? -1 : (p.sel ? past + tq : past + r / p.G);
                sc[x][hrow] = p.scale * kscale * kLog2e;
                if constexpr (!FP8) {
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        qf[x][c][hrow] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * c + 2 * j) : 0u;
                        qf[x][c][2 + hrow] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * c + 8 + 2 * j) : 0u;
                    }
                } else {
                    uint32_t raw[KS][2], big = 0;
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        const uint2 w = on ? *reinterpret_cast<const uint2 *>(src + 16 * c + 4 * j) : make_uint2(0u, 0u);
                        raw[c][0] = w.x;
                        raw[c][1] = w.y;
                        big = __vmaxu2(big, __vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu));
                    }
                    big = big >> 16 > (big & 0xffffu) ? big >> 16 : big & 0xffffu;
#pragma unroll
                    for (int m = 1; m < 4; m <<= 1) {
                        const uint32_t y = __shfl_xor_sync(0xffffffffu, big, m);
                        big = y > big ? y : big;
                    }
                    int e = (int)(big >> 7);                 // biased exponent of the largest element
                    e = e < 16 ? 16 : e;
                    const bool plain = e == 255;             // infinities and NaN go through unscaled
                    const float up = plain ? 1.f : __int_as_float((268 - e) << 23);
                    sc[x][hrow] *= plain ? 1.f : __int_as_float((e - 14) << 23);
#pragma unroll
                    for (int c = 0; c < KS; ++c)
#pragma unroll
                        for (int z = 0; z < 2; ++z) {
                            const __half2 h = __floats2half2_rn(bf16_lo(raw[c][z]) * up, bf16_hi(raw[c][z]) * up);
                            qf[x][c][2 * z + hrow] = *reinterpret_cast<const uint32_t *>(&h);
                        }
                }
            }

        // ---- copies.  Group `warp` of tile kt: 16 keys of one page, contiguous in memory.
        auto block_of = [&](int kt) -> int {  // logical block that holds the group (sparse: from the list)
            const int key = kt * kTile + warp * kGroup;
            const int entry = key >> p.pshift;
            if (!p.sel) return entry < p.max_blocks ? entry : -1;
            const int blk = entry < p.n_select ? list[entry] : -1;
            return blk < p.max_blocks ? blk : -1;
        };
        auto page_of = [&](int blk) -> int {
            const int pg = blk >= 0 ? table[blk] : -1;
            return pg < p.n_pages ? pg : -1;
        };
        auto issue = [&](int kt, int stage, int blk, int pg) {
            const int in_page = (kt * kTile + warp * kGroup) & ((1 << p.pshift) - 1);
            const int tok = pg >= 0 ? (blk << p.pshift) + in_page : kNoKeys;
            const int n_on = tok > lim_hi ? 0 : (lim_hi - tok + 1 < kGroup ? lim_hi - tok + 1 : kGroup);
            const size_t off = pg >= 0 ? ((((size_t)pg * p.Hkv + hk) << p.pshift) + in_page) * RB : 0;
            const uint32_t dst = region + stage * 2 * GB;
#pragma unroll
            for (int x = 0; x < GB / 512; ++x) {
                const int ch = x * 32 + lane, r = ch / CPR;
                const bool on = r < n_on;
                const size_t o = on ? off + ch * 16 : 0;
                const uint32_t d = dst + swizzled<RB>(r, ch % CPR);
                cp_async16_or_zero(d, p.k + o, on);
                cp_async16_or_zero(d + GB, p.v + o, on);
            }
            if (lane == 0) s_tok[warp][stage] = tok;
        };

        // the first tiles' lookups in one round: lane s looks up tile k0 + s
        const int n = k1 - k0;
        const int blk_l = lane <= NS && lane < n ? block_of(k0 + lane) : -1, pg_l = page_of(blk_l);
#pragma unroll
        for (int s = 0; s < NS - 1; ++s) {
            const int blk_s = __shfl_sync(0xffffffffu, blk_l, s), pg_s = __shfl_sync(0xffffffffu, pg_l, s);
            if (s < n) issue(k0 + s, s, blk_s, pg_s);
            cp_async_commit();
        }
        int blk = __shfl_sync(0xffffffffu, blk_l, NS - 1), pg = __shfl_sync(0xffffffffu, pg_l, NS - 1);
        int nblk = __shfl_sync(0xffffffffu, blk_l, NS);

        float m[RT][2], l[RT][2], acc[RT][NT][4];
#pragma unroll
        for (int x = 0; x < RT; ++x) {
            m[x][0] = m[x][1] = -INFINITY;
            l[x][0] = l[x][1] = 0.f;
#pragma unroll
            for (int t = 0; t < NT; ++t) acc[x][t][0] = acc[x][t][1] = acc[x][t][2] = acc[x][t][3] = 0.f;
        }

        for (int it = 0, stage = 0, ahead = NS - 1; it < n; ++it) {
            cp_async_wait<NS - 2>();
            if (WR == 1) __syncwarp();
            else __syncthreads();
            if (it + NS - 1 < n) issue(k0 + it + NS - 1, ahead, blk, pg);
            cp_async_commit();
            // the next tile's page and the one after's block, looked up while this tile runs
            blk = nblk;
            pg = page_of(blk);
            nblk = it + NS + 1 < n ? block_of(k0 + it + NS + 1) : -1;

#pragma unroll 1
            for (int grp = WR == 1 ? warp : 0; grp < (WR == 1 ? warp + 1 : 4); ++grp) {
                const uint32_t kb = smem_u32(smem) + grp * REGION + stage * 2 * GB, vb = kb + GB;
                const int tok = s_tok[grp][stage];
                // ---- scores of 16 keys
                float s[RT][2][4];
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int t = 0; t < 2; ++t) s[x][t][0] = s[x][t][1] = s[x][t][2] = s[x][t][3] = 0.f;
                if constexpr (!FP8) {
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        uint32_t f[4];  // keys 0-7: chunks 2c, 2c+1; keys 8-15: chunks 2c, 2c+1
                        ldmatrix_x4(f, kb + swizzled<RB>((lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)));
#pragma unroll
                        for (int x = 0; x < RT; ++x) {
                            mma_bf16_16816(s[x][0], qf[x][c][0], qf[x][c][1], qf[x][c][2], qf[x][c][3], f[0], f[1]);
                            mma_bf16_16816(s[x][1], qf[x][c][0], qf[x][c][1], qf[x][c][2], qf[x][c][3], f[2], f[3]);
                        }
                    }
                } else {
#pragma unroll
                    for (int c = 0; c < KS; c += 2) {
                        uint32_t f[4];  // keys 0-7: chunks c, c+1; keys 8-15: chunks c, c+1
                        ldmatrix_x4(f, kb + swizzled<RB>((lane & 7) + ((lane >> 4) << 3), c + ((lane >> 3) & 1)));
#pragma unroll
                        for (int z = 0; z < 4; ++z) {
                            const uint32_t b0 = e4m3x2_to_f16x2(f[z] & 0xffffu), b1 = e4m3x2_to_f16x2(f[z] >> 16);
#pragma unroll
                            for (int x = 0; x < RT; ++x)
                                mma_f16_16816(s[x][z >> 1], qf[x][c + (z & 1)][0], qf[x][c + (z & 1)][1],
                                              qf[x][c + (z & 1)][2], qf[x][c + (z & 1)][3], b0, b1);
                        }
                    }
                }
                // ---- scale, mask, running maximum
                const bool edge = tok + kGroup - 1 > lim_lo;  // some row does not see all 16
                bool grew = false;
                float mn[RT][2];
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        float top = m[x][hrow];
#pragma unroll
                        for (int t = 0; t < 2; ++t)
#pragma unroll
                            for (int e = 0; e < 2; ++e) {
                                float &v = s[x][t][2 * hrow + e];
                                v *= sc[x][hrow];
                                if (edge && tok + 8 * t + 2 * j + e > lim[x][hrow]) v = -INFINITY;
                                top = fmaxf(top, v);
                            }
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 1));
                        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, 2));
                        grew |= top > m[x][hrow];
                        mn[x][hrow] = top;
                    }
                if (__any_sync(0xffffffffu, grew)) {
#pragma unroll
                    for (int x = 0; x < RT; ++x)
#pragma unroll
                        for (int hrow = 0; hrow < 2; ++hrow) {
                            const float a = m[x][hrow] == -INFINITY ? 0.f : ex2(m[x][hrow] - mn[x][hrow]);
                            m[x][hrow] = mn[x][hrow];
                            l[x][hrow] *= a;
#pragma unroll
                            for (int t = 0; t < NT; ++t) {
                                acc[x][t][2 * hrow] *= a;
                                acc[x][t][2 * hrow + 1] *= a;
                            }
                        }
                }
                // ---- weights.  They meet V as bf16 (fp16 for an 8-bit cache, times 2^14 so that fp16 holds weights
                // down to 2^-39 of the largest); the sum l keeps fp32.  A bf16 output rounds by 2^-9 itself, so one
                // rounding of each weight, which averages out over the keys, is below it; an fp32 output gets the
                // rounded-off part in a second product, which leaves 2^-17.
                uint32_t ph[RT][4], pl[RT][4];
#pragma unroll
                for (int x = 0; x < RT; ++x)
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const float base = m[x][hrow] == -INFINITY ? 0.f : m[x][hrow] - (FP8 ? 14.f : 0.f);
#pragma unroll
                        for (int t = 0; t < 2; ++t) {
                            const float a = ex2(s[x][t][2 * hrow] - base), c = ex2(s[x][t][2 * hrow + 1] - base);
                            l[x][hrow] += a + c;
                            const int w = 2 * t + hrow;
                            if constexpr (!FP8) {
                                ph[x][w] = pack_bf16x2(a, c);
                                if (!p.o_bf16) pl[x][w] = pack_bf16x2(a - bf16_lo(ph[x][w]), c - bf16_hi(ph[x][w]));
                            } else {
                                const __half2 h = __floats2half2_rn(a, c);
                                ph[x][w] = *reinterpret_cast<const uint32_t *>(&h);
                                if (!p.o_bf16) {
                                    const float2 f = __half22float2(h);
                                    const __half2 r = __floats2half2_rn(a - f.x, c - f.y);
                                    pl[x][w] = *reinterpret_cast<const uint32_t *>(&r);
                                }
                            }
                        }
                    }
                // ---- o += P V
                // The window's own last keys are seen by some rows only.  A weight of zero does not hide an
                // infinity or NaN of such a key's value, so where one is there, these keys go one at a time
                // and a row takes up only what it sees.
                const int over = lim_hi - (tok > lim_lo + 1 ? tok : lim_lo + 1) + 1;  // keys that some rows do not see
                bool odd = false;
                if (over > 0 && tok + kGroup - 1 > lim_lo)
                    odd = strange_value<D, FP8>(smem + (vb - smem_u32(smem)), lim_lo + 1 - tok, lim_hi - tok, lane);
                if (!odd) {
#pragma unroll
                    for (int t = 0; t < NT; t += 2) {
                        uint32_t f[4];  // B fragments of accumulator tiles t (f[0], f[1]) and t + 1
                        v_fragments<D, FP8>(f, vb, t, lane);
#pragma unroll
                        for (int x = 0; x < RT; ++x) {
                            mma_pv<FP8>(acc[x][t], ph[x], f[0], f[1]);
                            mma_pv<FP8>(acc[x][t + 1], ph[x], f[2], f[3]);
                            if (!p.o_bf16) {
                                mma_pv<FP8>(acc[x][t], pl[x], f[0], f[1]);
                                mma_pv<FP8>(acc[x][t + 1], pl[x], f[2], f[3]);
                            }
                        }
                    }
                } else {
                    for (int y = tok > lim_lo + 1 ? tok - 1 : lim_lo; y <= lim_hi && y < tok + kGroup; ++y) {
                        // first pass: the keys up to lim_lo, which all rows see; then key y alone
                        const bool all = y <= lim_lo || y < tok;
                        auto keep = [&](int key) -> uint32_t { return all ? tok + key <= lim_lo : tok + key == y; };
                        const uint32_t lo = (keep(2 * j) ? 0xffffu : 0u) | (keep(2 * j + 1) ? 0xffff0000u : 0u),
                                       hi = (keep(2 * j + 8) ? 0xffffu : 0u) | (keep(2 * j + 9) ? 0xffff0000u : 0u);
#pragma unroll
                        for (int t = 0; t < NT; t += 2) {
                            uint32_t f[4];
                            v_fragments<D, FP8>(f, vb, t, lane);
#pragma unroll
                            for (int x = 0; x < RT; ++x)
#pragma unroll
                                for (int z = 0; z < 2; ++z) {
                                    float d[4] = {0.f, 0.f, 0.f, 0.f};
                                    mma_pv<FP8>(d, ph[x], f[2 * z] & lo, f[2 * z + 1] & hi);
                                    if (!p.o_bf16) mma_pv<FP8>(d, pl[x], f[2 * z] & lo, f[2 * z + 1] & hi);
#pragma unroll
                                    for (int e = 0; e < 4; ++e)
                                        if (all || y <= lim[x][e >> 1]) acc[x][t + z][e] += d[e];
                                }
                        }
                    }
                }
            }
            stage = stage + 1 == NS ? 0 : stage + 1;
            ahead = ahead + 1 == NS ? 0 : ahead + 1;
        }
        cp_async_wait<0>();
#pragma unroll
        for (int x = 0; x < RT; ++x)
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                l[x][hrow] += __shfl_xor_sync(0xffffffffu, l[x][hrow], 1);
                l[x][hrow] += __shfl_xor_sync(0xffffffffu, l[x][hrow], 2);
                // fmaxf passes over NaN scores: such a row may have no maximum, but it has seen keys and is NaN
                if (l[x][hrow] != l[x][hrow]) m[x][hrow] = INFINITY;
            }

        // ---- out: the unit whole, or a piece for the join.  Slot 2 c + 1 of CTA c holds a piece that begins its
        // unit, slot 2 c any other.
        const bool whole = k0 == 0 && k1 == nt;
        const size_t slot = 2 * (size_t)blockIdx.x + (k0 == 0);
        const float vscale = FP8 ? p.v_scale[hk] : 1.f;
        if constexpr (WR == 1) {
            float *buf = reinterpret_cast<float *>(smem + warp * REGION);
            __syncwarp();
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) {
                    const int r = 16 * x + 8 * hrow + i;
                    if (j == 0) {
                        s_m[warp][r] = m[x][hrow];
                        s_l[warp][r] = l[x][hrow];
                    }
                    if constexpr (!FP8) {
#pragma unroll
                        for (int t = 0; t < NT; ++t)
                            *reinterpret_cast<float2 *>(buf + r * PITCH + 8 * t + 2 * j) =
                                make_float2(acc[x][t][2 * hrow], acc[x][t][2 * hrow + 1]);
                    } else {
#pragma unroll
                        for (int c = 0; c < KS; ++c)
                            *reinterpret_cast<float4 *>(buf + r * PITCH + 16 * c + 4 * j) =
                                make_float4(acc[x][2 * c][2 * hrow], acc[x][2 * c + 1][2 * hrow],
                                            acc[x][2 * c][2 * hrow + 1], acc[x][2 * c + 1][2 * hrow + 1]);
                    }
                }
            __syncthreads();
            for (int y = tid; y < M * (D / 4); y += kAttnThreads) {
                const int r = y / (D / 4), c = 4 * (y % (D / 4));
                if (row0 + r >= rows) break;
                float top = s_m[0][r];
#pragma unroll
                for (int w = 1; w < 4; ++w) top = fmaxf(top, s_m[w][r]);
                float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
                float ls = 0.f;
#pragma unroll
                for (int w = 0; w < 4; ++w) {
                    const float a = s_m[w][r] == -INFINITY ? 0.f : ex2(s_m[w][r] - top);
                    const float4 f = *reinterpret_cast<const float4 *>(smem + w * REGION + (r * PITCH + c) * 4);
                    if (s_m[w][r] != -INFINITY) {
                        o.x += a * f.x; o.y += a * f.y; o.z += a * f.z; o.w += a * f.w;
                    }
                    ls += a * s_l[w][r];
                }
                if (whole) {
                    const float inv = top == -INFINITY ? 0.f : vscale / ls;
                    const size_t to = row_at(row0 + r) + c;
                    store_out(p, to, o.x * inv, o.y * inv);
                    store_out(p, to + 2, o.z * inv, o.w * inv);
                } else {
                    *reinterpret_cast<float4 *>(p.part_o + (slot * M + r) * D + c) = o;
                    if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * M + r) * 2) = make_float2(top, ls);
                }
            }
        } else {
#pragma unroll
            for (int x = 0; x < RT; ++x)
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) {
                    const int r = (warp * RT + x) * 16 + 8 * hrow + i;
                    if (rt * M + r >= rows) continue;
                    const float inv = !whole ? 1.f : (m[x][hrow] == -INFINITY ? 0.f : vscale / l[x][hrow]);
                    const size_t to = row_at(rt * M + r);
                    float *po = p.part_o + (slot * M + r) * D;
                    if (!whole && j == 0)
                        *reinterpret_cast<float2 *>(p.part_ml + (slot * M + r) * 2) = make_float2(m[x][hrow], l[x][hrow]);
#pragma unroll
                    for (int c = 0; c < NT / 2; ++c) {
                        const float *a0 = &acc[x][2 * c][2 * hrow], *a1 = &acc[x][2 * c + 1][2 * hrow];
                        // the two float pairs of this lane in tiles 2c, 2c+1 and their channels
                        const int c0 = FP8 ? 16 * c + 4 * j : 16 * c + 2 * j, c1 = FP8 ? c0 + 2 : c0 + 8;
                        const float2 f0 = FP8 ? make_float2(a0[0] * inv, a1[0] * inv) : make_float2(a0[0] * inv, a0[1] * inv);
                        const float2 f1 = FP8 ? make_float2(a0[1] * inv, a1[1] * inv) : make_float2(a1[0] * inv, a1[1] * inv);
                        if (whole) {
                            store_out(p, to + c0, f0.x, f0.y);
                            store_out(p, to + c1, f1.x, f1.y);
                        } else {
                            *reinterpret_cast<float2 *>(po + c0) = f0;
                            *reinterpret_cast<float2 *>(po + c1) = f1;
                        }
                    }
                }
        }
        __syncthreads();  // the merge buffer and s_tok are free for the next piece
    }
}

// Adds the pieces of the units that several CTAs share, in tile order, and writes zeros for the rows of
// sequences without tiles.  One block per (unit, row of the unit).
template <int D>
__global__ void __launch_bounds__(kAttnThreads) attn_join_kernel(const AttnParams p, int M, int grid) {
    __shared__ long long s_pre[kMaxBatch + 1];
    __shared__ float s_w[kAttnThreads];
    __shared__ float s_red[8];
    const int tid = threadIdx.x;
    pdl_wait_trigger();
    tile_prefix(p, s_pre);
    const int b = blockIdx.x / p.units_per_b;
    int u = blockIdx.x % p.units_per_b;
    const int r = blockIdx.y, nt = (int)(s_pre[b + 1] - s_pre[b]);
    const long long share = cta_share(p, s_pre[p.B] * p.units_per_b, grid);
    const long long first = s_pre[b] * p.units_per_b + (long long)u * nt;
    const int c_first = (int)(first / share), c_last = (int)((first + nt - 1) / share);
    if (nt > 0 && c_first == c_last) return;  // written whole
    const int rt = u % p.row_tiles;
    u /= p.row_tiles;
    const int hk = u % p.Hkv, tq = u / p.Hkv;
    const int row = rt * M + r;
    if (row >= (p.sel ? p.G : p.T * p.G)) return;
    const int t = p.sel ? tq : row / p.G, g = p.sel ? row : row % p.G;
    const size_t to = ((size_t)(b * p.T + t) * p.H + hk * p.G + g) * D;

    float o = 0.f, total = 0.f;
    float top = -INFINITY;
    const int n = nt > 0 ? c_last - c_first + 1 : 0;
    // slot of piece x of the unit
    auto slot = [&](int x) -> size_t { return 2 * (size_t)(c_first + x) + (x == 0); };
    for (int x = tid; x < n; x += kAttnThreads) top = fmaxf(top, p.part_ml[(slot(x) * M + r) * 2]);
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, m));
    if ((tid & 31) == 0) s_red[tid >> 5] = top;
    __syncthreads();
    top = fmaxf(fmaxf(s_red[0], s_red[1]), fmaxf(s_red[2], s_red[3]));
    for (int x0 = 0; x0 < n; x0 += kAttnThreads) {
        __syncthreads();
        const int x = x0 + tid;
        float w = 0.f, lw = 0.f;
        if (x < n) {
            const float2 ml = *reinterpret_cast<const float2 *>(p.part_ml + (slot(x) * M + r) * 2);
            w = ml.x == -INFINITY ? 0.f : ex2(ml.x - top);
            lw = ml.x == -INFINITY ? 0.f : w * ml.y;
        }
        s_w[tid] = w;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, m);
        if ((tid & 31) == 0) s_red[4 + (tid >> 5)] = lw;
        __syncthreads();
        total += (s_red[4] + s_red[5]) + (s_red[6] + s_red[7]);
        const int lim = n - x0 < kAttnThreads ? n - x0 : kAttnThreads;
        if (tid < D) {
#pragma unroll 8
            for (int y = 0; y < lim; ++y) {
                const float f = p.part_o[(slot(x0 + y) * M + r) * D + tid];
                if (s_w[y] != 0.f) o += s_w[y] * f;
            }
        }
    }
    if (tid < D) {
        const float inv = top == -INFINITY ? 0.f : (p.v_scale ? p.v_scale[hk] : 1.f) / total;
        const float x = o * inv;
        if (p.o_bf16) reinterpret_cast<uint16_t *>(p.o)[to + tid] = float_to_bf16_bits(x);
        else reinterpret_cast<float *>(p.o)[to + tid] = x;
    }
}

// Rows of a unit's tile: the smallest of 16, 32, 64 that holds them, 64 at most.
int tile_rows(int rows) { return rows <= 16 ? 16 : (rows <= 32 ? 32 : 64); }

int attn_grid_limit() { return 2 * sm_count(); }

size_t attn_ws(const hla_kv_cache *C, int B, int T, int H, bool sparse) {
    if (check_cache(C, false, false) != HLA_OK || check_window(C, B, T, H, 1) != HLA_OK) return 0;
    const int G = H / C->kv_heads, M = tile_rows(sparse ? G : T * G);
    return (size_t)2 * attn_grid_limit() * M * (C->head_dim + 2) * sizeof(float);
}

template <int D, bool FP8, int RT, int WR>
cudaError_t launch_attn(const AttnParams &p, int grid, cudaStream_t st) {
    constexpr size_t smem = 4 * (size_t)warp_region<D, FP8>();
    // the shared-memory limit is a per-device attribute: raise it once on every device used
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(attn_kernel<D, FP8, RT, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    return launch_kernel(attn_kernel<D, FP8, RT, WR>, dim3(grid), dim3(kAttnThreads), smem, st, p);
}

template <int D, bool FP8>
cudaError_t launch_rows(int M, const AttnParams &p, int grid, cudaStream_t st) {
    switch (M) {
        case 16: return launch_attn<D, FP8, 1, 1>(p, grid, st);
        case 32: return launch_attn<D, FP8, 2, 1>(p, grid, st);
        default: return launch_attn<D, FP8, 1, 4>(p, grid, st);
    }
}

int run_attn(const hla_kv_cache *C, int B, int T, int H, int max_blocks, const int32_t *block_table,
             const int32_t *past_len, int n_select, const int32_t *sel, bool sparse, float scale, const hla_bf16 *q,
             void *o, int o_dtype, void *ws, size_t ws_bytes, cudaStream_t st) {
    int e = check_cache(C, true, false);
    if (e != HLA_OK) return e;
    e = check_window(C, B, T, H, max_blocks);
    if (e != HLA_OK) return e;
    HLA_REQUIRE(block_table && past_len && q && o, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(o_dtype == HLA_F32 || o_dtype == HLA_BF16, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(scale == scale && scale - scale == 0.f, HLA_ERR_INVALID_ARG);  // finite
    if (sparse) {
        HLA_REQUIRE(sel && n_select >= 1, HLA_ERR_INVALID_ARG);
        HLA_REQUIRE((long)n_select * C->page_size < (1L << 30), HLA_ERR_UNSUPPORTED);
    }
    HLA_REQUIRE(aligned16(block_table) && aligned16(past_len) && aligned16(q) && aligned16(o) && aligned16(sel),
                HLA_ERR_MISALIGNED);
    HLA_REQUIRE(ws && ws_bytes >= attn_ws(C, B, T, H, sparse), HLA_ERR_WORKSPACE);
    HLA_REQUIRE(aligned16(ws), HLA_ERR_MISALIGNED);

    AttnParams p = {};
    p.k = static_cast<const uint8_t *>(C->k);
    p.v = static_cast<const uint8_t *>(C->v);
    const bool fp8 = C->dtype == HLA_E4M3;
    p.k_scale = fp8 ? C->k_scale : nullptr;
    p.v_scale = fp8 ? C->v_scale : nullptr;
    p.q = q; p.o = o; p.table = block_table; p.past = past_len; p.sel = sparse ? sel : nullptr;
    p.scale = scale;
    p.B = B; p.T = T; p.H = H; p.Hkv = C->kv_heads; p.G = H / C->kv_heads;
    p.max_blocks = max_blocks; p.n_pages = C->n_pages; p.pshift = page_shift(C->page_size);
    p.n_select = sparse ? n_select : 0;
    const int rows = sparse ? p.G : T * p.G, M = tile_rows(rows);
    p.row_tiles = (rows + M - 1) / M;
    p.units_per_b = (sparse ? T : 1) * p.Hkv * p.row_tiles;
    p.min_share = 1;
    p.o_bf16 = o_dtype == HLA_BF16;
    // no more CTAs than the longest possible sequences have tiles
    const long per_unit = ((long)(sparse ? n_select : max_blocks) * C->page_size + kTile - 1) / kTile;
    const long most = (long)B * p.units_per_b * per_unit;
    const int grid = most < attn_grid_limit() ? (int)most : attn_grid_limit();
    const int D = C->head_dim;
    p.part_o = static_cast<float *>(ws);
    p.part_ml = p.part_o + (size_t)2 * grid * M * D;

    set_variant("attn_%s<d%d,%s,m%d>", sparse ? "sparse" : "paged", D, fp8 ? "e4m3" : "bf16", M);
    PdlChain chain(st, pdl_default(B * T));
    cudaError_t ce = D == 128 ? (fp8 ? launch_rows<128, true>(M, p, grid, st) : launch_rows<128, false>(M, p, grid, st))
                              : (fp8 ? launch_rows<64, true>(M, p, grid, st) : launch_rows<64, false>(M, p, grid, st));
    e = launched(ce);
    if (e != HLA_OK) return e;
    const dim3 jg((unsigned)(B * p.units_per_b), (unsigned)(rows < M ? rows : M));
    ce = D == 128 ? launch_kernel(attn_join_kernel<128>, jg, dim3(kAttnThreads), 0, st, p, M, grid)
                  : launch_kernel(attn_join_kernel<64>, jg, dim3(kAttnThreads), 0, st, p, M, grid);
    return launched(ce);
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" size_t attn_paged_decode_workspace_size(const hla_kv_cache *C, int B, int T, int H) {
    return attn_ws(C, B, T, H, false);
}

extern "C" int attn_paged_decode(const hla_kv_cache *C, int B, int T, int H, int max_blocks, const int32_t *block_table,
                                 const int32_t *past_len, float scale, const hla_bf16 *q, void *o, int o_dtype, void *ws,
                                 size_t ws_bytes, hla_stream stream) {
    return run_attn(C, B, T, H, max_blocks, block_table, past_len, 0, nullptr, false, scale, q, o, o_dtype, ws, ws_bytes,
                    (cudaStream_t)stream);
}

extern "C" size_t attn_paged_sparse_workspace_size(const hla_kv_cache *C, int B, int T, int H) {
    return attn_ws(C, B, T, H, true);
}

extern "C" int attn_paged_sparse(const hla_kv_cache *C, int B, int T, int H, int max_blocks, const int32_t *block_table,
                                 const int32_t *past_len, int n_select, const int32_t *sel, float scale, const hla_bf16 *q,
                                 void *o, int o_dtype, void *ws, size_t ws_bytes, hla_stream stream) {
    return run_attn(C, B, T, H, max_blocks, block_table, past_len, n_select, sel, true, scale, q, o, o_dtype, ws, ws_bytes,
                    (cudaStream_t)stream);
}
