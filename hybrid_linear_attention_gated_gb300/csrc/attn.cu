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
// 1400 cycles of an SM's share of HBM for their 32 KB), which takes the rows in tiles of 16, 32 or 64;
// attn_tc.cu takes more on tcgen05.
//
// Work split.  A tile is 64 or 128 keys of one unit; a unit is (sequence, kv head, row tile), and for the
// sparse form (sequence, token, kv head, row tile).  The lengths live on the device, so the grid is
// fixed and every CTA takes an equal, contiguous share of all tiles, whatever the lengths are: it may
// finish one unit, run others whole and begin a last one.  A unit that one CTA holds whole is written
// out by it; the pieces of the others go to the workspace and attn_join_kernel adds them in order.
//
// Within a CTA a tile's keys are copied 16 or 32 to a warp, each warp into its own ring of cp.async stages.
// With 16 query rows a warp also runs its own keys against all rows and meets the other warps only at the end
// of a unit; with 32 or 64 rows, two or four warps take 16 rows each and run all keys that they copied together.
//
// Measured (CUDA graph, d = 128, 32 query heads on 8 kv heads): 64 sequences of 500 to 15500 tokens, bf16, 314 us (6.7
// TB/s) and 30000 to 65000 tokens, e4m3, 908 us (6.8 TB/s), both the copy rate; one sequence of 1021 tokens 6.1 us
// (this kernel about 4, the join the rest; 10 us called one at a time from Python), all of it dependent loads.  CTAs per SM and keys per step were swept: 32
// keys and 3 CTAs of d = 64, 2 of d = 128 (accumulators, query and scores take 255 registers a thread there).

#include <type_traits>

#include "attn.cuh"
#include "tcgen05.cuh"

namespace hla {
namespace {

// Keys that a warp copies per stage: 32, or 16 where a key's row is 256 bytes.
template <int D, bool FP8>
__host__ __device__ constexpr int warp_keys() {
    return D * (FP8 ? 1 : 2) <= 128 ? 32 : 16;
}
// CTAs per SM, which bounds the registers per thread, and stages of the copy ring.
template <int D, bool FP8, int WR>
__host__ __device__ constexpr int ctas_per_sm() {
    return D == 128 ? 2 : 3;
}
template <int D, bool FP8, int WR>
__host__ __device__ constexpr int ring_stages() {
    constexpr int tile_bytes = 8 * warp_keys<D, FP8>() * D * (FP8 ? 1 : 2), room = 216 * 1024 / ctas_per_sm<D, FP8, WR>() - 3 * 1024;
    return room / tile_bytes < 6 ? room / tile_bytes : 6;
}
template <int D, bool FP8, int WR>
__host__ __device__ constexpr int warp_region() {  // shared memory of one warp's keys over all stages
    return ring_stages<D, FP8, WR>() * 2 * warp_keys<D, FP8>() * D * (FP8 ? 1 : 2);
}

// B fragments (16 keys x 8 channels) of accumulator tiles t and t + 1 (t even) from a group's V rows: f[0], f[1]
// for t and f[2], f[3] for t + 1.  The k index of a fragment is the key.  An 8-bit transposed matrix gives a lane
// rows 4 j .. 4 j + 3, of which the product takes 0, 1 as k = 2 j, 2 j + 1 and 2, 3 as k = 2 j + 8, 2 j + 9: its
// rows are addressed in that order of keys.
template <int D, bool FP8>
__device__ __forceinline__ void v_fragments(uint32_t (&f)[4], uint32_t vb, int t, int lane) {
    constexpr int RB = D * (FP8 ? 1 : 2);
    if constexpr (!FP8) {
        ldmatrix_x4_trans(f, vb + swizzled<RB>(lane & 15, t + (lane >> 4)));
    } else {
        const int key = 2 * ((lane & 15) >> 2) + (lane & 1) + 4 * (lane & 2);
        uint32_t a, b;
        ldmatrix_trans8(a, b, vb + swizzled<RB>(key, t >> 1));
        e4m3x4_to_f16x4(a, f[0], f[1]);
        e4m3x4_to_f16x4(b, f[2], f[3]);
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

// WR: warps that divide the rows, 16 to a warp; the other 4 / WR ways divide the keys.
template <int D, bool FP8, int WR>
__global__ void __launch_bounds__(kAttnThreads, ctas_per_sm<D, FP8, WR>()) attn_kernel(const AttnParams p) {
    constexpr int ES = FP8 ? 1 : 2, RB = D * ES, CPR = RB / 16;
    constexpr int KW = warp_keys<D, FP8>(), KG = KW / kGroup, TILE = 4 * KW;
    constexpr int NS = ring_stages<D, FP8, WR>();
    constexpr int GB = kGroup * RB;           // bytes of one group's K (or V) rows
    constexpr int REGION = warp_region<D, FP8, WR>(), STAGE = 2 * KG * GB;
    constexpr int SG = KG * WR < 4 ? KG * WR : 4;  // groups that a warp scores at a time
    constexpr int M = 16 * WR, WK = 4 / WR;
    constexpr int KS = D / 16, NT = D / 8;
    constexpr uint32_t ONES = FP8 ? 0x3c003c00u : 0x3f803f80u;
    constexpr unsigned ALL = 0xffffffffu;
    static_assert(NS >= 2 && 16 * D * 4 <= STAGE, "a warp's part of a stage holds its 16 rows in fp32");
    extern __shared__ __align__(128) uint8_t smem[];
    int *const s_pre = reinterpret_cast<int *>(smem + 4 * REGION), *const s_past = s_pre + p.B + 1;  // [B + 1], [B]
    __shared__ int s_tok[4][NS][KG];          // first token of each staged group
    __shared__ float s_m[4][16], s_l[4][16];

    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int j = lane & 3, i = lane >> 2;    // fragment column pair and row
    const int wr = warp % WR, kp = warp / WR; // 16 rows and share of the keys
    pdl_wait_trigger();
    tile_prefix(p, s_pre, s_past);
    const int total = s_pre[p.B] * p.units_per_b;
    const int share = cta_share(total, gridDim.x);
    const int begin = share * (int)blockIdx.x;
    if ((long)share * blockIdx.x >= total) return;
    const int N = share < total - begin ? share : total - begin;  // this CTA's tiles
    const uint32_t ring = smem_u32(smem);
    const int rows = p.sel ? p.G : p.T * p.G;

    // The piece of a unit that tile t of all belongs to: the unit, and which of its nt tiles t is.
    struct Unit {
        int b, tq, hk, rt, nt, k;  // tq: the window token of the sparse form
    };
    auto unit_of = [&](int t) {
        Unit u;
        u.b = find_sequence(s_pre, p.B, p.units_per_b, t);
        u.nt = s_pre[u.b + 1] - s_pre[u.b];
        const int rem = t - s_pre[u.b] * p.units_per_b;
        int x = rem / u.nt;
        u.k = rem - x * u.nt;
        const int y = divided(x, p.by_row_tiles);
        u.rt = x - y * p.row_tiles;
        u.tq = divided(y, p.by_Hkv);
        u.hk = y - u.tq * p.Hkv;
        return u;
    };
    // row r of a unit: token t, head h of q and o
    auto row_at = [&](const Unit &u, int r) -> size_t {
        const int t = p.sel ? u.tq : divided(r, p.by_G), g = p.sel ? r : r - t * p.G;
        return ((size_t)(u.b * p.T + t) * p.H + u.hk * p.G + g) * D;
    };

    // ---- copies.  They run through the CTA's tiles without regard to units.  The groups that this warp copies are
    // numbered; lane l looks up group l of each 32, one batch ahead: where its 16 rows are (in units of 16 rows; -1:
    // no keys), its first token, and how many of its rows hold a key for any row of the unit.
    auto look = [&](int g0, int *at, int *tok, int *on) {
        const int g = g0 + lane;
        *at = -1;
        *tok = kNoKeys;
        *on = 0;
        if (g >= N * KG) return;
        const Unit u = unit_of(begin + g / KG);
        const int key = u.k * TILE + warp * KW + g % KG * kGroup;
        int blk = key >> p.pshift;
        if (p.sel) blk = blk < listed(p, s_past[u.b] + u.tq) ? p.sel[((size_t)(u.b * p.T + u.tq) * p.Hkv + u.hk) * p.n_select + blk] : -1;
        if (blk < 0 || blk >= p.max_blocks) return;
        const int page = p.table[(size_t)u.b * p.max_blocks + blk];
        if (page < 0 || page >= p.n_pages) return;
        const int row = key & ((1 << p.pshift) - 1), t = (blk << p.pshift) + row;
        const int seen = s_past[u.b] + (p.sel ? u.tq : p.T - 1) - t + 1;
        *tok = t;
        *on = seen < 0 ? 0 : seen < kGroup ? seen : kGroup;
        if (*on) *at = ((page * p.Hkv + u.hk) << (p.pshift - 4)) + (row >> 4);
    };
    int at_now, tok_now, on_now, at_next, tok_next, on_next;
    look(0, &at_now, &tok_now, &on_now);
    // where this lane's 16-byte chunks of a group go: chunk x * 32 + lane
    uint32_t to[GB / 512];
#pragma unroll
    for (int x = 0; x < GB / 512; ++x)
        to[x] = ring + warp * REGION + swizzled<RB>((x * 32 + lane) / CPR, lane % CPR);
    auto issue = [&](int ti, int stage) {
#pragma unroll
        for (int g = 0; g < KG; ++g) {
            const int src = (ti * KG + g) & 31;
            const int from16 = __shfl_sync(ALL, at_now, src), on = __shfl_sync(ALL, on_now, src), tok = __shfl_sync(ALL, tok_now, src);
            const uint32_t off = stage * STAGE + g * 2 * GB;
            const size_t from = (size_t)(from16 < 0 ? 0 : from16) * GB + lane * 16;
            const uint8_t *k = p.k + from, *v = p.v + from;
            if (on == kGroup) {
#pragma unroll
                for (int x = 0; x < GB / 512; ++x) {
                    cp_async16_s(to[x] + off, k + x * 512);
                    cp_async16_s(to[x] + off + GB, v + x * 512);
                }
            } else {  // rows without a key are zero: a weight of zero must not meet what the page holds there
#pragma unroll
                for (int x = 0; x < GB / 512; ++x) {
                    const bool in = (x * 32 + lane) / CPR < on;
                    cp_async16_or_zero(to[x] + off, in ? k + x * 512 : p.k, in);
                    cp_async16_or_zero(to[x] + off + GB, in ? v + x * 512 : p.v, in);
                }
            }
            if (lane == 0) s_tok[warp][stage][g] = tok;
        }
        const int seen = (ti + 1) * KG;
        if ((seen & 31) == 16) look(seen + 16, &at_next, &tok_next, &on_next);  // half a batch ahead
        if ((seen & 31) == 0) {
            at_now = at_next;
            tok_now = tok_next;
            on_now = on_next;
        }
    };

    // ---- query rows as they are in memory.  bf16: element pairs (8 c + 2 j) of chunk c.  e4m3 keys come out of ldmatrix
    // four bytes to a lane, so lane j takes elements 16 c + 4 j .. + 3 of k-step c.
    uint32_t qf[KS][4];
    auto load_q = [&](const Unit &u) {
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
            const int r = u.rt * M + 16 * wr + 8 * hrow + i;
            const bool on = r < rows;
            const uint16_t *src = p.q + (on ? row_at(u, r) : 0);
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                if constexpr (!FP8) {
                    qf[c][hrow] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * c + 2 * j) : 0u;
                    qf[c][2 + hrow] = on ? *reinterpret_cast<const uint32_t *>(src + 16 * c + 8 + 2 * j) : 0u;
                } else {
                    const uint2 w = on ? *reinterpret_cast<const uint2 *>(src + 16 * c + 4 * j) : make_uint2(0u, 0u);
                    qf[c][hrow] = w.x;
                    qf[c][2 + hrow] = w.y;
                }
            }
        }
    };

    Unit u = unit_of(begin);
    load_q(u);  // ahead of the copies in the memory system's queues
#pragma unroll
    for (int st = 0; st < NS - 1; ++st) {
        if (st < N) issue(st, st);
        cp_async_commit();
    }

    int stage = 0, ahead = NS - 1;
    for (int done = 0; done < N;) {
        // ---- the piece of a unit that this CTA runs: tiles [k0, k1) of nt
        const int nt = u.nt, k0 = u.k, k1 = nt - k0 < N - done ? nt : k0 + (N - done), first = done;
        done += k1 - k0;
        const int rt = u.rt, hk = u.hk;
        const int past = s_past[u.b];
        // last visible token of any row of the unit, and of the row with the fewest
        const int lim_hi = p.sel ? past + u.tq : past + p.T - 1, lim_lo = p.sel ? past + u.tq : past;

        // ---- query fragments.  Score scales are positive (a negative one is taken into the query), so that the running
        // maximum is that of the unscaled products.  With an 8-bit cache the rows go to fp16, scaled by a power of two
        // that puts their largest element in [2^14, 2^15): exact down to 2^-28 of it; the factor comes back in the row's
        // score scale.
        float sc[2];
        int lim[2];
        const float scale = p.scale * (FP8 ? p.k_scale[hk] : 1.f) * kLog2e;
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
            const int r = rt * M + 16 * wr + 8 * hrow + i;
            lim[hrow] = r >= rows ? -1 : past + (p.sel ? u.tq : divided(r, p.by_G));
            sc[hrow] = fmaxf(fabsf(scale), 1e-37f);  // above zero, so that -infinity stays itself
            if constexpr (!FP8) {
                if (scale < 0.f)
#pragma unroll
                    for (int c = 0; c < KS; ++c) {
                        qf[c][hrow] ^= 0x80008000u;
                        qf[c][2 + hrow] ^= 0x80008000u;
                    }
            } else {
                uint32_t big = 0;
#pragma unroll
                for (int c = 0; c < KS; ++c) big = __vmaxu2(big, __vmaxu2(qf[c][hrow] & 0x7fff7fffu, qf[c][2 + hrow] & 0x7fff7fffu));
                big = big >> 16 > (big & 0xffffu) ? big >> 16 : big & 0xffffu;
#pragma unroll
                for (int x = 1; x < 4; x <<= 1) {
                    const uint32_t y = __shfl_xor_sync(ALL, big, x);
                    big = y > big ? y : big;
                }
                int e = (int)(big >> 7);                 // biased exponent of the largest element
                e = e < 16 ? 16 : e;
                const bool plain = e == 255;             // infinities and NaN go through unscaled
                const float up = (plain ? 1.f : __int_as_float((268 - e) << 23)) * (scale < 0.f ? -1.f : 1.f);
                sc[hrow] *= plain ? 1.f : __int_as_float((e - 14) << 23);
                sc[hrow] = fmaxf(sc[hrow], 1e-37f);
#pragma unroll
                for (int c = 0; c < KS; ++c)
#pragma unroll
                    for (int z = 0; z < 4; z += 2) {
                        const __half2 h = __floats2half2_rn(bf16_lo(qf[c][z + hrow]) * up, bf16_hi(qf[c][z + hrow]) * up);
                        qf[c][z + hrow] = *reinterpret_cast<const uint32_t *>(&h);
                    }
            }
        }

        // m: running maximum of the products; base: the same, 0 while there is none.  Weights are powers of the difference
        // s - base times the scale, not of a difference of scaled products, whose rounding passes 2^127 from scores of 2^31
        // on.  The last accumulator tile is the sum of the weights as they meet V (a product with ones).
        float m[2] = {-INFINITY, -INFINITY}, base[2] = {0.f, 0.f}, acc[NT + 1][4];
#pragma unroll
        for (int t = 0; t <= NT; ++t) acc[t][0] = acc[t][1] = acc[t][2] = acc[t][3] = 0.f;

        int last = 0;  // stage of the piece's last tile
        for (int it = first; it < done; ++it) {
            cp_async_wait<NS - 2>();
            if (WR == 1) __syncwarp();
            else if (WR == 2) asm volatile("bar.sync %0, 64;" ::"r"(1 + kp) : "memory");
            else __syncthreads();
            if (it + NS - 1 < N) issue(it + NS - 1, ahead);
            cp_async_commit();

#pragma unroll 1
            for (int step = 0; step < KG * WR / SG; ++step) {
                // group g of the step: copied by warp w0 + g / KG, as its group g % KG
                const int w0 = kp * WR + step * (SG / KG);
                const uint32_t base_s = ring + w0 * REGION + stage * STAGE;
                auto group_at = [&](int g) -> uint32_t { return base_s + g / KG * REGION + g % KG * 2 * GB; };
                // ---- scores: tile 2 g + x holds keys 8 x + 2 j, + 1 of group g
                float s[2 * SG][4];
#pragma unroll
                for (int t = 0; t < 2 * SG; ++t) s[t][0] = s[t][1] = s[t][2] = s[t][3] = 0.f;
                if constexpr (!FP8) {
#pragma unroll
                    for (int c = 0; c < KS; ++c)
#pragma unroll
                        for (int g = 0; g < SG; ++g) {
                            uint32_t f[4];  // keys 0-7: chunks 2c, 2c+1; keys 8-15: chunks 2c, 2c+1
                            ldmatrix_x4(f, group_at(g) + swizzled<RB>((lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1)));
                            mma_bf16_16816(s[2 * g], qf[c][0], qf[c][1], qf[c][2], qf[c][3], f[0], f[1]);
                            mma_bf16_16816(s[2 * g + 1], qf[c][0], qf[c][1], qf[c][2], qf[c][3], f[2], f[3]);
                        }
                } else {
#pragma unroll
                    for (int c = 0; c < KS; c += 2)
#pragma unroll
                        for (int g = 0; g < SG; ++g) {
                            uint32_t f[4];  // keys 0-7: chunks c, c+1; keys 8-15: chunks c, c+1
                            ldmatrix_x4(f, group_at(g) + swizzled<RB>((lane & 7) + ((lane >> 4) << 3), c + ((lane >> 3) & 1)));
#pragma unroll
                            for (int z = 0; z < 4; ++z) {
                                uint32_t b0, b1;
                                e4m3x4_to_f16x4(f[z], b0, b1);
                                mma_f16_16816(s[2 * g + (z >> 1)], qf[c + (z & 1)][0], qf[c + (z & 1)][1], qf[c + (z & 1)][2],
                                              qf[c + (z & 1)][3], b0, b1);
                            }
                        }
                }
                // ---- mask, running maximum
                int tok[SG];
                float top[2] = {m[0], m[1]};
#pragma unroll
                for (int g = 0; g < SG; ++g) {
                    tok[g] = s_tok[w0 + g / KG][stage][g % KG];
                    if (tok[g] + kGroup - 1 > lim_lo) {  // some row does not see all 16
#pragma unroll
                        for (int x = 0; x < 2; ++x)
#pragma unroll
                            for (int e = 0; e < 4; ++e)
                                if (tok[g] + 8 * x + 2 * j + (e & 1) > lim[e >> 1]) s[2 * g + x][e] = -INFINITY;
                    }
#pragma unroll
                    for (int x = 0; x < 2; ++x)
#pragma unroll
                        for (int e = 0; e < 4; ++e) top[e >> 1] = fmaxf(top[e >> 1], s[2 * g + x][e]);
                }
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) {
                    top[hrow] = fmaxf(top[hrow], __shfl_xor_sync(ALL, top[hrow], 1));
                    top[hrow] = fmaxf(top[hrow], __shfl_xor_sync(ALL, top[hrow], 2));
                }
                if (__any_sync(ALL, top[0] > m[0] || top[1] > m[1])) {
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const float a = m[hrow] == -INFINITY ? 0.f : (m[hrow] == top[hrow] ? 1.f : ex2((m[hrow] - top[hrow]) * sc[hrow]));
                        m[hrow] = top[hrow];
                        base[hrow] = top[hrow] == -INFINITY ? 0.f : top[hrow];
#pragma unroll
                        for (int t = 0; t <= NT; ++t) {
                            acc[t][2 * hrow] *= a;
                            acc[t][2 * hrow + 1] *= a;
                        }
                    }
                }
                // ---- weights.  They meet V as bf16 (fp16 for an 8-bit cache, times 2^14 so that fp16 holds weights
                // down to 2^-39 of the largest), and what rounding took off goes through further products as long as the
                // output can show it.  One bf16 part, 2^-8, is as coarse as a bf16 output: 1.95e-3 off the exact result
                // over 64 x 8k tokens where the output's rounding alone is 1.67e-3.  With two, 2^-16, that rounding is all
                // that is left: 16 rows, which the cache bounds, have two (64 x 8k tokens 309 -> 314 us, 32 x 210k of d 64
                // 493 -> 497).  More rows, which the products bound, keep one (with two 32 rows of d 128 501 -> 527, of d 64
                // 496 -> 590, 64 of d 128 718 -> 960).  fp16's 2^-11 adds 1% to the error.  An fp32 output takes three parts
                // (fp16: two), 2^-24; with two bf16 ones it was 1.4e-6 off, twice what fp32 arithmetic is.
                auto weigh = [&](auto f32) {
                    // further products with what rounding took off: fp16 keeps 11 bits of a weight a time, bf16 8
                    constexpr bool F32 = decltype(f32)::value;
                    constexpr int EX = F32 ? (FP8 ? 1 : 2) : !FP8 && WR == 1 ? 1 : 0;
                    uint32_t ph[SG][4], pl[EX > 0 ? EX : 1][SG][4];
#pragma unroll
                    for (int hrow = 0; hrow < 2; ++hrow) {
                        const float2 minus = make_float2(-base[hrow], -base[hrow]), scale2 = make_float2(sc[hrow], sc[hrow]);
#pragma unroll
                        for (int t = 0; t < 2 * SG; ++t) {
                            float2 x = __fadd2_rn(make_float2(s[t][2 * hrow], s[t][2 * hrow + 1]), minus);
                            x = FP8 ? __ffma2_rn(x, scale2, make_float2(14.f, 14.f)) : __fmul2_rn(x, scale2);
                            const float a = ex2(x.x), c = ex2(x.y);
                            const int w = 2 * (t & 1) + hrow;
                            if constexpr (!FP8) {
                                const uint32_t h = pack_bf16x2(a, c);
                                ph[t >> 1][w] = h;
                                if constexpr (EX > 0) {
                                    const float a1 = a - bf16_lo(h), c1 = c - bf16_hi(h);
                                    const uint32_t l = pack_bf16x2(a1, c1);
                                    pl[0][t >> 1][w] = l;
                                    if constexpr (EX > 1) pl[1][t >> 1][w] = pack_bf16x2(a1 - bf16_lo(l), c1 - bf16_hi(l));
                                }
                            } else {
                                const __half2 h = __floats2half2_rn(a, c);
                                ph[t >> 1][w] = *reinterpret_cast<const uint32_t *>(&h);
                                if constexpr (EX > 0) {
                                    const float2 f = __half22float2(h);
                                    const __half2 l = __floats2half2_rn(a - f.x, c - f.y);
                                    pl[0][t >> 1][w] = *reinterpret_cast<const uint32_t *>(&l);
                                }
                            }
                        }
                    }
                    // o += P V.  The window's own last keys are seen by some rows only, and a weight of zero does not hide an
                    // infinity or NaN of such a key's value: where one is there, these keys go one at a time and a row takes
                    // up only what it sees.
#pragma unroll
                    for (int g = 0; g < SG; ++g) {
                        const uint32_t vb = group_at(g) + GB;
                        mma_pv<FP8>(acc[NT], ph[g], ONES, ONES);
#pragma unroll
                        for (int x = 0; x < EX; ++x) mma_pv<FP8>(acc[NT], pl[x][g], ONES, ONES);
                        bool odd = false;
                        if (lim_lo < lim_hi && tok[g] + kGroup - 1 > lim_lo && tok[g] <= lim_hi)
                            odd = strange_value<D, FP8>(smem + (vb - ring), lim_lo + 1 - tok[g], lim_hi - tok[g], lane);
                        if (__builtin_expect(!odd, 1)) {
#pragma unroll
                            for (int t = 0; t < NT; t += 2) {
                                uint32_t f[4];
                                v_fragments<D, FP8>(f, vb, t, lane);
                                mma_pv<FP8>(acc[t], ph[g], f[0], f[1]);
                                mma_pv<FP8>(acc[t + 1], ph[g], f[2], f[3]);
#pragma unroll
                                for (int x = 0; x < EX; ++x) {
                                    mma_pv<FP8>(acc[t], pl[x][g], f[0], f[1]);
                                    mma_pv<FP8>(acc[t + 1], pl[x][g], f[2], f[3]);
                                }
                            }
                        } else {
                            // first pass: the keys up to lim_lo, which all rows see; then key y alone
                            for (int y = tok[g] > lim_lo ? tok[g] - 1 : lim_lo; y <= lim_hi && y < tok[g] + kGroup; ++y) {
                                const bool all = y <= lim_lo || y < tok[g];
                                auto keep = [&](int key) -> bool { return all ? tok[g] + key <= lim_lo : tok[g] + key == y; };
                                const uint32_t lo = (keep(2 * j) ? 0xffffu : 0u) | (keep(2 * j + 1) ? 0xffff0000u : 0u),
                                               hi = (keep(2 * j + 8) ? 0xffffu : 0u) | (keep(2 * j + 9) ? 0xffff0000u : 0u);
#pragma unroll
                                for (int t = 0; t < NT; t += 2) {
                                    uint32_t f[4];
                                    v_fragments<D, FP8>(f, vb, t, lane);
#pragma unroll
                                    for (int z = 0; z < 2; ++z) {
                                        float d[4] = {0.f, 0.f, 0.f, 0.f};
                                        mma_pv<FP8>(d, ph[g], f[2 * z] & lo, f[2 * z + 1] & hi);
#pragma unroll
                                        for (int x = 0; x < EX; ++x) mma_pv<FP8>(d, pl[x][g], f[2 * z] & lo, f[2 * z + 1] & hi);
#pragma unroll
                                        for (int e = 0; e < 4; ++e)
                                            if (all || y <= lim[e >> 1]) acc[t + z][e] += d[e];
                                    }
                                }
                            }
                        }
                    }
                };
                if (p.o_bf16) weigh(std::false_type{});
                else weigh(std::true_type{});
            }
            last = stage;
            stage = stage + 1 == NS ? 0 : stage + 1;
            ahead = ahead + 1 == NS ? 0 : ahead + 1;
        }
        const Unit now = u;
        if (done < N) {  // the next unit's rows are on their way while this one is written out
            u = unit_of(begin + done);
            load_q(u);
        }

        // ---- the warps' parts together, each warp's in its part of the stage just read (the other stages are being filled
        // for the next unit), and out: the unit whole, or a piece for the join.  Slot 2 c + 1 of CTA c holds a piece that
        // begins its unit, slot 2 c any other.
        const bool whole = k0 == 0 && k1 == nt;
        const size_t slot = 2 * (size_t)blockIdx.x + (k0 == 0);
        const float vscale = FP8 ? p.v_scale[hk] : 1.f;
        if (WR == 1) __syncwarp();
        else __syncthreads();  // other warps read this warp's stages
        // 8-byte pairs of a row, permuted so that the eight rows of a store fall into different banks
        auto pair_at = [](int r, int c) -> int { return r * D + 2 * (c ^ 4 * (r & 7)); };
        float *const buf = reinterpret_cast<float *>(smem + warp * REGION + last * STAGE);
#pragma unroll
        for (int hrow = 0; hrow < 2; ++hrow) {
            const int r = 8 * hrow + i;
            if (j == 0) {
                // fmaxf passes over NaN scores: such a row may have no maximum, but it has seen keys and is NaN
                const float l = acc[NT][2 * hrow];
                s_m[warp][r] = l != l ? INFINITY : (m[hrow] == -INFINITY ? -INFINITY : fmaxf(m[hrow] * sc[hrow], -3e38f));
                s_l[warp][r] = l;
            }
#pragma unroll
            for (int t = 0; t < NT; ++t)
                *reinterpret_cast<float2 *>(buf + pair_at(r, 4 * t + j)) = make_float2(acc[t][2 * hrow], acc[t][2 * hrow + 1]);
        }
        __syncthreads();
        for (int y = tid; y < M * (D / 4); y += kAttnThreads) {
            const int r = y / (D / 4), c = 4 * (y % (D / 4)), rr = r & 15;
            if (rt * M + r >= rows) break;
            float top = -INFINITY, ls = 0.f;
#pragma unroll
            for (int x = 0; x < WK; ++x) top = fmaxf(top, s_m[x * WR + (r >> 4)][rr]);
            float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
            for (int x = 0; x < WK; ++x) {
                const int w = x * WR + (r >> 4);
                if (s_m[w][rr] == -INFINITY) continue;
                const float a = s_m[w][rr] == top && top != INFINITY ? 1.f : ex2(s_m[w][rr] - top);
                const float4 f = *reinterpret_cast<const float4 *>(smem + w * REGION + last * STAGE + 4 * pair_at(rr, c / 2));
                o.x += a * f.x; o.y += a * f.y; o.z += a * f.z; o.w += a * f.w;
                ls += a * s_l[w][rr];
            }
            if (whole) {
                const float inv = top == -INFINITY ? 0.f : vscale / ls;
                const size_t dst = row_at(now, rt * M + r) + c;
                store_out(p, dst, o.x * inv, o.y * inv);
                store_out(p, dst + 2, o.z * inv, o.w * inv);
            } else {
                *reinterpret_cast<float4 *>(p.part_o + (slot * M + r) * D + c) = o;
                if (c == 0) *reinterpret_cast<float2 *>(p.part_ml + (slot * M + r) * 2) = make_float2(top, ls);
            }
        }
        __syncthreads();  // the stage is free for the next tiles
    }
    cp_async_wait<0>();
}

// Adds the pieces of the units that several CTAs share, in tile order, and writes zeros for the rows of
// sequences without tiles.  Launched as a programmatic dependent of attn_kernel: what it needs first are the
// lengths, which that kernel does not write, so the blocks find out before their wait whether they have anything
// to do; block 0 always waits, so that the kernel does not complete before attn_kernel.
// A block takes one row of a unit, the blockIdx.x-th of all (by_end = 0), or with more units than CTAs in
// attn_kernel's grid, of the unit that CTA blockIdx.x begins and does not finish, if there is one: 1024 sequences
// of 200 to 600 tokens 262 us in all, 319 by unit.
template <int D>
__global__ void __launch_bounds__(D) attn_join_kernel(const AttnParams p, int M, int grid, int by_end) {
    constexpr int kAhead = 4;
    __shared__ float4 s_o[D];
    extern __shared__ int s_pre[];  // [B + 1]
    __shared__ float s_w[D];
    __shared__ float s_red[2][D / 32];
    const int tid = threadIdx.x;
    tile_prefix(p, s_pre);
    const int r = blockIdx.y, total_tiles = s_pre[p.B] * p.units_per_b, share = cta_share(total_tiles, grid);
    int b = 0, u = 0;
    bool mine = true, empty = false;  // a unit to write; sequences without tiles (by_end)
    if (!by_end) {
        b = blockIdx.x / p.units_per_b;
        u = blockIdx.x - b * p.units_per_b;
    } else {
        const long end = ((long)blockIdx.x + 1) * share;
        mine = end < total_tiles;
        if (mine) {
            b = find_sequence(s_pre, p.B, p.units_per_b, (int)end - 1);
            u = ((int)end - 1 - s_pre[b] * p.units_per_b) / (s_pre[b + 1] - s_pre[b]);
        }
        for (int x = blockIdx.x; x < p.B; x += gridDim.x) empty |= s_pre[x + 1] == s_pre[x];
    }
    const int nt = s_pre[b + 1] - s_pre[b];
    const int first = s_pre[b] * p.units_per_b + u * nt;
    const int c_first = first / share, c_last = (first + nt - 1) / share;
    const int rt = u % p.row_tiles;
    u /= p.row_tiles;
    const int hk = u % p.Hkv, tq = u / p.Hkv;
    const int row = rt * M + r;
    // written whole, no row, or another block's
    if ((nt > 0 && c_first == c_last) || row >= (p.sel ? p.G : p.T * p.G) || (by_end && c_first != blockIdx.x)) mine = false;
    if (!mine && !empty && (blockIdx.x | blockIdx.y) != 0) return;
    pdl_wait_trigger();
    if (p.force_timeout) return;
    if (empty)
        for (int x = blockIdx.x; x < p.B; x += gridDim.x)
            if (s_pre[x + 1] == s_pre[x])
                for (int y = blockIdx.y; y < p.T * p.H; y += gridDim.y) {
                    const size_t to = ((size_t)x * p.T * p.H + y) * D + tid;
                    if (p.o_bf16) reinterpret_cast<uint16_t *>(p.o)[to] = 0;
                    else reinterpret_cast<float *>(p.o)[to] = 0.f;
                }
    if (!mine) return;
    const int t = p.sel ? tq : row / p.G, g = p.sel ? row : row % p.G;
    const size_t to = ((size_t)(b * p.T + t) * p.H + hk * p.G + g) * D;

    // A quarter of the block to a piece, 4 channels to a thread, 4 pieces a thread on their way at once and the first ones
    // before their weights are known: one sequence at 1k 6.0 us, with a channel to a thread and piece after piece 7.4.
    float4 o = make_float4(0.f, 0.f, 0.f, 0.f);
    float total = 0.f, top = -INFINITY;
    const int ch = 4 * (tid % (D / 4));
    const int n = nt > 0 ? c_last - c_first + 1 : 0;
    // slot of piece x of the unit
    auto slot = [&](int x) -> size_t { return 2 * (size_t)(c_first + x) + (x == 0); };
    for (int x0 = 0; x0 < n; x0 += D) {  // the sums so far rescaled to the new maximum, as within a CTA
        const int x = x0 + tid, lim = n - x0 < D ? n - x0 : D, y1 = tid / (D / 4);
        float4 f[kAhead];  // the next pieces of this thread's, on their way before the last are used
        auto load = [&](int y0) {
#pragma unroll
            for (int y = 0; y < kAhead; ++y)
                if (y0 + 4 * y < lim) f[y] = *reinterpret_cast<const float4 *>(p.part_o + (slot(x0 + y0 + 4 * y) * M + r) * D + ch);
        };
        load(y1);
        float2 ml = make_float2(-INFINITY, 0.f);
        if (x < n) ml = *reinterpret_cast<const float2 *>(p.part_ml + (slot(x) * M + r) * 2);
        float mx = ml.x;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, m));
        if ((tid & 31) == 0) s_red[0][tid >> 5] = mx;
        __syncthreads();
        float now = top;
#pragma unroll
        for (int w = 0; w < D / 32; ++w) now = fmaxf(now, s_red[0][w]);
        const float w = ml.x == -INFINITY ? 0.f : ex2(ml.x - now);
        s_w[tid] = w;
        float lw = ml.x == -INFINITY ? 0.f : w * ml.y;
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) lw += __shfl_xor_sync(0xffffffffu, lw, m);
        if ((tid & 31) == 0) s_red[1][tid >> 5] = lw;
        __syncthreads();
        const float old = top == -INFINITY ? 0.f : ex2(top - now);
        top = now;
        o.x *= old; o.y *= old; o.z *= old; o.w *= old;
        total *= old;
#pragma unroll
        for (int y = 0; y < D / 32; ++y) total += s_red[1][y];
#pragma unroll 1
        for (int y0 = y1; y0 < lim; y0 += 4 * kAhead) {
            if (y0 != y1) load(y0);
#pragma unroll
            for (int y = 0; y < kAhead; ++y) {
                const float w = y0 + 4 * y < lim ? s_w[y0 + 4 * y] : 0.f;
                if (w != 0.f) {
                    o.x += w * f[y].x;
                    o.y += w * f[y].y;
                    o.z += w * f[y].z;
                    o.w += w * f[y].w;
                }
            }
        }
        __syncthreads();
    }
    s_o[tid] = o;
    __syncthreads();
    const float inv = top == -INFINITY ? 0.f : (p.v_scale ? p.v_scale[hk] : 1.f) / total;
    const float *const q = reinterpret_cast<const float *>(s_o) + tid;
    const float sum = (q[0] + q[D]) + (q[2 * D] + q[3 * D]);
    if (p.o_bf16) reinterpret_cast<uint16_t *>(p.o)[to + tid] = float_to_bf16_bits(sum * inv);
    else reinterpret_cast<float *>(p.o)[to + tid] = sum * inv;
}

// Rows of a unit's tile: the smallest of 16, 32, 64 that holds them, 64 at most; 128 on tcgen05 (attn_tc.cu).
int tile_rows(int rows, bool tc) { return tc ? kTcRows : rows <= 16 ? 16 : rows <= 32 ? 32 : 64; }

// More than 64 rows of bf16 keys and a bf16 output go to tcgen05.  Measured over 32 sequences of 180k to 240k tokens and
// one kv head, tcgen05 / mma.sync: 128 rows, d 128 647 / 1407 us, d 64 444 / 770.  A tile of 128 rows costs the same half
// empty: 64 rows (two kv heads of 90k to 120k tokens) take 643 / 721 and 441 / 397, and 4 sequences of 3k to 4k tokens
// 28 / 24 and 19 / 14.  (Short calls of 128 rows lose too, 26 / 22 and 22 / 16 over 4 x 6k to 8k tokens, but lengths are not
// known at launch.)
bool use_tc(int rows, int dtype, int o_dtype) { return rows > 64 && dtype == HLA_BF16 && o_dtype == HLA_BF16; }

int attn_grid_limit() { return 3 * sm_count(); }  // the most of any configuration

size_t pieces_bytes(int M, int d) { return (size_t)2 * attn_grid_limit() * M * (d + 2) * sizeof(float); }

size_t attn_ws(const hla_kv_cache *C, int B, int T, int H, bool sparse) {
    if (check_cache(C, false, false) != HLA_OK || check_window(C, B, T, H, 1) != HLA_OK) return 0;
    const int G = H / C->kv_heads, rows = sparse ? G : T * G;
    const size_t a = pieces_bytes(tile_rows(rows, false), C->head_dim), b = pieces_bytes(kTcRows, C->head_dim);
    return use_tc(rows, C->dtype, HLA_BF16) && b > a ? b : a;  // for either output type
}

template <int D, bool FP8, int WR>
cudaError_t launch_attn(const AttnParams &p, int *grid, long most, cudaStream_t st) {
    constexpr size_t ring = 4 * (size_t)warp_region<D, FP8, WR>();
    const size_t smem = ring + (2 * p.B + 1) * sizeof(int);
    // the shared-memory limit is a per-device attribute: raise it once on every device used
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(attn_kernel<D, FP8, WR>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 (int)(ring + (2 * kMaxBatch + 1) * sizeof(int)));
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    // one wave of CTAs, and no more than the longest possible sequences have tiles
    const int slots = ctas_per_sm<D, FP8, WR>() * sm_count();
    *grid = most < slots ? (int)most : slots;
    return launch_kernel(attn_kernel<D, FP8, WR>, dim3(*grid), dim3(kAttnThreads), smem, st, p);
}

template <int D, bool FP8>
cudaError_t launch_rows(int M, const AttnParams &p, int *grid, long most, cudaStream_t st) {
    switch (M) {
        case 16: return launch_attn<D, FP8, 1>(p, grid, most, st);
        case 32: return launch_attn<D, FP8, 2>(p, grid, most, st);
        default: return launch_attn<D, FP8, 4>(p, grid, most, st);
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
    const int rows = sparse ? p.G : T * p.G;
    const bool tc = use_tc(rows, C->dtype, o_dtype);
    const int M = tile_rows(rows, tc);
    p.row_tiles = (rows + M - 1) / M;
    p.units_per_b = (sparse ? T : 1) * p.Hkv * p.row_tiles;
    p.by_G = divisor(p.G); p.by_Hkv = divisor(p.Hkv); p.by_row_tiles = divisor(p.row_tiles);
    p.o_bf16 = o_dtype == HLA_BF16;
    const int tile = tc ? kTcTile
             : C->head_dim == 128 ? (fp8 ? 4 * warp_keys<128, true>() : 4 * warp_keys<128, false>())
                                : (fp8 ? 4 * warp_keys<64, true>() : 4 * warp_keys<64, false>());
    const long per_unit = ((long)(sparse ? n_select : max_blocks) * C->page_size + tile - 1) / tile;
    p.tshift = __builtin_ctz(tile);
    const long most = (long)B * p.units_per_b * per_unit;  // tiles, if every sequence filled its table
    // (share * CTA, up to a grid above it, stays in 32 bits)
    HLA_REQUIRE(most < 2000000000L && (long)C->n_pages * C->kv_heads * (C->page_size / kGroup) < (1L << 31), HLA_ERR_UNSUPPORTED);
    const int D = C->head_dim;
    p.part_o = static_cast<float *>(ws);
    p.part_ml = p.part_o + (size_t)2 * attn_grid_limit() * M * D;
    if (tc) {
        p.status = device_status_word();
        HLA_REQUIRE(p.status, HLA_ERR_CUDA);
        p.force_timeout = wait_timeout_forced();
    }

    set_variant("attn_%s<d%d,%s,m%d>", sparse ? "sparse" : "paged", D, fp8 ? "e4m3" : "bf16", M);
    // the join always follows attn_kernel programmatically (HLA_PDL=0 turns that off as everywhere)
    PdlChain chain(st, pdl_default(1));
    int grid = 0;
    cudaError_t ce = tc ? launch_attn_tc(D, p, &grid, most, st)
                     : D == 128 ? (fp8 ? launch_rows<128, true>(M, p, &grid, most, st) : launch_rows<128, false>(M, p, &grid, most, st))
                              : (fp8 ? launch_rows<64, true>(M, p, &grid, most, st) : launch_rows<64, false>(M, p, &grid, most, st));
    e = launched(ce);
    if (e != HLA_OK) return e;
    const bool by_end = B * p.units_per_b > grid;
    const dim3 jg((unsigned)(by_end ? grid : B * p.units_per_b), (unsigned)(rows < M ? rows : M));
    const size_t js = (B + 1) * sizeof(int);
    ce = D == 128 ? launch_kernel(attn_join_kernel<128>, jg, dim3(128), js, st, p, M, grid, (int)by_end)
                  : launch_kernel(attn_join_kernel<64>, jg, dim3(64), js, st, p, M, grid, (int)by_end);
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
