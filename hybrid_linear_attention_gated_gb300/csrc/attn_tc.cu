// The paged attention of more than 64 query rows per kv head (a speculative window of a model with few kv heads) on
// tcgen05: there mma.sync, not memory, bounds the warps' form in attn.cu.
//
// A CTA owns 128 rows (padded), one per thread, and runs the same equal share of tiles as attn_kernel, 64 keys a
// tile.  Per tile
//     S = Q K^T        tcgen05.mma 128 x 64 x d, both operands K-major in shared memory, S in tensor memory;
//     P = 2^(S - m)    a thread reads its row of S, keeps m and l, writes its row of P as bf16 to shared memory;
//     O += P V         tcgen05.mma 128 x d x 64, V as it lies in the cache (its channels contiguous: MN-major).
// O stays in tensor memory.  A row's m is raised, and O rescaled, only when a score passes it by 2^8 (a known way to spare
// rescaling: any m near the maximum will do, since it cancels): until then the weights stay below 2^8, which bf16 and the
// fp32 sums hold as well as 1.
//
// Keys and values come through two stages of cp.async in the 128-byte swizzle.  A tile is a chain of short steps
// (product, row of S, weights, product: about 3700 cycles for d = 128), so what counts is CTAs per SM that fill one
// another's gaps: two of d = 128 and three of d = 64 with 64-key tiles and two stages (when compared, 727 and 516 us for
// 128 rows over 32 sequences of 180k to 240k tokens) against one with 128-key tiles or four stages (1021 to 1200 us, 526
// to 640).  Now 647 and 444 us, 5.3 and 3.9 TB/s; what is left of the time is that chain.
//
// The keys that all rows see (up to past) go through the tiles; the window's own T - 1 last keys, which a row sees in
// part, are taken up on CUDA cores at the end of the unit, row by row, so that no weight of zero meets their values.
// They are fetched into shared memory together: read by each row from global memory, one after another, they made 8-token
// windows of 4 sequences of 6k to 8k tokens 44 us for 33.
//
// Every wait is bounded (as in tc_gemm.cu): a wait that gives up sets the device status word, and after the next
// block barrier every thread leaves the loop; the MMAs issued are waited for once more before tensor memory is freed.
#include "attn.cuh"
#include "tcgen05.cuh"

namespace hla {
namespace {

constexpr uint64_t kWaitNs = 2000000000ull;  // 2 s of %globaltimer per bounded wait
constexpr uint32_t kSub = kTcRows * 128;     // bytes of 128 rows of one 128-byte-wide swizzled block (Q, P)
constexpr uint32_t kKvSub = kTcTile * 128;   // of the 64 rows of a tile's K or V
constexpr int kStages = 2;                   // tiles in shared memory: one on its way while one is worked on

// Sequences whose prefix sums of tiles and lengths a CTA keeps: all that there can be, or with more only every 2nd, 4th,
// 8th or 16th prefix sum, from which the lengths themselves lead on.
template <int D>
__host__ __device__ constexpr int kept() {
    return D == 64 ? kMaxBatch : 112;
}
template <int D>
__host__ __device__ constexpr uint32_t tc_smem(int B) {  // Q, K and V stages, P; barriers and the tensor memory's address; s_on; s_pre, s_past
    return (D / 64) * kSub + 2 * kStages * (D / 64) * kKvSub + kSub + 32 + kStages * 16 + (2 * (B < kept<D>() ? B : kept<D>()) + 1) * 4;
}
template <int D>
__host__ __device__ constexpr int tc_ctas() {  // per SM
    return D == 64 ? 3 : 2;
}
// A CTA's shared memory is rounded up to 128 bytes and costs 1 KB more.  With 8 bytes per sequence in it, two CTAs of
// d = 128 fitted up to 119 sequences only: 128 rows over 6.7 million tokens 681 us for 119 of them, 1067 for 120 and 1267
// for 1024 (now 683 and 877).
template <int D>
constexpr bool fits() {
    return tc_ctas<D>() * ((tc_smem<D>(kMaxBatch) + 127) / 128 * 128 + 1024) <= 228 * 1024;
}
static_assert(fits<64>() && fits<128>(), "tc_ctas CTAs on an SM, whatever the batch");
static_assert((kMaxBatch + 1) * sizeof(int) <= kSub, "the prefix sums of all sequences pass through P's place");
template <int D>
__host__ __device__ constexpr uint32_t tmem_columns() {  // 64 of S, D of O
    return D == 64 ? 128 : 256;
}

// A bounded wait whose first polls do not read the clock (a read of %globaltimer takes longer than most waits here).
__device__ __forceinline__ bool wait_phase(uint64_t *bar, uint32_t parity, int *status) {
    const uint32_t a = smem_u32(bar);
#pragma unroll 1
    for (int i = 0; i < 64; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(a), "r"(parity)
            : "memory");
        if (done) return true;
    }
    return mbar_wait_for(bar, parity, kWaitNs, status);
}

__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async.shared::cta;" ::: "memory"); }

template <int D>
__global__ void __launch_bounds__(kAttnThreads, tc_ctas<D>()) attn_tc_kernel(const AttnParams p) {
    constexpr int RB = 2 * D, CPR = RB / 16, GB = kGroup * RB, NB = D / 64, M = kTcRows;
    constexpr uint32_t IS = idesc_bf16(M, kTcTile), IO = idesc_bf16(M, D, true);
    constexpr unsigned ALL = 0xffffffffu;
    extern __shared__ __align__(1024) uint8_t smem[];  // (and no static shared memory in front of it)
    uint8_t *const sQ = smem, *const sK = sQ + NB * kSub, *const sV = sK + kStages * NB * kKvSub,
            *const sP = sV + kStages * NB * kKvSub;
    uint64_t &bar_s = reinterpret_cast<uint64_t *>(sP + kSub)[0], &bar_o = (&bar_s)[1], &bar_end = (&bar_s)[2];
    uint32_t &s_tmem = *reinterpret_cast<uint32_t *>(&bar_s + 3);
    int (*const s_on)[4] = reinterpret_cast<int (*)[4]>(&bar_s + 4);  // [kStages]: rows with a key of each staged group
    int *const s_pre = &s_on[kStages][0], *const s_past = s_pre + p.B + 1;  // [B + 1], [B]; with more than kept: [kept + 1], none
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    pdl_wait();
    if (p.force_timeout) {
        if (blockIdx.x == 0 && tid == 0) {
            mbar_init(&bar_s, 1);
            asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
            mbar_wait_for(&bar_s, 0, 1000000ull, p.status);  // nothing arrives: gives up after 1 ms
            asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(&bar_s)) : "memory");
        }
        return;
    }
    // s_pre[x]: tiles per unit of the sequences before sequence x << skip.  s_past: all lengths, if they fit
    int skip = 0;
    if constexpr (kept<D>() < kMaxBatch)
        while (p.B > kept<D>() << skip) ++skip;
    const int nx = (p.B + (1 << skip) - 1) >> skip;
    int *const pre = skip ? reinterpret_cast<int *>(sP) : s_pre;  // (P's place is not in use yet)
    tile_prefix(p, pre, skip ? nullptr : s_past);
    if (skip) {
        for (int x = tid; x <= nx; x += kAttnThreads) s_pre[x] = pre[x << skip < p.B ? x << skip : p.B];
        __syncthreads();
    }
    auto past_of = [&](int b) -> int { return skip ? cached(p, b) : s_past[b]; };
    const int total = s_pre[nx] * p.units_per_b;
    const int share = cta_share(total, gridDim.x);
    const int begin = (long)share * blockIdx.x < total ? share * (int)blockIdx.x : total;
    const int N = share < total - begin ? share : total - begin;  // this CTA's tiles
    if (N == 0) return;
    const int rows = p.sel ? p.G : p.T * p.G;

    if (tid == 0) {
        mbar_init(&bar_s, 1);
        mbar_init(&bar_o, 1);
        mbar_init(&bar_end, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == 0) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&s_tmem)),
                     "r"(tmem_columns<D>())
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    pdl_trigger();  // only now: a dependent that allocates tensor memory must not get it before this CTA
    const uint32_t tm_s = s_tmem, tm_o = s_tmem + kTcTile;  // 64 columns of S, D of O
    const uint32_t my_lanes = (uint32_t)(warp * 32) << 16;

    struct Unit {
        int b, tq, hk, rt, nt, k;
    };
    auto unit_of = [&](int t) {
        Unit u;
        const int x0 = find_sequence(s_pre, nx, p.units_per_b, t);
        int at = s_pre[x0];  // tiles per unit before sequence u.b
        u.b = x0 << skip;
        u.nt = skip ? unit_tiles(p, past_of(u.b)) : s_pre[x0 + 1] - at;
        if (skip)
            while (u.b + 1 < p.B && (at + u.nt) * p.units_per_b <= t) {
                at += u.nt;
                u.nt = unit_tiles(p, past_of(++u.b));
            }
        const int rem = t - at * p.units_per_b;
        const int x = rem / u.nt;
        u.k = rem - x * u.nt;
        const int y = divided(x, p.by_row_tiles);
        u.rt = x - y * p.row_tiles;
        u.tq = divided(y, p.by_Hkv);
        u.hk = y - u.tq * p.Hkv;
        return u;
    };
    auto row_at = [&](const Unit &u, int r) -> size_t {
        const int t = p.sel ? u.tq : divided(r, p.by_G), g = p.sel ? r : r - t * p.G;
        return ((size_t)(u.b * p.T + t) * p.H + u.hk * p.G + g) * D;
    };
    // page of logical block blk of sequence b, or -1
    auto page_of = [&](int b, int blk) -> int {
        if (blk < 0 || blk >= p.max_blocks) return -1;
        const int page = p.table[(size_t)b * p.max_blocks + blk];
        return page < p.n_pages ? page : -1;
    };

    // ---- copies, as in attn_kernel: 16 keys per warp and tile, lane l looks up tile l of each 32
    auto look = [&](int g0, int *at, int *on) {
        *at = -1;
        *on = 0;
        if (g0 + lane >= N) return;
        const Unit u = unit_of(begin + g0 + lane);
        const int key = u.k * kTcTile + warp * kGroup;
        const int limit = past_of(u.b) + (p.sel ? u.tq : 0);  // last position that all rows see
        int blk = key >> p.pshift;
        if (p.sel) blk = blk < listed(p, limit) ? p.sel[((size_t)(u.b * p.T + u.tq) * p.Hkv + u.hk) * p.n_select + blk] : -1;
        const int page = page_of(u.b, blk);
        if (page < 0) return;
        const int row = key & ((1 << p.pshift) - 1), seen = limit - ((blk << p.pshift) + row) + 1;
        *on = seen < 0 ? 0 : seen < kGroup ? seen : kGroup;
        if (*on) *at = ((page * p.Hkv + u.hk) << (p.pshift - 4)) + (row >> 4);
    };
    int at_now, on_now, at_next, on_next;
    look(0, &at_now, &on_now);
    uint32_t to[GB / 512];  // this lane's chunks of a group in a stage
#pragma unroll
    for (int x = 0; x < GB / 512; ++x) {
        const int r = (x * 32 + lane) / CPR, c = (x * 32 + lane) % CPR;
        to[x] = (c >> 3) * kKvSub + (warp * kGroup + r) * 128 + (((c & 7) ^ (r & 7)) << 4);
    }
    const uint32_t k_ring = smem_u32(sK), v_ring = smem_u32(sV);
    auto issue = [&](int ti) {
        const uint32_t st = ti % kStages * NB * kKvSub;
        const int from16 = __shfl_sync(ALL, at_now, ti & 31), on = __shfl_sync(ALL, on_now, ti & 31);
        const size_t from = (size_t)(from16 < 0 ? 0 : from16) * GB + lane * 16;
        const uint8_t *k = p.k + from, *v = p.v + from;
        if (on == kGroup) {
#pragma unroll
            for (int x = 0; x < GB / 512; ++x) {
                cp_async16_s(k_ring + st + to[x], k + x * 512);
                cp_async16_s(v_ring + st + to[x], v + x * 512);
            }
        } else {
#pragma unroll
            for (int x = 0; x < GB / 512; ++x) {
                const bool in = (x * 32 + lane) / CPR < on;
                cp_async16_or_zero(k_ring + st + to[x], in ? k + x * 512 : p.k, in);
                cp_async16_or_zero(v_ring + st + to[x], in ? v + x * 512 : p.v, in);
            }
        }
        if (lane == 0) s_on[ti % kStages][warp] = on;
        if ((ti & 31) == 15) look(ti + 17, &at_next, &on_next);
        if ((ti & 31) == 31) {
            at_now = at_next;
            on_now = on_next;
        }
    };

#pragma unroll
    for (int x = 0; x < kStages - 1; ++x) {
        if (x < N) issue(x);
        cp_async_commit();
    }
    const uint64_t q_desc = sw128_desc(smem_u32(sQ)), k_desc = sw128_desc(k_ring), p_desc = sw128_desc(smem_u32(sP)),
                   v_desc = sw128_desc_mn(v_ring, kKvSub);
    const float sc = fmaxf(fabsf(p.scale) * kLog2e, 1e-37f);  // a negative scale is taken into the query
    bool ok = true, all_ok = true;                            // no wait of this thread, of any thread, has given up
    for (int done = 0; done < N && all_ok;) {
        const Unit u = unit_of(begin + done);
        const int k0 = u.k, k1 = u.nt - k0 < N - done ? u.nt : k0 + (N - done), first = done;
        done += k1 - k0;
        const int past = past_of(u.b), lim_lo = p.sel ? past + u.tq : past, lim_hi = p.sel ? lim_lo : past + p.T - 1;
        const int r = u.rt * M + tid;  // this thread's row of the unit
        const bool live = r < rows;

        // ---- Q: thread's own row into the K-major tile (the last unit's products with it are complete)
        {
            const uint16_t *src = p.q + (live ? row_at(u, r) : 0);
            const uint32_t flip = p.scale < 0.f ? 0x80008000u : 0u;
#pragma unroll
            for (int c = 0; c < CPR; ++c) {
                uint4 w = live ? ld_act_v4(src + 8 * c) : make_uint4(0u, 0u, 0u, 0u);
                w.x ^= flip; w.y ^= flip; w.z ^= flip; w.w ^= flip;
                *reinterpret_cast<uint4 *>(sQ + (c >> 3) * kSub + tid * 128 + (((c & 7) ^ (tid & 7)) << 4)) = w;
            }
        }
        float m = 0.f, l = 0.f;   // of the products; weights are powers of (s - m) sc, as in attn_kernel
        bool none = true;         // no score yet
        for (int it = first; it < done; ++it) {
            const int st = it % kStages;
            cp_async_wait<kStages - 2>();
            fence_async();
            tc_fence_before();
            all_ok = __syncthreads_and(ok);  // tile `it` is in shared memory, and every thread is done with tile it - 1
            if (!all_ok) break;
            if (tid == 0) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < D / 16; ++c) {
                    const uint32_t off = (c & 3) * 32;  // (a descriptor counts addresses in 16 bytes)
                    umma_bf16(tm_s, q_desc + (((c >> 2) * kSub + off) >> 4),
                              k_desc + (st * NB * kKvSub >> 4) + (((c >> 2) * kKvSub + off) >> 4), IS, c > 0);
                }
                umma_commit(&bar_s);
            }
            // the previous tile's stage and P are free once its output product is complete
            if (it > 0) ok &= wait_phase(&bar_o, (it - 1) & 1, p.status);
            __syncwarp();
            if (it + kStages - 1 < N) issue(it + kStages - 1);
            cp_async_commit();
            ok &= wait_phase(&bar_s, it & 1, p.status);
            __syncwarp();
            tc_fence_after();

            // ---- this thread's row of S
            uint32_t sr[kTcTile];
#pragma unroll
            for (int c = 0; c < kTcTile; c += 32) tmem_ld32(tm_s + my_lanes + c, sr + c);
            tmem_wait_ld();
            float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
            for (int g = 0; g < kTcTile / kGroup; ++g) {
                const int on = s_on[st][g];
                if (on < kGroup) {
#pragma unroll
                    for (int x = 0; x < kGroup; ++x)
                        if (x >= on) sr[16 * g + x] = 0xff800000u;  // -infinity
                }
#pragma unroll
                for (int x = 0; x < kGroup; ++x) m4[x & 3] = fmaxf(m4[x & 3], __uint_as_float(sr[16 * g + x]));
            }
            const float mx = fmaxf(fmaxf(m4[0], m4[1]), fmaxf(m4[2], m4[3]));
            if (none && mx != -INFINITY) {
                m = mx;
                none = false;
            }
            const bool far = !none && (mx - m) * sc > 8.f;
            if (__any_sync(ALL, far)) {  // (never in the unit's first tile, where O is not there yet)
                const float a = far ? ex2((m - mx) * sc) : 1.f;
                if (far) m = mx;
                l *= a;
                uint32_t o[32];
#pragma unroll
                for (int c = 0; c < D; c += 32) {
                    tmem_ld32(tm_o + my_lanes + c, o);
                    tmem_wait_ld();
#pragma unroll
                    for (int x = 0; x < 32; ++x) o[x] = __float_as_uint(__uint_as_float(o[x]) * a);
                    tmem_st32(tm_o + my_lanes + c, o);
                }
                tmem_wait_st();
            }
            // ---- weights: rounded once to bf16, as in attn_kernel for more than 16 rows, and summed as they are then: a row
            // that one key dominates keeps that key's value (weights of 2^8 at most are no powers of two, so the sum before
            // rounding is up to 2^-8 off theirs)
            float2 ls[4] = {};
            const float2 sc2 = make_float2(sc, sc), m2 = make_float2(-m, -m);
#pragma unroll
            for (int c = 0; c < kTcTile / 8; ++c) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x) {
                    float2 y = __fmul2_rn(__fadd2_rn(make_float2(__uint_as_float(sr[8 * c + 2 * x]), __uint_as_float(sr[8 * c + 2 * x + 1])), m2), sc2);
                    y = make_float2(ex2(y.x), ex2(y.y));
                    w[x] = pack_bf16x2(y.x, y.y);
                    ls[x] = __fadd2_rn(ls[x], make_float2(bf16_lo(w[x]), bf16_hi(w[x])));
                }
                *reinterpret_cast<uint4 *>(sP + tid * 128 + ((c ^ (tid & 7)) << 4)) = make_uint4(w[0], w[1], w[2], w[3]);
            }
            l += ((ls[0].x + ls[0].y) + (ls[1].x + ls[1].y)) + ((ls[2].x + ls[2].y) + (ls[3].x + ls[3].y));
            fence_async();
            tc_fence_before();
            all_ok = __syncthreads_and(ok);
            if (!all_ok) break;
            if (tid == 0) {
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < kTcTile / 16; ++c)
                    umma_bf16(tm_o, p_desc + (c * 32 >> 4), v_desc + (st * NB * kKvSub >> 4) + (c * 2048 >> 4), IO,
                              it > first || c > 0);
                umma_commit(&bar_o);
            }
        }
        if (!all_ok) break;
        ok &= wait_phase(&bar_o, (done - 1) & 1, p.status);
        __syncwarp();

        // ---- the window's own keys: their rows go to P's place, which is free since its last product is complete
        const bool window = k1 == u.nt && lim_hi > lim_lo;
        int *const s_page = reinterpret_cast<int *>(sP + (kMaxWindowTokens - 1) * 2 * RB);
        if (window) {
#pragma unroll 1
            for (int x = tid; x < (lim_hi - lim_lo) * 2 * CPR; x += kAttnThreads) {
                const int own = x / (2 * CPR), c = lim_lo + 1 + own, pg = page_of(u.b, c >> p.pshift);
                if (x % (2 * CPR) == 0) s_page[own] = pg;
                if (pg < 0) continue;
                const size_t at = ((((size_t)pg * p.Hkv + u.hk) << p.pshift) + (c & ((1 << p.pshift) - 1))) * RB + x % CPR * 16;
                *reinterpret_cast<uint4 *>(sP + x * 16) = ld_act_v4((x % (2 * CPR) < CPR ? p.k : p.v) + at);
            }
            __syncthreads();
        }

        // ---- this thread's row of O, and those keys
        tc_fence_after();
        uint32_t o[D];
#pragma unroll
        for (int c = 0; c < D; c += 32) tmem_ld32(tm_o + my_lanes + c, o + c);
        tmem_wait_ld();
        tc_fence_before();
        const int lim = live ? past + (p.sel ? u.tq : divided(r, p.by_G)) : -1;
        if (window)
            for (int c = lim_lo + 1; c <= lim_hi && c <= lim; ++c) {
                const int own = c - lim_lo - 1;
                if (s_page[own] < 0) continue;
                const uint8_t *const kr = sP + own * 2 * RB, *const vr = kr + RB;
                float s = 0.f;
#pragma unroll 4
                for (int x = 0; x < CPR; ++x) {
                    const uint4 a = *reinterpret_cast<const uint4 *>(sQ + (x >> 3) * kSub + tid * 128 + (((x & 7) ^ (tid & 7)) << 4)),
                                b = *reinterpret_cast<const uint4 *>(kr + 16 * x);
                    s += bf16_lo(a.x) * bf16_lo(b.x) + bf16_hi(a.x) * bf16_hi(b.x);
                    s += bf16_lo(a.y) * bf16_lo(b.y) + bf16_hi(a.y) * bf16_hi(b.y);
                    s += bf16_lo(a.z) * bf16_lo(b.z) + bf16_hi(a.z) * bf16_hi(b.z);
                    s += bf16_lo(a.w) * bf16_lo(b.w) + bf16_hi(a.w) * bf16_hi(b.w);
                }
                float a = 1.f;
                if (s != -INFINITY && (none || s > m)) {
                    a = none ? 1.f : ex2((m - s) * sc);
                    m = s;
                    none = false;
                }
                const float w = ex2((s - m) * sc);
                l = l * a + w;
#pragma unroll
                for (int x = 0; x < CPR; ++x) {
                    const uint4 b = *reinterpret_cast<const uint4 *>(vr + 16 * x);
                    const uint32_t bw[4] = {b.x, b.y, b.z, b.w};
#pragma unroll
                    for (int y = 0; y < 4; ++y) {
                        uint32_t &lo = o[8 * x + 2 * y], &hi = o[8 * x + 2 * y + 1];
                        lo = __float_as_uint(fmaf(w, bf16_lo(bw[y]), __uint_as_float(lo) * a));
                        hi = __float_as_uint(fmaf(w, bf16_hi(bw[y]), __uint_as_float(hi) * a));
                    }
                }
            }
        // ---- out: the unit whole, or a piece for the join (slots as in attn_kernel).  A row of NaN scores only has no
        // maximum, but it has seen keys and is NaN.
        const float top = l != l ? INFINITY : none ? -INFINITY : fmaxf(m * sc, -3e38f);
        if (live && k0 == 0 && k1 == u.nt) {
            const float inv = top == -INFINITY ? 0.f : 1.f / l;
            uint16_t *dst = static_cast<uint16_t *>(p.o) + row_at(u, r);
#pragma unroll
            for (int c = 0; c < D; c += 8) {
                uint32_t w[4];
#pragma unroll
                for (int x = 0; x < 4; ++x)
                    w[x] = pack_bf16x2(__uint_as_float(o[c + 2 * x]) * inv, __uint_as_float(o[c + 2 * x + 1]) * inv);
                *reinterpret_cast<uint4 *>(dst + c) = make_uint4(w[0], w[1], w[2], w[3]);
            }
        } else if (live) {
            const size_t slot = (2 * (size_t)blockIdx.x + (k0 == 0)) * M + tid;
#pragma unroll
            for (int c = 0; c < D; c += 4)
                *reinterpret_cast<uint4 *>(p.part_o + slot * D + c) = make_uint4(o[c], o[c + 1], o[c + 2], o[c + 3]);
            *reinterpret_cast<float2 *>(p.part_ml + slot * 2) = make_float2(top, l);
        }
    }
    // After a wait that gave up, products may still run: they read operands that are in shared memory, so they end.
    cp_async_wait<0>();
    all_ok = __syncthreads_and(ok && all_ok);
    if (!all_ok && tid == 0) {
        umma_commit(&bar_end);
        mbar_wait_for(&bar_end, 0, 8 * kWaitNs, p.status);
    }
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 0) asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(s_tmem), "r"(tmem_columns<D>()) : "memory");
}

template <int D>
cudaError_t launch(const AttnParams &p, int *grid, long most, cudaStream_t st) {
    // the shared-memory limit is a per-device attribute: raise it once on every device used
    static bool done[64] = {};
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev >= 64 || !done[dev]) {
        e = cudaFuncSetAttribute(attn_tc_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)tc_smem<D>(kMaxBatch));
        if (e != cudaSuccess) return e;
        if (dev < 64) done[dev] = true;
    }
    const int slots = tc_ctas<D>() * sm_count();
    *grid = most < slots ? (int)most : slots;
    return launch_kernel(attn_tc_kernel<D>, dim3(*grid), dim3(kAttnThreads), tc_smem<D>(p.B), st, p);
}

}  // namespace

cudaError_t launch_attn_tc(int D, const AttnParams &p, int *grid, long most, cudaStream_t st) {
    return D == 128 ? launch<128>(p, grid, most, st) : launch<64>(p, grid, most, st);
}

}  // namespace hla
