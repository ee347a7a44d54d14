// The whole mixture-of-experts layer for up to 64 tokens over 8-bit weights with block scales.
//
//   logits = x W_r^T, the k largest, w = sigmoid / sum; xq = e4m3 blocks of x;
//   h = SiLU(xq Wg^T) * (xq Wu^T) per chosen and shared expert, hq = e4m3 blocks of h;  y = residual + sum w (hq Wd^T).
//
// Bound by HBM: the weights of the distinct chosen experts, 3 Hd I bytes each, are read once; everything else is small.
//
//  1. `moe_prep_kernel`: the router's logits (mma.sync, clusters of four CTAs cut K) beside the conversion of x, and the last
//     kernel's counters set to zero.
//  2. `moe_choose_kernel`, more than 8 tokens only: the choice, a warp per token.  Fewer are chosen by every CTA of the next kernel for
//     itself, a launch less.  The whole layer without and with this kernel, 256 experts, top 8: 64 tokens of hidden 1024 124, 113 us;
//     of hidden 512 16 tokens 33.3, 31.4, 12 tokens 29.0, 28.5, 6 tokens 23.7, 24.0; one token of hidden 256, 16 experts 10.7, 12.0.
//  3. `moe_fp8_kernel`, one CTA per SM, a cooperative launch: every CTA derives the list of active experts from the choice, and
//     streams an equal, contiguous share of all gate and up tiles, then, after one grid barrier, of all down tiles (small
//     layers: some of the CTAs).  A tile is 128 weight rows x 128 of K.  The weight rows lie on the lanes of tcgen05 and all tokens of the
//     batch on the columns (16, 32 or 64): tokens that did not choose the expert cost nothing that the memory does not hide, and
//     nothing has to be gathered.  Products of one block of K are read back and added, scaled, to sums in registers.
//     Items cut between CTAs leave their parts in the workspace, and the CTA that comes last adds them in order: no CTA waits
//     for a part, and the order does not depend on who comes last.  Down tiles run through all experts of one block of output
//     rows, so that the mixture over experts is one sum in registers.  The copying thread runs ahead across the
//     barrier: the first down tiles, which depend on no other CTA, are on their way before it.
//
// Every wait is bounded (see tc_gemm.cu): a wait that gives up sets the device status word, and what follows still passes
// every block barrier and the grid barrier's count, without waiting.
#include "fp8.cuh"

namespace hla {
namespace {

constexpr int kMaxExperts = 1024;   // routed and shared together
constexpr int kMaxTopK = 16;
constexpr int kMaxTokens = 64;
constexpr int kChooseInside = 8;    // the most tokens that moe_fp8_kernel chooses for itself

// ----------------------------------------------------------------------------- workspace

struct MoeSpace {
    size_t logits, idx, w, xq, xs, hq, hs, part, count, total;
};

inline int tokens_padded(int M) { return M <= 16 ? 16 : M <= 32 ? 32 : 64; }
inline int moe_units_most(const hla_moe_fp8 *L, int M) {
    const long r = (long)M * L->top_k;
    return (int)(r < L->n_experts ? r : L->n_experts) + L->n_shared;
}

MoeSpace moe_space(const hla_moe_fp8 *L, int M) {
    const size_t NT = tokens_padded(M), U = moe_units_most(L, M), G = sm_count();
    MoeSpace s;
    size_t at = 0;
    auto take = [&](size_t bytes) {
        const size_t r = at;
        at += round_up(bytes, 256);
        return r;
    };
    s.logits = take((size_t)M * L->n_experts * 4);
    s.idx = take(M > kChooseInside ? (size_t)M * L->top_k * 4 : 0);
    s.w = take(M > kChooseInside ? (size_t)M * L->top_k * 4 : 0);
    s.xq = take((size_t)M * L->hidden);
    s.xs = take(NT * (L->hidden / kFp8Block) * 4);
    s.hq = take(U * NT * L->inter);
    s.hs = take(U * NT * (L->inter / kFp8Block) * 4);
    s.part = take(G * 2 * 2 * NT * 128 * 4);
    s.count = take((2 * G + 1) * 4);
    s.total = at;
    return s;
}

// ----------------------------------------------------------------------------- logits and conversion

constexpr int kPrepThreads = 256;
constexpr int kPrepCluster = 4;
constexpr int kPrepExperts = 8;     // experts per cluster: the columns of one mma.sync
// K steps of 32 whose weights are loaded at once.  A warp has hidden / 1024 steps, so that 7168 takes one round trip; it matters
// little: 64 tokens, inner 256, 256 + 1 experts of hidden 7168 with 4, 7, 8, 12 at once 247.6, 246.1, 247.0, 247.3 us; hidden 2048, 64 + 1
// experts 49.4, 49.9, 49.9, 51.2; hidden 3200, 8 + 1 experts 44.3, 44.5, 44.9, 45.5.
constexpr int kPrepAhead = 7;

struct PrepParams {
    int M, Hd, E, NT, router_clusters, counters;
    const uint16_t *x, *Wr;
    float *logits;
    uint8_t *xq;
    float *xs;
    int *count;
};

__global__ void __launch_bounds__(kPrepThreads) __cluster_dims__(kPrepCluster, 1, 1) moe_prep_kernel(const PrepParams p) {
    __shared__ float s_part[kPrepThreads / 32][kMaxTokens][kPrepExperts];
    __shared__ float s_sum[kMaxTokens][kPrepExperts];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int cluster = blockIdx.x / kPrepCluster, rank = blockIdx.x % kPrepCluster;
    if (cluster >= p.router_clusters) {  // conversion of x: 8 lanes a block of 128
        pdl_wait_trigger();
        const int KB = p.Hd / kFp8Block;
        const long b = ((long)(cluster - p.router_clusters) * kPrepCluster + rank) * (kPrepThreads / 8) + (tid >> 3);
        if (cluster == p.router_clusters && rank == 0)
            for (int i = tid; i < p.counters; i += kPrepThreads) p.count[i] = 0;
        const bool live = b < (long)p.M * KB;
        const int m = live ? (int)(b / KB) : 0, kb = live ? (int)(b - (long)m * KB) : 0;
        const size_t at = (size_t)m * p.Hd + kb * kFp8Block + (tid & 7) * 16;
        const uint4 a = ld_act_v4(p.x + at), c = ld_act_v4(p.x + at + 8);
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, c.x, c.y, c.z, c.w};
        float top = 0.f;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = max_magnitude(top, max_magnitude(bf16_lo(w[i]), bf16_hi(w[i])));
#pragma unroll
        for (int s = 4; s; s >>= 1) top = max_magnitude(top, __shfl_xor_sync(~0u, top, s));
        const float sc = fp8_scale_of(top), inv = fp8_inverse(sc);
        if (live) {
            uint32_t r[4];
#pragma unroll
            for (int i = 0; i < 4; ++i)
                r[i] = e4m3x4(bf16_lo(w[2 * i]) * inv, bf16_hi(w[2 * i]) * inv, bf16_lo(w[2 * i + 1]) * inv, bf16_hi(w[2 * i + 1]) * inv);
            *reinterpret_cast<uint4 *>(p.xq + at) = make_uint4(r[0], r[1], r[2], r[3]);
            if ((tid & 7) == 0) p.xs[(size_t)kb * p.NT + m] = sc;
        }
        return;
    }
    // Logits of 8 experts: the cluster's warps cut K into shares of whole steps of 32.  Lane (g, t) holds 8 values of K for
    // expert g and for tokens g and g + 8; the same permutation of K on both sides leaves the product as it is.
    const int g = lane >> 2, t = lane & 3, e0 = cluster * kPrepExperts;
    const int share = rank * (kPrepThreads / 32) + warp, shares = kPrepCluster * (kPrepThreads / 32), steps = p.Hd / 32;
    const int s0 = (int)((long)steps * share / shares), s1 = (int)((long)steps * (share + 1) / shares);
    const int e = e0 + g < p.E ? e0 + g : p.E - 1;
    const uint16_t *const wr = p.Wr + (size_t)e * p.Hd + t * 8;
    uint4 w[kPrepAhead];
#pragma unroll
    for (int i = 0; i < kPrepAhead; ++i)
        if (s0 + i < s1) w[i] = ld_weight_v4(wr + (s0 + i) * 32);
    pdl_wait_trigger();
    float acc[kMaxTokens / 16][4] = {};
    for (int s = s0; s < s1; s += kPrepAhead) {
        if (s > s0) {
#pragma unroll
            for (int i = 0; i < kPrepAhead; ++i)
                if (s + i < s1) w[i] = ld_weight_v4(wr + (s + i) * 32);
        }
#pragma unroll
        for (int mt = 0; mt < kMaxTokens / 16; ++mt) {
            if (mt * 16 >= p.M) break;
            const int ma = mt * 16 + g, mb = ma + 8;
            const uint16_t *const xa = p.x + (size_t)(ma < p.M ? ma : 0) * p.Hd + t * 8, *const xb = p.x + (size_t)(mb < p.M ? mb : 0) * p.Hd + t * 8;
            uint4 a[kPrepAhead], b[kPrepAhead];
#pragma unroll
            for (int i = 0; i < kPrepAhead; ++i)
                if (s + i < s1) {
                    a[i] = ld_act_v4(xa + (s + i) * 32);
                    b[i] = ld_act_v4(xb + (s + i) * 32);
                }
#pragma unroll
            for (int i = 0; i < kPrepAhead; ++i)
                if (s + i < s1) {
                    mma_bf16_16816(acc[mt], a[i].x, b[i].x, a[i].y, b[i].y, w[i].x, w[i].y);
                    mma_bf16_16816(acc[mt], a[i].z, b[i].z, a[i].w, b[i].w, w[i].z, w[i].w);
                }
        }
    }
#pragma unroll
    for (int mt = 0; mt < kMaxTokens / 16; ++mt) {
        if (mt * 16 >= p.M) break;
        *reinterpret_cast<float2 *>(&s_part[warp][mt * 16 + g][2 * t]) = make_float2(acc[mt][0], acc[mt][1]);
        *reinterpret_cast<float2 *>(&s_part[warp][mt * 16 + g + 8][2 * t]) = make_float2(acc[mt][2], acc[mt][3]);
    }
    __syncthreads();
    for (int i = tid; i < p.M * kPrepExperts; i += kPrepThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kPrepThreads / 32; ++k) v += (&s_part[k][0][0])[i];
        (&s_sum[0][0])[i] = v;
    }
    cluster_sync();
    for (int i = rank * kPrepThreads + tid; i < p.M * kPrepExperts; i += kPrepCluster * kPrepThreads) {
        float v = 0.f;
#pragma unroll
        for (int k = 0; k < kPrepCluster; ++k) v += peer_float(&s_sum[0][0] + i, k);
        const int m = i / kPrepExperts, n = e0 + i % kPrepExperts;
        if (n < p.E) p.logits[(size_t)m * p.E + n] = v;
    }
    cluster_sync();
}

// ----------------------------------------------------------------------------- the choice

__device__ __forceinline__ uint32_t ordered(float v) {  // larger floats have larger keys; none is 0
    const uint32_t b = __float_as_uint(v), k = b & 0x80000000u ? ~b : b | 0x80000000u;
    return k ? k : 1u;
}
__device__ __forceinline__ float unordered(uint32_t k) { return __uint_as_float(k & 0x80000000u ? k & 0x7FFFFFFFu : ~k); }

// The k largest of a token's E <= 32 PER logits by one warp, ties to the lower index: lane j gets the jth index and its logit.
template <int PER>
__device__ __forceinline__ void choose(const float *logits, int E, int k, int lane, int *idx, float *logit) {
    uint32_t key[PER], top = 0;
    int at = 0;  // the largest of this lane's own, the first of equal ones
#pragma unroll
    for (int i = 0; i < PER; ++i) {
        const int e = i * 32 + lane;
        const float v = __ldcg(logits + (e < E ? e : E - 1));
        key[i] = e < E ? ordered(v) : 0u;
    }
#pragma unroll
    for (int i = 0; i < PER; ++i)
        if (key[i] > top) top = key[i], at = i;
#pragma unroll 1
    for (int j = 0; j < k; ++j) {
        const uint32_t best = __reduce_max_sync(~0u, top);
        const uint32_t e = __reduce_min_sync(~0u, top == best ? (uint32_t)(at * 32 + lane) : ~0u);
        if (lane == j) {
            *idx = (int)e;
            *logit = unordered(best);
        }
        const bool mine = (e & 31) == lane;
        top = 0;
#pragma unroll
        for (int i = 0; i < PER; ++i) {
            key[i] &= mine && i == (int)(e >> 5) ? 0u : ~0u;
            if (key[i] > top) top = key[i], at = i;
        }
    }
}

// Lane j's jth choice of a token and its weight in the mixture: its sigmoid over the sum of the k.  Relative to the largest one's
// exponential where all logits are negative: their scores may all be below fp32.
__device__ __forceinline__ void choose_token(const float *logits, int E, int k, int lane, int *idx, float *w) {
    float logit = 0.f;
    *idx = 0;
    if (E <= 256) choose<8>(logits, E, k, lane, idx, &logit);
    else choose<32>(logits, E, k, lane, idx, &logit);
    const float top = fminf(__shfl_sync(~0u, logit, 0), 0.f);
    const float score = logit >= 0.f ? 1.f / (1.f + expf(-logit)) : expf(logit - top) / (1.f + expf(logit));
    float sum = 0.f;
    for (int j = 0; j < k; ++j) sum += __shfl_sync(~0u, score, j);
    *w = score / sum;
}

// The choice of many tokens, a warp each.
struct ChooseParams {
    int E, k;
    const float *logits;
    int32_t *idx, *topk_idx;
    float *w, *topk_w;
};
__global__ void __launch_bounds__(32) moe_choose_kernel(const ChooseParams p) {
    pdl_wait_trigger();
    const int lane = threadIdx.x, m = blockIdx.x;
    int idx;
    float w;
    choose_token(p.logits + (size_t)m * p.E, p.E, p.k, lane, &idx, &w);
    if (lane < p.k) {
        const int at = m * p.k + lane;
        p.idx[at] = idx;
        p.w[at] = w;
        if (p.topk_idx) p.topk_idx[at] = idx;
        if (p.topk_w) p.topk_w[at] = w;
    }
}

// ----------------------------------------------------------------------------- the experts

constexpr int kMoeThreads = 384;    // copies, products, scales, a warp of the choice only, two groups of four warps of sums
constexpr int kSumThreads = 256;
constexpr int kSumWarp0 = 4;
constexpr int kSparse = 0x8000;     // of a unit's entry: few tokens chose it

struct MoeMaps {
    CUtensorMap x, h, hfew, gate, up, down, sgate, sup, sdown;
};

struct MoeParams {
    int M, Hd, I, E, k, n_shared;
    const float *logits, *xs;
    const float *gate_s, *up_s, *down_s, *sgate_s, *sup_s, *sdown_s;
    const uint16_t *residual;
    uint16_t *y;
    int32_t *topk_idx;
    float *topk_w;
    const int32_t *idx;        // the choice [M, k] of more than kChooseInside tokens, or NULL
    const float *w;
    uint8_t *hq;
    float *hs, *part;
    int *count;                // [G] parts of cut gate/up items, [G] parts of cut output blocks, [1] grid barrier
    int *status;
    int force_timeout;
};

template <int NT>
struct Moe {
    static constexpr int kSlots = NT == 16 ? 10 : NT == 32 ? 8 : 7;
    static constexpr int kAcc = 4;                                    // accumulators of 2 NT columns
    static constexpr uint32_t kTile = 128 * 128, kTokens = NT * 128, kScales = NT * 4;
    static constexpr uint32_t kColumns = kAcc * 2 * NT;
    // 64 tokens: an expert that at most 8 tokens of each half of the batch chose is sparse: its sums and its rows of h
    // are the 16 positions of those tokens, not the 64 tokens
    static constexpr bool kLists = NT == 64;
    static constexpr int kSums = NT == 16 ? 16 : 32;                  // of a thread, for gate and for up
    static constexpr size_t kExchange = (NT == 16 ? 16 : 32) * 1024;  // where the groups' sums meet; y's sums of 64 tokens
    static constexpr size_t kTables = NT * kMaxTopK * 8 + kMaxExperts * 2 + kMaxExperts * 8;
    static constexpr size_t kSmem = 1024 + kSlots * (kTile + kTokens + kScales) + kAcc * 2 * NT * 4 + kExchange + (2 * kSlots + 2 * kAcc + 2) * 8 + 16 + kTables;
    static_assert((2 * kSlots + 2 * kAcc + 2) * 8 % 16 == 0, "the tables are aligned");
    static_assert(kSmem <= 227 * 1024, "one CTA to an SM");
};

// The shares of one phase: T steps of `step` blocks of K over `ctas` CTAs, as equal as whole steps can be.  All in 32 bits: 2^24
// blocks are 256 GB of weights.
struct Share {
    uint32_t T, ctas, step;
    __device__ __forceinline__ void set(uint32_t blocks, uint32_t per_step, uint32_t G) {
        step = per_step;
        T = blocks / per_step;
        ctas = T < G ? T : G;
    }
    __device__ __forceinline__ int start(uint32_t c) const { return c < ctas ? (int)(step * (T * c / ctas)) : (int)(step * T); }
    __device__ __forceinline__ int owner(uint32_t t) const { return (int)(((t + 1) * ctas - 1) / T); }  // of block t, at step 1
};

// Position in the order of the gate/up items: block of 128 of the inner width, unit, block of K.  The units run inside, so that
// those that many tokens chose, whose sums cost more, are spread over the CTAs.
struct GateAt {
    int u, ib, kb;
    __device__ __forceinline__ void set(uint32_t t, uint32_t U, uint32_t KB) {
        const uint32_t item = t / KB;
        kb = (int)(t - item * KB);
        ib = (int)(item / U);
        u = (int)(item - ib * U);
    }
    __device__ __forceinline__ void next(int U, int KB) {
        if (++kb == KB) {
            kb = 0;
            if (++u == U) u = 0, ++ib;
        }
    }
};
// Position in the order of the down items: block of output rows, unit, block of K.
struct DownAt {
    int rb, u, kb;
    __device__ __forceinline__ void set(uint32_t t, uint32_t U, uint32_t KB) {
        rb = (int)(t / (U * KB));
        const uint32_t r = t - rb * U * KB;
        u = (int)(r / KB);
        kb = (int)(r - u * KB);
    }
    __device__ __forceinline__ void next(int U, int KB) {
        if (++kb == KB) {
            kb = 0;
            if (++u == U) u = 0, ++rb;
        }
    }
};
// A place in a ring and how often the ring has gone round.
template <int N>
struct Ring {
    int s = 0, turn = 0;
    __device__ __forceinline__ void next() {
        if (++s == N) s = 0, ++turn;
    }
    __device__ __forceinline__ uint32_t filled() const { return turn & 1; }            // parity of this use's completion
    __device__ __forceinline__ uint32_t freed() const { return (turn - 1) & 1; }       // and of the one before, from the second use on
};

// Scales of the down products: +0 stands for a token that did not choose the expert, and for nothing else.  A chosen one's that
// is 0 (weights' scale 0, underflow) is -0: its products are added, so that NaN weights reach it all the same.
__device__ __forceinline__ float chosen(float scale) { return scale == 0.f ? -0.f : scale; }
__device__ __forceinline__ bool is_chosen(float scale) { return __float_as_uint(scale) != 0u; }

__device__ __forceinline__ int load_acquire(const int *p) {
    int v;
    asm volatile("ld.acquire.gpu.global.b32 %0, [%1];" : "=r"(v) : "l"(p) : "memory");
    return v;
}
// The bounded wait at the grid barrier.
__device__ __forceinline__ bool wait_grid(const int *barrier, int ctas, int *status) {
    uint64_t began = 0;
    for (uint32_t i = 0; load_acquire(barrier) < ctas; ++i)
        if ((i & 63) == 63) {
            const uint64_t now = global_ns();
            if (!began) began = now;
            else if (now - began > kFp8WaitNs) {
                atomicExch(status, HLA_ERR_DEVICE_TIMEOUT);
                return false;
            }
        }
    return true;
}
__device__ __forceinline__ int add_acq_rel(int *p, int v) {
    int old;
    asm volatile("atom.add.acq_rel.gpu.global.s32 %0, [%1], %2;" : "=r"(old) : "l"(p), "r"(v) : "memory");
    return old;
}
__device__ __forceinline__ void fence_async() { asm volatile("fence.proxy.async;" ::: "memory"); }
__device__ __forceinline__ void mbar_arrive_n(uint64_t *bar, uint32_t n) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)), "r"(n) : "memory");
}
__device__ __forceinline__ void tmem_ld1(uint32_t taddr, uint32_t &v) {
    asm volatile("tcgen05.ld.sync.aligned.32x32b.x1.b32 {%0}, [%1];" : "=r"(v) : "r"(taddr));
}

// Adds an item's parts in order: CTA c0 left its in slot `second`, the CTAs up to c1 in their first slot.  Four are loaded at once.
__device__ __forceinline__ void add_parts(const float *at, size_t to_up, size_t part, int c0, int c1, bool second, float4 *g, float4 *u) {
    for (int k = c0; k <= c1; k += 4) {
        float4 a[4], b[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            // the last part again behind it: loads under conditions wait for one another (64 tokens, 256 experts: 1607 us, 1592)
            const int from = k + i <= c1 ? k + i : c1;
            const float *const q = at + ((size_t)from * 2 + (from == c0 && second)) * part;
            a[i] = __ldcg(reinterpret_cast<const float4 *>(q));
            b[i] = __ldcg(reinterpret_cast<const float4 *>(q + to_up));
        }
#pragma unroll
        for (int i = 0; i < 4; ++i)
            if (k + i <= c1) {
                g->x += a[i].x, g->y += a[i].y, g->z += a[i].z, g->w += a[i].w;
                u->x += b[i].x, u->y += b[i].y, u->z += b[i].z, u->w += b[i].w;
            }
    }
}

// The most CTAs that share an item of `blocks` blocks.  n of them stream it in about 600 blocks / n cycles, and the last adds n
// parts at 400 + 8 M cycles each: least at the root of the quotient.  It counts for layers of few items.  With all CTAs, when this
// came in: 64 tokens, hidden 256, inner 1024, 64 + 1 experts 120 us, 81 so; one token, hidden 256, inner 128, 16 experts 13.9,
// 12.1.  Now, and with 250 + 5 M and 600 + 8 M: 61 tokens, hidden 3200, inner 512, 8 + 1 experts 44.3, 49.9, 45.1 us; 23 tokens,
// hidden 384, inner 768, 8 + 1 experts 20.9, 24.0, 21.5; the one token 12.2, 14.3, 12.3.
__device__ __forceinline__ uint32_t sharers(int blocks, int M) {
    const float p = sqrtf(600.f * blocks / (400.f + 8.f * M));
    return p < 1.f ? 1u : p > 1024.f ? 1024u : (uint32_t)p;
}

template <int NT>
__global__ void __launch_bounds__(kMoeThreads, 1) moe_fp8_kernel(const __grid_constant__ MoeMaps maps, const MoeParams p) {
    using F = Moe<NT>;
    constexpr int NS = F::kSlots, NB = F::kAcc, S = F::kSums, H = NT / 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const sA = smem, *const sB = smem + NS * F::kTile;
    float *const sX = reinterpret_cast<float *>(sB + NS * F::kTokens);  // [NS][NT]: the tokens' scales
    float *const sS = sX + NS * NT;  // [NB][2 NT]: what each accumulator's columns are multiplied by
    float *const s_sums = sS + NB * 2 * NT;
    uint64_t *const full = reinterpret_cast<uint64_t *>(s_sums + F::kExchange / 4);
    uint64_t *const empty = full + NS, *const acc_full = empty + NS, *const acc_empty = acc_full + NB, *const done = acc_empty + NB;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(done + 2);  // 16-byte aligned, as the tables behind it
    int *const s_int = reinterpret_cast<int *>(tmem_slot + 1);           // active experts, products issued, last part?
    uint2 *const s_mask = reinterpret_cast<uint2 *>(tmem_slot + 4);      // tokens that chose each expert, by half of the batch
    int *const s_idx = reinterpret_cast<int *>(s_mask + kMaxExperts);    // [M][k]
    float *const s_w = reinterpret_cast<float *>(s_idx + NT * kMaxTopK);
    uint16_t *const s_unit = reinterpret_cast<uint16_t *>(s_w + NT * kMaxTopK);  // routed units' experts

    if (p.force_timeout) {
        forced_timeout(done, p.status);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 2);  // the products, and the warp that reads the scales
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&acc_full[b], 2);  // the products and their scales
            mbar_init(&acc_empty[b], kSumThreads / 32);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_async();
    }
    if (warp == 3 && lane < 9) asm volatile("prefetch.tensormap [%0];" ::"l"(reinterpret_cast<uint64_t>(&maps.x + lane)) : "memory");
    if (warp == 1) tmem_alloc(tmem_slot, F::kColumns);
    for (int i = tid; i < p.E; i += kMoeThreads) s_mask[i] = make_uint2(0u, 0u);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_trigger();

    // ---- the choice: of few tokens by every CTA for itself, and the first one writes it out
    const auto record = [&](int m, int lane, int idx, float w) {
        s_idx[m * p.k + lane] = idx;
        s_w[m * p.k + lane] = w;
        atomicOr(m < 32 ? &s_mask[idx].x : &s_mask[idx].y, 1u << (m & 31));
    };
    if (NT == 16 && !p.idx) {
#pragma unroll 1
        for (int m = warp; m < p.M; m += kMoeThreads / 32) {
            int idx;
            float w;
            choose_token(p.logits + (size_t)m * p.E, p.E, p.k, lane, &idx, &w);
            if (lane < p.k) {
                record(m, lane, idx, w);
                if (blockIdx.x == 0) {
                    if (p.topk_idx) p.topk_idx[m * p.k + lane] = idx;
                    if (p.topk_w) p.topk_w[m * p.k + lane] = w;
                }
            }
        }
    } else {
        for (int i = tid; i < p.M * p.k; i += kMoeThreads) record(i / p.k, i % p.k, __ldcg(p.idx + i), __ldcg(p.w + i));
    }
    __syncthreads();
    // units: the shared experts, then the active ones in order
    if (warp == 0) {
        int n = 0;
        for (int e0 = 0; e0 < p.E; e0 += 32) {
            const uint2 mask = e0 + lane < p.E ? s_mask[e0 + lane] : make_uint2(0u, 0u);
            const bool any = (mask.x | mask.y) != 0;
            const uint32_t active = __ballot_sync(~0u, any);
            const bool sparse = F::kLists && __popc(mask.x) <= 8 && __popc(mask.y) <= 8;
            if (any) s_unit[n + __popc(active & ((1u << lane) - 1))] = (uint16_t)(e0 + lane | (sparse ? kSparse : 0));
            n += __popc(active);
        }
        if (lane == 0) s_int[0] = n;
    }
    __syncthreads();
    const int U = s_int[0] + p.n_shared, G = gridDim.x, c = blockIdx.x;
    const int nI = p.I / 128, nR = p.Hd / 128, KB1 = p.Hd / kFp8Block, KB2 = p.I / kFp8Block;
    Share s1, s2;
    // Gate/up items for three quarters of the CTAs or more, but no more than one each, stay whole: what is idle costs nothing while the
    // rest fills the memory, and no parts are joined.  One token of 8 + 1 experts, whole and cut: 144 items on 152 CTAs 75.9, 78.4 us
    // of hidden 7168 and 20.5, 23.4 of 512; 117 items 65.4, 67.3 and 19.9, 22.3.  The border is a careful one: 108 items gain so, too
    // (62.0, 63.6 and 19.5, 22.3), 81 of hidden 7168 lose (54.3, 52.3).
    const int items = U * nI;
    s1.set(items * KB1, items <= G && items * 4 >= G * 3 ? KB1 : 1, min((uint32_t)G, items * sharers(KB1, p.M)));
    s2.set(nR * U * KB2, 1, min((uint32_t)G, nR * sharers(U * KB2, p.M)));
    const int a0 = s1.start(c), a1 = s1.start(c + 1), b0 = s2.start(c), b1 = s2.start(c + 1);
    int *const barrier = p.count + 2 * G;
    const auto shared_unit = [&](int u) { return u < p.n_shared; };
    const auto expert_of = [&](int u) { return u < p.n_shared ? u : (int)s_unit[u - p.n_shared] & (kSparse - 1); };
    const auto sparse_unit = [&](int u) { return F::kLists && u >= p.n_shared && (s_unit[u - p.n_shared] & kSparse) != 0; };
    int issued = 0;  // slots filled, up to multiples of 2 NS

    if (warp == 0 && lane == 0) {
        // ---- copies
        bool ok = true;
        Ring<NS> r;
        GateAt at;
        at.set(a0, U, KB1);
        for (int t = a0; t < a1 && ok; ++t, at.next(U, KB1)) {
            const bool sh = shared_unit(at.u);
            const int row = expert_of(at.u) * p.I + at.ib * 128, col = at.kb * kFp8Block;
#pragma unroll
            for (int half = 0; half < 2; ++half) {
                if (r.turn > 0 && !(ok = fp8_wait(&empty[r.s], r.freed(), p.status))) break;
                mbar_expect_tx(&full[r.s], F::kTile + (half ? 0 : F::kTokens + F::kScales));
                tma_tile(sA + r.s * F::kTile, half ? (sh ? &maps.sup : &maps.up) : (sh ? &maps.sgate : &maps.gate), col, row, &full[r.s]);
                if (!half) {
                    tma_tile(sB + r.s * F::kTokens, &maps.x, col, 0, &full[r.s]);
                    bulk_g2s(sX + r.s * NT, p.xs + (size_t)at.kb * NT, F::kScales, &full[r.s]);
                }
                r.next();
            }
        }
        // the first down tiles go out before the grid barrier, their tokens after it
        const int n2 = b1 - b0;
        const int pre = n2 < NS ? n2 : NS;
        DownAt w, h;
        w.set(b0, U, KB2);
        h = w;
        const auto weights = [&](int s) {
            mbar_expect_tx(&full[s], F::kTile + F::kScales + (sparse_unit(w.u) ? 16 * 128 : F::kTokens));
            tma_tile(sA + s * F::kTile, shared_unit(w.u) ? &maps.sdown : &maps.down, w.kb * kFp8Block, expert_of(w.u) * p.Hd + w.rb * 128, &full[s]);
            w.next(U, KB2);
        };
        const auto tokens = [&](int s) {
            tma_tile(sB + s * F::kTokens, sparse_unit(h.u) ? &maps.hfew : &maps.h, h.kb * kFp8Block, h.u * NT, &full[s]);
            bulk_g2s(sX + s * NT, p.hs + ((size_t)h.u * KB2 + h.kb) * NT, F::kScales, &full[s]);
            h.next(U, KB2);
        };
        const Ring<NS> first = r;
        int sent = 0;
        for (; sent < pre && ok; ++sent) {
            if (r.turn > 0 && !(ok = fp8_wait(&empty[r.s], r.freed(), p.status))) break;
            weights(r.s);
            r.next();
        }
        if (n2 > 0 && ok) {
            ok = wait_grid(barrier, G, p.status);
            fence_async();
        }
        Ring<NS> q = first;
        for (int i = 0; i < sent; ++i, q.next()) tokens(q.s);  // after a barrier that gave up, too: the fills complete
        for (int t = sent; t < n2 && ok; ++t) {
            if (r.turn > 0 && !(ok = fp8_wait(&empty[r.s], r.freed(), p.status))) break;
            weights(r.s);
            tokens(r.s);
            r.next();
        }
        issued = r.turn > 1 ? (r.turn & 1 ? NS : 2 * NS) + r.s : r.turn * NS + r.s;
    } else if (warp == 1) {
        // ---- products
        bool ok = true;
        Ring<NS> r;
        Ring<NB> b;
        for (int t = a0; t < a1; ++t) {
            const int s = r.s;
            ok = (b.turn == 0 || fp8_wait(&acc_empty[b.s], b.freed(), p.status)) && fp8_wait(&full[s], r.filled(), p.status);
            r.next();
            ok = __all_sync(~0u, ok && fp8_wait(&full[r.s], r.filled(), p.status));
            if (!ok) break;
            tc_fence_after();
            umma_block(tmem + b.s * 2 * NT, smem_u32(sA + s * F::kTile), smem_u32(sB + s * F::kTokens), idesc_e4m3(128, NT));
            umma_block(tmem + b.s * 2 * NT + NT, smem_u32(sA + r.s * F::kTile), smem_u32(sB + s * F::kTokens), idesc_e4m3(128, NT));
            umma_commit_elected(&empty[s]);
            umma_commit_elected(&empty[r.s]);
            umma_commit_elected(&acc_full[b.s]);
            r.next();
            b.next();
        }
        DownAt at;
        at.set(b0, U, KB2);
        for (int t = b0; t < b1 && ok; ++t, at.next(U, KB2)) {
            ok = __all_sync(~0u, (b.turn == 0 || fp8_wait(&acc_empty[b.s], b.freed(), p.status)) && fp8_wait(&full[r.s], r.filled(), p.status));
            if (!ok) break;
            tc_fence_after();
            umma_block(tmem + b.s * 2 * NT, smem_u32(sA + r.s * F::kTile), smem_u32(sB + r.s * F::kTokens),
                       sparse_unit(at.u) ? idesc_e4m3(128, 16) : idesc_e4m3(128, NT));
            umma_commit_elected(&empty[r.s]);
            umma_commit_elected(&acc_full[b.s]);
            r.next();
            b.next();
        }
        if (lane == 0) s_int[1] = ok;
        umma_commit_elected(done);
        if (!fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else if (warp == 2) {
        // ---- scales: token scale (copied with the tiles) times weight scale of every column of an accumulator.  Lane i loads the
        // weight scales of the ith of 32 blocks, 32 blocks ahead: under full memory traffic a load takes microseconds.
        bool ok = true;
        Ring<NS> r;
        Ring<NB> b;
        float sg = 0.f, su = 0.f, next_g = 0.f, next_u = 0.f;
        const auto gate_scales = [&](int t) {
            if (t + lane >= a1) return;
            GateAt at;
            at.set(t + lane, U, KB1);
            const size_t q = ((size_t)expert_of(at.u) * nI + at.ib) * KB1 + at.kb;
            next_g = __ldg((shared_unit(at.u) ? p.sgate_s : p.gate_s) + q);
            next_u = __ldg((shared_unit(at.u) ? p.sup_s : p.up_s) + q);
        };
        const auto down_scales = [&](int t) {
            if (t + lane >= b1) return;
            DownAt at;
            at.set(t + lane, U, KB2);
            next_g = __ldg((shared_unit(at.u) ? p.sdown_s : p.down_s) + ((size_t)expert_of(at.u) * nR + at.rb) * KB2 + at.kb);
        };
        const auto ready = [&]() {
            ok = __all_sync(~0u, (b.turn == 0 || fp8_wait(&acc_empty[b.s], b.freed(), p.status)) && fp8_wait(&full[r.s], r.filled(), p.status));
        };
        GateAt at;
        at.set(a0, U, KB1);
        gate_scales(a0);
        int from = -1;  // the token of lanes 0..15 in a sparse unit
        for (int t = a0; t < a1 && ok; ++t, at.next(U, KB1)) {
            const int i = (t - a0) & 31;
            if (i == 0) {
                sg = next_g;
                su = next_u;
                gate_scales(t + 32);
            }
            const bool sparse = sparse_unit(at.u);
            if (sparse && (at.kb == 0 || t == a0)) {
                const uint2 mask = s_mask[expert_of(at.u)];
                uint32_t left = lane < 8 ? mask.x : lane < 16 ? mask.y : 0u;
                for (int j = 0; j < (lane & 7); ++j) left &= left - 1;
                from = left ? (lane >> 3) * 32 + __ffs(left) - 1 : -1;
            }
            ready();
            if (!ok) break;
            const float g = __shfl_sync(~0u, sg, i), u = __shfl_sync(~0u, su, i);
            const float *const x = sX + r.s * NT;
            float *const sc = sS + b.s * 2 * NT;
#pragma unroll
            for (int m = lane; m < NT; m += 32) {
                if (sparse && m >= 16) break;
                const float v = !sparse ? x[m] : from >= 0 ? x[from] : 0.f;
                sc[m] = v * g;
                sc[NT + m] = v * u;
            }
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&acc_full[b.s]);
                mbar_arrive(&empty[r.s]);
            }
            r.next();
            // The up tile's slot is given back once this use of it has begun: earlier, the arrival could count for the use before,
            // whose products may still be reading (with seven slots it was a gate tile's).
            ok = __all_sync(~0u, fp8_wait(&full[r.s], r.filled(), p.status));
            if (ok && lane == 0) mbar_arrive(&empty[r.s]);
            r.next();
            b.next();
        }
        if (ok) down_scales(b0);
        for (int t = b0; t < b1 && ok; ++t) {
            const int i = (t - b0) & 31;
            if (i == 0) {
                sg = next_g;
                down_scales(t + 32);
            }
            ready();
            if (!ok) break;
            const float g = __shfl_sync(~0u, sg, i);
            const float *const x = sX + r.s * NT;
            float *const sc = sS + b.s * 2 * NT;
#pragma unroll
            for (int m = lane; m < NT; m += 32) sc[m] = is_chosen(x[m]) ? chosen(x[m] * g) : 0.f;  // whatever the weights' scale (NaN, infinity)
            __syncwarp();
            if (lane == 0) {
                mbar_arrive(&acc_full[b.s]);
                mbar_arrive(&empty[r.s]);
            }
            r.next();
            b.next();
        }
    } else if (warp >= kSumWarp0) {
        // ---- sums, each thread of one weight row.  Up to 32 tokens, and for the gate and up products of a sparse unit, the two
        // groups of four warps take every other block of K and all tokens (or positions), and their sums meet in shared
        // memory where a segment ends; otherwise each takes its half of the tokens of every block.
        const int grp = warp >= kSumWarp0 + 4, q4 = warp & 3, row = q4 * 32 + lane;
        const int st = tid - kSumWarp0 * 32;
        const uint32_t my = tmem + (static_cast<uint32_t>(q4 * 32) << 16);
        constexpr size_t kPart = 2 * NT * 128;  // floats of a part: gate and up, position, row
        bool ok = true;
        Ring<NB> b;
        int turn = 0;  // which group's block the next one is
        // waits for an accumulator and its scales
        const auto ready = [&]() {
            ok = __all_sync(~0u, ok && fp8_wait(&acc_full[b.s], b.filled(), p.status));
            tc_fence_after();
            return ok;
        };
        // leaves a part behind (already stored): true in the CTA that comes last, whose parts are all there
        const auto last_part = [&](int *count, int parts) {
            named_sync(1, kSumThreads);
            if (st == 0) s_int[2] = add_acq_rel(count, 1) == parts - 1;
            named_sync(1, kSumThreads);
            return s_int[2] != 0;
        };
        {
            float ga[S], ua[S];
            GateAt at;
            at.set(a0, U, KB1);
            int begin = a0;            // of the segment
            bool sparse = false, both = false;
            uint32_t lists[2] = {0u, 0u};  // tokens of a sparse unit, by half of the batch
            for (int t = a0; t < a1; ++t, turn ^= 1) {
                if (t == begin) {
#pragma unroll
                    for (int j = 0; j < S; ++j) ga[j] = ua[j] = 0.f;
                    sparse = sparse_unit(at.u);
                    both = F::kLists && !sparse;
                    if (sparse) {
                        const uint2 mask = s_mask[expert_of(at.u)];
                        lists[0] = mask.x;
                        lists[1] = mask.y;
                    }
                }
                if ((both || turn == grp) && ready()) {
                    const uint32_t acc = my + b.s * 2 * NT;
                    const float *const sc = sS + b.s * 2 * NT;
                    if (sparse) {
                        uint32_t vg[16], vu[16];
                        const int n[2] = {__popc(lists[0]), __popc(lists[1])};
#pragma unroll
                        for (int h = 0; h < 2; ++h) {
                            uint32_t left = lists[h];
#pragma unroll
                            for (int j = 0; j < 8; ++j) {
                                if (j >= n[h]) break;
                                const int m = h * 32 + __ffs(left) - 1;
                                tmem_ld1(acc + m, vg[h * 8 + j]);
                                tmem_ld1(acc + NT + m, vu[h * 8 + j]);
                                left &= left - 1;
                            }
                        }
                        tmem_wait(vg);
                        tmem_wait(vu);
#pragma unroll
                        for (int h = 0; h < 2; ++h)
#pragma unroll
                            for (int j = h * 8; j < h * 8 + 8; j += 2) {  // a pair's second value may be none: its sum is not used
                                if (j - h * 8 >= n[h]) break;
                                const float2 f = *reinterpret_cast<const float2 *>(sc + j), e = *reinterpret_cast<const float2 *>(sc + NT + j);
                                fma2(ga[j], ga[j + 1], vg[j], vg[j + 1], f.x, f.y);
                                fma2(ua[j], ua[j + 1], vu[j], vu[j + 1], e.x, e.y);
                            }
                    } else {
                        // columns of this thread: all NT, or its half of 64; C of gate and of up at a time
                        constexpr int C = F::kLists ? 8 : 16, N = F::kLists ? H : NT;
                        const int m0 = F::kLists ? grp * H : 0;
#pragma unroll
                        for (int cc = 0; cc < N; cc += C) {
                            uint32_t vg[C], vu[C];
                            tmem_ld<C>(acc + m0 + cc, vg);
                            tmem_ld<C>(acc + NT + m0 + cc, vu);
                            tmem_wait(vg);
                            tmem_wait(vu);
#pragma unroll
                            for (int j = 0; j < C; j += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(sc + m0 + cc + j), e = *reinterpret_cast<const float4 *>(sc + NT + m0 + cc + j);
                                fma2(ga[cc + j], ga[cc + j + 1], vg[j], vg[j + 1], f.x, f.y);
                                fma2(ga[cc + j + 2], ga[cc + j + 3], vg[j + 2], vg[j + 3], f.z, f.w);
                                fma2(ua[cc + j], ua[cc + j + 1], vu[j], vu[j + 1], e.x, e.y);
                                fma2(ua[cc + j + 2], ua[cc + j + 3], vu[j + 2], vu[j + 3], e.z, e.w);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&acc_empty[b.s], both ? 1 : 2);
                }
                b.next();
                if (at.kb == KB1 - 1 || t + 1 == a1) {
                    // The segment ends: a whole item, or a part of one.  The sums meet in shared memory, [gate, up][position]
                    // [row], and each warp takes every eighth position: its token's h of 128 columns, their scale, times the
                    // token's weight in the mixture.
                    const int e = expert_of(at.u), n = sparse ? 16 : both ? 32 : NT;  // positions at a time
                    const int i0 = t - at.kb, i1 = i0 + KB1;
                    const bool whole = begin == i0 && t + 1 == i1;
                    float *const mine = p.part + ((size_t)c * 2 + (begin != a0)) * kPart;
                    // the token at a position, p.M if there is none
                    const auto token_at = [&](int at_pos) {
                        if (!sparse) return at_pos;
                        uint32_t left = at_pos < 8 ? lists[0] : lists[1];
                        for (int j = 0; j < (at_pos & 7); ++j) left &= left - 1;
                        return left ? (at_pos >> 3) * 32 + __ffs(left) - 1 : p.M;
                    };
                    const auto finish = [&](int pos, float4 g, float4 u) {
                        const int m = token_at(pos);
                        float *const hs = p.hs + ((size_t)at.u * KB2 + at.ib) * NT + pos;
                        const bool hit = m < p.M && (shared_unit(at.u) ? lane == 0 : lane < p.k && s_idx[m * p.k + lane] == e);
                        const uint32_t hits = __ballot_sync(~0u, hit);
                        if (!hits) {  // this token did not choose the expert
                            if (lane == 0) *hs = 0.f;
                            return;
                        }
                        const float h0 = silu_f(g.x) * u.x, h1 = silu_f(g.y) * u.y, h2 = silu_f(g.z) * u.z, h3 = silu_f(g.w) * u.w;
                        const float own = max_magnitude(max_magnitude(h0, h1), max_magnitude(h2, h3));
                        const float sc = fp8_scale_of(__uint_as_float(__reduce_max_sync(~0u, __float_as_uint(own)))), inv = fp8_inverse(sc);
                        *reinterpret_cast<uint32_t *>(p.hq + ((size_t)at.u * NT + pos) * p.I + at.ib * 128 + lane * 4) =
                            e4m3x4(h0 * inv, h1 * inv, h2 * inv, h3 * inv);
                        if (hit) *hs = shared_unit(at.u) ? sc : chosen(sc * s_w[m * p.k + lane]);
                    };
                    if (!both) {
                        if (grp) {
#pragma unroll
                            for (int j = 0; j < S; ++j)
                                if (j < n) {
                                    s_sums[j * 128 + row] = ga[j];
                                    s_sums[(n + j) * 128 + row] = ua[j];
                                }
                        }
                        named_sync(1, kSumThreads);
                        if (!grp) {
#pragma unroll
                            for (int j = 0; j < S; ++j)
                                if (j < n) {
                                    s_sums[j * 128 + row] += ga[j];
                                    s_sums[(n + j) * 128 + row] += ua[j];
                                }
                        }
                    }
#pragma unroll
                    for (int round = 0; round < (F::kLists ? 2 : 1); ++round) {
                        if (round > 0 && !both) break;
                        if (both) {  // 16 tokens of each half at a time
#pragma unroll
                            for (int j = 0; j < 16; ++j) {
                                s_sums[(grp * 16 + j) * 128 + row] = ga[(round * 16 + j) % S];
                                s_sums[(32 + grp * 16 + j) * 128 + row] = ua[(round * 16 + j) % S];
                            }
                        }
                        named_sync(1, kSumThreads);
#pragma unroll 1
                        for (int j = st >> 5; j < n; j += kSumThreads / 32) {
                            const int pos = both ? (j >> 4) * 32 + round * 16 + (j & 15) : j;
                            if (!sparse && pos >= p.M) {
                                if (whole && lane == 0) p.hs[((size_t)at.u * KB2 + at.ib) * NT + pos] = 0.f;
                                continue;
                            }
                            const float4 g = *reinterpret_cast<const float4 *>(s_sums + j * 128 + lane * 4),
                                         u = *reinterpret_cast<const float4 *>(s_sums + (n + j) * 128 + lane * 4);
                            if (whole) {
                                finish(pos, g, u);
                            } else {
                                __stcg(reinterpret_cast<float4 *>(mine + pos * 128 + lane * 4), g);
                                __stcg(reinterpret_cast<float4 *>(mine + (NT + pos) * 128 + lane * 4), u);
                            }
                        }
                        named_sync(1, kSumThreads);
                    }
                    if (!whole) {
                        const int c0 = s1.owner(i0), c1 = s1.owner(i1 - 1);
                        if (last_part(p.count + c0, c1 - c0 + 1)) {
#pragma unroll 1
                            for (int pos = st >> 5; pos < (both ? 2 : 1) * n; pos += kSumThreads / 32) {
                                float4 g = make_float4(0.f, 0.f, 0.f, 0.f), u = g;
                                if (sparse || pos < p.M)
                                    add_parts(p.part + pos * 128 + lane * 4, NT * 128, kPart, c0, c1, s1.start(c0) != i0, &g, &u);
                                finish(pos, g, u);
                            }
                        }
                    }
                    begin = t + 1;
                }
                at.next(U, KB1);
            }
        }
        fence_async();
        named_sync(1, kSumThreads);
        if (st == 0) {
            fence_async();
            add_acq_rel(barrier, 1);
        }
        {
            float acc[S];
            DownAt at;
            at.set(b0, U, KB2);
            int begin = b0;
            const int per = U * KB2;
            for (int t = b0; t < b1; ++t, turn ^= 1) {
                if (t == begin) {
#pragma unroll
                    for (int j = 0; j < S; ++j) acc[j] = 0.f;
                    if (F::kLists)
                        for (int j = 0; j < H; ++j) s_sums[(grp * H + j) * 128 + row] = 0.f;
                }
                const bool sparse = sparse_unit(at.u);
                if ((F::kLists || turn == grp) && ready()) {
                    const uint32_t a = my + b.s * 2 * NT;
                    const float *const sc = sS + b.s * 2 * NT;
                    if (sparse) {
                        uint32_t v[8];
                        tmem_ld<8>(a + grp * 8, v);
                        tmem_wait(v);
#pragma unroll
                        for (int j = 0; j < 8; j += 4) {
                            const float4 f = *reinterpret_cast<const float4 *>(sc + grp * 8 + j);
                            fma2(acc[j], acc[j + 1], v[j], v[j + 1], f.x, f.y);
                            fma2(acc[j + 2], acc[j + 3], v[j + 2], v[j + 3], f.z, f.w);
                        }
                    } else {
                        constexpr int C = 16, N = F::kLists ? H : NT;
                        const int m0 = F::kLists ? grp * H : 0;
#pragma unroll
                        for (int cc = 0; cc < N; cc += C) {
                            uint32_t v[C];
                            tmem_ld<C>(a + m0 + cc, v);
                            tmem_wait(v);
#pragma unroll
                            for (int j = 0; j < C; j += 4) {
                                const float4 f = *reinterpret_cast<const float4 *>(sc + m0 + cc + j);
                                const float x[4] = {f.x, f.y, f.z, f.w};
#pragma unroll
                                for (int i = 0; i < 4; ++i)
                                    if (is_chosen(x[i])) acc[cc + j + i] = fmaf(__uint_as_float(v[j + i]), x[i], acc[cc + j + i]);
                            }
                        }
                    }
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_n(&acc_empty[b.s], F::kLists ? 1 : 2);
                }
                b.next();
                const bool ends = (at.u == U - 1 && at.kb == KB2 - 1) || t + 1 == b1;
                if (F::kLists && (at.kb == KB2 - 1 || ends)) {
                    // 64 tokens: a unit's sums go to their tokens' (each token belongs to one group)
                    if (sparse) {
                        const uint2 mask = s_mask[expert_of(at.u)];
                        uint32_t left = grp ? mask.y : mask.x;
#pragma unroll
                        for (int j = 0; j < 8; ++j) {
                            if (left) {
                                s_sums[(grp * H + __ffs(left) - 1) * 128 + row] += acc[j];
                                left &= left - 1;
                            }
                            acc[j] = 0.f;
                        }
                    } else {
#pragma unroll
                        for (int j = 0; j < S; ++j) {
                            s_sums[(grp * H + j) * 128 + row] += acc[j];
                            acc[j] = 0.f;
                        }
                    }
                }
                if (ends) {
                    // [token][row] in shared memory; each warp takes every eighth token
                    if (!F::kLists) {
                        if (grp) {
#pragma unroll
                            for (int j = 0; j < NT; ++j) s_sums[j * 128 + row] = acc[j % S];
                        }
                        named_sync(1, kSumThreads);
                        if (!grp) {
#pragma unroll
                            for (int j = 0; j < NT; ++j) s_sums[j * 128 + row] += acc[j % S];
                        }
                    }
                    named_sync(1, kSumThreads);
                    const int i0 = at.rb * per, i1 = i0 + per;
                    const bool whole = begin == i0 && t + 1 == i1;
                    float *const mine = p.part + ((size_t)c * 2 + (begin != b0)) * kPart;
                    const auto finish = [&](int m, float4 v) {
                        const size_t o = (size_t)m * p.Hd + at.rb * 128 + lane * 4;
                        if (p.residual) {
                            const uint2 w = *reinterpret_cast<const uint2 *>(p.residual + o);
                            v.x += bf16_lo(w.x), v.y += bf16_hi(w.x), v.z += bf16_lo(w.y), v.w += bf16_hi(w.y);
                        }
                        *reinterpret_cast<uint2 *>(p.y + o) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
                    };
#pragma unroll 1
                    for (int m = st >> 5; m < p.M; m += kSumThreads / 32) {
                        const float4 v = *reinterpret_cast<const float4 *>(s_sums + m * 128 + lane * 4);
                        if (whole) finish(m, v);
                        else __stcg(reinterpret_cast<float4 *>(mine + m * 128 + lane * 4), v);
                    }
                    named_sync(1, kSumThreads);
                    if (!whole) {
                        const int c0 = s2.owner(i0), c1 = s2.owner(i1 - 1);
                        if (last_part(p.count + G + c0, c1 - c0 + 1)) {
#pragma unroll 1
                            for (int m = st >> 5; m < p.M; m += 2 * (kSumThreads / 32)) {  // a second token beside it: 64 of hidden 1024 104 us, 96
                                const int m2 = m + kSumThreads / 32 < p.M ? m + kSumThreads / 32 : m;
                                float4 v = make_float4(0.f, 0.f, 0.f, 0.f), v2 = v;
                                add_parts(p.part + m * 128 + lane * 4, (m2 - m) * 128, kPart, c0, c1, s2.start(c0) != i0, &v, &v2);
                                finish(m, v);
                                if (m2 != m) finish(m2, v2);
                            }
                        }
                    }
                    begin = t + 1;
                }
                at.next(U, KB2);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && !s_int[1]) drain_fills<NS>(full, issued, p.status);
    __syncwarp();
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, F::kColumns);
}

// ----------------------------------------------------------------------------- host

template <int NT>
cudaError_t launch_moe(const MoeMaps &maps, const MoeParams &p, int grid, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(moe_fp8_kernel<NT>, Moe<NT>::kSmem, done);
    if (e != cudaSuccess) return e;
    return launch_kernel_as(moe_fp8_kernel<NT>, dim3((unsigned)grid), dim3(kMoeThreads), Moe<NT>::kSmem, st, 1, true, maps, p);
}

int check_moe(const hla_moe_fp8 *L) {
    HLA_REQUIRE(L && L->hidden >= 1 && L->inter >= 1 && L->n_experts >= 1 && L->top_k >= 1 && L->n_shared >= 0, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(L->top_k <= L->n_experts, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(L->hidden % 128 == 0 && L->inter % 128 == 0 && L->top_k <= kMaxTopK, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE((long)L->n_experts + L->n_shared <= kMaxExperts && L->n_shared <= 16, HLA_ERR_UNSUPPORTED);
    // rows of the weight stacks and bytes of one row stay in 31 bits, and blocks (256 GB of a matrix) in 24
    HLA_REQUIRE(L->hidden <= 1 << 20 && L->inter <= 1 << 20, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(((long)L->n_experts + L->n_shared) * (L->hidden / 128) * (L->inter / 128) < 1L << 24, HLA_ERR_UNSUPPORTED);
    return HLA_OK;
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" size_t moe_fp8_forward_workspace_size(const hla_moe_fp8 *L, int M) {
    if (check_moe(L) != HLA_OK || M < 1 || M > kMaxTokens) return 0;
    return moe_space(L, M).total;
}

extern "C" int moe_fp8_forward(const hla_moe_fp8 *L, int M, const hla_bf16 *x, const hla_bf16 *residual, hla_bf16 *y,
                               int32_t *topk_idx, float *topk_w, void *ws, size_t ws_bytes, hla_stream stream) {
    int e = check_moe(L);
    if (e != HLA_OK) return e;
    HLA_REQUIRE(M >= 1 && x && y, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(M <= kMaxTokens, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(L->W_router && L->W_gate && L->W_up && L->W_down && L->S_gate && L->S_up && L->S_down, HLA_ERR_INVALID_ARG);
    const bool sh = L->n_shared > 0;
    HLA_REQUIRE(!sh || (L->Ws_gate && L->Ws_up && L->Ws_down && L->Ss_gate && L->Ss_up && L->Ss_down), HLA_ERR_INVALID_ARG);
    for (const void *q : {(const void *)x, (const void *)residual, (const void *)y, (const void *)topk_idx, (const void *)topk_w,
                          (const void *)L->W_router, (const void *)L->W_gate, (const void *)L->W_up, (const void *)L->W_down,
                          (const void *)L->S_gate, (const void *)L->S_up, (const void *)L->S_down})
        HLA_REQUIRE(aligned16(q), HLA_ERR_MISALIGNED);
    if (sh)
        for (const void *q : {(const void *)L->Ws_gate, (const void *)L->Ws_up, (const void *)L->Ws_down, (const void *)L->Ss_gate,
                              (const void *)L->Ss_up, (const void *)L->Ss_down})
            HLA_REQUIRE(aligned16(q), HLA_ERR_MISALIGNED);
    const MoeSpace sp = moe_space(L, M);
    HLA_REQUIRE(ws && ws_bytes >= sp.total, HLA_ERR_WORKSPACE);
    HLA_REQUIRE(aligned16(ws), HLA_ERR_MISALIGNED);

    const int NT = tokens_padded(M), Hd = L->hidden, I = L->inter, E = L->n_experts, U = moe_units_most(L, M), sms = sm_count();
    uint8_t *const w = static_cast<uint8_t *>(ws);
    // no more CTAs than the largest phase can have blocks
    const long most = (long)U * (I / 128) * (Hd / 128);
    const int grid = (int)(most < sms ? most : sms);

    MoeParams p = {};
    p.M = M; p.Hd = Hd; p.I = I; p.E = E; p.k = L->top_k; p.n_shared = L->n_shared;
    p.logits = reinterpret_cast<float *>(w + sp.logits);
    p.xs = reinterpret_cast<float *>(w + sp.xs);
    p.gate_s = L->S_gate; p.up_s = L->S_up; p.down_s = L->S_down;
    p.sgate_s = L->Ss_gate; p.sup_s = L->Ss_up; p.sdown_s = L->Ss_down;
    p.residual = residual; p.y = y; p.topk_idx = topk_idx; p.topk_w = topk_w;
    p.hq = w + sp.hq;
    p.hs = reinterpret_cast<float *>(w + sp.hs);
    p.part = reinterpret_cast<float *>(w + sp.part);
    p.count = reinterpret_cast<int *>(w + sp.count);
    p.status = device_status_word();
    HLA_REQUIRE(p.status, HLA_ERR_CUDA);
    p.force_timeout = wait_timeout_forced();
    MoeMaps maps;
    bool ok = byte_tile_map(&maps.x, w + sp.xq, M, Hd, NT) && byte_tile_map(&maps.h, p.hq, (uint64_t)U * NT, I, NT) && byte_tile_map(&maps.hfew, p.hq, (uint64_t)U * NT, I, 16) &&
              byte_tile_map(&maps.gate, L->W_gate, (uint64_t)E * I, Hd, 128) && byte_tile_map(&maps.up, L->W_up, (uint64_t)E * I, Hd, 128) &&
              byte_tile_map(&maps.down, L->W_down, (uint64_t)E * Hd, I, 128);
    if (sh)
        ok = ok && byte_tile_map(&maps.sgate, L->Ws_gate, (uint64_t)L->n_shared * I, Hd, 128) &&
             byte_tile_map(&maps.sup, L->Ws_up, (uint64_t)L->n_shared * I, Hd, 128) &&
             byte_tile_map(&maps.sdown, L->Ws_down, (uint64_t)L->n_shared * Hd, I, 128);
    else
        maps.sgate = maps.gate, maps.sup = maps.up, maps.sdown = maps.down;
    HLA_REQUIRE(ok, HLA_ERR_CUDA);

    const cudaStream_t st = (cudaStream_t)stream;
    set_variant("moe_fp8<tokens%d,ctas%d>", NT, grid);
    PdlChain chain(st, pdl_default(1));
    PrepParams q = {};
    q.M = M; q.Hd = Hd; q.E = E; q.NT = NT;
    q.router_clusters = (E + kPrepExperts - 1) / kPrepExperts;
    q.counters = 2 * grid + 1;
    q.x = x; q.Wr = L->W_router; q.logits = const_cast<float *>(p.logits); q.xq = w + sp.xq; q.xs = const_cast<float *>(p.xs); q.count = p.count;
    const int per = kPrepCluster * (kPrepThreads / 8);
    const long convert = ((long)M * (Hd / kFp8Block) + per - 1) / per;
    e = launched(launch_kernel(moe_prep_kernel, dim3((unsigned)((q.router_clusters + convert) * kPrepCluster)), dim3(kPrepThreads), 0, st, q));
    if (e != HLA_OK) return e;
    if (M > kChooseInside) {
        const ChooseParams r = {E, L->top_k, p.logits, reinterpret_cast<int32_t *>(w + sp.idx), topk_idx, reinterpret_cast<float *>(w + sp.w), topk_w};
        p.idx = r.idx;
        p.w = r.w;
        e = launched(launch_kernel(moe_choose_kernel, dim3((unsigned)M), dim3(32), 0, st, r));
        if (e != HLA_OK) return e;
    }
    const cudaError_t ce = NT == 16 ? launch_moe<16>(maps, p, grid, st) : NT == 32 ? launch_moe<32>(maps, p, grid, st) : launch_moe<64>(maps, p, grid, st);
    return launched(ce);
}
