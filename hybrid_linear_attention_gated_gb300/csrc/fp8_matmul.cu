// Matrix product of e4m3 matrices with a scale for each block of 128 along K:
//   y[m, n] = sum_b (x_scale[m, b] * w_scale[n / 128, b]) * sum_{k in b} x[m, k] W[n, k]  (+ residual[m, n]).
//
// Each block's product runs on tcgen05 (kind::f8f6f4, fp32 accumulator in tensor memory, overwritten by every block);
// warps of their own read it back and add it, scaled, to sums in registers, while the next block's product runs into another
// accumulator.  One warp copies tiles by TMA into a ring, one issues the products.
//
//  * Up to 32 tokens (`few_kernel`): bound by HBM, every weight byte is read once.  128 weight rows lie on the lanes and
//    16 or 32 tokens on the columns, so that a product of few tokens still fills the tensor core's rows.  K is cut among the
//    1 to 8 CTAs of a cluster, which add their sums through distributed shared memory in rank order: one launch, no
//    workspace, no atomics.
//  * More tokens (`many_kernel`, `pair_kernel`): 128 tokens on the lanes of a CTA, 128 weight rows (192 or 256 of a pair of CTAs) on the
//    columns.  A thread's row has one token scale and its columns one or two weight scales per block, so scaling is one
//    multiplication per block and one FMA per value; a warp copies the scales eight blocks ahead.
//
// Every wait is bounded (see tc_gemm.cu for the drain order): a wait that gives up sets the device status word, the roles
// leave their loops, issued products and copies are waited for, and tensor memory is freed.
#include "fp8.cuh"

namespace hla {
namespace {

struct MatmulParams {
    int M, N, K, KB;           // KB: blocks of 128 along K
    int split;                 // CTAs per cluster, each a share of the blocks
    int row_tiles, col_tiles;  // many_kernel: tiles of tokens and of weight rows
    const float *xs, *ws;
    const uint16_t *residual;
    void *y;
    int y_bf16;
    int direct;                // rows of y keep 32-byte stores aligned
    int *status;
    int force_timeout;
};

__device__ __forceinline__ void store_y(const MatmulParams &p, size_t at, float v) {
    if (p.residual) v += bf16_bits_to_float(p.residual[at]);
    if (p.y_bf16) static_cast<uint16_t *>(p.y)[at] = float_to_bf16_bits(v);
    else static_cast<float *>(p.y)[at] = v;
}

// Four columns of token m from a column that is a multiple of 4 on: one access where y's rows keep it aligned.
__device__ __forceinline__ void store_y4(const MatmulParams &p, int m, int col, float4 v) {
    const size_t at = (size_t)m * p.N + col;
    if (p.N % 4 == 0) {
        if (col >= p.N) return;
        if (p.residual) {
            const uint2 r = *reinterpret_cast<const uint2 *>(p.residual + at);
            v.x += bf16_lo(r.x), v.y += bf16_hi(r.x), v.z += bf16_lo(r.y), v.w += bf16_hi(r.y);
        }
        if (p.y_bf16)
            *reinterpret_cast<uint2 *>(static_cast<uint16_t *>(p.y) + at) = make_uint2(pack_bf16x2(v.x, v.y), pack_bf16x2(v.z, v.w));
        else
            *reinterpret_cast<float4 *>(static_cast<float *>(p.y) + at) = v;
        return;
    }
    const float x[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
    for (int j = 0; j < 4; ++j)
        if (col + j < p.N) store_y(p, at + j, x[j]);
}

// ----------------------------------------------------------------------------- up to 32 tokens

constexpr int kFewThreads = 192;       // copies, products, four warps of sums
constexpr int kScaleChunk = 32;        // blocks whose scales are in shared memory at once
constexpr uint32_t kTileBytes = 128 * 128;

template <int NT>
struct Few {
    static constexpr int kStages = NT == 16 ? 6 : 5;                 // about 100 KB: two CTAs to an SM
    static constexpr int kAcc = 4;                                   // accumulators in tensor memory
    static constexpr uint32_t kTokenBytes = NT * 128;
    static constexpr uint32_t kColumns = kAcc * NT;
    static constexpr size_t kSmem = 1024 + kStages * (kTileBytes + kTokenBytes) + kScaleChunk * NT * 4 + (2 * kStages + 2 * kAcc + 1) * 8 + 16;
    static_assert(NT * 128 * 4 <= kStages * kTileBytes, "the sums of the join take the place of the tiles");
};

template <int NT>
__global__ void __launch_bounds__(kFewThreads, 2)
    few_kernel(const __grid_constant__ CUtensorMap tmW, const __grid_constant__ CUtensorMap tmX, const MatmulParams p) {
    using F = Few<NT>;
    constexpr int NS = F::kStages, NB = F::kAcc;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const sW = smem, *const sX = smem + NS * kTileBytes;
    float *const sScale = reinterpret_cast<float *>(sX + NS * F::kTokenBytes);
    uint64_t *const full = reinterpret_cast<uint64_t *>(sScale + kScaleChunk * NT);
    uint64_t *const empty = full + NS, *const acc_full = empty + NS, *const acc_empty = acc_full + NB, *const done = acc_empty + NB;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    int *const consumed_slot = reinterpret_cast<int *>(tmem_slot + 1);

    if (p.force_timeout) {
        forced_timeout(done, p.status);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int rb = blockIdx.x / p.split, rank = blockIdx.x - rb * p.split;
    const int c0 = (int)((long)p.KB * rank / p.split), n = (int)((long)p.KB * (rank + 1) / p.split) - c0;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 4);
        }
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(tmem_slot, F::kColumns);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    if (warp != 0) pdl_wait_trigger();  // the copying thread waits after its first weight tiles

    int issued = 0;
    float acc[NT];
    bool ok = true;
    if (warp == 0) {
        // two weight tiles go out before the kernel that writes the tokens is done, the rest once the first scales are on their
        // way: behind a whole ring of tiles they would arrive microseconds later
        const int pre = n < 2 ? n : 2;
        if (lane == 0)
            for (int i = 0; i < pre; ++i) {
                mbar_expect_tx(&full[i], kTileBytes + F::kTokenBytes);
                tma_tile(sW + i * kTileBytes, &tmW, (c0 + i) * kFp8Block, rb * 128, &full[i]);
            }
        pdl_wait_trigger();
        named_sync(2, 160);
        if (lane == 0) {
            for (int i = 0; i < pre; ++i) tma_tile(sX + i * F::kTokenBytes, &tmX, (c0 + i) * kFp8Block, 0, &full[i]);
            issued = pre;
            for (int i = pre; i < n; ++i) {
                const int s = i % NS;
                if (i >= NS && !fp8_wait(&empty[s], (i / NS - 1) & 1, p.status)) break;
                mbar_expect_tx(&full[s], kTileBytes + F::kTokenBytes);
                tma_tile(sW + s * kTileBytes, &tmW, (c0 + i) * kFp8Block, rb * 128, &full[s]);
                tma_tile(sX + s * F::kTokenBytes, &tmX, (c0 + i) * kFp8Block, 0, &full[s]);
                issued = i + 1;
            }
        }
    } else if (warp == 1) {
        int i = 0;
        for (; i < n; ++i) {
            const int s = i % NS, b = i % NB;
            if (!__all_sync(~0u, (i < NB || fp8_wait(&acc_empty[b], (i / NB - 1) & 1, p.status)) && fp8_wait(&full[s], (i / NS) & 1, p.status)))
                break;
            tc_fence_after();
            umma_block(tmem + b * NT, smem_u32(sW + s * kTileBytes), smem_u32(sX + s * F::kTokenBytes), idesc_e4m3(128, NT));
            umma_commit_elected(&empty[s]);
            umma_commit_elected(&acc_full[b]);
        }
        if (lane == 0) *consumed_slot = i;
        umma_commit_elected(done);
        if (!fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else if (warp >= 2) {
        const int t = tid - 64;
        const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
        constexpr int kPer = NT * kScaleChunk / 128;
        float sx[kPer], sw = 0.f;  // this thread's block of a chunk, and every fourth token's scale
        const auto load_scales = [&](int i0) {
            const int k = i0 + t % kScaleChunk;
            if (k < n) sw = p.ws[(size_t)rb * p.KB + c0 + k];
#pragma unroll
            for (int j = 0; j < kPer; ++j) {
                const int tok = t / kScaleChunk + j * (128 / kScaleChunk);
                sx[j] = k < n && tok < p.M ? p.xs[(size_t)tok * p.KB + c0 + k] : 0.f;
            }
        };
        load_scales(0);
        named_sync(2, 160);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = 0.f;
        for (int i = 0; i < n; ++i) {  // to the end even after a wait that gave up: the four warps meet at each chunk
            if (i % kScaleChunk == 0) {  // x_scale * w_scale of the next blocks, a row of tokens per block; those behind them are loaded
                if (i > 0) named_sync(1, 128);
#pragma unroll
                for (int j = 0; j < kPer; ++j) sScale[(t % kScaleChunk) * NT + t / kScaleChunk + j * (128 / kScaleChunk)] = sx[j] * sw;
                load_scales(i + kScaleChunk);
                named_sync(1, 128);
            }
            const int b = i % NB;
            ok = __all_sync(~0u, ok && fp8_wait(&acc_full[b], (i / NB) & 1, p.status));
            if (!ok) continue;
            tc_fence_after();
            const float *const sc = sScale + (i % kScaleChunk) * NT;
            uint32_t v[NT];
            tmem_ld<NT>(my + b * NT, v);
            tmem_wait(v);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
#pragma unroll
            for (int j = 0; j < NT; j += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(sc + j);
                acc[j] = fmaf(__uint_as_float(v[j]), f.x, acc[j]);
                acc[j + 1] = fmaf(__uint_as_float(v[j + 1]), f.y, acc[j + 1]);
                acc[j + 2] = fmaf(__uint_as_float(v[j + 2]), f.z, acc[j + 2]);
                acc[j + 3] = fmaf(__uint_as_float(v[j + 3]), f.w, acc[j + 3]);
            }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && *consumed_slot < issued) drain_fills<NS>(full, issued, p.status);
    __syncwarp();
    __syncthreads();
    // the tiles are used up: their place takes the sums [token][weight row]
    float *const sums = reinterpret_cast<float *>(smem);
    if (warp >= 2) {
        const int row = (warp & 3) * 32 + lane;
#pragma unroll
        for (int j = 0; j < NT; ++j) sums[j * 128 + row] = acc[j];
    }
    if (p.split > 1) cluster_sync();
    else __syncthreads();
#pragma unroll 1
    for (int e = (rank * kFewThreads + tid) * 4; e < p.M * 128; e += p.split * kFewThreads * 4) {
        const int m = e >> 7, col = rb * 128 + (e & 127);
        float4 part[8];
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < p.split) part[r] = peer_float4(sums + e, r);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int r = 0; r < 8; ++r)
            if (r < p.split) v.x += part[r].x, v.y += part[r].y, v.z += part[r].z, v.w += part[r].w;
        store_y4(p, m, col, v);
    }
    if (p.split > 1) cluster_sync();  // no CTA leaves while another reads its sums
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, F::kColumns);
}

// ----------------------------------------------------------------------------- more tokens

constexpr int kManyThreads = 384;  // a warpgroup of copies and products, two of sums
// registers a thread: 168 at launch; the sums and what is on its way take more, which the first warpgroup leaves
constexpr int kFewRegs = 56, kManyRegs = 224;
static_assert(kFewRegs + 2 * kManyRegs <= 3 * 168, "shares of the registers at launch");
constexpr int kOutPitch = 33;
constexpr size_t kOutBytes = 8 * 32 * kOutPitch * 4;  // a warp's 32 rows x 32 columns on their way out

// Tiles in bands of `kBand` row tiles, down a band's columns: the tiles in flight share their operands in L2.
__device__ __forceinline__ void tile_at(const MatmulParams &p, int t, int *rt, int *ct) {
    constexpr int kBand = 16;
    const int band = t / (kBand * p.col_tiles), first = band * kBand;
    const int rows = p.row_tiles - first < kBand ? p.row_tiles - first : kBand;
    const int r = t - first * p.col_tiles;
    *ct = r / rows;
    *rt = first + r - *ct * rows;
}

// Scales in shared memory, kScaleRing blocks of K ahead: a warp copies the 128 tokens' and, for `blocks` blocks of weight rows
// from `wb` on, one each.  An entry is 128 + 4 floats; its `full` barrier counts every lane's copies, its `empty` the eight
// warps of sums.
constexpr int kScaleRing = 8, kScaleEntry = 132;
constexpr size_t kScaleBytes = kScaleRing * kScaleEntry * 4;

struct ScaleRing {
    float *entries;
    uint64_t *full, *empty;
    int e = 0, turn = 0;
    __device__ __forceinline__ void init() const {
        for (int i = 0; i < kScaleRing; ++i) {
            mbar_init(&full[i], 32);
            mbar_init(&empty[i], 8);
        }
    }
    __device__ __forceinline__ void next() {
        if (++e == kScaleRing) e = 0, ++turn;
    }
    // one tile's blocks [c0, c0 + n), tokens from `tok` on; false if a wait gave up
    __device__ __forceinline__ bool copy_tile(const MatmulParams &p, int tok, int wb, int c0, int n, int lane) {
        const int last = (p.N - 1) >> 7;  // columns behind the last are not stored, whatever their scale
        const float *x[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) x[j] = p.xs + (size_t)(tok + j * 32 + lane < p.M ? tok + j * 32 + lane : p.M - 1) * p.KB + c0;
        const float *const w = p.ws + (size_t)(wb + lane < last ? wb + lane : last) * p.KB + c0;
        for (int i = 0; i < n; ++i) {
            if (!__all_sync(~0u, turn == 0 || fp8_wait(&empty[e], (turn - 1) & 1, p.status))) return false;
            float *const to = entries + e * kScaleEntry;
#pragma unroll
            for (int j = 0; j < 4; ++j) cp_async4(to + j * 32 + lane, x[j] + i);
            if (lane < 2) cp_async4(to + 128 + lane, w + i);
            asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(&full[e])) : "memory");
            next();
        }
        return true;
    }
};

// acc += the accumulator's COLS columns at `at`, times the scales: `s0` up to column `cut` * 32, `s1` from there on.  `early` is
// called while the first columns are on their way, `release` once the last have been read.  16 columns at a time: 128 at
// 357 cycles beside the products; with 32 the registers spill (575).
template <int COLS, typename Early, typename Release>
__device__ __forceinline__ void add_block(float (&acc)[COLS], uint32_t at, float s0, float s1, int cut, Early early, Release release) {
    constexpr int C = 16;
    uint32_t v[2][C];
    tmem_ld<C>(at, v[0]);
    early();
#pragma unroll
    for (int c = 0; c < COLS / C; ++c) {
        tmem_wait(v[c & 1]);
        if (c + 1 < COLS / C) tmem_ld<C>(at + (c + 1) * C, v[(c + 1) & 1]);
        else release();
        const float sc = c * C < cut * 32 ? s0 : s1;
#pragma unroll
        for (int j = 0; j < C; j += 2) fma2(acc[c * C + j], acc[c * C + j + 1], v[c & 1][j], v[c & 1][j + 1], sc, sc);
    }
}

__device__ __forceinline__ void st32b(void *p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]),
                 "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7])
                 : "memory");
}
// A thread's row of COLS columns, straight from registers: 32 bytes a store, whole sectors.  What is added is loaded 64 columns
// at once.
template <int COLS>
__device__ __forceinline__ void store_row(const MatmulParams &p, size_t at, int columns, const float (&acc)[COLS]) {
    constexpr int B = COLS == 128 ? 64 : 32;
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += B) {
        uint4 w[B / 8] = {};
        if (p.residual) {
#pragma unroll
            for (int c = 0; c < B; c += 8)
                if (c0 + c < COLS && c0 + c < columns) w[c / 8] = ld_act_v4(p.residual + at + c0 + c);
        }
#pragma unroll
        for (int c = 0; c < B; c += 16) {
            if (c0 + c >= COLS || c0 + c >= columns) break;
            float v[16];
#pragma unroll
            for (int j = 0; j < 16; j += 2) {
                const uint4 &q = w[(c + j) / 8];
                const uint32_t r = j % 8 == 0 ? q.x : j % 8 == 2 ? q.y : j % 8 == 4 ? q.z : q.w;
                v[j] = acc[(c0 + c + j) % COLS] + bf16_lo(r);
                v[j + 1] = acc[(c0 + c + j + 1) % COLS] + bf16_hi(r);
            }
            uint32_t r[8];
            if (p.y_bf16) {
#pragma unroll
                for (int j = 0; j < 8; ++j) r[j] = pack_bf16x2(v[2 * j], v[2 * j + 1]);
                st32b(static_cast<uint16_t *>(p.y) + at + c0 + c, r);
            } else {
#pragma unroll
                for (int h = 0; h < 2; ++h) {
#pragma unroll
                    for (int j = 0; j < 8; ++j) r[j] = __float_as_uint(v[8 * h + j]);
                    st32b(static_cast<float *>(p.y) + at + c0 + c + 8 * h, r);
                }
            }
        }
    }
}

// A warp's 32 tokens from `tok` on (lane = token), COLS columns from n0 on.
template <int COLS>
__device__ __forceinline__ void store_tile(const MatmulParams &p, int tok, int n0, int lane, const float (&acc)[COLS], float *out) {
    const int rows = p.M - tok < 32 ? p.M - tok : 32;
    if (p.direct) {
        if (lane < rows && n0 < p.N) store_row(p, (size_t)(tok + lane) * p.N + n0, p.N - n0, acc);
        return;
    }
    // Rows that keep no alignment leave through shared memory, 32 rows x 32 columns at a time, so that a warp's stores are 64
    // bytes of one row.  What is added is loaded as many rows at once as the registers hold beside the sums.  Behind the last row
    // and column those themselves are loaded: with a condition at each load they wait for one another (280 tokens to rows of 5115 of
    // K 224: 13.2 us, 8.8 without; 333 to rows of 7001 of 4112: 27.3, 24.8).
    constexpr int R = COLS == 64 ? 16 : 32;
#pragma unroll
    for (int c0 = 0; c0 < COLS; c0 += 32) {
        const int col = n0 + c0 + lane;
        uint16_t o[R];
        const auto load = [&](int k0) {
            const uint16_t *const at = p.residual + (size_t)tok * p.N + (col < p.N ? col : p.N - 1);
#pragma unroll
            for (int k = 0; k < R; ++k) o[k] = at[(size_t)(k0 + k < rows ? k0 + k : rows - 1) * p.N];
        };
        if (p.residual && R == 32 && rows > 0) load(0);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 32; ++j) out[lane * kOutPitch + j] = acc[c0 + j];
        __syncwarp();
#pragma unroll 1
        for (int k0 = 0; k0 < rows; k0 += R) {
            if (p.residual && R < 32) load(k0);
            if (col >= p.N) break;
            const size_t at = (size_t)(tok + k0) * p.N + col;
#pragma unroll
            for (int k = 0; k < R; ++k) {
                if (k0 + k >= rows) break;
                float v = out[(k0 + k) * kOutPitch + lane];
                if (p.residual) v += bf16_bits_to_float(o[k]);
                if (p.y_bf16) static_cast<uint16_t *>(p.y)[at + (size_t)k * p.N] = float_to_bf16_bits(v);
                else static_cast<float *>(p.y)[at + (size_t)k * p.N] = v;
            }
        }
    }
}

// The rows that store_tile adds come to L2 while the products run.
template <int COLS>
__device__ __forceinline__ void prefetch_residual(const MatmulParams &p, int m, int n0) {
    if (!p.residual || m >= p.M) return;
#pragma unroll
    for (int c = 0; c < COLS; c += 32)
        if (n0 + c < p.N) asm volatile("prefetch.global.L2 [%0];" ::"l"(p.residual + (size_t)m * p.N + n0 + c));
}

// ---- one CTA a tile of 128 tokens x 128 weight rows; K cut among the CTAs of a cluster

struct Many {
    static constexpr int kCols = 64;      // columns of a warpgroup
    static constexpr int kStages = 5;     // 160 KB
    static constexpr int kAcc = 4;        // accumulators: all of tensor memory
    static constexpr int kPitch = 132;    // floats of a row of the join
    static constexpr size_t kRing = kStages * 2 * kTileBytes;
    static constexpr size_t kSmem = 1024 + kRing + kOutBytes + kScaleBytes + (2 * kStages + 2 * kAcc + 2 * kScaleRing + 1) * 8 + 16;
    static_assert(128 * kPitch * 4 <= kRing, "the sums of the join take the place of the tiles");
    static_assert(kSmem <= 227 * 1024, "one CTA to an SM");
};

// This CTA's share of the tile's rows: the sums of the cluster's CTAs, in rank order.
__device__ __forceinline__ void join_tile(const MatmulParams &p, int unit, int rank, const float *sums) {
    int rt, ct;
    tile_at(p, unit, &rt, &ct);
#pragma unroll 1
    for (int e = rank * kManyThreads + threadIdx.x; e < 128 * 32; e += p.split * kManyThreads) {
        const int r = e >> 5, c = (e & 31) * 4, tok = rt * 128 + r;
        if (tok >= p.M) continue;
        float4 part[8];
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < p.split) part[k] = peer_float4(sums + r * Many::kPitch + c, k);
        float4 v = make_float4(0.f, 0.f, 0.f, 0.f);
#pragma unroll
        for (int k = 0; k < 8; ++k)
            if (k < p.split) v.x += part[k].x, v.y += part[k].y, v.z += part[k].z, v.w += part[k].w;
        store_y4(p, tok, ct * 128 + c, v);
    }
}

__global__ void __launch_bounds__(kManyThreads, 1)
    many_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const MatmulParams p) {
    using F = Many;
    constexpr int NS = F::kStages, NB = F::kAcc, COLS = F::kCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const sX = smem, *const sW = smem + NS * kTileBytes;
    float *const sOut = reinterpret_cast<float *>(smem + F::kRing);
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + F::kRing + kOutBytes + kScaleBytes);
    uint64_t *const empty = full + NS, *const acc_full = empty + NS, *const acc_empty = acc_full + NB, *const done = acc_empty + NB;
    ScaleRing scales;
    scales.entries = reinterpret_cast<float *>(smem + F::kRing + kOutBytes);
    scales.full = done + 1;
    scales.empty = scales.full + kScaleRing;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(scales.empty + kScaleRing);
    int *const failed_slot = reinterpret_cast<int *>(tmem_slot + 1);

    if (p.force_timeout) {
        forced_timeout(done, p.status);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int unit = blockIdx.x / p.split, units = gridDim.x / p.split, rank = blockIdx.x - unit * p.split;
    const int c0 = (int)((long)p.KB * rank / p.split), n = (int)((long)p.KB * (rank + 1) / p.split) - c0;
    const int tiles = p.row_tiles * p.col_tiles;

    if (tid == 0) {
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        scales.init();
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(tmem_slot, 512);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_trigger();

    const int group = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;  // which half of the columns, and which token of the tile
    float acc[COLS];
    int issued = 0;  // fills so far, up to multiples of 2 NS
    if (warp == 0 && lane == 0) {
        bool ok = true;
        int s = 0, turn = 0;    // the stage, and how often the ring went round
        for (int t = unit; t < tiles && ok; t += units) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            for (int i = 0; i < n; ++i) {
                if (turn > 0 && !(ok = fp8_wait(&empty[s], (turn - 1) & 1, p.status))) break;
                mbar_expect_tx(&full[s], 2 * kTileBytes);
                tma_tile(sX + s * kTileBytes, &tmX, (c0 + i) * kFp8Block, rt * 128, &full[s]);
                tma_tile(sW + s * kTileBytes, &tmW, (c0 + i) * kFp8Block, ct * 128, &full[s]);
                if (++s == NS) s = 0, ++turn;
            }
        }
        issued = turn > 1 ? (turn & 1 ? NS : 2 * NS) + s : turn * NS + s;
    } else if (warp == 1) {
        bool ok = true;
        int s = 0, ring = 0, b = 0, turn = 0;  // stage and its parity, accumulator and how often it was used
        for (int t = unit; t < tiles && ok; t += units)
            for (int i = 0; i < n; ++i) {
                ok = __all_sync(~0u, (turn == 0 || fp8_wait(&acc_empty[b], (turn - 1) & 1, p.status)) && fp8_wait(&full[s], ring, p.status));
                if (!ok) break;
                tc_fence_after();
                umma_block(tmem + b * 128, smem_u32(sX + s * kTileBytes), smem_u32(sW + s * kTileBytes), idesc_e4m3(128, 128));
                umma_commit_elected(&empty[s]);
                umma_commit_elected(&acc_full[b]);
                if (++s == NS) s = 0, ring ^= 1;
                if (++b == NB) b = 0, ++turn;
            }
        if (lane == 0) *failed_slot = !ok;
        umma_commit_elected(done);
        if (!fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else if (warp == 2) {
        bool ok = true;
        for (int t = unit; t < tiles && ok; t += units) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            ok = scales.copy_tile(p, rt * 128, ct, c0, n, lane);
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= 4) {
        const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + group * COLS;
        bool ok = true, early = false;  // early: the next block was seen to be ready
        int b = 0, ring = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            const int m = rt * 128 + row, n0 = ct * 128 + group * COLS;
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
            if (p.split == 1) prefetch_residual<COLS>(p, m, n0);
            for (int i = 0; i < n; ++i) {
                ok = early || __all_sync(~0u, fp8_wait(&scales.full[scales.e], scales.turn & 1, p.status) && fp8_wait(&acc_full[b], ring, p.status));
                if (!ok) break;
                tc_fence_after();
                const float *const sc = scales.entries + scales.e * kScaleEntry;
                const float s0 = sc[row] * sc[128];
                const int this_b = b, this_e = scales.e;
                scales.next();
                if (++b == NB) b = 0, ring ^= 1;
                bool next = false;
                add_block<COLS>(acc, my + this_b * 128, s0, s0, COLS,
                                [&] { next = mbar_test(&scales.full[scales.e], scales.turn & 1) && mbar_test(&acc_full[b], ring); },
                                [&] {
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) {
                                        mbar_arrive(&acc_empty[this_b]);
                                        mbar_arrive(&scales.empty[this_e]);
                                    }
                                });
                early = __all_sync(~0u, next);
            }
            if (ok && p.split == 1) store_tile<COLS>(p, rt * 128 + (warp & 3) * 32, n0, lane, acc, sOut + (warp - 4) * 32 * kOutPitch);
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && *failed_slot) drain_fills<NS>(full, issued, p.status);
    __syncwarp();
    __syncthreads();
    if (p.split > 1) {
        // one tile per cluster; the tiles of the ring are used up: their place takes the sums, a row per token
        float *const sums = reinterpret_cast<float *>(smem);
        if (warp >= 4) {
#pragma unroll
            for (int j = 0; j < COLS; j += 4)
                *reinterpret_cast<float4 *>(sums + row * F::kPitch + group * COLS + j) = make_float4(acc[j], acc[j + 1], acc[j + 2], acc[j + 3]);
        }
        cluster_sync();
        join_tile(p, unit, rank, sums);
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, 512);
}

// ---- a pair of CTAs a tile of 256 tokens x NT weight rows: each CTA copies 128 tokens and half of the weight rows, the even one
// issues the products of both (cta_group::2), and each adds up its own tokens.  A CTA reads (128 + NT / 2) x 128 bytes per
// 128 x NT of output, where one that is alone reads (128 + NT) x 128.  What bounds both is the sums: reading
// 128 x 256 accumulators back and the barriers take about 900 cycles a block, the products 512.

template <int NT>
struct Pair {
    static constexpr int kCols = NT / 2;                    // columns of a warpgroup
    static constexpr uint32_t kWeightBytes = NT / 2 * 128;  // of a CTA
    static constexpr int kStages = 5;
    static constexpr int kAcc = 2, kPlace = 256;            // accumulators, and columns between them
    static constexpr size_t kRing = kStages * (kTileBytes + kWeightBytes);
    static constexpr size_t kSmem = 1024 + kRing + kOutBytes + kScaleBytes + (2 * kStages + 2 * kAcc + 2 * kScaleRing + 1) * 8 + 16;
    static_assert(kSmem <= 227 * 1024, "one CTA to an SM");
};

// After a wait that gave up in the even CTA, and once neither copies any more: waits for the last fill of each stage.  Both CTAs'
// copies, `bytes` each, complete on the even one's barriers, which expect them together.  A stage that one of them filled once more
// than the other (no more than once: the fill behind it waits for a product of both halves) gets what is missing: the arrival and the
// bytes of the other's, or the other's bytes as if they had come.  Where the even CTA did not give up, its products waited for all.
template <int NS>
__device__ __forceinline__ void drain_pair(uint64_t *full, int even, int odd, uint32_t bytes, int *status) {
    for (int s = 0; s < NS; ++s) {
        const int a = (even + NS - 1 - s) / NS, b = (odd + NS - 1 - s) / NS, last = (a > b ? a : b) - 1;
        if (last < 0) continue;
        if (a < b) mbar_expect_tx(&full[s], bytes);
        if (a > b) mbar_complete_tx(&full[s], bytes);
        if (!fp8_wait(&full[s], last & 1, status)) fp8_wait(&full[s], last & 1, status, 8 * kFp8WaitNs);
    }
}

template <int NT>
__global__ void __launch_bounds__(kManyThreads, 1) __cluster_dims__(2, 1, 1)
    pair_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const MatmulParams p) {
    using F = Pair<NT>;
    constexpr int NS = F::kStages, NB = F::kAcc, COLS = F::kCols;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const sX = smem, *const sW = smem + NS * kTileBytes;
    float *const sOut = reinterpret_cast<float *>(smem + F::kRing);
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + F::kRing + kOutBytes + kScaleBytes);  // the even CTA's serve both
    uint64_t *const empty = full + NS, *const acc_full = empty + NS, *const acc_empty = acc_full + NB, *const done = acc_empty + NB;
    ScaleRing scales;
    scales.entries = reinterpret_cast<float *>(smem + F::kRing + kOutBytes);
    scales.full = done + 1;
    scales.empty = scales.full + kScaleRing;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(scales.empty + kScaleRing);
    int *const failed_slot = reinterpret_cast<int *>(tmem_slot + 1), *const fills_slot = failed_slot + 1, *const drain_slot = failed_slot + 2;

    if (p.force_timeout) {
        forced_timeout(done, p.status);
        return;
    }
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int pair = blockIdx.x >> 1, pairs = gridDim.x >> 1, rank = blockIdx.x & 1, n = p.KB;
    const int tiles = p.row_tiles * p.col_tiles;

    if (tid == 0) {
        *failed_slot = *drain_slot = 0;
        for (int s = 0; s < NS; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < NB; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 16);
        }
        scales.init();
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc_pair(tmem_slot, 512);
    tc_fence_before();
    cluster_sync();  // the other CTA's barriers are set up too
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_trigger();

    const int group = (warp >> 2) - 1, row = (warp & 3) * 32 + lane;
    if (group < 0) {
        registers_down<kFewRegs>();
        if (warp == 0 && lane == 0) {
            bool ok = true;
            int s = 0, turn = 0;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int rt, ct;
                tile_at(p, t, &rt, &ct);
                for (int i = 0; i < n; ++i) {
                    if (turn > 0 && !(ok = fp8_wait(&empty[s], (turn - 1) & 1, p.status))) break;
                    if (rank == 0) mbar_expect_tx(&full[s], 2 * (kTileBytes + F::kWeightBytes));
                    const uint32_t bar = peer_address(&full[s], 0);
                    tma_tile_pair(sX + s * kTileBytes, &tmX, i * kFp8Block, rt * 256 + rank * 128, bar);
                    tma_tile_pair(sW + s * F::kWeightBytes, &tmW, i * kFp8Block, ct * NT + rank * (NT / 2), bar);
                    if (++s == NS) s = 0, ++turn;
                }
            }
            *fills_slot = turn * NS + s;
            if (!ok) *failed_slot = 1;
        } else if (warp == 1 && rank == 0) {
            bool ok = true;
            int s = 0, ring = 0, b = 0, turn = 0;
            for (int t = pair; t < tiles && ok; t += pairs)
                for (int i = 0; i < n; ++i) {
                    ok = __all_sync(~0u, (turn == 0 || fp8_wait(&acc_empty[b], (turn - 1) & 1, p.status)) && fp8_wait(&full[s], ring, p.status));
                    if (!ok) break;
                    tc_fence_after();
                    umma_block_pair(tmem + b * F::kPlace, smem_u32(sX + s * kTileBytes), smem_u32(sW + s * F::kWeightBytes), idesc_e4m3_pair(NT));
                    umma_commit_pair(&empty[s]);
                    umma_commit_pair(&acc_full[b]);
                    if (++s == NS) s = 0, ring ^= 1;
                    if (++b == NB) b = 0, ++turn;
                }
            if (!ok && lane == 0) *failed_slot = 1;
            umma_commit_pair(done);
        }
        if (warp == 2) {
            bool ok = true;
            for (int t = pair; t < tiles && ok; t += pairs) {
                int rt, ct;
                tile_at(p, t, &rt, &ct);
                ok = scales.copy_tile(p, rt * 256 + rank * 128, (ct * NT) >> 7, 0, n, lane);
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
        // in both CTAs: the products are done, and what they signal has arrived
        if (warp == 1 && !fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else {
        registers_up<kManyRegs>();
        const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + group * COLS;
        float acc[COLS];
        bool ok = true, early = false;
        int b = 0, ring = 0;
        for (int t = pair; t < tiles && ok; t += pairs) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            const int tok = rt * 256 + rank * 128, m = tok + row, n0 = ct * NT + group * COLS, cut = (128 - (n0 & 127)) / 32;
#pragma unroll
            for (int j = 0; j < COLS; ++j) acc[j] = 0.f;
            prefetch_residual<COLS>(p, m, n0);
            // this warpgroup's first block of weight rows among the tile's two, and its second, if it has one
            const int w0 = (n0 >> 7) - ((ct * NT) >> 7), w1 = NT == 192 && w0 == 0 ? 1 : w0;
            for (int i = 0; i < n; ++i) {
                ok = early || __all_sync(~0u, fp8_wait(&scales.full[scales.e], scales.turn & 1, p.status) && fp8_wait(&acc_full[b], ring, p.status));
                if (!ok) break;
                tc_fence_after();
                const float *const sc = scales.entries + scales.e * kScaleEntry;
                const float x = sc[row], s0 = x * sc[128 + w0], s1 = NT == 192 ? x * sc[128 + w1] : s0;
                const int this_b = b, this_e = scales.e;
                scales.next();
                if (++b == NB) b = 0, ring ^= 1;
                bool next = false;
                add_block<COLS>(acc, my + this_b * F::kPlace, s0, s1, NT == 192 ? cut : COLS,
                                [&] { next = mbar_test(&scales.full[scales.e], scales.turn & 1) && mbar_test(&acc_full[b], ring); },
                                [&] {
                                    tc_fence_before();
                                    __syncwarp();
                                    if (lane == 0) {
                                        mbar_arrive_peer(peer_address(&acc_empty[this_b], 0));
                                        mbar_arrive(&scales.empty[this_e]);
                                    }
                                });
                early = __all_sync(~0u, next);
            }
            if (ok) store_tile<COLS>(p, tok + (warp & 3) * 32, n0, lane, acc, sOut + (warp - 4) * 32 * kOutPitch);
        }
        if (!ok && lane == 0) *failed_slot = 1;
    }
    __syncwarp();
    __syncthreads();
    if (rank == 0 && tid < 2 && *failed_slot) peer_store(drain_slot, tid, 1);
    tc_fence_before();
    cluster_sync();  // no CTA leaves while the other's products, commits or arrivals may reach it
    if (*drain_slot) {  // in both: copies may be on their way into either
        if (rank == 0 && tid == 0)
            drain_pair<NS>(full, *fills_slot, __float_as_int(peer_float(reinterpret_cast<const float *>(fills_slot), 1)), kTileBytes + F::kWeightBytes, p.status);
        cluster_sync();
    }
    if (warp == 1) tmem_free_pair(tmem, 512);
}

// ----------------------------------------------------------------------------- host

template <int NT>
cudaError_t launch_few(const MatmulParams &p, const void *x, const void *W, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(few_kernel<NT>, Few<NT>::kSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mw, mx;
    if (!byte_tile_map(&mw, W, p.N, p.K, 128) || !byte_tile_map(&mx, x, p.M, p.K, NT)) return cudaErrorInvalidValue;
    return launch_kernel_as(few_kernel<NT>, dim3((unsigned)((p.N + 127) / 128 * p.split)), dim3(kFewThreads), Few<NT>::kSmem, st,
                            p.split, false, mw, mx, p);
}

cudaError_t launch_many(MatmulParams p, const void *x, const void *W, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(many_kernel, Many::kSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mw, mx;
    if (!byte_tile_map(&mw, W, p.N, p.K, 128) || !byte_tile_map(&mx, x, p.M, p.K, 128)) return cudaErrorInvalidValue;
    p.row_tiles = (p.M + 127) / 128;
    p.col_tiles = (p.N + 127) / 128;
    const long tiles = (long)p.row_tiles * p.col_tiles, slots = sm_count();
    const long grid = p.split > 1 ? tiles * p.split : tiles < slots ? tiles : slots;
    return launch_kernel_as(many_kernel, dim3((unsigned)grid), dim3(kManyThreads), Many::kSmem, st, p.split, false, mx, mw, p);
}

template <int NT>
cudaError_t launch_pair(MatmulParams p, const void *x, const void *W, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(pair_kernel<NT>, Pair<NT>::kSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mw, mx;
    if (!byte_tile_map(&mw, W, p.N, p.K, NT / 2) || !byte_tile_map(&mx, x, p.M, p.K, 128)) return cudaErrorInvalidValue;
    p.row_tiles = (p.M + 255) / 256;
    p.col_tiles = (p.N + NT - 1) / NT;
    const long tiles = (long)p.row_tiles * p.col_tiles, slots = sm_count() / 2;
    return launch_kernel(pair_kernel<NT>, dim3((unsigned)(2 * (tiles < slots ? tiles : slots))), dim3(kManyThreads), Pair<NT>::kSmem, st, mx, mw, p);
}

// CTAs per cluster: as many as keep at least `least` blocks each and do not pass the CTAs that run at once.
int split_of(long tiles, int KB, int slots, int least) {
    int s = 1;
    while (s < 8 && tiles * s * 2 <= slots && KB / (s * 2) >= least) s *= 2;
    return s;
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" int fp8_matmul(int M, int N, int K, const uint8_t *x, const float *x_scale, const uint8_t *W, const float *w_scale,
                          const hla_bf16 *residual, void *y, int y_dtype, hla_stream stream) {
    HLA_REQUIRE(M >= 1 && N >= 1 && K >= 1 && x && x_scale && W && w_scale && y, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(y_dtype == HLA_F32 || y_dtype == HLA_BF16, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(K % 16 == 0 && M <= 1 << 30 && N <= 1 << 30 && K <= 1 << 30, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(aligned16(x) && aligned16(x_scale) && aligned16(W) && aligned16(w_scale) && aligned16(residual) && aligned16(y),
                HLA_ERR_MISALIGNED);
    MatmulParams p = {};
    p.M = M; p.N = N; p.K = K;
    p.KB = K / kFp8Block + (K % kFp8Block != 0);
    p.xs = x_scale; p.ws = w_scale; p.residual = residual; p.y = y; p.y_bf16 = y_dtype == HLA_BF16;
    p.status = device_status_word();
    HLA_REQUIRE(p.status, HLA_ERR_CUDA);
    p.force_timeout = wait_timeout_forced();
    const cudaStream_t st = (cudaStream_t)stream;
    const int sms = sm_count();
    cudaError_t ce;
    if (M <= 32) {
        const int nt = M <= 16 ? 16 : 32;
        p.split = split_of((N + 127) / 128, p.KB, 2 * sms, 2);
        set_variant("fp8_matmul<tokens%d,split%d>", nt, p.split);
        ce = nt == 16 ? launch_few<16>(p, x, W, st) : launch_few<32>(p, x, W, st);
    } else {
        p.direct = N % 16 == 0 && (reinterpret_cast<uintptr_t>(y) & 31) == 0;
        // The variant whose waves of tiles take the fewest cycles a block of K, measured at 512 to 8192 tokens: 600 for a CTA's
        // 128 x 128, 900 and 970 for a pair's 256 x 192 and 256 x 256 (512 tokens to 7168 of 4096: 24.2, 20.0, 22.3 us; 256 to 16416
        // of 7168: 38, 53, 34 us; 256 to 7168 of 4096: 14, 19, 21 us; 8192 to 16416 of 7168: 920, 877, 801 us).  Neither the tile's end nor
        // the cutting of K is counted.  Where stores decide, that costs up to 9%: 8192 to 16416 of K 128 84.7, 77.8, 84.7 us (the last is
        // taken), 256 to 16416 of K 256 7.0, 8.5, 7.4 (the last).  Few tiles of long K are cut by the 128 x 128 variant alone, which the
        // waves prefer there anyway: 256 to 2048 of 7168 11.2, 27.7, 31.2, 1000 to 2048 of 7168 20.4, 28.7, 32.5.
        const auto waves = [](long tiles, long slots) { return (tiles + slots - 1) / slots; };
        const long rows = (M + 127) / 128L, pairs = (M + 255) / 256L, one = rows * ((N + 127) / 128L);
        const long cost1 = 600 * waves(one, sms), cost192 = 900 * waves(pairs * ((N + 191) / 192L), sms / 2),
                   cost256 = 970 * waves(pairs * ((N + 255) / 256L), sms / 2);
        HLA_REQUIRE(one < 1L << 30, HLA_ERR_UNSUPPORTED);
        if (cost1 <= cost192 && cost1 <= cost256) {
            p.split = split_of(one, p.KB, sms, 4);
            set_variant("fp8_matmul<tile128x128,split%d>", p.split);
            ce = launch_many(p, x, W, st);
        } else {
            p.split = 1;
            set_variant("fp8_matmul<pair256x%d>", cost192 < cost256 ? 192 : 256);
            ce = cost192 < cost256 ? launch_pair<192>(p, x, W, st) : launch_pair<256>(p, x, W, st);
        }
    }
    return launched(ce);
}
