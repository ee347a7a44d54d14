// Matrix product of e4m3 matrices with a scale for each block of 128 along K:
//   y[m, n] = sum_b (x_scale[m, b] * w_scale[n / 128, b]) * sum_{k in b} x[m, k] W[n, k]  (+ residual[m, n]).
//
// Each block's product runs on tcgen05 (kind::f8f6f4, fp32 accumulator in tensor memory, overwritten by every block);
// warps of their own read it back and add it, scaled, to sums in registers, while the next block's product runs into another
// accumulator.  One warp copies tiles by TMA into a ring, one issues the products.
//
//  * Up to 64 tokens (`few_kernel`): bound by HBM, every weight byte is read once.  128 weight rows lie on the lanes and
//    16 to 64 tokens on the columns, so that a product of few tokens still fills the tensor core's rows.  K is cut among the
//    1 to 8 CTAs of a cluster, which add their sums through distributed shared memory in rank order: one launch, no
//    workspace, no atomics.
//  * More tokens (`many_kernel`): 128 tokens on the lanes, 128 or 256 weight rows on the columns.  A thread's row has one
//    token scale and its columns one weight scale per block, so scaling is one multiplication per block and one FMA per
//    value.
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
    int *status;
    int force_timeout;
};

__device__ __forceinline__ void store_y(const MatmulParams &p, size_t at, float v) {
    if (p.residual) v += bf16_bits_to_float(p.residual[at]);
    if (p.y_bf16) static_cast<uint16_t *>(p.y)[at] = float_to_bf16_bits(v);
    else static_cast<float *>(p.y)[at] = v;
}

// ----------------------------------------------------------------------------- up to 64 tokens

constexpr int kFewThreads = 192;       // copies, products, four warps of sums
constexpr int kScaleChunk = 32;        // blocks whose scales are in shared memory at once
constexpr uint32_t kTileBytes = 128 * 128;

template <int NT>
struct Few {
    static constexpr int kStages = NT == 16 ? 6 : NT == 32 ? 5 : 4;  // about 100 KB: two CTAs to an SM
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
    if (tid != 0) pdl_wait_trigger();  // the copying thread waits after its first weight tiles

    int issued = 0;
    float acc[NT];
    bool ok = true;
    if (warp == 0 && lane == 0) {
        const int pre = n < NS ? n : NS;
        for (int i = 0; i < pre; ++i) {
            mbar_expect_tx(&full[i], kTileBytes + F::kTokenBytes);
            tma_tile(sW + i * kTileBytes, &tmW, (c0 + i) * kFp8Block, rb * 128, &full[i]);
        }
        pdl_wait_trigger();
        for (int i = 0; i < pre; ++i) tma_tile(sX + i * F::kTokenBytes, &tmX, (c0 + i) * kFp8Block, 0, &full[i]);
        issued = pre;
        for (int i = pre; i < n; ++i) {
            const int s = i % NS;
            if (!fp8_wait(&empty[s], (i / NS - 1) & 1, p.status)) break;
            mbar_expect_tx(&full[s], kTileBytes + F::kTokenBytes);
            tma_tile(sW + s * kTileBytes, &tmW, (c0 + i) * kFp8Block, rb * 128, &full[s]);
            tma_tile(sX + s * F::kTokenBytes, &tmX, (c0 + i) * kFp8Block, 0, &full[s]);
            issued = i + 1;
        }
    } else if (warp == 1 && lane == 0) {
        int i = 0;
        for (; i < n; ++i) {
            const int s = i % NS, b = i % NB;
            if (i >= NB && !fp8_wait(&acc_empty[b], (i / NB - 1) & 1, p.status)) break;
            if (!fp8_wait(&full[s], (i / NS) & 1, p.status)) break;
            tc_fence_after();
            umma_block(tmem + b * NT, smem_u32(sW + s * kTileBytes), smem_u32(sX + s * F::kTokenBytes), idesc_e4m3(128, NT));
            umma_commit(&empty[s]);
            umma_commit(&acc_full[b]);
        }
        *consumed_slot = i;
        umma_commit(done);
        if (!fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else if (warp >= 2) {
        const int t = tid - 64, row = (warp & 3) * 32 + lane;  // a warp reads the quarter of the lanes of its number mod 4
        const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16);
#pragma unroll
        for (int j = 0; j < NT; ++j) acc[j] = 0.f;
        for (int i = 0; i < n; ++i) {  // to the end even after a wait that gave up: the four warps meet at each chunk
            if (i % kScaleChunk == 0) {  // x_scale * w_scale of the next blocks, a row of tokens per block
                named_sync(1, 128);
                const int m = n - i < kScaleChunk ? n - i : kScaleChunk;
                for (int e = t; e < NT * kScaleChunk; e += 128) {
                    const int tok = e / kScaleChunk, k = e % kScaleChunk;
                    if (tok < p.M && k < m)
                        sScale[k * NT + tok] = p.xs[(size_t)tok * p.KB + c0 + i + k] * p.ws[(size_t)rb * p.KB + c0 + i + k];
                }
                named_sync(1, 128);
            }
            const int b = i % NB;
            ok = __all_sync(~0u, ok && fp8_wait(&acc_full[b], (i / NB) & 1, p.status));
            if (!ok) continue;
            tc_fence_after();
            uint32_t v[NT];
            tmem_ld<NT>(my + b * NT, v);
            tmem_wait_ld();
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&acc_empty[b]);
            const float *const sc = sScale + (i % kScaleChunk) * NT;
#pragma unroll
            for (int j = 0; j < NT; j += 4) {
                const float4 f = *reinterpret_cast<const float4 *>(sc + j);
                acc[j] = fmaf(__uint_as_float(v[j]), f.x, acc[j]);
                acc[j + 1] = fmaf(__uint_as_float(v[j + 1]), f.y, acc[j + 1]);
                acc[j + 2] = fmaf(__uint_as_float(v[j + 2]), f.z, acc[j + 2]);
                acc[j + 3] = fmaf(__uint_as_float(v[j + 3]), f.w, acc[j + 3]);
            }
        }
        if (p.split == 1 && ok) {
            const int col = rb * 128 + row;
#pragma unroll
            for (int j = 0; j < NT; ++j)
                if (j < p.M && col < p.N) store_y(p, (size_t)j * p.N + col, acc[j]);
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0)  // fills that no product waited for (after a wait that gave up)
        for (int i = *consumed_slot; i < issued; ++i)
            if (!fp8_wait(&full[i % NS], (i / NS) & 1, p.status)) fp8_wait(&full[i % NS], (i / NS) & 1, p.status, 8 * kFp8WaitNs);
    __syncwarp();
    __syncthreads();
    if (p.split > 1) {  // the tiles are used up: their place takes the sums [token][weight row]
        float *const sums = reinterpret_cast<float *>(smem);
        if (warp >= 2) {
            const int row = (warp & 3) * 32 + lane;
#pragma unroll
            for (int j = 0; j < NT; ++j) sums[j * 128 + row] = acc[j];
        }
        cluster_sync();
        for (int e = rank * kFewThreads + tid; e < p.M * 128; e += p.split * kFewThreads) {
            const int m = e >> 7, col = rb * 128 + (e & 127);
            if (col >= p.N) continue;
            float v = 0.f;
            for (int r = 0; r < p.split; ++r) v += peer_float(sums + e, r);
            store_y(p, (size_t)m * p.N + col, v);
        }
        cluster_sync();  // no CTA leaves while another reads its sums
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, F::kColumns);
}

// ----------------------------------------------------------------------------- more tokens

constexpr int kManyThreads = 320;  // copies, products, eight warps of sums

template <int NT>
struct Many {
    static constexpr int kStages = NT == 256 ? 4 : 3;  // 192 KB, or 96 KB for two CTAs to an SM
    static constexpr int kCtas = NT == 256 ? 1 : 2;
    static constexpr uint32_t kWeightBytes = NT * 128;
    static constexpr int kHalf = NT / 2;               // columns per warp: two groups of four warps
    static constexpr int kPad = 33;
    static constexpr size_t kSums = 128 * (NT + 1) * 4;                  // of the join
    static constexpr size_t kRing = kStages * (kTileBytes + kWeightBytes);
    static constexpr size_t kOut = 8 * 16 * kPad * 4;                    // a warp's 16 rows x 32 columns on their way out
    static constexpr size_t kSmem = 1024 + kRing + kOut + (2 * kStages + 5) * 8 + 16;
    static_assert(kSums <= kRing, "the sums of the join take the place of the tiles");
};

// Tiles in bands of 16 row tiles, down a band's columns: the 152 or 304 tiles in flight share their operands in L2.
__device__ __forceinline__ void tile_at(const MatmulParams &p, int t, int *rt, int *ct) {
    constexpr int kBand = 16;
    const int band = t / (kBand * p.col_tiles), first = band * kBand;
    const int rows = p.row_tiles - first < kBand ? p.row_tiles - first : kBand;
    const int r = t - first * p.col_tiles;
    *ct = r / rows;
    *rt = first + r - *ct * rows;
}

template <int NT>
__global__ void __launch_bounds__(kManyThreads, Many<NT>::kCtas)
    many_kernel(const __grid_constant__ CUtensorMap tmX, const __grid_constant__ CUtensorMap tmW, const MatmulParams p) {
    using F = Many<NT>;
    constexpr int NS = F::kStages, NB = 2;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *const smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *const sX = smem, *const sW = smem + NS * kTileBytes;
    float *const sOut = reinterpret_cast<float *>(smem + F::kRing);
    uint64_t *const full = reinterpret_cast<uint64_t *>(smem + F::kRing + F::kOut);
    uint64_t *const empty = full + NS, *const acc_full = empty + NS, *const acc_empty = acc_full + NB, *const done = acc_empty + NB;
    uint32_t *const tmem_slot = reinterpret_cast<uint32_t *>(done + 1);
    int *const consumed_slot = reinterpret_cast<int *>(tmem_slot + 1);

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
        mbar_init(done, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 1) tmem_alloc(tmem_slot, NB * NT);
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = *tmem_slot;
    pdl_wait_trigger();

    long issued = 0;
    float acc[F::kHalf];
    bool ok = true;
    const int half = warp >= 6;                               // which half of the columns
    const int row = (warp & 3) * 32 + lane;                   // which token of the tile
    if (warp == 0 && lane == 0) {
        for (int t = unit; t < tiles && ok; t += units) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            for (int i = 0; i < n; ++i, ++issued) {
                const int s = (int)(issued % NS);
                if (issued >= NS && !(ok = fp8_wait(&empty[s], (uint32_t)(issued / NS - 1) & 1, p.status))) break;
                mbar_expect_tx(&full[s], kTileBytes + F::kWeightBytes);
                tma_tile(sX + s * kTileBytes, &tmX, (c0 + i) * kFp8Block, rt * 128, &full[s]);
                tma_tile(sW + s * F::kWeightBytes, &tmW, (c0 + i) * kFp8Block, ct * NT, &full[s]);
            }
        }
    } else if (warp == 1 && lane == 0) {
        long g = 0;
        for (int t = unit; t < tiles && ok; t += units)
            for (int i = 0; i < n; ++i, ++g) {
                const int s = (int)(g % NS), b = (int)(g % NB);
                if (g >= NB && !(ok = fp8_wait(&acc_empty[b], (uint32_t)(g / NB - 1) & 1, p.status))) break;
                if (!(ok = fp8_wait(&full[s], (uint32_t)(g / NS) & 1, p.status))) break;
                tc_fence_after();
                umma_block(tmem + b * NT, smem_u32(sX + s * kTileBytes), smem_u32(sW + s * F::kWeightBytes), idesc_e4m3(128, NT));
                umma_commit(&empty[s]);
                umma_commit(&acc_full[b]);
            }
        *consumed_slot = (int)(g % (2 * NS)) | (int)(ok ? 0 : 1 << 30);
        umma_commit(done);
        if (!fp8_wait(done, 0, p.status)) fp8_wait(done, 0, p.status, 8 * kFp8WaitNs);
    } else if (warp >= 2) {
        const uint32_t my = tmem + (static_cast<uint32_t>((warp & 3) * 32) << 16) + half * F::kHalf;
        long g = 0;
        for (int t = unit; t < tiles && ok; t += units) {
            int rt, ct;
            tile_at(p, t, &rt, &ct);
            const int m = rt * 128 + row;
            int wb = (ct * NT + half * F::kHalf) >> 7;
            const int last_wb = (p.N - 1) >> 7;
            if (wb > last_wb) wb = last_wb;  // columns behind the last: their values are not stored
            const float *const xs = p.xs + (size_t)(m < p.M ? m : p.M - 1) * p.KB + c0, *const ws = p.ws + (size_t)wb * p.KB + c0;
#pragma unroll
            for (int j = 0; j < F::kHalf; ++j) acc[j] = 0.f;
            float sx = xs[0], sw = ws[0];
            for (int i = 0; i < n; ++i, ++g) {
                const float sc = sx * sw;
                if (i + 1 < n) {  // the next block's scales are on their way during this one
                    sx = xs[i + 1];
                    sw = ws[i + 1];
                }
                const int b = (int)(g % NB);
                ok = __all_sync(~0u, fp8_wait(&acc_full[b], (uint32_t)(g / NB) & 1, p.status));
                if (!ok) break;
                tc_fence_after();
#pragma unroll
                for (int c = 0; c < F::kHalf; c += 32) {
                    uint32_t v[32];
                    tmem_ld<32>(my + b * NT + c, v);
                    tmem_wait_ld();
                    if (c + 32 == F::kHalf) {
                        tc_fence_before();
                        __syncwarp();
                        if (lane == 0) mbar_arrive(&acc_empty[b]);
                    }
#pragma unroll
                    for (int j = 0; j < 32; ++j) acc[c + j] = fmaf(__uint_as_float(v[j]), sc, acc[c + j]);
                }
            }
            if (!ok || p.split > 1) continue;
            // out through shared memory, 16 rows x 32 columns a warp at a time: a row's 32 columns leave together
            float *const out = sOut + (warp - 2) * 16 * F::kPad;
            const int n0 = ct * NT + half * F::kHalf;
#pragma unroll
            for (int c = 0; c < F::kHalf; c += 32)
#pragma unroll
                for (int h = 0; h < 2; ++h) {
                    __syncwarp();
                    if (lane >> 4 == h) {
#pragma unroll
                        for (int j = 0; j < 32; ++j) out[(lane & 15) * F::kPad + j] = acc[c + j];
                    }
                    __syncwarp();
                    const int col = n0 + c + lane;
                    if (col < p.N) {
#pragma unroll 4
                        for (int r = 0; r < 16; ++r) {
                            const int tok = rt * 128 + (warp & 3) * 32 + h * 16 + r;
                            if (tok < p.M) store_y(p, (size_t)tok * p.N + col, out[r * F::kPad + lane]);
                        }
                    }
                }
        }
    }
    __syncwarp();
    __syncthreads();
    if (tid == 0 && (*consumed_slot >> 30)) {
        // after a wait that gave up: at most one fill per stage is waited for by no product
        for (int s = 0; s < NS; ++s) {
            // the last fill of stage s, if any, has index (issued - 1) - ((issued - 1 - s) mod NS)
            if (issued <= s) continue;
            const long f = issued - 1 - (issued - 1 - s) % NS;
            if (!fp8_wait(&full[s], (uint32_t)(f / NS) & 1, p.status)) fp8_wait(&full[s], (uint32_t)(f / NS) & 1, p.status, 8 * kFp8WaitNs);
        }
    }
    __syncwarp();
    __syncthreads();
    if (p.split > 1) {
        // one tile per cluster; the tiles of the ring are used up: their place takes the sums [token][NT + 1]
        float *const sums = reinterpret_cast<float *>(smem);
        if (warp >= 2) {
#pragma unroll
            for (int j = 0; j < F::kHalf; ++j) sums[row * (NT + 1) + half * F::kHalf + j] = acc[j];
        }
        cluster_sync();
        int rt, ct;
        tile_at(p, unit, &rt, &ct);
        for (int e = rank * kManyThreads + tid; e < 128 * NT; e += p.split * kManyThreads) {
            const int r = e / NT, c = e - r * NT, tok = rt * 128 + r, col = ct * NT + c;
            if (tok >= p.M || col >= p.N) continue;
            float v = 0.f;
            for (int k = 0; k < p.split; ++k) v += peer_float(sums + r * (NT + 1) + c, k);
            store_y(p, (size_t)tok * p.N + col, v);
        }
        cluster_sync();
    }
    tc_fence_before();
    __syncthreads();
    if (warp == 1) tmem_free(tmem, NB * NT);
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

template <int NT>
cudaError_t launch_many(MatmulParams p, const void *x, const void *W, cudaStream_t st) {
    static bool done[64] = {};
    const cudaError_t e = allow_smem(many_kernel<NT>, Many<NT>::kSmem, done);
    if (e != cudaSuccess) return e;
    CUtensorMap mw, mx;
    if (!byte_tile_map(&mw, W, p.N, p.K, NT) || !byte_tile_map(&mx, x, p.M, p.K, 128)) return cudaErrorInvalidValue;
    p.row_tiles = (p.M + 127) / 128;
    p.col_tiles = (p.N + NT - 1) / NT;
    const long tiles = (long)p.row_tiles * p.col_tiles, slots = (long)Many<NT>::kCtas * sm_count();
    const long grid = p.split > 1 ? tiles * p.split : tiles < slots ? tiles : slots;
    return launch_kernel_as(many_kernel<NT>, dim3((unsigned)grid), dim3(kManyThreads), Many<NT>::kSmem, st, p.split, false, mx, mw, p);
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
    HLA_REQUIRE(K % 16 == 0, HLA_ERR_UNSUPPORTED);
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
    if (M <= 64) {
        const int nt = M <= 16 ? 16 : M <= 32 ? 32 : 64;
        p.split = split_of((N + 127) / 128, p.KB, 2 * sms, 2);
        set_variant("fp8_matmul<tokens%d,split%d>", nt, p.split);
        ce = nt == 16 ? launch_few<16>(p, x, W, st) : nt == 32 ? launch_few<32>(p, x, W, st) : launch_few<64>(p, x, W, st);
    } else {
        const long rows = (M + 127) / 128, wide = rows * ((N + 255) / 256);
        const bool use_wide = wide >= sms;
        p.split = use_wide ? 1 : split_of(rows * ((N + 127) / 128), p.KB, 2 * sms, 4);
        set_variant("fp8_matmul<tile128x%d,split%d>", use_wide ? 256 : 128, p.split);
        ce = use_wide ? launch_many<256>(p, x, W, st) : launch_many<128>(p, x, W, st);
    }
    return launched(ce);
}
