// What the kernels over e4m3 values with block scales share: conversion, tiles, instructions, launches.
//
// A block is 128 consecutive values along K (of one row of activations, or of 128 rows of a weight matrix) with one
// fp32 scale; the product of a block is exact in the tensor core's fp32 accumulator up to its own additions, and the
// scales are applied to it outside, in fp32.
#pragma once

#include <cuda.h>

#include "tcgen05.cuh"

namespace hla {

constexpr int kFp8Block = 128;                      // values per scale along K: one 128-byte swizzle atom
constexpr uint64_t kFp8WaitNs = 2000000000ull;      // 2 s of %globaltimer per bounded wait

// 2-D map over a row-major [rows, K] matrix of bytes, box = 128 columns x box_rows rows, 128-byte swizzle; what lies
// outside the matrix reads as zeros.
bool byte_tile_map(CUtensorMap *map, const void *base, uint64_t rows, uint64_t K, uint32_t box_rows);

// ----------------------------------------------------------------------------- conversion

// Bits of the smallest power of two 2^e, e >= -126, with 448 * 2^e >= top (448 = 1.75 * 2^8); NaN for NaN and infinities.
__device__ __forceinline__ float fp8_scale_of(float top) {
    const uint32_t b = __float_as_uint(top);
    const int e = static_cast<int>(b >> 23) - 8 + ((b & 0x7FFFFFu) > 0x600000u);
    if (b >= 0x7F800000u) return __uint_as_float(0x7FC00000u);
    return __uint_as_float(static_cast<uint32_t>(e < 1 ? 1 : e) << 23);
}

// 1 / 2^e for the normal powers of two that fp8_scale_of gives (2^-126 .. 2^120); NaN stays NaN.
__device__ __forceinline__ float fp8_inverse(float scale) {
    return scale == scale ? __uint_as_float(0x7F000000u - __float_as_uint(scale)) : scale;
}

// Two values as e4m3, to nearest even, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    uint16_t r;
    asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;" : "=h"(r) : "f"(hi), "f"(lo));
    return r;
}
__device__ __forceinline__ uint32_t e4m3x4(float a, float b, float c, float d) { return e4m3x2(a, b) | e4m3x2(c, d) << 16; }

// Larger magnitude, NaN if either is (fmaxf drops it): magnitudes order like their bits, NaN above infinity.
__device__ __forceinline__ float max_magnitude(float a, float b) {
    const uint32_t x = __float_as_uint(a) & 0x7FFFFFFFu, y = __float_as_uint(b) & 0x7FFFFFFFu;
    return __uint_as_float(x > y ? x : y);
}

// ----------------------------------------------------------------------------- tensor cores

// Instruction descriptor, kind::f8f6f4: fp32 accumulator, e4m3 A and B, both K-major.
__host__ __device__ constexpr uint32_t idesc_e4m3(int m, int n) {
    return (1u << 4) | (static_cast<uint32_t>(n >> 3) << 17) | (static_cast<uint32_t>(m >> 4) << 24);
}

// The issuing warp runs converged and one elected lane issues: the operands stay in uniform registers, where a lane that
// issues alone spends 90 cycles an instruction on moving them (128x128x32 takes 64).
__device__ __forceinline__ void umma_e4m3(uint32_t d_tmem, uint64_t a, uint64_t b, uint32_t idesc, uint32_t accumulate) {
    asm volatile(
        "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
        "l"(a), "l"(b), "r"(idesc), "r"(accumulate)
        : "memory");
}
__device__ __forceinline__ void umma_commit_elected(uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n" ::"r"(smem_u32(bar))
        : "memory");
}

// D = A x B^T over one block of 128 along K (four instructions of 32); the whole warp.
__device__ __forceinline__ void umma_block(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint32_t idesc) {
    const uint64_t da = sw128_desc(a_smem), db = sw128_desc(b_smem);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk) umma_e4m3(d_tmem, da + 2 * kk, db + 2 * kk, idesc, kk > 0);
}

__device__ __forceinline__ void tma_tile(void *dst, const CUtensorMap *map, int x, int y, uint64_t *bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(smem_u32(bar))
        : "memory");
}

// Counts `bytes` as copied that were expected and will not come.
__device__ __forceinline__ void mbar_complete_tx(uint64_t *bar, uint32_t bytes) {
    asm volatile("mbarrier.complete_tx.relaxed.cluster.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(bytes) : "memory");
}

__device__ __forceinline__ void mbar_arrive(uint64_t *bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// A bounded wait for the phase with the given parity; false (and the status word set) after `limit` ns of %globaltimer, which
// is read every 256 polls only: a read takes longer than most waits here, and the loop is small because every role has several.
__device__ __forceinline__ bool fp8_wait(uint64_t *bar, uint32_t parity, int *status, uint64_t limit = kFp8WaitNs) {
    const uint32_t a = smem_u32(bar);
    uint64_t began = 0;
#pragma unroll 1
    for (uint32_t i = 1;; ++i) {
        uint32_t done;
        asm volatile(
            "{\n .reg .pred p;\n mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
            : "=r"(done)
            : "r"(a), "r"(parity)
            : "memory");
        if (done) return true;
        if ((i & 255) == 0) {
            const uint64_t now = global_ns();
            if (began == 0) began = now;
            else if (now - began > limit) break;
        }
    }
    atomicExch(status, HLA_ERR_DEVICE_TIMEOUT);
    return false;
}

// After a wait that gave up: waits for the last fill of each stage of a ring of NS, which no product may have waited for.  `issued`
// counts the fills, up to multiples of 2 NS.
template <int NS>
__device__ __forceinline__ void drain_fills(uint64_t *full, int issued, int *status) {
    for (int s = 0; s < NS; ++s) {
        if (issued <= s) continue;
        const int f = issued - 1 - (issued - 1 - s) % NS;
        if (!fp8_wait(&full[s], f / NS & 1, status)) fp8_wait(&full[s], f / NS & 1, status, 8 * kFp8WaitNs);
    }
}

// Whether the phase has completed, without waiting.
__device__ __forceinline__ bool mbar_test(uint64_t *bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n .reg .pred p;\n mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done)
        : "r"(smem_u32(bar)), "r"(parity)
        : "memory");
    return done != 0;
}

// COLS consecutive 32-bit tensor-memory columns of this thread's lane; tmem_wait(v) before v is used: the values pass
// through the wait, so that nothing which uses them moves ahead of it.
template <int COLS>
__device__ __forceinline__ void tmem_ld(uint32_t taddr, uint32_t (&v)[COLS]) {
    static_assert(COLS == 8 || COLS == 16 || COLS == 32, "columns per load");
    if constexpr (COLS == 8) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7])
                     : "r"(taddr));
    } else if constexpr (COLS == 16) {
        asm volatile(
            "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15}, [%16];"
            : "=r"(v[0]), "=r"(v[1]), "=r"(v[2]), "=r"(v[3]), "=r"(v[4]), "=r"(v[5]), "=r"(v[6]), "=r"(v[7]), "=r"(v[8]),
              "=r"(v[9]), "=r"(v[10]), "=r"(v[11]), "=r"(v[12]), "=r"(v[13]), "=r"(v[14]), "=r"(v[15])
            : "r"(taddr));
    } else {
        tmem_ld32(taddr, v);
    }
}
template <int COLS>
__device__ __forceinline__ void tmem_wait(uint32_t (&v)[COLS]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;" : "+r"(v[0]), "+r"(v[1]), "+r"(v[2]), "+r"(v[3]), "+r"(v[4]), "+r"(v[5]), "+r"(v[6]), "+r"(v[7])::"memory");
#pragma unroll
    for (int c = 8; c < COLS; c += 8)
        asm volatile("" : "+r"(v[c]), "+r"(v[c + 1]), "+r"(v[c + 2]), "+r"(v[c + 3]), "+r"(v[c + 4]), "+r"(v[c + 5]), "+r"(v[c + 6]), "+r"(v[c + 7])::"memory");
}

// (a0, a1) += (v0, v1) * (s0, s1), each rounded once: one packed instruction.
__device__ __forceinline__ void fma2(float &a0, float &a1, uint32_t v0, uint32_t v1, float s0, float s1) {
    asm("{\n .reg .b64 a, v, s;\n mov.b64 a, {%0, %1};\n mov.b64 v, {%2, %3};\n mov.b64 s, {%4, %5};\n"
        " fma.rn.f32x2 a, v, s, a;\n mov.b64 {%0, %1}, a;\n}\n"
        : "+f"(a0), "+f"(a1)
        : "r"(v0), "r"(v1), "f"(s0), "f"(s1));
}

// Allocate / free `columns` (a power of two from 32) of tensor memory; one whole warp.
__device__ __forceinline__ void tmem_alloc(uint32_t *slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free(uint32_t taddr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
}

// ---- pairs of CTAs (cta_group::2): the even CTA of a cluster issues products of 256 rows, whose operands and accumulator lie
// half in each CTA's shared and tensor memory, at the same places
__host__ __device__ constexpr uint32_t idesc_e4m3_pair(int n) { return idesc_e4m3(256, n); }
__device__ __forceinline__ void umma_block_pair(uint32_t d_tmem, uint32_t a_smem, uint32_t b_smem, uint32_t idesc) {
    const uint64_t da = sw128_desc(a_smem), db = sw128_desc(b_smem);
#pragma unroll
    for (int kk = 0; kk < 4; ++kk)
        asm volatile(
            "{\n .reg .pred p, q;\n setp.ne.b32 p, %4, 0;\n elect.sync _|q, 0xffffffff;\n"
            " @q tcgen05.mma.cta_group::2.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n" ::"r"(d_tmem),
            "l"(da + 2 * kk), "l"(db + 2 * kk), "r"(idesc), "r"(static_cast<uint32_t>(kk > 0))
            : "memory");
}
// Arrives at the barrier at this place in both CTAs once the products issued so far are done.
__device__ __forceinline__ void umma_commit_pair(uint64_t *bar) {
    asm volatile(
        "{\n .reg .pred q;\n elect.sync _|q, 0xffffffff;\n"
        " @q tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;\n}\n" ::"r"(
            smem_u32(bar)),
        "h"(static_cast<uint16_t>(3))
        : "memory");
}
__device__ __forceinline__ uint32_t peer_address(const void *p, uint32_t rank) {
    uint32_t a;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    return a;
}
// A copy into this CTA's shared memory that completes on a barrier of the pair's even CTA.
__device__ __forceinline__ void tma_tile_pair(void *dst, const CUtensorMap *map, int x, int y, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile.mbarrier::complete_tx::bytes.cta_group::2 [%0], [%1, {%2, %3}], [%4];" ::"r"(
            smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(x), "r"(y), "r"(bar)
        : "memory");
}
__device__ __forceinline__ void mbar_arrive_peer(uint32_t bar) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" ::"r"(bar) : "memory");
}
__device__ __forceinline__ void tmem_alloc_pair(uint32_t *slot, uint32_t columns) {
    asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(slot)), "r"(columns) : "memory");
    asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
}
__device__ __forceinline__ void tmem_free_pair(uint32_t taddr, uint32_t columns) {
    asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(taddr), "r"(columns) : "memory");
}

__device__ __forceinline__ void cluster_sync() {
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release.aligned;\n barrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void peer_store(int *p, uint32_t rank, int v) {
    asm volatile("st.shared::cluster.s32 [%0], %1;" ::"r"(peer_address(p, rank)), "r"(v) : "memory");
}
__device__ __forceinline__ float peer_float(const float *p, uint32_t rank) {
    uint32_t a;
    float v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(a));
    return v;
}
__device__ __forceinline__ float4 peer_float4(const float *p, uint32_t rank) {
    uint32_t a;
    float4 v;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(a) : "r"(smem_u32(p)), "r"(rank));
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(a));
    return v;
}
// The register share of a warpgroup (all four of its warps); a block's shares add up to what it was launched with.
template <int N>
__device__ __forceinline__ void registers_down() { asm volatile("setmaxnreg.dec.sync.aligned.u32 %0;" ::"n"(N)); }
template <int N>
__device__ __forceinline__ void registers_up() { asm volatile("setmaxnreg.inc.sync.aligned.u32 %0;" ::"n"(N)); }
// A barrier among `threads` threads of the block (whole warps).
__device__ __forceinline__ void named_sync(int id, int threads) {
    asm volatile("bar.sync %0, %1;" ::"r"(id), "r"(threads) : "memory");
}

// The CTAs whose bounded waits are made to give up (hla_test_force_wait_timeout): CTA 0 waits for a barrier at which
// nothing arrives, and every CTA returns before it allocates, copies or multiplies.
__device__ __forceinline__ void forced_timeout(uint64_t *bar, int *status) {
    if (blockIdx.x == 0 && threadIdx.x == 0) {
        mbar_init(bar, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fp8_wait(bar, 0, status, 1000000ull);
        asm volatile("mbarrier.inval.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
    }
}

// ----------------------------------------------------------------------------- launches

// Raises a kernel's shared-memory limit once on every device used (`done` belongs to the kernel).
template <typename K>
inline cudaError_t allow_smem(K kernel, size_t bytes, bool (&done)[64]) {
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 64 && done[dev]) return cudaSuccess;
    e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)bytes);
    if (e == cudaSuccess && dev < 64) done[dev] = true;
    return e;
}

// As launch_kernel, in clusters of `cluster` blocks, or as a cooperative launch.
template <typename... KArgs, typename... Args>
inline cudaError_t launch_kernel_as(void (*kernel)(KArgs...), dim3 grid, dim3 block, size_t smem, cudaStream_t st,
                                    int cluster, bool cooperative, Args... args) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = block;
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[3];
    int n = 0;
    if (pdl_for(st)) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n++].val.programmaticStreamSerializationAllowed = 1;
    }
    if (cluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = cluster;
        attr[n].val.clusterDim.y = 1;
        attr[n++].val.clusterDim.z = 1;
    }
    if (cooperative) {
        attr[n].id = cudaLaunchAttributeCooperative;
        attr[n++].val.cooperative = 1;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, static_cast<KArgs>(args)...);
    if (e == cudaSuccess) pdl_launched(st);
    return e;
}

}  // namespace hla
