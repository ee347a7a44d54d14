// What the paged-cache kernels share: the checks of a cache descriptor, page lookup, the 8-bit
// conversions and the tensor-core fragments of swizzled shared-memory rows.
#pragma once

#include <cuda_fp16.h>

#include "common.cuh"

namespace hla {

constexpr int kMaxBatch = 1024;         // sequences per call (their length prefix sums sit in shared memory)
constexpr int kMaxWindowTokens = 8;     // tokens per sequence, as the KDA speculative window
constexpr int kMaxKvHeads = 256;

// ----------------------------------------------------------------------------- host side

// log2 of a supported page size (16, 32, 64, 128), or -1
inline int page_shift(int page_size) {
    for (int s = 4; s <= 7; ++s)
        if (page_size == 1 << s) return s;
    return -1;
}

// Checks of the descriptor alone; need_kv / need_bounds say which of its tensors the call uses.
inline int check_cache(const hla_kv_cache *C, bool need_kv, bool need_bounds) {
    HLA_REQUIRE(C, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(C->n_pages >= 1 && C->kv_heads >= 1 && C->page_size >= 1 && C->head_dim >= 1, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(C->dtype == HLA_BF16 || C->dtype == HLA_E4M3, C->dtype == HLA_F32 ? HLA_ERR_UNSUPPORTED : HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(C->head_dim == 64 || C->head_dim == 128, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(page_shift(C->page_size) >= 0 && C->kv_heads <= kMaxKvHeads, HLA_ERR_UNSUPPORTED);
    if (need_kv) {
        HLA_REQUIRE(C->k && C->v, HLA_ERR_INVALID_ARG);
        HLA_REQUIRE(aligned16(C->k) && aligned16(C->v), HLA_ERR_MISALIGNED);
        if (C->dtype == HLA_E4M3) {
            HLA_REQUIRE(C->k_scale && C->v_scale, HLA_ERR_INVALID_ARG);
            HLA_REQUIRE(aligned16(C->k_scale) && aligned16(C->v_scale), HLA_ERR_MISALIGNED);
        }
    }
    HLA_REQUIRE((C->k_min != nullptr) == (C->k_max != nullptr), HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(!need_bounds || C->k_min, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(aligned16(C->k_min) && aligned16(C->k_max), HLA_ERR_MISALIGNED);
    return HLA_OK;
}

// Sizes of the calls that read the cache for T new tokens of B sequences.
inline int check_window(const hla_kv_cache *C, int B, int T, int H, int max_blocks) {
    HLA_REQUIRE(B >= 1 && T >= 1 && H >= 1 && max_blocks >= 1, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(H % C->kv_heads == 0, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(B <= kMaxBatch && T <= kMaxWindowTokens && H <= 1024, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE((long)max_blocks * C->page_size < (1L << 30), HLA_ERR_UNSUPPORTED);
    return HLA_OK;
}

// ----------------------------------------------------------------------------- device side

// x / d for x d < 2^31 by a multiplication: a few instructions, where a short kernel pays for each one's fetch.
__host__ __device__ constexpr uint32_t divisor(int d) { return (uint32_t)(((1ull << 31) + d - 1) / d); }
__device__ __forceinline__ int divided(int x, uint32_t by) { return (int)__umulhi(2u * (uint32_t)x, by); }

__device__ __forceinline__ uint32_t min2(uint32_t a, uint32_t b) {  // of two bf16, NaN kept
    const __nv_bfloat162 r = __hmin2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}
__device__ __forceinline__ uint32_t max2(uint32_t a, uint32_t b) {
    const __nv_bfloat162 r = __hmax2_nan(*reinterpret_cast<const __nv_bfloat162 *>(&a), *reinterpret_cast<const __nv_bfloat162 *>(&b));
    return *reinterpret_cast<const uint32_t *>(&r);
}

// Inclusive prefix sums over a warp's lanes.
__device__ __forceinline__ int warp_prefix(int x, int lane) {
#pragma unroll
    for (int m = 1; m < 32; m <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, x, m);
        if (lane >= m) x += y;
    }
    return x;
}
// Turns the counts pre[1..n] that the block's threads have just written into prefix sums pre[0..n].  A lane of the first
// warp sums an odd number of neighbours (different banks across the lanes).  The caller's block barrier ends it.
__device__ __forceinline__ void block_prefix(int *pre, int n) {
    __syncthreads();
    if (threadIdx.x < 32) {
        const int each = ((n + 31) / 32) | 1, first = threadIdx.x * each, last = first + each < n ? first + each : n;
        int sum = 0;
        for (int b = first; b < last; ++b) sum += pre[b + 1];
        sum = warp_prefix(sum, threadIdx.x) - sum;
        for (int b = first; b < last; ++b) pre[b + 1] = sum += pre[b + 1];
        if (threadIdx.x == 0) pre[0] = 0;
    }
}

// Four e4m3 values as fp16 (exact): bytes 0, 1 in lo and 2, 3 in hi.
__device__ __forceinline__ void e4m3x4_to_f16x4(uint32_t four, uint32_t &lo, uint32_t &hi) {
    asm("{\n .reg .b16 a, b;\n mov.b32 {a, b}, %2;\n cvt.rn.f16x2.e4m3x2 %0, a;\n cvt.rn.f16x2.e4m3x2 %1, b;\n}\n"
        : "=r"(lo), "=r"(hi)
        : "r"(four));
}
// Two fp32 values as e4m3, rounded to nearest even and saturated at +-448 (NaN stays NaN); lo in the low byte.
__device__ __forceinline__ uint32_t f32x2_to_e4m3x2(float lo, float hi) {
    uint32_t r;
    asm("{\n .reg .b16 t;\n cvt.rn.satfinite.e4m3x2.f32 t, %1, %2;\n cvt.u32.u16 %0, t;\n}\n" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

__device__ __forceinline__ void ldmatrix_x4(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}
__device__ __forceinline__ void ldmatrix_x4_trans(uint32_t (&r)[4], uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0,%1,%2,%3}, [%4];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                 : "r"(addr)
                 : "memory");
}

// A 16x16 matrix of bytes, transposed: lane l (0-15) gives the address of row l; lane (i, j) = (l / 4, l % 4) gets rows
// 4 j .. 4 j + 3 of column i in a and of column i + 8 in b.
__device__ __forceinline__ void ldmatrix_trans8(uint32_t &a, uint32_t &b, uint32_t addr) {
    asm volatile("ldmatrix.sync.aligned.m16n16.x1.trans.shared.b8 {%0,%1}, [%2];" : "=r"(a), "=r"(b) : "r"(addr) : "memory");
}

// D(16x8 fp32) += A(16x16 fp16, row) * B(16x8 fp16, col)
__device__ __forceinline__ void mma_f16_16816(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
        "{%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, {%0,%1,%2,%3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// 16 bytes into shared memory, or 16 zero bytes where `on` is false (src is not read then, but is a valid address)
__device__ __forceinline__ void cp_async16_or_zero(uint32_t dst, const void *src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}

// 16 bytes from global into shared memory through L2
__device__ __forceinline__ void cp_async16_s(uint32_t dst, const void *src) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(dst), "l"(src) : "memory");
}

// Byte offset of 16-byte chunk c of row r in rows of RB bytes (64, 128 or 256), the chunks of a row permuted so
// that eight rows read at one chunk index fall into different banks, both rows 0-7 (or 8-15) of a group and the
// rows 0, 1, 8, 9, 2, 3, 10, 11 (4, 5, 12, 13, ...) that an 8-bit transposed read takes together.
template <int RB>
__device__ __forceinline__ uint32_t swizzled(int r, int c) {
    constexpr int CPR = RB / 16;
    const int y = r ^ ((r >> 1) & 4);
    const int x = CPR >= 8 ? (y & 7) : ((y >> 1) & (CPR - 1));
    return (uint32_t)(r * RB + ((c ^ x) << 4));
}

__device__ __forceinline__ float ex2(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

}  // namespace hla
