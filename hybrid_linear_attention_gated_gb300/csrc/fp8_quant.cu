// Conversion of bf16 or fp32 matrices to e4m3 with a power-of-two scale for each block of 128 values.
//
// q = e4m3(x / s), s = the smallest power of two with max|x| <= 448 s over the block: the division is exact, so the
// only rounding is the one to e4m3, and it falls the same way whatever precision computes it.
//
// Bound by HBM: 3 (5) bytes per bf16 (fp32) value.  A block of one row is 8 lanes of 16 values, each loaded as
// whole 32-byte sectors and stored as 16 bytes; the maximum is three shuffles.  A block of 128 rows is one CTA with its 64
// values a thread in registers between the maximum and the conversion, so either way x is read once.
#include "fp8.cuh"

namespace hla {
namespace {

constexpr int kQuantThreads = 256;

struct QuantParams {
    const void *x;
    uint8_t *q;
    float *scale;
    long M;
    int K, KB;
};

// 16 consecutive values as fp32; 32 bytes a load.
__device__ __forceinline__ void ld32b(const void *p, uint32_t (&r)[8]) {
    asm volatile("ld.global.v8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                 : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                 : "l"(p)
                 : "memory");
}

// Values stay packed as loaded (8 registers of bf16, 16 of fp32) until they are converted.
template <bool BF16>
struct Values {
    uint32_t w[BF16 ? 8 : 16];
    __device__ __forceinline__ void load(const void *x, size_t at) {
        if constexpr (BF16) {
            if ((reinterpret_cast<uintptr_t>(x) & 31) == 0 && (at & 15) == 0) {
                ld32b(static_cast<const uint16_t *>(x) + at, w);
            } else {
                const uint4 a = ld_act_v4(static_cast<const uint16_t *>(x) + at), b = ld_act_v4(static_cast<const uint16_t *>(x) + at + 8);
                w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w; w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 a = ld_act_v4(static_cast<const float *>(x) + at + 4 * i);
                w[4 * i] = a.x; w[4 * i + 1] = a.y; w[4 * i + 2] = a.z; w[4 * i + 3] = a.w;
            }
        }
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int i = 0; i < (BF16 ? 8 : 16); ++i) w[i] = 0;
    }
    __device__ __forceinline__ float at(int i) const {
        if constexpr (BF16) return i & 1 ? bf16_hi(w[i >> 1]) : bf16_lo(w[i >> 1]);
        else return __uint_as_float(w[i]);
    }
    // the largest magnitude: magnitudes order like their bits (two bf16 at a time), NaN above infinity
    __device__ __forceinline__ float top() const {
        uint32_t t = 0;
        if constexpr (BF16) {
#pragma unroll
            for (int i = 0; i < 8; ++i) asm("max.u16x2 %0, %0, %1;" : "+r"(t) : "r"(w[i] & 0x7FFF7FFFu));
            t = max(t << 16, t & 0xFFFF0000u);
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i) t = max(t, w[i] & 0x7FFFFFFFu);
        }
        return __uint_as_float(t);
    }
    __device__ __forceinline__ void store(uint8_t *q, float inv) const {
        uint32_t r[4];
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float v[4];
#pragma unroll
            for (int j = 0; j < 4; j += 2)
                asm("{\n .reg .b64 a, s;\n mov.b64 a, {%2, %3};\n mov.b64 s, {%4, %4};\n mul.rn.f32x2 a, a, s;\n mov.b64 {%0, %1}, a;\n}\n"
                    : "=f"(v[j]), "=f"(v[j + 1])
                    : "f"(at(4 * i + j)), "f"(at(4 * i + j + 1)), "f"(inv));
            r[i] = e4m3x4(v[0], v[1], v[2], v[3]);
        }
        *reinterpret_cast<uint4 *>(q) = make_uint4(r[0], r[1], r[2], r[3]);
    }
};

// One scale per row and 128 columns: each group of 8 lanes takes every (groups of the grid)th block.  One block in flight a
// group, 49 KB an SM: 8191 rows of 7168 at 28.6 us (6.2 TB/s), one row at 1.8 us; two, three and four blocks 31.2, 29.0 and
// 28.4 us, but 2.0 to 2.3 us for one row.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quant_rows_kernel(const QuantParams p) {
    pdl_wait_trigger();
    const int sub = threadIdx.x & 7;
    const long groups = (long)gridDim.x * (kQuantThreads / 8), blocks = p.M * p.KB;
    for (long b = (long)blockIdx.x * (kQuantThreads / 8) + (threadIdx.x >> 3); b - (threadIdx.x >> 3 & 3) < blocks;
         b += groups) {  // the four groups of a warp end together: the shuffles need all of it
        const long row = b < 1l << 31 ? (long)((uint32_t)b / (uint32_t)p.KB) : b / p.KB;
        const int col = (int)(b - row * p.KB) * kFp8Block + sub * 16;
        const bool live = b < blocks && col < p.K;
        const size_t at = (size_t)row * p.K + col;
        Values<BF16> v;
        if (live) v.load(p.x, at);
        else v.zero();
        float top = v.top();
#pragma unroll
        for (int m = 4; m; m >>= 1) top = max_magnitude(top, __shfl_xor_sync(~0u, top, m));
        const float s = fp8_scale_of(top);
        if (live) v.store(p.q + at, fp8_inverse(s));
        if (sub == 0 && b < blocks) p.scale[b] = s;
    }
}

// One scale per 128 rows and 128 columns: one CTA, 16 values of four rows a thread.
template <bool BF16>
__global__ void __launch_bounds__(kQuantThreads) quant_tiles_kernel(const QuantParams p) {
    __shared__ float s_top[kQuantThreads / 32];
    pdl_wait_trigger();
    const long rb = blockIdx.x / p.KB;
    const int kb = (int)(blockIdx.x - rb * p.KB);
    const int col = kb * kFp8Block + (threadIdx.x & 7) * 16;
    Values<BF16> v[4];
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long row = rb * 128 + i * 32 + (threadIdx.x >> 3);
        // the last row again behind it: without conditions the four are loaded together (16416 x 7168 fp32: 85.5 us, 83.3)
        v[i].load(p.x, (size_t)(row < p.M ? row : p.M - 1) * p.K + (col < p.K ? col : 0));
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        if (col >= p.K) v[i].zero();
#pragma unroll
    for (int i = 0; i < 4; ++i) top = max_magnitude(top, v[i].top());
#pragma unroll
    for (int m = 16; m; m >>= 1) top = max_magnitude(top, __shfl_xor_sync(~0u, top, m));
    if ((threadIdx.x & 31) == 0) s_top[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int i = 0; i < kQuantThreads / 32; ++i) top = max_magnitude(top, s_top[i]);
    const float s = fp8_scale_of(top), inv = fp8_inverse(s);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const long row = rb * 128 + i * 32 + (threadIdx.x >> 3);
        if (row < p.M && col < p.K) v[i].store(p.q + (size_t)row * p.K + col, inv);
    }
    if (threadIdx.x == 0) p.scale[blockIdx.x] = s;
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" int fp8_quantize(int M, int K, const void *x, int x_dtype, int rows_per_scale, uint8_t *q, float *scale,
                            hla_stream stream) {
    HLA_REQUIRE(M >= 1 && K >= 1 && x && q && scale, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(x_dtype == HLA_F32 || x_dtype == HLA_BF16, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(K % 16 == 0 && (rows_per_scale == 1 || rows_per_scale == 128), HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(aligned16(x) && aligned16(q) && aligned16(scale), HLA_ERR_MISALIGNED);
    QuantParams p;
    p.x = x; p.q = q; p.scale = scale; p.M = M; p.K = K;
    p.KB = K / kFp8Block + (K % kFp8Block != 0);
    const cudaStream_t st = (cudaStream_t)stream;
    const bool bf = x_dtype == HLA_BF16;
    set_variant("fp8_quantize<%s,rows%d>", bf ? "bf16" : "f32", rows_per_scale);
    if (rows_per_scale == 1) {
        constexpr int kPerCta = kQuantThreads / 8;
        const long ctas = ((long)M * p.KB + kPerCta - 1) / kPerCta, most = 8L * sm_count();
        const dim3 grid((unsigned)(ctas < most ? ctas : most));
        return launched(launch_kernel(bf ? quant_rows_kernel<true> : quant_rows_kernel<false>, grid, dim3(kQuantThreads), 0, st, p));
    }
    const long tiles = ((long)M + 127) / 128 * p.KB;
    HLA_REQUIRE(tiles < (1L << 31), HLA_ERR_UNSUPPORTED);
    return launched(launch_kernel(bf ? quant_tiles_kernel<true> : quant_tiles_kernel<false>, dim3((unsigned)tiles),
                                  dim3(kQuantThreads), 0, st, p));
}
