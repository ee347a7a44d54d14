// Choice of the cache blocks that a query attends to, by bounds on their keys.
//
// A block is one page.  Its bounds are the per-channel minimum and maximum of its keys, and
//     s_j = max over the G heads of a kv head of  sum_d max(q_d, 0) kmax_jd + min(q_d, 0) kmin_jd
// is an upper bound on every q.k of block j.  The highest n blocks are wanted, ties to the lower index, and
// exactly: two blocks at the border may differ by less than fp32 sums hold.
//
// attn_score_kernel computes all scores on mma.sync (bf16 products are exact in fp32; the sums are not) and is
// bound by reading the bounds, 4 d bytes per block.  attn_choose_kernel then needs only fp32's word on most
// blocks: with e a bound on the error of any score and t the n-th highest fp32 score, blocks above t + 2 e are
// in and blocks below t - 2 e are out; the few between are scored again in fp64 and ranked.
#include "paged.cuh"

namespace hla {
namespace {

constexpr int kScoreBlocks = 64;      // blocks scored per CTA
constexpr int kScoreThreads = 128;
constexpr int kChooseThreads = 256;
constexpr int kMaxBlocks = 65536;     // blocks per sequence (a bit each in shared memory)
constexpr int kStaged = 6144;         // scores of a row kept in shared memory; longer rows are read through L2
constexpr int kListed = 1024;         // blocks near the border kept in shared memory

struct SelectParams {
    const uint16_t *q, *k_min, *k_max;
    const int32_t *table, *past;
    int32_t *sel;
    float *score;                 // [B, T, Hkv, stride]
    unsigned long long *exact;    // [B, T, Hkv, stride]: fp64 scores of the blocks near the border, when too many to list
    float *absmax;                // [B, Hkv, chunks]
    int B, T, H, Hkv, G, d;
    int max_blocks, n_pages, pshift;
    int n_select, n_first, n_last;
    int stride, chunks;
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

// Scores of 64 blocks of one (sequence, kv head) for all T x G queries.  Warp w scores blocks 16 w .. 16 w + 15;
// the rows go in tiles of 16 that hold whole groups of G heads (or a part of one group, for G > 16).
template <int D>
__global__ void __launch_bounds__(kScoreThreads) attn_score_kernel(const SelectParams p) {
    constexpr int RB = 2 * D, CPR = RB / 16, KS = D / 16;
    __shared__ __align__(128) uint8_t s_max[kScoreBlocks * RB], s_min[kScoreBlocks * RB];
    __shared__ float s_tile[4][16][17];
    __shared__ uint32_t s_abs[4];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, i = lane >> 2, j = lane & 3;
    pdl_wait_trigger();
    const int chunk = blockIdx.x, b = blockIdx.y / p.Hkv, hk = blockIdx.y % p.Hkv;
    const int nb = visible_blocks(p, b, p.T - 1), j0 = chunk * kScoreBlocks + warp * 16;
    if (chunk * kScoreBlocks >= nb) return;

    // bounds of this warp's 16 blocks: lane l looks up block l, then rows are copied chunk by chunk
    const int blk = j0 + (lane & 15);
    int pg = blk < nb ? p.table[(size_t)b * p.max_blocks + blk] : -1;
    if (pg >= p.n_pages) pg = -1;
    const uint32_t bmax = smem_u32(s_max) + warp * 16 * RB, bmin = smem_u32(s_min) + warp * 16 * RB;
#pragma unroll
    for (int x = 0; x < 16 * CPR / 32; ++x) {
        const int r = (x * 32 + lane) / CPR, c = (x * 32 + lane) % CPR;
        const int rp = __shfl_sync(0xffffffffu, pg, r);
        const size_t o = rp >= 0 ? ((size_t)rp * p.Hkv + hk) * D + c * 8 : 0;
        cp_async16_or_zero(bmax + swizzled<RB>(r, c), p.k_max + o, rp >= 0);
        cp_async16_or_zero(bmin + swizzled<RB>(r, c), p.k_min + o, rp >= 0);
    }
    cp_async_commit();
    cp_async_wait<0>();
    __syncwarp();

    // largest magnitude among the bounds, as the bits of a bf16 (a NaN's are the largest)
    uint32_t big = 0;
#pragma unroll
    for (int x = 0; x < 16 * CPR / 32; ++x) {
        const uint4 u = reinterpret_cast<const uint4 *>(s_max + warp * 16 * RB)[x * 32 + lane],
                    w = reinterpret_cast<const uint4 *>(s_min + warp * 16 * RB)[x * 32 + lane];
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(u.x & 0x7fff7fffu, u.y & 0x7fff7fffu), __vmaxu2(u.z & 0x7fff7fffu, u.w & 0x7fff7fffu)));
        big = __vmaxu2(big, __vmaxu2(__vmaxu2(w.x & 0x7fff7fffu, w.y & 0x7fff7fffu), __vmaxu2(w.z & 0x7fff7fffu, w.w & 0x7fff7fffu)));
    }
    big = big >> 16 > (big & 0xffffu) ? big >> 16 : big & 0xffffu;
    big = __reduce_max_sync(0xffffffffu, big);
    if (lane == 0) s_abs[warp] = big;
    __syncthreads();
    if (tid == 0) {
        uint32_t m = s_abs[0];
        for (int w = 1; w < 4; ++w) m = s_abs[w] > m ? s_abs[w] : m;
        p.absmax[((size_t)b * p.Hkv + hk) * p.chunks + chunk] = bf16_bits_to_float((uint16_t)m);
    }

    const int per = p.G <= 16 ? 16 / p.G : 1;     // tokens per row tile
    const int parts = (p.G + 15) / 16;            // row tiles per token
    for (int t0 = 0; t0 < p.T; t0 += per) {
        float best = 0.f;                         // of (token t0 + y / 16, block y % 16) for outputs y of this lane
        float keep[8];
#pragma unroll
        for (int y = 0; y < 8; ++y) keep[y] = -INFINITY;
        for (int part = 0; part < parts; ++part) {
            float s[2][4] = {};
            const uint16_t *src[2];
            bool on[2];
#pragma unroll
            for (int hrow = 0; hrow < 2; ++hrow) {
                const int r = i + 8 * hrow;
                const int t = t0 + (parts == 1 ? r / p.G : 0), g = parts == 1 ? r % p.G : part * 16 + r;
                on[hrow] = t < p.T && g < p.G && (parts > 1 || r < per * p.G);
                src[hrow] = p.q + (on[hrow] ? ((size_t)(b * p.T + t) * p.H + hk * p.G + g) * D : 0);
            }
#pragma unroll
            for (int c = 0; c < KS; ++c) {
                uint32_t a[4], f[4], g[4];
#pragma unroll
                for (int hrow = 0; hrow < 2; ++hrow) {
                    a[hrow] = on[hrow] ? *reinterpret_cast<const uint32_t *>(src[hrow] + 16 * c + 2 * j) : 0u;
                    a[2 + hrow] = on[hrow] ? *reinterpret_cast<const uint32_t *>(src[hrow] + 16 * c + 8 + 2 * j) : 0u;
                }
                const uint32_t at = swizzled<RB>((lane & 7) + ((lane >> 4) << 3), 2 * c + ((lane >> 3) & 1));
                ldmatrix_x4(f, bmax + at);
                ldmatrix_x4(g, bmin + at);
#pragma unroll
                for (int x = 0; x < 2; ++x) {
                    mma_bf16_16816(s[x], relu2(a[0]), relu2(a[1]), relu2(a[2]), relu2(a[3]), f[2 * x], f[2 * x + 1]);
                    mma_bf16_16816(s[x], neg2(a[0]), neg2(a[1]), neg2(a[2]), neg2(a[3]), g[2 * x], g[2 * x + 1]);
                }
            }
            __syncwarp();
#pragma unroll
            for (int x = 0; x < 2; ++x)
#pragma unroll
                for (int e = 0; e < 4; ++e) s_tile[warp][i + 8 * (e >> 1)][8 * x + 2 * j + (e & 1)] = s[x][e];
            __syncwarp();
            // maximum over the heads (a NaN stays)
            const int rows = parts == 1 ? p.G : (p.G - part * 16 < 16 ? p.G - part * 16 : 16);
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                const int o = y * 32 + lane, tl = o >> 4, bl = o & 15;
                if (tl >= per) break;
                best = keep[y];
                for (int g = 0; g < rows; ++g) {
                    const float v = s_tile[warp][(parts == 1 ? tl * p.G : 0) + g][bl];
                    best = v > best || v != v ? v : best;
                }
                keep[y] = best;
            }
        }
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const int o = y * 32 + lane, tl = o >> 4, bl = o & 15, t = t0 + tl;
            const bool has = __shfl_sync(0xffffffffu, pg, bl) >= 0;
            if (tl < per && t < p.T && j0 + bl < nb)
                p.score[((size_t)(b * p.T + t) * p.Hkv + hk) * p.stride + j0 + bl] = has ? keep[y] : -INFINITY;
        }
    }
}

// Unsigned integers in the order of the values (-0 and +0 alike, NaN above all; never 0).
__device__ __forceinline__ uint32_t ordered(float x) {
    if (x != x) return 0xffffffffu;
    const uint32_t u = __float_as_uint(x + 0.f);
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ float unordered(uint32_t k) {
    return __uint_as_float(k & 0x80000000u ? k & 0x7fffffffu : ~k);
}
__device__ __forceinline__ unsigned long long ordered(double x) {
    if (x != x) return ~0ull;
    const unsigned long long u = (unsigned long long)__double_as_longlong(x + 0.0);
    return u >> 63 ? ~u : u | 1ull << 63;
}

__device__ __forceinline__ int block_sum(int x, int *s_red) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    x = __reduce_add_sync(0xffffffffu, x);
    __syncthreads();
    if (lane == 0) s_red[warp] = x;
    __syncthreads();
    int all = 0;
#pragma unroll
    for (int w = 0; w < kChooseThreads / 32; ++w) all += s_red[w];
    return all;
}

// One CTA per (sequence, token, kv head).
__global__ void __launch_bounds__(kChooseThreads) attn_choose_kernel(const SelectParams p) {
    __shared__ float s_score[kStaged];
    __shared__ uint32_t s_bits[kMaxBlocks / 32];       // the choice
    __shared__ unsigned long long s_key[kListed];
    __shared__ int s_blk[kListed];
    __shared__ int s_red[kChooseThreads / 32];
    __shared__ uint32_t s_lo, s_hi;
    __shared__ float s_f[2][kChooseThreads / 32];
    __shared__ int s_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int NW = kChooseThreads / 32;
    pdl_wait_trigger();
    const int row = blockIdx.x, hk = row % p.Hkv, t = row / p.Hkv % p.T, b = row / p.Hkv / p.T;
    int32_t *sel = p.sel + (size_t)row * p.n_select;
    const int nb = visible_blocks(p, b, t);
    if (nb <= p.n_select) {
        for (int x = tid; x < p.n_select; x += kChooseThreads) sel[x] = x < nb ? x : -1;
        return;
    }
    // the first and last blocks are in; k of those between, [e0, e1), are to be chosen
    const int e0 = p.n_first, e1 = nb - p.n_last, k = p.n_select - p.n_first - p.n_last;
    const int words = (nb + 31) >> 5;
    const float *row_score = p.score + (size_t)row * p.stride;
    const bool staged = nb <= kStaged;
    uint32_t lo = ~0u, hi = 0;
    for (int x = tid; x < nb; x += kChooseThreads) {
        const float v = row_score[x];
        if (staged) s_score[x] = v;
        if (x >= e0 && x < e1) {
            const uint32_t o = ordered(v);
            lo = o < lo ? o : lo;
            hi = o > hi ? o : hi;
        }
    }
    for (int x = tid; x < words; x += kChooseThreads) {
        uint32_t m = 0;
        for (int y = 0; y < 32; ++y)
            if (32 * x + y < e0 || (32 * x + y >= e1 && 32 * x + y < nb)) m |= 1u << y;
        s_bits[x] = m;
    }
    const float *src = staged ? s_score : row_score;

    // bound on any score's error: 2^-14 sum |q| max |bound|.  A score is a chain of 2 d / 16 products of 16 terms; a
    // sum of 17 values that keeps 23 bits of the largest errs by at most 17 2^-23 of it, 2 d / 16 <= 16 times over.
    float absq = 0.f, absb = 0.f;
    const uint16_t *qrow = p.q + ((size_t)(b * p.T + t) * p.H + hk * p.G) * p.d;
    for (int g = warp; g < p.G; g += NW) {
        float a = 0.f;
        for (int c = lane; c < p.d; c += 32) a += fabsf(bf16_bits_to_float(qrow[g * p.d + c]));
#pragma unroll
        for (int m = 16; m > 0; m >>= 1) a += __shfl_xor_sync(0xffffffffu, a, m);
        absq = a > absq || a != a ? a : absq;
    }
    const int chunks = (visible_blocks(p, b, p.T - 1) + kScoreBlocks - 1) / kScoreBlocks;
    for (int c = tid; c < chunks; c += kChooseThreads) {
        const float a = p.absmax[((size_t)b * p.Hkv + hk) * p.chunks + c];
        absb = a > absb || a != a ? a : absb;
    }
#pragma unroll
    for (int m = 16; m > 0; m >>= 1) {
        const float a = __shfl_xor_sync(0xffffffffu, absb, m);
        absb = a > absb || a != a ? a : absb;
    }
    lo = __reduce_min_sync(0xffffffffu, lo);
    hi = __reduce_max_sync(0xffffffffu, hi);
    if (tid == 0) {
        s_lo = ~0u;
        s_hi = 0;
        s_n = 0;
    }
    __syncthreads();
    if (lane == 0) {
        s_f[0][warp] = absq;
        s_f[1][warp] = absb;
        atomicMin(&s_lo, lo);
        atomicMax(&s_hi, hi);
    }
    __syncthreads();
    for (int w = 0; w < NW; ++w) {
        absq = s_f[0][w] > absq || s_f[0][w] != s_f[0][w] ? s_f[0][w] : absq;
        absb = s_f[1][w] > absb || s_f[1][w] != s_f[1][w] ? s_f[1][w] : absb;
    }
    const float size = absq * absb, err = size * 6.103515625e-05f;
    lo = s_lo;
    hi = s_hi;

    // [low, high]: the band in which fp32 does not decide.  Infinities, NaN and sums near fp32's range decide nothing.
    float low = -INFINITY, high = INFINITY;
    const bool usable = size < 1e37f;
    if (k > 0 && usable) {
        // lo <= t < hi: halve until the ends are equal or closer than the error
        if (hi != ~0u) ++hi;
        while (hi - lo > 1 && unordered(hi) - unordered(lo) > err) {
            const uint32_t mid = lo + (hi - lo) / 2;
            int n = 0;
            for (int x = e0 + tid; x < e1; x += kChooseThreads) n += ordered(src[x]) >= mid;
            if (block_sum(n, s_red) >= k) lo = mid;
            else hi = mid;
        }
        low = unordered(lo) - 2.f * err;
        high = unordered(hi) + 2.f * err;
    }
    __syncthreads();
    int sure = 0, near = 0;
    if (k > 0) {
        for (int x = e0 + tid; x < e1; x += kChooseThreads) {
            const float v = src[x];
            if (usable && v > high) {
                ++sure;
                atomicOr(&s_bits[x >> 5], 1u << (x & 31));
            } else if (!usable || v >= low) {
                ++near;
                const int at = atomicAdd(&s_n, 1);  // any order: they are ranked by score and index below
                if (at < kListed) s_blk[at] = x;
            }
        }
    }
    sure = block_sum(sure, s_red);
    near = block_sum(near, s_red);
    const int want = k - sure;
    if (want > 0 && near > want) {
        // fp64 scores of the blocks in the band, a warp each
        auto score64 = [&](int x) -> unsigned long long {
            int pg = p.table[(size_t)b * p.max_blocks + x];
            if (pg < 0 || pg >= p.n_pages) return ordered(-INFINITY + 0.0);
            const uint16_t *bx = p.k_max + ((size_t)pg * p.Hkv + hk) * p.d, *bn = p.k_min + ((size_t)pg * p.Hkv + hk) * p.d;
            unsigned long long best = 0;
            for (int g = 0; g < p.G; ++g) {
                double s = 0.0;
                for (int ch = lane; ch < p.d; ch += 32) {
                    const float qv = bf16_bits_to_float(qrow[g * p.d + ch]);
                    const float up = qv > 0.f || qv != qv ? qv : 0.f, dn = qv < 0.f || qv != qv ? qv : 0.f;
                    s += (double)up * (double)bf16_bits_to_float(bx[ch]) + (double)dn * (double)bf16_bits_to_float(bn[ch]);
                }
#pragma unroll
                for (int m = 16; m > 0; m >>= 1) s += __shfl_xor_sync(0xffffffffu, s, m);
                const unsigned long long o = ordered(s);
                best = o > best ? o : best;
            }
            return best;
        };
        if (near <= kListed) {  // ranked one against another
            for (int c = warp; c < near; c += NW) {
                const unsigned long long o = score64(s_blk[c]);
                if (lane == 0) s_key[c] = o;
            }
            __syncthreads();
            for (int c = tid; c < near; c += kChooseThreads) {
                const unsigned long long o = s_key[c];
                const int x = s_blk[c];
                int rank = 0;
                for (int y = 0; y < near; ++y) rank += s_key[y] > o || (s_key[y] == o && s_blk[y] < x);
                if (rank < want) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
            }
        } else {  // many equals (keys never written, say): by block in the workspace, 0 for those outside the band
            unsigned long long *key = p.exact + (size_t)row * p.stride;
            for (int x = e0 + warp; x < e1; x += NW) {
                const bool in = !usable || (src[x] >= low && !(src[x] > high));
                const unsigned long long o = in ? score64(x) : 0;
                if (lane == 0) key[x] = o;
            }
            __syncthreads();
            // the want-th highest key: the largest klo with count(key >= klo) >= want
            unsigned long long klo = 1, khi = ~0ull;
            while (klo < khi) {
                const unsigned long long mid = khi - (khi - klo) / 2;
                int n = 0;
                for (int x = e0 + tid; x < e1; x += kChooseThreads) n += key[x] >= mid;
                if (block_sum(n, s_red) >= want) klo = mid;
                else khi = mid - 1;
            }
            int above = 0;
            for (int x = e0 + tid; x < e1; x += kChooseThreads) {
                if (key[x] > klo) {
                    ++above;
                    atomicOr(&s_bits[x >> 5], 1u << (x & 31));
                }
            }
            // and the lowest indexes among its equals: those below the largest cut that takes `equal` of them
            const int equal = want - block_sum(above, s_red);
            int clo = e0, chi = e1;
            while (clo < chi) {
                const int mid = chi - (chi - clo) / 2;
                int n = 0;
                for (int x = e0 + tid; x < mid; x += kChooseThreads) n += key[x] == klo;
                if (block_sum(n, s_red) <= equal) clo = mid;
                else chi = mid - 1;
            }
            for (int x = e0 + tid; x < clo; x += kChooseThreads)
                if (key[x] == klo) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
        }
    } else if (want > 0) {  // the whole band
        for (int x = e0 + tid; x < e1; x += kChooseThreads)
            if (!usable || (src[x] >= low && !(src[x] > high))) atomicOr(&s_bits[x >> 5], 1u << (x & 31));
    }
    __syncthreads();

    // the chosen indexes in ascending order
    int base = 0;
    for (int w0 = 0; w0 < words; w0 += kChooseThreads) {
        const uint32_t m = w0 + tid < words ? s_bits[w0 + tid] : 0u;
        int n = __popc(m);
        const int mine = n;
#pragma unroll
        for (int s = 1; s < 32; s <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, n, s);
            if (lane >= s) n += y;
        }
        __syncthreads();
        if (lane == 31) s_red[warp] = n;
        __syncthreads();
        int at = base + n - mine;
        for (int w = 0; w < NW; ++w) {
            if (w < warp) at += s_red[w];
            base += s_red[w];
        }
        for (uint32_t x = m; x; x &= x - 1) {
            if (at < p.n_select) sel[at] = 32 * (w0 + tid) + __ffs(x) - 1;
            ++at;
        }
    }
}

size_t row_stride(int max_blocks) { return round_up((size_t)max_blocks, 4); }

size_t select_ws(const hla_kv_cache *C, int B, int T, int H, int max_blocks) {
    if (check_cache(C, false, false) != HLA_OK || check_window(C, B, T, H, max_blocks) != HLA_OK || max_blocks > kMaxBlocks)
        return 0;
    const size_t rows = (size_t)B * T * C->kv_heads, chunks = (max_blocks + kScoreBlocks - 1) / kScoreBlocks;
    return rows * row_stride(max_blocks) * (sizeof(unsigned long long) + sizeof(float)) + round_up((size_t)B * C->kv_heads * chunks * sizeof(float), 16);
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
    HLA_REQUIRE((long)B * C->kv_heads <= 65535, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(aligned16(block_table) && aligned16(past_len) && aligned16(q) && aligned16(sel), HLA_ERR_MISALIGNED);
    HLA_REQUIRE(ws && ws_bytes >= select_ws(C, B, T, H, max_blocks), HLA_ERR_WORKSPACE);
    HLA_REQUIRE(aligned16(ws), HLA_ERR_MISALIGNED);
    SelectParams p = {};
    p.q = q; p.k_min = C->k_min; p.k_max = C->k_max; p.table = block_table; p.past = past_len; p.sel = sel;
    p.B = B; p.T = T; p.H = H; p.Hkv = C->kv_heads; p.G = H / C->kv_heads; p.d = C->head_dim;
    p.max_blocks = max_blocks; p.n_pages = C->n_pages; p.pshift = page_shift(C->page_size);
    p.n_select = n_select; p.n_first = n_first; p.n_last = n_last;
    p.stride = (int)row_stride(max_blocks);
    p.chunks = (max_blocks + kScoreBlocks - 1) / kScoreBlocks;
    const size_t rows = (size_t)B * T * p.Hkv;
    p.exact = static_cast<unsigned long long *>(ws);
    p.score = reinterpret_cast<float *>(p.exact + rows * p.stride);
    p.absmax = p.score + rows * p.stride;
    const cudaStream_t st = (cudaStream_t)stream;
    set_variant("attn_select<d%d>", p.d);
    PdlChain chain(st, pdl_default(B * T));
    const dim3 grid((unsigned)p.chunks, (unsigned)(B * p.Hkv));
    e = launched(p.d == 128 ? launch_kernel(attn_score_kernel<128>, grid, dim3(kScoreThreads), 0, st, p)
                            : launch_kernel(attn_score_kernel<64>, grid, dim3(kScoreThreads), 0, st, p));
    if (e != HLA_OK) return e;
    return launched(launch_kernel(attn_choose_kernel, dim3((unsigned)rows), dim3(kChooseThreads), 0, st, p));
}
