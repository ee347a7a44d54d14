// Appending new tokens to a paged key-value cache, with the position rotation of q and k on the way and the
// per-channel key bounds of the touched pages.
//
// Rotation: channel pair (x, y) of frequency f at position p becomes (x cos a - y sin a, x sin a + y cos a) with
// a = p f.  Far positions lose their angle in fp32, so a is kept as a fraction of a turn in 64 bits:
// F = 2^64 frac(f / 2 pi), from f's own bits in integers, and p F modulo 2^64 is exact; its top 32 bits, less the nearest
// quarter, give the sine and cosine.  (fp64 would do too, but a page's keys take one angle per pair and token, and the fp64
// rate of this part is far below that.)
//
// Every value is read and written once, so the step is bound by memory, and at decode sizes by latency.  One grid
// does both halves: blocks that own a touched page for some kv heads, and blocks that own some tokens of q.
// Measured (CUDA graph, 32 query and 8 kv heads of 128): one token 3.5 us; 64 x 4 tokens, e4m3, 6.1 us; 60 single
// tokens and 4 chunks of 512 14.3 us; 8 prompts of 4093 tokens 129 us, 6.2 TB/s of reads and writes.
#include "paged.cuh"

namespace hla {
namespace {

constexpr int kThreads = 128;
constexpr int kMaxQTokens = 4;    // tokens of q per CTA

struct AppendParams {
    const uint16_t *q, *k, *v;
    uint16_t *q_out;
    uint8_t *k_cache, *v_cache;
    const float *k_scale, *v_scale;
    uint16_t *k_min, *k_max;
    const int32_t *cu, *past, *table;
    const double *inv_freq;
    int N, B, H, Hkv, pshift, n_pages, max_blocks;
    int half;                 // rotated channel pairs per head (0: none)
    int heads_per_cta, q_tokens, kv_ctas, head_groups;
    uint32_t by_half, by_H, by_head_groups;  // for divided()
};

// Fraction of a turn per position, in units of 2^-64 turn, cut off: the fp64 value m 2^e times 2^128 / 2 pi in integers.
__device__ __forceinline__ uint64_t turn_fraction(double inv_freq) {
    const uint64_t bits = (uint64_t)__double_as_longlong(inv_freq), hi = 0x28be60db9391054aull, lo = 0x7f09d5f47d4d3770ull;
    const int ex = (int)(bits >> 52 & 0x7ff);
    const uint64_t m = (bits & 0xfffffffffffffull) | (ex ? 1ull << 52 : 0ull);
    const uint64_t w0 = m * lo, x = __umul64hi(m, lo), y = m * hi, w1 = x + y, w2 = __umul64hi(m, hi) + (w1 < x);
    const int s = 64 + 1075 - (ex ? ex : 1);  // the product, w2 w1 w0, in units of 2^-64 turn: shifted right by s
    uint64_t u = 0;
    if (s >= 128) u = s < 192 ? w2 >> (s - 128) : 0;
    else if (s > 64) u = w2 << (128 - s) | w1 >> (s - 64);
    else if (s > 0) u = s == 64 ? w1 : w1 << (64 - s) | w0 >> s;
    return bits >> 63 ? 0 - u : u;
}
// The angle in units of 2^-32 turn, rounded, is taken to within an eighth of a turn of a quarter before it meets fp32, whose
// 24 bits would otherwise leave 2^-26 of a turn.  There the Taylor series of sine and cosine end soon: what follows the last
// terms here is below 2^-28 of the sums.
__device__ __forceinline__ float2 cos_sin(uint64_t turns, int pos) {
    const uint32_t top = (uint32_t)((turns * (uint64_t)(uint32_t)pos + 0x80000000ull) >> 32);
    const uint32_t quarter = (top + 0x20000000u) >> 30;
    const float a = (float)(int32_t)(top - (quarter << 30)) * 1.4629180792671596e-09f, q = a * a;  // 2 pi / 2^32
    float s = fmaf(q, 1.f / 362880.f, -1.f / 5040.f);
    s = fmaf(s, q, 1.f / 120.f);
    s = fmaf(s, q, -1.f / 6.f);
    s = fmaf(s * q, a, a);
    float c = fmaf(q, -1.f / 3628800.f, 1.f / 40320.f);
    c = fmaf(c, q, -1.f / 720.f);
    c = fmaf(c, q, 1.f / 24.f);
    c = fmaf(c, q, -0.5f);
    c = fmaf(c, q, 1.f);
    const float x = quarter & 1 ? s : c, y = quarter & 1 ? c : s;
    return make_float2((quarter + 1) & 2 ? -x : x, quarter & 2 ? -y : y);
}

// First token and number of new tokens of sequence b, clamped to the N rows there are; 0 for an idle slot.
__device__ __forceinline__ int new_tokens(const AppendParams &p, int b, int *first) {
    int a = p.cu[b], e = p.cu[b + 1];
    a = a < 0 ? 0 : a;
    e = e > p.N ? p.N : e;
    *first = a;
    return p.past[b] >= 0 && e > a ? e - a : 0;
}

// Pages of sequence b that its new tokens touch (inside its table).
__device__ __forceinline__ int touched_pages(const AppendParams &p, int b) {
    int first;
    const int n = new_tokens(p, b, &first);
    if (n == 0) return 0;
    const long j0 = (long)p.past[b] >> p.pshift, j1 = ((long)p.past[b] + n - 1) >> p.pshift;
    if (j0 >= p.max_blocks) return 0;
    return (int)((j1 < p.max_blocks - 1 ? j1 : p.max_blocks - 1) - j0 + 1);
}

// Two 16-byte chunks of a head (channels 8 c0.. and 8 c1..) that are rotated together.  half == 0, or chunks behind
// the rotated ones: unchanged.
template <bool INTER>
__device__ __forceinline__ void item_chunks(const AppendParams &p, int x, int *c0, int *c1) {
    const int hc = p.half >> 3;  // chunks of one half
    if (!INTER && x < hc) {
        *c0 = x;
        *c1 = x + hc;
    } else {  // the x-th pair of neighbouring chunks (the first 2 hc are the hc rotated items above)
        *c0 = 2 * x;
        *c1 = 2 * x + 1;
    }
}

__device__ __forceinline__ void unpack8(const uint4 w, float (&f)[8]) {
    f[0] = bf16_lo(w.x); f[1] = bf16_hi(w.x); f[2] = bf16_lo(w.y); f[3] = bf16_hi(w.y);
    f[4] = bf16_lo(w.z); f[5] = bf16_hi(w.z); f[6] = bf16_lo(w.w); f[7] = bf16_hi(w.w);
}
__device__ __forceinline__ uint4 pack8(const float (&f)[8]) {
    return make_uint4(pack_bf16x2(f[0], f[1]), pack_bf16x2(f[2], f[3]), pack_bf16x2(f[4], f[5]), pack_bf16x2(f[6], f[7]));
}

// Place of a pair's (cos, sin) in its row: the eight pairs of an item lie one item count apart and a row is 64 bytes
// longer than a round of the banks, so that the items and rows of a warp read side by side.
template <int D>
__device__ __forceinline__ int angle_at(int pair) {
    return (pair & 7) * (D / 16) + (pair >> 3);
}

// Rotates the item's 16 channels; cs: (cos, sin) of the row's pairs.
template <int D, bool INTER>
__device__ __forceinline__ void rotate(const AppendParams &p, int x, float (&a)[8], float (&b)[8], const float2 *cs) {
    if (8 * x >= p.half) return;
    if constexpr (INTER) {
#pragma unroll
        for (int y = 0; y < 8; y += 2) {
            const float2 u = cs[(y >> 1) * (D / 16) + x], w = cs[(4 + (y >> 1)) * (D / 16) + x];
            const float a0 = a[y], b0 = b[y];
            a[y] = a0 * u.x - a[y + 1] * u.y;
            a[y + 1] = a0 * u.y + a[y + 1] * u.x;
            b[y] = b0 * w.x - b[y + 1] * w.y;
            b[y + 1] = b0 * w.y + b[y + 1] * w.x;
        }
    } else {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            const float2 u = cs[y * (D / 16) + x];
            const float a0 = a[y];
            a[y] = a0 * u.x - b[y] * u.y;
            b[y] = a0 * u.y + b[y] * u.x;
        }
    }
}

__device__ __forceinline__ uint4 e4m3x8_to_bf16x8(const uint2 t) {  // exact
    uint32_t h[4], o[4];
    e4m3x4_to_f16x4(t.x, h[0], h[1]);
    e4m3x4_to_f16x4(t.y, h[2], h[3]);
#pragma unroll
    for (int y = 0; y < 4; ++y) {
        const float2 g = __half22float2(*reinterpret_cast<const __half2 *>(&h[y]));
        o[y] = pack_bf16x2(g.x, g.y);
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// 8 values as the cache holds them; returns them as bf16 (an e4m3 value is one exactly).
template <bool FP8>
__device__ __forceinline__ uint4 store8(uint8_t *row, int c, float (&f)[8], float scale) {
    if constexpr (!FP8) {
        const uint4 w = pack8(f);
        reinterpret_cast<uint4 *>(row)[c] = w;
        return w;
    } else {
        // values beyond the largest e4m3 saturate, infinities too
        uint32_t r[4];
#pragma unroll
        for (int y = 0; y < 4; ++y) r[y] = f32x2_to_e4m3x2(__fdiv_rn(f[2 * y], scale), __fdiv_rn(f[2 * y + 1], scale));
        const uint2 t = make_uint2(r[0] | r[1] << 16, r[2] | r[3] << 16);
        reinterpret_cast<uint2 *>(row)[c] = t;
        return e4m3x8_to_bf16x8(t);
    }
}

// 8 cached values as bf16.
template <bool FP8>
__device__ __forceinline__ uint4 load8(const uint8_t *row, int c) {
    if constexpr (!FP8) {
        return reinterpret_cast<const uint4 *>(row)[c];
    } else {
        return e4m3x8_to_bf16x8(reinterpret_cast<const uint2 *>(row)[c]);
    }
}

// (lo, hi) of 16 channels, taking up the item's two chunks.
struct Bounds {
    uint32_t lo[8], hi[8];
    __device__ __forceinline__ void clear() {
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            lo[y] = 0x7f807f80u;  // +inf
            hi[y] = 0xff80ff80u;  // -inf
        }
    }
    __device__ __forceinline__ void take(const uint4 a, const uint4 b) {
        const uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int y = 0; y < 8; ++y) {
            lo[y] = min2(lo[y], w[y]);
            hi[y] = max2(hi[y], w[y]);
        }
    }
};

template <int D, bool FP8, bool INTER>
__global__ void __launch_bounds__(kThreads, 6) kv_append_kernel(const AppendParams p) {
    constexpr int ITEMS = D / 16;              // pairs of chunks per head row
    constexpr int LANES = kThreads / ITEMS;    // rows in flight
    constexpr int ES = FP8 ? 1 : 2;
    constexpr int MAXH = D / 2;                // channel pairs
    __shared__ uint64_t s_turn[MAXH];
    // angles of one pass of LANES cache rows, and of the next (or of the tokens of q)
    __shared__ float2 s_cs[2][LANES][MAXH + 8];
    __shared__ uint32_t s_lo[4][ITEMS][8], s_hi[4][ITEMS][8];
    __shared__ int s_warp[4], s_b, s_j;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int item = tid % ITEMS, rl = tid / ITEMS;
    pdl_wait_trigger();
    if (tid < p.half) s_turn[tid] = turn_fraction(p.inv_freq[tid]);
    int c0, c1;
    item_chunks<INTER>(p, item, &c0, &c1);

    if ((int)blockIdx.x >= p.kv_ctas) {
        // ---- q of some tokens: all heads
        const int n0 = (blockIdx.x - p.kv_ctas) * p.q_tokens;
        const int nt = p.N - n0 < p.q_tokens ? p.N - n0 : p.q_tokens, rows = nt * p.H;
        __shared__ int s_pos[kMaxQTokens];
        // four rows at a time: their loads are in flight together, the first ones while the positions are found
        uint4 wa[4], wb[4];
        auto load = [&](int r0) {
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = r0 + y * LANES;
                if (r >= rows) break;
                const size_t o = ((size_t)n0 * p.H + r) * D;
                wa[y] = ld_act_v4(p.q + o + 8 * c0);
                wb[y] = ld_act_v4(p.q + o + 8 * c1);
            }
        };
        load(rl);
        for (int x = 0; x < nt; ++x) {
            // the sequence of token n0 + x: the number of offsets cu[1..B] at or below it
            int n = 0;
            for (int y0 = 0; y0 < p.B; y0 += kThreads)
                n += __syncthreads_count(y0 + tid < p.B && p.cu[y0 + tid + 1] <= n0 + x);
            if (tid == 0) {
                int pos = -1;
                if (n < p.B && n0 + x >= p.cu[n] && p.past[n] >= 0) pos = p.past[n] + (n0 + x - p.cu[n]);
                s_pos[x] = pos;
            }
        }
        __syncthreads();
        for (int x = tid; x < nt * p.half; x += kThreads) {
            const int t = divided(x, p.by_half), h = x - t * p.half;
            s_cs[0][t][angle_at<D>(h)] = cos_sin(s_turn[h], s_pos[t]);
        }
        __syncthreads();
        for (int r0 = rl; r0 < rows; r0 += 4 * LANES) {
            if (r0 != rl) load(r0);
#pragma unroll
            for (int y = 0; y < 4; ++y) {
                const int r = r0 + y * LANES, t = divided(r, p.by_H);
                if (r >= rows) break;
                if (s_pos[t] < 0) continue;  // no sequence's token, or an idle one's: left as it was
                const size_t o = ((size_t)n0 * p.H + r) * D;
                float a[8], b[8];
                unpack8(wa[y], a);
                unpack8(wb[y], b);
                rotate<D, INTER>(p, item, a, b, s_cs[0][t]);
                *reinterpret_cast<uint4 *>(p.q_out + o + 8 * c0) = pack8(a);
                *reinterpret_cast<uint4 *>(p.q_out + o + 8 * c1) = pack8(b);
            }
        }
        return;
    }

    // ---- one touched page, some kv heads.  Which: the u-th of all sequences' touched pages.
    const int u = divided(blockIdx.x, p.by_head_groups), h0 = (blockIdx.x - u * p.head_groups) * p.heads_per_cta;
    const int h1 = h0 + p.heads_per_cta < p.Hkv ? h0 + p.heads_per_cta : p.Hkv;
    if (tid == 0) s_b = -1;
    int base = 0;
    for (int b0 = 0; b0 < p.B && base <= u; b0 += kThreads) {
        const int np = b0 + tid < p.B ? touched_pages(p, b0 + tid) : 0;
        int x = np;
#pragma unroll
        for (int m = 1; m < 32; m <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, x, m);
            if (lane >= m) x += y;
        }
        __syncthreads();
        if (lane == 31) s_warp[warp] = x;
        __syncthreads();
        int before = base + x - np;
        for (int w = 0; w < 4; ++w) {
            if (w < warp) before += s_warp[w];
            base += s_warp[w];
        }
        if (u >= before && u < before + np) {
            s_b = b0 + tid;
            s_j = u - before;
        }
    }
    __syncthreads();
    const int b = s_b;
    if (b < 0) return;  // fewer touched pages than the grid allows for
    int first;
    const int n = new_tokens(p, b, &first), past = p.past[b];
    const int j = (past >> p.pshift) + s_j, start = j << p.pshift;
    const int pg = p.table[(size_t)b * p.max_blocks + j];
    if (pg < 0 || pg >= p.n_pages) return;  // no page: its tokens are dropped
    const int r0 = past > start ? past - start : 0;
    const long rest = (long)n + (past - start);
    const int P = 1 << p.pshift, r1 = rest < P ? (int)rest : P;
    const int t0 = first + start - past;  // token of page row 0
    const bool bounds = p.k_min != nullptr;

    for (int h = h0; h < h1; ++h) {
        uint8_t *kp = p.k_cache + (((size_t)pg * p.Hkv + h) << p.pshift) * (D * ES);
        uint8_t *vp = p.v_cache + (((size_t)pg * p.Hkv + h) << p.pshift) * (D * ES);
        const float ks = FP8 ? p.k_scale[h] : 1.f, vs = FP8 ? p.v_scale[h] : 1.f;
        Bounds bd;
        bd.clear();
        // LANES rows a pass, one to a thread; the next pass's rows and angles are on their way during this one's work
        uint4 ka, kb, va, vb;
        auto load = [&](int r) {
            if (r >= r1) return;
            const size_t o = ((size_t)(t0 + r) * p.Hkv + h) * D;
            ka = ld_act_v4(p.k + o + 8 * c0);
            kb = ld_act_v4(p.k + o + 8 * c1);
            va = ld_act_v4(p.v + o + 8 * c0);
            vb = ld_act_v4(p.v + o + 8 * c1);
        };
        auto angles = [&](int buf, int rr) {
            const int n = (r1 - rr < LANES ? r1 - rr : LANES) * p.half;
            for (int x = tid; x < n; x += kThreads) {
                const int r = divided(x, p.by_half), y = x - r * p.half;
                s_cs[buf][r][angle_at<D>(y)] = cos_sin(s_turn[y], start + rr + r);
            }
        };
        const bool many = r1 - r0 > LANES;  // otherwise the angles of the one pass serve all heads
        load(r0 + rl);
        if (bounds)  // keys that were there
#pragma unroll 1
            for (int r = rl; r < r0; r += 2 * LANES) {
                uint4 oa[2], ob[2];
#pragma unroll
                for (int y = 0; y < 2; ++y) {
                    const int x = r + y * LANES < r0 ? r + y * LANES : r;
                    oa[y] = load8<FP8>(kp + x * (D * ES), c0);
                    ob[y] = load8<FP8>(kp + x * (D * ES), c1);
                }
#pragma unroll
                for (int y = 0; y < 2; ++y) bd.take(oa[y], ob[y]);
            }
        if (h == h0 || many) {
            __syncthreads();  // (the last head's rows are done with the angles; s_turn is there)
            angles(0, r0);
            __syncthreads();
        }
        for (int rr = r0, buf = 0; rr < r1; rr += LANES, buf ^= 1) {
            const int r = rr + rl;
            const uint4 ca = ka, cb = kb, da = va, db = vb;
            load(r + LANES);
            if (r < r1) {
                float a[8], c[8];
                unpack8(ca, a);
                unpack8(cb, c);
                rotate<D, INTER>(p, item, a, c, s_cs[buf][rl]);
                uint8_t *krow = kp + r * (D * ES), *vrow = vp + r * (D * ES);
                const uint4 wa = store8<FP8>(krow, c0, a, ks), wb = store8<FP8>(krow, c1, c, ks);
                if (bounds) bd.take(wa, wb);
                if constexpr (!FP8) {
                    reinterpret_cast<uint4 *>(vrow)[c0] = da;
                    reinterpret_cast<uint4 *>(vrow)[c1] = db;
                } else {
                    unpack8(da, a);
                    unpack8(db, c);
                    store8<true>(vrow, c0, a, vs);
                    store8<true>(vrow, c1, c, vs);
                }
            }
            if (rr + LANES < r1) {
                angles(buf ^ 1, rr + LANES);
                __syncthreads();
            }
        }
        if (!bounds) continue;
        // over the rows: lanes of a warp that share an item, then the warps
#pragma unroll
        for (int m = ITEMS; m < 32; m <<= 1)
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                bd.lo[y] = min2(bd.lo[y], __shfl_xor_sync(0xffffffffu, bd.lo[y], m));
                bd.hi[y] = max2(bd.hi[y], __shfl_xor_sync(0xffffffffu, bd.hi[y], m));
            }
        __syncthreads();
        if (lane < ITEMS)
#pragma unroll
            for (int y = 0; y < 8; ++y) {
                s_lo[warp][item][y] = bd.lo[y];
                s_hi[warp][item][y] = bd.hi[y];
            }
        __syncthreads();
        if (tid < ITEMS * 8) {
            const int it = tid / 8, y = tid % 8;
            uint32_t lo = s_lo[0][it][y], hi = s_hi[0][it][y];
            for (int w = 1; w < 4; ++w) {
                lo = min2(lo, s_lo[w][it][y]);
                hi = max2(hi, s_hi[w][it][y]);
            }
            int a, c;
            item_chunks<INTER>(p, it, &a, &c);
            const size_t o = ((size_t)pg * p.Hkv + h) * D + 8 * (y < 4 ? a : c) + 2 * (y & 3);
            *reinterpret_cast<uint32_t *>(p.k_min + o) = lo;
            *reinterpret_cast<uint32_t *>(p.k_max + o) = hi;
        }
    }
}

}  // namespace
}  // namespace hla

using namespace hla;

extern "C" int kv_cache_append(const hla_kv_cache *C, int N, int B, const int32_t *cu_seqlens, const int32_t *past_len,
                               int max_blocks, const int32_t *block_table, int H, const hla_bf16 *q, const hla_bf16 *k,
                               const hla_bf16 *v, int rope_dim, int rope_interleaved, const double *inv_freq,
                               hla_bf16 *q_out, hla_stream stream) {
    int e = check_cache(C, true, false);
    if (e != HLA_OK) return e;
    HLA_REQUIRE(N >= 1, HLA_ERR_INVALID_ARG);
    e = check_window(C, B, 1, H, max_blocks);
    if (e != HLA_OK) return e;
    HLA_REQUIRE(cu_seqlens && past_len && block_table && q && k && v && q_out, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(rope_dim >= 0 && (rope_interleaved == 0 || rope_interleaved == 1), HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(rope_dim <= C->head_dim && rope_dim % 16 == 0, HLA_ERR_UNSUPPORTED);
    HLA_REQUIRE(rope_dim == 0 || inv_freq, HLA_ERR_INVALID_ARG);
    HLA_REQUIRE(aligned16(cu_seqlens) && aligned16(past_len) && aligned16(block_table) && aligned16(q) && aligned16(k) &&
                    aligned16(v) && aligned16(q_out) && aligned16(inv_freq),
                HLA_ERR_MISALIGNED);
    AppendParams p = {};
    p.q = q; p.k = k; p.v = v; p.q_out = q_out;
    p.k_cache = static_cast<uint8_t *>(C->k); p.v_cache = static_cast<uint8_t *>(C->v);
    p.k_scale = C->k_scale; p.v_scale = C->v_scale; p.k_min = C->k_min; p.k_max = C->k_max;
    p.cu = cu_seqlens; p.past = past_len; p.table = block_table; p.inv_freq = inv_freq;
    p.N = N; p.B = B; p.H = H; p.Hkv = C->kv_heads; p.pshift = page_shift(C->page_size);
    p.n_pages = C->n_pages; p.max_blocks = max_blocks;
    p.half = rope_dim / 2;
    // n new tokens touch at most n pages, and at most n / page_size + 2
    const long by_size = (long)N / C->page_size + 2L * B, pages = N < by_size ? N : by_size;
    // Heads of a page share its angles; one head per CTA until the pages alone fill the SMs several times: two heads per
    // CTA take prompts from 133 to 131 us, but a mixed batch, whose longest CTA sets the pace, from 18 to 26.
    p.heads_per_cta = 1;
    while (p.heads_per_cta < p.Hkv && pages * ((p.Hkv + 2 * p.heads_per_cta - 1) / (2 * p.heads_per_cta)) >= 8L * sm_count()) p.heads_per_cta *= 2;
    p.head_groups = (p.Hkv + p.heads_per_cta - 1) / p.heads_per_cta;
    const long kv = pages * p.head_groups;
    p.by_half = divisor(p.half ? p.half : 1); p.by_H = divisor(p.H); p.by_head_groups = divisor(p.head_groups);
    p.q_tokens = 1;  // four rows in flight per thread want four tokens of 32 heads, once there are tokens enough
    while (p.q_tokens < kMaxQTokens && N / (2 * p.q_tokens) >= 3L * sm_count()) p.q_tokens *= 2;
    const long qc = (N + p.q_tokens - 1) / p.q_tokens;
    HLA_REQUIRE(kv * p.head_groups < (1L << 31) && kv + qc < (1L << 31), HLA_ERR_UNSUPPORTED);
    p.kv_ctas = (int)kv;
    const bool fp8 = C->dtype == HLA_E4M3;
    const int D = C->head_dim;
    set_variant("kv_append<d%d,%s,rope%d%s>", D, fp8 ? "e4m3" : "bf16", rope_dim, rope_interleaved ? "i" : "");
    const cudaStream_t st = (cudaStream_t)stream;
    const dim3 grid((unsigned)(kv + qc));
    auto go = [&](auto kernel) { return launched(launch_kernel(kernel, grid, dim3(kThreads), 0, st, p)); };
    const bool in = rope_interleaved != 0;
    if (D == 128) {
        if (fp8) return in ? go(kv_append_kernel<128, true, true>) : go(kv_append_kernel<128, true, false>);
        return in ? go(kv_append_kernel<128, false, true>) : go(kv_append_kernel<128, false, false>);
    }
    if (fp8) return in ? go(kv_append_kernel<64, true, true>) : go(kv_append_kernel<64, true, false>);
    return in ? go(kv_append_kernel<64, false, true>) : go(kv_append_kernel<64, false, false>);
}
