// What the two attention kernels share: parameters, the split of the work by the lengths on the device, and the
// output's stores.
#pragma once

#include "paged.cuh"

namespace hla {

constexpr int kGroup = 16;      // keys that are copied and masked together: never more than one page
constexpr int kAttnThreads = 128;
constexpr int kNoKeys = 1 << 30;  // token index of a group without keys: behind every row's last key
constexpr float kLog2e = 1.44269504088896340736f;

struct AttnParams {
    const uint8_t *k, *v;
    const float *k_scale, *v_scale;
    const uint16_t *q;
    void *o;
    const int32_t *table, *past, *sel;  // sel: null for the dense form
    float *part_o, *part_ml;
    float scale;
    int B, T, H, Hkv, G;
    int max_blocks, n_pages, pshift, n_select;
    int row_tiles;    // row tiles of a unit's rows
    int units_per_b;  // units of one sequence
    int min_share;    // least tiles per CTA
    int tile;         // keys per tile
    uint32_t by_G, by_Hkv, by_row_tiles;  // for divided()
    int o_bf16;
    int *status;       // attn_tc_kernel: the device status word
    int force_timeout; // test hook, see hla_test_force_wait_timeout
};

// Cached tokens of sequence b; negative: an idle slot.  Held below 2^30 so that token indexes stay in 32 bits
// (the table covers fewer).
__device__ __forceinline__ int cached(const AttnParams &p, int b) {
    const int x = p.past[b];
    return x < kNoKeys - 16 ? x : kNoKeys - 16;
}

// Entries of its list that the token at position pos reads: no more than the blocks it sees.
__device__ __forceinline__ int listed(const AttnParams &p, int pos) {
    const int n = (pos >> p.pshift) + 1;
    return n < p.n_select ? n : p.n_select;
}

// Tiles of one unit of a sequence with `past` cached tokens.
__device__ __forceinline__ int unit_tiles(const AttnParams &p, int past) {
    if (past < 0) return 0;
    if (p.sel) return (int)((((long)listed(p, past + p.T - 1) << p.pshift) + p.tile - 1) / p.tile);
    const long cap = (long)p.max_blocks << p.pshift;
    const long len = (long)past + p.T < cap ? (long)past + p.T : cap;
    return (int)((len + p.tile - 1) / p.tile);
}

// Prefix sums of the sequences' tiles per unit into pre[0..B], and their cached tokens into past[0..B-1] where
// that is wanted; ends with a block barrier.
__device__ __forceinline__ void tile_prefix(const AttnParams &p, int *pre, int *past = nullptr) {
    const int lane = threadIdx.x;
    if (lane < 32) {
        int base = 0;
        for (int b0 = 0; b0 < p.B; b0 += 32) {
            const int b = b0 + lane;
            const int c = b < p.B ? cached(p, b) : -1;
            int x = unit_tiles(p, c);
            if (past && b < p.B) past[b] = c;
#pragma unroll
            for (int m = 1; m < 32; m <<= 1) {
                const int y = __shfl_up_sync(0xffffffffu, x, m);
                if (lane >= m) x += y;
            }
            if (b < p.B) pre[b + 1] = base + x;
            base += __shfl_sync(0xffffffffu, x, 31);
        }
        if (lane == 0) pre[0] = 0;
    }
    __syncthreads();
}

// Tiles that each CTA of the attention grid takes.
__device__ __forceinline__ int cta_share(const AttnParams &p, int total, int grid) {
    const int s = (int)(((long)total + grid - 1) / grid);
    return s < p.min_share ? p.min_share : s;
}

// The sequence whose units hold tile t: pre[b] * units <= t < pre[b + 1] * units.
__device__ __forceinline__ int find_sequence(const int *pre, int B, int units, int t) {
    int lo = 0, hi = B;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] * units <= t) lo = mid;
        else hi = mid;
    }
    return lo;
}

__device__ __forceinline__ void store_out(const AttnParams &p, size_t at, float x, float y) {
    if (p.o_bf16)
        *reinterpret_cast<uint32_t *>(reinterpret_cast<uint16_t *>(p.o) + at) = pack_bf16x2(x, y);
    else
        *reinterpret_cast<float2 *>(reinterpret_cast<float *>(p.o) + at) = make_float2(x, y);
}

// attn_tc.cu: the same pieces on tcgen05, rows in tiles of 128.  *grid: CTAs launched, at most `most`.
constexpr int kTcRows = 128;
constexpr int kTcTile = 64;   // keys per tile
cudaError_t launch_attn_tc(int D, const AttnParams &p, int *grid, long most, cudaStream_t st);

}  // namespace hla
