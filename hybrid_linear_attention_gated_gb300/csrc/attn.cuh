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
    int tshift;       // log2 of keys per tile
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
    const int cap = p.max_blocks << p.pshift;  // (below 2^30, as the cached tokens and the listed ones)
    const int len = p.sel ? listed(p, past + p.T - 1) << p.pshift : past + p.T < cap ? past + p.T : cap;
    return (len + (1 << p.tshift) - 1) >> p.tshift;
}

// (out of line: a short call's time goes into fetching its instructions, and these would lie among them)
static __device__ __noinline__ void many_prefix(const AttnParams &p, int *pre, int *past) {
    for (int b = threadIdx.x; b < p.B; b += blockDim.x) {
        const int c = cached(p, b);
        if (past) past[b] = c;
        pre[b + 1] = unit_tiles(p, c);
    }
    block_prefix(pre, p.B);
}

// Prefix sums of the sequences' tiles per unit into pre[0..B], and their cached tokens into past[0..B-1] where
// that is wanted; ends with a block barrier.
__device__ __forceinline__ void tile_prefix(const AttnParams &p, int *pre, int *past = nullptr) {
    const int lane = threadIdx.x;
    if (p.B <= 32) {
        if (lane < 32) {
            const int c = lane < p.B ? cached(p, lane) : -1;
            if (past && lane < p.B) past[lane] = c;
            const int x = warp_prefix(unit_tiles(p, c), lane);
            if (lane < p.B) pre[lane + 1] = x;
            if (lane == 0) pre[0] = 0;
        }
    } else {
        many_prefix(p, pre, past);
    }
    __syncthreads();
}

// Tiles that each CTA of the attention grid takes.
__device__ __forceinline__ int cta_share(int total, int grid) {
    const int s = (int)(((unsigned)total + grid - 1u) / (unsigned)grid);
    return s < 1 ? 1 : s;
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
