// Shared by the kernels of ep_expert_matmul: which rows an expert owns, which
// x row an output row reads, and the prefix of the experts' row tiles.
#pragma once

#include <cuda_bf16.h>

#include "ep_kernels.cuh"

namespace ep {
namespace mm {

constexpr unsigned kFull = 0xffffffffu;

// Number of rows of expert e, and its first position in expert-major order,
// for any contents of the offsets: clamped to the rows that the output holds.
__device__ __forceinline__ int expert_rows(const MatmulArgs& a, int e, int& begin) {
    const int limit = a.layout == 0 ? a.rows : INT32_MAX;
    begin = max(0, min(__ldg(a.expert_offsets + e), limit));
    const int end = max(begin, min(__ldg(a.expert_offsets + e + 1), limit));
    return a.layout == 0 ? end - begin : min(end - begin, a.cap);
}

// Row of x that row i of expert e reads, -1 for none.
__device__ __forceinline__ int source_row(const MatmulArgs& a, int e, int begin, int i) {
    if (a.row_src == nullptr) return a.layout == 0 ? begin + i : e * a.cap + i;
    const long long p = (long long)begin + i;
    if (p >= a.n_src) return -1;
    const int r = __ldg(a.row_src + p);
    return (r >= 0 && r < a.x_rows) ? r : -1;
}

// First output row of expert e.
__device__ __forceinline__ size_t first_row(const MatmulArgs& a, int e, int begin) {
    return a.layout == 0 ? (size_t)begin : (size_t)e * a.cap;
}

// Row tiles of the experts: s_tiles[i] = tiles of ceil(rows_e / tile) rows over
// the experts before 8 i (an eighth of a full table, so that it takes half a KB
// of shared memory); s_tiles[kTileGroups] = all of them.  Computed by the
// block's first 128 threads, 8 experts each; every thread calls it, and it ends
// with a barrier.  (Offsets whose ranges overlap can count a row more than once;
// sums are taken in 64 bits and held at 2^31 - 1, so that they stay in order.)
constexpr int kPerGroup = 8;
constexpr int kTileGroups = kMaxE / kPerGroup;
__device__ __forceinline__ int tile_count(int rows, int tile) {
    return (int)(((uint32_t)rows + tile - 1) / (uint32_t)tile);
}
__device__ __forceinline__ void tile_prefix(const MatmulArgs& a, int tile, int* s_tiles, long long* s_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    long long sum = 0, incl = 0;
    if (tid < kTileGroups) {
#pragma unroll
        for (int j = 0; j < kPerGroup; ++j) {
            const int e = tid * kPerGroup + j;
            int begin;
            sum += e < a.E ? tile_count(expert_rows(a, e, begin), tile) : 0;
        }
        incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const long long o = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) s_warp[warp] = incl;
    }
    __syncthreads();
    if (tid < kTileGroups) {
        long long run = incl - sum;
        for (int w = 0; w < warp; ++w) run += s_warp[w];
        s_tiles[tid] = (int)min(run, (long long)INT32_MAX);
        if (tid == kTileGroups - 1) s_tiles[kTileGroups] = (int)min(run + sum, (long long)INT32_MAX);
    }
    __syncthreads();
}

struct ExpertTile {
    int e, begin, rows;   // the expert, its first position in expert-major order, its rows
    int first, count;     // its first tile, its number of tiles
};

// Among the experts of group g, the one that owns tile t: s_tiles[g] <= t <
// s_tiles[g + 1].  Their offsets load together.
__device__ __forceinline__ ExpertTile expert_in_group(const MatmulArgs& a, int tile, const int* s_tiles, int g, int t) {
    int begin[kPerGroup], rows[kPerGroup];
#pragma unroll
    for (int j = 0; j < kPerGroup; ++j) {
        begin[j] = rows[j] = 0;
        if (g * kPerGroup + j < a.E) rows[j] = expert_rows(a, g * kPerGroup + j, begin[j]);
    }
    ExpertTile x = {g * kPerGroup, begin[0], rows[0], s_tiles[g], tile_count(rows[0], tile)};
#pragma unroll
    for (int j = 1; j < kPerGroup; ++j)
        if (t - x.first >= x.count && g * kPerGroup + j < a.E)
            x = {g * kPerGroup + j, begin[j], rows[j], x.first + x.count, tile_count(rows[j], tile)};
    return x;
}

// The expert that owns tile t < s_tiles[kTileGroups].
__device__ __forceinline__ ExpertTile expert_of_tile(const MatmulArgs& a, int tile, const int* s_tiles, int t) {
    int lo = 0, hi = kTileGroups;  // s_tiles[lo] <= t < s_tiles[hi]
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tiles[mid] <= t) lo = mid; else hi = mid;
    }
    return expert_in_group(a, tile, s_tiles, lo, t);
}

}  // namespace mm
}  // namespace ep
