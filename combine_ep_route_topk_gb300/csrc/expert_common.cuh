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

// s_tiles[e] = exclusive prefix over the experts of ceil(rows_e / tile), by the
// block's first 256 threads (4 experts each); every thread calls it, and it
// ends with a barrier.
__device__ __forceinline__ void tile_prefix(const MatmulArgs& a, int tile, int* s_tiles, int* s_warp) {
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    constexpr int kPer = kMaxE / 256;
    int n[kPer], sum = 0, incl = 0;
    if (tid < 256) {
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = tid * kPer + j;
            int begin;
            n[j] = e < a.E ? (expert_rows(a, e, begin) + tile - 1) / tile : 0;
            sum += n[j];
        }
        incl = sum;
#pragma unroll
        for (int off = 1; off < 32; off <<= 1) {
            const int o = __shfl_up_sync(kFull, incl, off);
            if (lane >= off) incl += o;
        }
        if (lane == 31) s_warp[warp] = incl;
    }
    __syncthreads();
    if (tid < 256) {
        int run = incl - sum;
        for (int w = 0; w < warp; ++w) run += s_warp[w];
#pragma unroll
        for (int j = 0; j < kPer; ++j) {
            const int e = tid * kPer + j;
            if (e < a.E) s_tiles[e] = run;
            run += n[j];
            if (e == a.E - 1) s_tiles[a.E] = run;
        }
    }
    __syncthreads();
}

// The expert that owns tile t (s_tiles[e] <= t < s_tiles[e + 1]).
__device__ __forceinline__ int expert_of_tile(const int* s_tiles, int E, int t) {
    int lo = 0, hi = E;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (s_tiles[mid] <= t) lo = mid; else hi = mid;
    }
    return lo;
}

}  // namespace mm
}  // namespace ep
