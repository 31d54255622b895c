// Experts' products in 8-bit integers for sm_103a (ep_expert_matmul).
//
//   out[r, n] = xs[r] * ws[e, n] * sum_k x[r, k] * w[e, n, k]
//
// for the rows r of expert e.  The sum is an exact 32-bit integer (Kd <= 65536
// keeps it below 2^31); the scales are applied in float32 and the output is
// rounded once.
//
// A work unit is (expert, group of up to 8 of its rows, 32 channels): each of
// the block's 8 warps owns 4 channels, streams their weights with 16-byte
// loads and multiplies them with the group's rows, staged in shared memory,
// by dp4a.  Bound by the weight bytes while the experts have few rows.
#include "expert_common.cuh"

namespace ep {
namespace {

using namespace mm;

constexpr int kWarps = 8;
constexpr int kRows = 8;       // rows per unit
constexpr int kChannels = 4;   // channels per warp
constexpr int kChunk = 2048;   // bytes of a row staged at a time

__device__ __forceinline__ void store_out(const MatmulArgs& a, size_t at, float v) {
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.out)[at] = v;
}

__global__ void __launch_bounds__(kWarps * 32)
matmul_rows_kernel(MatmulArgs a) {
    __shared__ int s_units[kMaxE + 1];  // exclusive prefix of the experts' row groups
    __shared__ int s_warp[kWarps];
    __shared__ __align__(16) int8_t s_x[kRows][kChunk];
    __shared__ int s_src[kRows];
    pdl_prologue();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    if (a.status != nullptr && blockIdx.x == 0 && tid == 0) *a.status = 0;
    tile_prefix(a, kRows, s_units, s_warp);

    const int blocks_n = (a.Nc + kWarps * kChannels - 1) / (kWarps * kChannels);
    const long long units = (long long)s_units[a.E] * blocks_n;
    for (long long u = blockIdx.x; u < units; u += gridDim.x) {
        const int group = (int)(u / blocks_n), nb = (int)(u % blocks_n);
        const int e = expert_of_tile(s_units, a.E, group);
        int begin;
        const int rows_e = expert_rows(a, e, begin);
        const int first = (group - s_units[e]) * kRows;
        const int rows = min(kRows, rows_e - first);
        if (tid < kRows) s_src[tid] = tid < rows ? source_row(a, e, begin, first + tid) : -1;
        const int n0 = (nb * kWarps + warp) * kChannels;
        int acc[kChannels][kRows];
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int r = 0; r < kRows; ++r) acc[c][r] = 0;
        for (int k0 = 0; k0 < a.Kd; k0 += kChunk) {
            const int len = min(kChunk, a.Kd - k0);  // a multiple of 16
            __syncthreads();
            for (int i = tid * 16; i < kRows * kChunk; i += kWarps * 32 * 16) {
                const int r = i / kChunk, k = i % kChunk;
                int4 q = make_int4(0, 0, 0, 0);
                if (k < len && s_src[r] >= 0)
                    q = __ldg(reinterpret_cast<const int4*>(a.x + (size_t)s_src[r] * a.Kd + k0 + k));
                *reinterpret_cast<int4*>(&s_x[r][k]) = q;
            }
            __syncthreads();
            for (int k = lane * 16; k < len; k += 512) {
                int4 w[kChannels];
#pragma unroll
                for (int c = 0; c < kChannels; ++c)
                    w[c] = n0 + c < a.Nc
                        ? __ldg(reinterpret_cast<const int4*>(
                              a.w + ((size_t)e * a.Nc + n0 + c) * a.Kd + k0 + k))
                        : make_int4(0, 0, 0, 0);
#pragma unroll
                for (int r = 0; r < kRows; ++r) {
                    const int4 x = *reinterpret_cast<const int4*>(&s_x[r][k]);
#pragma unroll
                    for (int c = 0; c < kChannels; ++c) {
                        acc[c][r] = __dp4a(w[c].x, x.x, acc[c][r]);
                        acc[c][r] = __dp4a(w[c].y, x.y, acc[c][r]);
                        acc[c][r] = __dp4a(w[c].z, x.z, acc[c][r]);
                        acc[c][r] = __dp4a(w[c].w, x.w, acc[c][r]);
                    }
                }
            }
        }
        // lane c * 8 + r takes the sum of (channel c, row r)
        int mine = 0;
#pragma unroll
        for (int c = 0; c < kChannels; ++c)
#pragma unroll
            for (int r = 0; r < kRows; ++r) {
                const int v = __reduce_add_sync(kFull, acc[c][r]);
                if (lane == c * kRows + r) mine = v;
            }
        const int r = lane % kRows, ch = n0 + lane / kRows;
        if (r < rows && ch < a.Nc) {
            const int src = s_src[r];
            const float xs = src >= 0 ? __ldg(a.x_scales + src) : 0.0f;
            const size_t to = first_row(a, e, begin) + first + r;
            store_out(a, to * a.Nc + ch, (float)mine * xs * __ldg(a.w_scales + (size_t)e * a.Nc + ch));
        }
        __syncthreads();  // s_src is rewritten by the next unit
    }
}

}  // namespace

cudaError_t launch_expert_matmul(const MatmulArgs& a, cudaStream_t s) {
    if (a.rows == 0)
        return a.status != nullptr ? cudaMemsetAsync(a.status, 0, sizeof(int32_t), s) : cudaSuccess;
    const int per = a.layout == 0 ? (a.rows + a.E - 1) / a.E : a.cap;  // rows per expert
    cudaError_t err;
    if (per <= 2 || a.x_rows == 0)
        err = launch(matmul_rows_kernel, dim3(sm_count() * 4), dim3(kWarps * 32), 0, s, a);
    else
        err = launch_matmul_tc(a, per, s);
    note_launch();
    return err;
}

}  // namespace ep
