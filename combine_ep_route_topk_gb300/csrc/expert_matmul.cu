// Experts' products in 8-bit integers for sm_103a, a few rows per expert
// (ep_expert_matmul; expert_matmul_tc.cu has the kernel for more).
//
//   out[r, n] = xs[r] * ws[e, n] * sum_k x[r, k] * w[e, n, k]
//
// The sum is an exact 32-bit integer (Kd <= 65536 keeps it below 2^31); the
// scales are applied in float32 and the output is rounded once.
//
// Bound by the weight bytes: each weight is read once and used for up to 8
// rows.  The (row group, channel) pairs lie on a line that is divided evenly
// among the warps of the grid, so that no SM ends much later than another; a
// warp takes two channels at a time, with 16-byte loads, two rounds of them in
// flight, and multiplies them by dp4a with the group's rows, which stay in L1.
// The row loop is compiled for 1, 2, 4 and 8 rows; that of 8 spills (48 registers a
// thread at 5 blocks an SM: 504 bytes stored, 672 loaded).  8 rows of as many experts
// (4096 x 7168, 235 MB): 39.4 us = 6.0 TB/s; with 4 or 6 blocks per SM 41.6 and
// 40.6 us, with 3 or 4 channels at a time 40.1 and 41.6 us.
#include "expert_common.cuh"

namespace ep {
namespace {

using namespace mm;

constexpr int kWarps = 8;
constexpr int kRows = 8;          // rows per group
constexpr int kBlocksPerSm = 5;
constexpr int kChannels = 2;      // a warp's, at a time

__device__ __forceinline__ void store_out(const MatmulArgs& a, size_t at, float v) {
    if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(v);
    else static_cast<float*>(a.out)[at] = v;
}

__device__ __forceinline__ int dot16(int4 a, int4 b, int acc) {
    acc = __dp4a(a.x, b.x, acc);
    acc = __dp4a(a.y, b.y, acc);
    acc = __dp4a(a.z, b.z, acc);
    return __dp4a(a.w, b.w, acc);
}

// Channels [n, end) of expert e for R rows; src: the lane's row of x (lanes
// 0 .. R-1), -1 for none.
template <int R>
__device__ __forceinline__ void channels(const MatmulArgs& a, int e, int n, int end, int src, int rows,
                                         size_t first, int lane) {
    constexpr int CH = kChannels;
    const int8_t* x[R];
#pragma unroll
    for (int r = 0; r < R; ++r) x[r] = a.x + (size_t)max(0, __shfl_sync(kFull, src, r)) * a.Kd;
    const float xs = src >= 0 ? __ldg(a.x_scales + src) : 0.0f;
    for (; n < end; n += CH) {
        const int8_t* w[CH];  // past the end, the last channel again: it is read from L1
#pragma unroll
        for (int c = 0; c < CH; ++c) w[c] = a.w + ((size_t)e * a.Nc + min(n + c, end - 1)) * a.Kd;
        int acc[CH][R];
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) acc[c][r] = 0;
        for (int k = lane * 16; k < a.Kd; k += 1024) {
            const bool more = k + 512 < a.Kd;
            int4 p[CH], q[CH];
#pragma unroll
            for (int c = 0; c < CH; ++c) {
                p[c] = __ldcs(reinterpret_cast<const int4*>(w[c] + k));
                q[c] = make_int4(0, 0, 0, 0);
                if (more) q[c] = __ldcs(reinterpret_cast<const int4*>(w[c] + k + 512));
            }
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int4 y = __ldg(reinterpret_cast<const int4*>(x[r] + k));
#pragma unroll
                for (int c = 0; c < CH; ++c) acc[c][r] = dot16(p[c], y, acc[c][r]);
            }
            if (more) {
#pragma unroll
                for (int r = 0; r < R; ++r) {
                    const int4 y = __ldg(reinterpret_cast<const int4*>(x[r] + k + 512));
#pragma unroll
                    for (int c = 0; c < CH; ++c) acc[c][r] = dot16(q[c], y, acc[c][r]);
                }
            }
        }
        // lane c * 8 + r takes the sum of (channel n + c, row r)
        int mine = 0;
#pragma unroll
        for (int c = 0; c < CH; ++c)
#pragma unroll
            for (int r = 0; r < R; ++r) {
                const int v = __reduce_add_sync(kFull, acc[c][r]);
                if (lane == c * kRows + r) mine = v;
            }
        const int r = lane % kRows, ch = n + lane / kRows;
        const float s = __shfl_sync(kFull, xs, r);
        if (lane < CH * kRows && r < rows && ch < end)
            store_out(a, (first + r) * a.Nc + ch, (float)mine * s * __ldg(a.w_scales + (size_t)e * a.Nc + ch));
    }
}

__global__ void __launch_bounds__(kWarps * 32, kBlocksPerSm)
matmul_rows_kernel(MatmulArgs a) {
    __shared__ int s_groups[kTileGroups + 1];  // prefix of the experts' row groups
    __shared__ long long s_warp[kTileGroups / 32];
    pdl_prologue();
    const int lane = threadIdx.x & 31;
    if (a.status != nullptr && blockIdx.x == 0 && threadIdx.x == 0) *a.status = 0;
    tile_prefix(a, kRows, s_groups, s_warp);

    // this warp's share of the line of (group, channel)
    const long long total = (long long)s_groups[kTileGroups] * a.Nc;
    const long long warps = (long long)gridDim.x * kWarps, w = (long long)(threadIdx.x >> 5) * gridDim.x + blockIdx.x;
    long long at = total / warps * w + min(w, total % warps);
    const long long stop = at + total / warps + (w < total % warps ? 1 : 0);
    while (at < stop) {
        const int group = (int)(at / a.Nc), n = (int)(at - (long long)group * a.Nc);
        const int end = (int)min((long long)a.Nc, n + (stop - at));
        at += end - n;
        const ExpertTile t = expert_of_tile(a, kRows, s_groups, group);
        const int first = (group - t.first) * kRows;
        const int rows = min(kRows, t.rows - first);
        // a row that reads nothing takes row 0 and the scale 0
        const int src = lane < rows && a.x_rows > 0 ? source_row(a, t.e, t.begin, first + lane) : -1;
        const size_t to = first_row(a, t.e, t.begin) + first;
        if (a.x_rows == 0) {  // nothing to read: rows of zeros
            for (int i = lane; i < rows * (end - n); i += 32)
                store_out(a, (to + i / (end - n)) * a.Nc + n + i % (end - n), 0.0f);
        } else if (rows == 1) {
            channels<1>(a, t.e, n, end, src, rows, to, lane);
        } else if (rows == 2) {
            channels<2>(a, t.e, n, end, src, rows, to, lane);
        } else if (rows <= 4) {
            channels<4>(a, t.e, n, end, src, rows, to, lane);
        } else {
            channels<8>(a, t.e, n, end, src, rows, to, lane);
        }
    }
}

}  // namespace

cudaError_t launch_expert_matmul(const MatmulArgs& a, cudaStream_t s) {
    if (a.rows == 0)
        return a.status != nullptr ? cudaMemsetAsync(a.status, 0, sizeof(int32_t), s) : cudaSuccess;
    // Few rows, most of them alone with their expert: this kernel.  It takes a time per
    // row; the tensor cores one per expert with rows, so that rows which pick
    // independently and meet count against it.  Mean of 20 draws, us, rows alone with
    // their expert / rows that pick independently (tensor cores in brackets):
    //   32 experts of 4096 x 7168:  8 rows 41 (47) / 39 (47), 12 60 (67) / 53 (60),
    //                               16 78 (87) / 68 (68)
    //   128 of 2880 x 1440:  32 rows 28 (34) / 27 (31), 48 38 (46) / 37 (39),
    //                        64 48 (59) / 48 (47)
    //   128 of 7168 x 2048:  48 rows 117 (117) / 112 (99), 64 154 (194) / 151 (151)
    //   256 of 4096 x 2048:  32 rows 48 (50) / 47 (48), 64 90 (91) / 94 (82),
    //                        96 133 (130) / 136 (110), 128 176 (169) / 177 (134)
    //   512 of 1024 x 2048:  64 rows 27 (31) / 27 (29), 128 49 (50) / 51 (44),
    //                        256 91 (90) / 94 (72)
    //   1024 of 512 x 1024:  128 rows 17 (18) / 17 (18), 512 52 (66) / 52 (53)
    // Past 64 rows that pick independently, large experts would so be faster on the
    // tensor cores (up to 25 %) and small ones slower; the rule does not tell them apart.
    // One expert of 4096 x 4096: 2 rows 8 (12), 4 rows 12 (12), 5 rows 22 (12).
    cudaError_t err;
    if (a.x_rows == 0 || a.rows <= 4 || 2ll * a.rows <= a.E) {
        err = launch(matmul_rows_kernel, dim3(sm_count() * kBlocksPerSm), dim3(kWarps * 32), 0, s, a);
    } else {
        err = launch_matmul_tc(a, s);
    }
    note_launch();
    return err;
}

}  // namespace ep
