// Root-mean-square norm of rows with the residual's addition, and its gradient,
// for sm_103a (ep_rms_norm, ep_rms_norm_backward).
//
//   z = x + residual, rounded to the rows' type;  r = 1 / sqrt(mean(z^2) + eps)
//   y = z r w, as rows and / or as E4M3 codes with a scale for every 128 columns
//   with n = z r and g = d_y w:
//   d_x = r (g - n mean(g n)) + d_residual,  d_w = sum over the rows of d_y n
//
// One pass: a block (a warp for short rows) holds its row in registers, joins the
// sum in shared memory and writes every output, so the bytes moved are the rows
// read and written.  Sums are float32, over at most 64 terms a thread and then a
// tree.  In the gradient a block takes rows blockIdx.x, + gridDim.x, ... with the
// same columns in a thread throughout, which sums d_w of its columns in
// registers; the blocks' sums are joined by a second kernel in a fixed order.
#include <algorithm>

#include "rows_common.cuh"

namespace ep {
namespace {

using namespace rows;

// Sum over the row's threads: whole warps, nt of them (NT at most), one warp
// without shared memory.  s_part: NT / 32 floats that nothing else uses until the
// block's next barrier but one.
template <int NT>
__device__ __forceinline__ float row_sum(float v, int nt, float* s_part) {
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    if constexpr (NT > 32) {
        if ((threadIdx.x & 31) == 0) s_part[threadIdx.x >> 5] = v;
        __syncthreads();
        v = 0.0f;
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
            if (w * 32 < nt) v += s_part[w];
    }
    return v;
}

template <bool STREAM>
__device__ __forceinline__ void load_weight(const NormArgs& a, int c, float (&w)[kVec]) {
    if (a.weight_bf16) load16<STREAM>(static_cast<const __nv_bfloat16*>(a.weight) + c, w);
    else load16<STREAM>(static_cast<const float*>(a.weight) + c, w);
}

__device__ __forceinline__ float rounded(float v, const __nv_bfloat16*) {
    return __bfloat162float(__float2bfloat16_rn(v));
}
__device__ __forceinline__ float rounded(float v, const float*) { return v; }

// Up to NT threads a row, whole warps, HELD vectors of 16 each; ROWS rows a block
// (more than 1: a warp each).
template <typename T, int NT, int ROWS, int HELD>
__global__ void __launch_bounds__(NT * ROWS) rms_norm_kernel(NormArgs a) {
    static_assert(ROWS == 1 || NT == 32, "a warp per row");
    __shared__ float s_part[NT / 32];
    pdl_prologue();
    const int nt = ROWS > 1 ? NT : (int)blockDim.x;
    const int tid = ROWS > 1 ? (int)threadIdx.x % NT : (int)threadIdx.x;
    const long long r = (long long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / NT : 0);
    if (r >= a.rows) return;  // a whole warp, or none of the block
    const size_t at = (size_t)r * a.cols;
    const T* x = static_cast<const T*>(a.x) + at;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + at : nullptr;
    float z[HELD][kVec];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * nt + tid) * kVec;
#pragma unroll
        for (int j = 0; j < kVec; ++j) z[i][j] = 0.0f;
        if (c < a.cols) {
            load16<true>(x + c, z[i]);
            if (res != nullptr) {
                float t[kVec];
                load16<true>(res + c, t);
#pragma unroll
                for (int j = 0; j < kVec; ++j) z[i][j] = rounded(z[i][j] + t[j], x);
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum = fmaf(z[i][j], z[i][j], sum);
    }
    if (a.residual_out != nullptr) {
        T* to = static_cast<T*>(a.residual_out) + at;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < a.cols) store16(to + c, z[i]);
        }
    }
    sum = row_sum<NT>(sum, nt, s_part);
    const float rstd = __fdiv_rn(1.0f, __fsqrt_rn(__fdiv_rn(sum, (float)a.cols) + a.eps));
    if (tid == 0 && a.rstd != nullptr) a.rstd[r] = rstd;
    if (a.y == nullptr && a.q == nullptr) return;
    const int blocks = scale_blocks(a.cols);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * nt + tid) * kVec;
        if (c < a.cols) {
            float w[kVec];
            load_weight<false>(a, c, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) z[i][j] = z[i][j] * rstd * w[j];
            if (a.y != nullptr) store16(static_cast<T*>(a.y) + at + c, z[i]);
        }
        if (a.q != nullptr) {  // every lane takes part in the blocks' maxima
            float scale;
            const uint4 codes = encode16(z[i], scale);
            if (c < a.cols) {
                *reinterpret_cast<uint4*>(a.q + at + c) = codes;
                if (c % kScaleBlock == 0) a.scales[(size_t)r * blocks + c / kScaleBlock] = scale;
            }
        }
    }
}

template <typename T, int NT, int ROWS, int HELD>
cudaError_t norm_shape(const NormArgs& a, cudaStream_t s) {
    const int vectors = (a.cols + kVec - 1) / kVec;
    const int nt = ROWS > 1 ? NT : std::min(NT, ((vectors + HELD - 1) / HELD + 31) / 32 * 32);
    return launch(rms_norm_kernel<T, NT, ROWS, HELD>, dim3((unsigned)((a.rows + ROWS - 1ll) / ROWS)),
                  dim3(nt * ROWS), 0, s, a);
}

template <typename T>
cudaError_t norm_t(const NormArgs& a, cudaStream_t s) {
    if (a.cols <= 512) return norm_shape<T, 32, 8, 1>(a, s);
    if (a.cols <= 1024) return norm_shape<T, 32, 4, 2>(a, s);
    if (a.cols <= 4096) return norm_shape<T, 256, 1, 1>(a, s);
    if (a.cols <= 8192) return norm_shape<T, 256, 1, 2>(a, s);
    return norm_shape<T, 512, 1, 2>(a, s);
}

// ---- gradient --------------------------------------------------------------------

constexpr int kGradVec = 8;
constexpr int kGradWarps = 8;  // warps of a block whose warps take a row each

__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[kGradVec]) {
    unpack8(__ldcs(reinterpret_cast<const uint4*>(p)), v);
}
__device__ __forceinline__ void load8(const float* p, float (&v)[kGradVec]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p)), b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w; v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}
__device__ __forceinline__ void store8(__nv_bfloat16* p, const float (&v)[kGradVec]) {
    *reinterpret_cast<uint4*>(p) = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
}
__device__ __forceinline__ void store8(float* p, const float (&v)[kGradVec]) {
    reinterpret_cast<float4*>(p)[0] = make_float4(v[0], v[1], v[2], v[3]);
    reinterpret_cast<float4*>(p)[1] = make_float4(v[4], v[5], v[6], v[7]);
}

template <typename T, int NT, int ROWS, int HELD>
__global__ void __launch_bounds__(NT * ROWS) rms_norm_backward_kernel(NormGradArgs a) {
    static_assert(ROWS == 1 || NT == 32, "a warp per row");
    __shared__ float s_part[2][NT / 32];
    extern __shared__ float s_dw[];  // ROWS > 1: [ROWS][cols]
    pdl_prologue();
    const int nt = ROWS > 1 ? NT : (int)blockDim.x;
    const int tid = ROWS > 1 ? (int)threadIdx.x % NT : (int)threadIdx.x;
    const int sub = ROWS > 1 ? (int)threadIdx.x / NT : 0;
    float dw[HELD][kGradVec];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
#pragma unroll
        for (int j = 0; j < kGradVec; ++j) dw[i][j] = 0.0f;
    int turn = 0;
    for (long long r = (long long)blockIdx.x * ROWS + sub; r < a.rows; r += (long long)gridDim.x * ROWS) {
        const size_t at = (size_t)r * a.cols;
        const float rstd = __ldg(a.rstd + r);
        float n[HELD][kGradVec], g[HELD][kGradVec];
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kGradVec;
            if (c < a.cols) {
                load8(static_cast<const T*>(a.z) + at + c, n[i]);
                load8(static_cast<const T*>(a.d_y) + at + c, g[i]);
            } else {
#pragma unroll
                for (int j = 0; j < kGradVec; ++j) n[i][j] = g[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kGradVec;
            if (c < a.cols) {
                float w[kGradVec];
                if (a.weight_bf16) {
                    unpack8(__ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.weight) + c)), w);
                } else {
                    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.weight) + c);
                    const float4 lo = __ldg(p), hi = __ldg(p + 1);
                    w[0] = lo.x; w[1] = lo.y; w[2] = lo.z; w[3] = lo.w;
                    w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
                }
#pragma unroll
                for (int j = 0; j < kGradVec; ++j) {
                    n[i][j] *= rstd;
                    dw[i][j] = fmaf(g[i][j], n[i][j], dw[i][j]);
                    g[i][j] *= w[j];
                    sum = fmaf(g[i][j], n[i][j], sum);
                }
            }
        }
        // two buffers in turn: a warp may be one row ahead of another
        sum = row_sum<NT>(sum, nt, s_part[turn]);
        turn ^= 1;
        const float mean = __fdiv_rn(sum, (float)a.cols);
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kGradVec;
            if (c < a.cols) {
                float d[kGradVec];
#pragma unroll
                for (int j = 0; j < kGradVec; ++j) d[j] = 0.0f;
                if (a.d_residual != nullptr) load8(static_cast<const T*>(a.d_residual) + at + c, d);
#pragma unroll
                for (int j = 0; j < kGradVec; ++j) d[j] = fmaf(rstd, fmaf(-n[i][j], mean, g[i][j]), d[j]);
                store8(static_cast<T*>(a.d_x) + at + c, d);
            }
        }
    }
    if (a.d_weight == nullptr) return;
    float* to = a.partial + (size_t)blockIdx.x * a.cols;
    if constexpr (ROWS > 1) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kGradVec;
            if (c < a.cols) store8(s_dw + (size_t)sub * a.cols + c, dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += NT * ROWS) {
            float v = 0.0f;
            for (int k = 0; k < ROWS; ++k) v += s_dw[(size_t)k * a.cols + c];
            to[c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kGradVec;
            if (c < a.cols) store8(to + c, dw[i]);
        }
    }
}

// Sum of the blocks' partial sums: 32 columns a block, 32 strands of partial sums
// each, joined in a fixed order.
__global__ void __launch_bounds__(1024) weight_grad_kernel(NormGradArgs a, int parts) {
    __shared__ float s[32][33];
    pdl_prologue();
    const int lane = threadIdx.x & 31, strand = threadIdx.x >> 5, c = blockIdx.x * 32 + lane;
    float v = 0.0f;
    if (c < a.cols)
        for (int p = strand; p < parts; p += 32) v += __ldcs(a.partial + (size_t)p * a.cols + c);
    s[strand][lane] = v;
    __syncthreads();
    v = s[lane][strand];
#pragma unroll
    for (int off = 16; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    if (lane == 0 && blockIdx.x * 32 + strand < (unsigned)a.cols) a.d_weight[blockIdx.x * 32 + strand] = v;
}

template <typename T, int NT, int ROWS, int HELD>
cudaError_t grad_shape(const NormGradArgs& a, cudaStream_t s) {
    const int vectors = (a.cols + kGradVec - 1) / kGradVec;
    const int nt = ROWS > 1 ? NT : std::min(NT, ((vectors + HELD - 1) / HELD + 31) / 32 * 32);
    const size_t smem = ROWS > 1 ? (size_t)ROWS * a.cols * sizeof(float) : 0;
    return launch(rms_norm_backward_kernel<T, NT, ROWS, HELD>, dim3(norm_grad_blocks(a.rows, a.cols)),
                  dim3(nt * ROWS), smem, s, a);
}

template <typename T>
cudaError_t grad_t(const NormGradArgs& a, cudaStream_t s) {
    if (a.cols <= 256) return grad_shape<T, 32, kGradWarps, 1>(a, s);
    if (a.cols <= 512) return grad_shape<T, 32, kGradWarps, 2>(a, s);
    if (a.cols <= 2048) return grad_shape<T, 256, 1, 1>(a, s);
    if (a.cols <= 4096) return grad_shape<T, 256, 1, 2>(a, s);
    if (a.cols <= 8192) return grad_shape<T, 512, 1, 2>(a, s);
    return grad_shape<T, 512, 1, 4>(a, s);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& a, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    const cudaError_t err = a.bf16 ? norm_t<__nv_bfloat16>(a, s) : norm_t<float>(a, s);
    note_launch();
    return err;
}

int norm_grad_blocks(int rows, int cols) {
    const int per = cols <= 512 ? kGradWarps : 1;
    return (int)std::min<long long>(2ll * sm_count(), ((long long)rows + per - 1) / per);
}

cudaError_t launch_rms_norm_backward(const NormGradArgs& a, cudaStream_t s) {
    if (a.rows == 0)
        return a.d_weight != nullptr ? cudaMemsetAsync(a.d_weight, 0, (size_t)a.cols * sizeof(float), s) : cudaSuccess;
    cudaError_t err = a.bf16 ? grad_t<__nv_bfloat16>(a, s) : grad_t<float>(a, s);
    note_launch();
    if (err != cudaSuccess || a.d_weight == nullptr) return err;
    err = launch(weight_grad_kernel, dim3((a.cols + 31) / 32), dim3(1024), 0, s, a, norm_grad_blocks(a.rows, a.cols));
    note_launch();
    return err;
}

}  // namespace ep
