// Quantisation of activation rows to 8-bit integers for sm_103a
// (ep_quantize_rows), optionally of the SwiGLU of a row's two halves.
//
//   v_c   = x_c, or x_c / (1 + exp(-x_c)) * x_{c+cols}
//   scale = max_c |v_c| / 127      (1 for a row of zeros)
//   q_c   = round-to-nearest-even(v_c * (127 / max|v|))
//
// One pass over the row: a block holds its values in registers, reduces the
// maximum and writes the codes, so the bytes moved are the row read and the
// codes written (HBM-bound).  The values, the maximum and the scale are
// float32; the code is the only rounding to fewer bits.
#include <cuda_bf16.h>

#include "ep_kernels.cuh"

namespace ep {
namespace {

// Eight consecutive elements.
__device__ __forceinline__ void load8(const __nv_bfloat16* p, float (&v)[8]) {
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(p));
    const uint32_t x[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int j = 0; j < 4; ++j) {
        v[2 * j] = __uint_as_float(x[j] << 16);
        v[2 * j + 1] = __uint_as_float(x[j] & 0xffff0000u);
    }
}
__device__ __forceinline__ void load8(const float* p, float (&v)[8]) {
    const float4 a = __ldcs(reinterpret_cast<const float4*>(p));
    const float4 b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    v[0] = a.x; v[1] = a.y; v[2] = a.z; v[3] = a.w;
    v[4] = b.x; v[5] = b.y; v[6] = b.z; v[7] = b.w;
}

template <typename T, bool SWIGLU>
__device__ __forceinline__ void values8(const T* row, int cols, int c, float (&v)[8]) {
    load8(row + c, v);
    if constexpr (SWIGLU) {
        float u[8];
        load8(row + cols + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) v[j] = __fdiv_rn(v[j], 1.0f + expf(-v[j])) * u[j];
    }
}

__device__ __forceinline__ uint32_t code(float v, float inv) {
    const int q = __float2int_rn(v * inv);  // NaN -> 0
    return (uint32_t)max(-127, min(127, q)) & 0xffu;
}

__device__ __forceinline__ void store8(int8_t* p, const float (&v)[8], float inv) {
    uint2 q;
    q.x = code(v[0], inv) | code(v[1], inv) << 8 | code(v[2], inv) << 16 | code(v[3], inv) << 24;
    q.y = code(v[4], inv) | code(v[5], inv) << 8 | code(v[6], inv) << 16 | code(v[7], inv) << 24;
    *reinterpret_cast<uint2*>(p) = q;
}

// NT threads per row; HELD > 0: the row fits HELD vectors of 8 a thread, held
// in registers; HELD == 0: any length, the values computed twice.
template <typename T, bool SWIGLU, int NT, int HELD>
__global__ void __launch_bounds__(NT) quantize_kernel(QuantArgs a) {
    __shared__ float s_max[NT / 32];
    pdl_prologue();
    const long long r = blockIdx.x;
    if (a.expert_offsets != nullptr) {  // block-uniform: rows that hold no token
        if (a.layout == 0) {
            if (r >= __ldg(a.expert_offsets + a.E)) return;
        } else {
            const int e = (int)(r / a.cap), slot = (int)(r % a.cap);
            if (slot >= __ldg(a.expert_offsets + e + 1) - __ldg(a.expert_offsets + e)) return;
        }
    }
    const int wide = SWIGLU ? 2 * a.cols : a.cols;
    const T* row = static_cast<const T*>(a.x) + r * wide;
    int8_t* out = a.q + r * a.cols;
    constexpr int H = HELD > 0 ? HELD : 1;
    float v[H][8];
    float top = 0.0f;
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int c = (i * NT + threadIdx.x) * 8;
            if (c < a.cols) {
                values8<T, SWIGLU>(row, a.cols, c, v[i]);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.0f;
            }
        }
#pragma unroll
        for (int i = 0; i < H; ++i)
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[i][j]));
    } else {
        for (int c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
            values8<T, SWIGLU>(row, a.cols, c, v[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = fmaxf(top, fabsf(v[0][j]));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, off));
    if ((threadIdx.x & 31) == 0) s_max[threadIdx.x >> 5] = top;
    __syncthreads();
#pragma unroll
    for (int w = 0; w < NT / 32; ++w) top = fmaxf(top, s_max[w]);
    const float inv = top > 0.0f ? __fdiv_rn(127.0f, top) : 1.0f;
    if (threadIdx.x == 0) a.scales[r] = top > 0.0f ? __fdiv_rn(top, 127.0f) : 1.0f;
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int c = (i * NT + threadIdx.x) * 8;
            if (c < a.cols) store8(out + c, v[i], inv);
        }
    } else {
        for (int c = threadIdx.x * 8; c < a.cols; c += NT * 8) {
            values8<T, SWIGLU>(row, a.cols, c, v[0]);
            store8(out + c, v[0], inv);
        }
    }
}

template <typename T, bool SWIGLU>
cudaError_t launch_quantize_t(const QuantArgs& a, cudaStream_t s) {
    const dim3 grid((unsigned)a.rows);
    if (a.cols <= 1024)
        return launch(quantize_kernel<T, SWIGLU, 128, 1>, grid, dim3(128), 0, s, a);
    if (a.cols <= 2048)
        return launch(quantize_kernel<T, SWIGLU, 128, 2>, grid, dim3(128), 0, s, a);
    if (a.cols <= 4096)
        return launch(quantize_kernel<T, SWIGLU, 256, 2>, grid, dim3(256), 0, s, a);
    if (a.cols <= 8192)
        return launch(quantize_kernel<T, SWIGLU, 256, 4>, grid, dim3(256), 0, s, a);
    return launch(quantize_kernel<T, SWIGLU, 256, 0>, grid, dim3(256), 0, s, a);
}

}  // namespace

cudaError_t launch_quantize(const QuantArgs& a, cudaStream_t s) {
    if (a.rows == 0) return cudaSuccess;
    cudaError_t err;
    if (a.bf16)
        err = a.swiglu ? launch_quantize_t<__nv_bfloat16, true>(a, s)
                       : launch_quantize_t<__nv_bfloat16, false>(a, s);
    else
        err = a.swiglu ? launch_quantize_t<float, true>(a, s) : launch_quantize_t<float, false>(a, s);
    note_launch();
    return err;
}

}  // namespace ep
