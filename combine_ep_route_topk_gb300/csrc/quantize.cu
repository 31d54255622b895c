// Quantisation of activation rows to 8-bit integers for sm_103a
// (ep_quantize_rows), optionally of the SwiGLU of a row's two halves.
//
//   v_c   = x_c, or x_c / (1 + exp(-x_c)) * x_{c+cols}
//   scale = max_c |v_c| / 127      (1 for a row of zeros; not finite, with codes
//           of 0, where a v is not: the products of such a row are NaN)
//   q_c   = round-to-nearest-even(v_c * (127 / max|v|)), quotient and product
//           each rounded to float32
//
// One pass over the row: a block (a warp for short rows) holds its values in
// registers, reduces the maximum and writes the codes, so the bytes moved are
// the row read and the codes written (HBM-bound).  The values, the maximum and
// the scale are float32; the code is the only rounding to fewer bits.
#include <cuda_bf16.h>

#include <algorithm>
#include <cfloat>

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

// SwiGLU's exponential and quotient by the hardware's exp2 and reciprocal: the
// product with log2 e rounds at 2^-24 of |x| and each result at about 2^-23,
// together far below the 1/254 of the row's maximum that a code rounds.
template <typename T, bool SWIGLU>
__device__ __forceinline__ void values8(const T* row, int cols, int c, float (&v)[8]) {
    load8(row + c, v);
    if constexpr (SWIGLU) {
        float u[8];
        load8(row + cols + c, u);
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float e, inv;
            asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(v[j] * -1.4426950408889634f));
            asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(inv) : "f"(1.0f + e));
            v[j] = v[j] * inv * u[j];
        }
    }
}

// Four codes: with 1.5 * 2^23 added, a float32 of magnitude up to 127 is rounded
// to the nearest integer (ties to even), which is its lowest byte.  The product is
// rounded to float32 first: in one fused step the error of inv would decide the
// products that lie exactly between two codes (0.07 % of the codes of bf16 rows).
// Products are taken two an instruction, sums one by one: a sum of two would be
// fused with them.  32768 x 7168 bf16: 106.7 us as in one step, 109.6 with single
// products.
__device__ __forceinline__ void codes2(float x, float y, float inv, uint32_t& a, uint32_t& b) {
    float p, q;
    asm("{\n.reg .b64 v, f;\nmov.b64 v, {%2, %3};\nmov.b64 f, {%4, %4};\n"
        "mul.rn.f32x2 v, v, f;\nmov.b64 {%0, %1}, v;\n}\n"
        : "=f"(p), "=f"(q) : "f"(x), "f"(y), "f"(inv));
    a = __float_as_uint(__fadd_rn(p, 12582912.0f));
    b = __float_as_uint(__fadd_rn(q, 12582912.0f));
}
__device__ __forceinline__ uint32_t codes4(const float* v, float inv) {
    uint32_t a, b, c, d;
    codes2(v[0], v[1], inv, a, b);
    codes2(v[2], v[3], inv, c, d);
    return __byte_perm(__byte_perm(a, b, 0x0040), __byte_perm(c, d, 0x0040), 0x5410);
}

__device__ __forceinline__ void store8(int8_t* p, const float (&v)[8], float inv) {
    *reinterpret_cast<uint2*>(p) = make_uint2(codes4(v, inv), codes4(v + 4, inv));
}

__device__ __forceinline__ void scale8(float (&v)[8], float f) {
#pragma unroll
    for (int j = 0; j < 8; ++j) v[j] *= f;
}

// The larger one; NaN where either is, so that a NaN reaches the row's scale.
__device__ __forceinline__ float max_nan(float a, float b) {
    float m;
    asm("max.NaN.f32 %0, %1, %2;" : "=f"(m) : "f"(a), "f"(b));
    return m;
}

// Whether row r holds a token.
__device__ __forceinline__ bool holds_token(const QuantArgs& a, long long r) {
    if (a.expert_offsets == nullptr) return true;
    if (a.layout == 0) return r < __ldg(a.expert_offsets + a.E);
    const int e = (int)(r / a.cap), slot = (int)(r % a.cap);
    return slot < __ldg(a.expert_offsets + e + 1) - __ldg(a.expert_offsets + e);
}

// Up to NT threads per row, whole warps, and ROWS rows per block (ROWS > 1: a warp
// each); HELD > 0: the row fits HELD vectors of 8 a thread, held in registers;
// HELD == 0: any length, the values computed twice.
template <typename T, bool SWIGLU, int NT, int ROWS, int HELD>
__global__ void __launch_bounds__(NT * ROWS) quantize_kernel(QuantArgs a) {
    static_assert(ROWS == 1 || NT == 32, "a warp per row");
    pdl_prologue();
    const int nt = ROWS > 1 ? NT : (int)blockDim.x;  // threads of a row
    const int tid = ROWS > 1 ? (int)threadIdx.x % NT : (int)threadIdx.x;
    const long long r = (long long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / NT : 0);
    if (r >= a.rows || !holds_token(a, r)) return;  // uniform over the row's threads
    const int wide = SWIGLU ? 2 * a.cols : a.cols;
    const T* row = static_cast<const T*>(a.x) + r * wide;
    int8_t* out = a.q + r * a.cols;
    constexpr int H = HELD > 0 ? HELD : 1;
    float v[H][8];
    float top = 0.0f;
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int c = (i * nt + tid) * 8;
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
            for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(v[i][j]));
    } else {
        for (int c = tid * 8; c < a.cols; c += nt * 8) {
            values8<T, SWIGLU>(row, a.cols, c, v[0]);
#pragma unroll
            for (int j = 0; j < 8; ++j) top = max_nan(top, fabsf(v[0][j]));
        }
    }
#pragma unroll
    for (int off = 16; off > 0; off >>= 1)
        top = max_nan(top, __shfl_xor_sync(0xffffffffu, top, off));
    if constexpr (NT > 32) {
        __shared__ float s_max[NT / 32];
        if ((tid & 31) == 0) s_max[tid >> 5] = top;
        __syncthreads();
#pragma unroll
        for (int w = 0; w < NT / 32; ++w)
            if (w * 32 < nt) top = max_nan(top, s_max[w]);
    }
    // a row whose largest value is below 1e-30 is scaled up first: 127 / top would
    // leave the range of a float32
    const float up = top < 1e-30f ? 0x1p96f : 1.0f;
    const float inv = top > 0.0f ? __fdiv_rn(127.0f, top * up) : 1.0f;
    if (tid == 0) a.scales[r] = top == 0.0f ? 1.0f : __fdiv_rn(top, 127.0f);
    if (!(top <= FLT_MAX)) {  // uniform over the row
        for (int c = tid * 8; c < a.cols; c += nt * 8) *reinterpret_cast<uint2*>(out + c) = make_uint2(0, 0);
        return;
    }
    if constexpr (HELD > 0) {
#pragma unroll
        for (int i = 0; i < H; ++i) {
            const int c = (i * nt + tid) * 8;
            if (up != 1.0f) scale8(v[i], up);  // uniform over the row
            if (c < a.cols) store8(out + c, v[i], inv);
        }
    } else {
        for (int c = tid * 8; c < a.cols; c += nt * 8) {
            values8<T, SWIGLU>(row, a.cols, c, v[0]);
            if (up != 1.0f) scale8(v[0], up);
            store8(out + c, v[0], inv);
        }
    }
}

template <typename T, bool SWIGLU, int NT, int ROWS, int HELD>
cudaError_t launch_shape(const QuantArgs& a, cudaStream_t s) {
    const int vectors = (a.cols + 7) / 8, held = HELD > 0 ? HELD : 1;
    const int nt = ROWS > 1 ? NT : std::min(NT, ((vectors + held - 1) / held + 31) / 32 * 32);
    return launch(quantize_kernel<T, SWIGLU, NT, ROWS, HELD>, dim3((unsigned)((a.rows + ROWS - 1ll) / ROWS)),
                  dim3(nt * ROWS), 0, s, a);
}

// Measured on a GB300 (bf16, us; floor at the measured copy rate): 32768 x 7168
// 105.4 (105), with 256 threads for its 224 x 4 vectors 111.2; 8192 x 9216 37.5
// (34), with 512 threads for 288 54.8; SwiGLU 32768 x 2048 54.1 (50), with 64 and
// 256 threads a row 59.1 and 56.2.  A warp a row: 65536 x 1024 28.1 (30), with
// 128 threads 66.1 (a block a nanosecond is what the chip starts); 32768 x 1440
// 18.6 (21), with 96 threads 33.3, but SwiGLU of 65536 x 1440 97.7 against 78.4
// (71), and one token's 8 rows 2.1 against 1.5.  Four vectors a thread: 32768 x
// 4096 59.5 (60), with two 70.3, but SwiGLU of them 118.0 against 111.8 (100).
template <typename T, bool SWIGLU>
cudaError_t launch_quantize_t(const QuantArgs& a, cudaStream_t s) {
    if (a.cols <= 256) return launch_shape<T, SWIGLU, 32, 8, 1>(a, s);
    if (a.cols <= 512) return launch_shape<T, SWIGLU, 32, 8, 2>(a, s);
    if (a.cols <= 1024 && a.rows >= 4096) return launch_shape<T, SWIGLU, 32, 4, 4>(a, s);
    if constexpr (!SWIGLU)
        if (a.cols <= 1536 && a.rows >= 4096) return launch_shape<T, SWIGLU, 32, 4, 6>(a, s);
    if (a.cols <= 1024) return launch_shape<T, SWIGLU, 128, 1, 1>(a, s);
    if (a.cols <= 2048) return launch_shape<T, SWIGLU, 128, 1, 2>(a, s);
    if constexpr (!SWIGLU)
        if (a.cols <= 4096 && a.rows >= 4096) return launch_shape<T, SWIGLU, 128, 1, 4>(a, s);
    if (a.cols <= 4096) return launch_shape<T, SWIGLU, 256, 1, 2>(a, s);
    if (a.cols <= 8192) return launch_shape<T, SWIGLU, 256, 1, 4>(a, s);
    if (a.cols <= 16384) return launch_shape<T, SWIGLU, 512, 1, 4>(a, s);
    return launch_shape<T, SWIGLU, 512, 1, 0>(a, s);
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
