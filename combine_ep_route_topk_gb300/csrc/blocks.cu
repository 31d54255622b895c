// Rows to E4M3 codes with a scale for every 128 columns and back, and SwiGLU's
// gradient from rows or from such codes, for sm_103a (ep_quantize_blocks,
// ep_dequantize_blocks, ep_swiglu_backward).
//
//   v      = x, or g / (1 + exp(-g)) * u with (g, u) the row's halves
//   scale  = max|v| / 448 over 128 columns (1 for zeros), code = E4M3(v / scale)
//   d_g    = d u s (1 + g (1 - s)),  d_u = d g s,  s = 1 / (1 + exp(-g))
//
// All three pass once over their rows.  A thread takes 16 columns, in accesses of
// 32 bytes: 8 threads share a block's maximum in registers.  Bound by those bytes,
// and where the codes are made nearly as much by instructions (186 a thread's 16
// columns, 56 to 67 % of the issue slots).  32768 rows of bf16: 7168 columns to codes
// 117 us = 6.0 TB/s and back 102 us = 6.9; SwiGLU of 2 x 2048 53 us = 6.3, with the
// checkpoint 90 = 5.2, its gradient from that 80 us = 6.7, from rows 92 = 7.3.  The same in
// float32: 88 us = 6.9 TB/s, with the checkpoint 109 = 6.8, the gradients 135 = 7.0 and
// 191 = 7.1.
#include <algorithm>

#include "rows_common.cuh"

namespace ep {
namespace {

using namespace rows;

constexpr int kThreads = 256;

// exp of a row's value.  Float32 rows: CUDA's own, within two last places.  bf16 rows: the
// hardware's 2^(x log2 e), off by some 2^-22 and, for the product's rounding, |x| 2^-23,
// relative, far below the 2^-8 of the value that it is taken of and of a bf16's rounding.
template <typename T>
__device__ __forceinline__ float exp_of(float x) {
    if constexpr (sizeof(T) == 4) return expf(x);
    float e;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(e) : "f"(x * 1.4426950408889634f));
    return e;
}
// 1 / x by the hardware's instruction, within a last place (0 below 2^-126).
__device__ __forceinline__ float fast_rcp(float x) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Item i of a kernel's thread: row i / pieces, columns 16 (i % pieces) and on.
struct Place {
    uint32_t row;
    int col;
};
__device__ __forceinline__ Place place(uint64_t i, uint32_t pieces) {
    Place p;
    if (i >> 32 == 0) {
        p.row = (uint32_t)i / pieces;
        p.col = (int)((uint32_t)i % pieces) * kVec;
    } else {
        p.row = (uint32_t)(i / pieces);
        p.col = (int)(i % pieces) * kVec;
    }
    return p;
}

// KEEP: also the codes of x, whose blocks lie on the halves' (cols a multiple of 128).  x
// stays as it lies in memory, so that registers allow 6, 5 or 4 blocks an SM (as float32,
// and 4 blocks with the checkpoint, 94 us where this takes 90; 57 and 53 without it).
template <typename T, bool SWIGLU, bool KEEP>
__global__ void __launch_bounds__(kThreads, !KEEP ? 6 : sizeof(T) == 2 ? 5 : 4) quantize_blocks_kernel(BlockQuantArgs a, Divisor per_row) {
    pdl_prologue();
    const int blocks = (int)per_row.d;
    // the block of 128 that this thread's 8 lanes hold, below 2^31 of them
    const uint32_t block = blockIdx.x * (kThreads / kLanes) + threadIdx.x / kLanes;
    Place p;
    p.row = per_row.divide(block);
    p.col = (int)((block - p.row * (uint32_t)blocks) * kScaleBlock + threadIdx.x % kLanes * kVec);
    // the lanes of a block decide together; all lanes take part in the maxima
    const bool row_on = p.row < (uint32_t)a.rows && holds_token(a.tokens, p.row);
    const bool on = row_on && p.col < a.cols;
    const size_t r = p.row;
    const T* row = static_cast<const T*>(a.x) + r * (SWIGLU ? 2 * (size_t)a.cols : (size_t)a.cols) + p.col;
    Raw<T> g, u;
    g.zero();
    u.zero();
    if (on) {
        g.load(row, a.wide);
        if constexpr (SWIGLU) u.load(row + a.cols, a.wide);
    }
    float v[kVec], scale;  // the values' negatives, as encode16 takes them
    g.negatives(v);
    if constexpr (KEEP) {
        const uint4 g_codes = encode16(v, scale);
        const size_t wide = 2 * (size_t)a.cols;
        if (on) {
            *reinterpret_cast<uint4*>(a.x_q + r * wide + p.col) = g_codes;
            if (p.col % kScaleBlock == 0) a.x_scales[r * 2 * blocks + p.col / kScaleBlock] = scale;
        }
        float w[kVec];
        u.negatives(w);
        const uint4 u_codes = encode16(w, scale);
        if (on) {
            *reinterpret_cast<uint4*>(a.x_q + r * wide + a.cols + p.col) = u_codes;
            if (p.col % kScaleBlock == 0) a.x_scales[r * 2 * blocks + blocks + p.col / kScaleBlock] = scale;
        }
    }
    if constexpr (SWIGLU) {
        if constexpr (KEEP) g.negatives(v);
#pragma unroll
        for (int j = 0; j < kVec; ++j) v[j] = v[j] * fast_rcp(1.0f + exp_of<T>(v[j])) * u.at(j);
    }
    const uint4 codes = encode16(v, scale);
    if (on) {
        *reinterpret_cast<uint4*>(a.q + r * a.cols + p.col) = codes;
        if (p.col % kScaleBlock == 0) a.scales[r * blocks + p.col / kScaleBlock] = scale;
    }
}

template <typename T>
__global__ void __launch_bounds__(kThreads) dequantize_blocks_kernel(BlockRestoreArgs a) {
    pdl_prologue();
    const int blocks = scale_blocks(a.cols);
    const Place p = place((uint64_t)blockIdx.x * kThreads + threadIdx.x, (uint32_t)(a.cols / kVec));
    if (p.row >= (uint32_t)a.rows || !holds_token(a.tokens, p.row)) return;
    const size_t r = p.row;
    const uint4 q = __ldcs(reinterpret_cast<const uint4*>(a.q + r * a.cols + p.col));
    float v[kVec];
    decode16(q, __ldg(a.scales + r * blocks + p.col / kScaleBlock), v);
    store16(static_cast<T*>(a.out) + r * a.cols + p.col, v, a.wide);
}

template <typename T, bool CODES>
__global__ void __launch_bounds__(kThreads) swiglu_backward_kernel(SwigluGradArgs a) {
    pdl_prologue();
    const Place p = place((uint64_t)blockIdx.x * kThreads + threadIdx.x, (uint32_t)(a.cols / kVec));
    if (p.row >= (uint32_t)a.rows || !holds_token(a.tokens, p.row)) return;
    const size_t r = p.row, wide = 2 * (size_t)a.cols;
    float g[kVec], u[kVec], d[kVec];
    load16<true>(static_cast<const T*>(a.d_out) + r * a.cols + p.col, d, a.wide);
    if constexpr (CODES) {
        const uint8_t* q = static_cast<const uint8_t*>(a.x) + r * wide + p.col;
        const float* s = a.x_scales + r * scale_blocks(2 * a.cols);
        const uint4 gq = __ldcs(reinterpret_cast<const uint4*>(q));
        const uint4 uq = __ldcs(reinterpret_cast<const uint4*>(q + a.cols));
        decode16(gq, __ldg(s + p.col / kScaleBlock), g);
        decode16(uq, __ldg(s + (a.cols + p.col) / kScaleBlock), u);
    } else {
        const T* x = static_cast<const T*>(a.x) + r * wide + p.col;
        load16<true>(x, g, a.wide);
        load16<true>(x + a.cols, u, a.wide);
    }
#pragma unroll
    for (int j = 0; j < kVec; ++j) {
        // s and 1 - s from exp(-|g|), so that neither cancels or overflows
        const float e = exp_of<T>(-fabsf(g[j])), big = fast_rcp(1.0f + e), small = e * big;
        const float s = g[j] >= 0.0f ? big : small, rest = g[j] >= 0.0f ? small : big;
        const float slope = s * fmaf(g[j], rest, 1.0f);
        const float up = d[j] * g[j] * s;
        g[j] = d[j] * u[j] * slope;
        u[j] = up;
    }
    T* out = static_cast<T*>(a.d_x) + r * wide + p.col;
    store16(out, g, a.wide);
    store16(out + a.cols, u, a.wide);
}

template <typename Args>
cudaError_t run(void (*kernel)(Args), const Args& a, uint64_t pieces, cudaStream_t s) {
    const uint64_t blocks = (pieces * (uint64_t)a.rows + kThreads - 1) / kThreads;
    const cudaError_t err = launch(kernel, dim3((unsigned)blocks), dim3(kThreads), 0, s, a);
    note_launch();
    return err;
}

cudaError_t run_quantize(void (*kernel)(BlockQuantArgs, Divisor), const BlockQuantArgs& a, cudaStream_t s) {
    const uint64_t blocks = (uint64_t)scale_blocks(a.cols) * a.rows, per = kThreads / kLanes;
    const cudaError_t err = launch(kernel, dim3((unsigned)((blocks + per - 1) / per)), dim3(kThreads), 0, s, a,
                                   Divisor((uint32_t)scale_blocks(a.cols)));
    note_launch();
    return err;
}

template <typename T>
cudaError_t quantize_t(const BlockQuantArgs& a, cudaStream_t s) {
    if (!a.swiglu) return run_quantize(quantize_blocks_kernel<T, false, false>, a, s);
    if (a.x_q == nullptr) return run_quantize(quantize_blocks_kernel<T, true, false>, a, s);
    if (a.cols % kScaleBlock == 0) return run_quantize(quantize_blocks_kernel<T, true, true>, a, s);
    // a block of x straddles the halves: its codes in a pass of their own, which reads the
    // rows again (32768 x 1440 bf16: 90 us, of 41 for the values and 51 for the checkpoint;
    // 524 MB, where one reading would leave 335)
    BlockQuantArgs kept = a;
    kept.cols = 2 * a.cols;
    kept.q = a.x_q;
    kept.scales = a.x_scales;
    const cudaError_t err = run_quantize(quantize_blocks_kernel<T, false, false>, kept, s);
    return err != cudaSuccess ? err : run_quantize(quantize_blocks_kernel<T, true, false>, a, s);
}

}  // namespace

cudaError_t launch_quantize_blocks(const BlockQuantArgs& args, cudaStream_t s) {
    if (args.rows == 0) return cudaSuccess;
    BlockQuantArgs a = args;
    a.wide = aligned32(a.x);
    return a.bf16 ? quantize_t<__nv_bfloat16>(a, s) : quantize_t<float>(a, s);
}

cudaError_t launch_dequantize_blocks(const BlockRestoreArgs& args, cudaStream_t s) {
    if (args.rows == 0) return cudaSuccess;
    BlockRestoreArgs a = args;
    a.wide = aligned32(a.out);
    const uint64_t pieces = a.cols / kVec;
    return a.bf16 ? run(dequantize_blocks_kernel<__nv_bfloat16>, a, pieces, s)
                  : run(dequantize_blocks_kernel<float>, a, pieces, s);
}

cudaError_t launch_swiglu_backward(const SwigluGradArgs& args, cudaStream_t s) {
    if (args.rows == 0) return cudaSuccess;
    SwigluGradArgs a = args;
    a.wide = aligned32(a.d_out, a.d_x, a.x_scales == nullptr ? a.x : nullptr);
    const uint64_t pieces = a.cols / kVec;
    if (a.x_scales != nullptr)
        return a.bf16 ? run(swiglu_backward_kernel<__nv_bfloat16, true>, a, pieces, s)
                      : run(swiglu_backward_kernel<float, true>, a, pieces, s);
    return a.bf16 ? run(swiglu_backward_kernel<__nv_bfloat16, false>, a, pieces, s)
                  : run(swiglu_backward_kernel<float, false>, a, pieces, s);
}

}  // namespace ep
