// Rows of bf16 or float32 and their E4M3 codes with a scale for every 128 columns
// (the form that ep_dispatch writes), shared by the kernels that make and read
// them (blocks.cu, norm.cu).  A thread takes 16 consecutive columns, eight threads
// a block of 128; a row's last block may be shorter.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <cuda_fp8.h>

#include "ep_kernels.cuh"

namespace ep {
namespace rows {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kVec = 16;       // columns of a thread
constexpr int kLanes = kScaleBlock / kVec;

__device__ __forceinline__ float lo_of(uint32_t w) { return __uint_as_float(w << 16); }
__device__ __forceinline__ float hi_of(uint32_t w) { return __uint_as_float(w & 0xffff0000u); }

__device__ __forceinline__ void unpack8(const uint4& q, float* v) {
    v[0] = lo_of(q.x); v[1] = hi_of(q.x); v[2] = lo_of(q.y); v[3] = hi_of(q.y);
    v[4] = lo_of(q.z); v[5] = hi_of(q.z); v[6] = lo_of(q.w); v[7] = hi_of(q.w);
}

// 16 columns, once (streamed: nothing reads them again) or kept in cache.
template <bool STREAM>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[kVec]) {
    const uint4* q = reinterpret_cast<const uint4*>(p);
    const uint4 a = STREAM ? __ldcs(q) : __ldg(q), b = STREAM ? __ldcs(q + 1) : __ldg(q + 1);
    unpack8(a, v);
    unpack8(b, v + 8);
}
template <bool STREAM>
__device__ __forceinline__ void load16(const float* p, float (&v)[kVec]) {
    const float4* q = reinterpret_cast<const float4*>(p);
    float4 a[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) a[i] = STREAM ? __ldcs(q + i) : __ldg(q + i);
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        v[4 * i] = a[i].x; v[4 * i + 1] = a[i].y; v[4 * i + 2] = a[i].z; v[4 * i + 3] = a[i].w;
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[kVec]) {
    uint4* q = reinterpret_cast<uint4*>(p);
    q[0] = make_uint4(pack2(v[0], v[1]), pack2(v[2], v[3]), pack2(v[4], v[5]), pack2(v[6], v[7]));
    q[1] = make_uint4(pack2(v[8], v[9]), pack2(v[10], v[11]), pack2(v[12], v[13]), pack2(v[14], v[15]));
}
__device__ __forceinline__ void store16(float* p, const float (&v)[kVec]) {
    float4* q = reinterpret_cast<float4*>(p);
#pragma unroll
    for (int i = 0; i < 4; ++i) q[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// The values that 16 codes stand for.
__device__ __forceinline__ void decode16(const uint4& q, float scale, float (&v)[kVec]) {
    const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
#pragma unroll
        for (int h = 0; h < 2; ++h) {
            const __half2_raw r = __nv_cvt_fp8x2_to_halfraw2((__nv_fp8x2_storage_t)(w[i] >> (16 * h)), __NV_E4M3);
            const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&r));
            v[4 * i + 2 * h] = f.x * scale;
            v[4 * i + 2 * h + 1] = f.y * scale;
        }
    }
}

// Codes of a block's values as ep_dispatch makes them, by the 8 lanes that hold
// them (all lanes of the warp call it; lanes past the row's end hold zeros):
// scale = max|v| / 448 (1 where that is 0), code = E4M3(v / scale), both quotients by
// IEEE division.  A NaN takes no part in the maximum and stays NaN as a code; a
// block with an infinity gets the scale infinity, so that its values are NaN.
__device__ __forceinline__ uint4 encode16(const float (&v)[kVec], float& scale) {
    float top = 0.0f;
#pragma unroll
    for (int j = 0; j < kVec; ++j) top = fmaxf(top, fabsf(v[j]));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    scale = __fdiv_rn(top, 448.0f);
    if (scale == 0.0f) scale = 1.0f;
    uint32_t p[8];
#pragma unroll
    for (int j = 0; j < 8; ++j)
        p[j] = (uint32_t)__nv_cvt_float2_to_fp8x2(
            make_float2(__fdiv_rn(v[2 * j], scale), __fdiv_rn(v[2 * j + 1], scale)), __NV_SATFINITE, __NV_E4M3);
    return make_uint4(p[0] | p[1] << 16, p[2] | p[3] << 16, p[4] | p[5] << 16, p[6] | p[7] << 16);
}

// Whether row r holds a token.
__device__ __forceinline__ bool holds_token(const TokenRows& t, uint32_t r) {
    if (t.expert_offsets == nullptr) return true;
    if (t.layout == 0) return (long long)r < __ldg(t.expert_offsets + t.E);
    const uint32_t e = r / (uint32_t)t.cap, slot = r % (uint32_t)t.cap;
    return (long long)slot < (long long)__ldg(t.expert_offsets + e + 1) - __ldg(t.expert_offsets + e);
}

}  // namespace rows
}  // namespace ep
