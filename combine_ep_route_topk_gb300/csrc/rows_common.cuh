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

// 32 bytes that start on a boundary of 32, in one access (whole sectors of memory: two
// of 16 bytes by each thread, 32 apart, ask for every sector twice).
template <bool STREAM>
__device__ __forceinline__ void load32(const void* p, uint32_t (&r)[8]) {
    if (STREAM)
        asm volatile("ld.global.L1::no_allocate.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p) : "memory");
    else
        asm volatile("ld.global.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "l"(p) : "memory");
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(p), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}
template <bool STREAM>
__device__ __forceinline__ void load32(const void* p, uint32_t (&r)[8], bool wide) {
    if (wide) {
        load32<STREAM>(p, r);
    } else {
        const uint4* q = static_cast<const uint4*>(p);
        const uint4 a = STREAM ? __ldcs(q) : *q, b = STREAM ? __ldcs(q + 1) : q[1];
        r[0] = a.x; r[1] = a.y; r[2] = a.z; r[3] = a.w;
        r[4] = b.x; r[5] = b.y; r[6] = b.z; r[7] = b.w;
    }
}
__device__ __forceinline__ void store32(void* p, const uint32_t (&r)[8], bool wide) {
    if (wide) {
        store32(p, r);
    } else {
        static_cast<uint4*>(p)[0] = make_uint4(r[0], r[1], r[2], r[3]);
        static_cast<uint4*>(p)[1] = make_uint4(r[4], r[5], r[6], r[7]);
    }
}

// 16 columns, once (streamed: nothing reads them again) or kept in cache; wide: rows
// start on 32 bytes.
template <bool STREAM>
__device__ __forceinline__ void load16(const __nv_bfloat16* p, float (&v)[kVec], bool wide) {
    uint32_t r[8];
    load32<STREAM>(p, r, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[2 * i] = lo_of(r[i]);
        v[2 * i + 1] = hi_of(r[i]);
    }
}
template <bool STREAM>
__device__ __forceinline__ void load16(const float* p, float (&v)[kVec], bool wide) {
    uint32_t r[8], t[8];
    load32<STREAM>(p, r, wide);
    load32<STREAM>(p + 8, t, wide);
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        v[i] = __uint_as_float(r[i]);
        v[8 + i] = __uint_as_float(t[i]);
    }
}

__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}
__device__ __forceinline__ void store16(__nv_bfloat16* p, const float (&v)[kVec], bool wide) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = pack2(v[2 * i], v[2 * i + 1]);
    store32(p, r, wide);
}
__device__ __forceinline__ void store16(float* p, const float (&v)[kVec], bool wide) {
    uint32_t r[8];
#pragma unroll
    for (int h = 0; h < 16; h += 8) {
#pragma unroll
        for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(v[h + i]);
        store32(p + h, r, wide);
    }
}

// Sixteen columns as they lie in memory.
template <typename T>
struct Raw {
    uint32_t r[kVec * sizeof(T) / 32][8];
    __device__ __forceinline__ void load(const T* p, bool wide) {
#pragma unroll
        for (int h = 0; h < (int)(kVec * sizeof(T) / 32); ++h) load32<true>(p + h * (32 / sizeof(T)), r[h], wide);
    }
    __device__ __forceinline__ void zero() {
#pragma unroll
        for (int h = 0; h < (int)(kVec * sizeof(T) / 32); ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) r[h][i] = 0;
    }
    // What they hold, negated (encode16 takes that).
    __device__ __forceinline__ void negatives(float (&v)[kVec]) const {
#pragma unroll
        for (int h = 0; h < (int)(kVec * sizeof(T) / 32); ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                if (sizeof(T) == 4) {
                    v[h * 8 + i] = __uint_as_float(r[h][i] ^ 0x80000000u);
                } else {
                    v[2 * i] = lo_of(r[0][i] ^ 0x8000u);
                    v[2 * i + 1] = hi_of(r[0][i] ^ 0x80000000u);
                }
            }
    }
    // The sums with t's, rounded to the type.
    __device__ __forceinline__ void add(const Raw& t) {
#pragma unroll
        for (int h = 0; h < (int)(kVec * sizeof(T) / 32); ++h)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                r[h][i] = sizeof(T) == 4 ? __float_as_uint(__uint_as_float(r[h][i]) + __uint_as_float(t.r[h][i]))
                                         : pack2(lo_of(r[h][i]) + lo_of(t.r[h][i]), hi_of(r[h][i]) + hi_of(t.r[h][i]));
    }
    __device__ __forceinline__ void store(T* p, bool wide) const {
#pragma unroll
        for (int h = 0; h < (int)(kVec * sizeof(T) / 32); ++h) store32(p + h * (32 / sizeof(T)), r[h], wide);
    }
    __device__ __forceinline__ float at(int j) const {
        if (sizeof(T) == 4) return __uint_as_float(r[j / 8][j % 8]);
        return j % 2 ? hi_of(r[0][j / 2]) : lo_of(r[0][j / 2]);
    }
};

inline bool aligned32(const void* a, const void* b = nullptr, const void* c = nullptr, const void* d = nullptr) {
    return ((reinterpret_cast<uintptr_t>(a) | reinterpret_cast<uintptr_t>(b) | reinterpret_cast<uintptr_t>(c) |
             reinterpret_cast<uintptr_t>(d)) & 31u) == 0;
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

// Two E4M3 codes, the first in the low byte.
__device__ __forceinline__ uint32_t e4m3x2(float lo, float hi) {
    return (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(lo, hi), __NV_SATFINITE, __NV_E4M3);
}

__device__ __forceinline__ float max_abs3(float a, float b, float c) {
    float m;
    asm("max.abs.f32 %0, %1, %2, %3;" : "=f"(m) : "f"(a), "f"(b), "f"(c));
    return m;
}

// Codes of a block's values as ep_dispatch makes them, by the 8 lanes that hold
// them (all lanes of the warp call it; lanes past the row's end hold zeros):
// scale = max|v| / 448 (1 where that is 0), code = E4M3(v / scale), both quotients
// rounded as IEEE divisions are.  A NaN takes no part in the maximum and stays NaN
// as a code; a block with an infinity gets the scale infinity, so that its values
// are NaN.  The quotients are products with the reciprocal, corrected once
// by their remainder (Markstein, "Computation of elementary functions on the IBM
// RISC System/6000 processor", 1990), which is exact here: v has a remainder that
// a float32 holds, or a quotient far below the smallest code.  (The hardware's
// reciprocal is off by 2^-23 of itself, which leaves 2^-22 of a last place: a quotient
// that is a float32, like the borders between codes, comes out as itself.)  Given are the values'
// negatives, nv: the remainder q scale - v, taken from the quotient, keeps the sign of
// -0, and two values an instruction have no modifier for a sign.  32768 x 7168 bf16
// rows 117 us, with divisions 158.
__device__ __forceinline__ uint4 encode16(const float (&nv)[kVec], float& scale) {
    float top = max_abs3(nv[0], nv[1], nv[2]);
#pragma unroll
    for (int j = 3; j < kVec - 1; j += 2) top = max_abs3(top, nv[j], nv[j + 1]);
    top = fmaxf(top, fabsf(nv[kVec - 1]));
#pragma unroll
    for (int off = kLanes / 2; off > 0; off >>= 1) top = fmaxf(top, __shfl_xor_sync(kFull, top, off));
    uint32_t p[8];
    // zeros, of padded rows or of lanes past the row's end: scale 1 by the same way (the other,
    // with its divisions, made a norm of 65536 x 1040 rows take 170 us instead of 104)
    if (top == 0.0f) top = 448.0f;
    if (top >= 0x1p-100f && top <= 0x1.fffffep127f) {
        constexpr float kInv448 = 1.0f / 448.0f;
        scale = top * kInv448;
        scale = fmaf(fmaf(-scale, 448.0f, top), kInv448, scale);
        float ninv;
        asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(ninv) : "f"(-scale));
        uint64_t ninv2, scale2;
        asm("mov.b64 %0, {%1, %1};" : "=l"(ninv2) : "f"(ninv));
        asm("mov.b64 %0, {%1, %1};" : "=l"(scale2) : "f"(scale));
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            float x, y;
            asm("{\n.reg .b64 v, q, r;\n"
                "mov.b64 v, {%2, %3};\n"
                "mul.rn.f32x2 q, v, %4;\n"
                "fma.rn.f32x2 r, q, %5, v;\n"
                "fma.rn.f32x2 q, r, %4, q;\n"
                "mov.b64 {%0, %1}, q;\n}\n"
                : "=f"(x), "=f"(y) : "f"(nv[2 * j]), "f"(nv[2 * j + 1]), "l"(ninv2), "l"(scale2));
            p[j] = e4m3x2(x, y);
        }
    } else {
        scale = top == top ? __fdiv_rn(top, 448.0f) : 0.0f;  // nothing but NaN: 1 as for zeros
        if (scale == 0.0f) scale = 1.0f;
#pragma unroll
        for (int j = 0; j < 8; ++j) p[j] = e4m3x2(__fdiv_rn(-nv[2 * j], scale), __fdiv_rn(-nv[2 * j + 1], scale));
    }
    return make_uint4(__byte_perm(p[0], p[1], 0x5410), __byte_perm(p[2], p[3], 0x5410),
                      __byte_perm(p[4], p[5], 0x5410), __byte_perm(p[6], p[7], 0x5410));
}

// n / d for n below 2^31 by one product (Granlund and Montgomery, "Division by invariant
// integers using multiplication", 1994), made on the host.
struct Divisor {
    uint32_t d, m, shift;
    Divisor() = default;
    explicit Divisor(uint32_t by) : d(by), m(0), shift(0) {
        if (by > 1) {
            uint32_t l = 1;
            while ((1ull << l) < by) ++l;
            m = (uint32_t)((1ull << (31 + l)) / by + 1);
            shift = l - 1;
        }
    }
    __device__ __forceinline__ uint32_t divide(uint32_t n) const { return d == 1 ? n : __umulhi(n, m) >> shift; }
};

// Whether row r holds a token.
__device__ __forceinline__ bool holds_token(const TokenRows& t, uint32_t r) {
    if (t.expert_offsets == nullptr) return true;
    if (t.layout == 0) return (long long)r < __ldg(t.expert_offsets + t.E);
    const uint32_t e = r / (uint32_t)t.cap, slot = r % (uint32_t)t.cap;
    return (long long)slot < (long long)__ldg(t.expert_offsets + e + 1) - __ldg(t.expert_offsets + e);
}

}  // namespace rows
}  // namespace ep
