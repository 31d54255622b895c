// Root-mean-square norm of rows with the residual's addition, and its gradient,
// for sm_103a (ep_rms_norm, ep_rms_norm_backward).
//
//   z = x + residual, rounded to the rows' type;  r = 1 / sqrt(mean(z^2) + eps)
//   y = z r w, as rows and / or as E4M3 codes with a scale for every 128 columns
//   with n = z r and g = d_y w:
//   d_x = r (g - n mean(g n)) + d_residual,  d_w = sum over the rows of d_y n
//
// One pass: a block (a warp or a part of one for short rows) holds its row in
// registers, joins the sum in shared memory and writes every output, so the bytes
// moved are the rows read and written.  Sums are float32, over at most 32 terms a
// thread and then a tree.  In the gradient a block of 512 threads on each SM shares
// them among as many rows as they hold, takes rows in turn with the same columns in
// a thread throughout, has the next rows on their way to shared memory (registers
// for the shortest and longest rows) and sums d_w of its columns in registers; the
// blocks' sums are joined by a second kernel in a fixed order.
//
// Bound by those bytes, but where codes alone are written by instructions.  32768 x
// 7168 bf16: y, codes and the residual 311 us = 6.8 TB/s, y alone 141 = 6.7, codes
// alone 152 = 4.7 (70 % of the issue slots); the gradient with the residual's 284 us =
// 6.6 TB/s.  16384 x 7168 float32: 285 and 262 us = 7.0 and 7.2 TB/s.  Gradients of rows
// past 8192 columns hold two vectors a thread, of which 128 registers spill a part (88 bytes
// a thread for bf16, 468 for float32): 8192 x 16384 with the residual's 195 us = 5.5 TB/s in
// bf16, 557 = 3.9 in float32.
#include <algorithm>
#include <atomic>

#include "rows_common.cuh"

namespace ep {
namespace {

using namespace rows;

// Sum over the row's threads: NT of them where that is a warp or a part of one
// (a power of two), else nt <= NT in whole warps, whose partial sums meet in
// s_part (NT / 32 floats that nothing else uses until the block's next barrier but
// one); barrier `bar` counts nt threads.
template <int NT>
__device__ __forceinline__ float row_sum(float v, int nt, int tid, int bar, float* s_part) {
#pragma unroll
    for (int off = (NT < 32 ? NT : 32) / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    if constexpr (NT > 32) {
        if ((tid & 31) == 0) s_part[tid >> 5] = v;
        asm volatile("barrier.sync %0, %1;" ::"r"(bar), "r"(nt) : "memory");
        const int w = tid & (NT / 32 - 1);  // each NT / 32 lanes join all the warps' sums
        v = w * 32 < nt ? s_part[w] : 0.0f;
#pragma unroll
        for (int off = NT / 64; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    }
    return v;
}

template <typename Args>
__device__ __forceinline__ void load_weight(const Args& a, int c, float (&w)[kVec]) {
    if (a.weight_bf16) load16<false>(static_cast<const __nv_bfloat16*>(a.weight) + c, w, a.wide);
    else load16<false>(static_cast<const float*>(a.weight) + c, w, a.wide);
}

// 1 / sqrt(sum / cols + eps): the hardware's root (2^-22) and a Newton step, which leave
// 2^-23; every thread of a row computes it, and a root and two quotients in full took a
// quarter of the kernel's instructions (codes alone, 32768 x 7168: 184 us,
// 174 so).
__device__ __forceinline__ float rstd_of(float sum, const NormArgs& a) {
    const float v = fmaf(sum, a.inv_cols, a.eps), y = rsqrtf(v);
    const float r = fmaf(0.5f * y, fmaf(-v * y, y, 1.0f), y);
    return y == 0.0f ? 0.0f : r;  // v infinite
}

// Stores the negatives of what v holds.
__device__ __forceinline__ void store_negated(__nv_bfloat16* p, const float (&v)[kVec], bool wide) {
    uint32_t r[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) r[i] = pack2(v[2 * i], v[2 * i + 1]) ^ 0x80008000u;
    store32(p, r, wide);
}
__device__ __forceinline__ void store_negated(float* p, const float (&v)[kVec], bool wide) {
    float n[kVec];
#pragma unroll
    for (int i = 0; i < kVec; ++i) n[i] = -v[i];
    store16(p, n, wide);
}

// Blocks an SM that the registers are to allow.  Rows held as they lie in memory (bf16: half
// of the registers) and these bounds: 32768 x 7168 bf16 with the residual, y and codes 311 us,
// held as float32 with 4 blocks of 62 registers 344; 8192 x 16384 174 and 291 (one block).
template <typename T, int NT, int HELD>
constexpr int kMinBlocks = NT == 512 ? 2 : NT == 256 && (HELD == 1 || sizeof(T) == 2) ? 5 : 1;

// Up to NT threads a row, HELD vectors of 16 each: whole warps and a row a block
// (ROWS = 1), or NT = 8, 16 or 32 threads and ROWS rows a block.
template <typename T, int NT, int ROWS, int HELD>
__global__ void __launch_bounds__(NT * ROWS, kMinBlocks<T, NT, HELD>) rms_norm_kernel(NormArgs a) {
    static_assert(ROWS == 1 || NT <= 32, "a warp or a part of one for each of several rows");
    __shared__ float s_part[(NT + 31) / 32];
    pdl_prologue();
    const int nt = ROWS > 1 ? NT : (int)blockDim.x;
    const int tid = ROWS > 1 ? (int)threadIdx.x % NT : (int)threadIdx.x;
    const long long r = (long long)blockIdx.x * ROWS + (ROWS > 1 ? threadIdx.x / NT : 0);
    const int cols = r < a.rows ? a.cols : 0;  // past the last row, lanes only take part in sums
    const size_t at = (size_t)r * a.cols;
    const T* x = static_cast<const T*>(a.x) + at;
    const T* res = a.residual != nullptr ? static_cast<const T*>(a.residual) + at : nullptr;
    if (a.few) {  // the weight is on its way while the row is summed
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < cols)
                asm volatile("prefetch.global.L1 [%0];" ::"l"(static_cast<const char*>(a.weight) + (size_t)c * (a.weight_bf16 ? 2 : 4)));
        }
    }
    Raw<T> z[HELD];
    float sum = 0.0f;
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * nt + tid) * kVec;
        z[i].zero();
        if (c < cols) {
            z[i].load(x + c, a.wide);
            if (res != nullptr) {
                Raw<T> t;
                t.load(res + c, a.wide);
                z[i].add(t);
            }
        }
#pragma unroll
        for (int j = 0; j < kVec; ++j) sum = fmaf(z[i].at(j), z[i].at(j), sum);
    }
    if (a.residual_out != nullptr) {
        T* to = static_cast<T*>(a.residual_out) + at;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < cols) z[i].store(to + c, a.wide);
        }
    }
    sum = row_sum<NT>(sum, nt, tid, 0, s_part);
    const float rstd = rstd_of(sum, a);
    if (tid == 0 && cols > 0 && a.rstd != nullptr) a.rstd[r] = rstd;
    if (a.y == nullptr && a.q == nullptr) return;
    const int blocks = scale_blocks(a.cols);
#pragma unroll
    for (int i = 0; i < HELD; ++i) {
        const int c = (i * nt + tid) * kVec;
        float nv[kVec];  // the negatives, as encode16 takes them
#pragma unroll
        for (int j = 0; j < kVec; ++j) nv[j] = 0.0f;
        if (c < cols) {
            float w[kVec];
            load_weight(a, c, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) nv[j] = z[i].at(j) * -rstd * w[j];
            if (a.y != nullptr) store_negated(static_cast<T*>(a.y) + at + c, nv, a.wide);
        }
        if (a.q != nullptr) {  // every lane takes part in the blocks' maxima
            float scale;
            const uint4 codes = encode16(nv, scale);
            if (c < cols) {
                *reinterpret_cast<uint4*>(a.q + at + c) = codes;
                if (c % kScaleBlock == 0) a.scales[(size_t)r * blocks + c / kScaleBlock] = scale;
            }
        }
    }
}

// bf16 rows without a residual, of up to 512 vectors, a thread's vector each: blocks stay
// and take rows blockIdx.x, + gridDim.x, ..., the weight in registers, the next row on its
// way to shared memory (two rows ahead: 150 us where one takes 143).  A warp fetches its own
// 1 KB of a row in 16-byte pieces, so that only its own lanes wait for them.  Where codes
// are wanted, bound by its 300 instructions a vector.
constexpr int kAheadThreads = 512, kAheadRows = 2;

// Where piece c of a warp's lies, so that lanes that read their vectors' i-th pieces meet
// no bank conflicts.
template <typename T>
__device__ __forceinline__ uint32_t piece_place(uint32_t c) {
    return c ^ (c >> 3 & (sizeof(T) == 2 ? 1 : 3));
}
__device__ __forceinline__ void fetch_piece(uint32_t to, const void* from) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(to), "l"(from) : "memory");
}
__device__ __forceinline__ void take_piece(uint32_t from, uint32_t* r) {
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]) : "r"(from) : "memory");
}
// A lane's vector as it lies in memory, and its values.
template <typename T>
__device__ __forceinline__ void take_vector(const uint32_t (&own)[sizeof(T)], uint32_t slot, uint32_t (&r)[4 * sizeof(T)]) {
#pragma unroll
    for (int i = 0; i < (int)sizeof(T); ++i) take_piece(own[i] + slot, r + 4 * i);
}
__device__ __forceinline__ float value_of(const uint32_t (&r)[8], int j) { return j % 2 ? hi_of(r[j / 2]) : lo_of(r[j / 2]); }
__device__ __forceinline__ float value_of(const uint32_t (&r)[16], int j) { return __uint_as_float(r[j]); }

// Two values an instruction: a pair by a pair, or by twice the same.
__device__ __forceinline__ uint64_t pair(float lo, float hi) {
    uint64_t r;
    asm("mov.b64 %0, {%1, %2};" : "=l"(r) : "f"(lo), "f"(hi));
    return r;
}
__device__ __forceinline__ uint64_t mul2(uint64_t a, uint64_t b) {
    uint64_t r;
    asm("mul.rn.f32x2 %0, %1, %2;" : "=l"(r) : "l"(a), "l"(b));
    return r;
}
__device__ __forceinline__ uint64_t square2(uint64_t a, uint64_t sum) {
    uint64_t r;
    asm("fma.rn.f32x2 %0, %1, %1, %2;" : "=l"(r) : "l"(a), "l"(sum));
    return r;
}
__device__ __forceinline__ void apart(uint64_t a, float& lo, float& hi) { asm("mov.b64 {%0, %1}, %2;" : "=f"(lo), "=f"(hi) : "l"(a)); }

__global__ void __launch_bounds__(kAheadThreads, 2) rms_norm_ahead_kernel(NormArgs a) {
    extern __shared__ __align__(16) uint4 s_rows[];  // [kAheadRows][warps][64]
    __shared__ float s_part[2][kAheadThreads / 32];
    pdl_prologue();
    const int nt = (int)blockDim.x, tid = (int)threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int c = tid * kVec, pieces = a.cols / 8, blocks = scale_blocks(a.cols);
    const bool on = c < a.cols;
    const __nv_bfloat16* x = static_cast<const __nv_bfloat16*>(a.x);
    const int slot_pieces = nt * 2;
    const uint32_t first = (uint32_t)__cvta_generic_to_shared(s_rows + warp * 64), slot_bytes = slot_pieces * 16;
    // this lane's two pieces of a row, or none; what is never fetched stays 0
    const int p0 = warp * 64 + lane, p1 = p0 + 32;
    const uint32_t to0 = first + piece_place<__nv_bfloat16>(lane) * 16, to1 = first + piece_place<__nv_bfloat16>(32 + lane) * 16;
    for (int i = tid; i < kAheadRows * slot_pieces; i += nt) s_rows[i] = make_uint4(0, 0, 0, 0);
    __syncthreads();
    const auto fetch = [&](long long r, uint32_t slot) {
        if (r < a.rows) {
            const __nv_bfloat16* row = x + (size_t)r * a.cols;
            if (p0 < pieces) fetch_piece(to0 + slot, row + p0 * 8);
            if (p1 < pieces) fetch_piece(to1 + slot, row + p1 * 8);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int i = 0; i < kAheadRows - 1; ++i) fetch(blockIdx.x + (long long)i * gridDim.x, i * slot_bytes);
    uint64_t w[kVec / 2];
    {
        float f[kVec];
#pragma unroll
        for (int j = 0; j < kVec; ++j) f[j] = 0.0f;
        if (on) load_weight(a, c, f);
#pragma unroll
        for (int j = 0; j < kVec / 2; ++j) w[j] = pair(f[2 * j], f[2 * j + 1]);
    }
    const uint32_t own0 = first + piece_place<__nv_bfloat16>(2 * lane) * 16, own1 = first + piece_place<__nv_bfloat16>(2 * lane + 1) * 16;
    uint32_t slot = 0, next = (kAheadRows - 1) * slot_bytes;  // what next held was read before the last barrier
    int turn = 0;
    for (long long r = blockIdx.x; r < a.rows; r += gridDim.x) {
        fetch(r + (kAheadRows - 1ll) * gridDim.x, next);
        next = slot;
        asm volatile("cp.async.wait_group %0;" ::"n"(kAheadRows - 1) : "memory");
        __syncwarp();
        const size_t at = (size_t)r * a.cols + c;
        uint32_t p[8];
        take_piece(own0 + slot, p);
        take_piece(own1 + slot, p + 4);
        slot = slot == (kAheadRows - 1) * slot_bytes ? 0 : slot + slot_bytes;
        if (on && a.residual_out != nullptr) store32(static_cast<__nv_bfloat16*>(a.residual_out) + at, p, a.wide);
        uint64_t z[8], sums = 0;
#pragma unroll
        for (int j = 0; j < 8; ++j) {
            z[j] = pair(lo_of(p[j]), hi_of(p[j]));
            sums = square2(z[j], sums);
        }
        float sum, odd;
        apart(sums, sum, odd);
        sum = row_sum<kAheadThreads>(sum + odd, nt, tid, 0, s_part[turn]);
        turn ^= 1;
        const float rstd = rstd_of(sum, a);
        if (tid == 0 && a.rstd != nullptr) a.rstd[r] = rstd;
        // the negatives, as encode16 takes them
        const uint64_t by = pair(-rstd, -rstd);
        float nv[kVec];
#pragma unroll
        for (int j = 0; j < 8; ++j) apart(mul2(mul2(z[j], by), w[j]), nv[2 * j], nv[2 * j + 1]);
        if (on && a.y != nullptr) store_negated(static_cast<__nv_bfloat16*>(a.y) + at, nv, a.wide);
        if (a.q != nullptr) {  // every lane takes part in the blocks' maxima
            float scale;
            const uint4 codes = encode16(nv, scale);
            if (on) {
                *reinterpret_cast<uint4*>(a.q + at) = codes;
                if (c % kScaleBlock == 0) a.scales[(size_t)r * blocks + c / kScaleBlock] = scale;
            }
        }
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
}

cudaError_t norm_ahead(const NormArgs& a, cudaStream_t s) {
    const int nt = (a.cols / kVec + 31) / 32 * 32;
    const size_t smem = (size_t)kAheadRows * nt * 32;  // 32 KB at most
    const long long blocks = std::min<long long>(a.rows, (long long)sm_count() * (2 * kAheadThreads / nt));
    return launch(rms_norm_ahead_kernel, dim3((unsigned)blocks), dim3(nt), smem, s, a);
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
    // Us, one row a block / blocks that stay, 32768 rows: y of 7168 160 / 141, of 4096 86 / 82,
    // of 2048 43 / 41; codes of 7168 168 / 152, of 2048 47 / 47; both of 7168 203 / 184, of 2048
    // 53 / 55; one row 8.2 / 6.1.  With a residual the former are at the copy rate by
    // themselves (311, the latter 342).
    if (a.bf16 && a.residual == nullptr && a.cols > 1024 && a.cols <= kAheadThreads * kVec) return norm_ahead(a, s);
    if (a.cols <= 128) return norm_shape<T, 8, 32, 1>(a, s);
    if (a.cols <= 256) return norm_shape<T, 16, 16, 1>(a, s);
    if (a.cols <= 512) return norm_shape<T, 32, 8, 1>(a, s);
    if (a.cols <= 1024) return norm_shape<T, 32, 4, 2>(a, s);
    if (a.cols <= 4096) return norm_shape<T, 256, 1, 1>(a, s);
    if (a.cols <= 8192) return norm_shape<T, 256, 1, 2>(a, s);
    return norm_shape<T, 512, 1, 2>(a, s);
}

// ---- gradient --------------------------------------------------------------------

constexpr int kGradThreads = 512;  // of a block, one block an SM

__device__ __forceinline__ void store16f(float* p, const float (&v)[kVec]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) reinterpret_cast<float4*>(p)[i] = make_float4(v[4 * i], v[4 * i + 1], v[4 * i + 2], v[4 * i + 3]);
}

// How the threads share the rows: nt threads a row, `groups` rows at a time in a block.
struct GradShape {
    int nt, groups, blocks;
};
int grad_held(int cols) { return cols <= kGradThreads * kVec ? 1 : 2; }
GradShape grad_shape(int rows, int cols) {
    GradShape g;
    const int vectors = cols / kVec, held = grad_held(cols);
    g.nt = vectors <= 8 ? 8 : vectors <= 16 ? 16 : ((vectors + held - 1) / held + 31) / 32 * 32;
    g.groups = kGradThreads / g.nt;
    if (g.nt > 32) g.groups = std::min(g.groups, 15);  // a barrier each, and one for the block
    g.blocks = (int)std::min<long long>(sm_count(), ((long long)rows + g.groups - 1) / g.groups);
    return g;
}

// The block's partial sums of d_w: of one group from its registers, of more joined in s_dw.
template <int HELD>
__device__ __forceinline__ void join_groups(const NormGradArgs& a, const GradShape& g, const float (&dw)[HELD][kVec],
                                            float* s_dw, int group, int tid) {
    const int nt = g.nt;
    if (a.d_weight == nullptr) return;
    float* to = a.partial + (size_t)blockIdx.x * a.cols;
    if (g.groups > 1) {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < a.cols) store16f(s_dw + (size_t)group * a.cols + c, dw[i]);
        }
        __syncthreads();
        for (int c = threadIdx.x; c < a.cols; c += blockDim.x) {
            float v = 0.0f;
            for (int k = 0; k < g.groups; ++k) v += s_dw[(size_t)k * a.cols + c];
            to[c] = v;
        }
    } else {
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c < a.cols) store16f(to + c, dw[i]);
        }
    }
}

// Rows of a part of a warp (HELD = 1) or of more than 512 vectors (2): a row's three arrays
// load together, and with HELD = 1 while the row before is worked on.
template <typename T, int HELD>
__global__ void __launch_bounds__(kGradThreads, 1) rms_norm_backward_kernel(NormGradArgs a, GradShape g) {
    extern __shared__ __align__(16) float s_dw[];  // [groups][cols], for more than one group
    __shared__ float s_part[2][kGradThreads / 32];
    constexpr bool kAhead = HELD == 1;
    pdl_prologue();
    const int nt = g.nt, group = (int)threadIdx.x / nt, tid = (int)threadIdx.x % nt;
    const bool has_res = a.d_residual != nullptr, wide = a.wide;
    const long long first = (long long)blockIdx.x * g.groups + group;
    const int step = (int)gridDim.x * g.groups;
    Raw<T> z[HELD], dy[HELD], res[HELD];
    float rstd = 0.0f;
    const auto load = [&](long long r) {
        const bool on = r < a.rows;
        rstd = on ? __ldg(a.rstd + r) : 0.0f;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            z[i].zero();
            dy[i].zero();
            res[i].zero();
            if (on && c < a.cols) {
                const size_t at = (size_t)r * a.cols + c;
                z[i].load(static_cast<const T*>(a.z) + at, wide);
                dy[i].load(static_cast<const T*>(a.d_y) + at, wide);
                if (has_res) res[i].load(static_cast<const T*>(a.d_residual) + at, wide);
            }
        }
    };
    float dw[HELD][kVec];
#pragma unroll
    for (int i = 0; i < HELD; ++i)
#pragma unroll
        for (int j = 0; j < kVec; ++j) dw[i][j] = 0.0f;
    int turn = 0;
    if (kAhead) load(first);
    // a block's groups take turns together, so that a warp's lanes do; past the last row
    // they hold zeros
    for (long long base = (long long)blockIdx.x * g.groups; base < a.rows; base += step) {
        const long long r = base + group;
        if (!kAhead) load(r);
        float n[HELD][kVec], gy[HELD][kVec];
        Raw<T> d[HELD];
        const float scale = rstd;
        float sum = 0.0f;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
            if (c >= a.cols) {  // idle threads add nothing
#pragma unroll
                for (int j = 0; j < kVec; ++j) n[i][j] = gy[i][j] = 0.0f;
                continue;
            }
            float w[kVec];
            load_weight(a, c, w);
#pragma unroll
            for (int j = 0; j < kVec; ++j) {
                n[i][j] = z[i].at(j) * scale;
                gy[i][j] = dy[i].at(j);
                dw[i][j] = fmaf(gy[i][j], n[i][j], dw[i][j]);
                gy[i][j] *= w[j];
                sum = fmaf(gy[i][j], n[i][j], sum);
            }
        }
#pragma unroll
        for (int i = 0; i < HELD; ++i) d[i] = res[i];
        if (kAhead) load(r + step);
        // two buffers in turn: a warp may be one row ahead of another
        if (nt == 8) sum = row_sum<8>(sum, nt, tid, 0, nullptr);
        else if (nt == 16) sum = row_sum<16>(sum, nt, tid, 0, nullptr);
        else if (nt == 32) sum = row_sum<32>(sum, nt, tid, 0, nullptr);
        else sum = row_sum<kGradThreads>(sum, nt, tid, group + 1, s_part[turn] + group * (nt >> 5));
        turn ^= 1;
        const float mean = sum * a.inv_cols;
#pragma unroll
        for (int i = 0; i < HELD; ++i) {
            const int c = (i * nt + tid) * kVec;
#pragma unroll
            for (int j = 0; j < kVec; ++j) n[i][j] = fmaf(scale, fmaf(-n[i][j], mean, gy[i][j]), d[i].at(j));
            if (r < a.rows && c < a.cols) store16(static_cast<T*>(a.d_x) + (size_t)r * a.cols + c, n[i], wide);
        }
    }
    join_groups<HELD>(a, g, dw, s_dw, group, tid);
}

// Rows of whole warps, a thread's vector each: the next rows of a group (ROWS - 1 of them)
// are on their way to shared memory, as in rms_norm_ahead_kernel.  32768 x 7168 bf16 with the
// residual's gradient 283 us, with one row ahead in registers 313; 5003 x 2880 float32 31 us
// instead of 37.  Registers allow one block an SM (two of 64 a thread, the weight read twice
// from what is left of L1: 469).
template <typename T, int ROWS>
__global__ void __launch_bounds__(kGradThreads, 1) rms_norm_backward_ahead_kernel(NormGradArgs a, GradShape g) {
    constexpr int kPieces = sizeof(T);  // of 16 bytes in a vector
    constexpr bool kEarly = sizeof(T) == 2;
    extern __shared__ __align__(16) uint4 s_grad[];  // [ROWS][z, d_y, d_residual][warps][32 kPieces]
    __shared__ float s_part[2][kGradThreads / 32];
    pdl_prologue();
    const int nt = g.nt, group = (int)threadIdx.x / nt, tid = (int)threadIdx.x % nt, lane = tid & 31, warp = tid >> 5;
    const int c = tid * kVec, pieces = a.cols / kVec * kPieces;
    const bool on = c < a.cols, has_res = a.d_residual != nullptr;
    const uint32_t array_bytes = blockDim.x * 16 * kPieces, slot_bytes = (has_res ? 3 : 2) * array_bytes;
    const uint32_t first = (uint32_t)__cvta_generic_to_shared(s_grad) + threadIdx.x / 32 * (512 * kPieces);
    uint32_t to[kPieces], own[kPieces];  // the pieces that this lane fetches, and those of its vector
#pragma unroll
    for (int i = 0; i < kPieces; ++i) {
        to[i] = first + piece_place<T>(32 * i + lane) * 16;
        own[i] = first + piece_place<T>(kPieces * lane + i) * 16;
    }
    const auto fetch_row = [&](const void* rows, size_t at, uint32_t slot) {
        const uint4* row = reinterpret_cast<const uint4*>(static_cast<const T*>(rows) + at);
#pragma unroll
        for (int i = 0; i < kPieces; ++i) {
            const int p = (warp * kPieces + i) * 32 + lane;
            if (p < pieces) fetch_piece(to[i] + slot, row + p);
        }
    };
    const auto fetch = [&](long long r, uint32_t slot) {
        if (r < a.rows) {
            const size_t at = (size_t)r * a.cols;
            fetch_row(a.z, at, slot);
            fetch_row(a.d_y, at, slot + array_bytes);
            if (has_res) fetch_row(a.d_residual, at, slot + 2 * array_bytes);
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    const long long step = (long long)gridDim.x * g.groups;
    long long r = (long long)blockIdx.x * g.groups + group;
    for (int i = 0; i < ROWS - 1; ++i) fetch(r + i * step, i * slot_bytes);
    float w[kVec], dw[1][kVec];
#pragma unroll
    for (int j = 0; j < kVec; ++j) w[j] = dw[0][j] = 0.0f;
    if (on) load_weight(a, c, w);
    float next_scale = r < a.rows ? __ldg(a.rstd + r) : 0.0f;
    uint32_t slot = 0, next = (ROWS - 1) * slot_bytes;
    int turn = 0;
    for (; r < a.rows; r += step) {
        __syncwarp();  // what lies in next has been read
        fetch(r + (ROWS - 1) * step, next);
        next = slot;
        const float scale = next_scale;
        if (r + step < a.rows) next_scale = __ldg(a.rstd + r + step);
        asm volatile("cp.async.wait_group %0;" ::"n"(ROWS - 1) : "memory");
        __syncwarp();
        uint32_t z[4 * kPieces], d[4 * kPieces], res[4 * kPieces];
        take_vector<T>(own, slot, z);
        take_vector<T>(own, slot + array_bytes, d);
        // float32 has no registers for these before the sum
        if (kEarly && has_res) take_vector<T>(own, slot + 2 * array_bytes, res);
        float n[kVec], gy[kVec], sum = 0.0f;
#pragma unroll
        for (int j = 0; j < kVec; ++j) {
            n[j] = on ? value_of(z, j) * scale : 0.0f;
            gy[j] = on ? value_of(d, j) : 0.0f;
            dw[0][j] = fmaf(gy[j], n[j], dw[0][j]);
            gy[j] *= w[j];
            sum = fmaf(gy[j], n[j], sum);
        }
        if (nt == 32) sum = row_sum<32>(sum, nt, tid, 0, nullptr);
        else sum = row_sum<kGradThreads>(sum, nt, tid, group + 1, s_part[turn] + group * (nt >> 5));
        turn ^= 1;
        const float mean = sum * a.inv_cols;
        if (on) {
            if (!kEarly && has_res) take_vector<T>(own, slot + 2 * array_bytes, res);
#pragma unroll
            for (int j = 0; j < kVec; ++j)
                n[j] = fmaf(scale, fmaf(-n[j], mean, gy[j]), has_res ? value_of(res, j) : 0.0f);
            store16(static_cast<T*>(a.d_x) + (size_t)r * a.cols + c, n, a.wide);
        }
        slot = slot == (ROWS - 1) * slot_bytes ? 0 : slot + slot_bytes;
    }
    asm volatile("cp.async.wait_all;" ::: "memory");
    __syncthreads();  // the rows' memory takes the groups' sums
    join_groups<1>(a, g, dw, reinterpret_cast<float*>(s_grad), group, tid);
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

// More than 48 KB of dynamic shared memory, allowed once for each device.
cudaError_t allow_smem(const void* kernel, int bytes, std::atomic<bool> (&done)[64]) {
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess || (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed))) return err;
    err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
    if (err == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return err;
}

template <typename T, int ROWS>
cudaError_t grad_ahead(const NormGradArgs& a, const GradShape& g, cudaStream_t s) {
    static std::atomic<bool> done[64];
    constexpr int kBytes = ROWS * 16 * (int)sizeof(T);  // of a thread, of each array
    const int threads = g.nt * g.groups, arrays = a.d_residual != nullptr ? 3 : 2;
    const cudaError_t err = allow_smem(reinterpret_cast<const void*>(rms_norm_backward_ahead_kernel<T, ROWS>),
                                       (sizeof(T) == 4 && ROWS == 3 ? 2 : 3) * kBytes * kGradThreads, done);
    if (err != cudaSuccess) return err;
    return launch(rms_norm_backward_ahead_kernel<T, ROWS>, dim3(g.blocks), dim3(threads), (size_t)arrays * kBytes * threads,
                  s, a, g);
}

template <typename T>
cudaError_t grad_t(const NormGradArgs& a, const GradShape& g, cudaStream_t s) {
    // whole warps a row, a vector a thread: through shared memory, three rows of a group where
    // they fit (float32 with a residual's gradient: two, 196 KB)
    if (g.nt >= 32 && grad_held(a.cols) == 1) {
        if constexpr (sizeof(T) == 4)
            if (a.d_residual != nullptr) return grad_ahead<T, 2>(a, g, s);
        return grad_ahead<T, 3>(a, g, s);
    }
    const dim3 grid(g.blocks), block(g.nt * g.groups);
    // at most 512 threads of 16 columns: 32 KB
    const size_t smem = g.groups > 1 ? (size_t)g.groups * a.cols * sizeof(float) : 0;
    return grad_held(a.cols) == 1 ? launch(rms_norm_backward_kernel<T, 1>, grid, block, smem, s, a, g)
                                  : launch(rms_norm_backward_kernel<T, 2>, grid, block, smem, s, a, g);
}

}  // namespace

cudaError_t launch_rms_norm(const NormArgs& args, cudaStream_t s) {
    if (args.rows == 0) return cudaSuccess;
    NormArgs a = args;
    a.wide = aligned32(a.x, a.residual, a.residual_out, a.y) && aligned32(a.weight);
    // One row of 7168: 8.2 us instead of 10.2.  Many rows find the weight in L1 and only
    // pay: 65536 rows of 512 would take 168 us instead of 47.
    a.inv_cols = 1.0f / (float)a.cols;
    a.few = a.rows <= sm_count() && (a.y != nullptr || a.q != nullptr);
    const cudaError_t err = a.bf16 ? norm_t<__nv_bfloat16>(a, s) : norm_t<float>(a, s);
    note_launch();
    return err;
}

// The most blocks of any type and residual: a row a block.
int norm_grad_blocks(int rows) { return std::min(sm_count(), rows); }

cudaError_t launch_rms_norm_backward(const NormGradArgs& args, cudaStream_t s) {
    NormGradArgs a = args;
    a.wide = aligned32(a.d_y, a.z, a.d_residual, a.d_x) && aligned32(a.weight);
    a.inv_cols = 1.0f / (float)a.cols;
    if (a.rows == 0)
        return a.d_weight != nullptr ? cudaMemsetAsync(a.d_weight, 0, (size_t)a.cols * sizeof(float), s) : cudaSuccess;
    const GradShape g = grad_shape(a.rows, a.cols);
    cudaError_t err = a.bf16 ? grad_t<__nv_bfloat16>(a, g, s) : grad_t<float>(a, g, s);
    note_launch();
    if (err != cudaSuccess || a.d_weight == nullptr) return err;
    err = launch(weight_grad_kernel, dim3((a.cols + 31) / 32), dim3(1024), 0, s, a, g.blocks);
    note_launch();
    return err;
}

}  // namespace ep
