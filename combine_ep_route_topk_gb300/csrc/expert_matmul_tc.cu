// Experts' products in 8-bit integers on the tensor cores of sm_103a
// (ep_expert_matmul with more than a few rows per expert).
//
//   out[r, n] = xs[r] * ws[e, n] * sum_k x[r, k] * w[e, n, k]
//
// The integer tensor rate of this chip is a small fraction of its 16-bit rate,
// and every 8-bit integer is a float16: the codes are widened on the chip and
// multiplied by tcgen05.mma kind::f16 with float32 accumulators.  A product of
// two codes is an integer of at most 2^14, so sums below 2^24 in magnitude are
// exact; beyond, an addition rounds at 2^-24 relative, far below the output's.
//
// A tile is 128 channels a CTA (the M side: weights) x up to TN rows (the N
// side).  CG = 1: one CTA, TN = 128, two accumulators.  CG = 2: a pair of CTAs
// on 256 channels, TN = 256, each holding half of the rows' operand.
//   TMA warp        weights, [128 channels x 128 bytes] boxes, 128-byte swizzle
//   4 weight warps  shared memory -> float16 -> TMEM (the A operand's stages)
//   4 row warps     x rows (gathered, L2) -> float16 -> shared memory (B);
//                   warp w fills stage w, so four stages load at once
//   MMA warp        one thread issues 8 MMAs of K = 16 per stage
//   4 output warps  TMEM -> scales -> bf16 / float32 -> rows of out
// The weights go through TMEM so that their float16 form costs no shared
// memory bandwidth.  Every wait has a time limit: on expiry the CTA stops,
// writes status 1, waits for its own copies and frees its TMEM.
#include <cuda.h>

#include <atomic>

#include "expert_common.cuh"

namespace ep {
namespace {

using namespace mm;

constexpr int kStages = 4;            // stages of converted operands
constexpr int kWStages = 5;           // stages of 8-bit weights
constexpr int kBK = 128;              // K of a stage
constexpr int kWBytes = 128 * kBK;    // one stage of weights
constexpr int kBBytes = 128 * kBK * 2;  // one stage of rows, float16
constexpr int kBAtom = 128 * 128;     // 64 K of 128 rows
constexpr int kThreads = 14 * 32;
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kTmemA = 256;      // A stages start here: 64 columns each
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s

struct Shared {
    uint64_t w_full[kWStages], w_empty[kWStages];
    uint64_t full[kStages], empty[kStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drained;
    uint32_t tmem;
    int abort;
    int warp_sums[8];
    int tiles[kMaxE + 1];
};
constexpr int kSmemBytes = 1024 + kStages * kBBytes + kWStages * kWBytes + (int)sizeof(Shared);

__device__ __forceinline__ uint32_t smem_u32(const void* p) {
    return (uint32_t)__cvta_generic_to_shared(p);
}

__device__ __forceinline__ void mbar_init(uint64_t* bar, int count) {
    asm volatile("mbarrier.init.shared::cta.b64 [%0], %1;" ::"r"(smem_u32(bar)), "r"(count) : "memory");
}

__device__ __forceinline__ bool mbar_try(uint32_t bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(bar), "r"(parity) : "memory");
    return done != 0;
}

// Waits for the phase with this parity to complete.  False when the CTA gave
// up (here, after the time limit, or elsewhere).
__device__ __forceinline__ bool mbar_wait(Shared* sh, uint64_t* bar, uint32_t parity) {
    const uint32_t b = smem_u32(bar);
    if (mbar_try(b, parity)) return true;
    const long long start = clock64();
    while (!mbar_try(b, parity)) {
        if (*(volatile int*)&sh->abort) return false;
        if (clock64() - start > kWaitCycles) {
            *(volatile int*)&sh->abort = 1;
            return false;
        }
    }
    return true;
}

// The same by a whole warp, with one answer.
__device__ __forceinline__ bool mbar_wait_warp(Shared* sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, mbar_wait(sh, bar, parity));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.release.cta.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
}

// Arrives on the barrier at the same place in the pair's first CTA.
template <int CG>
__device__ __forceinline__ void mbar_arrive_leader(uint64_t* bar) {
    if constexpr (CG == 1) {
        mbar_arrive(bar);
    } else {
        asm volatile(
            "{\n.reg .b32 a;\n"
            "mapa.shared::cluster.u32 a, %0, 0;\n"
            "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_u32(bar))
            : "memory");
    }
}

__device__ __forceinline__ void mbar_expect_tx(uint64_t* bar, uint32_t bytes) {
    asm volatile("mbarrier.arrive.expect_tx.shared::cta.b64 _, [%0], %1;" ::"r"(smem_u32(bar)),
                 "r"(bytes) : "memory");
}

__device__ __forceinline__ void tma_load(const CUtensorMap* map, uint64_t* bar, void* dst, int k, int row) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%3, %4}], [%2];"
        ::"r"(smem_u32(dst)), "l"(map), "r"(smem_u32(bar)), "r"(k), "r"(row) : "memory");
}

template <int CG>
__device__ __forceinline__ void mma_f16(uint32_t d, uint32_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    const uint32_t acc = accumulate ? 1u : 0u;
    if constexpr (CG == 1)
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::1.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else
        asm volatile(
            "{\n.reg .pred p;\nsetp.ne.u32 p, %4, 0;\n"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], [%1], %2, %3, p;\n}\n"
            ::"r"(d), "r"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
}

// All MMAs issued so far by this thread arrive on the barrier when done (of
// both CTAs of a pair).
template <int CG>
__device__ __forceinline__ void mma_commit(uint64_t* bar) {
    if constexpr (CG == 1)
        asm volatile("tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];"
                     ::"r"(smem_u32(bar)) : "memory");
    else
        asm volatile(
            "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
            ::"r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
}

__device__ __forceinline__ void tmem_fence_before() {
    asm volatile("tcgen05.fence::before_thread_sync;" ::: "memory");
}
__device__ __forceinline__ void tmem_fence_after() {
    asm volatile("tcgen05.fence::after_thread_sync;" ::: "memory");
}

__device__ __forceinline__ void tmem_store32(uint32_t at, const uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x32.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31, %32};"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15]),
          "r"(r[16]), "r"(r[17]), "r"(r[18]), "r"(r[19]), "r"(r[20]), "r"(r[21]), "r"(r[22]), "r"(r[23]),
          "r"(r[24]), "r"(r[25]), "r"(r[26]), "r"(r[27]), "r"(r[28]), "r"(r[29]), "r"(r[30]), "r"(r[31])
        : "memory");
}

__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

// Four 8-bit integers -> four float16: with the sign bit flipped a byte u is
// v + 128, the half 0x6400 | u is 1024 + u, and 1152 less is v, exactly.
__device__ __forceinline__ void widen4(uint32_t x, uint32_t& lo, uint32_t& hi) {
    x ^= 0x80808080u;
    lo = __byte_perm(x, 0x64646464u, 0x4140);
    hi = __byte_perm(x, 0x64646464u, 0x4342);
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(lo) : "r"(0x64806480u));
    asm("sub.rn.f16x2 %0, %0, %1;" : "+r"(hi) : "r"(0x64806480u));
}

// K-major operand of 128-byte rows with the 128-byte swizzle: groups of 8 rows
// are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

struct Unit {
    int e, begin;    // expert, its first position in expert-major order
    int channel;     // first channel of the CTA pair (or CTA)
    int first, rows; // rows of the expert in this tile
    int n;           // rows rounded up to the MMA's granularity
};

template <int CG>
struct Tiles {
    static constexpr int TN = 128 * CG;
    static constexpr int kChannels = 128 * CG;
    static constexpr int kGrain = 16 * CG;
    int ct;           // channel tiles
    long long units;

    __device__ __forceinline__ Tiles(const MatmulArgs& a, const Shared* sh) {
        ct = (a.Nc + kChannels - 1) / kChannels;
        units = (long long)sh->tiles[a.E] * ct;
    }
    // An expert's units are consecutive, its row tiles innermost, so that CTAs
    // which run together share weights and rows in L2.
    __device__ __forceinline__ Unit get(const MatmulArgs& a, const Shared* sh, long long u) const {
        Unit t;
        t.e = expert_of_tile(sh->tiles, a.E, (int)(u / ct));
        const int t0 = sh->tiles[t.e], nt = sh->tiles[t.e + 1] - t0;
        const long long local = u - (long long)t0 * ct;
        const int c = (int)(local / nt), i = (int)(local - (long long)c * nt);
        const int rows = expert_rows(a, t.e, t.begin);
        const int per = ((rows + nt - 1) / nt + kGrain - 1) / kGrain * kGrain;
        t.channel = c * kChannels;
        t.first = i * per;
        t.rows = min(per, rows - t.first);
        t.n = (t.rows + kGrain - 1) / kGrain * kGrain;
        return t;
    }
};

template <int CG>
__global__ void __launch_bounds__(kThreads, 1)
matmul_tc_kernel(MatmulArgs a, const __grid_constant__ CUtensorMap w_map) {
    extern __shared__ uint8_t s_raw[];
    uint8_t* s_b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* s_w = s_b + kStages * kBBytes;
    Shared* sh = reinterpret_cast<Shared*>(s_w + kWStages * kWBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;
    constexpr int kAcc = CG == 1 ? 2 : 1;

    pdl_prologue();
    if (tid == 0) {
        sh->abort = 0;
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&sh->w_full[i], 1);
            mbar_init(&sh->w_empty[i], 4);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], 5 * CG);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 4 * CG);
        }
        mbar_init(&sh->drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (a.status != nullptr && blockIdx.x == 0) *a.status = 0;
    }
    if (warp == 13) {
        if constexpr (CG == 1)
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
    }
    tmem_fence_before();
    tile_prefix(a, Tiles<CG>::TN, sh->tiles, sh->warp_sums);
    if constexpr (CG == 2) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tmem_fence_after();
    const uint32_t tmem = sh->tmem;
    const Tiles<CG> tiles(a, sh);
    const int kblocks = (a.Kd + kBK - 1) / kBK;
    const long long u0 = blockIdx.x / CG, du = gridDim.x / CG;

    if (warp == 12) {
        // ---- weights: TMA ----
        if (lane == 0) {
            uint32_t c = 0;  // stages issued so far
            bool ok = true;
            for (long long u = u0; ok && u < tiles.units; u += du) {
                const Unit t = tiles.get(a, sh, u);
                const int row = t.e * a.Nc + t.channel + rank * 128;
                for (int kb = 0; kb < kblocks; ++kb, ++c) {
                    const uint32_t s = c % kWStages, round = c / kWStages;
                    ok = mbar_wait(sh, &sh->w_empty[s], (round & 1) ^ 1);
                    if (!ok) break;
                    mbar_expect_tx(&sh->w_full[s], kWBytes);
                    tma_load(&w_map, &sh->w_full[s], s_w + s * kWBytes, kb * kBK, row);
                }
            }
            if (!ok) {
                // the copies still in flight land before the CTA ends
                const uint32_t n = c < kWStages ? c : kWStages;
                const long long start = clock64();
                for (uint32_t i = c - n; i != c; ++i)
                    while (!mbar_try(smem_u32(&sh->w_full[i % kWStages]), (i / kWStages) & 1))
                        if (clock64() - start > kWaitCycles) break;
            }
        }
    } else if (warp == 13) {
        // ---- MMA ----
        if (rank == 0 && lane == 0) {
            uint32_t c = 0, it = 0;
            bool ok = true;
            for (long long u = u0; ok && u < tiles.units; u += du, ++it) {
                const Unit t = tiles.get(a, sh, u);
                const uint32_t acc = it % kAcc;
                // float32 accumulators, float16 operands, both K-major
                const uint32_t idesc = 1u << 4 | (uint32_t)(t.n >> 3) << 17 | (uint32_t)(128 * CG >> 4) << 24;
                ok = mbar_wait(sh, &sh->acc_empty[acc], (it / kAcc & 1) ^ 1);
                if (!ok) break;
                tmem_fence_after();
                for (int kb = 0; kb < kblocks; ++kb, ++c) {
                    const uint32_t s = c % kStages;
                    ok = mbar_wait(sh, &sh->full[s], c / kStages & 1);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint32_t b = smem_u32(s_b + s * kBBytes);
                    const int steps = min(kBK, a.Kd - kb * kBK) / 16;
#pragma unroll
                    for (int k = 0; k < kBK / 16; ++k)
                        if (k < steps)
                            mma_f16<CG>(tmem + acc * 128, tmem + kTmemA + s * 64 + k * 8,
                                        operand_desc(b + (k >> 2) * kBAtom + (k & 3) * 32), idesc,
                                        kb > 0 || k > 0);
                    mma_commit<CG>(&sh->empty[s]);
                }
                if (ok) mma_commit<CG>(&sh->acc_full[acc]);
            }
            if (!ok) {  // the MMAs in flight end before their operands' memory is given up
                mma_commit<CG>(&sh->drained);
                const long long start = clock64();
                while (!mbar_try(smem_u32(&sh->drained), 0))
                    if (clock64() - start > kWaitCycles) break;
            }
        }
    } else if (warp >= 8) {
        // ---- x rows -> float16 -> shared memory; warp w fills stage w ----
        const int s = warp - 8;
        uint32_t c = 0;
        bool ok = true;
        for (long long u = u0; ok && u < tiles.units; u += du) {
            const Unit t = tiles.get(a, sh, u);
            const int half = t.n / CG, r0 = rank * half;  // this CTA's rows of the tile
            int src[4];
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int r = r0 + i * 32 + lane;
                src[i] = (i * 32 + lane < half && r < t.rows) ? source_row(a, t.e, t.begin, t.first + r) : -1;
            }
            for (int kb = 0; kb < kblocks; ++kb, ++c) {
                if ((c % kStages) != (uint32_t)s) continue;
                const int chunk = lane & 7;
                const int k = kb * kBK + chunk * 16;
                const bool in_k = k < a.Kd;
                uint8_t* atom = s_b + s * kBBytes + (chunk >> 2) * kBAtom;
                const int c0 = (chunk & 3) * 2 + (chunk >> 2);  // the half stored first
                bool waited = false;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    if (i * 32 >= half) break;
                    uint4 q[8];
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int row = __shfl_sync(kFull, src[i], j * 4 + (lane >> 3));
                        q[j] = make_uint4(0u, 0u, 0u, 0u);
                        if (row >= 0 && in_k)
                            q[j] = __ldg(reinterpret_cast<const uint4*>(a.x + (size_t)row * a.Kd + k));
                    }
                    if (!waited) {
                        ok = mbar_wait_warp(sh, &sh->empty[s], (c / kStages & 1) ^ 1);
                        waited = true;
                        if (!ok) break;
                    }
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        const int r = i * 32 + j * 4 + (lane >> 3);
                        uint4 lo, hi;
                        widen4(q[j].x, lo.x, lo.y);
                        widen4(q[j].y, lo.z, lo.w);
                        widen4(q[j].z, hi.x, hi.y);
                        widen4(q[j].w, hi.z, hi.w);
                        // chunks 4..7 store their second half first: the 8 lanes of a row then
                        // cover all 8 bank groups
                        uint8_t* at = atom + r * 128;
                        const bool swap = (chunk >> 2) != 0;
                        *reinterpret_cast<uint4*>(at + ((c0 ^ (r & 7)) << 4)) = swap ? hi : lo;
                        *reinterpret_cast<uint4*>(at + (((c0 ^ 1) ^ (r & 7)) << 4)) = swap ? lo : hi;
                    }
                }
                if (!ok) break;
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_leader<CG>(&sh->full[s]);
            }
        }
        // the last MMAs' arrivals on this stage land before the CTA ends
        const uint32_t uses = c / kStages + (c % kStages > (uint32_t)s ? 1 : 0);
        if (ok && uses > 0) mbar_wait_warp(sh, &sh->empty[s], (uses - 1) & 1);
    } else if (warp >= 4) {
        // ---- weights -> float16 -> TMEM ----
        const int quarter = warp - 4;
        const int row = quarter * 32 + lane;
        uint32_t c = 0;
        bool ok = true;
        for (long long u = u0; ok && u < tiles.units; u += du) {
            for (int kb = 0; kb < kblocks; ++kb, ++c) {
                const uint32_t sw = c % kWStages, s = c % kStages;
                ok = mbar_wait_warp(sh, &sh->w_full[sw], c / kWStages & 1);
                if (!ok) break;
                const uint8_t* from = s_w + sw * kWBytes + row * 128;
                uint32_t r[64];
#pragma unroll
                for (int j = 0; j < 8; ++j) {
                    const uint4 q = *reinterpret_cast<const uint4*>(from + ((j ^ (row & 7)) << 4));
                    widen4(q.x, r[j * 8], r[j * 8 + 1]);
                    widen4(q.y, r[j * 8 + 2], r[j * 8 + 3]);
                    widen4(q.z, r[j * 8 + 4], r[j * 8 + 5]);
                    widen4(q.w, r[j * 8 + 6], r[j * 8 + 7]);
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->w_empty[sw]);
                ok = mbar_wait_warp(sh, &sh->empty[s], (c / kStages & 1) ^ 1);
                if (!ok) break;
                tmem_fence_after();
                const uint32_t at = tmem + ((uint32_t)quarter << 21) + kTmemA + s * 64;
                tmem_store32(at, reinterpret_cast<const uint32_t(&)[32]>(r[0]));
                tmem_store32(at + 32, reinterpret_cast<const uint32_t(&)[32]>(r[32]));
                asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
                tmem_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive_leader<CG>(&sh->full[s]);
            }
        }
    } else {
        // ---- accumulators -> out ----
        uint32_t it = 0;
        bool ok = true;
        for (long long u = u0; ok && u < tiles.units; u += du, ++it) {
            const Unit t = tiles.get(a, sh, u);
            const uint32_t acc = it % kAcc;
            const int ch = t.channel + rank * 128 + warp * 32 + lane;
            const float ws = ch < a.Nc ? __ldg(a.w_scales + (size_t)t.e * a.Nc + ch) : 0.0f;
            const size_t base = (first_row(a, t.e, t.begin) + t.first) * a.Nc + ch;
            ok = mbar_wait_warp(sh, &sh->acc_full[acc], it / kAcc & 1);
            if (!ok) break;
            tmem_fence_after();
            const uint32_t from = tmem + ((uint32_t)warp << 21) + acc * 128;
            float xs = 0.0f;
            for (int n0 = 0; n0 < t.n; n0 += 16) {
                if ((n0 & 31) == 0) {
                    const int r = n0 + lane;
                    const int src = r < t.rows ? source_row(a, t.e, t.begin, t.first + r) : -1;
                    xs = src >= 0 ? __ldg(a.x_scales + src) : 0.0f;
                }
                uint32_t v[16];
                tmem_load16(from + n0, v);
#pragma unroll
                for (int j = 0; j < 16; ++j) {
                    const float x = __shfl_sync(kFull, xs, (n0 & 16) + j);
                    const float y = __uint_as_float(v[j]) * x * ws;
                    if (n0 + j < t.rows && ch < a.Nc) {
                        const size_t at = base + (size_t)(n0 + j) * a.Nc;
                        if (a.out_bf16) static_cast<__nv_bfloat16*>(a.out)[at] = __float2bfloat16_rn(y);
                        else static_cast<float*>(a.out)[at] = y;
                    }
                }
            }
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_leader<CG>(&sh->acc_empty[acc]);
        }
    }

    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    if constexpr (CG == 2) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tmem_fence_after();
    if (warp == 13) {
        if constexpr (CG == 1) {
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        } else {
            asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
            asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
        }
    }
    if (tid == 0 && sh->abort != 0 && a.status != nullptr) *a.status = 1;
}

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

// The driver's tensor map encoder (a host function; looked up once).
EncodeTiled encode_tiled() {
    static std::atomic<void*> found{nullptr};
    void* f = found.load(std::memory_order_acquire);
    if (f == nullptr) {
        cudaDriverEntryPointQueryResult result;
        if (cudaGetDriverEntryPointByVersion("cuTensorMapEncodeTiled", &f, 12000, cudaEnableDefault,
                                             &result) != cudaSuccess ||
            result != cudaDriverEntryPointSuccess)
            return nullptr;
        found.store(f, std::memory_order_release);
    }
    return reinterpret_cast<EncodeTiled>(f);
}

// Grid of the persistent kernel on the current device: a CTA per SM, or as
// many pairs as the device holds at once (an SM without a neighbour in its
// cluster cannot host half a pair).  Looked up once per device.
template <int CG>
cudaError_t persistent_grid(int* grid) {
    static std::atomic<int> cached[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    int n = dev >= 0 && dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (n <= 0) {
        err = cudaFuncSetAttribute(matmul_tc_kernel<CG>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes);
        if (err != cudaSuccess) return err;
        n = sm_count();
        if (CG == 2) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(n / 2 * 2);
            cfg.blockDim = dim3(kThreads);
            cfg.dynamicSmemBytes = kSmemBytes;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = 2;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int pairs = 0;
            err = cudaOccupancyMaxActiveClusters(&pairs, matmul_tc_kernel<CG>, &cfg);
            if (err != cudaSuccess) return err;
            if (pairs < 1) return cudaErrorInvalidConfiguration;
            n = 2 * pairs;
        }
        if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    }
    *grid = n;
    return cudaSuccess;
}

template <int CG>
cudaError_t launch_tc(const MatmulArgs& a, cudaStream_t s) {
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    CUtensorMap map;
    const cuuint64_t dims[2] = {(cuuint64_t)a.Kd, (cuuint64_t)a.E * a.Nc};
    const cuuint64_t strides[1] = {(cuuint64_t)a.Kd};
    const cuuint32_t box[2] = {kBK, 128}, steps[2] = {1, 1};
    if (encode(&map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(a.w), dims, strides, box, steps,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    int grid = 0;
    const cudaError_t err = persistent_grid<CG>(&grid);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = kSmemBytes;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (CG == 2) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = 2;
        attr[n].val.clusterDim.y = attr[n].val.clusterDim.z = 1;
        ++n;
    }
    if (pdl_enabled()) {
        attr[n].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        attr[n].val.programmaticStreamSerializationAllowed = 1;
        ++n;
    }
    cfg.attrs = attr;
    cfg.numAttrs = n;
    return cudaLaunchKernelEx(&cfg, matmul_tc_kernel<CG>, a, map);
}

}  // namespace

cudaError_t launch_matmul_tc(const MatmulArgs& a, bool pair, cudaStream_t s) {
    return pair ? launch_tc<2>(a, s) : launch_tc<1>(a, s);
}

}  // namespace ep
