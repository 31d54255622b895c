// What the experts' products on the tensor cores share: barriers with a time limit,
// TMA and tcgen05 in inline PTX, the order in which a persistent CTA takes its
// tiles, and the tensor maps' encoder.
#pragma once

#include <cuda.h>

#include <atomic>

#include "expert_common.cuh"

namespace ep {
namespace tc {

using namespace mm;

constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWaitHint = 2000;  // ns that one poll of a barrier may sleep
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s

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
        "mbarrier.try_wait.parity.shared::cta.b64 p, [%1], %2, %3;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(bar), "r"(parity), "r"(kWaitHint) : "memory");
    return done != 0;
}

// Waits for the phase with this parity to complete.  False when the CTA gave
// up (here, after the time limit, or elsewhere).
template <class Shared>
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

__device__ __forceinline__ bool elect_one() {
    uint32_t one;
    asm volatile("{\n.reg .pred p;\nelect.sync _|p, 0xffffffff;\nselp.u32 %0, 1, 0, p;\n}\n" : "=r"(one));
    return one != 0;
}

// The same by a whole warp, with one answer.
template <class Shared>
__device__ __forceinline__ bool mbar_wait_warp(Shared* sh, uint64_t* bar, uint32_t parity) {
    return __all_sync(kFull, mbar_wait(sh, bar, parity));
}

__device__ __forceinline__ void mbar_arrive(uint64_t* bar) {
    asm volatile("mbarrier.arrive.shared::cta.b64 _, [%0];" ::"r"(smem_u32(bar)) : "memory");
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
            "mbarrier.arrive.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_u32(bar))
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

// Before a CTA that gave up ends, the copies of its last stages land (waited
// for with the same limit); c stages were issued.
template <int STAGES>
__device__ __forceinline__ void drain_copies(uint64_t* full, uint32_t c) {
    const uint32_t n = c < STAGES ? c : STAGES;
    const long long start = clock64();
    for (uint32_t i = c - n; i != c; ++i)
        while (!mbar_try(smem_u32(&full[i % STAGES]), (i / STAGES) & 1))
            if (clock64() - start > kWaitCycles) break;
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

__device__ __forceinline__ void tmem_load16(uint32_t at, uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x16.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, "
        "%15}, [%16];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]),
          "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15])
        : "r"(at) : "memory");
    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
}

// K-major operand of 128-byte rows with the 128-byte swizzle: groups of 8 rows
// are 1024 bytes apart.
__device__ __forceinline__ uint64_t operand_desc(uint32_t addr) {
    return (uint64_t)((addr >> 4) & 0x3fffu) | (uint64_t)1 << 16 | (uint64_t)(1024 >> 4) << 32 |
           (uint64_t)1 << 46 | (uint64_t)2 << 61;
}

// A shape S has tiles of S::TN rows, in multiples of S::kGrain, and S::kChannels channels.
// Units of one CTA (or pair): u0, u0 + du, ...  (A unit covers some 2^13
// elements of an output in memory, so all of them are fewer than 2^32, unless
// the offsets' ranges overlap: then the first 2^32 - 1 are taken.)
template <class S>
__device__ __forceinline__ uint32_t unit_count(const MatmulArgs& a, const int* tiles, uint32_t u0, uint32_t du) {
    const uint64_t ct = ((uint32_t)a.Nc + S::kChannels - 1) / S::kChannels;
    const uint32_t all = (uint32_t)min((uint64_t)UINT32_MAX, (uint64_t)tiles[kTileGroups] * ct);
    return all > u0 ? (all - 1 - u0) / du + 1 : 0;
}

// Steps through them, for a warp that publishes them.  An expert's units are
// consecutive, its row tiles innermost, so that CTAs which run together share
// weights and rows in L2.  The place moves without a division, and the groups
// of experts only forward.
template <class S>
struct Steps {
    uint32_t ct;             // channel tiles
    uint32_t tile, rest;     // the current unit is tile * ct + rest
    uint32_t dtile, drest;
    int group;

    __device__ __forceinline__ Steps(const MatmulArgs& a, uint32_t u0, uint32_t du) {
        ct = ((uint32_t)a.Nc + S::kChannels - 1) / S::kChannels;
        tile = u0 / ct;
        rest = u0 % ct;
        dtile = du / ct;
        drest = du % ct;
        group = 0;
    }
    // x: expert and rows of the tile; y: the expert's first position; z: channel
    // tile; w: first row of the tile among the expert's
    __device__ __forceinline__ int4 next(const MatmulArgs& a, const int* tiles) {
        while (tiles[group + 1] <= (int)tile) ++group;
        const ExpertTile x = expert_in_group(a, S::TN, tiles, group, (int)tile);
        uint32_t c = rest, i = 0, per = (uint32_t)x.rows;
        if (x.count > 1) {  // rows divided evenly among the tiles
            const uint32_t local = (tile - x.first) * ct + rest;
            c = local / (uint32_t)x.count;
            i = local - c * x.count;
            per = (per + x.count - 1) / (uint32_t)x.count;
        }
        per = (per + S::kGrain - 1) / S::kGrain * S::kGrain;
        const int first = (int)(i * per);
        tile += dtile;
        rest += drest;
        if (rest >= ct) {
            rest -= ct;
            ++tile;
        }
        return make_int4(x.e | min((int)per, x.rows - first) << 10, x.begin, (int)c, first);
    }
};

using EncodeTiled = CUresult (*)(CUtensorMap*, CUtensorMapDataType, cuuint32_t, void*, const cuuint64_t*,
                                 const cuuint64_t*, const cuuint32_t*, const cuuint32_t*,
                                 CUtensorMapInterleave, CUtensorMapSwizzle, CUtensorMapL2promotion,
                                 CUtensorMapFloatOOBfill);

// The driver's tensor map encoder (a host function; looked up once).
inline EncodeTiled encode_tiled() {
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

}  // namespace tc
}  // namespace ep
