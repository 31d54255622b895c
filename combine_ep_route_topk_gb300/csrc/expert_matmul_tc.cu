// Experts' products in 8-bit integers on the tensor cores of sm_103a
// (ep_expert_matmul with more than a few rows per expert).
//
//   out[r, n] = xs[r] * ws[e, n] * sum_k x[r, k] * w[e, n, k]
//
// The integer tensor rate of this chip is a small fraction of its 16-bit rate,
// and every 8-bit integer is a float16: the codes are widened on the chip and
// multiplied by tcgen05.mma kind::f16 with float32 accumulators.  A product of
// two codes is an integer of at most 2^14, so sums below 2^24 in magnitude are
// exact (always up to K = 1024).  Beyond, each of the K / 16 additions may lose up
// to 2^-23 of the sum so far: with every code 127, 4.6e-5 of the sum at K = 65536
// and nothing measurable at 7168; with random codes of one sign 7e-8 at 7168 and
// 1.5e-5 at 65536.  That is below a bf16 output's rounding (2e-3), not always below
// a float32's; codes of both signs do not get there.
//
// A tile is 128 channels a CTA (the M side: weights) x up to TN rows (the N
// side).  CG = 1: one CTA.  CG = 2: a pair of CTAs on 256 channels, each
// holding half of the rows' operand.
//   TMA warp        weights, [128 channels x 128 bytes] boxes, 128-byte swizzle
//   2 copying warps x rows, wherever they lie, by 16-byte background copies
//   8 weight warps  8-bit stages -> float16 -> TMEM (the A operand's stages)
//   row warps       8-bit stages -> float16 -> shared memory (B)
//   MMA warp        one elected thread issues 8 MMAs of K = 16 per stage
//   8 output warps  the list of tiles and of their rows of x, in turn;
//                   TMEM -> scales -> bf16 / float32 -> rows of out
// Within a block of 128 K, both operands hold the first 8 K of each 16 in one
// half of a stage and the second 8 in the other (a sum's order is free): a row's
// 8 lanes then store to 8 different banks' groups without exchanging halves.
// The weights go through TMEM so that their float16 form costs no shared
// memory bandwidth.  Every wait has a time limit: on expiry the CTA stops,
// writes status 1, waits for its own copies and MMAs and frees its TMEM.
//
// What bounds it: with few rows per expert the weights' bytes (32 experts of
// 4096 x 7168, 8 rows each: 150 us = 6.3 TB/s of the 6.7 that a copy reaches),
// with many the tensor cores (1024 rows each: 0.98 ms = 1.96 PFLOP/s, where a
// large library product of bf16 reaches 1.95; 1.72 M cycles, of which the MMAs
// take 1.55 M).  In between, shared memory (205 rows a tile: 110 to 136 KB a
// block and CTA, about 1000 of its 1150 cycles; the MMAs take 820) and, where K
// is short, a tile's start and end.
#include <cuda.h>

#include <algorithm>
#include <atomic>
#include <cmath>

#include "expert_common.cuh"

namespace ep {
namespace {

using namespace mm;

constexpr int kBK = 128;              // K of a stage
constexpr int kWBytes = 128 * kBK;    // one stage of 8-bit weights
constexpr int kOutWarps = 8, kWeightWarp0 = kOutWarps, kWeightWarps = 8;
constexpr int kTmaWarp = kWeightWarp0 + kWeightWarps, kMmaWarp = kTmaWarp + 1;
constexpr int kCopyWarp0 = kMmaWarp + 1, kCopyWarps = 2;
constexpr int kRowWarp0 = kCopyWarp0 + kCopyWarps;  // two row warps for every 32 rows of a stage
constexpr uint32_t kTmemCols = 512;
constexpr uint32_t kWaitHint = 2000;  // ns that one poll of a barrier may sleep
constexpr long long kWaitCycles = 4000000000ll;  // about 2 s

// Rows per tile TN, of which each CTA of the CG holds kRows in shared memory.
// KS > 1: the KS CTAs of a cluster divide a tile's K among them and join their
// sums through each other's shared memory.
template <int CG_, int TN_, int KS_ = 1>
struct Shape {
    static constexpr int CG = CG_, TN = TN_, KS = KS_;
    static constexpr int kCluster = CG * KS;
    static_assert(KS == 1 || (CG == 1 && TN == 64), "sums are joined in 4 groups of 16 rows");
    static constexpr int kRows = TN / CG;
    static constexpr int kBAtom = kRows * 128;       // 64 K of the rows, float16
    static constexpr int kBBytes = 2 * kBAtom;       // one stage
    static constexpr int kXBytes = kRows * kBK;      // one stage of 8-bit rows
    static constexpr int kStages = kRows <= 64 ? 4 : 3;   // converted operands
    static constexpr int kWStages = kRows <= 80 && KS == 1 ? 6 : 4;  // 8-bit weights in flight
    static constexpr int kXStages = kRows <= 80 ? 4 : 2;  // 8-bit rows in flight
    static constexpr int kRowWarps = 2 * ((kRows + 31) / 32);
    static constexpr int kThreads = (kRowWarp0 + kRowWarps) * 32;
    // accumulators of TN columns, then the weights' stages of 64
    static constexpr int kAcc = 2 * TN + kStages * 64 <= (int)kTmemCols ? 2 : 1;
    static constexpr uint32_t kTmemA = kAcc * TN;
    static constexpr int kChannels = 128 * CG;
    static constexpr int kGrain = 16;                // an MMA's N is a multiple
    static constexpr int kPartBytes = KS > 1 ? 4 * 16 * 128 * 4 : 0;  // [KS][4 / KS groups][16 rows][128 channels]
    static_assert(kBAtom % 1024 == 0 && kTmemA + kStages * 64 <= kTmemCols, "swizzle, TMEM");
};

constexpr int kMaxStages = 4, kMaxWStages = 6, kMaxXStages = 4;
// Units are published by the output warps in turn, kOutWarps ahead of the one
// whose sums they wait for: the waits for the offsets and for the index of the
// rows lie off the path of the operands.  A slot is written again when the MMAs
// of the unit kOutWarps - 1 after its own are over, and with them every other
// warp's reading of it (the output warps are at most 2 units apart).
constexpr int kUnitSlots = 2 * kOutWarps;
constexpr int kOutPitch = 80;
struct Shared {
    uint64_t w_full[kMaxWStages], w_empty[kMaxWStages];
    uint64_t x_full[kMaxXStages], x_empty[kMaxXStages];
    uint64_t full[kMaxStages], empty[kMaxStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t drained;
    uint64_t part_full, part_empty;
    uint64_t unit_full[kUnitSlots];
    int4 unit[kUnitSlots];
    int source[kUnitSlots][128];       // of a unit's rows in this CTA: rows of x
    float row_scales[kOutWarps][128];  // of the rows that an output warp stores
    // 16 rows x 32 channels of an output warp on their way to memory; rows 80
    // bytes apart, so that the 8 rows of a stored matrix hit different banks
    uint8_t out[kOutWarps][16 * kOutPitch];
    uint32_t tmem;
    int abort;
    long long warp_sums[kTileGroups / 32];
    int tiles[kTileGroups + 1];
};
template <class S>
constexpr int kSmemBytes = 1024 + S::kStages * S::kBBytes + S::kWStages * kWBytes + S::kXStages * S::kXBytes +
                           S::kPartBytes + (int)sizeof(Shared);

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

// The barrier's and a float's place in CTA `cta` of the cluster, with the order
// that data passed between CTAs by ordinary stores needs.
__device__ __forceinline__ void mbar_arrive_cluster(uint64_t* bar, uint32_t cta) {
    asm volatile(
        "{\n.reg .b32 a;\n"
        "mapa.shared::cluster.u32 a, %0, %1;\n"
        "mbarrier.arrive.release.cluster.shared::cluster.b64 _, [a];\n}\n" ::"r"(smem_u32(bar)), "r"(cta)
        : "memory");
}
__device__ __forceinline__ void store_cluster(uint32_t at, uint32_t cta, float v) {
    asm volatile(
        "{\n.reg .b32 a;\n"
        "mapa.shared::cluster.u32 a, %0, %1;\n"
        "st.shared::cluster.f32 [a], %2;\n}\n" ::"r"(at), "r"(cta), "f"(v) : "memory");
}
// A whole warp's wait for what other CTAs stored.
__device__ __forceinline__ bool mbar_wait_cluster(Shared* sh, uint64_t* bar, uint32_t parity) {
    const bool ok = mbar_wait_warp(sh, bar, parity);
    asm volatile("fence.acq_rel.cluster;" ::: "memory");
    return ok;
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

// 16 bytes to shared memory, in the background (zeros where !on).
__device__ __forceinline__ void copy16(uint32_t dst, const int8_t* src, bool on) {
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
// Arrives on the barrier once the thread's copies so far have landed.
__device__ __forceinline__ void copies_arrive(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
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

__device__ __forceinline__ void tmem_store16(uint32_t at, const uint32_t (&r)[16]) {
    asm volatile(
        "tcgen05.st.sync.aligned.32x32b.x16.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, "
        "%14, %15, %16};"
        ::"r"(at), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]),
          "r"(r[8]), "r"(r[9]), "r"(r[10]), "r"(r[11]), "r"(r[12]), "r"(r[13]), "r"(r[14]), "r"(r[15])
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

// 16 lanes (channels) x 16 columns: registers 4 g .. 4 g + 3 hold columns 8 g +
// 2 (lane % 4) and the next, of channel lane / 4 and of channel lane / 4 + 8.
__device__ __forceinline__ void tmem_load_tile(uint32_t at, float (&r)[8]) {
    asm volatile("tcgen05.ld.sync.aligned.16x256b.x2.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
                 : "=f"(r[0]), "=f"(r[1]), "=f"(r[2]), "=f"(r[3]), "=f"(r[4]), "=f"(r[5]), "=f"(r[6]), "=f"(r[7])
                 : "r"(at) : "memory");
}

// Four 8 x 8 matrices of 16-bit values, transposed; lane i gives the address of
// row i % 8 of matrix i / 8.
__device__ __forceinline__ void store_matrices(uint32_t at, uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    asm volatile("stmatrix.sync.aligned.m8n8.x4.trans.shared.b16 [%0], {%1, %2, %3, %4};"
                 ::"r"(at), "r"(a), "r"(b), "r"(c), "r"(d) : "memory");
}

__device__ __forceinline__ uint32_t pack_bf16(float lo, float hi) {
    const __nv_bfloat162 v = __floats2bfloat162_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&v);
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

__device__ __forceinline__ uint4 load_shared(uint32_t at) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(at) : "memory");
    return v;
}
__device__ __forceinline__ void store_shared(uint32_t at, uint4 v) {
    asm volatile("st.shared.v4.b32 [%0], {%1, %2, %3, %4};"
                 ::"r"(at), "r"(v.x), "r"(v.y), "r"(v.z), "r"(v.w) : "memory");
}

// 16 codes of a row, widened: the first 8 to one half of a stage, the second to
// the other.
template <int ATOM>
__device__ __forceinline__ void widen_row(uint32_t to, uint4 q) {
    uint4 v;
    widen4(q.x, v.x, v.y);
    widen4(q.y, v.z, v.w);
    store_shared(to, v);
    widen4(q.z, v.x, v.y);
    widen4(q.w, v.z, v.w);
    store_shared(to + ATOM, v);
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

// Units of one CTA (or pair): u0, u0 + du, ...  (A unit covers some 2^13
// elements of an output in memory, so all of them are fewer than 2^32, unless
// the offsets' ranges overlap: then the first 2^32 - 1 are taken.)
template <class S>
__device__ __forceinline__ uint32_t unit_count(const MatmulArgs& a, const Shared* sh, uint32_t u0, uint32_t du) {
    const uint64_t ct = ((uint32_t)a.Nc + S::kChannels - 1) / S::kChannels;
    const uint32_t all = (uint32_t)min((uint64_t)UINT32_MAX, (uint64_t)sh->tiles[kTileGroups] * ct);
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
    __device__ __forceinline__ int4 next(const MatmulArgs& a, const Shared* sh) {
        while (sh->tiles[group + 1] <= (int)tile) ++group;
        const ExpertTile x = expert_in_group(a, S::TN, sh->tiles, group, (int)tile);
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

template <class S>
__device__ __forceinline__ Unit unpack(int4 q) {
    Unit t;
    t.e = q.x & (kMaxE - 1);
    t.begin = q.y;
    t.channel = q.z * S::kChannels;
    t.first = q.w;
    t.rows = q.x >> 10;
    t.n = (t.rows + S::kGrain - 1) / S::kGrain * S::kGrain;
    return t;
}

// Unit u of this CTA, once it is published (by a whole warp).
template <class S>
__device__ __forceinline__ bool get_unit(Shared* sh, uint32_t u, Unit& t) {
    if (!mbar_wait_warp(sh, &sh->unit_full[u % kUnitSlots], u / kUnitSlots & 1)) return false;
    t = unpack<S>(sh->unit[u % kUnitSlots]);
    return true;
}

template <class S>
__global__ void __launch_bounds__(S::kThreads, 1)
matmul_tc_kernel(MatmulArgs a, const __grid_constant__ CUtensorMap w_map) {
    constexpr int CG = S::CG, kAcc = S::kAcc, kStages = S::kStages, kWStages = S::kWStages, kXStages = S::kXStages;
    constexpr int kBBytes = S::kBBytes, kBAtom = S::kBAtom, KS = S::KS;
    extern __shared__ uint8_t s_raw[];
    uint8_t* s_b = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
    uint8_t* s_w = s_b + kStages * kBBytes;
    uint8_t* s_x = s_w + kWStages * kWBytes;
    uint8_t* s_part = s_x + kXStages * S::kXBytes;
    Shared* sh = reinterpret_cast<Shared*>(s_part + S::kPartBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int rank = CG == 2 ? (int)(blockIdx.x & 1) : 0;  // of the pair
    const int part = KS > 1 ? (int)(blockIdx.x % KS) : 0;   // of K

    pdl_prologue();
    if (tid == 0) {
        sh->abort = 0;
        for (int i = 0; i < kWStages; ++i) {
            mbar_init(&sh->w_full[i], 1);
            mbar_init(&sh->w_empty[i], 4);
        }
        for (int i = 0; i < kXStages; ++i) {
            mbar_init(&sh->x_full[i], kCopyWarps * 32);
            mbar_init(&sh->x_empty[i], S::kRowWarps / 2);
        }
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], (4 + S::kRowWarps / 2) * CG);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], kOutWarps * CG);
        }
        for (int i = 0; i < kUnitSlots; ++i) mbar_init(&sh->unit_full[i], 1);
        mbar_init(&sh->drained, 1);
        mbar_init(&sh->part_full, kOutWarps * KS);
        mbar_init(&sh->part_empty, kOutWarps * KS);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (a.status != nullptr && blockIdx.x == 0) *a.status = 0;
    }
    if (warp == kMmaWarp) {
        if constexpr (CG == 1)
            asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
        else
            asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                         ::"r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
    }
    tmem_fence_before();
    tile_prefix(a, S::TN, sh->tiles, sh->warp_sums);
    if constexpr (S::kCluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tmem_fence_after();
    const uint32_t tmem = sh->tmem;
    const uint32_t cluster = blockIdx.x / S::kCluster, clusters = gridDim.x / S::kCluster;
    const uint32_t units = unit_count<S>(a, sh, cluster, clusters);
    // this CTA's blocks of K: kb0 .. kb1 - 1, at least one (the launcher sees to it)
    const int all_blocks = (a.Kd + kBK - 1) / kBK;
    const int kb0 = all_blocks * part / KS, kb1 = all_blocks * (part + 1) / KS, kblocks = kb1 - kb0;

    if (warp == kTmaWarp) {
        // ---- the weights' TMA boxes ----
        uint32_t c = 0;  // stages issued so far
        bool ok = true;
        for (uint32_t u = 0; ok && u < units; ++u) {
            Unit t;
            ok = get_unit<S>(sh, u, t);
            if (!ok) break;
            const int row = t.e * a.Nc + t.channel + rank * 128;
            for (int kb = kb0; kb < kb1; ++kb, ++c) {
                const uint32_t s = c % kWStages;
                ok = mbar_wait_warp(sh, &sh->w_empty[s], (c / kWStages & 1) ^ 1);
                if (!ok) break;
                if (elect_one()) {
                    mbar_expect_tx(&sh->w_full[s], kWBytes);
                    tma_load(&w_map, &sh->w_full[s], s_w + s * kWBytes, kb * kBK, row);
                }
                __syncwarp();
            }
        }
        if (!ok && lane == 0) drain_copies<kWStages>(sh->w_full, c);
    } else if (warp == kMmaWarp) {
        // ---- MMA: the warp waits together, one elected lane issues ----
        if (rank == 0) {
            const uint64_t desc0 = operand_desc(smem_u32(s_b));
            uint32_t c = 0, it = 0;
            bool ok = true;
            for (uint32_t u = 0; ok && u < units; ++u, ++it) {
                Unit t;
                ok = get_unit<S>(sh, u, t);
                if (!ok) break;
                const uint32_t acc = it % kAcc;
                // float32 accumulators, float16 operands, both K-major
                const uint32_t idesc = 1u << 4 | (uint32_t)(t.n >> 3) << 17 | (uint32_t)(128 * CG >> 4) << 24;
                ok = mbar_wait_warp(sh, &sh->acc_empty[acc], (it / kAcc & 1) ^ 1);
                if (!ok) break;
                const uint32_t d = tmem + acc * S::TN;
                for (int kb = kb0; kb < kb1; ++kb, ++c) {
                    const uint32_t s = c % kStages;
                    ok = mbar_wait_warp(sh, &sh->full[s], c / kStages & 1);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint32_t at = tmem + S::kTmemA + s * 64;
                    const uint64_t desc = desc0 + (uint64_t)(s * (kBBytes >> 4));
                    // 16-byte pieces of the block's rows: each gives 8 K to either atom
                    const int pieces = min(8, (a.Kd - kb * kBK) / 16);
                    if (elect_one()) {
                        if (pieces > 6) {
#pragma unroll
                            for (int k = 0; k < kBK / 16; ++k)
                                mma_f16<CG>(d, at + k * 8, desc + ((k >> 2) * kBAtom + (k & 3) * 32 >> 4), idesc,
                                            k > 0 || kb > kb0);
                        } else {  // the last, short block
                            for (int k = 0; k < kBK / 16; ++k)
                                if ((k & 3) * 2 < pieces)
                                    mma_f16<CG>(d, at + k * 8, desc + ((k >> 2) * kBAtom + (k & 3) * 32 >> 4),
                                                idesc, k > 0 || kb > kb0);
                        }
                        mma_commit<CG>(&sh->empty[s]);
                        if (kb == kb1 - 1) mma_commit<CG>(&sh->acc_full[acc]);
                    }
                    __syncwarp();
                }
            }
            if (!ok && c > 0) {  // the MMAs in flight end before their operands' memory is given up
                if (elect_one()) {
                    mma_commit<CG>(&sh->drained);
                    const long long start = clock64();
                    while (!mbar_try(smem_u32(&sh->drained), 0))
                        if (clock64() - start > kWaitCycles) break;
                }
                __syncwarp();
            }
        }
    } else if (warp >= kCopyWarp0 && warp < kRowWarp0) {
        // ---- x rows, wherever they lie, -> shared memory in the background;
        // 8 lanes a row, each copying warp half of the rows ----
        constexpr int kPer = S::kRows / kCopyWarps / 4;  // rows per lane
        const int chunk = lane & 7, l8 = lane >> 3;
        const int r0 = (warp - kCopyWarp0) * 4 + l8;     // then every 8th row
        const uint32_t to = smem_u32(s_x) + r0 * kBK + chunk * 16;
        uint32_t c = 0;
        bool ok = true;
        for (uint32_t u = 0; ok && u < units; ++u) {
            Unit t;
            ok = get_unit<S>(sh, u, t);
            if (!ok) break;
            const int half = t.n / CG;  // this CTA's rows of the tile, a multiple of 8
            const int8_t* src[kPer];
#pragma unroll
            for (int i = 0; i < kPer; ++i)
                src[i] = a.x + (size_t)sh->source[u % kUnitSlots][r0 + i * 8] * a.Kd + chunk * 16;
            for (int kb = kb0; kb < kb1; ++kb, ++c) {
                const uint32_t s = c % kXStages;
                ok = mbar_wait_warp(sh, &sh->x_empty[s], (c / kXStages & 1) ^ 1);
                if (!ok) break;
                const uint32_t dst = to + s * S::kXBytes;
                if (kb * kBK + kBK <= a.Kd) {
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (i * 8 < half) copy16(dst + i * 8 * kBK, src[i] + kb * kBK, true);
                } else {  // the last, short block: zeros past Kd
                    const bool on = kb * kBK + chunk * 16 < a.Kd;
#pragma unroll
                    for (int i = 0; i < kPer; ++i)
                        if (i * 8 < half) copy16(dst + i * 8 * kBK, on ? src[i] + kb * kBK : a.x, on);
                }
                copies_arrive(&sh->x_full[s]);
            }
        }
        asm volatile("cp.async.wait_all;" ::: "memory");
    } else if (warp >= kRowWarp0) {
        // ---- x rows -> float16 -> shared memory; two groups of warps take
        // turns, 32 rows a warp, 8 lanes a row ----
        constexpr int kGroup = S::kRowWarps / 2;
        const int group = (warp - kRowWarp0) / kGroup, r0 = (warp - kRowWarp0) % kGroup * 32;
        const int chunk = lane & 7, l8 = lane >> 3;
        const uint32_t from = smem_u32(s_x) + (r0 + l8) * kBK + chunk * 16;
        const uint32_t at = smem_u32(s_b) + (r0 + l8) * 128 + ((chunk ^ l8) << 4);
        uint32_t c = group, c1 = 0;
        bool ok = true;
        for (uint32_t u = 0; ok && u < units; ++u) {
            Unit t;
            ok = get_unit<S>(sh, u, t);
            if (!ok) break;
            const int mine = t.n / CG - r0;  // rows of this warp, if any, in eights
            c1 += kblocks;
            for (; c < c1; c += 2) {
                const uint32_t sx = c % kXStages, s = c % kStages;
                ok = mbar_wait_warp(sh, &sh->x_full[sx], c / kXStages & 1);
                if (!ok) break;
                uint4 q[8];
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (mine > j / 2 * 8) q[j] = load_shared(from + sx * S::kXBytes + j * 4 * kBK);
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->x_empty[sx]);
                ok = mbar_wait_warp(sh, &sh->empty[s], (c / kStages & 1) ^ 1);
                if (!ok) break;
                const uint32_t to = at + s * kBBytes;
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    if (mine > j / 2 * 8) widen_row<kBAtom>((to ^ (j & 1) * 64) + j * 4 * 128, q[j]);
                asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive_leader<CG>(&sh->full[s]);
            }
        }
        // the last MMAs' arrivals on each stage land before the CTA ends
        for (uint32_t i = c1 < kStages ? 0 : c1 - kStages; ok && i < c1; ++i)
            ok = mbar_wait_warp(sh, &sh->empty[i % kStages], i / kStages & 1);
    } else if (warp >= kWeightWarp0) {
        // ---- weights -> float16 -> TMEM; two groups of 4 warps take turns ----
        // (kWStages and kXStages are even, so that a group sees every phase of
        // the 8-bit stages it uses.  Of a converted stage it sees every second
        // phase; MMAs end in order, so its wait two blocks before has shown it
        // that the phase which has the same parity is over.)
        const int quarter = warp & 3, group = (warp - kWeightWarp0) >> 2;
        const int row = quarter * 32 + lane;
        const uint32_t from = smem_u32(s_w) + row * 128 + ((row & 7) << 4);
        const uint32_t to = tmem + ((uint32_t)quarter << 21) + S::kTmemA;
        const uint32_t total = units * kblocks;
        bool ok = true;
        for (uint32_t c = group; ok && c < total; c += 2) {
            const uint32_t sw = c % kWStages, s = c % kStages;
            ok = mbar_wait_warp(sh, &sh->w_full[sw], c / kWStages & 1);
            if (!ok) break;
            uint4 q[8];
#pragma unroll
            for (int j = 0; j < 8; ++j) q[j] = load_shared((from + sw * kWBytes) ^ (j * 16));
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->w_empty[sw]);
            ok = mbar_wait_warp(sh, &sh->empty[s], (c / kStages & 1) ^ 1);
            if (!ok) break;
            tmem_fence_after();
#pragma unroll
            for (int j = 0; j < 8; j += 4) {
                uint32_t lo[16], hi[16];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    widen4(q[j + i].x, lo[i * 4], lo[i * 4 + 1]);
                    widen4(q[j + i].y, lo[i * 4 + 2], lo[i * 4 + 3]);
                }
                tmem_store16(to + s * 64 + j * 4, lo);
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    widen4(q[j + i].z, hi[i * 4], hi[i * 4 + 1]);
                    widen4(q[j + i].w, hi[i * 4 + 2], hi[i * 4 + 3]);
                }
                tmem_store16(to + s * 64 + 32 + j * 4, hi);
            }
            asm volatile("tcgen05.wait::st.sync.aligned;" ::: "memory");
            tmem_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive_leader<CG>(&sh->full[s]);
        }
    } else {
        // ---- accumulators -> out; two warps per 32 channels, 16 of every 32 rows each ----
        const int quarter = warp & 3, h = warp >> 2;
        float* row_scales = sh->row_scales[warp];
        const uint32_t stage = smem_u32(sh->out[warp]);
        const bool vectors = KS == 1 && a.out_bf16 && a.Nc % 8 == 0;  // rows of out start on 16 bytes
        const int size = a.out_bf16 ? 2 : 4;
        const size_t pitch = (size_t)a.Nc * size;
        Steps<S> steps(a, cluster + warp * clusters, kOutWarps * clusters);
        const auto publish = [&](uint32_t u) {
            const int4 packed = steps.next(a, sh);
            const Unit t = unpack<S>(packed);
            const int half = t.n / CG;
#pragma unroll
            for (int i = 0; i < S::kRows; i += 32) {
                // a row that reads nothing takes row 0: its output is scaled by 0 or not stored
                const int r = i + lane, rr = rank * half + r;
                if (S::kRows % 32 == 0 || r < S::kRows)
                    sh->source[u % kUnitSlots][r] =
                        r < half && rr < t.rows ? max(0, source_row(a, t.e, t.begin, t.first + rr)) : 0;
            }
            __syncwarp();
            if (lane == 0) {
                sh->unit[u % kUnitSlots] = packed;
                mbar_arrive(&sh->unit_full[u % kUnitSlots]);
            }
            __syncwarp();
        };
        if (warp < units) publish(warp);
        for (uint32_t u = 0; u < units; ++u) {
            if (u % kOutWarps == warp && units - u > kOutWarps) publish(u + kOutWarps);
            Unit t;
            if (!get_unit<S>(sh, u, t)) break;
            const uint32_t acc = u % kAcc;
            const int ch0 = t.channel + rank * 128 + quarter * 32;  // this warp's channels
            uint8_t* to = static_cast<uint8_t*>(a.out) +
                          (first_row(a, t.e, t.begin) + t.first) * pitch + (size_t)ch0 * size;
            for (int i = lane; i < S::TN / 2; i += 32) {
                // the warp's rows; with K divided, those that this CTA joins (the first 64 / KS)
                const int r = KS == 1 ? (i >> 4) * 32 + h * 16 + (i & 15) : ((i >> 4) * KS + part) * 16 + (i & 15);
                const int src = r < t.rows ? source_row(a, t.e, t.begin, t.first + r) : -1;
                row_scales[i] = src >= 0 ? __ldg(a.x_scales + src) : 0.0f;
            }
            const float* ws_e = a.w_scales + (size_t)t.e * a.Nc;
            float ws[4];  // of channels lane / 4 + 8 i; or the lane's own
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const int ch = ch0 + (vectors ? (lane >> 2) + i * 8 : lane);
                ws[i] = ch < a.Nc ? __ldg(ws_e + ch) : 0.0f;
            }
            __syncwarp();
            if (!mbar_wait_warp(sh, &sh->acc_full[acc], u / kAcc & 1)) break;
            tmem_fence_after();
            const uint32_t from = tmem + ((uint32_t)quarter << 21) + acc * S::TN;
            if constexpr (KS > 1) {
                // Rows 16 g .. 16 g + 15 are joined by CTA g % KS: every CTA stores its
                // sums there, and their owner adds them in the order of K.
                const uint32_t parts = smem_u32(s_part);
                const float* mine = reinterpret_cast<const float*>(s_part);
                const int ch = quarter * 32 + lane;
                if (!mbar_wait_cluster(sh, &sh->part_empty, (u & 1) ^ 1)) break;
                for (int g = h; g * 16 < t.n; g += 2) {
                    uint32_t v[16];
                    tmem_load16(from + g * 16, v);
                    const uint32_t at = parts + (((part * (4 / KS) + g / KS) * 16) * 128 + ch) * 4;
#pragma unroll
                    for (int j = 0; j < 16; ++j) store_cluster(at + j * 128 * 4, g % KS, __uint_as_float(v[j]));
                }
                tmem_fence_before();
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->acc_empty[acc]);
                if (lane < KS) mbar_arrive_cluster(&sh->part_full, lane);
                if (!mbar_wait_cluster(sh, &sh->part_full, u & 1)) break;
                for (int gl = 0; gl < 4 / KS; ++gl) {
                    const int n0 = (gl * KS + part) * 16 + h * 8;  // two warps share the 16 rows
#pragma unroll
                    for (int j = 0; j < 8; ++j) {
                        float sum = 0.0f;
#pragma unroll
                        for (int p = 0; p < KS; ++p) sum += mine[((p * (4 / KS) + gl) * 16 + h * 8 + j) * 128 + ch];
                        const float y = sum * row_scales[gl * 16 + h * 8 + j] * ws[0];
                        if (n0 + j < t.rows && ch0 + lane < a.Nc) {
                            uint8_t* at = to + (size_t)(n0 + j) * pitch + lane * size;
                            if (a.out_bf16) *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(y);
                            else *reinterpret_cast<float*>(at) = y;
                        }
                    }
                }
                asm volatile("fence.acq_rel.cluster;" ::: "memory");
                __syncwarp();
                if (lane < KS) mbar_arrive_cluster(&sh->part_empty, lane);
                continue;
            }
            if (vectors) {
                const int piece = (lane & 3) * 8;  // 8 channels of one row: 16 bytes
                const bool in = ch0 + piece < a.Nc;
                for (int n0 = h * 16, i0 = 0; n0 < t.n; n0 += 32, i0 += 16) {
                    float lo[8], hi[8];  // channels 0 .. 15 and 16 .. 31
                    tmem_load_tile(from + n0, lo);
                    tmem_load_tile(from + n0 + (16u << 16), hi);
                    asm volatile("tcgen05.wait::ld.sync.aligned;" ::: "memory");
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const float2 xs = *reinterpret_cast<const float2*>(row_scales + i0 + g * 8 + (lane & 3) * 2);
                        const int j = g * 4;
                        store_matrices(stage + (g * 8 + (lane & 7)) * kOutPitch + (lane >> 3) * 16,
                                       pack_bf16(lo[j] * xs.x * ws[0], lo[j + 1] * xs.y * ws[0]),
                                       pack_bf16(lo[j + 2] * xs.x * ws[1], lo[j + 3] * xs.y * ws[1]),
                                       pack_bf16(hi[j] * xs.x * ws[2], hi[j + 1] * xs.y * ws[2]),
                                       pack_bf16(hi[j + 2] * xs.x * ws[3], hi[j + 3] * xs.y * ws[3]));
                    }
                    __syncwarp();
#pragma unroll
                    for (int g = 0; g < 2; ++g) {
                        const int r = g * 8 + (lane >> 2);
                        const uint4 v = load_shared(stage + r * kOutPitch + piece * 2);
                        if (in && n0 + r < t.rows) *reinterpret_cast<uint4*>(to + (n0 + r) * pitch + piece * 2) = v;
                    }
                    __syncwarp();  // the stage is free again
                }
            } else {
                const int rows = ch0 + lane < a.Nc ? t.rows : 0;
                for (int n0 = h * 16, i0 = 0; n0 < t.n; n0 += 32, i0 += 16) {
                    uint32_t v[16];
                    tmem_load16(from + n0, v);
                    uint8_t* p = to + n0 * pitch + lane * size;
#pragma unroll
                    for (int j = 0; j < 16; ++j, p += pitch) {
                        const float y = __uint_as_float(v[j]) * row_scales[i0 + j] * ws[0];
                        if (n0 + j < rows) {
                            if (a.out_bf16) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(y);
                            else *reinterpret_cast<float*>(p) = y;
                        }
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
    if constexpr (S::kCluster > 1) {
        asm volatile("barrier.cluster.arrive.release.aligned;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire.aligned;" ::: "memory");
    }
    tmem_fence_after();
    if (warp == kMmaWarp) {
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
// many clusters as the device holds at once (an SM without a neighbour in its
// cluster cannot host a part of one).  Looked up once per device.
template <class S>
cudaError_t persistent_grid(int* grid) {
    static std::atomic<int> cached[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    int n = dev >= 0 && dev < 64 ? cached[dev].load(std::memory_order_relaxed) : 0;
    if (n <= 0) {
        err = cudaFuncSetAttribute(matmul_tc_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<S>);
        if (err != cudaSuccess) return err;
        n = sm_count();
        if (S::kCluster > 1) {
            cudaLaunchConfig_t cfg = {};
            cfg.gridDim = dim3(n / S::kCluster * S::kCluster);
            cfg.blockDim = dim3(S::kThreads);
            cfg.dynamicSmemBytes = kSmemBytes<S>;
            cudaLaunchAttribute attr[1];
            attr[0].id = cudaLaunchAttributeClusterDimension;
            attr[0].val.clusterDim.x = S::kCluster;
            attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
            cfg.attrs = attr;
            cfg.numAttrs = 1;
            int clusters = 0;
            err = cudaOccupancyMaxActiveClusters(&clusters, matmul_tc_kernel<S>, &cfg);
            if (err != cudaSuccess) return err;
            if (clusters < 1) return cudaErrorInvalidConfiguration;
            n = S::kCluster * clusters;
        }
        if (dev >= 0 && dev < 64) cached[dev].store(n, std::memory_order_relaxed);
    }
    *grid = n;
    return cudaSuccess;
}

template <class S>
cudaError_t launch_tc(const MatmulArgs& a, cudaStream_t s) {
    static_assert(kSmemBytes<S> <= 227 * 1024, "a CTA's shared memory");
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    CUtensorMap w_map;
    const cuuint64_t dims[2] = {(cuuint64_t)a.Kd, (cuuint64_t)a.E * a.Nc};
    const cuuint64_t strides[1] = {(cuuint64_t)a.Kd};
    const cuuint32_t box[2] = {kBK, 128}, steps[2] = {1, 1};
    if (encode(&w_map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<int8_t*>(a.w), dims, strides, box, steps,
               CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
               CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) != CUDA_SUCCESS)
        return cudaErrorInvalidValue;
    int grid = 0;
    const cudaError_t err = persistent_grid<S>(&grid);
    if (err != cudaSuccess) return err;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(grid);
    cfg.blockDim = dim3(S::kThreads);
    cfg.dynamicSmemBytes = kSmemBytes<S>;
    cfg.stream = s;
    cudaLaunchAttribute attr[2];
    int n = 0;
    if (S::kCluster > 1) {
        attr[n].id = cudaLaunchAttributeClusterDimension;
        attr[n].val.clusterDim.x = S::kCluster;
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
    return cudaLaunchKernelEx(&cfg, matmul_tc_kernel<S>, a, w_map);
}

}  // namespace

namespace {

// Cycles that a shape would take, by the waves of its tiles.  A block of K takes
// `base` cycles and `slope` more for each row of the tile (measured; the weights
// arrive, are widened and multiplied), a tile's start and end 3000, sums that are
// joined 6500 more, the launch of pairs 2000 more.  The counts of several experts scatter around their mean as
// independent picks would, which decides whether an expert needs one tile more;
// one expert's count and a capacity are taken as they are, so that a capacity far
// above the rows gets wide tiles (32 experts of 4096 x 7168 with 8 rows each: 185 us
// under a capacity of 1024, 146 under one of 16).
template <class S>
double shape_cycles(const MatmulArgs& a, double base, double slope) {
    const double mean = a.layout == 0 ? (double)a.rows / a.E : a.cap;
    const double sigma = a.layout == 0 && a.E > 1 ? std::sqrt(mean) : 0.0;
    // An expert's tiles: those that it has for sure, and one more for each multiple
    // of TN that its count may exceed.
    const double sure = std::max(1.0, sigma == 0.0 ? std::ceil(mean / S::TN) : std::floor((mean - 4.0 * sigma) / S::TN));
    double more = 0.0;
    for (int k = (int)sure; sigma > 0.0 && k * (double)S::TN < mean + 4.0 * sigma; ++k)
        more += 0.5 * std::erfc((k * S::TN - mean) / (sigma * std::sqrt(2.0)));
    const double rows = std::min((double)S::TN, std::max(1.0, mean / (sure + more)));
    const double most = a.layout == 0 ? std::min(a.E, a.rows) + std::floor((double)a.rows / S::TN) : a.E * sure;
    const double tiles = std::min(a.E * sure, most), extra = std::min(a.E * more, most - tiles);
    const auto waves = [&](double t) {
        return std::ceil(t * std::ceil(a.Nc / (double)S::kChannels) / (sm_count() / S::kCluster));
    };
    // less than one tile more is the chance of one
    const double all = extra < 1.0 ? waves(tiles) + extra * (waves(tiles + 1.0) - waves(tiles)) : waves(tiles + extra);
    const double blocks = std::ceil(std::ceil(a.Kd / (double)kBK) / S::KS);
    return all * (blocks * (base + slope * rows) + (S::KS > 1 ? 9500.0 : 3000.0)) + (S::CG > 1 ? 2000.0 : 0.0);
}

}  // namespace

// A tile that holds an expert's rows whole reads and widens its weights once;
// narrow tiles leave shared memory for more weights in flight and TMEM for a
// second accumulator, wide ones use the tensor cores better, and where there are
// few tiles K is divided among CTAs.  The shape with the least estimated cycles
// is taken.  Measured on a GB300 (us; counts drawn around their mean) with
// TN = 64, 160, 256:
//   32 experts of 4096 x 7168: mean 8 150, 153, 184; 64 211, 167, 208;
//     128 355, 187, 228; 160 435, 265, 239; 320 779, 423, 420; 512 1214, 682, 559
//   128 experts of 2880 x 1440: mean 8 94, 104, 120; 64 147, 117, 137;
//     128 240, 136, 157; 200 355, 237, 187; 512 819, 503, 436
//   19 experts of 4096 x 7168, 128 rows each (4 whole waves of 160): 175, 109, 136
// and with K whole, in 2 and in 4 parts:
//   1 expert of 4096 x 4096: 8 rows 15.6, 13.6, 12.3; 64 rows 18.0, 15.4, 13.4
//   4 experts of 4096 x 4096, 64 rows: 18.2, 22.4, 28.6
//   6 experts of 500 x 1008, 64 rows: 8.4, 9.9, 10.0
cudaError_t launch_matmul_tc(const MatmulArgs& a, cudaStream_t s) {
    const int blocks = (a.Kd + kBK - 1) / kBK;
    const double c64 = shape_cycles<Shape<1, 64>>(a, 560.0, 3.2), c160 = shape_cycles<Shape<2, 160>>(a, 620.0, 1.55),
                 c256 = shape_cycles<Shape<2, 256>>(a, 820.0, 1.6);
    const double whole = std::min(c64, std::min(c160, c256));
    const double two = blocks >= 2 ? shape_cycles<Shape<1, 64, 2>>(a, 560.0, 3.2) : whole;
    const double four = blocks >= 4 ? shape_cycles<Shape<1, 64, 4>>(a, 560.0, 3.2) : whole;
    if (std::min(two, four) < whole)
        return four < two ? launch_tc<Shape<1, 64, 4>>(a, s) : launch_tc<Shape<1, 64, 2>>(a, s);
    if (c64 == whole) return launch_tc<Shape<1, 64>>(a, s);
    return c160 == whole ? launch_tc<Shape<2, 160>>(a, s) : launch_tc<Shape<2, 256>>(a, s);
}

}  // namespace ep
