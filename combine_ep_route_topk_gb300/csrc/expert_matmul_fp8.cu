// Experts' products of E4M3 codes with a scale for every 128 columns, for sm_103a
// (ep_expert_matmul_fp8).
//
//   out[r, n] = sum over the blocks b of 128 K of
//               xs[s, b] * ws[e, n / 128, b] * sum_{k in b} x[s, k] * w[e, n, k]
//
// The scales are float32 of any value, so they cannot ride along with the codes
// through the tensor cores: a block's sums leave them unscaled and are scaled and
// added in registers.  A tile is 128 rows (the M side, a row to a TMEM lane) by BN
// channels.  Every block of 128 K is four tcgen05.mma kind::f8f6f4 of K = 32 into
// an accumulator of its own; the accumulators of the next blocks fill while 8
// warps take one: a thread holds a row's sums of BN / 2 channels, all in one block
// of 128 channels, so one product xs * ws scales them all and each takes one fused
// multiply-add.
//   2 TMA warps weights in [BN x 128 bytes] boxes, rows of x in boxes of 32 or, with
//               row_src, 4 a copy; 128-byte swizzle
//   MMA warp    issues the MMAs
//   unit warp   the list of tiles, their rows and their scales, ahead of the others
//   8 warps     TMEM -> scales -> registers; at a tile's end -> rows of out
// Rows that a tile lacks are neither copied nor stored: what lies in their place in
// shared memory reaches their own lanes only.  Every wait has a time limit: on
// expiry the CTA stops, writes status 1, waits for its own copies and MMAs and
// frees its TMEM.
//
// What bounds it: with few rows per expert the weights' bytes (32 experts of 4096 x
// 7168, 64 rows each: 154 us = 6.3 TB/s).  With many (1024 rows each: 0.77 ms = 2.5
// PFLOP/s; 0.88 in a long loop at the 1.72 GHz that the power limit leaves) the summing
// warps: a step of 128 x 256 x 128 takes 900 cycles, of which the MMAs take 512 and a
// warp's 128 loads and multiply-adds 430 beside the other warp of its scheduler, the rest
// being its waits, arrivals and scales.  Without loads and multiply-adds the same steps
// take 830, and one accumulator for all of K (no scales) 770, which is what shared memory
// needs to be written and read (96 KB at 128 bytes a cycle).  Pairs of CTAs
// (cta_group::2), which halve that, gained nothing: 0.89 ms when this took 0.84.  Nor did
// 16 summing warps (1.03 when this took 0.77), accumulators of 128 or 160 channels (1.03,
// 1.19), taking the accumulator in two halves (0.90), two values a multiply-add (0.94)
// or spinning on the barriers (1.05).
#include <algorithm>
#include <atomic>
#include <cmath>

#include "rows_common.cuh"
#include "tc_common.cuh"

namespace ep {
namespace {

using namespace tc;

constexpr int kBK = kScaleBlock;  // K of a stage, and of a scale
constexpr int kSumWarps = 8, kTmaWarp = kSumWarps, kXWarp = kTmaWarp + 1, kMmaWarp = kXWarp + 1,
              kUnitWarp = kMmaWarp + 1, kThreads = (kUnitWarp + 1) * 32;
// Registers: 168 a thread at launch; the summing warps take 224 of what the other
// four warps give up (256 * 224 + 128 * 56 = 384 * 168).
constexpr int kLaunchRegs = 168;

template <int BN_>
struct Shape {
    static constexpr int BN = BN_;
    static constexpr int TN = 128, kGrain = 1, kChannels = BN;  // rows and channels of a tile
    static constexpr int kABytes = 128 * kBK;             // a stage's rows
    static constexpr int kBBytes = BN * kBK;              // a stage's weights
    static constexpr int kStageBytes = kABytes + kBBytes;
    static constexpr int kStages = 192 * 1024 / kStageBytes;
    static constexpr int kAcc = (int)kTmemCols / BN;      // accumulators
    static constexpr int kCols = BN / 2;                  // channels of a summing thread
    static constexpr bool kAnywhere = BN == 128;          // out's rows may start off 16 bytes
    static_assert(kStages >= kAcc, "no turn of a stage is missed");
    static_assert(kCols <= kScaleBlock && BN <= 256, "one scale a thread; a TMA box");
};

constexpr int kMaxStages = 6, kMaxAcc = 4, kUnitSlots = 4;
constexpr int kScaleGroup = 4, kScaleSlots = 6;  // blocks whose scales come together, groups under way
struct Shared {
    uint64_t full[kMaxStages], done[kMaxStages];  // a stage has landed; its MMAs are over
    uint64_t acc_empty[kMaxAcc];
    uint64_t unit_full[kUnitSlots], unit_empty[kUnitSlots];
    uint64_t scale_full[kScaleSlots], scale_empty[kScaleSlots];
    uint64_t drained;
    int4 unit[kUnitSlots];
    alignas(16) int source[kUnitSlots][128];   // rows of x of a unit's rows, -1 for none
    alignas(16) float x_scales[kScaleSlots][128][kScaleGroup];  // of a row in the blocks of a group
    alignas(16) float w_scales[kScaleSlots][2][kScaleGroup];           // of the channels' two halves
    float turn[kSumWarps][8][33];  // 8 channels of a summing warp's 32 rows on their way out
    uint32_t tmem;
    int abort;
    long long warp_sums[kTileGroups / 32];
    int tiles[kTileGroups + 1];
};
template <class S>
constexpr int kSmemBytes = 1024 + S::kStages * S::kStageBytes + (int)sizeof(Shared);

// By a whole warp, one lane of which issues: with the choice inside, the operands stay
// in uniform registers (four of these and the commit take 156 cycles, 240 in a branch).
__device__ __forceinline__ void mma_f8(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, bool accumulate) {
    asm volatile(
        "{\n.reg .pred p, one;\nelect.sync _|one, 0xffffffff;\nsetp.ne.u32 p, %4, 0;\n"
        "@one tcgen05.mma.cta_group::1.kind::f8f6f4 [%0], %1, %2, %3, p;\n}\n"
        ::"r"(d), "l"(a), "l"(b), "r"(idesc), "r"(accumulate ? 1u : 0u) : "memory");
}
__device__ __forceinline__ void commit_elected(uint64_t* bar) {
    asm volatile(
        "{\n.reg .pred one;\nelect.sync _|one, 0xffffffff;\n"
        "@one tcgen05.commit.cta_group::1.mbarrier::arrive::one.shared::cluster.b64 [%0];\n}\n"
        ::"r"(smem_u32(bar)) : "memory");
}

// 32 columns of this warp's 32 lanes, without the wait; then the wait, which the
// registers depend on.
__device__ __forceinline__ void tmem_start32(uint32_t at, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0, %1, %2, %3, %4, %5, %6, %7, %8, %9, %10, %11, %12, %13, %14, %15, %16, %17, %18, %19, %20, %21, %22, %23, %24, %25, %26, %27, %28, %29, %30, %31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]), "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]), "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]), "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(at) : "memory");
}
__device__ __forceinline__ void tmem_finish32(uint32_t (&r)[32]) {
    asm volatile("tcgen05.wait::ld.sync.aligned;"
                 : "+r"(r[0]), "+r"(r[1]), "+r"(r[2]), "+r"(r[3]), "+r"(r[4]), "+r"(r[5]), "+r"(r[6]), "+r"(r[7]), "+r"(r[8]), "+r"(r[9]), "+r"(r[10]), "+r"(r[11]), "+r"(r[12]), "+r"(r[13]), "+r"(r[14]), "+r"(r[15]), "+r"(r[16]), "+r"(r[17]), "+r"(r[18]), "+r"(r[19]), "+r"(r[20]), "+r"(r[21]), "+r"(r[22]), "+r"(r[23]), "+r"(r[24]), "+r"(r[25]), "+r"(r[26]), "+r"(r[27]), "+r"(r[28]), "+r"(r[29]), "+r"(r[30]), "+r"(r[31]) :: "memory");
}

// acc += v * s for 32 sums.
__device__ __forceinline__ void add_scaled32(float* acc, const uint32_t (&v)[32], float s) {
#pragma unroll
    for (int j = 0; j < 32; ++j) acc[j] = fmaf(__uint_as_float(v[j]), s, acc[j]);
}
// Four rows of x, one below the other in shared memory (row 0 for a row that reads
// nothing: its output is 0 or not stored).
__device__ __forceinline__ void load_rows(const CUtensorMap* map, uint64_t* bar, uint32_t dst, int k, int4 r) {
    asm volatile(
        "cp.async.bulk.tensor.2d.shared::cluster.global.tile::gather4.mbarrier::complete_tx::bytes "
        "[%0], [%1, {%3, %4, %5, %6, %7}], [%2];"
        ::"r"(dst), "l"(map), "r"(smem_u32(bar)), "r"(k), "r"(max(r.x, 0)), "r"(max(r.y, 0)), "r"(max(r.z, 0)),
          "r"(max(r.w, 0)) : "memory");
}

// 16 or 4 bytes to shared memory in the background (zeros where !on).
__device__ __forceinline__ void fetch16(uint32_t dst, const float* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(on ? 16 : 0) : "memory");
}
__device__ __forceinline__ void fetch4(uint32_t dst, const float* src, bool on) {
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(on ? 4 : 0) : "memory");
}

// A place in a ring of N and the parity of its turn.
template <int N>
struct Ring {
    uint32_t i = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++i == N) {
            i = 0;
            phase ^= 1;
        }
    }
};

// Whether the phase with this parity is over; does not wait.
__device__ __forceinline__ bool test_now(uint64_t* bar, uint32_t parity) {
    uint32_t done;
    asm volatile(
        "{\n.reg .pred p;\n"
        "mbarrier.test_wait.parity.shared::cta.b64 p, [%1], %2;\n"
        "selp.u32 %0, 1, 0, p;\n}\n"
        : "=r"(done) : "r"(smem_u32(bar)), "r"(parity) : "memory");
    return done != 0;
}
// A warp's wait.
template <class Shared>
__device__ __forceinline__ bool wait_warp(Shared* sh, uint64_t* bar, uint32_t parity) {
    if (__all_sync(kFull, mbar_try(smem_u32(bar), parity))) return true;
    return mbar_wait_warp(sh, bar, parity);
}

// Arrives on the barrier once the thread's copies so far have landed.
__device__ __forceinline__ void arrive_landed(uint64_t* bar) {
    asm volatile("cp.async.mbarrier.arrive.noinc.shared::cta.b64 [%0];" ::"r"(smem_u32(bar)) : "memory");
}

struct Unit {
    int e, begin;     // expert, its first position in expert-major order
    int channel;      // first channel
    int first, rows;  // rows of the expert in this tile
};
template <class S>
__device__ __forceinline__ Unit unpack_unit(int4 q) {
    Unit t;
    t.e = q.x & (kMaxE - 1);
    t.begin = q.y;
    t.channel = q.z * S::kChannels;
    t.first = q.w;
    t.rows = q.x >> 10;
    return t;
}

// Whether each row of out starts on 16 bytes (out does).
__host__ __device__ __forceinline__ bool rows_on_16(const MatmulArgs& a) {
    return (size_t)a.Nc * (a.out_bf16 ? 2 : 4) % 16 == 0;
}

// Eight channels of a row of out that starts on 16 bytes; cols: how many there are from here.
__device__ __forceinline__ void store8(const MatmulArgs& a, uint8_t* to, int cols, const float (&f)[8]) {
    if (a.out_bf16) {
        if (cols > 0)
            *reinterpret_cast<uint4*>(to) = make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7]));
    } else {
        if (cols > 0) *reinterpret_cast<float4*>(to) = make_float4(f[0], f[1], f[2], f[3]);
        if (cols > 4) *reinterpret_cast<float4*>(to + 16) = make_float4(f[4], f[5], f[6], f[7]);
    }
}
// 32 bytes that start on a boundary of 32: a whole sector of memory.
__device__ __forceinline__ void store32(uint8_t* to, const uint32_t (&r)[8]) {
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};"
                 ::"l"(to), "r"(r[0]), "r"(r[1]), "r"(r[2]), "r"(r[3]), "r"(r[4]), "r"(r[5]), "r"(r[6]), "r"(r[7]) : "memory");
}

template <class S>
__global__ void __launch_bounds__(kThreads, 1)
matmul_fp8_kernel(MatmulArgs a, const __grid_constant__ CUtensorMap w_map, const __grid_constant__ CUtensorMap x_map) {
    constexpr int kStages = S::kStages, kAcc = S::kAcc;
    extern __shared__ uint8_t s_raw[];
    uint8_t* s_stage = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(s_raw) + 1023) & ~(uintptr_t)1023);
    Shared* sh = reinterpret_cast<Shared*>(s_stage + kStages * S::kStageBytes);
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;

    pdl_prologue();
    if (tid == 0) {
        sh->abort = 0;
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], 2);
            mbar_init(&sh->done[i], 1);
        }
        for (int i = 0; i < kAcc; ++i) mbar_init(&sh->acc_empty[i], kSumWarps);
        for (int i = 0; i < kUnitSlots; ++i) {
            mbar_init(&sh->unit_full[i], 1);
            mbar_init(&sh->unit_empty[i], kSumWarps + 2);  // all that look rows up
        }
        for (int i = 0; i < kScaleSlots; ++i) {
            mbar_init(&sh->scale_full[i], 32);
            mbar_init(&sh->scale_empty[i], kSumWarps);
        }
        mbar_init(&sh->drained, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        if (a.status != nullptr && blockIdx.x == 0) *a.status = 0;
    }
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.alloc.cta_group::1.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(&sh->tmem)), "r"(kTmemCols) : "memory");
    }
    tmem_fence_before();
    tile_prefix(a, S::TN, sh->tiles, sh->warp_sums);
    tmem_fence_after();
    const uint32_t tmem = sh->tmem;
    const uint32_t units = unit_count<S>(a, sh->tiles, blockIdx.x, gridDim.x);
    const int kblocks = scale_blocks(a.Kd);

    if (warp >= kSumWarps) {
        asm volatile("setmaxnreg.dec.sync.aligned.u32 56;");
        if (warp < kMmaWarp) {
            // ---- operands.  The first warp fetches the weights' boxes; the second rows of x
            // that lie together, in boxes of 32.  Rows anywhere (row_src) are fetched 4 a copy,
            // half of them by each warp.  Such copies take some 55 cycles each wherever they
            // are issued, 128 rows 0.93 us: 1024 rows an expert 1.64 ms, rows that lie
            // together 0.77.  (16-byte copies by threads and the fence that orders them
            // before the MMAs: 1.43 ms, but 0.85 us a step however few the rows, 57 us for
            // one token's 8 rows where this takes 45.) ----
            const bool gather = a.row_src != nullptr, weights = warp == kTmaWarp;
            uint32_t c = 0;
            bool ok = true;
            for (uint32_t u = 0; ok && u < units; ++u) {
                const uint32_t slot = u % kUnitSlots;
                ok = mbar_wait_warp(sh, &sh->unit_full[slot], u / kUnitSlots & 1);
                if (!ok) break;
                const Unit t = unpack_unit<S>(sh->unit[slot]);
                const int w_row = t.e * a.Nc + t.channel, x_row = sh->source[slot][0];
                // copies of this warp: of 4 rows each, or of 32
                const int all = gather ? (t.rows + 3) / 4 : (t.rows + 31) / 32;
                const int first = !gather || weights ? 0 : all / 2;
                const int last = weights ? (gather ? all / 2 : 0) : all;
                const uint32_t bytes = (last - first) * (gather ? 4 : 32) * kBK + (weights ? S::kBBytes : 0);
                for (int kb = 0; kb < kblocks; ++kb, ++c) {
                    const uint32_t s = c % kStages;
                    ok = mbar_wait_warp(sh, &sh->done[s], (c / kStages & 1) ^ 1);
                    if (!ok) break;
                    if (elect_one()) {
                        uint8_t* stage = s_stage + s * S::kStageBytes;
                        mbar_expect_tx(&sh->full[s], bytes);
                        if (weights) tma_load(&w_map, &sh->full[s], stage + S::kABytes, kb * kBK, w_row);
                        if (gather) {
#pragma unroll 4
                            for (int i = first; i < last; ++i)
                                load_rows(&x_map, &sh->full[s], smem_u32(stage + i * 4 * kBK), kb * kBK,
                                          *reinterpret_cast<const int4*>(&sh->source[slot][i * 4]));
                        } else {
                            for (int i = first; i < last; ++i)
                                tma_load(&x_map, &sh->full[s], stage + i * 32 * kBK, kb * kBK, x_row + i * 32);
                        }
                    }
                    __syncwarp();
                }
                if (lane == 0) mbar_arrive(&sh->unit_empty[slot]);
            }
            // the last MMAs' arrivals on each stage land before the CTA ends
            for (uint32_t i = c < kStages ? 0 : c - kStages; ok && i < c; ++i)
                ok = mbar_wait_warp(sh, &sh->done[i % kStages], i / kStages & 1);
            if (!ok && lane == 0) drain_copies<kStages>(sh->full, c);
        } else if (warp == kMmaWarp) {
            // ---- MMA: the whole warp, an elected lane of which issues ----
            const uint64_t desc0 = operand_desc(smem_u32(s_stage));
            // float32 accumulators, E4M3 operands, both K-major
            constexpr uint32_t idesc = 1u << 4 | (uint32_t)(S::BN >> 3) << 17 | (uint32_t)(S::TN >> 4) << 24;
            Ring<kStages> st;
            Ring<kAcc> acc;
            bool ok = true, any = false;
            for (uint32_t u = 0; ok && u < units; ++u) {
#pragma unroll 1
                for (int kb = 0; kb < kblocks; ++kb) {
                    ok = wait_warp(sh, &sh->full[st.i], st.phase) && wait_warp(sh, &sh->acc_empty[acc.i], acc.phase ^ 1);
                    if (!ok) break;
                    tmem_fence_after();
                    const uint64_t da = desc0 + (uint64_t)(st.i * (S::kStageBytes >> 4)), db = da + (S::kABytes >> 4);
                    const uint32_t d = tmem + acc.i * S::BN;
#pragma unroll
                    for (int k = 0; k < 4; ++k) mma_f8(d, da + k * 2, db + k * 2, idesc, k > 0);
                    commit_elected(&sh->done[st.i]);
                    any = true;
                    st.next();
                    acc.next();
                }
            }
            if (!ok && any) {  // the MMAs in flight end before their operands' memory is given up
                commit_elected(&sh->drained);
                const long long start = clock64();
                while (!mbar_try(smem_u32(&sh->drained), 0))
                    if (clock64() - start > kWaitCycles) break;
                __syncwarp();
            }
        } else {
            // ---- units, their rows and their scales, a few ahead ----
            Steps<S> steps(a, blockIdx.x, gridDim.x);
            // fours of a row's scales start on 16 bytes
            const bool whole = kblocks % 4 == 0 && reinterpret_cast<uintptr_t>(a.x_scales) % 16 == 0;
            const int channel_blocks = scale_blocks(a.Nc);
            uint32_t g = 0;
            bool ok = true;
            for (uint32_t u = 0; ok && u < units; ++u) {
                const uint32_t slot = u % kUnitSlots;
                const int4 packed = steps.next(a, sh->tiles);
                const Unit t = unpack_unit<S>(packed);
                ok = mbar_wait_warp(sh, &sh->unit_empty[slot], (u / kUnitSlots & 1) ^ 1);
                if (!ok) break;
                for (int r = lane; r < 128; r += 32)
                    sh->source[slot][r] = r < t.rows && a.x_rows > 0 ? source_row(a, t.e, t.begin, t.first + r) : -1;
                __syncwarp();
                if (lane == 0) {
                    sh->unit[slot] = packed;
                    mbar_arrive(&sh->unit_full[slot]);
                }
                __syncwarp();
                // lanes 0 .. 7: a half of the channels and one of the group's blocks each
                const int block = min((t.channel + (lane >> 2 & 1) * S::kCols) / kScaleBlock, channel_blocks - 1);
                const float* ws = a.w_scales + ((size_t)t.e * channel_blocks + block) * kblocks + (lane & 3);
                for (int kb = 0; kb < kblocks; kb += kScaleGroup, ++g) {
                    const uint32_t sg = g % kScaleSlots;
                    ok = mbar_wait_warp(sh, &sh->scale_empty[sg], (g / kScaleSlots & 1) ^ 1);
                    if (!ok) break;
#pragma unroll 1
                    for (int r = lane; r < t.rows; r += 32) {
                        const int src = sh->source[slot][r];
                        // a row that reads nothing has no scales either: zeros, by copies of no bytes
                        // from where there is memory
                        const float* xs = src >= 0 ? a.x_scales + (size_t)src * kblocks + kb : reinterpret_cast<const float*>(a.w);
                        const uint32_t dst = smem_u32(sh->x_scales[sg][r]);
                        if (whole) {
                            fetch16(dst, xs, src >= 0);
                        } else {
                            for (int j = 0; j < kScaleGroup && kb + j < kblocks; ++j) fetch4(dst + j * 4, src >= 0 ? xs + j : xs, src >= 0);
                        }
                    }
                    if (lane < 8 && kb + (lane & 3) < kblocks)
                        fetch4(smem_u32(&sh->w_scales[sg][lane >> 2][lane & 3]), ws + kb, true);
                    arrive_landed(&sh->scale_full[sg]);
                }
            }
            asm volatile("cp.async.wait_all;" ::: "memory");
        }
    } else {
        // ---- accumulators -> sums -> out; a row a thread, half of the channels ----
        asm volatile("setmaxnreg.inc.sync.aligned.u32 224;");
        constexpr int kCols = S::kCols, kChunks = kCols / 32;
        const int quarter = warp & 3, half = warp >> 2;
        const uint32_t from = tmem + ((uint32_t)quarter << 21) + half * kCols;
        const int size = a.out_bf16 ? 2 : 4;
        // rows of out start on 32 bytes, or on 16
        const bool sectors = (size_t)a.Nc * size % 32 == 0 && reinterpret_cast<uintptr_t>(a.out) % 32 == 0;
        const bool vectors = rows_on_16(a);
        const int row = quarter * 32 + lane;
        uint32_t c = 0, g = 0;  // blocks and groups of scales so far
        Ring<kStages> st;
        bool ready = false, soon = false;  // the next block is there already
        bool ok = true;
        for (uint32_t u = 0; ok && u < units; ++u) {
            const uint32_t slot = u % kUnitSlots;
            ok = mbar_wait_warp(sh, &sh->unit_full[slot], u / kUnitSlots & 1);
            if (!ok) break;
            bool busy;  // the warp has rows and channels
            {
                const Unit t = unpack_unit<S>(sh->unit[slot]);
                busy = quarter * 32 < t.rows && t.channel + half * kCols < a.Nc;
            }
            float acc[kCols];
#pragma unroll
            for (int j = 0; j < kCols; ++j) acc[j] = 0.0f;
#pragma unroll 1
            for (int kb = 0; ok && kb < kblocks; kb += kScaleGroup, ++g) {
                const uint32_t sg = g % kScaleSlots;
                ok = wait_warp(sh, &sh->scale_full[sg], g / kScaleSlots & 1);
                if (!ok) break;
                float s[kScaleGroup];
                {
                    const float4 x = *reinterpret_cast<const float4*>(sh->x_scales[sg][row]);
                    const float4 w = *reinterpret_cast<const float4*>(sh->w_scales[sg][half]);
                    s[0] = x.x * w.x; s[1] = x.y * w.y; s[2] = x.z * w.z; s[3] = x.w * w.w;
                }
                __syncwarp();
                if (lane == 0) mbar_arrive(&sh->scale_empty[sg]);
#pragma unroll
                for (int j = 0; j < kScaleGroup; ++j) {
                    if (kb + j >= kblocks) break;
                    const uint32_t b = c % kAcc;
                    if (!ready) ok = wait_warp(sh, &sh->done[st.i], st.phase);
                    if (!ok) break;
                    tmem_fence_after();
                    if (busy) {
                        uint32_t v[2][32];
                        tmem_start32(from + b * S::BN, v[0]);
#pragma unroll
                        for (int i = 0; i < kChunks; ++i) {
                            tmem_finish32(v[i & 1]);
                            if (i + 1 < kChunks) {
                                tmem_start32(from + b * S::BN + (i + 1) * 32, v[(i + 1) & 1]);
                            } else {  // all of it is in registers: the next block may come
                                tmem_fence_before();
                                if (lane == 0) mbar_arrive(&sh->acc_empty[b]);
                                st.next();
                                soon = test_now(&sh->done[st.i], st.phase);  // answered behind the last sums
                            }
                            add_scaled32(acc + i * 32, v[i & 1], s[j]);
                        }
                    } else {
                        if (lane == 0) mbar_arrive(&sh->acc_empty[b]);
                        st.next();
                        soon = false;
                    }
                    ++c;
                    ready = __all_sync(kFull, soon);
                    if (!ok) break;
                }
            }
            if (!ok) break;
            const Unit t = unpack_unit<S>(sh->unit[slot]);
            const bool none = sh->source[slot][row] < 0;  // a row of zeros, whatever lay in its place
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->unit_empty[slot]);
            const int ch0 = t.channel + half * kCols;
            if constexpr (S::kAnywhere) {
                if (!vectors) {
                    // 8 channels at a time through shared memory, so that a store takes 8
                    // neighbours of four rows (6 experts of 500 x 1008, 64 rows each: 14 us,
                    // 22 by each thread's own row)
                    const int rows = min(t.rows - quarter * 32, 32), c = lane & 7;
                    uint8_t* to = static_cast<uint8_t*>(a.out) +
                                  ((first_row(a, t.e, t.begin) + t.first + quarter * 32) * (size_t)a.Nc + ch0 + c) * size;
#pragma unroll
                    for (int j = 0; j < kCols; j += 8) {
                        __syncwarp();
#pragma unroll
                        for (int i = 0; i < 8; ++i) sh->turn[warp][i][lane] = none ? 0.0f : acc[j + i];
                        __syncwarp();
                        if (ch0 + j + c < a.Nc)
                            for (int r = lane >> 3; r < rows; r += 4) {
                                const float y = sh->turn[warp][c][r];
                                uint8_t* at = to + ((size_t)r * a.Nc + j) * size;
                                if (a.out_bf16) *reinterpret_cast<__nv_bfloat16*>(at) = __float2bfloat16_rn(y);
                                else *reinterpret_cast<float*>(at) = y;
                            }
                    }
                    continue;
                }
            }
            if (row >= t.rows || !busy) continue;
            uint8_t* to = static_cast<uint8_t*>(a.out) +
                          ((first_row(a, t.e, t.begin) + t.first + row) * (size_t)a.Nc + ch0) * size;
            const int cols = a.Nc - ch0;
            if (sectors) {
#pragma unroll
                for (int j = 0; j < kCols; j += 16) {
                    float f[16];
#pragma unroll
                    for (int i = 0; i < 16; ++i) f[i] = none ? 0.0f : acc[j + i];
                    uint32_t r[8];
                    if (a.out_bf16) {
#pragma unroll
                        for (int i = 0; i < 8; ++i) r[i] = pack_bf16(f[2 * i], f[2 * i + 1]);
                        if (j < cols) store32(to + j * 2, r);
                    } else {
#pragma unroll
                        for (int h = 0; h < 16; h += 8) {
#pragma unroll
                            for (int i = 0; i < 8; ++i) r[i] = __float_as_uint(f[h + i]);
                            if (j + h < cols) store32(to + (j + h) * 4, r);
                        }
                    }
                }
            } else {
#pragma unroll
                for (int j = 0; j < kCols; j += 8) {
                    float f[8];
#pragma unroll
                    for (int i = 0; i < 8; ++i) f[i] = none ? 0.0f : acc[j + i];
                    store8(a, to + j * size, cols - j, f);
                }
            }
        }
    }

    __syncwarp();
    tmem_fence_before();
    __syncthreads();
    tmem_fence_after();
    if (warp == kMmaWarp) {
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::1.sync.aligned;" ::: "memory");
        asm volatile("tcgen05.dealloc.cta_group::1.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(kTmemCols) : "memory");
    }
    if (tid == 0 && sh->abort != 0 && a.status != nullptr) *a.status = 1;
}

// The persistent kernel's attributes on the current device, set once for each.
template <class S>
cudaError_t prepare_kernel() {
    static std::atomic<bool> done[64];
    int dev = 0;
    cudaError_t err = cudaGetDevice(&dev);
    if (err != cudaSuccess) return err;
    if (dev >= 0 && dev < 64 && done[dev].load(std::memory_order_relaxed)) return cudaSuccess;
    cudaFuncAttributes attr;
    err = cudaFuncGetAttributes(&attr, matmul_fp8_kernel<S>);
    if (err != cudaSuccess) return err;
    // the summing warps' registers come out of the launch's: with fewer they would wait forever
    if (attr.numRegs < kLaunchRegs) return cudaErrorInvalidConfiguration;
    err = cudaFuncSetAttribute(matmul_fp8_kernel<S>, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmemBytes<S>);
    if (err == cudaSuccess && dev >= 0 && dev < 64) done[dev].store(true, std::memory_order_relaxed);
    return err;
}

// Rows of bytes, copied in boxes of 128 columns.
bool rows_map(EncodeTiled encode, CUtensorMap* map, const void* base, uint64_t cols, uint64_t rows, uint32_t box_rows) {
    const cuuint64_t dims[2] = {cols, rows}, strides[1] = {cols};
    const cuuint32_t box[2] = {kBK, box_rows}, steps[2] = {1, 1};
    return encode(map, CU_TENSOR_MAP_DATA_TYPE_UINT8, 2, const_cast<void*>(base), dims, strides, box, steps,
                  CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                  CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

template <class S>
cudaError_t launch_shape(const MatmulArgs& a, cudaStream_t s) {
    static_assert(kSmemBytes<S> <= 227 * 1024, "a CTA's shared memory");
    const EncodeTiled encode = encode_tiled();
    if (encode == nullptr) return cudaErrorNotSupported;
    CUtensorMap w_map, x_map;
    // without rows of x nothing of it counts: a row of the weights stands in for them
    const void* x = a.x_rows > 0 ? a.x : a.w;
    if (!rows_map(encode, &w_map, a.w, a.Kd, (uint64_t)a.E * a.Nc, S::BN) ||
        !rows_map(encode, &x_map, x, a.Kd, std::max(a.x_rows, 1), a.row_src != nullptr ? 1 : 32))
        return cudaErrorInvalidValue;
    const cudaError_t err = prepare_kernel<S>();
    if (err != cudaSuccess) return err;
    return launch(matmul_fp8_kernel<S>, dim3(sm_count()), dim3(kThreads), kSmemBytes<S>, s, a, w_map, x_map);
}

}  // namespace

cudaError_t launch_expert_matmul_fp8(const MatmulArgs& a, cudaStream_t s) {
    if (a.rows == 0)
        return a.status != nullptr ? cudaMemsetAsync(a.status, 0, sizeof(int32_t), s) : cudaSuccess;
    // Wide tiles take half the steps at 900 cycles instead of 620; narrow ones have twice
    // the tiles and more weights in flight.  Us with 256 channels and with 128, 32 experts of
    // 4096 x 7168: 64 rows each 160, 154; 128 rows 188, 213; 1024 rows 772, 1085; one
    // expert of 4096 x 4096, 512 rows (64 wide tiles) 27, 20.  Rows fetched by 4 cost a
    // step more: 32 rows each 164, 195.  A capacity counts half, as nothing here knows how
    // many rows it holds.  Other sizes, with and without row_src: the rule's shape is within
    // 8 % of the better one at 8 to 512 rows each of 32 experts of 7168 x 2048 and x 512 and of
    // 128 of 2880 x 1440 (most at 96 rows of the last, wide 117 and narrow 111), and where a
    // capacity of 64 to 1024 holds 1 to 64 rows (4096 x 7168, one row each: wide 171 and
    // narrow 165).  Rows of out off 16 bytes are
    // narrow tiles' alone: the way through shared memory costs the wide ones registers that
    // their steps need (prefill 0.86 ms instead of 0.77).  32 experts of 4100 x 7168, 1024 rows
    // each: 1.23 ms, wide tiles with each thread's own stores 1.79.
    const double mean = a.layout == 0 ? (double)a.rows / a.E : 0.5 * a.cap;
    const double tiles = a.E * std::ceil(mean / 128) * ((a.Nc + 255) / 256);
    const bool wide = tiles >= sm_count() && mean >= (a.row_src != nullptr ? 16 : 96) && rows_on_16(a);
    const cudaError_t err = wide ? launch_shape<Shape<256>>(a, s) : launch_shape<Shape<128>>(a, s);
    note_launch();
    return err;
}

}  // namespace ep
