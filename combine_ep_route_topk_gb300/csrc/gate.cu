// Gate of an expert layer for sm_103a: scores, balance bias, groups, top-K and
// weights (ep_gate_topk), and the gradient of the weights with respect to the
// logits (ep_gate_topk_backward).
//
//   s_e   = 1 / (1 + exp(-l_e))                  (sigmoid), or
//           exp(l_e - m) / sum_a exp(l_a - m)    (softmax over the experts whose
//           logit is available: neither -inf nor NaN)
//   key_e = s_e + bias_e, or l_e without a bias (the scores grow with l)
//   group score = largest key of the group, or the sum of its two largest
//           s_e + bias_e; only experts of the best topk_groups groups remain
//   picks = the K largest keys, ties to the lower id
//   w_k   = scale * s_k [/ sum of the picks' s]
//
// One warp per token.  Lane i holds the VPL consecutive experts i*VPL ..
// i*VPL + VPL-1, so that a lower lane always means lower ids.  It sorts its
// keys (values alone, by a network of min and max); a round of the selection is
// then one redux.sync max over the lanes' heads and a ballot, the lowest lane
// that holds the maximum wins, and the winner moves its list up by one.  Which
// expert a pick is follows once, after the rounds, from its value, its lane and
// how many equal values that lane gave before it.  Scores are recomputed, in
// full accuracy, for the picks alone; the choice uses the hardware's exp2 and
// reciprocal (an absolute error below 3e-7 in a score of at most 1).
//
// What bounds it: instructions (523 a token of 256 experts with bias and groups;
// 75 % of the issue slots): 32768 tokens of float32, 33.6 MB, take 17.4 us where
// the bytes alone would take 5; one token 2.5 us.  Rows of finite numbers skip
// the tests for others and picks without equals in their lane the count of them
// (18.8 us with neither, and 15.3 against 12.6 for a softmax in one group).  That
// holds where the experts fill the lanes: 32, 64, 128, 160, 256, 384, 512 and 1024.
// Otherwise the padding past E, held as NaN, sends every row through the tests (a
// softmax of 32768 tokens: 96 experts 11.7 us, 128 10.5; 192 14.8, 256 12.6).  The
// gradient (32768 x 256, 8 picks a token) takes 11.2 us for its 33.5 MB of stores,
// 7.3 when they stay in L2, and 11.6 where every expert gets one (softmax, not
// renormalised).
#include <cuda_bf16.h>

#include <cfloat>

#include "ep_kernels.cuh"

namespace ep {
namespace {

constexpr unsigned kFull = 0xffffffffu;
constexpr int kGateWarps = 8;
constexpr int kGradManyTokens = 4096;  // from here four tokens a warp

// False for NaN and -inf.
__device__ __forceinline__ bool available(float v) { return v > -INFINITY; }

// A logit as the formulas use it: +inf counts as the largest finite number, so
// that no score is inf / inf.
__device__ __forceinline__ float clamp_logit(float v) { return fminf(v, FLT_MAX); }


__device__ __forceinline__ float load_one(const float* p) { return __ldg(p); }
__device__ __forceinline__ float load_one(const __nv_bfloat16* p) {
    return __uint_as_float((uint32_t)__ldg(reinterpret_cast<const unsigned short*>(p)) << 16);
}

__device__ __forceinline__ void load_four(const float* p, float* v) {
    const float4 q = __ldg(reinterpret_cast<const float4*>(p));
    v[0] = q.x; v[1] = q.y; v[2] = q.z; v[3] = q.w;
}
__device__ __forceinline__ void load_four(const __nv_bfloat16* p, float* v) {
    const uint2 q = __ldg(reinterpret_cast<const uint2*>(p));
    v[0] = __uint_as_float(q.x << 16); v[1] = __uint_as_float(q.x & 0xffff0000u);
    v[2] = __uint_as_float(q.y << 16); v[3] = __uint_as_float(q.y & 0xffff0000u);
}

// The hardware's exp2 and reciprocal.
constexpr float kLog2e = 1.4426950408889634f;
__device__ __forceinline__ float exp2_fast(float x) {
    float y;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
__device__ __forceinline__ float rcp_fast(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}

// Accurate to the last places, unlike the scores of the choice.
__device__ __forceinline__ float sigmoid(float l) { return rcp_fast(1.0f + expf(-l)); }

// Sum and maximum over aligned groups of G lanes.
template <int G>
__device__ __forceinline__ float lanes_sum(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v += __shfl_xor_sync(kFull, v, off);
    return v;
}
template <int G>
__device__ __forceinline__ float lanes_max(float v) {
#pragma unroll
    for (int off = G / 2; off > 0; off >>= 1) v = fmaxf(v, __shfl_xor_sync(kFull, v, off));
    return v;
}

// The share s_k / sum_j s_j of the lane's pick (logit l) among the picks of its
// token, which G lanes hold; 0 on lanes without one.  The scores are taken
// relative to the largest pick's, exp(l - c) with c = max l for the softmax and
// min(0, max l) for the sigmoid, so that no sum underflows however far below the
// others' the picks' scores lie.  Quotients by the hardware's reciprocal (1 ulp).
template <int G>
__device__ __forceinline__ float pick_share(float l, bool picked, int score) {
    float s = 0.0f;
    if (score == kScoreSigmoid) {
        // l > 0 (then c = 0): 1 / (1 + exp(-l)); else exp(l - c) / (1 + exp(l))
        const float e = expf(-fabsf(l));
        float num = l > 0.0f ? 1.0f : e;
        if (__any_sync(kFull, picked && l < 0.0f)) {  // some token's picks may all be negative
            const float c = lanes_max<G>(picked ? l : -INFINITY);
            if (c < 0.0f) num = expf(l - c);
        }
        if (picked) s = num * rcp_fast(1.0f + e);
    } else {
        const float c = lanes_max<G>(picked ? l : -INFINITY);
        if (picked) s = expf(l - c);
    }
    const float sum = lanes_sum<G>(s);  // at least 1/2 where anything is picked
    return picked ? s * rcp_fast(sum) : 0.0f;
}

// The two best of this lane's and the other lane's.
__device__ __forceinline__ void merge_two(float& best, float& second, int off) {
    const float o1 = __shfl_xor_sync(kFull, best, off);
    const float o2 = __shfl_xor_sync(kFull, second, off);
    second = fmaxf(fminf(best, o1), fmaxf(second, o2));
    best = fmaxf(best, o1);
}

// The lane's VPL logits (NaN past E), four at a time where rows allow it.
template <int VPL, typename T>
__device__ __forceinline__ void load_row(const T* row, int E, bool vec, int lane, float (&v)[VPL]) {
    const int e0 = lane * VPL;
    if constexpr (VPL % 4 == 0) {
        if (vec) {
#pragma unroll
            for (int j = 0; j < VPL; j += 4) {
                if (e0 + j < E) {
                    load_four(row + e0 + j, &v[j]);
                } else {
#pragma unroll
                    for (int i = 0; i < 4; ++i) v[j + i] = __int_as_float(0x7fffffff);
                }
            }
            return;
        }
    }
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        v[j] = (e0 + j < E) ? load_one(row + e0 + j) : __int_as_float(0x7fffffff);
}

// Sorts v descending: Batcher's odd-even merge sort (1968), one step a call.
template <int N, int P = 1, int K = 1>
__device__ __forceinline__ void sort_descending(float (&v)[N]) {
    if constexpr (P < N) {
#pragma unroll
        for (int x = K % P; x + K < N; ++x)
            if ((x - K % P) % (2 * K) < K && x / (2 * P) == (x + K) / (2 * P)) {
                const float hi = fmaxf(v[x], v[x + K]);
                v[x + K] = fminf(v[x], v[x + K]);
                v[x] = hi;
            }
        if constexpr (K > 1) sort_descending<N, P, K / 2>(v);
        else sort_descending<N, P * 2, P * 2>(v);
    }
}

// The L largest of v, descending: pieces of at most L are sorted, and joined by
// Batcher's bitonic merge, of which only the upper half is kept.
template <int L, int FROM = 0, int N>
__device__ __forceinline__ void largest(const float (&v)[N], float (&list)[L]) {
    if constexpr (FROM < N) {
        constexpr int R = N - FROM < L ? N - FROM : L;
        float piece[R];
#pragma unroll
        for (int i = 0; i < R; ++i) piece[i] = v[FROM + i];
        sort_descending(piece);
        if constexpr (FROM == 0) {
#pragma unroll
            for (int i = 0; i < L; ++i) list[i] = piece[i];
        } else {
#pragma unroll
            for (int i = 0; i < R; ++i) list[L - 1 - i] = fmaxf(list[L - 1 - i], piece[i]);
#pragma unroll
            for (int d = L / 2; d > 0; d /= 2)
#pragma unroll
                for (int i = 0; i < L; ++i)
                    if ((i & d) == 0) {
                        const float hi = fmaxf(list[i], list[i + d]);
                        list[i + d] = fminf(list[i], list[i + d]);
                        list[i] = hi;
                    }
        }
        largest<L, FROM + R>(v, list);
    }
}

// Maximum over the warp.
__device__ __forceinline__ float redux_max(float v) {
    float m;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(m) : "f"(v));
    return m;
}

__device__ __forceinline__ void two_best(float x, float& a, float& b) {
    b = fmaxf(b, fminf(a, x));
    a = fmaxf(a, x);
}

// For groups of L whole lanes: the lanes' two largest keys are merged, scored,
// and the number of groups that come before the lane's returned.  (Lanes past E
// hold groups of nothing, which come last.)
template <int L, typename F>
__device__ __forceinline__ int groups_before(float best, float second, int lane, F group_score) {
#pragma unroll
    for (int off = 1; off < L; off <<= 1) merge_two(best, second, off);
    const float score = group_score(best, second);
    int before = 0;
#pragma unroll
    for (int x = L; x < 32; x += L) {
        const float other = __shfl_xor_sync(kFull, score, x);
        before += (lane ^ x) < lane ? other >= score : other > score;
    }
    return before;
}

// KT > 0: K == KT, or for more than 8 experts a lane K <= KT, which lets a lane
// keep its KT largest keys alone (8192 tokens of 1024 experts 27.3 -> 22.1 us).
template <int VPL, typename T, int KT>
__global__ void __launch_bounds__(kGateWarps * 32)
gate_kernel(GateArgs a) {
    extern __shared__ float s_choice[];  // [warps][E], only for groups that cross lanes unevenly
    __shared__ float2 s_pick[kGateWarps][32];  // a pick's key and the lane that gave it
    pdl_prologue();
    const int lane = threadIdx.x & 31;
    const int warp = threadIdx.x >> 5;
    const uint32_t t = blockIdx.x * kGateWarps + warp;  // unsigned: past N near 2^31 too
    if (t >= (uint32_t)a.N) return;  // warp-uniform
    const int E = a.E, K = KT > 0 && VPL <= 8 ? KT : a.K;
    const T* row = static_cast<const T*>(a.logits) + (size_t)t * E;
    const int e0 = lane * VPL;
    const bool groups_sum = a.groups > 1 && a.group_top == 2;
    const bool sigmoids = a.score == kScoreSigmoid;
    const unsigned lower = (1u << lane) - 1;  // the lanes below

    float v[VPL], bias[VPL];
    load_row<VPL>(row, E, a.vec != 0, lane, v);
    if (a.bias != nullptr) {
        load_row<VPL>(a.bias, E, a.bias_vec != 0, lane, bias);
    }
    // Whether every logit and bias of the row is finite: 0 x is NaN otherwise (on
    // another pipe than the comparisons that are spared then).  False for every row
    // that does not fill the lanes, whose padding is NaN.
    float zero = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        zero = fmaf(v[j], 0.0f, zero);
        if (a.bias != nullptr) zero = fmaf(bias[j], 0.0f, zero);
    }
    const bool finite = __all_sync(kFull, zero == 0.0f);
    if (a.bias != nullptr && !finite) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) bias[j] = fmaxf(bias[j], -INFINITY);  // NaN: not available
    }

    // softmax: the largest available logit, and the sum where a score is needed
    float m = 0.0f, total = 1.0f;
    if (!sigmoids) {
        m = -INFINITY;
        if (finite) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) m = fmaxf(m, v[j]);
        } else {
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (available(v[j])) m = fmaxf(m, clamp_logit(v[j]));
        }
        m = redux_max(m);
        if (a.bias != nullptr || groups_sum || !a.renorm) {
            float sum = 0.0f;
#pragma unroll
            for (int j = 0; j < VPL; ++j)
                if (available(v[j])) sum += expf(clamp_logit(v[j]) - m);
            total = lanes_sum<32>(sum);
        }
    }

    // keys (-inf: not available)
    const float inv_total = rcp_fast(total);
    float key[VPL];
    if (a.bias == nullptr) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = v[j];
        if (!finite) {
#pragma unroll
            for (int j = 0; j < VPL; ++j) key[j] = clamp_logit(v[j]);
        }
    } else if (sigmoids) {
#pragma unroll
        for (int j = 0; j < VPL; ++j)  // a sigmoid of +inf is 1 without a clamp
            key[j] = rcp_fast(1.0f + exp2_fast(v[j] * -kLog2e)) + bias[j];
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            key[j] = exp2_fast((clamp_logit(v[j]) - m) * kLog2e) * inv_total + bias[j];
    }
    if (!finite) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) key[j] = available(v[j]) ? key[j] : -INFINITY;
    }
    // a group's score from its two largest keys
    const auto group_score = [&](float best, float second) {
        if (!groups_sum) return best;
        if (a.bias == nullptr) {  // the keys are logits
            best = !available(best) ? best
                   : sigmoids ? rcp_fast(1.0f + exp2_fast(best * -kLog2e))
                              : exp2_fast((best - m) * kLog2e) * inv_total;
            second = !available(second) ? second
                     : sigmoids ? rcp_fast(1.0f + exp2_fast(second * -kLog2e))
                                : exp2_fast((second - m) * kLog2e) * inv_total;
        }
        return available(second) ? best + second : best;
    };
    if (a.groups > 1 && a.lanes_per_group == 0) {
        // groups that share lanes: their keys through shared memory, L lanes a group
        const int per = E / a.groups, L = a.share_lanes;
        float* choice = s_choice + (size_t)warp * E;
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < E) choice[e0 + j] = key[j];
        __syncwarp();
        float best = -INFINITY, second = -INFINITY;
        const int g = lane / L;
        if (g < a.groups)
            for (int n = lane % L; n < per; n += L) two_best(choice[g * per + n], best, second);
        for (int off = 1; off < L; off <<= 1) merge_two(best, second, off);
        best = g < a.groups ? group_score(best, second) : -INFINITY;
        int before = 0;
        for (int o = 0; o < a.groups; ++o) {
            const float other = __shfl_sync(kFull, best, o * L);
            before += o < g ? other >= best : other > best;
        }
        const unsigned kept = __ballot_sync(kFull, g < a.groups && before < a.topk_groups);
        int group = e0 / per, next = (group + 1) * per - e0;  // the first of the lane's that is in the next group
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            while (j >= next) {
                ++group;
                next += per;
            }
            if (e0 + j < E && !(kept >> (group * L) & 1u)) key[j] = -INFINITY;
        }
    }

    // No more than KT of a lane are ever picked.
    constexpr int kBound = KT == 0 ? VPL : KT <= 4 ? 4 : 8;
    constexpr int L = kBound < VPL ? kBound : VPL;
    float list[L];
    largest<L>(key, list);

    if (a.groups > 1 && a.lanes_per_group > 0) {
        // whole lanes of one group next to each other, a power of two of them
        const float second = L > 1 ? list[L > 1 ? 1 : 0] : -INFINITY;
        int before = 0;
        switch (a.lanes_per_group) {
            case 1: before = groups_before<1>(list[0], second, lane, group_score); break;
            case 2: before = groups_before<2>(list[0], second, lane, group_score); break;
            case 4: before = groups_before<4>(list[0], second, lane, group_score); break;
            case 8: before = groups_before<8>(list[0], second, lane, group_score); break;
            default: before = groups_before<16>(list[0], second, lane, group_score); break;
        }
        if (before >= a.topk_groups) {
#pragma unroll
            for (int j = 0; j < L; ++j) list[j] = -INFINITY;
        }
    }

#pragma unroll(KT > 0 ? KT : 1)
    for (int k = 0; k < (KT > 0 ? KT : K); ++k) {
        if (k >= K) break;
        const float top = redux_max(list[0]);
        const unsigned heads = __ballot_sync(kFull, list[0] == top);
        if (list[0] == top && (heads & lower) == 0u) {  // the lowest of the lanes that hold it
            s_pick[warp][k] = make_float2(top, __int_as_float(lane));
#pragma unroll
            for (int j = 0; j + 1 < L; ++j)
                if (KT == 0 || j < KT - 1 - k) list[j] = list[j + 1];
            if (KT == 0 || L <= KT - 1 - k) list[L - 1] = -INFINITY;
        }
    }
    // Pick k is the (same + 1)-th of its lane's experts with this key, where
    // `same` picks right before it have the same key and lane.
    __syncwarp();
    float my_top = -INFINITY;
    int my_lane = 0;
    if (lane < K) {
        const float2 pick = s_pick[warp][lane];
        my_top = pick.x;
        my_lane = __float_as_int(pick.y);
    }
    const float up_top = __shfl_up_sync(kFull, my_top, 1);
    const int up_lane = __shfl_up_sync(kFull, my_lane, 1);
    const unsigned rest = ~__ballot_sync(kFull, lane > 0 && up_top == my_top && up_lane == my_lane);
    int same = lane - (31 - __clz(rest & (0xffffffffu >> (31 - lane))));
    int my_id = -1;
    if (__any_sync(kFull, lane < K && same > 0)) {
#pragma unroll
        for (int j = 0; j < VPL; ++j) {
            const float x = __shfl_sync(kFull, key[j], my_lane);
            if (x == my_top && same-- == 0) my_id = my_lane * VPL + j;
        }
    } else {  // the usual case: the lowest that has it
#pragma unroll
        for (int j = VPL - 1; j >= 0; --j) {
            const float x = __shfl_sync(kFull, key[j], my_lane);
            if (x == my_top) my_id = my_lane * VPL + j;
        }
    }
    if (lane >= K || !(my_top > -INFINITY)) my_id = -1;

    float l = -INFINITY, s = 0.0f;
    if (my_id >= 0) l = clamp_logit(load_one(row + my_id));
    if (a.renorm) {
        s = pick_share<KT == 0 ? 32 : 8>(l, my_id >= 0, a.score);  // the picks are in the first K lanes
    } else if (my_id >= 0) {
        s = sigmoids ? sigmoid(l) : expf(l - m) * inv_total;
    }
    if (lane < K) {
        if (a.picks != nullptr) a.picks[(size_t)t * K + lane] = my_id;
        int id = my_id;
        if (id >= 0 && a.emap != nullptr) {
            id = __ldg(a.emap + id);
            if (id < 0 || id >= E) id = -1;
        }
        a.topk_idx[(size_t)t * K + lane] = id;
        a.topk_w[(size_t)t * K + lane] = s * a.scale;
    }
}

template <int VPL, typename T, int KT>
cudaError_t launch_gate_k(const GateArgs& a, size_t smem, cudaStream_t s) {
    return launch(gate_kernel<VPL, T, KT>, dim3((a.N - 1) / kGateWarps + 1), dim3(kGateWarps * 32), smem,
                  s, a);
}

// The rounds unrolled for the usual numbers of picks: a round then moves only as
// much of the winner's list as the rounds left can need.
template <int VPL, typename T>
cudaError_t launch_gate_v(const GateArgs& a, size_t smem, cudaStream_t s) {
    switch (a.K) {
        case 4: return launch_gate_k<VPL, T, 4>(a, smem, s);
        case 6: return launch_gate_k<VPL, T, 6>(a, smem, s);
        case 8: return launch_gate_k<VPL, T, 8>(a, smem, s);
        default: return launch_gate_k<VPL, T, 0>(a, smem, s);
    }
}

template <typename T>
cudaError_t launch_gate_t(GateArgs a, cudaStream_t s) {
    int vpl = 1;
    while (vpl * 32 < a.E) vpl *= 2;
    // Fewer a lane where that covers the row: shorter lists, no idle lanes, and more
    // often groups of whole lanes.  32768 tokens (us): 160 experts in 8 groups, 6
    // picks, 8 a lane 29.1, 5 a lane 16.7; 160 in one 16.1 and 13.1; 384 in 8
    // groups, 8 picks, 16 a lane 58.7, 12 a lane 24.2; 384 in one 30.1 and 20.7.
    if (vpl == 8 && a.E <= 5 * 32) vpl = 5;
    if (vpl == 16 && a.E <= 12 * 32) vpl = 12;
    const int per = a.E / a.groups, lanes = per / vpl;
    a.lanes_per_group = per % vpl == 0 && (lanes & (lanes - 1)) == 0 ? lanes : 0;
    a.share_lanes = 1;
    while (a.share_lanes * 2 * a.groups <= 32) a.share_lanes *= 2;
    const size_t smem = a.groups > 1 && a.lanes_per_group == 0 ? sizeof(float) * kGateWarps * a.E : 0;
    switch (vpl) {
        case 1: return launch_gate_k<1, T, 0>(a, smem, s);
        case 2: return launch_gate_k<2, T, 0>(a, smem, s);
        case 4: return launch_gate_v<4, T>(a, smem, s);
        case 5: return launch_gate_v<5, T>(a, smem, s);
        case 8: return launch_gate_v<8, T>(a, smem, s);
        case 12: return a.K <= 8 ? launch_gate_k<12, T, 8>(a, smem, s) : launch_gate_k<12, T, 0>(a, smem, s);
        case 16: return a.K <= 8 ? launch_gate_k<16, T, 8>(a, smem, s) : launch_gate_k<16, T, 0>(a, smem, s);
        default: return a.K <= 8 ? launch_gate_k<32, T, 8>(a, smem, s) : launch_gate_k<32, T, 0>(a, smem, s);
    }
}

// ---- gradient ---------------------------------------------------------------
//
// With g_k the gradient of weight k, c the scale, q_k = s_k / sum_j s_j and
// h_k = c g_k - sum_j c g_j q_j:
//   sigmoid, renormalised   dl_k = h_k q_k (1 - s_k)
//   softmax, renormalised   dl_k = h_k q_k   (the full sum cancels)
//   sigmoid                 dl_k = c g_k s_k (1 - s_k)
//   softmax                 dl_e = s_e (c g_e - sum_j c g_j s_j), every expert
// and 0 elsewhere.  The choice of the experts and the bias are constants.

__device__ __forceinline__ void store_one(float* p, float v) { *p = v; }
__device__ __forceinline__ void store_one(__nv_bfloat16* p, float v) { *p = __float2bfloat16_rn(v); }
__device__ __forceinline__ void store_four(float* p, float4 v) {
    *reinterpret_cast<float4*>(p) = v;
}
__device__ __forceinline__ void store_four(__nv_bfloat16* p, float4 v) {
    const __nv_bfloat162 lo = __floats2bfloat162_rn(v.x, v.y), hi = __floats2bfloat162_rn(v.z, v.w);
    uint2 q;
    q.x = *reinterpret_cast<const uint32_t*>(&lo);
    q.y = *reinterpret_cast<const uint32_t*>(&hi);
    *reinterpret_cast<uint2*>(p) = q;
}

// Old ids of the mapped ones: inv[new] = the lowest expert that maps there, E for
// none.  Every thread of the block calls it.
__device__ __forceinline__ void invert_map(const int32_t* emap, int E, int* inv) {
    for (int e = threadIdx.x; e < E; e += kGateWarps * 32) inv[e] = E;
    __syncthreads();
    for (int e = threadIdx.x; e < E; e += kGateWarps * 32) {
        const int to = __ldg(emap + e);
        if (to >= 0 && to < E) atomicMin(inv + to, e);
    }
    __syncthreads();
}

// A pick of token t with the id that topk_idx gave and the gradient of its
// weight: its expert (-1: none, or not available), its logit and scale times the
// gradient (0 without an expert).
template <typename T>
__device__ __forceinline__ int load_pick(const GateGradArgs& a, uint32_t t, int id, const int* inv, float& l, float& g) {
    g *= a.scale;
    if (id < 0 || id >= a.E) id = -1;
    if (id >= 0 && a.emap != nullptr) {
        id = inv[id];
        if (id >= a.E) id = -1;
    }
    l = -INFINITY;
    if (id >= 0) l = load_one(static_cast<const T*>(a.logits) + (size_t)t * a.E + id);
    if (!available(l)) id = -1;
    if (id < 0) g = 0.0f;
    l = clamp_logit(l);
    return id;
}

// Gradients that only the picks get.  A warp takes TPW tokens, each with G = 32 /
// TPW lanes for its picks.  The rows' zeros are stored first, while the picks
// load; the picks' values follow (the barrier orders the two stores).
// 32768 tokens of 256 experts write 33.5 MB.
template <typename T, int TPW>
__global__ void __launch_bounds__(kGateWarps * 32)
gate_backward_kernel(GateGradArgs a) {
    extern __shared__ int s_inv[];
    pdl_prologue();
    constexpr int G = 32 / TPW;
    if (a.emap != nullptr) invert_map(a.emap, a.E, s_inv);
    const int lane = threadIdx.x & 31;
    const uint32_t t0 = (blockIdx.x * kGateWarps + (threadIdx.x >> 5)) * TPW, N = (uint32_t)a.N;
    if (t0 >= N) return;  // warp-uniform
    T* out = static_cast<T*>(a.d_logits) + (size_t)t0 * a.E;
    const int n = (int)min((uint32_t)TPW, N - t0) * a.E;
    const int i = lane / G, k = lane % G;
    const uint32_t t = t0 + i;
    const bool has = k < a.K && t < N;
    int id = -1;
    float g = 0.0f, l = -INFINITY, d = 0.0f;
    if (has) {
        id = __ldg(a.topk_idx + (size_t)t * a.K + k);
        g = __ldg(a.d_w + (size_t)t * a.K + k);
    }
    if (a.vec) {
        for (int e = lane * 4; e < n; e += 128) store_four(out + e, make_float4(0.0f, 0.0f, 0.0f, 0.0f));
    } else {
        for (int e = lane; e < n; e += 32) store_one(out + e, 0.0f);
    }
    if (has) id = load_pick<T>(a, t, id, s_inv, l, g);
    if (a.renorm) {
        const float q = pick_share<G>(l, id >= 0, a.score);
        d = (g - lanes_sum<G>(g * q)) * q;
        if (a.score == kScoreSigmoid && id >= 0) d *= sigmoid(-l);  // 1 - s, without cancellation
    } else {
        const float e = expf(-fabsf(l));
        if (id >= 0) d = g * __fdiv_rn(e, (1.0f + e) * (1.0f + e));  // s (1 - s), likewise
    }
    __syncwarp();
    if (id >= 0) store_one(out + (size_t)i * a.E + id, d);
}

// The softmax without renormalisation: every expert's logit gets a gradient.  One
// warp per token, the row in registers: -s_e sum_j c g_j s_j everywhere, then the
// picks' values over it.
template <int VPL, typename T>
__global__ void __launch_bounds__(kGateWarps * 32)
gate_backward_dense_kernel(GateGradArgs a) {
    extern __shared__ int s_inv[];
    pdl_prologue();
    if (a.emap != nullptr) invert_map(a.emap, a.E, s_inv);
    const int lane = threadIdx.x & 31;
    const uint32_t t = blockIdx.x * kGateWarps + (threadIdx.x >> 5);
    if (t >= (uint32_t)a.N) return;  // warp-uniform
    const int E = a.E, e0 = lane * VPL;
    T* out = static_cast<T*>(a.d_logits) + (size_t)t * E;
    float v[VPL];
    load_row<VPL>(static_cast<const T*>(a.logits) + (size_t)t * E, E, a.vec != 0, lane, v);
    int id = -1;
    float g = 0.0f, l = -INFINITY;
    if (lane < a.K) {
        id = __ldg(a.topk_idx + (size_t)t * a.K + lane);
        g = __ldg(a.d_w + (size_t)t * a.K + lane);
        id = load_pick<T>(a, t, id, s_inv, l, g);
    }
    float m = -INFINITY;
#pragma unroll
    for (int j = 0; j < VPL; ++j)
        if (available(v[j])) m = fmaxf(m, clamp_logit(v[j]));
    m = redux_max(m);
    float sum = 0.0f;
#pragma unroll
    for (int j = 0; j < VPL; ++j) {
        v[j] = available(v[j]) ? expf(clamp_logit(v[j]) - m) : 0.0f;
        sum += v[j];
    }
    sum = lanes_sum<32>(sum);
    const float inv = sum > 0.0f ? __fdiv_rn(1.0f, sum) : 0.0f;
    const float s = id >= 0 ? expf(l - m) * inv : 0.0f;
    const float dot = lanes_sum<32>(g * s);
    const float f = -dot * inv;
    if (VPL >= 4 && a.vec) {
        if constexpr (VPL >= 4) {
#pragma unroll
            for (int j = 0; j < VPL; j += 4)
                if (e0 + j < E)
                    store_four(out + e0 + j, make_float4(v[j] * f, v[j + 1] * f, v[j + 2] * f, v[j + 3] * f));
        }
    } else {
#pragma unroll
        for (int j = 0; j < VPL; ++j)
            if (e0 + j < E) store_one(out + e0 + j, v[j] * f);
    }
    __syncwarp();
    if (id >= 0) store_one(out + id, s * (g - dot));
}

template <int VPL, typename T>
cudaError_t launch_dense(const GateGradArgs& a, size_t smem, cudaStream_t s) {
    return launch(gate_backward_dense_kernel<VPL, T>, dim3((a.N - 1) / kGateWarps + 1),
                  dim3(kGateWarps * 32), smem, s, a);
}

template <typename T, int TPW>
cudaError_t launch_sparse(const GateGradArgs& a, size_t smem, cudaStream_t s) {
    constexpr int per = kGateWarps * TPW;
    return launch(gate_backward_kernel<T, TPW>, dim3((a.N - 1) / per + 1), dim3(kGateWarps * 32), smem, s, a);
}

template <typename T>
cudaError_t launch_backward_t(const GateGradArgs& a, cudaStream_t s) {
    const size_t smem = a.emap != nullptr ? sizeof(int) * a.E : 0;
    if (a.score == kScoreSoftmax && !a.renorm) {
        if (a.E <= 32) return launch_dense<1, T>(a, smem, s);
        if (a.E <= 64) return launch_dense<2, T>(a, smem, s);
        if (a.E <= 128) return launch_dense<4, T>(a, smem, s);
        if (a.E <= 256) return launch_dense<8, T>(a, smem, s);
        if (a.E <= 512) return launch_dense<16, T>(a, smem, s);
        return launch_dense<32, T>(a, smem, s);
    }
    // four tokens a warp where their picks fit 8 lanes each and there are tokens enough
    if (a.K <= 8 && a.N >= kGradManyTokens) return launch_sparse<T, 4>(a, smem, s);
    return launch_sparse<T, 1>(a, smem, s);
}

}  // namespace

cudaError_t launch_gate(const GateArgs& a, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    const cudaError_t err = a.bf16 ? launch_gate_t<__nv_bfloat16>(a, s) : launch_gate_t<float>(a, s);
    note_launch();
    return err;
}

cudaError_t launch_gate_backward(const GateGradArgs& a, cudaStream_t s) {
    if (a.N == 0) return cudaSuccess;
    const cudaError_t err = a.bf16 ? launch_backward_t<__nv_bfloat16>(a, s) : launch_backward_t<float>(a, s);
    note_launch();
    return err;
}

}  // namespace ep
