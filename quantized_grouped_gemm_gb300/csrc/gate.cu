// gate.cu -- the gate over given router logits (moe_gate): scores, groups, top-k, weights.
//
// One warp per token, no memory traffic but the logits in and the choice out.  The lanes are shared out
// among the groups (all 32 to the one group where there are none); a lane holds up to P consecutive
// experts of its group, so the order (lane, position) is the order of the expert indices.
//
// The kernel is bound by instructions, not by its bytes (256 fp32 logits are 32 a lane), so the top k are
// found without sorting E values.  Each lane takes the maximum of each of S parts of its values; the k-th
// largest of these 32 S samples is a lower bound B of the k-th largest value (k samples are >= B), so only
// values >= B can be chosen -- about 9 of 256 for k = 8.  Those are compacted through shared memory, and each
// finds its rank by counting the ones above it (and, when the ranks turn out not to be a permutation, the equal ones
// before it).  More than 64 candidates go to gate_slow.
//
// Measured: 65536 x 256 fp32 sigmoid scores with a bias in 8 groups, k = 8: 33 us = 2.2 TB/s of logits and choices (31.6 where
// these stay in L2), 523 instructions a token (86 % of the issue slots; 10.5 us would be the bytes); 4096 x 512 bf16 with a
// bias, k = 10: 5.3 us; up to 512 tokens of 256: 2.0-2.7 us, a launch and one token's chain of dependent reductions.
#include "moe_internal.cuh"

#include <cuda_fp16.h>

namespace moe {
namespace {

constexpr int kGateWarps = 8;
constexpr int kMaxCand = 64;   // candidates ranked by counting: up to two a lane
constexpr uint32_t kAll = 0xffffffffu;
constexpr float kInf = __builtin_huge_valf(), kMaxF = 3.402823466e+38f, kMinNormal = 1.175494351e-38f;

// How the choice values come about.
enum GateMode {
    kLogits,        // neither bias nor groups: scores rise with the logits, which are compared themselves, before any
                    // rounding (those whose score is 0 as equals); only the chosen experts' scores are computed
    kLogitsTotal,   // the same, with the softmax's sum over all experts (weights not renormalised)
    kScores,        // a bias: every expert's score
    kGroups         // groups, with or without a bias
};

__device__ __forceinline__ float warp_max(float v) {   // a NaN operand is dropped
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o >= 1; o >>= 1) v += __shfl_xor_sync(kAll, v, o);
    return v;
}

// 2^t by the hardware, good to about 2^-22, results below 2^-126 as 0.
__device__ __forceinline__ float exp2_f32(float t) {
    float p;
    asm("ex2.approx.ftz.f32 %0, %1;" : "=f"(p) : "f"(t));
    return p;
}
constexpr float kLog2e = 1.44269504f;
// Logits (softmax: less the largest) from which on a score is 0, next to the smallest normal number.
constexpr float kLowest = -87.0f;
// Scores.  The argument's rounding, 2^-24 |x log2 e| and a little from log2 e itself, is a relative error of 7.3e-8 |x|:
// under 1e-6 for scores down to exp(-8) of the largest (a sigmoid near 1 has a (1 - s)-th of it), 6e-6 for those near
// exp(-80), which only a bias can choose; a two-part product for every expert would cost three instructions on each.
// -inf and NaN (fmaxf drops it) give 0.
__device__ __forceinline__ float sigmoid_score(float l) {
    float r;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(r) : "f"(1.0f + exp2_f32(fmaxf(l, -__builtin_huge_valf()) * -kLog2e)));
    return r;
}
__device__ __forceinline__ float softmax_term(float x) { return exp2_f32(fmaxf(x, -__builtin_huge_valf()) * kLog2e); }

template <typename T> __device__ __forceinline__ float logit_f32(T v, bool f16);
template <> __device__ __forceinline__ float logit_f32<float>(float v, bool) { return v; }
template <> __device__ __forceinline__ float logit_f32<uint16_t>(uint16_t v, bool f16) {
    return f16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}

// A token whose candidates are too many to rank by counting: many equal values, as when experts are switched off.
// Where fewer than k values are above `bound` (its equals make them enough), these and as many of the equals as are
// wanted, in index order, are ranked by counting; else the distinct values are taken in turn, from the largest, each with
// all the experts that have it in index order, until k are chosen (there are at least k).  e0, cnt: the lane's experts
// that can be chosen.  Lane j < k gets slot j's expert and score.
// Not inlined, as the usual path has to fit the instruction cache, and the values are worked out again, as handing them
// over costs the usual path registers (12875 x 728, k = 23 in bf16: 33.9 against 24.8 us then, 26 now).
struct Chosen {
    int e;
    float s;
};
template <typename T, int P>
__device__ __noinline__ Chosen gate_slow(const GateArgs& a, long long tok, int e0, int cnt, float bound, float m,
                                         float inv) {
    __shared__ uint16_t order[kGateWarps][32];
    __shared__ float value[kGateWarps][32];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const T* row = static_cast<const T*>(a.logits) + tok * a.stride;
    const bool by_score = a.bias || a.groups > 1;
    const auto logit = [&](T l) { return fminf(fmaxf(logit_f32<T>(l, a.f16), -kInf), kMaxF); };
    const auto score = [&](float x) { return a.sigmoid ? sigmoid_score(x) : softmax_term(x) * inv; };
    float v[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        v[i] = -kInf;
        if (i < cnt) {
            const float l = logit(row[e0 + i]), x = l - m;
            if (a.bias) v[i] = fmaxf(score(x) + __ldg(a.bias + e0 + i), -kMaxF);
            else if (by_score) v[i] = score(x);
            else if (a.sigmoid) v[i] = fmaxf(x, kLowest);
            else v[i] = x > kLowest ? (m > -kMaxF ? l : x) : -kMaxF;
        }
    }
    if (bound == -kInf) {   // the samples ran out among equals: the least of the lanes' largest values
        float least = -kInf;
#pragma unroll
        for (int i = 0; i < P; ++i) least = fmaxf(least, v[i]);
        bound = -warp_max(cnt > 0 ? -least : -kInf);
    }
    int n = 0;   // values above the bound; 2^16: values equal to it
#pragma unroll
    for (int i = 0; i < P; ++i) n += (v[i] > bound) + ((v[i] == bound) << 16);
    const int mine = n;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int other = __shfl_up_sync(kAll, n, o);
        if (lane >= o) n += other;
    }
    const int total = __shfl_sync(kAll, n, 31), wanted = a.k - (total & 0xffff);   // equals to take
    n -= mine;
    if (wanted > 0 && wanted <= total >> 16) {
        int equals = n >> 16, at = (n & 0xffff) + min(equals, wanted);
#pragma unroll
        for (int i = 0; i < P; ++i) {
            if (v[i] > bound || (v[i] == bound && equals++ < wanted)) {
                value[warp][at] = v[i];
                order[warp][at++] = (uint16_t)(e0 + i);
            }
        }
        __syncwarp();
        const int e = order[warp][lane < a.k ? lane : 0];
        const float x = value[warp][lane < a.k ? lane : 0];
        int rank = 0;
        for (int j = 0; j < a.k; ++j) {
            const float o = value[warp][j];
            rank += o > x || (o == x && j < lane);
        }
        __syncwarp();
        if (lane < a.k) order[warp][rank] = (uint16_t)e;
    } else {
        float last = 0.0f;
        // the first round looks at every value, +inf (an infinite bias) among them; a round takes one expert at least
        for (int slots = 0, round = 0; slots < a.k && round < a.k; ++round) {
            float best = -kInf;
#pragma unroll
            for (int i = 0; i < P; ++i) best = fmaxf(best, round == 0 || v[i] < last ? v[i] : -kInf);
            last = warp_max(best);
            int mine = 0;
#pragma unroll
            for (int i = 0; i < P; ++i) mine += v[i] == last;
            int at = mine;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int other = __shfl_up_sync(kAll, at, o);
                if (lane >= o) at += other;
            }
            const int total = __shfl_sync(kAll, at, 31);
            at += slots - mine;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (v[i] == last) {
                    if (at < a.k) order[warp][at] = (uint16_t)(e0 + i);
                    ++at;
                }
            }
            slots += total;
        }
    }
    __syncwarp();
    Chosen c{0, 0.0f};
    if (lane < a.k) {
        c.e = order[warp][lane];
        const float x = logit(row[c.e]) - m;
        c.s = x > kLowest || by_score ? score(x) : 0.0f;
    }
    return c;
}

// P: the most experts a lane holds (fewer at the end of a group); S: samples a lane gives to the bound.
// Two CTAs to an SM where a lane holds up to 64: 128 registers with a few spills against 150 (20000 x 1020 in 17 groups,
// bias: 83 against 116 us in bf16, 75 against 105 in fp32; 300 tokens 9.2-9.8 against 8.9-9.6).
template <typename T, int P, int S, GateMode kMode>
__global__ void __launch_bounds__(32 * kGateWarps, P > 32 ? 2 : 0) gate_kernel(const __grid_constant__ GateArgs a) {
    constexpr bool kByScore = kMode == kScores || kMode == kGroups;
    constexpr int kCap = 32 * P < kMaxCand ? 32 * P : kMaxCand;
    __shared__ __align__(16) float c_v[kGateWarps][kCap];   // the candidates' values,
    __shared__ float2 c_se[kGateWarps][kCap];               // scores (or logits) and indices
    __shared__ uint8_t c_win[kGateWarps][kMaxCand];
    // A candidate's score is kept where a lane holds few experts.  Else it is worked out again from the logit of the
    // chosen, so that the scores need no registers after the choice values (4096 x 512, k = 10 in bf16 with bias:
    // 5.8 against 6.9 us; one token of 256 experts 2.6 against 2.1 us, the reload's latency).  By logits the value
    // is the logit.
    constexpr bool kKeep = kByScore && P <= 8;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tok = (long long)blockIdx.x * kGateWarps + warp;
    pdl_wait();
    pdl_launch_dependents();
    if (tok >= a.T) return;
    // this lane's experts: e0 .. e0 + cnt - 1
    const int lpg = 1 << a.lane_shift, g = lane >> a.lane_shift, sub = lane & (lpg - 1);
    const int e0 = g * a.per + sub * a.lane_experts;
    const int cnt = a.full ? P : g < a.groups ? max(0, min(a.lane_experts, a.per - sub * a.lane_experts)) : 0;
    const T* row = static_cast<const T*>(a.logits) + tok * a.stride + e0;

    float s[P];   // logits, then with kByScore scores
    constexpr int V = 16 / (int)sizeof(T) < P ? 16 / (int)sizeof(T) : P;   // elements of a vector load
    if (V * sizeof(T) == 16 && a.vec) {
#pragma unroll
        for (int c = 0; c < P; c += V) {
            if (a.full || c + V <= cnt) {
                const uint4 q = ld_nc_v4(row + c);
                const uint32_t w[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int i = 0; i < V; ++i) {
                    if (sizeof(T) == 4) s[c + i] = __uint_as_float(w[i % 4]);
                    else s[c + i] = logit_f32<uint16_t>((uint16_t)(w[(i / 2) % 4] >> (16 * (i % 2))), a.f16);
                }
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i) s[c + i] = c + i < cnt ? logit_f32<T>(row[c + i], a.f16) : -kInf;
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) s[i] = i < cnt ? logit_f32<T>(row[i], a.f16) : -kInf;
    }

    float inv = 1.0f, m = 0.0f, peak = 0.0f;   // softmax: the largest logit, and what the largest of s is
    if (!a.sigmoid) {
        m = s[0];
#pragma unroll
        for (int i = 1; i < P; ++i) m = fmaxf(m, s[i]);   // fmaxf drops a NaN
        m = warp_max(m);
        peak = m;
        if (!(m > -kMaxF && m <= kMaxF)) {   // +inf counts as the largest number; nothing left: every score is 0
            const bool lowest = m == -kMaxF;
            m = m > 0.0f ? kMaxF : lowest ? m : 0.0f;
            peak = m;
#pragma unroll
            for (int i = 0; i < P; ++i) s[i] = fminf(fmaxf(s[i], -kInf), kMaxF);
            if (!kByScore && lowest) {   // -FLT_MAX will mark a score of 0
                peak = 0.0f;
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] -= m;
            }
        }
        if (kMode != kLogits) {
            float z = 0.0f;
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const float x = softmax_term(s[i] - peak);
                z += x;
                if (kByScore) s[i] = x;
            }
            z = warp_sum(z);
            inv = z > 0.0f ? 1.0f / z : 0.0f;
            if (kByScore) {
#pragma unroll
                for (int i = 0; i < P; ++i) s[i] *= inv;
            }
        }
    } else if (kByScore) {
#pragma unroll
        for (int i = 0; i < P; ++i) s[i] = sigmoid_score(s[i]);
    }

    // choice values (at least -FLT_MAX, also for NaN; +inf with an infinite bias); -inf marks what cannot be chosen
    float v[P];
    if (kByScore) {
        if (a.bias) {
            if (P % 4 == 0 && a.bias_vec) {
#pragma unroll
                for (int c = 0; c < P; c += 4) {
                    if (a.full || c + 4 <= cnt) {
                        const float4 b = ld_nc_f4(a.bias + e0 + c);
                        v[c] = s[c] + b.x; v[(c + 1) % P] = s[(c + 1) % P] + b.y;
                        v[(c + 2) % P] = s[(c + 2) % P] + b.z; v[(c + 3) % P] = s[(c + 3) % P] + b.w;
                    } else {
#pragma unroll
                        for (int i = c; i < c + 4 && i < P; ++i) v[i] = i < cnt ? s[i] + __ldg(a.bias + e0 + i) : 0.0f;
                    }
                }
            } else {
#pragma unroll
                for (int i = 0; i < P; ++i) v[i] = i < cnt ? s[i] + __ldg(a.bias + e0 + i) : 0.0f;
            }
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = fmaxf(v[i], -kMaxF);
        } else {
#pragma unroll
            for (int i = 0; i < P; ++i) v[i] = s[i];
        }
    } else if (a.sigmoid) {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = fminf(fmaxf(s[i], kLowest), kMaxF);
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i) v[i] = s[i] - peak > kLowest ? s[i] : -kMaxF;
    }
    if (!a.full) {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (i >= cnt) v[i] = -kInf;
    }

    float lane_max = v[0];
    bool kept = true;   // this lane's experts can be chosen from
    if (kMode == kGroups) {
        // the two best of the lane, then of the group's lanes
        float v1 = v[0], v2 = -kInf;
#pragma unroll
        for (int i = 1; i < P; ++i) {
            v2 = fmaxf(v2, fminf(v1, v[i]));
            v1 = fmaxf(v1, v[i]);
        }
        lane_max = v1;
        for (int o = lpg >> 1; o >= 1; o >>= 1) {
            const float o1 = __shfl_xor_sync(kAll, v1, o), o2 = __shfl_xor_sync(kAll, v2, o);
            v2 = fmaxf(fmaxf(v2, o2), fminf(v1, o1));
            v1 = fmaxf(v1, o1);
        }
        // the group_topk best groups: those of at least the value that group_topk rounds of a maximum reach, unless ties
        // make them more; then one group a round, the lowest lane (so the lowest group) first
        const float worth = g < a.groups ? fmaxf(a.group_max ? v1 : v1 + v2, -kMaxF) : -kInf;
        float left = worth, least = 0.0f;
#pragma unroll 4
        for (int j = 0; j < a.group_topk; ++j) {
            least = warp_max(left);
            if (left == least) left = -kInf;
        }
        kept = worth >= least && g < a.groups;
        if (__builtin_expect(__popc(__ballot_sync(kAll, kept)) != a.group_topk << a.lane_shift, 0)) {
            kept = false;
            left = worth;
            for (int j = 0; j < a.group_topk; ++j) {
                const float top = warp_max(left);
                if (g == (__ffs(__ballot_sync(kAll, left == top)) - 1) >> a.lane_shift) {
                    kept = true;
                    left = -kInf;
                }
            }
        }
    } else {
#pragma unroll
        for (int i = 1; i < P; ++i) lane_max = fmaxf(lane_max, v[i]);
    }

    // candidates: one a lane where a lane holds one expert anyway
    bool slow = false;
    float cv = kept ? v[0] : -kInf, cs = kKeep ? s[0] : v[0];
    int ce = e0, cand = 32;
    float bound = -kMaxF;
    if (P > 1) {
        float h[S];
#pragma unroll
        for (int q = 0; q < S; ++q) {
            h[q] = S == 1 ? lane_max : v[q * (P / S)];
#pragma unroll
            for (int i = 1; i < P / S && S > 1; ++i) h[q] = fmaxf(h[q], v[q * (P / S) + i]);
            h[q] = kept ? h[q] : -kInf;
        }
#pragma unroll 4
        for (int j = 0; j < a.rounds; ++j) {   // equal samples leave together, which only lowers the bound
            float best = h[0];
#pragma unroll
            for (int q = 1; q < S; ++q) best = fmaxf(best, h[q]);
            const float top = warp_max(best);
            bound = top;
#pragma unroll
            for (int q = 0; q < S; ++q)
                if (h[q] == top) h[q] = -kInf;
        }
        const float least = kept ? bound : __int_as_float(0x7fffffff);   // (no value is >= NaN, +inf neither)
        c_v[warp][lane] = -kInf;          // ranks are counted in fours
        int mine = 0;
#pragma unroll
        for (int i = 0; i < P; ++i) mine += v[i] >= least;
        int at = mine;   // inclusive sum over the lanes, so candidates are kept in the order of their indices
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int other = __shfl_up_sync(kAll, at, o);
            if (lane >= o) at += other;
        }
        cand = __shfl_sync(kAll, at, 31);
        slow = cand > kCap;               // (a bound of -inf, when the samples ran out among equals, counts every lane's P)
        at -= mine;
        __syncwarp();
        if (!slow) {
#pragma unroll
            for (int i = 0; i < P; ++i) {
                if (v[i] >= least) {
                    c_v[warp][at] = v[i];
                    c_se[warp][at] = make_float2(kKeep ? s[i] : v[i], __int_as_float(e0 + i));
                    ++at;
                }
            }
        }
        __syncwarp();
        if (cand <= 32) {
            const float2 se = c_se[warp][lane < cand ? lane : 0];
            cv = lane < cand ? c_v[warp][lane] : -kInf;
            cs = se.x;
            ce = __float_as_int(se.y);
        }
    }

    int slot = -1;   // the chosen expert of this lane, if any: slot, index, score (or logit)
    if (P > 1 && cand <= 32) {
        int rank = 0;
        if (cand <= 16) {   // two lanes to a candidate, each counts eight
            const float x = c_v[warp][lane & 15];
            const float4* half = reinterpret_cast<const float4*>(&c_v[warp][(lane & 16) >> 1]);
#pragma unroll
            for (int j = 0; j < 2; ++j) rank += (half[j].x > x) + (half[j].y > x) + (half[j].z > x) + (half[j].w > x);
            rank += __shfl_xor_sync(kAll, rank, 16);
        } else {
            for (int j = 0; j < cand; j += 4) {
                const float4 o = *reinterpret_cast<const float4*>(&c_v[warp][j]);
                rank += (o.x > cv) + (o.y > cv) + (o.z > cv) + (o.w > cv);
            }
        }
        // no ties: the ranks of the candidates are 0 .. cand - 1
        if (__reduce_or_sync(kAll, lane < cand ? 1u << rank : 0u) != kAll >> (32 - cand)) {
            // ties: equals have one rank, and the candidates are in index order
            rank += __popc(__match_any_sync(kAll, lane < cand ? rank : 64 + lane) & ((1u << lane) - 1u));
        }
        if (lane < cand && rank < a.k) slot = rank;
    } else if (P > 1 && !slow) {
        // two a lane; chosen when the ranks below k are all there, once each
        if (lane < 4 && cand + lane < kCap) c_v[warp][cand + lane] = -kInf;
        __syncwarp();
        const float v0 = c_v[warp][lane], v1 = lane + 32 < cand ? c_v[warp][(lane + 32) % kCap] : -kInf;
        int r0 = 0, r1 = 0;
        for (int j = 0; j < cand; j += 4) {
            const float4 o = *reinterpret_cast<const float4*>(&c_v[warp][j]);
            r0 += (o.x > v0) + (o.y > v0) + (o.z > v0) + (o.w > v0);
            r1 += (o.x > v1) + (o.y > v1) + (o.z > v1) + (o.w > v1);
        }
        bool in0 = r0 < a.k, in1 = lane + 32 < cand && r1 < a.k;
        const uint32_t ranks = __reduce_or_sync(kAll, (in0 ? 1u << r0 : 0u) | (in1 ? 1u << r1 : 0u));
        const int count = __popc(__ballot_sync(kAll, in0)) + __popc(__ballot_sync(kAll, in1));
        if (count != a.k || __popc(ranks) != a.k) {   // ties, as above
            c_win[warp][lane] = c_win[warp][lane + 32] = 0;   // by rank: how many of the first 32 have it
            __syncwarp();
            const uint32_t m0 = __match_any_sync(kAll, r0);
            const uint32_t m1 = __match_any_sync(kAll, lane + 32 < cand ? r1 : 64 + lane);
            c_win[warp][r0] = (uint8_t)__popc(m0);
            __syncwarp();
            if (lane + 32 < cand) r1 += c_win[warp][r1] + __popc(m1 & ((1u << lane) - 1u));
            r0 += __popc(m0 & ((1u << lane) - 1u));
            __syncwarp();
            in0 = r0 < a.k;
            in1 = lane + 32 < cand && r1 < a.k;
        }
        if (in0) c_win[warp][r0] = (uint8_t)lane;
        if (in1) c_win[warp][r1] = (uint8_t)(lane + 32);
        __syncwarp();
        if (lane < a.k) {
            const float2 se = c_se[warp][c_win[warp][lane]];
            slot = lane;
            cs = se.x;
            ce = __float_as_int(se.y);
        }
    }
    if (P == 1) {   // k rounds over the lanes, which hold the experts in index order
        for (int j = 0; j < a.k; ++j) {
            const float top = warp_max(cv);
            if (lane == __ffs(__ballot_sync(kAll, cv == top)) - 1) {
                slot = j;
                cv = -kInf;
            }
        }
    }

    float w = cs;
    if (!kKeep) {
        if (kByScore && slot >= 0) {
            const float l = logit_f32<T>(static_cast<const T*>(a.logits)[tok * a.stride + ce], a.f16);
            cs = fminf(fmaxf(l, -kInf), kMaxF);
        }
        cs -= kByScore ? m : peak;
        w = cs > kLowest ? (a.sigmoid ? sigmoid_score(cs) : softmax_term(cs) * inv) : 0.0f;
    }
    if (P > 1 && slow) {
        const Chosen c = gate_slow<T, P>(a, tok, e0, kept ? cnt : 0, bound, m, inv);
        slot = lane < a.k ? lane : -1;
        ce = c.e;
        w = c.s;
    }
    if (slot < 0) w = 0.0f;
    if (a.renormalise) {
        const float z = warp_sum(w);
        w *= z >= kMinNormal ? __fdividef(1.0f, z) : 0.0f;   // (1 / z stays finite; scale / z need not)
        w *= a.scale;
    } else {
        w *= a.scale;
    }
    if (slot >= 0) {
        a.topk_idx[tok * a.k + slot] = ce;
        a.topk_w[tok * a.k + slot] = w;
    }
}

template <typename T, int P, int S>
cudaError_t launch_ps(const GateArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.T + kGateWarps - 1) / kGateWarps)), block(32 * kGateWarps);
    if (a.groups > 1) return launch_with_pdl(gate_kernel<T, P, S, kGroups>, grid, block, 0, st, a);
    if constexpr (P <= 32) {   // a lane holds more than 32 experts only where groups leave lanes idle
        if (a.bias) return launch_with_pdl(gate_kernel<T, P, S, kScores>, grid, block, 0, st, a);
        if (!a.sigmoid && !a.renormalise) return launch_with_pdl(gate_kernel<T, P, S, kLogitsTotal>, grid, block, 0, st, a);
        return launch_with_pdl(gate_kernel<T, P, S, kLogits>, grid, block, 0, st, a);
    }
    return cudaErrorInvalidValue;
}

// Samples: the fewest parts to a lane, of 1, 4 and 8, with which k is at most 9/16 of the samples (about 1.4 k candidates
// then, 25 for k = 18 of 256); a round costs as many times as much.  All are candidates where they are at most 64 and k
// is large.
template <typename T, int P>
cudaError_t launch_p(GateArgs a, cudaStream_t st) {
    const int lanes = (a.groups > 1 ? a.group_topk : 1) * ((a.per + a.lane_experts - 1) / a.lane_experts);   // that can matter
    const auto enough = [&](int s) { return 16 * a.k <= 9 * lanes * ((a.lane_experts * s + P - 1) / P); };
    a.full = a.lane_experts == P && a.per == P << a.lane_shift && a.groups << a.lane_shift == 32;
    a.rounds = a.k;
    if (P > 1 && lanes * a.lane_experts <= kMaxCand && 4 * a.k > lanes) a.rounds = 0;
    else if constexpr (P >= 4) {
        if (!enough(1)) {
            if constexpr (P >= 8)
                if (!enough(4)) return launch_ps<T, P, 8>(a, st);
            return launch_ps<T, P, 4>(a, st);
        }
    }
    return launch_ps<T, P, 1>(a, st);
}

template <typename T>
cudaError_t launch_t(GateArgs a, cudaStream_t st) {
    int lanes = 32;   // of a group: a power of two
    while (lanes * a.groups > 32) lanes /= 2;
    a.lane_shift = lanes == 32 ? 5 : lanes == 16 ? 4 : lanes == 8 ? 3 : lanes == 4 ? 2 : lanes == 2 ? 1 : 0;
    int need = (a.per + lanes - 1) / lanes;
    // vector loads: every group and lane starts at a multiple of 16 bytes (lanes of at least four experts: a short one
    // is loaded by elements anyway)
    constexpr int kVec = 16 / (int)sizeof(T);
    a.vec = a.vec && (a.groups == 1 || a.per % kVec == 0) && need >= kVec;
    if (a.vec) need = (need + kVec - 1) / kVec * kVec;
    a.lane_experts = need;
    a.bias_vec = reinterpret_cast<uintptr_t>(a.bias) % 16 == 0 && (a.groups == 1 || a.per % 4 == 0) && need % 4 == 0;
    if (need <= 1) return launch_p<T, 1>(a, st);
    if (need <= 2) return launch_p<T, 2>(a, st);
    if (need <= 4) return launch_p<T, 4>(a, st);
    if (need <= 8) return launch_p<T, 8>(a, st);
    if (need <= 16) return launch_p<T, 16>(a, st);
    if (need <= 32) return launch_p<T, 32>(a, st);
    return launch_p<T, 64>(a, st);
}

}  // namespace

cudaError_t launch_gate(const GateArgs& a, int logits_type, cudaStream_t st, unsigned long long* launches) {
    *launches += 1;
    return logits_type == MOE_F32 ? launch_t<float>(a, st) : launch_t<uint16_t>(a, st);
}

}  // namespace moe
