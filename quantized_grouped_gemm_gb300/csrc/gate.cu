// gate.cu -- the gate over given router logits (moe_gate): scores, groups, top-k, weights.
//
// One warp per token.  Lane l holds the P = 2^p >= E/32 consecutive experts l*P .. l*P + P-1, so the
// order (lane, position) is the order of the expert indices and ties resolve to the lower index by
// taking the lowest lane.
#include "moe_internal.cuh"

#include <cuda_bf16.h>
#include <cuda_fp16.h>
#include <math_constants.h>

namespace moe {
namespace {

constexpr int kGateWarps = 8;

__device__ __forceinline__ uint32_t warp_max_u32(uint32_t v) { return __reduce_max_sync(0xffffffffu, v); }

// Order-preserving key of a choice value (+0 and -0 alike); -inf maps to 0x007fffff, so 0 stays free
// for "cannot be chosen".  NaN counts as -inf.
__device__ __forceinline__ uint32_t choice_key(float v) {
    if (!(v == v)) v = -CUDART_INF_F;
    v += 0.0f;
    const uint32_t u = __float_as_uint(v);
    return (u & 0x80000000u) ? ~u : (u | 0x80000000u);
}

template <typename T> __device__ __forceinline__ float to_f32(T v);
template <> __device__ __forceinline__ float to_f32<float>(float v) { return v; }
template <> __device__ __forceinline__ float to_f32<__nv_bfloat16>(__nv_bfloat16 v) { return __bfloat162float(v); }
template <> __device__ __forceinline__ float to_f32<__half>(__half v) { return __half2float(v); }

template <typename T, int P, bool kSigmoid, bool kGroups>
__global__ void __launch_bounds__(32 * kGateWarps) gate_kernel(GateArgs a) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const long long tok = (long long)blockIdx.x * kGateWarps + warp;
    __shared__ float s_group[kGateWarps][32];
    pdl_wait();
    pdl_launch_dependents();
    if (tok >= a.T) return;
    const int E = a.E, e0 = lane * P;
    const T* row = static_cast<const T*>(a.logits) + tok * a.stride;

    float s[P];   // logits, then scores
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = -CUDART_INF_F;
    constexpr int V = 16 / (int)sizeof(T) < P ? 16 / (int)sizeof(T) : P;   // elements of a vector load
    if (a.vec && V * sizeof(T) == 16) {
#pragma unroll
        for (int c = 0; c < P; c += V) {
            if (e0 + c + V <= E) {
                const uint4 q = ld_nc_v4(row + e0 + c);
                const T* t = reinterpret_cast<const T*>(&q);
#pragma unroll
                for (int i = 0; i < V; ++i) s[c + i] = to_f32(t[i]);
            } else {
#pragma unroll
                for (int i = 0; i < V; ++i)
                    if (e0 + c + i < E) s[c + i] = to_f32(row[e0 + c + i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (e0 + i < E) s[i] = to_f32(row[e0 + i]);
    }
    // NaN counts as -inf, +inf as the largest finite number (fmaxf drops a NaN operand)
#pragma unroll
    for (int i = 0; i < P; ++i) s[i] = fminf(fmaxf(s[i], -CUDART_INF_F), CUDART_MAX_NORMAL_F);

    if (kSigmoid) {
#pragma unroll
        for (int i = 0; i < P; ++i) s[i] = __fdividef(1.0f, 1.0f + expf(-s[i]));   // exp(inf): 1 / inf = 0
    } else {
        float m = s[0];
#pragma unroll
        for (int i = 1; i < P; ++i) m = fmaxf(m, s[i]);
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
        if (m == -CUDART_INF_F) m = 0.0f;   // nothing left: every score is exp(-inf) = 0
        float z = 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) {
            s[i] = expf(s[i] - m);
            z += s[i];
        }
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        const float r = z > 0.0f ? 1.0f / z : 0.0f;
#pragma unroll
        for (int i = 0; i < P; ++i) s[i] *= r;
    }

    // choice values as keys; experts beyond E cannot be chosen
    uint32_t key[P];
#pragma unroll
    for (int i = 0; i < P; ++i) {
        const float v = a.bias && e0 + i < E ? s[i] + __ldg(a.bias + e0 + i) : s[i];
        key[i] = e0 + i < E ? choice_key(v) : 0u;
    }

    if (kGroups) {
        // worth of group g, then the groups kept: a bit per group
        const int per = E / a.groups;
        for (int g = 0; g < a.groups; ++g) {
            uint32_t k1 = 0, k2 = 0;   // this lane's two best of the group
#pragma unroll
            for (int i = 0; i < P; ++i) {
                const int e = e0 + i;
                if (e >= g * per && e < (g + 1) * per) {
                    k2 = max(k2, min(k1, key[i]));
                    k1 = max(k1, key[i]);
                }
            }
            const uint32_t b1 = warp_max_u32(k1);
            const uint32_t has = __ballot_sync(0xffffffffu, k1 == b1);
            const uint32_t b2 = warp_max_u32(lane == __ffs(has) - 1 ? k2 : k1);
            const auto val = [](uint32_t k) { return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k); };
            if (lane == g) s_group[warp][g] = a.group_max ? val(b1) : val(b1) + val(b2);
        }
        __syncwarp();
        uint32_t mine = lane < a.groups ? choice_key(s_group[warp][lane]) : 0u;
        int rank = 0;
        for (int g = 0; g < a.groups; ++g) {
            const uint32_t other = choice_key(s_group[warp][g]);
            rank += other > mine || (other == mine && g < lane);
        }
        const uint32_t kept = __ballot_sync(0xffffffffu, lane < a.groups && rank < a.group_topk);
#pragma unroll
        for (int i = 0; i < P; ++i)
            if (e0 + i < E && !((kept >> ((e0 + i) / per)) & 1u)) key[i] = 0u;
    }

    // k rounds: the warp's largest key, the lowest lane that has it, that lane's first position
    int my_e = 0;
    float my_s = 0.0f;
    for (int j = 0; j < a.k; ++j) {
        uint32_t best = key[0];
#pragma unroll
        for (int i = 1; i < P; ++i) best = max(best, key[i]);
        const uint32_t top = warp_max_u32(best);
        const int from = __ffs(__ballot_sync(0xffffffffu, best == top)) - 1;
        int e = 0;
        float sc = 0.0f;
        if (lane == from) {
            bool found = false;
#pragma unroll
            for (int i = 0; i < P; ++i)
                if (!found && key[i] == top) {
                    found = true;
                    key[i] = 0u;
                    e = e0 + i;
                    sc = s[i];
                }
        }
        e = __shfl_sync(0xffffffffu, e, from);
        sc = __shfl_sync(0xffffffffu, sc, from);
        if (lane == j) {
            my_e = e;
            my_s = sc;
        }
    }
    float w = lane < a.k ? my_s : 0.0f;
    if (a.renormalise) {
        float z = w;
#pragma unroll
        for (int o = 16; o >= 1; o >>= 1) z += __shfl_xor_sync(0xffffffffu, z, o);
        w = z > 0.0f ? w / z : 0.0f;
    }
    if (lane < a.k) {
        a.topk_idx[tok * a.k + lane] = my_e;
        a.topk_w[tok * a.k + lane] = w * a.scale;
    }
}

template <typename T, int P>
cudaError_t launch_p(const GateArgs& a, cudaStream_t st) {
    const dim3 grid((unsigned)((a.T + kGateWarps - 1) / kGateWarps)), block(32 * kGateWarps);
    if (a.sigmoid)
        return a.groups > 1 ? launch_with_pdl(gate_kernel<T, P, true, true>, grid, block, 0, st, a)
                            : launch_with_pdl(gate_kernel<T, P, true, false>, grid, block, 0, st, a);
    return a.groups > 1 ? launch_with_pdl(gate_kernel<T, P, false, true>, grid, block, 0, st, a)
                        : launch_with_pdl(gate_kernel<T, P, false, false>, grid, block, 0, st, a);
}

template <typename T>
cudaError_t launch_t(const GateArgs& a, cudaStream_t st) {
    if (a.E <= 32) return launch_p<T, 1>(a, st);
    if (a.E <= 64) return launch_p<T, 2>(a, st);
    if (a.E <= 128) return launch_p<T, 4>(a, st);
    if (a.E <= 256) return launch_p<T, 8>(a, st);
    if (a.E <= 512) return launch_p<T, 16>(a, st);
    return launch_p<T, 32>(a, st);
}

}  // namespace

cudaError_t launch_gate(const GateArgs& a, int logits_type, cudaStream_t st, unsigned long long* launches) {
    *launches += 1;
    if (logits_type == MOE_BF16) return launch_t<__nv_bfloat16>(a, st);
    if (logits_type == MOE_F16) return launch_t<__half>(a, st);
    return launch_t<float>(a, st);
}

}  // namespace moe
