// linear_common.cuh -- what the kernels of moe_linear share: element types, the epilogue's activation
// functions and the store of one output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

#ifdef __CUDACC__

// act(z) in fp32.  kExact (fp32 outputs): CUDA's full-precision functions.  Else the result is rounded
// to bf16 or fp16 (8 or 11 bits), and the exponential is the hardware one: its relative error,
// a few 2^-23 and another 2^-24 |z|, disappears in that rounding.
template <bool kExact>
__device__ __forceinline__ float sigmoid_f32(float z) {
    return kExact ? 1.0f / (1.0f + expf(-z)) : __fdividef(1.0f, 1.0f + __expf(-z));
}

template <bool kExact>
__device__ __forceinline__ float apply_act(int act, float z) {
    switch (act) {
        case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;   // a NaN stays one
        case MOE_ACT_SILU: return z * sigmoid_f32<kExact>(z);
        // z Phi(z): erfc keeps the relative accuracy where Phi is small
        case MOE_ACT_GELU: return 0.5f * z * erfcf(-0.70710678f * z);
        // tanh form: 0.5 z (1 + tanh u) = z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
        case MOE_ACT_GELU_TANH: return z * sigmoid_f32<kExact>(1.5957691216f * (z + 0.044715f * z * z * z));
        default: return z;
    }
}

template <bool kF16>
__device__ __forceinline__ float elem_f32(uint16_t v) {
    return kF16 ? __half2float(__ushort_as_half(v)) : bf16f(v);
}

template <bool kF16>
__device__ __forceinline__ uint16_t elem_from_f32(float v) {
    return kF16 ? __half_as_ushort(__float2half_rn(v)) : f32_to_bf16_rn(v);
}

// y[t][n] = v + residual[t][n] in the output's type (one rounding).
template <bool kF16, bool kOutF32>
__device__ __forceinline__ void store_output(const LinearArgs& a, long long t, int n, float v) {
    if (kOutF32) {
        if (a.residual) v += static_cast<const float*>(a.residual)[t * a.r_stride + n];
        static_cast<float*>(a.y)[t * a.y_stride + n] = v;
    } else {
        if (a.residual) v += elem_f32<kF16>(static_cast<const uint16_t*>(a.residual)[t * a.r_stride + n]);
        static_cast<uint16_t*>(a.y)[t * a.y_stride + n] = elem_from_f32<kF16>(v);
    }
}

__device__ __forceinline__ void mma_f16_16816(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                              uint32_t b0, uint32_t b1) {
    asm volatile(
        "mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0,%1,%2,%3}, {%4,%5,%6,%7}, {%8,%9}, "
        "{%0,%1,%2,%3};"
        : "+f"(c[0]), "+f"(c[1]), "+f"(c[2]), "+f"(c[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

#endif  // __CUDACC__

}  // namespace moe
