// linear_common.cuh -- what the kernels of moe_linear share: element types, the epilogue's activation
// functions and the store of one output.
#pragma once

#include <cuda_bf16.h>
#include <cuda_fp16.h>

#include "moe_internal.cuh"

namespace moe {

constexpr int kLK = 64;                 // columns of K per block: one 128-byte swizzle row
constexpr int kLM = 128;                // M of a CTA: token rows (linear_pair) or weight rows (linear_feat)
// Blocks of 64 columns to a stage of the ring.  Waiting for a stage, issuing its products and releasing it cost
// the issuer and the producer about 0.1 us whatever its size, so small blocks share a stage (one weight tile of
// 2048 columns: 8.7 us with one block of 16 tokens to a stage, 6.9 with two, 6.1 with four; of 128 tokens 10.6
// and 9.3 with two).
__host__ __device__ constexpr int feat_sub(int block) { return block <= 20480 ? 4 : block <= 36864 ? 2 : 1; }

// How the tensor cores do a product (linear.cu): by linear_pair, or by linear_feat with tt tokens to a tile and K in
// slices; us: the time expected.
struct LinearPlan {
    bool pair;
    int tt, slices;
    double us;
};
LinearPlan linear_plan(const LinearArgs& l);
cudaError_t launch_linear_tc_bf16(const LinearArgs& l, cudaStream_t st);   // rows at multiples of 16 bytes
cudaError_t launch_linear_tc_f16(const LinearArgs& l, cudaStream_t st);

#ifdef __CUDACC__

// act(z) in fp32.  kExact (fp32 outputs): the exponential is good to a few 2^-23.  Else the result is rounded
// to bf16 or fp16 (8 or 11 bits), and the exponential is the hardware one: its relative error, a few 2^-23 and
// another 2^-24 |z|, disappears in that rounding.
template <bool kExact>
__device__ __forceinline__ float sigmoid_f32(float z) {
    return __fdividef(1.0f, 1.0f + (kExact ? exp_f32(fminf(fmaxf(-z, -88.0f), 88.0f)) : __expf(-z)));
}

// z Phi(z).  The upper tail of |z| is 0.5 exp(-z^2 / 2) times the scaled complementary error function, for which
// a polynomial in t = 1 / (1 + 0.43 x), x = |z| / sqrt 2, was fitted here in 64 bits by least squares of the
// relative error (1e-7 for x up to 9.3; 4e-7 with its terms in fp32), so that small values keep their digits.
// Beyond |z| of about 13.2 the exponential is below 2^-126 and comes out as 0, from 20 on in either form: z is held there for
// its argument only, so that z times the tail is 0 however large z is.
template <bool kExact>
__device__ __forceinline__ float gelu_f32(float z) {
    const float x = fminf(fabsf(z), 20.0f), t = __fdividef(1.0f, fmaf(0.43f * 0.70710678f, x, 1.0f));
    float p = 0.0737080984f;
    p = fmaf(p, t, -0.310374153f);
    p = fmaf(p, t, 0.383707111f);
    p = fmaf(p, t, -0.0857271134f);
    p = fmaf(p, t, 0.246845185f);
    p = fmaf(p, t, 0.20495087f);
    p = fmaf(p, t, 0.244375479f);
    p = fmaf(p, t, 0.242514606f);
    const float s = -0.5f * x * x, q = 0.5f * t * p * (kExact ? exp_f32(s) : __expf(s));
    return z * (z < 0.0f ? q : 1.0f - q);
}

template <bool kExact>
__device__ __forceinline__ float apply_act(int act, float z) {
    switch (act) {
        case MOE_ACT_RELU: return z < 0.0f ? 0.0f : z;   // a NaN stays one
        case MOE_ACT_SILU: return z * sigmoid_f32<kExact>(z);
        case MOE_ACT_GELU: return gelu_f32<kExact>(z);
        // tanh form: 0.5 z (1 + tanh u) = z / (1 + exp(-2u)), u = sqrt(2/pi) (z + 0.044715 z^3)
        case MOE_ACT_GELU_TANH: return z * sigmoid_f32<kExact>(1.5957691216f * (z + 0.044715f * z * z * z));
        default: return z;
    }
}

// The same for an array, the choice taken once (unrolled around a switch for each element the code outgrows the
// instruction cache).
template <bool kExact, int kCnt>
__device__ __forceinline__ void apply_act_all(int act, float (&v)[kCnt]) {
    const auto all = [&](auto one) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) v[j] = one(v[j]);
    };
    if (act == MOE_ACT_NONE) return;
    if (act == MOE_ACT_RELU) all([](float z) { return apply_act<kExact>(MOE_ACT_RELU, z); });
    else if (act == MOE_ACT_SILU) all([](float z) { return apply_act<kExact>(MOE_ACT_SILU, z); });
    else if (act == MOE_ACT_GELU) all([](float z) { return apply_act<kExact>(MOE_ACT_GELU, z); });
    else all([](float z) { return apply_act<kExact>(MOE_ACT_GELU_TANH, z); });
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
