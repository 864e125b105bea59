// linear.cu -- y = act(x w^T + bias) + residual (moe_linear): the kernel for few tokens and the choice of
// kernel.
//
// linear_rows: a CTA owns 16 output features (16 rows of w; with SwiGLU the 16 gate and the 16 up rows)
// of 8 NT tokens.  Its eight warps take the 128-column slices of K in turn; each multiplies its slice with
// m16n8k16 products whose 16 rows are weight rows and whose 8 columns are tokens, straight from global
// memory: a sum over k does not depend on the order of k, so lane (g, q) of a quad reads the 8
// consecutive columns 8q .. 8q+7 of a 32-column piece of its rows (one 16-byte load) and uses them as the
// k indices the fragment layout gives it; the tokens' columns are read the same way.  The eight partial
// sums go through shared memory and are added in warp order.
#include "linear_common.cuh"

namespace moe {
namespace {

constexpr int kRowsWarps = 8;
constexpr int kRowsSlice = 128;   // columns of K a warp takes at a time

// Elements p[0..7] of a row of which `left` remain (zeros beyond); kVec: p is 16-byte aligned.
template <bool kVec>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int left) {
    if (kVec && left >= 8) return ld_nc_v4(p);
    uint32_t r[4] = {0u, 0u, 0u, 0u};
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < left) r[i / 2] |= (uint32_t)__ldg(p + i) << (16 * (i % 2));
    return make_uint4(r[0], r[1], r[2], r[3]);
}

template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if (kF16) mma_f16_16816(c, a0, a1, a2, a3, b0, b1);
    else mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
}

template <bool kF16, bool kOutF32, bool kGated, int NT, bool kVec>
__global__ void __launch_bounds__(32 * kRowsWarps) linear_rows(LinearArgs a) {
    constexpr int S = kGated ? 2 : 1, kTok = 8 * NT, kPitch = 17;
    __shared__ float red[kRowsWarps][S][kTok * kPitch];
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, g = lane >> 2, q = lane & 3;
    const int n0 = blockIdx.x * 16;
    const long long t0 = (long long)blockIdx.y * kTok;
    pdl_wait();
    pdl_launch_dependents();

    // rows and tokens beyond the end repeat the last one; their products are not stored
    const uint16_t* wp[S][2];
    const uint16_t* xp[NT];
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int h = 0; h < 2; ++h)
            wp[s][h] = static_cast<const uint16_t*>(a.w) + ((long long)s * a.N + min(n0 + g + 8 * h, a.N - 1)) * a.w_stride;
#pragma unroll
    for (int j = 0; j < NT; ++j) {
        const long long t = t0 + 8 * j + g;
        xp[j] = static_cast<const uint16_t*>(a.x) + (t < a.T ? t : a.T - 1) * a.x_stride;
    }
    float acc[S][NT][4] = {};
    for (int kc = warp * kRowsSlice; kc < a.K; kc += kRowsWarps * kRowsSlice) {
        uint4 wv[S][4][2];
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = kc + 32 * u + 8 * q;
#pragma unroll
            for (int s = 0; s < S; ++s)
#pragma unroll
                for (int h = 0; h < 2; ++h) wv[s][u][h] = load8<kVec>(wp[s][h] + k, a.K - k);
        }
#pragma unroll
        for (int u = 0; u < 4; ++u) {
            const int k = kc + 32 * u + 8 * q;
#pragma unroll
            for (int j = 0; j < NT; ++j) {
                const uint4 xv = load8<kVec>(xp[j] + k, a.K - k);
#pragma unroll
                for (int s = 0; s < S; ++s) {
                    const uint4 w0 = wv[s][u][0], w1 = wv[s][u][1];
                    mma16<kF16>(acc[s][j], w0.x, w1.x, w0.y, w1.y, xv.x, xv.y);
                    mma16<kF16>(acc[s][j], w0.z, w1.z, w0.w, w1.w, xv.z, xv.w);
                }
            }
        }
    }
#pragma unroll
    for (int s = 0; s < S; ++s)
#pragma unroll
        for (int j = 0; j < NT; ++j)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                red[warp][s][(8 * j + 2 * q + (i & 1)) * kPitch + g + 8 * (i >> 1)] = acc[s][j][i];
    __syncthreads();
    for (int i = threadIdx.x; i < 16 * kTok; i += 32 * kRowsWarps) {
        const int r = i % 16, n = n0 + r;
        const long long t = t0 + i / 16;
        if (n >= a.N || t >= a.T) continue;
        float z[S];
#pragma unroll
        for (int s = 0; s < S; ++s) {
            z[s] = 0.0f;
#pragma unroll
            for (int w = 0; w < kRowsWarps; ++w) z[s] += red[w][s][(i / 16) * kPitch + r];
            if (a.bias) z[s] += __ldg(a.bias + (long long)s * a.N + n);
        }
        const float v = kGated ? z[0] * sigmoid_f32<kOutF32>(z[0]) * z[S - 1] : apply_act<kOutF32>(a.act, z[0]);
        store_output<kF16, kOutF32>(a, t, n, v);
    }
}

template <bool kF16, bool kOutF32, bool kGated, bool kVec>
cudaError_t launch_rows_nt(const LinearArgs& a, cudaStream_t st) {
    const int nt = a.T <= 8 ? 1 : a.T <= 16 ? 2 : 4;
    const dim3 grid((a.N + 15) / 16, (a.T + 8 * nt - 1) / (8 * nt)), block(32 * kRowsWarps);
    if (nt == 1) return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 1, kVec>, grid, block, 0, st, a);
    if (nt == 2) return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 2, kVec>, grid, block, 0, st, a);
    return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 4, kVec>, grid, block, 0, st, a);
}

template <bool kF16, bool kOutF32>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t st) {
    const bool vec = a.x_stride % 8 == 0 && a.w_stride % 8 == 0;
    if (a.act == MOE_ACT_SWIGLU)
        return vec ? launch_rows_nt<kF16, kOutF32, true, true>(a, st) : launch_rows_nt<kF16, kOutF32, true, false>(a, st);
    return vec ? launch_rows_nt<kF16, kOutF32, false, true>(a, st) : launch_rows_nt<kF16, kOutF32, false, false>(a, st);
}

}  // namespace

// Operands whose rows do not start at multiples of 16 bytes are copied to rows that do, for the tensor-core
// kernels (TMA reads rows at such addresses only).
constexpr int kFewTokens = 32;   // at most this many: linear_rows

static bool straight(long long stride) { return stride % 8 == 0; }
static long long padded(int K) { return (K + 7) / 8 * 8; }

__global__ void __launch_bounds__(256) realign_rows(const uint16_t* __restrict__ src, long long src_stride, int K,
                                                    uint16_t* __restrict__ dst, long long dst_stride) {
    pdl_wait();
    pdl_launch_dependents();
    const uint16_t* s = src + (long long)blockIdx.x * src_stride;
    uint4* d = reinterpret_cast<uint4*>(dst + (long long)blockIdx.x * dst_stride);
    for (int c = threadIdx.x; c < (int)(dst_stride / 8); c += blockDim.x) d[c] = load8<false>(s + 8 * c, K - 8 * c);
}

size_t linear_workspace(const LinearArgs& a) {
    size_t n = 256;
    if (a.T > kFewTokens) {
        if (!straight(a.w_stride)) n += align_up((size_t)a.rows * padded(a.K) * 2, 256);
        if (!straight(a.x_stride)) n += align_up((size_t)a.T * padded(a.K) * 2, 256);
    }
    return n;
}

cudaError_t launch_linear(const LinearArgs& args, cudaStream_t st, unsigned long long* launches) {
    LinearArgs a = args;
    *launches += 1;
    if (a.T <= kFewTokens) {
        if (a.f16) return a.out_f32 ? launch_rows<true, true>(a, st) : launch_rows<true, false>(a, st);
        return a.out_f32 ? launch_rows<false, true>(a, st) : launch_rows<false, false>(a, st);
    }
    uint8_t* at = a.ws + 256;
    const long long stride = padded(a.K);
    if (!straight(a.w_stride)) {
        const cudaError_t e = launch_with_pdl(realign_rows, dim3(a.rows), dim3(256), 0, st, static_cast<const uint16_t*>(a.w),
                                              a.w_stride, a.K, reinterpret_cast<uint16_t*>(at), stride);
        if (e != cudaSuccess) return e;
        a.w = at;
        a.w_stride = stride;
        at += align_up((size_t)a.rows * stride * 2, 256);
        *launches += 1;
    }
    if (!straight(a.x_stride)) {
        const cudaError_t e = launch_with_pdl(realign_rows, dim3(a.T), dim3(256), 0, st, static_cast<const uint16_t*>(a.x),
                                              a.x_stride, a.K, reinterpret_cast<uint16_t*>(at), stride);
        if (e != cudaSuccess) return e;
        a.x = at;
        a.x_stride = stride;
        *launches += 1;
    }
    return launch_linear_tc(a, st);
}

}  // namespace moe
