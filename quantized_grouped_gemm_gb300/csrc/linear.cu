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
    const int nt = a.T <= 8 ? 1 : 2;
    const dim3 grid((a.N + 15) / 16, (a.T + 8 * nt - 1) / (8 * nt)), block(32 * kRowsWarps);
    if (nt == 1) return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 1, kVec>, grid, block, 0, st, a);
    return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 2, kVec>, grid, block, 0, st, a);
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
constexpr int kFewTokens = 16;   // at most this many: linear_rows may be taken

static bool straight(long long stride) { return stride % 8 == 0; }
static long long padded(int K) { return (K + 7) / 8 * 8; }

// One operand to copy: rows of K elements from any element address to rows at multiples of 16 bytes, zeros beyond K.
struct Realign {
    const uint16_t* src;
    uint16_t* dst;
    long long src_stride;
    int rows;
};

// A thread writes 16 bytes, from five 4-byte words where the row starts in the middle of one (else four).
__global__ void __launch_bounds__(256) realign_rows(Realign r0, Realign r1, int K, int pieces) {
    pdl_wait();
    pdl_launch_dependents();
    long long i = (long long)blockIdx.x * blockDim.x + threadIdx.x;
    const long long n0 = (long long)r0.rows * pieces;
    Realign r = r0;
    if (i >= n0) {
        i -= n0;
        r = r1;
        if (i >= (long long)r.rows * pieces) return;
    }
    const int row = (int)(i / pieces), c = 8 * (int)(i - (long long)row * pieces), left = K - c;   // elements left
    const uint16_t* p = r.src + row * r.src_stride + c;
    const bool odd = reinterpret_cast<uintptr_t>(p) & 2;
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - (odd ? 1 : 0));   // aligned words
    uint32_t w[5];
#pragma unroll
    for (int u = 0; u < 5; ++u) w[u] = 2 * u - (odd ? 1 : 0) < left && (u < 4 || odd) ? __ldg(q + u) : 0u;
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        o[u] = odd ? __funnelshift_r(w[u], w[u + 1], 16) : w[u];
        if (2 * u + 1 >= left) o[u] = 2 * u < left ? o[u] & 0xffffu : 0u;
    }
    reinterpret_cast<uint4*>(r.dst)[i] = make_uint4(o[0], o[1], o[2], o[3]);
}

// Whether linear_rows does it: few tokens, and not longer than the tensor-core kernels would take.  Its time,
// fitted like theirs: an iteration of its eight warps covers 1024 columns of K and is a load's latency; large
// weights stream from HBM, which the tensor-core kernels do at the full rate.
bool linear_takes_rows(const LinearArgs& a) {
    if (a.T > kFewTokens) return false;
    const double bytes = 2.0 * a.rows * a.K, iterations = (a.K + 1023) / 1024;
    const bool vec = straight(a.w_stride) && straight(a.x_stride);
    const double step = (a.T <= 8 ? 0.9 : 1.65) * (vec ? 1.0 : 1.6);
    const double rate = (a.T <= 8 ? 6.4e6 / (1 + 0.015 * a.T) : 4.1e6) / (vec ? 1.0 : 1.8);   // element loads
    const double rows_us = 1.9 + (iterations * step > bytes / rate ? iterations * step : bytes / rate);
    const double stream = bytes > 100e6 ? 1.4 + bytes / 6.7e6 : 0.0, loop = linear_tc_us(a);   // past L2: HBM's rate
    const double copy = straight(a.w_stride) ? straight(a.x_stride) ? 0.0 : 2.0 : 2.0 + bytes / 3e6;
    return rows_us <= copy + (loop > stream ? loop : stream);
}

size_t linear_workspace(const LinearArgs& a) {
    size_t n = 256;
    if (!a.few) {
        if (!straight(a.w_stride)) n += align_up((size_t)a.rows * padded(a.K) * 2, 256);
        if (!straight(a.x_stride)) n += align_up((size_t)a.T * padded(a.K) * 2, 256);
    }
    return n;
}

cudaError_t launch_linear(const LinearArgs& args, cudaStream_t st, unsigned long long* launches) {
    LinearArgs a = args;
    *launches += 1;
    if (a.few) {
        if (a.f16) return a.out_f32 ? launch_rows<true, true>(a, st) : launch_rows<true, false>(a, st);
        return a.out_f32 ? launch_rows<false, true>(a, st) : launch_rows<false, false>(a, st);
    }
    const bool copy_w = !straight(a.w_stride), copy_x = !straight(a.x_stride);
    if (copy_w || copy_x) {
        const long long stride = padded(a.K);
        uint8_t* at = a.ws + 256;
        Realign r[2] = {};
        if (copy_w) {
            r[0] = Realign{static_cast<const uint16_t*>(a.w), reinterpret_cast<uint16_t*>(at), a.w_stride, a.rows};
            a.w = at;
            a.w_stride = stride;
            at += align_up((size_t)a.rows * stride * 2, 256);
        }
        if (copy_x) {
            r[1] = Realign{static_cast<const uint16_t*>(a.x), reinterpret_cast<uint16_t*>(at), a.x_stride, a.T};
            a.x = at;
            a.x_stride = stride;
        }
        const int pieces = (int)(stride / 8);
        const long long threads = ((long long)r[0].rows + r[1].rows) * pieces;
        const cudaError_t e = launch_with_pdl(realign_rows, dim3((unsigned)((threads + 255) / 256)), dim3(256), 0, st, r[0],
                                              r[1], a.K, pieces);
        if (e != cudaSuccess) return e;
        *launches += 1;
    }
    return launch_linear_tc(a, st);
}

}  // namespace moe
