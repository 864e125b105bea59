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
//
// Bound by the weights' way into the registers: few tokens leave no reuse, and a tile in shared memory would only add a
// copy and a barrier.  Measured: 1 x 2048 x 2048 in bf16 2.6 us = 3.2 TB/s, which is the launch and two loads' latency;
// 8 x 4096 x 2048 3.5 us = 4.8 TB/s (out of L2); fp32 outputs 1 x 256 x 2048 2.4 us, 1 x 2048 x 16384 10.0 us = 6.7 TB/s out of
// L2 and 20 us from HBM.
#include <type_traits>

#include "linear_common.cuh"

namespace moe {
namespace {

constexpr int kRowsWarps = 8;
constexpr int kRowsSlice = 128;   // columns of K a warp takes at a time
constexpr int kRowsChunk = 4;     // slices of a warp summed in the tensor cores' accumulator for fp32 outputs: 512 columns

// Elements p[0..7] of a row of which `left` remain (zeros beyond), from the aligned 4-byte words that hold them.
__device__ __forceinline__ uint4 load8_words(const uint16_t* p, int left) {
    const int odd = (int)(reinterpret_cast<uintptr_t>(p) >> 1) & 1;   // the row starts in the middle of a word
    const uint32_t* q = reinterpret_cast<const uint32_t*>(p - odd);
    uint32_t w[5];
#pragma unroll
    for (int u = 0; u < 5; ++u) {   // word u holds elements 2u - odd and 2u + 1 - odd (the one before p among them)
        w[u] = 0u;
        if (u < 4 || odd) {
            if (2 * u + 1 - odd < left) w[u] = __ldg(q + u);
            else if (2 * u - odd < left) w[u] = __ldg(reinterpret_cast<const uint16_t*>(q + u));   // the row's last element
        }
    }
    uint32_t o[4];
#pragma unroll
    for (int u = 0; u < 4; ++u) {
        o[u] = odd ? __funnelshift_r(w[u], w[u + 1], 16) : w[u];
        if (2 * u + 1 >= left) o[u] = 2 * u < left ? o[u] & 0xffffu : 0u;
    }
    return make_uint4(o[0], o[1], o[2], o[3]);
}

// The same for linear_rows.  kInside: 8 elements (16 without kVec) are known to remain, so that there is no branch and
// many loads go out together.  kVec: p is 16-byte aligned; else the two aligned 16-byte blocks that hold the elements are
// loaded and shifted together (in range: a row that does not start at such a block has the one before it in front of it).
template <bool kVec, bool kInside>
__device__ __forceinline__ uint4 load8(const uint16_t* p, int left) {
    if (!kInside) return load8_words(p, left);
    if (kVec) return ld_nc_v4(p);
    const uint32_t sh = (uint32_t)(reinterpret_cast<uintptr_t>(p) & 15u);   // bytes into the first block
    const char* base = reinterpret_cast<const char*>(p) - sh;
    const uint4 a = ld_nc_v4(base), b = ld_nc_v4(base + 16);
    uint32_t w[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
    if (sh & 8u) {
#pragma unroll
        for (int i = 0; i < 6; ++i) w[i] = w[i + 2];
    }
    if (sh & 4u) {
#pragma unroll
        for (int i = 0; i < 5; ++i) w[i] = w[i + 1];
    }
    const uint32_t bits = (sh & 2u) * 8u;
    return make_uint4(__funnelshift_r(w[0], w[1], bits), __funnelshift_r(w[1], w[2], bits), __funnelshift_r(w[2], w[3], bits),
                      __funnelshift_r(w[3], w[4], bits));
}

template <bool kF16>
__device__ __forceinline__ void mma16(float (&c)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                      uint32_t b1) {
    if (kF16) mma_f16_16816(c, a0, a1, a2, a3, b0, b1);
    else mma_bf16_16816(c, a0, a1, a2, a3, b0, b1);
}

// kLong: fp32 outputs of rows of which a warp has more than a chunk: a chunk's sums leave the accumulator and are added in
// ordinary fp32 (see linear_tc.cuh).  A form of its own, as its loop costs the others registers (1 x 4096 x 2048: 3.95 against
// 3.2 us, fewer CTAs of two launches side by side on an SM).
template <bool kF16, bool kOutF32, bool kGated, int NT, bool kVec, bool kLong>
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
    // the loads of 128 columns go out together, of 64 where each takes two (registers)
    constexpr int kAtOnce = kVec ? 4 : 2;
    const auto slice = [&](int kc, auto inside) {
        constexpr bool kInside = decltype(inside)::value;
#pragma unroll
        for (int u0 = 0; u0 < 4; u0 += kAtOnce) {
            uint4 wv[S][kAtOnce][2];
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int k = kc + 32 * (u0 + u) + 8 * q;
#pragma unroll
                for (int s = 0; s < S; ++s)
#pragma unroll
                    for (int h = 0; h < 2; ++h) wv[s][u][h] = load8<kVec, kInside>(wp[s][h] + k, a.K - k);
            }
#pragma unroll
            for (int u = 0; u < kAtOnce; ++u) {
                const int k = kc + 32 * (u0 + u) + 8 * q;
#pragma unroll
                for (int j = 0; j < NT; ++j) {
                    const uint4 xv = load8<kVec, kInside>(xp[j] + k, a.K - k);
#pragma unroll
                    for (int s = 0; s < S; ++s) {
                        const uint4 w0 = wv[s][u][0], w1 = wv[s][u][1];
                        mma16<kF16>(acc[s][j], w0.x, w1.x, w0.y, w1.y, xv.x, xv.y);
                        mma16<kF16>(acc[s][j], w0.z, w1.z, w0.w, w1.w, xv.z, xv.w);
                    }
                }
            }
        }
    };
    int kc = warp * kRowsSlice;
    for (bool first = true;; first = false) {
        const int end = kLong ? min(a.K, kc + kRowsChunk * kRowsWarps * kRowsSlice) : a.K;
        for (; kc < end; kc += kRowsWarps * kRowsSlice) {
            if (kc + kRowsSlice + (kVec ? 0 : 8) <= a.K) slice(kc, std::true_type{});
            else slice(kc, std::false_type{});
        }
        // the warp's sums, to where they meet the other warps' (a place is one thread's until the barrier)
#pragma unroll
        for (int s = 0; s < S; ++s)
#pragma unroll
            for (int j = 0; j < NT; ++j)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    float& r = red[warp][s][(8 * j + 2 * q + (i & 1)) * kPitch + g + 8 * (i >> 1)];
                    r = !kLong || first ? acc[s][j][i] : r + acc[s][j][i];
                    if (kLong) acc[s][j][i] = 0.0f;
                }
        if (!kLong || kc >= a.K) break;
    }
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
    if constexpr (kOutF32) {
        if (a.K > kRowsChunk * kRowsWarps * kRowsSlice) {
            if (nt == 1) return launch_with_pdl(linear_rows<kF16, true, kGated, 1, kVec, true>, grid, block, 0, st, a);
            return launch_with_pdl(linear_rows<kF16, true, kGated, 2, kVec, true>, grid, block, 0, st, a);
        }
    }
    if (nt == 1) return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 1, kVec, false>, grid, block, 0, st, a);
    return launch_with_pdl(linear_rows<kF16, kOutF32, kGated, 2, kVec, false>, grid, block, 0, st, a);
}

template <bool kF16, bool kOutF32>
cudaError_t launch_rows(const LinearArgs& a, cudaStream_t st) {
    const bool vec = a.x_stride % 8 == 0 && a.w_stride % 8 == 0;
    if (a.act == MOE_ACT_SWIGLU)
        return vec ? launch_rows_nt<kF16, kOutF32, true, true>(a, st) : launch_rows_nt<kF16, kOutF32, true, false>(a, st);
    return vec ? launch_rows_nt<kF16, kOutF32, false, true>(a, st) : launch_rows_nt<kF16, kOutF32, false, false>(a, st);
}

}  // namespace

// Which kernel and tile: the least of an estimate in microseconds, fitted to runs of every form on products of
// 1..4096 tokens (of 86 sizes 68 take at most 1.05 times the best form's time, 81 at most 1.25, one 2.0).  Per tile a CTA, or a pair, needs the longer of its K loop
// and its epilogue, as the two overlap; the launch, the last epilogue and joining slices come once.
// Clusters of a size that run at a time with one CTA to an SM, as the device reports it: 152 SMs hold 76 of 2, 36
// of 4 and 15 of 8.  For the estimate only: more of them take turns.
static int clusters_at_once(int size, int num_sms) {
    return size == 1 ? num_sms : size == 2 ? num_sms / 2 : size == 4 ? num_sms * 36 / 152 : num_sms * 15 / 152;
}

LinearPlan linear_plan(const LinearArgs& l) {
    const bool gated = l.act == MOE_ACT_SWIGLU, res = l.residual != nullptr;
    // what the activation adds to the epilogue of a tile, in units of silu's (about 6 ns a token of 128 features)
    const double act = l.act == MOE_ACT_SILU || l.act == MOE_ACT_GELU_TANH ? 1.0 : l.act == MOE_ACT_GELU ? 2.0 : 0.0;
    const int nkb = (l.K + kLK - 1) / kLK, G = gated ? 2 : 1;
    const double kLaunch = 1.4, kL2 = 17e6;                        // us; bytes a us that L2 gives all SMs together
    const double kLoop[5] = {0.142, 0.155, 0.19, 0.215, 0.30};     // us of 64 columns for 16, 32, .. 256 tokens
    const double kLoopGated[4] = {0.26, 0.28, 0.34, 0.41};
    LinearPlan best{false, 0, 1, 1e300};
    const auto consider = [&](bool pair, int tt, int s, int sub, double tiles, double slots, double block_us,
                              double block_bytes, double epilogue, double once) {
        const double waves = s > 1 ? 1 : (double)(((long long)tiles + (long long)slots - 1) / (long long)slots);
        const double busy = tiles * s < slots ? tiles * s : slots, shared = block_bytes * busy / kL2;
        // few weight rows: every CTA asks the same few L2 slices for them
        if (!pair && l.rows < kLM) block_us += 0.003 * busy * (1.0 - (double)l.rows / kLM);
        const int stages = (nkb + sub - 1) / sub;
        const double loop = (double)((stages + s - 1) / s) * sub * (block_us > shared ? block_us : shared);
        const double us = kLaunch + once + waves * (loop > epilogue ? loop : epilogue) + epilogue;
        if (us < best.us) best = LinearPlan{pair, tt, s, us};
    };
    const int most = l.out_f32 ? (gated ? 64 : 128) : (gated ? 128 : 256);
    for (int tt = 16, i = 0; tt <= most; tt *= 2, ++i) {
        const double tiles = (double)((l.N + kLM - 1) / kLM) * ((l.T + tt - 1) / tt);
        const int bytes = (G * kLM + tt) * 128, sub = feat_sub(bytes);
        const double epilogue = (gated ? 0.75 + 0.0145 * tt + (res ? 0.004 * tt : 0.0)
                                       : 0.5 + 0.0068 * tt + act * (0.15 + 0.006 * tt) + (res ? 0.1 + 0.004 * tt : 0.0)) *
                                (l.out_f32 ? tt == 128 ? 1.5 : 1.17 : 1.0);
        for (int s = 1; s <= 8; s *= 2) {
            if (s > 1 && (tiles > clusters_at_once(s, l.num_sms) || (nkb + sub - 1) / sub < s || tt / s < 4 || G * tt > 128))
                break;
            consider(false, tt, s, sub, tiles, l.num_sms, gated ? kLoopGated[i] : kLoop[i], bytes, epilogue,
                     s > 1 ? 1.7 + 0.010 * tt * G : 0.0);
        }
        if (tt >= l.T) break;
    }
    if (l.T > kLM) {
        const int tn = l.out_f32 ? 128 : 256;
        const double tiles = (double)((l.T + 2 * kLM - 1) / (2 * kLM)) * ((l.rows + tn - 1) / tn);
        // rows of y or the residual at other than multiples of 16 bytes: element stores and loads
        const int size = l.out_f32 ? 4 : 2;
        const double slow = (res && l.r_stride * size % 16 ? 20.0 : 0.0) + (l.y_stride * size % 16 ? 2.0 : 0.0);
        consider(true, 0, 1, 1, tiles, l.num_sms / 2, tn == 256 ? 0.32 : 0.25, (2 * kLM + tn) * 128,
                 2.6 + 2.2 * act + (res ? (l.out_f32 ? 3.0 : 1.6) : 0.0) + slow, 0.0);
    }
    return best;
}

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

// A thread writes 16 bytes.  Bound by latency at the sizes where it matters: 333 x 777 x 1001 takes 8.8-9.0 us with it and
// 6.3 where the rows are aligned.
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
    const int row = (int)(i / pieces), c = 8 * (int)(i - (long long)row * pieces);
    reinterpret_cast<uint4*>(r.dst)[i] = load8_words(r.src + row * r.src_stride + c, K - c);
}

// Whether linear_rows does it: few tokens, and not longer than the tensor-core kernels would take.  Its time,
// fitted like theirs: an iteration of its eight warps covers 1024 columns of K and is a load's latency; large
// weights stream from HBM, which the tensor-core kernels do at the full rate.
bool linear_takes_rows(const LinearArgs& a) {
    if (a.T > kFewTokens) return false;
    // on 152 SMs whatever the device at hand: the workspace's size, asked for anywhere, rests on this
    LinearArgs nominal = a;
    nominal.num_sms = 152;
    const double bytes = 2.0 * a.rows * a.K, iterations = (a.K + 1023) / 1024;
    const bool vec = straight(a.w_stride) && straight(a.x_stride);
    const double waves = (a.N + 15) / 16 / 456.0;   // of CTAs, three to an SM
    double step = a.T <= 8 ? 0.68 : 1.3, rate = a.T <= 8 ? 6.4e6 / (1 + 0.015 * a.T) : 4.1e6;
    if (!vec) {   // two loads and shifts for one
        step *= a.T <= 8 ? 2.1 : 1.6;
        rate /= 1.4;
    }
    double wave = iterations * step;
    if (a.K < 1024) wave = step * (0.6 + 0.4 * a.K / 1024);
    const double least = a.act == MOE_ACT_SWIGLU ? 2.3 : 1.15;   // of a wave among others
    const double steps = waves > 1.0 ? waves * (wave > least ? wave : least) : wave;
    const double rows_us = 1.5 + (steps > bytes / rate ? steps : bytes / rate);
    const double stream = bytes > 100e6 ? 1.4 + bytes / 6.7e6 : 0.0, loop = linear_plan(nominal).us;   // past L2: HBM's rate
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
    return a.f16 ? launch_linear_tc_f16(a, st) : launch_linear_tc_bf16(a, st);
}

}  // namespace moe
