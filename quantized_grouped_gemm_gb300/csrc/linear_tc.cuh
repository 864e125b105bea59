// linear_tc.cuh -- moe_linear on the 5th-generation tensor cores (more than a few tokens).
//
// Operands are K-major and come in by TMA as 64-column blocks with the 128-byte swizzle (TMA fills what lies
// beyond T, N or K with zeros); the fp32 accumulators are in TMEM.
//
//   linear_pair   large products.  D[token][feature]: two CTAs (a cluster) share one 256-token x kTN-row tile,
//                 each holds 128 tokens' rows and half of the weight rows, so a byte of shared memory feeds
//                 twice the products of a single-CTA tile.  Persistent; while the epilogue empties one
//                 accumulator the next tile's products go into another.
//   linear_feat   few tokens, or few tiles.  D[feature][token]: a tile is 128 features x 16..256 tokens of one
//                 CTA.  Persistent over the tiles where they are many (a stream of the weights); where they are
//                 few, the 2..8 CTAs of a cluster take slices of K of one tile and add their fp32 partial sums
//                 through distributed shared memory, in slice order, so that a small product uses most SMs.
//
// The tensor cores truncate when they add to the accumulator (about half a unit of 2^-23 of the running sum at each
// 16-column step, always towards zero), so after chunk_blocks blocks the partial sum leaves it and the next is added in
// ordinary fp32.  fp32 outputs: every 512 columns (384 with SwiGLU), the sums held in registers.  16-bit outputs: every 8192
// (measured: 9e-6 of sums of products of either sign; where all have one sign 3e-5 in bf16 and 5e-5 in fp16, whose half unit
// is 2.4e-4 at least), the sums held in the other accumulator, which costs the issuer a wait at each of these.
#include <atomic>
#include <type_traits>

#include "linear_common.cuh"

namespace moe {
namespace {

// Blocks summed in the accumulator.  fp32 outputs: the relative error is 4.7e-7 (bf16) or 6.5e-7 (fp16) after 8, up to 3e-6
// where all products have one sign (in each of two factors with SwiGLU, so 6 there); it grows with their number.
__host__ __device__ constexpr int chunk_blocks(bool out_f32, bool gated) { return !out_f32 ? 128 : gated ? 6 : 8; }
// Threads: four warps (producer, issuer, TMEM, spare) and `groups` warpgroups of the epilogue, each with its share of
// a tile's columns.  Four groups where the tile is wide: short K loops leave the time to the epilogue.
__host__ __device__ constexpr int tc_threads(int groups) { return 128 * (1 + groups); }

constexpr int kPairMaxStages = 6;
constexpr int kStageBuf = 128 * 128;    // a warpgroup's output staging: 128 rows of 128 bytes

struct PairSmem {
    uint64_t full[kPairMaxStages], empty[kPairMaxStages];
    uint64_t acc_full[4], acc_empty[4];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ uint32_t map_to_rank(const void* p, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(smem_u32(p)), "r"(rank));
    return r;
}

// TMA load whose bytes are counted on a barrier of either CTA of the pair (bar: a shared::cluster address).
__device__ __forceinline__ void tma_load_2d_pair(void* dst, const CUtensorMap* map, int c0, int c1, uint32_t bar) {
    asm volatile(
        "cp.async.bulk.tensor.2d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, "
        "%3}], [%4];" ::"r"(smem_u32(dst)),
        "l"(reinterpret_cast<uint64_t>(map)), "r"(c0), "r"(c1), "r"(bar)
        : "memory");
}

__device__ __forceinline__ void tma_store_2d(const CUtensorMap* map, const void* src, int c0, int c1) {
    asm volatile("cp.async.bulk.tensor.2d.global.shared::cta.bulk_group [%0, {%1, %2}], [%3];" ::"l"(
                     reinterpret_cast<uint64_t>(map)),
                 "r"(c0), "r"(c1), "r"(smem_u32(src))
                 : "memory");
}
__device__ __forceinline__ void bulk_commit() { asm volatile("cp.async.bulk.commit_group;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_read() { asm volatile("cp.async.bulk.wait_group.read 0;" ::: "memory"); }
__device__ __forceinline__ void bulk_wait_all() { asm volatile("cp.async.bulk.wait_group 0;" ::: "memory"); }

template <bool kPair>
__device__ __forceinline__ void tc_mma_f16kind(uint32_t d, uint64_t ad, uint64_t bd, uint32_t idesc, uint32_t acc) {
    if (kPair)
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "setp.ne.b32 p, %4, 0;\n\t"
            "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}" ::"r"(d),
            "l"(ad), "l"(bd), "r"(idesc), "r"(acc)
            : "memory");
    else
        tc_mma_bf16(d, ad, bd, idesc, acc);
}

// Arrive on the barrier at this offset in both CTAs of the pair once the MMAs issued so far are done.
__device__ __forceinline__ void tc_commit_pair(uint64_t* bar) {
    asm volatile(
        "tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;" ::"r"(
            smem_u32(bar)),
        "h"((uint16_t)3)
        : "memory");
}

// 16-bit operands of one type (bf16 or fp16), fp32 accumulator, both K-major.
__device__ __forceinline__ uint32_t idesc_f16kind(bool f16, int M, int N) {
    return f16 ? idesc_bf16_f32(M, N) & ~((1u << 7) | (1u << 10)) : idesc_bf16_f32(M, N);
}

__device__ __forceinline__ void tmem_ld32(uint32_t taddr, uint32_t (&r)[32]) {
    asm volatile(
        "tcgen05.ld.sync.aligned.32x32b.x32.b32 {%0,%1,%2,%3,%4,%5,%6,%7,%8,%9,%10,%11,%12,%13,%14,%15,%16,%17,%18,"
        "%19,%20,%21,%22,%23,%24,%25,%26,%27,%28,%29,%30,%31}, [%32];"
        : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7]), "=r"(r[8]),
          "=r"(r[9]), "=r"(r[10]), "=r"(r[11]), "=r"(r[12]), "=r"(r[13]), "=r"(r[14]), "=r"(r[15]), "=r"(r[16]),
          "=r"(r[17]), "=r"(r[18]), "=r"(r[19]), "=r"(r[20]), "=r"(r[21]), "=r"(r[22]), "=r"(r[23]), "=r"(r[24]),
          "=r"(r[25]), "=r"(r[26]), "=r"(r[27]), "=r"(r[28]), "=r"(r[29]), "=r"(r[30]), "=r"(r[31])
        : "r"(taddr));
}

// One 16-byte piece of the swizzled staging row r (128 bytes, eight pieces).
__device__ __forceinline__ uint4* stage_piece(uint8_t* buf, int r, int piece) {
    return reinterpret_cast<uint4*>(buf + r * 128 + ((piece ^ (r & 7)) << 4));
}

template <int kCols>
__device__ __forceinline__ void tmem_ld_cols(uint32_t taddr, uint32_t (&r)[kCols]) {   // the wait is the caller's
    static_assert(kCols == 8 || kCols == 16 || kCols == 32, "columns of a TMEM load");
    if constexpr (kCols == 8)
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(taddr));
    else if constexpr (kCols == 16) tmem_ld16(taddr, r);
    else tmem_ld32(taddr, r);
}
__device__ __forceinline__ void tmem_st8(uint32_t taddr, const float* r) {
    asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};" ::"r"(taddr),
                 "f"(r[0]), "f"(r[1]), "f"(r[2]), "f"(r[3]), "f"(r[4]), "f"(r[5]), "f"(r[6]), "f"(r[7])
                 : "memory");
}

// fp32 outputs in several chunks: adds this chunk's kCols columns (of each of G accumulators, kNext columns apart)
// to the running sums; after the last chunk the sums go back to TMEM, where the epilogue finds the products of
// one-chunk tiles too.
template <int G, int kCols, int kNext>
__device__ __forceinline__ void add_chunk(uint32_t acc, float (&sum)[G * kCols], bool first, bool last) {
    constexpr int kB = kCols < 32 ? kCols : 32;
#pragma unroll
    for (int g = 0; g < G; ++g)
#pragma unroll
        for (int j = 0; j < kCols; j += kB) {
            uint32_t q[kB];
            tmem_ld_cols<kB>(acc + g * kNext + j, q);
            tmem_ld_wait();
#pragma unroll
            for (int u = 0; u < kB; ++u)
                sum[g * kCols + j + u] = first ? __uint_as_float(q[u]) : sum[g * kCols + j + u] + __uint_as_float(q[u]);
        }
    if (last) {
#pragma unroll
        for (int g = 0; g < G; ++g)
#pragma unroll
            for (int j = 0; j < kCols; j += 8) tmem_st8(acc + g * kNext + j, &sum[g * kCols + j]);
        tmem_st_wait();
    }
}

// 16-bit outputs in several chunks: adds the sums so far, kCols columns (of each of G accumulators, kNext columns apart) at
// `from`, to the chunk at `acc`.
template <int G, int kCols, int kNext>
__device__ __forceinline__ void add_sums(uint32_t from, uint32_t acc) {
    constexpr int kB = kCols < 32 ? kCols : 32;
#pragma unroll 1
    for (int j = 0; j < G * kCols; j += kB) {
        const int at = j < kCols ? j : j - kCols + kNext;
        uint32_t p[kB], q[kB];
        tmem_ld_cols<kB>(from + at, p);
        tmem_ld_cols<kB>(acc + at, q);
        tmem_ld_wait();
        float v[kB];
#pragma unroll
        for (int u = 0; u < kB; ++u) v[u] = __uint_as_float(p[u]) + __uint_as_float(q[u]);
#pragma unroll
        for (int u = 0; u < kB; u += 8) tmem_st8(acc + at + u, &v[u]);
    }
    tmem_st_wait();
}

struct TcArgs {
    LinearArgs l;
    int tiles_m, tiles_n, nkb;
    bool y_tma;        // y rows start at multiples of 16 bytes: stores by TMA
    bool r_vec;        // residual rows too: 16-byte loads
};

// Which tile: bands of kBand token tiles, token tile innermost, so the tiles in flight at one time share
// both their x and their w rows in L2.
constexpr int kBand = 8;
__device__ __forceinline__ void tile_at(int i, int tiles_m, int tiles_n, int* m, int* n) {
    const int band = i / (kBand * tiles_n), first = band * kBand;
    const int h = min(kBand, tiles_m - first), j = i - band * kBand * tiles_n;
    *m = first + j % h;
    *n = j / h;
}

// The residual of 32 outputs (features n0.. of token t; `valid` of them exist) as stored, zeros beyond.
template <bool kOutF32>
struct Residual32 {
    uint4 q[kOutF32 ? 8 : 4];
};
template <bool kOutF32>
__device__ __forceinline__ void load_residual32(const TcArgs& a, long long t, int n0, int valid, Residual32<kOutF32>& r) {
    constexpr int kVecs = kOutF32 ? 8 : 4, kPer = kOutF32 ? 4 : 8;
    using Elem = typename std::conditional<kOutF32, uint32_t, uint16_t>::type;
    const Elem* p = static_cast<const Elem*>(a.l.residual) + t * a.l.r_stride + n0;
    if (a.r_vec && valid == 32) {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) r.q[i] = *reinterpret_cast<const uint4*>(p + kPer * i);
    } else {
#pragma unroll
        for (int i = 0; i < kVecs; ++i) {
            uint32_t w[4] = {0u, 0u, 0u, 0u};
#pragma unroll
            for (int j = 0; j < kPer; ++j)
                if (kPer * i + j < valid) w[j * 4 / kPer] |= (uint32_t)p[kPer * i + j] << (kOutF32 ? 0 : 16 * (j % 2));
            r.q[i] = make_uint4(w[0], w[1], w[2], w[3]);
        }
    }
}
template <bool kF16, bool kOutF32>
__device__ __forceinline__ void add_residual32(const Residual32<kOutF32>& r, float (&v)[32]) {
#pragma unroll
    for (int i = 0; i < (kOutF32 ? 8 : 4); ++i) {
        const uint32_t u[4] = {r.q[i].x, r.q[i].y, r.q[i].z, r.q[i].w};
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            if (kOutF32) {
                v[(4 * i + j) % 32] += __uint_as_float(u[j]);
            } else {
                v[(8 * i + 2 * j) % 32] += elem_f32<kF16>((uint16_t)(u[j] & 0xffffu));
                v[(8 * i + 2 * j + 1) % 32] += elem_f32<kF16>((uint16_t)(u[j] >> 16));
            }
        }
    }
}

template <bool kF16>
__device__ __forceinline__ uint32_t pack2(float lo, float hi) {
    uint32_t r;
    if (kF16) asm("cvt.rn.f16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    else asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(r) : "f"(hi), "f"(lo));
    return r;
}

template <bool kOutF32>
using OutElem = typename std::conditional<kOutF32, float, uint16_t>::type;

// The residual of one feature n of kCnt consecutive tokens from t0, as stored (0 beyond the last token).
template <bool kOutF32, int kCnt>
__device__ __forceinline__ void load_residual(const LinearArgs& l, long long t0, int n, OutElem<kOutF32> (&r)[kCnt]) {
    using Elem = OutElem<kOutF32>;
    const char* row = static_cast<const char*>(l.residual) + t0 * l.r_stride * (long long)sizeof(Elem);   // uniform
    const uint32_t off = n * (uint32_t)sizeof(Elem);
    const bool in = n < l.N;
    if (t0 + kCnt <= l.T) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) {
            r[j] = in ? *reinterpret_cast<const Elem*>(row + off) : (Elem)0;
            row += l.r_stride * (long long)sizeof(Elem);
        }
    } else {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) {
            r[j] = in && t0 + j < l.T ? *reinterpret_cast<const Elem*>(row + off) : (Elem)0;
            row += l.r_stride * (long long)sizeof(Elem);
        }
    }
}

// Bias, activation, residual (r, as stored) and store of one feature n < N of kCnt consecutive tokens from t0 (z:
// products, u: the up projection's).
template <bool kF16, bool kOutF32, bool kGated, int kCnt, int kUp>
__device__ __forceinline__ void finish_column(const LinearArgs& l, long long t0, int n, float b0, float b1,
                                              float (&z)[kCnt], const float (&u)[kUp], const OutElem<kOutF32> (&r)[kCnt]) {
    using Elem = OutElem<kOutF32>;
    if (l.bias) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) z[j] += b0;
    }
    if (kGated) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) z[j] = z[j] * sigmoid_f32<kOutF32>(z[j]) * (u[kGated ? j : 0] + b1);
    } else {
        apply_act_all<kOutF32>(l.act, z);
    }
    if (l.residual) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) {
            if constexpr (kOutF32) z[j] += r[j];
            else z[j] += elem_f32<kF16>(r[j]);
        }
    }
    char* row = static_cast<char*>(l.y) + t0 * l.y_stride * (long long)sizeof(Elem);   // uniform
    const uint32_t off = n * (uint32_t)sizeof(Elem);
    const auto put = [&](int j) {
        if constexpr (kOutF32) *reinterpret_cast<float*>(row + off) = z[j];
        else *reinterpret_cast<uint16_t*>(row + off) = elem_from_f32<kF16>(z[j]);
        row += l.y_stride * (long long)sizeof(Elem);
    };
    if (t0 + kCnt <= l.T) {
#pragma unroll
        for (int j = 0; j < kCnt; ++j) put(j);
    } else {
#pragma unroll
        for (int j = 0; j < kCnt; ++j)
            if (t0 + j < l.T) put(j);
    }
}

// Bound by the tensor cores: a stage's 64 columns are 512 clocks of products for 32 KB a CTA, which L2 delivers just in
// time.  Measured in bf16: 4096 x 8192 x 2048 74-76 us = 1.81-1.85 PFLOP/s; 16384 x 8192 x 2048 with silu 280-327 us = 1.7-2.0,
// by the clock that the power limit leaves; 4096 x 2048 x 4096 43-46 us = 1.5-1.6 (128 tiles on 76 pairs); 4096 x 2048 x 16384,
// two chunks, 153-166 us.
// kTN: weight rows of a tile (256, or 128 with fp32 outputs so that a thread's running sums fit its
// registers); with kGated half of them are gate rows and half the up rows of the same features.  kGroups: warpgroups of
// the epilogue.
template <bool kF16, bool kOutF32, bool kGated, int kTN, int kGroups>
__global__ void __launch_bounds__(tc_threads(kGroups), 1)
    linear_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_y, TcArgs a) {
    constexpr int kBRows = kTN / 2;                          // weight rows a CTA holds
    constexpr int kABytes = kLM * 128, kBBytes = kBRows * 128, kStage = kABytes + kBBytes;
    constexpr int kBufs = 512 / kTN;                         // accumulators in TMEM
    constexpr bool kChunks = kOutF32 || kGroups == 2;        // four groups only take short rows
    static_assert(kOutF32 || kBufs == 2, "the sums of long rows go from one accumulator to the other");
    constexpr int kFeat = kGated ? kTN / 2 : kTN;            // outputs of a tile
    constexpr int kHalf = kFeat / kGroups;                   // outputs a warpgroup handles
    constexpr int kPairStages = kGroups == 2 ? 6 : 5;
    constexpr int kGrp = kOutF32 ? 32 : 64;                  // outputs of one staging row (128 bytes)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* staging = smem + kPairStages * kStage;          // a buffer per warpgroup
    float* s_bias = reinterpret_cast<float*>(staging + kGroups * kStageBuf);   // [warpgroup][gate, up][64]
    PairSmem* sh = reinterpret_cast<PairSmem*>(s_bias + 256);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const int tiles = a.tiles_m * a.tiles_n;
    const int nkb = a.nkb, chunk = kChunks ? chunk_blocks(kOutF32, kGated) : nkb, nch = kChunks ? (nkb + chunk - 1) / chunk : 1;
    int* status = reinterpret_cast<int*>(a.l.ws);
    volatile int* abort = &sh->abort;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
        if (a.y_tma) prefetch_tmap(&tm_y);
        for (int i = 0; i < kPairStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], 2 * 4 * kGroups);
        }
        sh->abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(&sh->tmem)), "r"(512u)
                     : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    tc_fence_before();
    __syncthreads();
    cluster_arrive();
    cluster_wait();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        // ------------------------------ producer: x rows and half of the w rows ------------------------------
        int s = 0;
        uint32_t ph = 1;   // the first pass over the ring finds every slot free
        bool ok = true;
        for (int i = cluster; i < tiles && ok; i += clusters) {
            int m, n;
            tile_at(i, a.tiles_m, a.tiles_n, &m, &n);
            const int t0 = m * 2 * kLM + (int)rank * kLM;
            const int w0 = kGated ? n * kFeat + (rank ? a.l.N : 0) : n * kTN + (int)rank * kBRows;
            for (int kb = 0; kb < nkb; ++kb) {
                if (!mbar_wait_warp(&sh->empty[s], ph, abort)) { ok = false; break; }
#ifdef MOE_TEST_DROP_LINEAR_BLOCK
                // timeout test only: both CTAs leave this block of the first tile out, so the issuer's wait on it never ends
                const bool drop = i == 0 && kb == MOE_TEST_DROP_LINEAR_BLOCK;
#else
                constexpr bool drop = false;
#endif
                if (!drop && elect_one()) {
                    if (rank == 0) mbar_arrive_expect_tx(&sh->full[s], 2 * kStage);
                    const uint32_t bar = map_to_rank(&sh->full[s], 0);
                    uint8_t* st = smem + s * kStage;
                    tma_load_2d_pair(st, &tm_x, kb * kLK, t0, bar);
                    tma_load_2d_pair(st + kABytes, &tm_w, kb * kLK, w0, bar);
                }
                if (++s == kPairStages) { s = 0; ph ^= 1; }
            }
        }
        // every slot released: no arrival of the issuer's commits is still on its way to this CTA
        for (int i = 0; i < kPairStages && ok; ++i) {
            if (!mbar_wait_warp(&sh->empty[s], ph, abort)) ok = false;
            if (++s == kPairStages) { s = 0; ph ^= 1; }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp == 1 && rank == 0) {
        // ------------------------------ MMA issuer (one CTA of the pair) ------------------------------
        const uint32_t idesc = idesc_f16kind(kF16, 2 * kLM, kTN);
        int s = 0, buf = 0;
        uint32_t ph = 0, eph = 1;
        bool ok = true;
        for (int i = cluster; i < tiles && ok; i += clusters) {
            for (int c = 0; c < nch && ok; ++c) {
                if (!mbar_wait_warp(&sh->acc_empty[buf], eph, abort)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d = tmem + buf * kTN;
                const int k1 = min(nkb, (c + 1) * chunk);
                for (int kb = c * chunk; kb < k1; ++kb) {
                    if (!mbar_wait_warp(&sh->full[s], ph, abort)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sa = smem_u32(smem + s * kStage);
                        const uint64_t ad = sw128_desc(sa), bd = sw128_desc(sa + kABytes);
#pragma unroll
                        for (int k = 0; k < kLK / 16; ++k)
                            tc_mma_f16kind<true>(d, ad + 2 * k, bd + 2 * k, idesc, kb > c * chunk || k > 0);
                        tc_commit_pair(&sh->empty[s]);
                        if (kb == k1 - 1) tc_commit_pair(&sh->acc_full[buf]);
                    }
                    __syncwarp();
                    if (++s == kPairStages) { s = 0; ph ^= 1; }
                }
                if (++buf == kBufs) { buf = 0; eph ^= 1; }
            }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp >= 4) {
        // ------------------------------ epilogue ------------------------------
        const int ew = warp - 4, half = ew >> 2, quarter = ew & 3;   // share of the columns, TMEM lanes
        const int r = 32 * quarter + lane;                           // token row in the CTA's tile
        uint8_t* stg = staging + half * kStageBuf;
        float* sb = s_bias + half * (256 / kGroups);
        const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
        const bool issuer = (ew & 3) == 0 && lane == 0;              // stores of this warpgroup
        int buf = 0;
        uint32_t fph = 0;
        bool ok = true;
        // the residual of the next 32 outputs is loaded while these are worked on (16-bit; fp32 residuals, whose registers
        // the running sums need, when they are added)
        Residual32<kOutF32> res = {};
        const auto fetch = [&](int tile, int col) {
            int m, n;
            tile_at(tile, a.tiles_m, a.tiles_n, &m, &n);
            const long long t = (long long)m * 2 * kLM + (int)rank * kLM + r;
            const int nj = n * kFeat + half * kHalf + col;
            if (t < a.l.T && nj < a.l.N) load_residual32<kOutF32>(a, t, nj, min(32, a.l.N - nj), res);
        };
        if (a.l.residual && !kOutF32) fetch(cluster, 0);
        for (int i = cluster; i < tiles && ok; i += clusters) {
            int m, n;
            tile_at(i, a.tiles_m, a.tiles_n, &m, &n);
            const long long t0 = (long long)m * 2 * kLM + (int)rank * kLM;
            const int n0 = n * kFeat + half * kHalf;
            const uint32_t cols = tmem + lane_addr + half * kHalf;
            float sum[kOutF32 ? (kGated ? 2 : 1) * kHalf : 1];
            for (int c = 0; c < nch; ++c) {
                // one answer for the warpgroup, so that its barriers below are reached by all or none
                const bool got = mbar_wait(&sh->acc_full[buf], fph, abort);
                if (named_bar_or(1 + half, 128, !got)) { ok = false; break; }
                tc_fence_after();
                if constexpr (kOutF32) {
                    if (nch > 1) add_chunk<kGated ? 2 : 1, kHalf, kFeat>(cols + buf * kTN, sum, c == 0, c == nch - 1);
                } else if constexpr (kChunks) {
                    if (c > 0) add_sums<kGated ? 2 : 1, kHalf, kFeat>(cols + (buf ^ 1) * kTN, cols + buf * kTN);
                }
                // an accumulator whose sums have gone on (the last one is released below)
                if (kOutF32 ? c < nch - 1 : c > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_release(&sh->acc_empty[kOutF32 ? buf : buf ^ 1], 0);
                }
                if (c < nch - 1) {
                    if (++buf == kBufs) { buf = 0; fph ^= 1; }
                }
            }
            if (!ok) break;
            const uint32_t acc = cols + buf * kTN;
            // 128 bytes of outputs a row at a time (rolled: the code of every activation, unrolled for the whole tile,
            // does not fit the instruction cache)
#pragma unroll 1
            for (int g0 = 0; g0 < kHalf; g0 += kGrp) {
                if (issuer) bulk_wait_read();         // the previous store has read the buffer
                if (a.l.bias && (r & 63) < kGrp && (kGated || r < 64)) {   // bias of these outputs (and of their up rows)
                    const int nb = n0 + g0 + (r & 63);
                    sb[r] = nb < a.l.N ? __ldg(a.l.bias + (r < 64 ? 0 : a.l.N) + nb) : 0.0f;
                }
                named_bar_sync(1 + half, 128);
#pragma unroll 1
                for (int j = 0; j < kGrp; j += 32) {
                    float v[32], up[32];
                    uint32_t q[32], p[32];
                    tmem_ld32(acc + g0 + j, q);
                    if (kGated) tmem_ld32(acc + kFeat + g0 + j, p);
                    tmem_ld_wait();
#pragma unroll
                    for (int u = 0; u < 32; ++u) {
                        v[u] = __uint_as_float(q[u]);
                        if (kGated) up[u] = __uint_as_float(p[u]);
                    }
                    if (a.l.bias) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            v[u] += sb[j + u];
                            if (kGated) up[u] += sb[64 + j + u];
                        }
                    }
                    if (kGated) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) v[u] = v[u] * sigmoid_f32<kOutF32>(v[u]) * up[u];
                    } else {
                        apply_act_all<kOutF32>(a.l.act, v);
                    }
                    if (a.l.residual) {
                        if (kOutF32) fetch(i, g0 + j);
                        add_residual32<kF16, kOutF32>(res, v);
                        if (kOutF32) {}
                        else if (g0 + j + 32 < kHalf) fetch(i, g0 + j + 32);
                        else if (i + clusters < tiles) fetch(i + clusters, 0);
                    }
                    if (kOutF32) {
#pragma unroll
                        for (int u = 0; u < 8; ++u)
                            *stage_piece(stg, r, u) = make_uint4(__float_as_uint(v[4 * u]), __float_as_uint(v[4 * u + 1]),
                                                                 __float_as_uint(v[4 * u + 2]), __float_as_uint(v[4 * u + 3]));
                    } else {
#pragma unroll
                        for (int u = 0; u < 4; ++u)
                            *stage_piece(stg, r, j / 8 + u) =
                                make_uint4(pack2<kF16>(v[8 * u], v[8 * u + 1]), pack2<kF16>(v[8 * u + 2], v[8 * u + 3]),
                                           pack2<kF16>(v[8 * u + 4], v[8 * u + 5]), pack2<kF16>(v[8 * u + 6], v[8 * u + 7]));
                    }
                }
                if (g0 + kGrp >= kHalf) {   // the accumulator has been read: the issuer may reuse it
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_release(&sh->acc_empty[buf], 0);
                }
                if (a.y_tma) fence_proxy_async_smem();
                named_bar_sync(1 + half, 128);
                const int ng = n0 + g0;
                if (a.y_tma) {
                    if (issuer && ng < a.l.N && t0 < a.l.T) {
                        tma_store_2d(&tm_y, stg, ng, (int)t0);
                        bulk_commit();
                    }
                } else {
                    // rows at any alignment: a warp writes 32 rows, lanes along the row
                    constexpr int kSize = kOutF32 ? 4 : 2;
                    for (int rr = 32 * quarter; rr < 32 * quarter + 32; ++rr) {
                        if (t0 + rr >= a.l.T) break;
                        uint8_t* dst = static_cast<uint8_t*>(a.l.y) + ((t0 + rr) * a.l.y_stride + ng) * kSize;
#pragma unroll
                        for (int e = lane; e < kGrp; e += 32) {
                            if (ng + e >= a.l.N) break;
                            const uint8_t* src = stg + rr * 128 + ((((e * kSize) >> 4) ^ (rr & 7)) << 4) + ((e * kSize) & 15);
                            if (kOutF32) *reinterpret_cast<float*>(dst + 4 * e) = *reinterpret_cast<const float*>(src);
                            else *reinterpret_cast<uint16_t*>(dst + 2 * e) = *reinterpret_cast<const uint16_t*>(src);
                        }
                    }
                }
            }
            if (++buf == kBufs) { buf = 0; fph ^= 1; }
        }
        if (issuer) bulk_wait_all();
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    }
    __syncthreads();
    if (*abort) {   // unwinding: let copies and products in flight land before shared memory and TMEM go
        const long long from = clock64();
        while (clock64() - from < 4000000) {}
    }
    tc_fence_before();
    cluster_arrive();
    cluster_wait();
    if (warp == 2) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem), "r"(512u) : "memory");
    }
}

// ---------------------------------------------------------------------------------------------------------

constexpr int kFeatStages = 12;
struct FeatSmem {
    uint64_t full[kFeatStages], empty[kFeatStages];
    uint64_t acc_full[2], acc_empty[2];
    uint64_t joined;           // the other slices' partial sums have arrived
    uint32_t tmem;
    int abort;
};

// Contiguous bytes from this CTA's shared memory to another's, counted on a barrier there (both shared::cluster).
__device__ __forceinline__ void bulk_s2s(uint32_t dst, const void* src, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];" ::"r"(dst),
                 "r"(smem_u32(src)), "r"(bytes), "r"(bar)
                 : "memory");
}

// Sums the slices' partial sums of kCnt tokens of feature f, in slice order, and finishes them.  own: this CTA's
// sums of these tokens; in: the same of slice 0 in its inbound buffer; rows of 128 features.
template <bool kF16, bool kOutF32, bool kGated, int kCnt>
__device__ __forceinline__ void join_slices(const LinearArgs& l, const float* own, int own_g, const float* in, int in_g,
                                            int slices, int rank, long long t, int n, float b0, float b1) {
    float v[kCnt] = {}, up[kCnt] = {};
    OutElem<kOutF32> res[kCnt] = {};
    if (l.residual) load_residual<kOutF32, kCnt>(l, t, n, res);
    for (int q = 0; q < slices; ++q) {
        const float* p = q == rank ? own : in + q * (kGated ? 2 : 1) * in_g;
        const int gg = q == rank ? own_g : in_g;
#pragma unroll
        for (int u = 0; u < kCnt; ++u) {
            v[u] += p[u * kLM];
            if (kGated) up[u] += p[gg + u * kLM];
        }
    }
    finish_column<kF16, kOutF32, kGated, kCnt>(l, t, n, b0, b1, v, up, res);
}

__host__ __device__ constexpr int feat_groups(int tokens) { return tokens >= 64 ? 4 : 2; }   // warpgroups of the epilogue

struct FeatArgs {
    LinearArgs l;
    int tiles_n, tiles_t, nkb, slices, stages;
    int ring;          // bytes of the operand ring (with slices: at least of a tile's partial sums)
};

// Bound by HBM where the weights are large (16 x 131072 x 2048: 82 us = 6.6 TB/s), else by its stages: 64 columns of a
// 128 x 64 tile take 0.18 us whether one CTA runs or 128 (4096 x 256 x 2048, fp32 out: 9.6 us), and loading the weight rows
// once for two or four CTAs by multicast changes nothing there (10.9 us, the cluster's barriers being extra).
// Weight rows as the M side: lane = feature, column = token, so a warp stores 32 consecutive features of a
// token at once whatever the alignment of y, and a tile costs as many token columns as there are tokens.
// kTT: tokens of a tile.  kGated: a tile has 128 gate rows and the 128 up rows of the same features, each with
// its own accumulator.
template <bool kF16, bool kOutF32, bool kGated, int kTT>
__global__ void __launch_bounds__(tc_threads(feat_groups(kTT)), 1)
    linear_feat(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, FeatArgs a) {
    constexpr int G = kGated ? 2 : 1;
    constexpr int kABytes = G * kLM * 128, kBlock = kABytes + kTT * 128, kSub = feat_sub(kBlock), kStage = kSub * kBlock;
    constexpr int kGroups = feat_groups(kTT), kThreads = tc_threads(kGroups);
    constexpr int kHalf = kTT / kGroups;                     // tokens a warpgroup handles
    constexpr int kBlk = kHalf < 16 ? kHalf : 16;            // of them, at a time
    constexpr int kAcc = G * kTT;                            // TMEM columns of a tile's accumulators
    constexpr int kBufs = 2 * kAcc <= 512 ? 2 : 1;
    constexpr int kTmem = kBufs * kAcc <= 32 ? 32 : kBufs * kAcc;
    static_assert((kTmem & (kTmem - 1)) == 0 && kTmem <= 512, "TMEM columns");
    static_assert(kOutF32 || kBufs == 2, "the sums of long rows go from one accumulator to the other");
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    __shared__ FeatSmem sh;
    const int lane = threadIdx.x & 31, warp = __shfl_sync(0xffffffffu, threadIdx.x >> 5, 0);   // (known to be uniform)
    const int S = a.slices, rank = S > 1 ? (int)cluster_ctarank() : 0, stages = a.stages;
    // slices > 1: this CTA's partial sums [G][kTT][128 features] take the ring's place, those of the other slices
    // for its share of the tokens arrive in [slice][G][per][128]
    float* own = reinterpret_cast<float*>(smem);
    float* inbound = reinterpret_cast<float*>(smem + a.ring);
    const int per = kTT / S;                                 // tokens of the share
    const int first = S > 1 ? blockIdx.x / S : blockIdx.x, step = S > 1 ? INT32_MAX / 2 : (int)gridDim.x;
    const int tiles = a.tiles_n * a.tiles_t;
    const int kb0 = (int)((long long)a.nkb * rank / S), kb1 = (int)((long long)a.nkb * (rank + 1) / S);
    const int chunk = chunk_blocks(kOutF32, kGated) / kSub, nch = (kb1 - kb0 + chunk - 1) / chunk;
    int* status = reinterpret_cast<int*>(a.l.ws);
    volatile int* abort = &sh.abort;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
        for (int i = 0; i < stages; ++i) {
            mbar_init(&sh.full[i], 1);
            mbar_init(&sh.empty[i], 1);
        }
        for (int i = 0; i < kBufs; ++i) {
            mbar_init(&sh.acc_full[i], 1);
            mbar_init(&sh.acc_empty[i], 4 * kGroups);
        }
        mbar_init(&sh.joined, 1);
        sh.abort = 0;
        fence_barrier_init();
        if (S > 1) mbar_arrive_expect_tx(&sh.joined, (S - 1) * G * per * kLM * 4);
    }
    if (warp == 2) {
        tmem_alloc(&sh.tmem, kTmem);
        tmem_relinquish();
    }
    if (warp == 3 && lane < stages && kb0 + lane < kb1) {
        // warm L2 with the first weight blocks while the previous kernel on the stream finishes (only a hint:
        // what that kernel may still write is read after the wait below)
        const int n0 = first % a.tiles_n * kLM;
        for (int u = 0; u < kSub; ++u) {
            prefetch_l2_tile(&tm_w, ((kb0 + lane) * kSub + u) * kLK, n0);
            if (kGated) prefetch_l2_tile(&tm_w, ((kb0 + lane) * kSub + u) * kLK, a.l.N + n0);
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh.tmem;
    if (S > 1) cluster_arrive();
    pdl_wait();
    pdl_launch_dependents();
    if (S > 1) cluster_wait();   // every CTA of the cluster runs: its shared memory may be written

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        for (int i = first; i < tiles && ok; i += step) {
            const int n0 = i % a.tiles_n * kLM, t0 = i / a.tiles_n * kTT;
            for (int kb = kb0; kb < kb1; ++kb) {
                if (!mbar_wait_warp(&sh.empty[s], ph, abort)) { ok = false; break; }
#ifdef MOE_TEST_DROP_LINEAR_BLOCK
                const bool drop = i == 0 && kb == MOE_TEST_DROP_LINEAR_BLOCK;   // as in linear_pair
#else
                constexpr bool drop = false;
#endif
                if (!drop && elect_one()) {
                    uint8_t* st = smem + s * kStage;
                    mbar_arrive_expect_tx(&sh.full[s], kStage);
#pragma unroll
                    for (int u = 0; u < kSub; ++u) {
                        const int c = (kb * kSub + u) * kLK;
                        uint8_t* at = st + u * kBlock;
                        tma_load_2d(at, &tm_w, c, n0, &sh.full[s]);
                        if (kGated) tma_load_2d(at + kLM * 128, &tm_w, c, a.l.N + n0, &sh.full[s]);
                        tma_load_2d(at + kABytes, &tm_x, c, t0, &sh.full[s]);
                    }
                }
                if (++s == stages) { s = 0; ph ^= 1; }
            }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_f16kind(kF16, kLM, kTT);
        int s = 0, buf = 0;
        uint32_t ph = 0, eph = 1;
        bool ok = true;
        for (int i = first; i < tiles && ok; i += step) {
            for (int c = 0; c < nch && ok; ++c) {
                if (!mbar_wait_warp(&sh.acc_empty[buf], eph, abort)) { ok = false; break; }
                tc_fence_after();
                const int f = kb0 + c * chunk, k1 = min(kb1, f + chunk);
                const uint32_t d = tmem + buf * kAcc;
                for (int kb = f; kb < k1; ++kb) {
                    if (!mbar_wait_warp(&sh.full[s], ph, abort)) { ok = false; break; }
                    tc_fence_after();
                    if (elect_one()) {
                        const uint32_t sa = smem_u32(smem + s * kStage);
#pragma unroll
                        for (int u = 0; u < kSub; ++u) {
                            const uint64_t bd = sw128_desc(sa + u * kBlock + kABytes);
#pragma unroll
                            for (int g = 0; g < G; ++g) {
                                const uint64_t ad = sw128_desc(sa + u * kBlock + g * kLM * 128);
#pragma unroll
                                for (int k = 0; k < kLK / 16; ++k)
                                    tc_mma_f16kind<false>(d + g * kTT, ad + 2 * k, bd + 2 * k, idesc,
                                                          kb > f || u > 0 || k > 0);
                            }
                        }
                        tc_commit(&sh.empty[s]);
                        if (kb == k1 - 1) tc_commit(&sh.acc_full[buf]);
                    }
                    __syncwarp();
                    if (++s == stages) { s = 0; ph ^= 1; }
                }
                if (++buf == kBufs) { buf = 0; eph ^= 1; }
            }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp >= 4) {
        const int ew = warp - 4, half = ew >> 2, quarter = ew & 3, r = 32 * quarter + lane;   // feature in the tile
        int buf = 0;
        uint32_t fph = 0;
        bool ok = true;
        // the residual of the next kBlk outputs is loaded while these are worked on
        const bool has_res = a.l.residual && S == 1;
        OutElem<kOutF32> res[kBlk] = {};
        if (has_res && first < tiles)
            load_residual<kOutF32, kBlk>(a.l, (long long)(first / a.tiles_n) * kTT + half * kHalf,
                                         first % a.tiles_n * kLM + r, res);
        for (int i = first; i < tiles && ok; i += step) {
            const int n = i % a.tiles_n * kLM + r;
            const long long t0 = (long long)(i / a.tiles_n) * kTT + half * kHalf;
            const uint32_t cols = tmem + ((uint32_t)(32 * quarter) << 16) + half * kHalf;
            float sum[kOutF32 ? G * kHalf : 1];
            for (int c = 0; c < nch; ++c) {
                const bool got = mbar_wait_warp(&sh.acc_full[buf], fph, abort);
                if (!got) { ok = false; break; }
                tc_fence_after();
                if constexpr (kOutF32) {
                    if (nch > 1) add_chunk<G, kHalf, kTT>(cols + buf * kAcc, sum, c == 0, c == nch - 1);
                } else if (c > 0) {
                    add_sums<G, kHalf, kTT>(cols + (buf ^ 1) * kAcc, cols + buf * kAcc);
                }
                // an accumulator whose sums have gone on (the last one is released below)
                if (kOutF32 ? c < nch - 1 : c > 0) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive(&sh.acc_empty[kOutF32 ? buf : buf ^ 1]);
                }
                if (c < nch - 1) {
                    if (++buf == kBufs) { buf = 0; fph ^= 1; }
                }
            }
            if (!ok) break;
            const uint32_t acc = cols + buf * kAcc;
            const float b0 = a.l.bias && n < a.l.N ? __ldg(a.l.bias + n) : 0.0f;
            const float b1 = kGated && a.l.bias && n < a.l.N ? __ldg(a.l.bias + a.l.N + n) : 0.0f;
#pragma unroll 1
            for (int j = 0; j < kHalf; j += kBlk) {   // rolled: see linear_pair
                float v[kBlk], up[kGated ? kBlk : 1];
                uint32_t q[kBlk], p[kBlk];
                tmem_ld_cols<kBlk>(acc + j, q);
                if (kGated) tmem_ld_cols<kBlk>(acc + kTT + j, p);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < kBlk; ++u) {
                    v[u] = __uint_as_float(q[u]);
                    if (kGated) up[kGated ? u : 0] = __uint_as_float(p[u]);
                }
                if (S > 1) {
                    // the ring is free: this CTA's products are complete, in order, with the last accumulator
#pragma unroll
                    for (int u = 0; u < kBlk; ++u) {
                        own[(half * kHalf + j + u) * kLM + r] = v[u];
                        if (kGated) own[(kTT + half * kHalf + j + u) * kLM + r] = up[kGated ? u : 0];
                    }
                } else {
                    OutElem<kOutF32> now[kBlk];
#pragma unroll
                    for (int u = 0; u < kBlk; ++u) now[u] = res[u];
                    if (has_res) {
                        if (j + kBlk < kHalf) {
                            load_residual<kOutF32, kBlk>(a.l, t0 + j + kBlk, n, res);
                        } else if (i + step < tiles) {
                            const int ni = i + step;
                            load_residual<kOutF32, kBlk>(a.l, (long long)(ni / a.tiles_n) * kTT + half * kHalf,
                                                         ni % a.tiles_n * kLM + r, res);
                        }
                    }
                    if (n < a.l.N) finish_column<kF16, kOutF32, kGated, kBlk>(a.l, t0 + j, n, b0, b1, v, up, now);
                }
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh.acc_empty[buf]);
            if (++buf == kBufs) { buf = 0; fph ^= 1; }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
        if (S > 1 && ok) fence_proxy_async_smem();   // the partial sums, before they are copied
    }
    __syncthreads();
    if (S > 1) {
        // the cluster's CTAs share out the tile's tokens: each sends the others theirs
        if (warp == 4 && !*abort && elect_one()) {
            for (int q = 1; q < S; ++q) {
                const int to = (rank + q) % S;
#pragma unroll
                for (int g = 0; g < G; ++g)
                    bulk_s2s(map_to_rank(inbound + (rank * G + g) * per * kLM, to), own + (g * kTT + to * per) * kLM,
                             per * kLM * 4,
                             map_to_rank(&sh.joined, to));
            }
        }
        __syncwarp();
        const bool got = mbar_wait_warp(&sh.joined, 0, abort);
        if (!got && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
        cluster_arrive();   // everything for this CTA has arrived; it leaves when that holds for all
        const int f = threadIdx.x & 127, n = first % a.tiles_n * kLM + f;
        const long long tt = (long long)(first / a.tiles_n) * kTT + rank * per;
        if (got && n < a.l.N) {
            const float b0 = a.l.bias ? __ldg(a.l.bias + n) : 0.0f;
            const float b1 = kGated && a.l.bias ? __ldg(a.l.bias + a.l.N + n) : 0.0f;
            const int have = (int)min((long long)per, a.l.T - tt);   // tokens of the share that exist
            const float* mine = own + rank * per * kLM + f;
            if (per >= 8) {
                for (int j = 8 * (threadIdx.x >> 7); j < have; j += 8 * (kThreads / 128))
                    join_slices<kF16, kOutF32, kGated, 8>(a.l, mine + j * kLM, kTT * kLM, inbound + j * kLM + f, per * kLM, S, rank,
                                                    tt + j, n, b0, b1);
            } else if (threadIdx.x < 128 && have > 0) {
                join_slices<kF16, kOutF32, kGated, 4>(a.l, mine, kTT * kLM, inbound + f, per * kLM, S, rank, tt, n, b0, b1);
            }
        }
        __syncwarp();
        cluster_wait();
    }
    if (*abort) {   // unwinding: let copies and products in flight land first
        const long long from = clock64();
        while (clock64() - from < 4000000) {}
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, kTmem);
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, int threads, size_t smem, int cluster_x, cudaStream_t st,
                            Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster_x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    const cudaError_t e = cudaLaunchKernelEx(&cfg, kernel, std::forward<Args>(args)...);
    return e == cudaSuccess ? cudaGetLastError() : e;
}

// Tensor maps of x, w and y for tiles of `wbox` weight rows.
cudaError_t make_maps(const LinearArgs& l, int wbox, bool store, CUtensorMap* x, CUtensorMap* w, CUtensorMap* y) {
    cudaError_t e = make_tmap_bf16_2d(x, l.x, l.T, l.K, l.x_stride * 2, kLK, kLM);
    if (e == cudaSuccess) e = make_tmap_bf16_2d(w, l.w, l.rows, l.K, l.w_stride * 2, kLK, wbox);
    if (e == cudaSuccess && store)
        e = l.out_f32 ? make_tmap_f32_2d(y, l.y, l.T, l.N, l.y_stride * 4, 32, kLM)
                      : make_tmap_bf16_2d(y, l.y, l.T, l.N, l.y_stride * 2, 64, kLM);
    return e;
}

TcArgs tc_args(const LinearArgs& l) {
    TcArgs a{};
    a.l = l;
    a.nkb = (l.K + kLK - 1) / kLK;
    const int size = l.out_f32 ? 4 : 2;
    a.y_tma = (l.y_stride * size) % 16 == 0;
    a.r_vec = (l.r_stride * size) % 16 == 0;
    return a;
}

// Clusters of two that fit the device at one time (each takes both SMs' shared memory whole).
template <typename Kernel>
int pair_clusters(Kernel kernel, int threads, size_t smem, int num_sms) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(num_sms / 2 * 2);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    return n;
}

template <bool kF16, bool kOutF32, bool kGated, int kGroups>
cudaError_t launch_pair(const LinearArgs& l, cudaStream_t st) {
    constexpr int kTN = kOutF32 ? 128 : 256, kFeat = kGated ? kTN / 2 : kTN;
    constexpr int kStages = kGroups == 2 ? 6 : 5, kThreads = tc_threads(kGroups);
    constexpr size_t kSmem = 1024 + kStages * (kLM * 128 + kTN / 2 * 128) + kGroups * kStageBuf + 256 * 4 + sizeof(PairSmem);
    static_assert(kSmem <= 232448, "shared memory of one CTA");
    auto* kernel = linear_pair<kF16, kOutF32, kGated, kTN, kGroups>;
    static std::atomic<int> clusters[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int nc = clusters[dev].load();
    if (nc == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        nc = pair_clusters(kernel, kThreads, kSmem, l.num_sms);
        if (nc <= 0) return cudaErrorNotSupported;
        clusters[dev].store(nc);
    }
    TcArgs a = tc_args(l);
    a.tiles_m = (l.T + 2 * kLM - 1) / (2 * kLM);
    a.tiles_n = (l.N + kFeat - 1) / kFeat;
    CUtensorMap x{}, w{}, y{};
    if ((e = make_maps(l, kTN / 2, a.y_tma, &x, &w, &y)) != cudaSuccess) return e;
    const long long tiles = (long long)a.tiles_m * a.tiles_n;
    if (tiles > INT32_MAX) return cudaErrorInvalidValue;
    return launch_clusters(kernel, dim3(2 * (unsigned)(tiles < nc ? tiles : nc)), kThreads, kSmem, 2, st, x, w, y, a);
}

template <bool kF16, bool kOutF32, bool kGated, int kTT>
cudaError_t launch_feat_tt(const LinearArgs& l, int slices, cudaStream_t st) {
    constexpr int G = kGated ? 2 : 1, kBlock = G * kLM * 128 + kTT * 128, kSub = feat_sub(kBlock), kStage = kSub * kBlock;
    constexpr int kPart = G * kTT * kLM * 4;         // bytes of a slice's partial sums
    constexpr int kMost = 220 * 1024;   // the barriers are in static shared memory
    auto* kernel = linear_feat<kF16, kOutF32, kGated, kTT>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, 1024 + kMost);
        if (e == cudaSuccess && slices > 8) e = cudaErrorInvalidValue;
        if (e != cudaSuccess) return e;
        set[dev].store(true);
    }
    FeatArgs a{};
    a.l = l;
    a.nkb = (l.K + kSub * kLK - 1) / (kSub * kLK);
    a.tiles_n = (l.N + kLM - 1) / kLM;
    a.tiles_t = (l.T + kTT - 1) / kTT;
    a.slices = slices;
    const long long tiles = (long long)a.tiles_n * a.tiles_t;
    if (tiles > INT32_MAX / 16 || slices > a.nkb) return cudaErrorInvalidValue;
    const int blocks_of = (a.nkb + slices - 1) / slices;
    const long long blocks = tiles * slices > l.num_sms && slices == 1 ? l.num_sms : tiles * slices;
    const long long work = blocks_of * ((tiles * slices + blocks - 1) / blocks);   // K blocks a CTA goes through
    if (kTT / slices < 4 || (slices > 1 && 2 * kPart > kMost)) return cudaErrorInvalidValue;
    const int room = kMost - (slices > 1 ? kPart : 0);
    a.stages = room / kStage < kFeatStages ? room / kStage : kFeatStages;
    if (work < a.stages) a.stages = (int)work;   // no more than it uses: the next kernel's CTAs may start beside
    a.ring = a.stages * kStage;
    if (slices > 1 && a.ring < kPart) a.ring = kPart;
    size_t smem = (size_t)a.ring + (slices > 1 ? kPart : 0);
    // CTAs on one SM have to get their TMEM columns without waiting for each other (those of one cluster wait at
    // its barriers): no more of them than 512 / kTmem fit in the 228 KB
    constexpr int kAcc = G * kTT, kCols = 2 * kAcc <= 512 ? 2 * kAcc : kAcc, kFit = 512 / (kCols < 32 ? 32 : kCols);
    constexpr size_t kLeast = 228 * 1024 / (kFit + 1);
    if (smem < kLeast) smem = kLeast;
    CUtensorMap x{}, w{};
    e = make_tmap_bf16_2d(&x, l.x, l.T, l.K, l.x_stride * 2, kLK, kTT);
    if (e == cudaSuccess) e = make_tmap_bf16_2d(&w, l.w, l.rows, l.K, l.w_stride * 2, kLK, kLM);
    if (e != cudaSuccess) return e;
    return launch_clusters(kernel, dim3((unsigned)blocks), tc_threads(feat_groups(kTT)), 1024 + smem, slices, st, x, w, a);
}

template <bool kF16, bool kOutF32, bool kGated>
cudaError_t launch_feat(const LinearArgs& l, int tt, int slices, cudaStream_t st) {
    switch (tt) {
        case 16: return launch_feat_tt<kF16, kOutF32, kGated, 16>(l, slices, st);
        case 32: return launch_feat_tt<kF16, kOutF32, kGated, 32>(l, slices, st);
        case 64: return launch_feat_tt<kF16, kOutF32, kGated, 64>(l, slices, st);
        case 128:
            if constexpr (!(kOutF32 && kGated)) return launch_feat_tt<kF16, kOutF32, kGated, 128>(l, slices, st);
            break;
        case 256:
            if constexpr (!kOutF32 && !kGated) return launch_feat_tt<kF16, kOutF32, kGated, 256>(l, slices, st);
            break;
    }
    return cudaErrorInvalidValue;
}

template <bool kF16, bool kOutF32, bool kGated>
cudaError_t launch_tc(const LinearArgs& l, cudaStream_t st) {
    const LinearPlan p = linear_plan(l);
    if (!p.pair) return launch_feat<kF16, kOutF32, kGated>(l, p.tt, p.slices, st);
    // Short K loops leave the time to the epilogue, and four warpgroups of it pay for a stage less in the ring (K = 512 with
    // GELU: 52 against 58 us at 4096 x 8192; K = 2048: 344 against 336 us at 16384 x 8192).
    if constexpr (!kOutF32 && !kGated)
        if (l.K < 1024) return launch_pair<kF16, false, false, 4>(l, st);
    return launch_pair<kF16, kOutF32, kGated, 2>(l, st);
}

template <bool kF16>
cudaError_t launch_tc_type(const LinearArgs& l, cudaStream_t st) {
    const bool g = l.act == MOE_ACT_SWIGLU;
    if (l.out_f32) return g ? launch_tc<kF16, true, true>(l, st) : launch_tc<kF16, true, false>(l, st);
    return g ? launch_tc<kF16, false, true>(l, st) : launch_tc<kF16, false, false>(l, st);
}

}  // namespace
}  // namespace moe
