// linear_tc.cu -- moe_linear on the 5th-generation tensor cores (more than a few tokens).
//
// Both kernels compute D[token][feature] = sum_k x[token][k] w[feature][k] with x rows as the M and w rows
// as the N side of tcgen05.mma: both are K-major, both come in by TMA as 64-column blocks with the
// 128-byte swizzle (TMA fills what lies beyond T, N or K with zeros), the fp32 accumulator is in TMEM.
//
//   linear_pair   large products.  Two CTAs (a cluster) share one 256-token x TN-feature tile: each holds
//                 128 tokens' rows and half of the weight rows, so a byte of shared memory feeds twice the
//                 products of a single-CTA tile.  Persistent; while the epilogue empties one accumulator
//                 the next tile's products go into another.
//   linear_split  few tiles.  One CTA per 128-token x TN-feature tile and slice of K; the 1..8 CTAs of a
//                 cluster hold the slices of one tile and add their fp32 partial sums through
//                 distributed shared memory, in slice order, so that a small product still uses most SMs.
//
// fp32 outputs: the tensor cores truncate when they add to the accumulator (about half a unit of 2^-23 of
// the running sum at each 16-column step, always towards zero), so after kChunk blocks the epilogue
// takes the partial sum into registers and adds the next in ordinary fp32.  For 16-bit outputs that
// error is far below the rounding of the output, and the whole of K stays in the accumulator.
#include <atomic>

#include "linear_common.cuh"

namespace moe {
namespace {

constexpr int kLK = 64;                 // columns of K per block: one 128-byte swizzle row
constexpr int kLM = 128;                // token rows a CTA holds
constexpr int kChunk = 8;               // blocks summed in the accumulator for fp32 outputs
constexpr int kEpiWarps = 8;            // two warpgroups, each half of the columns
constexpr int kTcThreads = 32 * (4 + kEpiWarps);   // warps 0..3: producer, issuer, TMEM, spare

constexpr int kPairStages = 6;
constexpr int kStageBuf = 128 * 128;    // a warpgroup's output staging: 128 rows of 128 bytes

struct PairSmem {
    uint64_t full[kPairStages], empty[kPairStages];
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

// Adds the residual to 32 outputs (features n0.. of token t; valid of them exist) held as fp32.
template <bool kF16, bool kOutF32>
__device__ __forceinline__ void add_residual(const TcArgs& a, long long t, int n0, int valid, float (&v)[32]) {
    if (kOutF32) {
        const float* p = static_cast<const float*>(a.l.residual) + t * a.l.r_stride + n0;
        if (a.r_vec && valid == 32) {
#pragma unroll
            for (int i = 0; i < 8; ++i) {
                const float4 q = *reinterpret_cast<const float4*>(p + 4 * i);
                v[4 * i] += q.x; v[4 * i + 1] += q.y; v[4 * i + 2] += q.z; v[4 * i + 3] += q.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < valid) v[i] += p[i];
        }
    } else {
        const uint16_t* p = static_cast<const uint16_t*>(a.l.residual) + t * a.l.r_stride + n0;
        if (a.r_vec && valid == 32) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                const uint4 q = *reinterpret_cast<const uint4*>(p + 8 * i);
                const uint32_t u[4] = {q.x, q.y, q.z, q.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    v[8 * i + 2 * j] += elem_f32<kF16>((uint16_t)(u[j] & 0xffffu));
                    v[8 * i + 2 * j + 1] += elem_f32<kF16>((uint16_t)(u[j] >> 16));
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < 32; ++i)
                if (i < valid) v[i] += elem_f32<kF16>(p[i]);
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

// kTN: weight rows of a tile (256, or 128 with fp32 outputs so that a thread's running sums fit its
// registers); with kGated half of them are gate rows and half the up rows of the same features.
template <bool kF16, bool kOutF32, bool kGated, int kTN>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_pair(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w,
                const __grid_constant__ CUtensorMap tm_y, TcArgs a) {
    constexpr int kBRows = kTN / 2;                          // weight rows a CTA holds
    constexpr int kABytes = kLM * 128, kBBytes = kBRows * 128, kStage = kABytes + kBBytes;
    constexpr int kBufs = 512 / kTN;                         // accumulators in TMEM
    constexpr int kFeat = kGated ? kTN / 2 : kTN;            // outputs of a tile
    constexpr int kHalf = kFeat / 2;                         // outputs a warpgroup handles
    constexpr int kGrp = kOutF32 ? 32 : 64;                  // outputs of one staging row (128 bytes)
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    uint8_t* staging = smem + kPairStages * kStage;          // two buffers, one per warpgroup
    float* s_bias = reinterpret_cast<float*>(staging + 2 * kStageBuf);   // [warpgroup][2][64]
    PairSmem* sh = reinterpret_cast<PairSmem*>(s_bias + 2 * 128);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const uint32_t rank = cluster_ctarank();
    const int cluster = blockIdx.x >> 1, clusters = gridDim.x >> 1;
    const int tiles = a.tiles_m * a.tiles_n;
    const int nkb = a.nkb, chunk = kOutF32 ? kChunk : nkb, nch = (nkb + chunk - 1) / chunk;
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
            mbar_init(&sh->acc_empty[i], 2 * kEpiWarps);
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
                if (elect_one()) {
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
        const int ew = warp - 4, half = ew >> 2, quarter = ew & 3;   // columns, TMEM lanes
        const int r = 32 * quarter + lane;                           // token row in the CTA's tile
        uint8_t* stg = staging + half * kStageBuf;
        float* sb = s_bias + half * 128;
        const uint32_t lane_addr = (uint32_t)(32 * quarter) << 16;
        const bool issuer = (ew & 3) == 0 && lane == 0;              // stores of this warpgroup
        int buf = 0;
        uint32_t fph = 0;
        bool ok = true;
        for (int i = cluster; i < tiles && ok; i += clusters) {
            int m, n;
            tile_at(i, a.tiles_m, a.tiles_n, &m, &n);
            const long long t0 = (long long)m * 2 * kLM + (int)rank * kLM;
            const int n0 = n * kFeat + half * kHalf;
            float sum[kOutF32 ? (kGated ? 2 : 1) * kHalf : 1];
            for (int c = 0; c < nch; ++c) {
                // one answer for the warpgroup, so that its barriers below are reached by all or none
                const bool got = mbar_wait(&sh->acc_full[buf], fph, abort);
                if (named_bar_or(1 + half, 128, !got)) { ok = false; break; }
                tc_fence_after();
                const uint32_t acc = tmem + lane_addr + buf * kTN + half * kHalf;
                if (kOutF32) {
#pragma unroll
                    for (int g = 0; g < (kGated ? 2 : 1); ++g)
#pragma unroll
                        for (int j = 0; j < kHalf; j += 32) {
                            uint32_t q[32];
                            tmem_ld32(acc + g * kFeat + j, q);
                            tmem_ld_wait();
#pragma unroll
                            for (int u = 0; u < 32; ++u)
                                sum[g * kHalf + j + u] =
                                    c == 0 ? __uint_as_float(q[u]) : sum[g * kHalf + j + u] + __uint_as_float(q[u]);
                        }
                }
                if (kOutF32 || c < nch - 1) {   // (16-bit outputs: one chunk, released below)
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_release(&sh->acc_empty[buf], 0);
                }
                if (c < nch - 1 && ++buf == kBufs) { buf = 0; fph ^= 1; }
            }
            if (!ok) break;
            const uint32_t acc = tmem + lane_addr + buf * kTN + half * kHalf;
            const bool row_in = t0 + r < a.l.T;
            // 128 bytes of outputs a row at a time
#pragma unroll
            for (int g0 = 0; g0 < kHalf; g0 += kGrp) {
                if (issuer) bulk_wait_read();         // the previous store has read the buffer
                if (a.l.bias && (r & 63) < kGrp && (kGated || r < 64)) {   // bias of these outputs (and of their up rows)
                    const int nb = n0 + g0 + (r & 63);
                    sb[r] = nb < a.l.N ? __ldg(a.l.bias + (r < 64 ? 0 : a.l.N) + nb) : 0.0f;
                }
                named_bar_sync(1 + half, 128);
#pragma unroll
                for (int j = 0; j < kGrp; j += 32) {
                    const int nj = n0 + g0 + j, valid = max(0, min(32, a.l.N - nj));
                    float v[32], up[32];
                    if (kOutF32) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            v[u] = sum[g0 + j + u];
                            if (kGated) up[u] = sum[(kGated ? kHalf : 0) + g0 + j + u];
                        }
                    } else {
                        uint32_t q[32], p[32];
                        tmem_ld32(acc + g0 + j, q);
                        if (kGated) tmem_ld32(acc + kFeat + g0 + j, p);
                        tmem_ld_wait();
#pragma unroll
                        for (int u = 0; u < 32; ++u) {
                            v[u] = __uint_as_float(q[u]);
                            if (kGated) up[u] = __uint_as_float(p[u]);
                        }
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
                    } else if (a.l.act != MOE_ACT_NONE) {
#pragma unroll
                        for (int u = 0; u < 32; ++u) v[u] = apply_act<kOutF32>(a.l.act, v[u]);
                    }
                    if (a.l.residual && row_in) add_residual<kF16, kOutF32>(a, t0 + r, nj, valid, v);
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
                if (!kOutF32 && g0 + kGrp >= kHalf) {   // the accumulator has been read: the issuer may reuse it
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

struct SplitSmem {
    uint64_t full[8], empty[8];
    uint64_t acc_full[2], acc_empty[2];
    uint32_t tmem;
    int abort;
};

__device__ __forceinline__ float4 ld_dsmem_f4(uint32_t addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0,%1,%2,%3}, [%4];" : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(addr) : "memory");
    return v;
}

template <int kTN> struct SplitShape {
    static constexpr int kStage = kLM * 128 + kTN * 128;
    static constexpr int kStages = kTN == 128 ? 6 : 8;
    static constexpr int kPitch = kTN + 4;                  // floats of a partial-sum row
    static constexpr int kBytes = 1024 + kStages * kStage + (int)sizeof(SplitSmem);
    static_assert(kLM * kPitch * 4 <= kStages * kStage, "the partial sums reuse the operand ring");
};

template <bool kF16, bool kOutF32, bool kGated, int kTN>
__global__ void __launch_bounds__(kTcThreads, 1)
    linear_split(const __grid_constant__ CUtensorMap tm_x, const __grid_constant__ CUtensorMap tm_w, TcArgs a) {
    using Sh = SplitShape<kTN>;
    constexpr int kStage = Sh::kStage, kStages = Sh::kStages, kPitch = Sh::kPitch;
    constexpr int kFeat = kGated ? kTN / 2 : kTN;
    constexpr int kCols = kTN / 2;                           // accumulator columns a warpgroup takes
    extern __shared__ uint8_t smem_raw[];
    uint8_t* smem = smem_raw + ((1024 - (smem_u32(smem_raw) & 1023)) & 1023);
    SplitSmem* sh = reinterpret_cast<SplitSmem*>(smem + kStages * kStage);
    float* part = reinterpret_cast<float*>(smem);
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slices = gridDim.x, rank = blockIdx.x;         // the cluster spans x
    const int m = blockIdx.z, n = blockIdx.y;
    const int kb0 = (int)((long long)a.nkb * rank / slices), kb1 = (int)((long long)a.nkb * (rank + 1) / slices);
    const int chunk = kOutF32 ? kChunk : a.nkb, nch = (kb1 - kb0 + chunk - 1) / chunk;
    int* status = reinterpret_cast<int*>(a.l.ws);
    volatile int* abort = &sh->abort;

    if (threadIdx.x == 0) {
        prefetch_tmap(&tm_x);
        prefetch_tmap(&tm_w);
        for (int i = 0; i < kStages; ++i) {
            mbar_init(&sh->full[i], 1);
            mbar_init(&sh->empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sh->acc_full[i], 1);
            mbar_init(&sh->acc_empty[i], kEpiWarps);
        }
        sh->abort = 0;
        fence_barrier_init();
    }
    if (warp == 2) {
        tmem_alloc(&sh->tmem, 2 * kTN);
        tmem_relinquish();
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = sh->tmem;
    pdl_wait();
    pdl_launch_dependents();

    if (warp == 0) {
        int s = 0;
        uint32_t ph = 1;
        bool ok = true;
        const int t0 = m * kLM, w0 = n * kFeat;
        for (int kb = kb0; kb < kb1; ++kb) {
            if (!mbar_wait_warp(&sh->empty[s], ph, abort)) { ok = false; break; }
            if (elect_one()) {
                uint8_t* st = smem + s * kStage;
                mbar_arrive_expect_tx(&sh->full[s], kStage);
                tma_load_2d(st, &tm_x, kb * kLK, t0, &sh->full[s]);
                tma_load_2d(st + kLM * 128, &tm_w, kb * kLK, w0, &sh->full[s]);
                if (kGated) tma_load_2d(st + kLM * 128 + kFeat * 128, &tm_w, kb * kLK, a.l.N + w0, &sh->full[s]);
            }
            if (++s == kStages) { s = 0; ph ^= 1; }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp == 1) {
        const uint32_t idesc = idesc_f16kind(kF16, kLM, kTN);
        int s = 0, buf = 0;
        uint32_t ph = 0, eph = 1;
        bool ok = true;
        for (int c = 0; c < nch && ok; ++c) {
            if (!mbar_wait_warp(&sh->acc_empty[buf], eph, abort)) { ok = false; break; }
            tc_fence_after();
            const int f = kb0 + c * chunk, k1 = min(kb1, f + chunk);
            for (int kb = f; kb < k1; ++kb) {
                if (!mbar_wait_warp(&sh->full[s], ph, abort)) { ok = false; break; }
                tc_fence_after();
                if (elect_one()) {
                    const uint32_t sa = smem_u32(smem + s * kStage);
                    const uint64_t ad = sw128_desc(sa), bd = sw128_desc(sa + kLM * 128);
#pragma unroll
                    for (int k = 0; k < kLK / 16; ++k)
                        tc_mma_f16kind<false>(tmem + buf * kTN, ad + 2 * k, bd + 2 * k, idesc, kb > f || k > 0);
                    tc_commit(&sh->empty[s]);
                    if (kb == k1 - 1) tc_commit(&sh->acc_full[buf]);
                }
                __syncwarp();
                if (++s == kStages) { s = 0; ph ^= 1; }
            }
            if (++buf == 2) { buf = 0; eph ^= 1; }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
    } else if (warp >= 4) {
        const int ew = warp - 4, half = ew >> 2, quarter = ew & 3, r = 32 * quarter + lane;
        float sum[kCols];
        int buf = 0;
        uint32_t fph = 0;
        bool ok = true;
        for (int c = 0; c < nch; ++c) {
            const bool got = mbar_wait(&sh->acc_full[buf], fph, abort);
            if (!__all_sync(0xffffffffu, got)) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tmem + ((uint32_t)(32 * quarter) << 16) + buf * kTN + half * kCols;
#pragma unroll
            for (int j = 0; j < kCols; j += 32) {
                uint32_t q[32];
                tmem_ld32(acc + j, q);
                tmem_ld_wait();
#pragma unroll
                for (int u = 0; u < 32; ++u)
                    sum[j + u] = c == 0 ? __uint_as_float(q[u]) : sum[j + u] + __uint_as_float(q[u]);
            }
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&sh->acc_empty[buf]);
            if (++buf == 2) { buf = 0; fph ^= 1; }
        }
        if (!ok && lane == 0) { *abort = 1; set_status(status, MOE_STATUS_TIMEOUT); }
        // the last accumulator is complete: every product has read its operands, and the ring is free
        // (with several chunks too: commits complete in order)
        if (ok) {
#pragma unroll
            for (int j = 0; j < kCols; j += 4)
                *reinterpret_cast<float4*>(part + r * kPitch + half * kCols + j) =
                    make_float4(sum[j], sum[j + 1], sum[j + 2], sum[j + 3]);
        }
    }
    __syncthreads();
    if (*abort) {   // unwinding: let copies and products in flight land first
        const long long from = clock64();
        while (clock64() - from < 4000000) {}
    }
    if (slices > 1) {
        cluster_arrive();
        cluster_wait();
    }
    // the cluster's CTAs share out the tile's rows; each sums the slices' partial sums in order
    {
        const int rows = kLM / slices;
        constexpr int kQuads = kFeat / 4;
        for (int i = threadIdx.x; i < rows * kQuads; i += kTcThreads) {
            const int r = rank * rows + i / kQuads, c = 4 * (i % kQuads);
            const long long t = (long long)m * kLM + r;
            const int nn = n * kFeat + c;
            if (t >= a.l.T || nn >= a.l.N) continue;
            const float* mine = part + r * kPitch + c;
            float z[4] = {0.f, 0.f, 0.f, 0.f}, u[4] = {0.f, 0.f, 0.f, 0.f};
            for (int q = 0; q < slices; ++q) {
                const uint32_t at = slices > 1 ? map_to_rank(mine, q) : smem_u32(mine);
                const float4 p = slices > 1 ? ld_dsmem_f4(at) : *reinterpret_cast<const float4*>(mine);
                z[0] += p.x; z[1] += p.y; z[2] += p.z; z[3] += p.w;
                if (kGated) {
                    const float4 v = slices > 1 ? ld_dsmem_f4(at + kFeat * 4) : *reinterpret_cast<const float4*>(mine + kFeat);
                    u[0] += v.x; u[1] += v.y; u[2] += v.z; u[3] += v.w;
                }
            }
            const int valid = min(4, a.l.N - nn);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                if (j >= valid) break;
                if (a.l.bias) {
                    z[j] += __ldg(a.l.bias + nn + j);
                    if (kGated) u[j] += __ldg(a.l.bias + a.l.N + nn + j);
                }
                z[j] = kGated ? z[j] * sigmoid_f32<kOutF32>(z[j]) * u[j] : apply_act<kOutF32>(a.l.act, z[j]);
            }
            constexpr int kSize = kOutF32 ? 4 : 2;
            if (valid == 4 && a.y_tma && (!a.l.residual || a.r_vec)) {   // rows of whole 16 bytes: vectors
                if (a.l.residual) {
                    const uint8_t* p = static_cast<const uint8_t*>(a.l.residual) + (t * a.l.r_stride + nn) * kSize;
                    if (kOutF32) {
                        const float4 q = *reinterpret_cast<const float4*>(p);
                        z[0] += q.x; z[1] += q.y; z[2] += q.z; z[3] += q.w;
                    } else {
                        const uint2 q = *reinterpret_cast<const uint2*>(p);
                        z[0] += elem_f32<kF16>((uint16_t)(q.x & 0xffffu)); z[1] += elem_f32<kF16>((uint16_t)(q.x >> 16));
                        z[2] += elem_f32<kF16>((uint16_t)(q.y & 0xffffu)); z[3] += elem_f32<kF16>((uint16_t)(q.y >> 16));
                    }
                }
                uint8_t* p = static_cast<uint8_t*>(a.l.y) + (t * a.l.y_stride + nn) * kSize;
                if (kOutF32) *reinterpret_cast<float4*>(p) = make_float4(z[0], z[1], z[2], z[3]);
                else *reinterpret_cast<uint2*>(p) = make_uint2(pack2<kF16>(z[0], z[1]), pack2<kF16>(z[2], z[3]));
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    if (j < valid) store_output<kF16, kOutF32>(a.l, t, nn + j, z[j]);
            }
        }
    }
    tc_fence_before();
    if (slices > 1) {   // no CTA leaves while another may read its partial sums
        cluster_arrive();
        cluster_wait();
    } else {
        __syncthreads();
    }
    if (warp == 2) {
        tc_fence_after();
        tmem_dealloc(tmem, 2 * kTN);
    }
}

template <typename... KArgs, typename... Args>
cudaError_t launch_clusters(void (*kernel)(KArgs...), dim3 grid, size_t smem, int cluster_x, cudaStream_t st, Args&&... args) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = cluster_x;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.gridDim = grid;
    cfg.blockDim = dim3(kTcThreads);
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
int pair_clusters(Kernel kernel, size_t smem, int num_sms) {
    cudaLaunchConfig_t cfg{};
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = 2;
    attr[0].val.clusterDim.y = attr[0].val.clusterDim.z = 1;
    cfg.gridDim = dim3(num_sms / 2 * 2);
    cfg.blockDim = dim3(kTcThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    int n = 0;
    if (cudaOccupancyMaxActiveClusters(&n, kernel, &cfg) != cudaSuccess) return 0;
    return n;
}

template <bool kF16, bool kOutF32, bool kGated>
cudaError_t launch_pair(const LinearArgs& l, cudaStream_t st) {
    constexpr int kTN = kOutF32 ? 128 : 256, kFeat = kGated ? kTN / 2 : kTN;
    constexpr size_t kSmem = 1024 + kPairStages * (kLM * 128 + kTN / 2 * 128) + 2 * kStageBuf + 2 * 128 * 4 + sizeof(PairSmem);
    static_assert(kSmem <= 232448, "shared memory of one CTA");
    auto* kernel = linear_pair<kF16, kOutF32, kGated, kTN>;
    static std::atomic<int> clusters[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    int nc = clusters[dev].load();
    if (nc == 0) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmem);
        if (e != cudaSuccess) return e;
        nc = pair_clusters(kernel, kSmem, l.num_sms);
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
    return launch_clusters(kernel, dim3(2 * (unsigned)(tiles < nc ? tiles : nc)), kSmem, 2, st, x, w, y, a);
}

template <bool kF16, bool kOutF32, bool kGated, int kTN>
cudaError_t launch_split_tn(const LinearArgs& l, int slices, cudaStream_t st) {
    constexpr int kFeat = kGated ? kTN / 2 : kTN, kSmem = SplitShape<kTN>::kBytes;
    static_assert(kSmem <= 232448, "shared memory of one CTA");
    auto* kernel = linear_split<kF16, kOutF32, kGated, kTN>;
    static std::atomic<bool> set[64];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= 64) return cudaErrorInvalidDevice;
    if (!set[dev].load()) {
        e = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kSmem);
        if (e != cudaSuccess) return e;
        set[dev].store(true);
    }
    const TcArgs a = tc_args(l);
    CUtensorMap x{}, w{};
    if ((e = make_maps(l, kGated ? kTN / 2 : kTN, false, &x, &w, nullptr)) != cudaSuccess) return e;
    const dim3 grid(slices, (l.N + kFeat - 1) / kFeat, (l.T + kLM - 1) / kLM);
    return launch_clusters(kernel, grid, kSmem, slices, st, x, w, a);
}

// Which kernel.  linear_split while its 64-feature tiles are few; each tile gets as many slices of K (a
// power of two, at least four blocks each) as there are SMs to take them.
template <bool kF16, bool kOutF32, bool kGated>
cudaError_t launch_tc(const LinearArgs& l, cudaStream_t st) {
    const long long tm = (l.T + kLM - 1) / kLM;
    const long long t64 = tm * ((l.rows + 63) / 64), t128 = tm * ((l.rows + 127) / 128);
    const int nkb = (l.K + kLK - 1) / kLK;
    if (t128 <= l.num_sms) {
        const bool wide = t64 > l.num_sms;
        const long long tiles = wide ? t128 : t64;
        int s = 1;
        while (s < 8 && tiles * s * 2 <= l.num_sms && nkb >= 8 * s) s *= 2;
        return wide ? launch_split_tn<kF16, kOutF32, kGated, 128>(l, s, st) : launch_split_tn<kF16, kOutF32, kGated, 64>(l, s, st);
    }
    return launch_pair<kF16, kOutF32, kGated>(l, st);
}

}  // namespace

cudaError_t launch_linear_tc(const LinearArgs& l, cudaStream_t st) {
    const bool g = l.act == MOE_ACT_SWIGLU;
    if (l.f16) {
        if (l.out_f32) return g ? launch_tc<true, true, true>(l, st) : launch_tc<true, true, false>(l, st);
        return g ? launch_tc<true, false, true>(l, st) : launch_tc<true, false, false>(l, st);
    }
    if (l.out_f32) return g ? launch_tc<false, true, true>(l, st) : launch_tc<false, true, false>(l, st);
    return g ? launch_tc<false, false, true>(l, st) : launch_tc<false, false, false>(l, st);
}

}  // namespace moe
