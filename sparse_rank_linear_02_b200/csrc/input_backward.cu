// input_backward.cu -- gradient of the layer's input on the tensor cores.
//
//   dX = dY S + G V,   G = dY U        (Y = X S^T + (X V^T) U^T)
//
// S is 2:4 along d_in, which is the output dimension here and not the one that
// is summed over, so the sparse MMA does not apply (its sparse operand is sparse
// along K): the kernel expands S to a dense operand on the fly, on the way into
// shared memory, and runs dense MMAs.
//
//   A = S^T tile  256 input columns x 64 output rows (K), MN-major: a row of S is
//                 contiguous along d_in, as tcgen05 reads it with the operand's
//                 major-ness in the instruction descriptor,
//   B = dY tile   n tokens x 64 K, K-major, by TMA,
//   D = dX^T tile 256 x n fp32 in TMEM, two accumulators of up to 256 columns.
// After the d_out / 64 stages of S, ceil(r / 64) rank stages add A = V tile (64
// ranks x 256 columns, MN-major, by TMA), B = G tile.  G is formed before by the
// product kernel of the factors' gradients (tc_gemm.cuh) and rounded to bf16, as
// there: the tensor cores read bf16.
//
// A cluster of two CTAs on neighbouring SMs shares a tile (cta_group::2): each
// expands 128 of its columns and loads half of its tokens.
//   warp 0       TMA producer (dY; V and G),
//   warp 1       MMA issue (leader CTA),
//   warps 2..5   epilogue: TMEM -> bf16 -> shared memory -> TMA store,
//   warps 6..13  expanders, four groups of two warps that take the stages in
//                turn: a thread loads 16 bytes of kept values (four groups of
//                S) and their two metadata bytes straight into registers, one
//                turn ahead, and writes 32 bytes of the dense tile in the
//                128-byte swizzle.  The byte permutes that place two values
//                among four positions take their selectors from arithmetic: the
//                selector of position p is byte p of 0x44444444 (zero), turned
//                into 0x10 (first value) or 0x32 (second) by an exclusive or.
// The follower's expanders announce a stage to the leader with 16-byte bulk
// copies that complete on its barrier, since a release-ordered remote arrive
// would stall them for most of a microsecond each.
//
// Few tiles (short batches): the K stages are split over the pairs that would
// idle; slices leave fp32 partial tiles in the workspace, which a second kernel
// adds in slice order.
//
// Every wait is bounded; on expiry an error word is set (slr_check_kernel_error).
#include <cuda.h>

#include <cstring>

#include "tc_gemm.cuh"

namespace slr {

// Error word of this file's bounded waits (read by slr_check_kernel_error).
__device__ unsigned int g_dx_error = 0;

namespace {

unsigned int *dx_err() {
    static unsigned int *addr[64] = {};
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0 || dev >= 64) return nullptr;
    if (addr[dev] == nullptr) {
        void *q = nullptr;
        if (cudaGetSymbolAddress(&q, g_dx_error) == cudaSuccess) addr[dev] = static_cast<unsigned int *>(q);
    }
    return addr[dev];
}

constexpr int kCols = 128;                    // input columns per CTA (half of a pair's tile)
constexpr int kK = 64;                        // output rows (K) per stage
constexpr int kMaxN = 256;                    // tokens per tile
constexpr int kABytes = kCols * kK * 2;       // 16 KB: two 64-column panels of 64 K rows
constexpr int kBBytes = kMaxN / 2 * kK * 2;   // 16 KB
constexpr int kStage = kABytes + kBBytes;
constexpr int kNS = 6;
constexpr int kOutBytes = 32 * kCols * 2;     // 32 tokens x 128 columns
constexpr int kOutOff = kNS * kStage;
constexpr int kBarOff = kOutOff + 2 * kOutBytes;
constexpr int kGroups = 4, kGWarps = 2;       // expander groups, which take the stages in turn, and their warps
constexpr int kGRows = 64 / (kGWarps * 4);    // K rows of a stage per expander thread
constexpr int kSigOff = kBarOff + 256;        // landing places of the follower's signals, and their source
constexpr int kDxSmem = kSigOff + 16 * (kNS * kGWarps + 1) + 1024;
constexpr int kDxThreads = (6 + kGroups * kGWarps) * 32;
static_assert(kDxSmem <= 232448, "shared memory budget");

struct DxMaps {
    CUtensorMap dy, g, v, x32, x16;
};
struct DxParams {
    const uint16_t *vals;
    const uint8_t *meta;
    float *part;               // [ks][M][d_in], ks > 1
    int32_t M, d_out, d_in;
    int32_t nk, nlr;           // K stages, rank stages
    int32_t n, ttiles, ks;     // tokens per tile, token tiles, K slices
    int32_t items;             // tiles x slices
    unsigned int *err;
};

// One tile's K slice.
struct DxItem {
    int32_t d0, tok0, k0, k1, lr, q;
    __device__ __forceinline__ DxItem(const DxParams &p, int w) {
        const int tile = w / p.ks;
        q = w - tile * p.ks;
        const int rt = tile / p.ttiles;
        d0 = rt * 2 * kCols;
        tok0 = (tile - rt * p.ttiles) * p.n;
        k0 = (int)((int64_t)p.nk * q / p.ks);
        k1 = (int)((int64_t)p.nk * (q + 1) / p.ks);
        lr = q == 0 ? p.nlr : 0;
    }
};

// Two kept values (v: low half first) at positions i0 < i1 of four, zeros
// elsewhere; nib = i0 | i1 << 2 in the low bits.
__device__ __forceinline__ uint2 expand_group(uint32_t v, uint32_t nib) {
    const uint32_t sel = 0x44444444u ^ (0x54u << ((nib << 3) & 0x18u)) ^ (0x76u << ((nib << 1) & 0x18u));
    return make_uint2(__byte_perm(v, 0, sel), __byte_perm(v, 0, sel >> 16));
}

// The verdicts of a group's threads joined: all go on, or none does and no named
// barrier is left waiting for one that gave up.
__device__ __forceinline__ bool group_and(uint32_t id, uint32_t n, bool ok) {
    uint32_t all;
    asm volatile(
        "{\n\t.reg .pred p, q;\n\t"
        "setp.ne.u32 p, %3, 0;\n\t"
        "barrier.cta.red.and.pred q, %1, %2, p;\n\t"
        "selp.u32 %0, 1, 0, q;\n\t}"
        : "=r"(all)
        : "r"(id), "r"(n), "r"((uint32_t)ok)
        : "memory");
    return all != 0;
}

__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kDxThreads, 1)
    input_backward_kernel(const __grid_constant__ DxMaps maps, const __grid_constant__ DxParams p) {
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bfull = reinterpret_cast<uint64_t *>(smem + kBarOff);   // leader: both CTAs' TMA bytes of a stage
    uint64_t *afull = bfull + kNS;       // leader: its expanders and the follower's signals
    uint64_t *empty = afull + kNS;       // the stage's MMAs are done (both CTAs)
    uint64_t *acc_full = empty + kNS;
    uint64_t *acc_empty = acc_full + 2;  // leader: drained by both CTAs' epilogues
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(acc_empty + 2);
    uint8_t *signals = smem + kSigOff;

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int half = p.n / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < kNS; ++s) {
            mbar_init(&bfull[s], 1);
            mbar_init(&afull[s], kGWarps);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 8);
        }
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        fence_proxy_async_smem();
    }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;" ::"r"(smem_u32(tmem_slot)),
                     "r"(512u));
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;");
    }
    tc_fence_before();
    cluster_sync_all();   // both CTAs' barriers initialised and TMEM allocated
    tc_fence_after();
    const uint32_t tmem_base = *tmem_slot;

    if (warp == 0) {
        // ------------------------------------------------------------ producer (each CTA)
        const uint32_t bar0 = mapa_shared(smem_u32(&bfull[0]), 0);
        uint32_t s = 0, ph = 0;
        bool ok = true, g_ready = false;
        for (int w = pair; w < p.items && ok; w += npairs) {
            const DxItem it(p, w);
            const int tok = it.tok0 + (int)rank * half, d0 = it.d0 + (int)rank * kCols;
            for (int i = it.k0; i < it.k1 + it.lr; ++i) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&empty[s], ph ^ 1))) {
                    if (lane == 0) atomicOr(p.err, 1u);
                    ok = false;
                    break;
                }
                const uint32_t a = smem_u32(smem + s * kStage), b = a + kABytes, bar = bar0 + s * 8;
                if (i >= it.k1 && !g_ready) {
                    asm volatile("griddepcontrol.wait;" ::: "memory");   // G may still be in production
                    g_ready = true;
                }
                if (elect_one()) {
                    if (i < it.k1) {
                        if (leader) mbar_expect_tx(&bfull[s], (uint32_t)p.n * 128u);
                        tma_load_2d_pair(&maps.dy, b, bar, i * kK, tok);
                    } else {
                        const int j = (i - it.k1) * kK;
                        if (leader) mbar_expect_tx(&bfull[s], (uint32_t)p.n * 128u + 2u * kABytes);
                        tma_load_2d_pair(&maps.v, a, bar, d0, j);
                        tma_load_2d_pair(&maps.v, a + kABytes / 2, bar, d0 + 64, j);
                        tma_load_2d_pair(&maps.g, b, bar, j, tok);
                    }
                }
                __syncwarp();
                if (++s == kNS) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else if (warp == 1) {
        // ------------------------------------------------------------ MMA issue (leader CTA)
        if (leader) {
            const uint32_t idesc = idesc_bf16(2 * kCols, p.n, false) | (1u << 15);   // A is MN-major
            uint32_t s = 0, ph = 0, aph = 0;   // aph: bit s, the phase of afull[s]
            int t = 0;
            bool ok = true;
            for (int w = pair; w < p.items && ok; w += npairs, ++t) {
                const DxItem it(p, w);
                const int buf = t & 1;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&acc_empty[buf], (uint32_t)(((t >> 1) & 1) ^ 1)));
                if (!ok) {
                    if (lane == 0) atomicOr(p.err, 2u);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * kMaxN);
                for (int i = it.k0; i < it.k1 + it.lr; ++i) {
                    bool got = mbar_wait_cluster(&bfull[s], ph);
                    if (got && i < it.k1) got = mbar_wait_cluster(&afull[s], (aph >> s) & 1u);
                    if (!__all_sync(0xFFFFFFFFu, got)) {
                        ok = false;
                        break;
                    }
                    if (i < it.k1) aph ^= 1u << s;
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + s * kStage), b = a + kABytes;
                    if (elect_one()) {
#pragma unroll
                        for (int c = 0; c < 4; ++c)   // K = 16 each: two 8-row groups of A, 32 bytes along B's rows
                            mma_dense_pair(d, desc_mn_sw128(a + 2048 * c), desc_sw128(b + 32 * c), idesc,
                                           (i > it.k0 || c > 0) ? 1u : 0u);
                        mma_commit_pair(&empty[s]);
                    }
                    __syncwarp();
                    if (++s == kNS) {
                        s = 0;
                        ph ^= 1;
                    }
                }
                if (!ok) {
                    if (lane == 0) atomicOr(p.err, 4u);
                    break;
                }
                if (elect_one()) mma_commit_pair(&acc_full[buf]);
                __syncwarp();
            }
        }
    } else if (warp < 6) {
        // ------------------------------------------------------------ epilogue (each CTA, its 128 columns)
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;   // input column within the CTA's tile
        const bool store_thread = warp == 2 && lane == 0;
        const uint32_t empty0 = mapa_shared(smem_u32(&acc_empty[0]), 0);
        uint32_t piece = 0;
        int t = 0;
        for (int w = pair; w < p.items; w += npairs, ++t) {
            const DxItem it(p, w);
            const int d0 = it.d0 + (int)rank * kCols;
            const int buf = t & 1;
            const bool ok = group_and(1, 128, mbar_wait_cluster(&acc_full[buf], (uint32_t)((t >> 1) & 1)));
            if (!ok) {
                if (lane == 0) atomicOr(p.err, 8u);
                break;
            }
            tc_fence_after();
            const uint32_t acc = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)(buf * kMaxN);
            const int nq = (p.n + 31) / 32;
#pragma unroll 1
            for (int q = 0; q < nq; ++q) {
                const bool wide = p.n - q * 32 >= 32;   // else a last piece of 16 tokens
                uint32_t v[32];
                if (wide) {
                    tmem_ld_32x32b_x32(acc + (uint32_t)(q * 32), v);
                } else {
                    uint32_t h[16];
                    tmem_ld_32x32b_x16(acc + (uint32_t)(q * 32), h);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = h[j];
                }
                if (q == nq - 1) {
                    tc_fence_before();
                    __syncwarp();
                    if (lane == 0) mbar_arrive_remote_relaxed(empty0 + (uint32_t)(buf * 8));
                }
                const int tq = it.tok0 + q * 32, lim = min(p.M, it.tok0 + p.n);
                if (tq >= lim) continue;   // uniform across the epilogue warps
                if (p.ks > 1) {
                    if (d0 + row < p.d_in) {
                        float *dst = p.part + ((int64_t)it.q * p.M + tq) * p.d_in + d0 + row;
#pragma unroll
                        for (int j = 0; j < 32; ++j)
                            if (tq + j < lim && (wide || j < 16)) dst[(int64_t)j * p.d_in] = __uint_as_float(v[j]);
                    }
                    continue;
                }
                if (store_thread) bulk_wait_read1();
                named_bar_sync(2, 128);
                uint16_t *out = reinterpret_cast<uint16_t *>(smem + kOutOff + (piece & 1) * kOutBytes);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (wide || j < 16) out[j * kCols + row] = f32_to_bf16_bits(__uint_as_float(v[j]));
                fence_proxy_async_smem();
                named_bar_sync(2, 128);
                if (store_thread) {
                    tma_store_2d(wide ? &maps.x32 : &maps.x16, smem_u32(out), d0, tq);
                    bulk_commit();
                }
                ++piece;
            }
        }
        if (store_thread) bulk_wait_all();
    } else {
        // ------------------------------------------------------------ expanders (each CTA, its 128 columns)
        // Eight consecutive threads write two K rows (k, k + 1) of one 64-column
        // panel: their 16-byte stores fall into eight different bank groups.
        const int grp = (warp - 6) / kGWarps, gw = (warp - 6) % kGWarps;
        const int e = gw * 32 + lane;
        const int krow = (e >> 4) * 2 + ((e >> 2) & 1);              // and every 4 * kGWarps rows after it
        const int col = ((e >> 3) & 1) * 64 + (e & 3) * 16;
        const uint32_t off = (uint32_t)(((e >> 3) & 1) * (kABytes / 2) + krow * 128);
        const uint32_t c0 = off + (uint32_t)((((e & 3) * 2) ^ (krow & 7)) * 16);
        const uint32_t c1 = off + (uint32_t)((((e & 3) * 2 + 1) ^ (krow & 7)) * 16);
        const uint32_t afull0 = mapa_shared(smem_u32(&afull[0]), 0), sig0 = mapa_shared(smem_u32(signals), 0);
        const uint32_t sig_src = smem_u32(signals + 16 * kNS * kGWarps);
        const int64_t vld = p.d_in / 2, mld = p.d_in / 8;
        // Stage number `pos` of the pair's sequence sits in slot pos % kNS and
        // belongs to group pos % kGroups.  A group waits for every slot of its
        // turns, rank stages too: a skipped phase could be taken for the next.
        uint32_t pos = 0;    // of the item's first stage
        bool ok = true;
        for (int w = pair; w < p.items && ok; w += npairs) {
            const DxItem it(p, w);
            const int d = it.d0 + (int)rank * kCols + col;
            const bool in = d < p.d_in;
            const uint16_t *vp = p.vals + (int64_t)krow * vld + d / 2;
            const uint8_t *mp = p.meta + (int64_t)krow * mld + d / 8;
            uint4 v[kGRows];
            uint32_t m[kGRows];
            auto load = [&](int h, int i) {
                const int64_t k = (int64_t)i * kK + 4 * kGWarps * h;
                v[h] = make_uint4(0, 0, 0, 0);
                m[h] = 0x4444u;   // a valid pattern for the zeros
                if (in && i < it.k1 && k + krow < p.d_out) {
                    v[h] = ld_stream_v4(vp + k * vld);
                    m[h] = __ldg(reinterpret_cast<const unsigned short *>(mp + k * mld));
                }
            };
            const int first = (int)((uint32_t)(grp - (int)pos) % kGroups), nst = it.k1 - it.k0 + it.lr;
#pragma unroll
            for (int h = 0; h < kGRows; ++h) load(h, it.k0 + first);
            for (int i = first; i < nst; i += kGroups) {
                const uint32_t at = pos + (uint32_t)i, s = at % kNS, use = at / kNS;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&empty[s], (use & 1) ^ 1))) {
                    if (lane == 0) atomicOr(p.err, 16u);
                    ok = false;
                    break;
                }
                if (it.k0 + i >= it.k1) continue;   // a rank stage
                uint8_t *a = smem + s * kStage;
#pragma unroll
                for (int h = 0; h < kGRows; ++h) {
                    const uint2 g0 = expand_group(v[h].x, m[h]), g1 = expand_group(v[h].y, m[h] >> 4);
                    const uint2 g2 = expand_group(v[h].z, m[h] >> 8), g3 = expand_group(v[h].w, m[h] >> 12);
                    *reinterpret_cast<uint4 *>(a + c0 + h * (4 * kGWarps * 128)) = make_uint4(g0.x, g0.y, g1.x, g1.y);
                    *reinterpret_cast<uint4 *>(a + c1 + h * (4 * kGWarps * 128)) = make_uint4(g2.x, g2.y, g3.x, g3.y);
                    load(h, it.k0 + i + kGroups);
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    if (!leader)
                        bulk_signal_peer(sig0 + 16 * (s * kGWarps + gw), sig_src, afull0 + s * 8);
                    else if (gw == 0)
                        mbar_expect_tx(&afull[s], 16 * kGWarps);
                    else
                        mbar_arrive(&afull[s]);
                }
            }
            pos += (uint32_t)nst;
        }
    }

    tc_fence_before();
    cluster_sync_all();   // the pair's MMAs, signals and stores are done before TMEM is freed
    if (warp == 1) {
        tc_fence_after();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(512u));
    }
}

// dX = the sum over the K slices, in slice order, rounded to bf16.
__global__ void __launch_bounds__(256) input_backward_sum_kernel(const float *__restrict__ part, int ks, int64_t total,
                                                                uint16_t *__restrict__ dX) {
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int64_t e = ((int64_t)blockIdx.x * 256 + threadIdx.x) * 4;
    if (e >= total) return;
    float4 acc = make_float4(0.f, 0.f, 0.f, 0.f);
    for (int q = 0; q < ks; ++q) {
        const uint4 v = ld_dep_v4(part + q * total + e);
        acc.x += __uint_as_float(v.x);
        acc.y += __uint_as_float(v.y);
        acc.z += __uint_as_float(v.z);
        acc.w += __uint_as_float(v.w);
    }
    uint2 o;
    o.x = (uint32_t)f32_to_bf16_bits(acc.x) | ((uint32_t)f32_to_bf16_bits(acc.y) << 16);
    o.y = (uint32_t)f32_to_bf16_bits(acc.z) | ((uint32_t)f32_to_bf16_bits(acc.w) << 16);
    *reinterpret_cast<uint2 *>(dX + e) = o;
}

}  // namespace

// Tokens per tile and K slices for a problem, by the estimated cycles of the
// busiest pair: rounds of tiles x stages, a stage at the larger of its MMAs (2 n
// cycles), its bytes at the 44 a cycle that an SM takes in, and the expanders
// (~240); a slice's partial tile and the second kernel cost extra.
DxPlan input_backward_plan(int64_t M, int64_t d_out, int64_t d_in, int64_t r, int sms) {
    const int64_t ut = (M + 15) / 16, rows = (d_in + 255) / 256, nk = (d_out + kK - 1) / kK, nlr = (r + 63) / 64;
    const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
    DxPlan best{0, 0, 1};
    double best_cost = 0;
    const int64_t tmin = (ut + kMaxN / 16 - 1) / (kMaxN / 16);
    for (int64_t tt = tmin; tt <= tmin + 6 && tt <= ut; ++tt) {
        const int64_t nu = (ut + tt - 1) / tt, ttiles = (ut + nu - 1) / nu;
        const double n = 16.0 * nu, bytes = (9216.0 + 64.0 * n) / 44.0;
        double stage = 2.0 * n > bytes ? 2.0 * n : bytes;
        if (stage < 240.0) stage = 240.0;
        for (int64_t ks = 1; ks <= 8 && ks * 4 <= nk + 3; ++ks) {
            const int64_t rounds = (rows * ttiles * ks + pairs - 1) / pairs;
            double cost = rounds * (((nk + ks - 1) / ks + nlr) * stage + 1500.0);
            if (ks > 1) cost += 5000.0 + (double)ks * M * d_in * 8.0 / (pairs * 40.0);
            if (best.n == 0 || cost < best_cost) {
                best = DxPlan{(int)(16 * nu), (int)ttiles, (int)ks};
                best_cost = cost;
            }
        }
    }
    return best;
}

size_t input_backward_workspace(int64_t M, int64_t d_out, int64_t d_in, int64_t r, int sms) {
    const DxPlan plan = input_backward_plan(M, d_out, d_in, r, sms);
    const size_t g = ((size_t)M * (size_t)r * 2 + 255) / 256 * 256;
    return g + (plan.ks > 1 ? (size_t)plan.ks * M * d_in * 4 : 0);
}

cudaError_t launch_input_backward(const uint16_t *dY, int64_t M, const uint16_t *vals, const uint8_t *meta, int64_t d_out,
                                  int64_t d_in, const uint16_t *U, const uint16_t *V, int64_t r, uint16_t *dX, uint8_t *ws,
                                  int sms, cudaStream_t stream) {
    if (dx_err() == nullptr) return cudaErrorInvalidValue;
    uint16_t *G = reinterpret_cast<uint16_t *>(ws);
    if (r > 0) {
        // G = dY U (A = dY K-major, K = d_out; B = U [d_out][r] MN-major).
        cudaError_t e;
        if (r <= 64)
            e = gemm_tc<false, true, 64, kOutBF16>(dY, nullptr, d_out, U, nullptr, r, M, r, d_out, G, dx_err(), stream);
        else if (r <= 128)
            e = gemm_tc<false, true, 128, kOutBF16>(dY, nullptr, d_out, U, nullptr, r, M, r, d_out, G, dx_err(), stream);
        else
            e = gemm_tc<false, true, 256, kOutBF16>(dY, nullptr, d_out, U, nullptr, r, M, r, d_out, G, dx_err(), stream);
        if (e != cudaSuccess) return e;
    }
    const DxPlan plan = input_backward_plan(M, d_out, d_in, r, sms);
    DxMaps maps;
    memset(&maps, 0, sizeof maps);
    bool ok = make_map(&maps.dy, kBF16, dY, d_out, M, d_out * 2, 64, plan.n / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
              make_map(&maps.x32, kBF16, dX, d_in, M, d_in * 2, kCols, 32, CU_TENSOR_MAP_SWIZZLE_NONE) &&
              make_map(&maps.x16, kBF16, dX, d_in, M, d_in * 2, kCols, 16, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (ok && r > 0)
        ok = make_map(&maps.g, kBF16, G, r, M, r * 2, 64, plan.n / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map(&maps.v, kBF16, V, d_in, r, d_in * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return cudaErrorInvalidValue;
    DxParams p;
    p.vals = vals;
    p.meta = meta;
    p.part = reinterpret_cast<float *>(ws + ((size_t)M * (size_t)r * 2 + 255) / 256 * 256);
    p.M = (int32_t)M;
    p.d_out = (int32_t)d_out;
    p.d_in = (int32_t)d_in;
    p.nk = (int32_t)((d_out + kK - 1) / kK);
    p.nlr = (int32_t)((r + 63) / 64);
    p.n = plan.n;
    p.ttiles = plan.ttiles;
    p.ks = plan.ks;
    const int64_t items = (d_in + 255) / 256 * plan.ttiles * plan.ks;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    p.items = (int32_t)items;
    p.err = dx_err();
    cudaError_t err =
        cudaFuncSetAttribute(input_backward_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, kDxSmem);
    if (err != cudaSuccess) return err;
    const int64_t pairs = items < sms / 2 ? items : sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(kDxThreads);
    cfg.dynamicSmemBytes = kDxSmem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = r > 0 ? 1 : 0;   // the kernel just before is the one that writes G
    err = cudaLaunchKernelEx(&cfg, input_backward_kernel, maps, p);
    if (err != cudaSuccess || plan.ks == 1) return err;
    const int64_t total = M * d_in;
    cfg.gridDim = dim3((unsigned)((total + 1023) / 1024));
    cfg.blockDim = dim3(256);
    cfg.dynamicSmemBytes = 0;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, input_backward_sum_kernel, (const float *)p.part, (int)plan.ks, total, dX);
}

cudaError_t read_and_clear_dx_error(unsigned *code) {
    unsigned v = 0;
    cudaError_t err = cudaMemcpyFromSymbol(&v, g_dx_error, sizeof v);
    if (err != cudaSuccess) return err;
    if (v != 0) {
        const unsigned zero = 0;
        err = cudaMemcpyToSymbol(g_dx_error, &zero, sizeof zero);
    }
    *code = v;
    return err;
}

}  // namespace slr
