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
//   D = dX^T tile 256 x n fp32 in TMEM: two accumulators of up to 256 tokens, or
//                 two 256-column halves over the same tokens (up to 240), which
//                 read the dY tile once for twice the MMAs.
// After the d_out / 64 stages of S, ceil(r / 64) rank stages add A = V tile (64
// ranks x 256 columns, MN-major, by TMA), B = G tile.  G is formed before by the
// product kernel of the factors' gradients (tc_gemm.cuh) and rounded to bf16, as
// there: the tensor cores read bf16.  This kernel starts beside it on the SMs it
// leaves free and waits for it before the rank stages.
//
// A cluster of two CTAs on neighbouring SMs shares a tile (cta_group::2): each
// expands its half of the columns and loads half of the tokens.
//   warp 0       TMA producer (dY; V and G),
//   warp 1       MMA issue (leader CTA),
//   warps 2..9   epilogue: TMEM -> bf16 -> shared memory -> TMA store,
//   warps 10..   expanders, in groups that take the stages in turn: a thread
//                reads 16 bytes of kept values (four groups of S) and their two
//                metadata bytes from shared memory and writes 32 bytes of the
//                dense tile in the 128-byte swizzle,
//   last warp    TMA producer of the packed values.
// The follower's expanders announce a stage to the leader with 16-byte bulk
// copies that complete on its barrier, since a release-ordered remote arrive
// would stall them for most of a microsecond each.
//
// What bounds it: a stage of two halves takes about 1040 cycles whatever its tokens,
// for the expansion (reads, permutes and writes of shared memory); of one half, 620.
// Its MMAs take 2 n cycles a half, its 34 KB of dY, values and metadata (240 tokens)
// 890.  So at 240 tokens the tensor pipe is the bound beside it (87.5% active for
// 2048 tokens of 14336 x 4096), at 160 the expansion (55% active, the ALU pipe 60%,
// shared memory 45%, for 777 tokens of 4096 x 14336, 96 us), at 64 the expansion and
// the three launches (10% active, 64 tokens of 4096 x 4096, 15 us).  Measured, 2048 tokens of 14336 x 4096 without the rank term: 165 us = 1461 TF/s of the
// dense product (cuBLAS: 1670), 180 with it (r = 64).  Steps on the way there:
// all of S by 16-byte loads 186 us, one half 193, eight warps on every stage
// instead of groups in turn 252.
//
// Few tiles (short batches): the K stages are split over the pairs that would
// idle; slices leave fp32 partial tiles in the workspace, which a second kernel
// adds in slice order.
//
// Every wait is bounded; on expiry an error word is set (slr_check_kernel_error).
#include <cuda.h>

#include <cstdlib>
#include <cstring>

#include "tc_gemm.cuh"

namespace slr {

// Error word of this file's bounded waits (read by slr_check_kernel_error).
__device__ unsigned int g_dx_error = 0;

namespace {

unsigned int *dx_err() {
    static std::atomic<unsigned int *> at[kMaxCachedDevices] = {};
    return device_address(g_dx_error, at);
}

constexpr int kCols = 128;                    // input columns per CTA and half
constexpr int kK = 64;                        // output rows (K) per stage
constexpr int kABytes = kCols * kK * 2;       // 16 KB per half: two 64-column panels of 64 K rows
constexpr int kOutBytes = 32 * kCols * 2;     // 32 tokens x 128 columns
constexpr int kValBytes = kK * kCols;         // packed values of a stage and half: 64 rows of 128 bytes
constexpr int kMetaTurns = 2;                 // turns that an expander warp's metadata (32 rows of 16 bytes) is ahead
constexpr int kEWarps = 8;                    // epilogue warps, two groups of four
constexpr int kXFirst = 2 + kEWarps;          // first expander warp

// H = 1: tiles of 256 columns, two accumulators of up to 256 tokens.  H = 2: two
// such halves over the same tokens, one accumulator each of up to 240.
template <int H>
struct DxCfg {
    static constexpr int MAXN = H == 1 ? 256 : 240;
    static constexpr int B_BYTES = MAXN / 2 * kK * 2;
    static constexpr int STAGE = H * kABytes + B_BYTES;
    static constexpr int NS = H == 1 ? 4 : 3;
    static constexpr int NACC = H == 1 ? 2 : 1;
    // Expanders: groups, which take the stages in turn, of GWARPS warps, WPH to a
    // half; a thread has ROWS of the stage's K rows, eight apart.  (Two halves
    // with 8 warps in all: 172 us where 16 take 166, one half with 16 warps 17.6
    // us where 8 take 14.9 -- 2048 tokens of 14336 x 4096, 64 of 4096 x 4096, r = 0.)
    static constexpr int WPH = 2 * H, GWARPS = WPH * H, GROUPS = H == 1 ? 4 : 2, XWARPS = GWARPS * GROUPS;
    static constexpr int ROWS = 16 / WPH;
    static constexpr int THREADS = (3 + kEWarps + XWARPS) * 32;
    static constexpr int OUT_OFF = NS * STAGE;
    static constexpr int RAW_OFF = OUT_OFF + 2 * kOutBytes;   // ring of packed values
    static constexpr int NR = H == 1 ? 6 : 3;
    static constexpr int META_OFF = RAW_OFF + NR * H * kValBytes;
    static constexpr int BAR_OFF = META_OFF + XWARPS * kMetaTurns * ROWS * 64;
    static constexpr int SIG_OFF = BAR_OFF + 256;     // landing places of the follower's signals, and their source
    static constexpr int SMEM = SIG_OFF + 16 * (NS * GWARPS + 1) + 1024;
    static_assert(STAGE % 1024 == 0 && B_BYTES % 1024 == 0, "swizzled tiles start on 1 KB");
    static_assert(SMEM <= 232448, "shared memory budget");
    static_assert((3 * NS + 4 + 2 * NR) * 8 + 4 <= 256, "barrier area");
    static_assert(RAW_OFF % 1024 == 0, "swizzled tiles start on 1 KB");
    // A group's wait at its turn before (GROUPS positions back, for the slot's
    // use NS before that) must imply the use two before the present one, or its
    // parity could be taken for the next.
    static_assert(GROUPS <= NS, "a wait's parity would be ambiguous");
    // Likewise for the packed values: a group passes over the other groups' uses
    // of a slot, but the MMAs NS positions back, which it has waited for, came
    // after the landing of every use at least NS stages of S back.
    static_assert(NR >= NS, "a wait's parity would be ambiguous");
};

struct DxMaps {
    CUtensorMap dy, g, v, x32, x16, vals;
};
struct DxParams {
    const uint8_t *meta;
    float *part;               // [ks][M][d_in], ks > 1
    int32_t M, d_out, d_in;
    int32_t nk, nlr;           // K stages, rank stages
    int32_t n, ttiles, ks;     // tokens per tile, token tiles, K slices
    int32_t items;             // tiles x slices
    unsigned int *err;
};

// One tile's K slice.
template <int H>
struct DxItem {
    int32_t d0, tok0, k0, k1, lr, q;
    __device__ __forceinline__ DxItem(const DxParams &p, int w) {
        const int tile = w / p.ks;
        q = w - tile * p.ks;
        const int rt = tile / p.ttiles;
        d0 = rt * 2 * H * kCols;
        tok0 = (tile - rt * p.ttiles) * p.n;
        k0 = (int)((int64_t)p.nk * q / p.ks);
        k1 = (int)((int64_t)p.nk * (q + 1) / p.ks);
        lr = q == 0 ? p.nlr : 0;
    }
};

// Four groups of S from packed to dense: v holds the two kept values of each (low
// half first), m their index nibbles i0 | i1 << 2; out the 16 columns.
//
// A byte permute of (v, 0) with selector byte pair 0x10 (first value), 0x32
// (second) or 0x44 (zero) for each position places a group's values, so the work
// is in finding the selectors, for four groups at once: the six valid nibbles
// have different low three bits in Gray code (n ^ n >> 1: (0,1) 6, (0,2) 4,
// (1,2) 5, (0,3) 2, (1,3) 3, (2,3) 1), which one permute per position looks up
// in a table of eight bytes, one byte per group.  22 operations for 16 columns;
// selectors by shifts and exclusive ors took 46 and bound the kernel (205 us
// where 154 remained without them; integer operations issue at half rate).
__device__ __forceinline__ void expand4(const uint4 &v, uint32_t m, uint4 &lo, uint4 &hi) {
    const uint32_t g = (m ^ (m >> 1)) & 0x7777u;
    const uint32_t p0 = __byte_perm(0x44104444u, 0x44104410u, g), p1 = __byte_perm(0x10444444u, 0x44321044u, g);
    const uint32_t p2 = __byte_perm(0x44441044u, 0x44443232u, g), p3 = __byte_perm(0x32323244u, 0x44444444u, g);
    const uint32_t a = __byte_perm(p0, p1, 0x5140), b = __byte_perm(p0, p1, 0x7362);   // positions 0, 1 of groups 0, 1; 2, 3
    const uint32_t c = __byte_perm(p2, p3, 0x5140), d = __byte_perm(p2, p3, 0x7362);   // positions 2, 3
    lo = make_uint4(__byte_perm(v.x, 0, a), __byte_perm(v.x, 0, c), __byte_perm(v.y, 0, a >> 16), __byte_perm(v.y, 0, c >> 16));
    hi = make_uint4(__byte_perm(v.z, 0, b), __byte_perm(v.z, 0, d), __byte_perm(v.w, 0, b >> 16), __byte_perm(v.w, 0, d >> 16));
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

template <int H>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(DxCfg<H>::THREADS, 1)
    input_backward_kernel(const __grid_constant__ DxMaps maps, const __grid_constant__ DxParams p) {
    using C = DxCfg<H>;
    using Item = DxItem<H>;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint64_t *bfull = reinterpret_cast<uint64_t *>(smem + C::BAR_OFF);   // leader: both CTAs' TMA bytes of a stage
    uint64_t *afull = bfull + C::NS;       // leader: its expanders and the follower's signals
    uint64_t *empty = afull + C::NS;       // the stage's MMAs are done (both CTAs)
    uint64_t *acc_full = empty + C::NS;
    uint64_t *acc_empty = acc_full + 2;  // leader: drained by both CTAs' epilogues
    uint64_t *raw_full = acc_empty + 2;  // packed values landed / read by the group's warps (each CTA)
    uint64_t *raw_empty = raw_full + C::NR;
    uint32_t *tmem_slot = reinterpret_cast<uint32_t *>(raw_empty + C::NR);
    uint8_t *signals = smem + C::SIG_OFF;

    // The kernel that adds the slices may be scheduled now; it waits for this
    // grid before it reads a partial tile.
    asm volatile("griddepcontrol.launch_dependents;");
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_ctarank();
    const bool leader = rank == 0;
    const int pair = blockIdx.x >> 1, npairs = gridDim.x >> 1;
    const int half = p.n / 2;

    if (threadIdx.x == 0) {
        for (int s = 0; s < C::NS; ++s) {
            mbar_init(&bfull[s], 1);
            mbar_init(&afull[s], C::GWARPS);
            mbar_init(&empty[s], 1);
        }
        for (int b = 0; b < 2; ++b) {
            mbar_init(&acc_full[b], 1);
            mbar_init(&acc_empty[b], 2 * kEWarps);
        }
        for (int s = 0; s < C::NR; ++s) {
            mbar_init(&raw_full[s], 1);
            mbar_init(&raw_empty[s], C::GWARPS);
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
            const Item it(p, w);
            const int tok = it.tok0 + (int)rank * half, d0 = it.d0 + (int)rank * kCols;
            for (int i = it.k0; i < it.k1 + it.lr; ++i) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&empty[s], ph ^ 1))) {
                    if (lane == 0) atomicOr(p.err, 1u);
                    ok = false;
                    break;
                }
                const uint32_t a = smem_u32(smem + s * C::STAGE), b = a + H * kABytes, bar = bar0 + s * 8;
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
                        if (leader) mbar_expect_tx(&bfull[s], (uint32_t)p.n * 128u + 2u * H * kABytes);
#pragma unroll
                        for (int h = 0; h < 2 * H; ++h)   // 64-column panels, two to a half
                            tma_load_2d_pair(&maps.v, a + h * (kABytes / 2), bar, d0 + (h >> 1) * 2 * kCols + (h & 1) * 64, j);
                        tma_load_2d_pair(&maps.g, b, bar, j, tok);
                    }
                }
                __syncwarp();
                if (++s == C::NS) {
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
                const Item it(p, w);
                const int buf = C::NACC == 2 ? t & 1 : 0;
                ok = __all_sync(0xFFFFFFFFu, mbar_wait_cluster(&acc_empty[buf], (uint32_t)((t / C::NACC & 1) ^ 1)));
                if (!ok) {
                    if (lane == 0) atomicOr(p.err, 2u);
                    break;
                }
                tc_fence_after();
                const uint32_t d = tmem_base + (uint32_t)(buf * C::MAXN);
                for (int i = it.k0; i < it.k1 + it.lr; ++i) {
                    bool got = mbar_wait_cluster(&bfull[s], ph);
                    if (got && i < it.k1) got = mbar_wait_cluster(&afull[s], (aph >> s) & 1u);
                    if (!__all_sync(0xFFFFFFFFu, got)) {
                        ok = false;
                        break;
                    }
                    if (i < it.k1) aph ^= 1u << s;
                    tc_fence_after();
                    const uint32_t a = smem_u32(smem + s * C::STAGE), b = a + H * kABytes;
                    if (elect_one()) {
#pragma unroll
                        for (int h = 0; h < H; ++h)
#pragma unroll
                            for (int c = 0; c < 4; ++c)   // K = 16 each: two 8-row groups of A, 32 bytes along B's rows
                                mma_dense_pair(d + h * C::MAXN, desc_mn_sw128(a + h * kABytes + 2048 * c),
                                               desc_sw128(b + 32 * c), idesc, (i > it.k0 || c > 0) ? 1u : 0u);
                        mma_commit_pair(&empty[s]);
                    }
                    __syncwarp();
                    if (++s == C::NS) {
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
    } else if (warp < kXFirst) {
        // ------------------------------------------------------------ epilogue (each CTA, its 128 columns)
        // Two groups of four warps (one per TMEM lane quarter): each drains one
        // half, or every other piece of a tile of one half.
        const int grp = (warp - 2) >> 2, quarter = warp & 3;
        const int row = quarter * 32 + lane;   // input column within the CTA's tile
        const bool store_thread = ((warp - 2) & 3) == 0 && lane == 0;
        uint16_t *out = reinterpret_cast<uint16_t *>(smem + C::OUT_OFF + grp * kOutBytes);
        const uint32_t empty0 = mapa_shared(smem_u32(&acc_empty[0]), 0);
        int t = 0;
        for (int w = pair; w < p.items; w += npairs, ++t) {
            const Item it(p, w);
            const int buf = C::NACC == 2 ? t & 1 : 0;
            const bool ok = group_and(1 + grp, 128, mbar_wait_cluster(&acc_full[buf], (uint32_t)(t / C::NACC & 1)));
            if (!ok) {
                if (lane == 0) atomicOr(p.err, 8u);
                break;
            }
            tc_fence_after();
            const int nq = (p.n + 31) / 32;
            if (H == 1 && grp >= nq) {   // one piece: nothing for the second group
                tc_fence_before();
                if (lane == 0) mbar_arrive_remote_relaxed(empty0 + (uint32_t)(buf * 8));
            }
#pragma unroll 1
            for (int q = H == 1 ? grp : 0; q < nq; q += H == 1 ? 2 : 1) {
                const int h = H == 1 ? 0 : grp;
                const int d0 = it.d0 + h * 2 * kCols + (int)rank * kCols;
                const uint32_t acc = tmem_base + ((uint32_t)(quarter * 32) << 16) + (uint32_t)((buf + h) * C::MAXN);
                const bool wide = p.n - q * 32 >= 32;   // else a last piece of 16 tokens
                uint32_t v[32];
                if (wide) {
                    tmem_ld_32x32b_x32(acc + (uint32_t)(q * 32), v);
                } else {
                    uint32_t u[16];
                    tmem_ld_32x32b_x16(acc + (uint32_t)(q * 32), u);
#pragma unroll
                    for (int j = 0; j < 16; ++j) v[j] = u[j];
                }
                if (q + (H == 1 ? 2 : 1) >= nq) {
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
                if (store_thread) bulk_wait_read0();
                named_bar_sync(3 + grp, 128);
#pragma unroll
                for (int j = 0; j < 32; ++j)
                    if (wide || j < 16) out[j * kCols + row] = f32_to_bf16_bits(__uint_as_float(v[j]));
                fence_proxy_async_smem();
                named_bar_sync(3 + grp, 128);
                if (store_thread) {
                    tma_store_2d(wide ? &maps.x32 : &maps.x16, smem_u32(out), d0, tq);
                    bulk_commit();
                }
            }
        }
        if (store_thread) bulk_wait_all();
    } else if (warp == kXFirst + C::XWARPS) {
        // ------------------------------------------------------------ packed values (each CTA)
        uint32_t s = 0, ph = 0;
        bool ok = true;
        for (int w = pair; w < p.items && ok; w += npairs) {
            const Item it(p, w);
            const int d0 = it.d0 + (int)rank * kCols;
            for (int i = it.k0; i < it.k1; ++i) {
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&raw_empty[s], ph ^ 1))) {
                    if (lane == 0) atomicOr(p.err, 32u);
                    ok = false;
                    break;
                }
                if (elect_one()) {
                    mbar_expect_tx(&raw_full[s], H * kValBytes);
#pragma unroll
                    for (int h = 0; h < H; ++h)
                        tma_load_2d(&maps.vals, smem_u32(smem + C::RAW_OFF + (s * H + h) * kValBytes), &raw_full[s],
                                    (d0 + h * 2 * kCols) / 2, i * kK);
                }
                __syncwarp();
                if (++s == C::NR) {
                    s = 0;
                    ph ^= 1;
                }
            }
        }
    } else {
        // ------------------------------------------------------------ expanders (each CTA, its 128 columns)
        // A thread's 16 bytes of row k of the packed tile become two 16-byte pieces
        // of row k of the dense one, both in the 128-byte swizzle.  Eight
        // consecutive threads take rows k and k ^ 5 of one 64-column panel: bit 2
        // tells their reads apart, bit 0 their writes, so that each falls into
        // eight different bank groups.
        const int grp = (warp - kXFirst) / C::GWARPS, gw = (warp - kXFirst) % C::GWARPS;
        const int mine = ((lane >> 4) & 1) + (gw & 1) * 2;           // the pair of rows, of eight
        const int krow = ((lane >> 2) & 1) ? mine ^ 5 : mine;        // and every eighth row after it
        const int panel = (lane >> 3) & 1, quad = lane & 3;
        const int base = C::WPH == 4 ? (gw & 2) * 16 : 0;            // four warps to a half: its first or second 32 rows
        const int half = gw / C::WPH, hcol = half * 2 * kCols;                      // the warp's half
        const uint32_t off = (uint32_t)(half * kABytes + panel * (kABytes / 2) + (base + krow) * 128);
        const uint32_t c0 = off + (uint32_t)(((quad * 2) ^ krow) * 16);
        const uint32_t c1 = off + (uint32_t)(((quad * 2 + 1) ^ krow) * 16);
        const uint32_t rv = (uint32_t)(half * kValBytes + (base + krow) * 128 + (((panel * 4 + quad) ^ krow) * 16));
        // The warp's metadata come by cp.async, 16 bytes a lane: K row
        // `mrow(lane)`, the lanes of a row pair in the pairs' order.  (As TMA boxes
        // the 16-byte rows would cost as much as the 128-byte rows of the values;
        // two-byte loads into registers, and all of S by 16-byte loads, held the
        // SM's intake to 52 GB/s, where TMA takes in 66.)
        uint8_t *meta0 = smem + C::META_OFF + (warp - kXFirst) * (kMetaTurns * C::ROWS * 64);
        const int mpair = ((lane >> 1) & 1) + (gw & 1) * 2;
        const int mrow = base + ((lane & 1) ? mpair ^ 5 : mpair) + 8 * (lane >> 2);   // of ROWS eights
        const uint32_t rm = (uint32_t)((((lane >> 4) & 1) * 2 + ((lane >> 2) & 1)) * 16 + panel * 8 + quad * 2);
        const uint32_t afull0 = mapa_shared(smem_u32(&afull[0]), 0), sig0 = mapa_shared(smem_u32(signals), 0);
        const uint32_t sig_src = smem_u32(signals + 16 * C::NS * C::GWARPS);
        const int64_t mld = p.d_in / 8;
        // Stage number `pos` of the pair's sequence sits in slot pos % NS and
        // belongs to group pos % GROUPS.  A group waits for every slot of its
        // turns, rank stages too: a skipped phase could be taken for the next.
        uint32_t pos = 0;    // of the item's first stage
        uint32_t rpos = 0;   // its number among the stages of S: the packed values' ring
        bool ok = true;
        for (int w = pair; w < p.items && ok; w += npairs) {
            const Item it(p, w);
            const int d = it.d0 + (int)rank * kCols + hcol;
            const bool in = d < p.d_in;
            // Rows past d_out and stages past the slice come as zeros, which place
            // zeros.
            auto copy = [&](int b, int i) {
                if (i < it.k1 && lane < 4 * C::ROWS) {
                    const int64_t k = (int64_t)i * kK + mrow;
                    const bool there = in && k < p.d_out;
                    const uint8_t *src = there ? p.meta + k * mld + d / 8 : p.meta;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(smem_u32(meta0 + b * C::ROWS * 64 + lane * 16)),
                                 "l"(src), "r"(there ? 16 : 0)
                                 : "memory");
                }
                asm volatile("cp.async.commit_group;" ::: "memory");
            };
            const int first = (grp + C::GROUPS - (int)(pos % C::GROUPS)) % C::GROUPS, nst = it.k1 - it.k0 + it.lr;
            int b = 0;
#pragma unroll
            for (int t = 0; t < kMetaTurns; ++t) copy(t, it.k0 + first + t * C::GROUPS);
            for (int i = first; i < nst; i += C::GROUPS) {
                const uint32_t at = pos + (uint32_t)i, s = at % C::NS, use = at / C::NS;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait_cluster(&empty[s], (use & 1) ^ 1))) {
                    if (lane == 0) atomicOr(p.err, 16u);
                    ok = false;
                    break;
                }
                if (it.k0 + i >= it.k1) continue;   // a rank stage
                asm volatile("cp.async.wait_group %0;" ::"n"(kMetaTurns - 1) : "memory");
                const uint32_t rat = rpos + (uint32_t)i, rs = rat % C::NR;
                if (!__all_sync(0xFFFFFFFFu, mbar_wait(&raw_full[rs], (rat / C::NR) & 1))) {
                    if (lane == 0) atomicOr(p.err, 64u);
                    ok = false;
                    break;
                }
                __syncwarp();
                uint8_t *a = smem + s * C::STAGE;
                const uint8_t *raw = smem + C::RAW_OFF + rs * (H * kValBytes), *meta = meta0 + b * C::ROWS * 64;
#pragma unroll
                for (int h = 0; h < C::ROWS; ++h) {
                    const uint4 v = *reinterpret_cast<const uint4 *>(raw + rv + h * 1024);
                    const uint32_t m = *reinterpret_cast<const uint16_t *>(meta + rm + h * 64);
                    uint4 lo, hi;
                    expand4(v, m, lo, hi);
                    *reinterpret_cast<uint4 *>(a + c0 + h * 1024) = lo;
                    *reinterpret_cast<uint4 *>(a + c1 + h * 1024) = hi;
                }
                fence_proxy_async_smem();
                __syncwarp();
                if (lane == 0) {
                    mbar_arrive(&raw_empty[rs]);
                    if (!leader)
                        bulk_signal_peer(sig0 + 16 * (s * C::GWARPS + gw), sig_src, afull0 + s * 8);
                    else if (gw == 0)
                        mbar_expect_tx(&afull[s], 16 * C::GWARPS);
                    else
                        mbar_arrive(&afull[s]);
                }
                copy(b, it.k0 + i + kMetaTurns * C::GROUPS);
                b = b + 1 == kMetaTurns ? 0 : b + 1;
            }
            asm volatile("cp.async.wait_group 0;" ::: "memory");
            pos += (uint32_t)nst;
            rpos += (uint32_t)(it.k1 - it.k0);
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

// Halves, tokens per tile and K slices for a problem, by the estimated cycles of
// the busiest pair: rounds of tiles x stages, a stage at the largest of its MMAs
// (1.7 n cycles a half as fitted, 2 n by the pipe's rate), its bytes at the 38 a cycle
// that an SM takes in, and the expansion (620 cycles, 1040 for two halves: the
// largest of the three up to 224 tokens for one half, and always for two); the drains
// that are not overlapped, and a slice's partial tile and the second kernel, cost
// extra.
// The constants are fitted to the times of up to 14 plans for each of 107 problems
// (1 to 2048 tokens, 520 x 1408 to 8192 x 28672), where the choice is then within
// 2.1% of the fastest; on 120 drawn at random it is within 5%, and within 11% for
// ten that take less than 12 us.  SLR_DX_HALVES=1|2 forces the halves; used by the tests.
DxPlan input_backward_plan(int64_t M, int64_t d_out, int64_t d_in, int64_t r, int sms) {
    const int64_t ut = (M + 15) / 16, nk = (d_out + kK - 1) / kK, nlr = (r + 63) / 64;
    const int64_t pairs = sms / 2 < 1 ? 1 : sms / 2;
    DxPlan best{1, 0, 0, 1};
    double best_cost = 0;
    const char *force = getenv("SLR_DX_HALVES");
    for (int h = 1; h <= 2; ++h) {
        if (force != nullptr && (force[0] == '1' || force[0] == '2') && h != force[0] - '0') continue;
        const int64_t rows = (d_in + 256 * h - 1) / (256 * h), chu = (h == 1 ? DxCfg<1>::MAXN : DxCfg<2>::MAXN) / 16;
        const int64_t tmin = (ut + chu - 1) / chu;
        for (int64_t tt = tmin; tt <= tmin + 6 && tt <= ut; ++tt) {
            const int64_t nu = (ut + tt - 1) / tt, ttiles = (ut + nu - 1) / nu;
            const double n = 16.0 * nu, bytes = (9216.0 * h + 64.0 * n) / 38.0;
            double stage = 1.7 * n * h > bytes ? 1.7 * n * h : bytes;
            if (stage < (h == 1 ? 620.0 : 1040.0)) stage = h == 1 ? 620.0 : 1040.0;
            for (int64_t ks = 1; ks <= 8 && ks * 4 <= nk + 3; ++ks) {
                const int64_t rounds = (rows * ttiles * ks + pairs - 1) / pairs;
                double cost = rounds * (((nk + ks - 1) / ks + nlr) * stage + (h == 1 ? 2000.0 : 2000.0 + 22.0 * n)) + n;
                if (ks > 1) cost += 2750.0 + (double)ks * M * d_in * 8.0 / (pairs * 78.0);
                if (best.n == 0 || cost < best_cost) {
                    best = DxPlan{h, (int)(16 * nu), (int)ttiles, (int)ks};
                    best_cost = cost;
                }
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
              make_map(&maps.vals, kBF16, vals, d_in / 2, d_out, d_in, 64, kK, CU_TENSOR_MAP_SWIZZLE_128B) &&
              make_map(&maps.x32, kBF16, dX, d_in, M, d_in * 2, kCols, 32, CU_TENSOR_MAP_SWIZZLE_NONE) &&
              make_map(&maps.x16, kBF16, dX, d_in, M, d_in * 2, kCols, 16, CU_TENSOR_MAP_SWIZZLE_NONE);
    if (ok && r > 0)
        ok = make_map(&maps.g, kBF16, G, r, M, r * 2, 64, plan.n / 2, CU_TENSOR_MAP_SWIZZLE_128B) &&
             make_map(&maps.v, kBF16, V, d_in, r, d_in * 2, 64, 64, CU_TENSOR_MAP_SWIZZLE_128B);
    if (!ok) return cudaErrorInvalidValue;
    DxParams p;
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
    const int64_t items = (d_in + 256 * plan.halves - 1) / (256 * plan.halves) * plan.ttiles * plan.ks;
    if (items > INT32_MAX) return cudaErrorInvalidValue;
    p.items = (int32_t)items;
    p.err = dx_err();
    const auto kernel = plan.halves == 1 ? input_backward_kernel<1> : input_backward_kernel<2>;
    const int smem = plan.halves == 1 ? DxCfg<1>::SMEM : DxCfg<2>::SMEM;
    cudaError_t err = cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
    if (err != cudaSuccess) return err;
    const int64_t pairs = items < sms / 2 ? items : sms / 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(2 * pairs));
    cfg.blockDim = dim3(plan.halves == 1 ? DxCfg<1>::THREADS : DxCfg<2>::THREADS);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = r > 0 ? 1 : 0;   // the kernel just before is the one that writes G
    err = cudaLaunchKernelEx(&cfg, kernel, maps, p);
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
