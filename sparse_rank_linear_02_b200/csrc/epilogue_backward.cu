// epilogue_backward.cu -- gradient through the layer's bias and activation.
//
//   dZ = dY * act'(Z)        db_j = sum over the tokens m of dZ[m][j]
//
// for Y = act(Z) + R, Z = X S^T + T U^T + b: one pass over dY and Z.  The sums
// take the fp32 products before their rounding to bf16.
//
// It cannot do with less than 6 bytes of HBM traffic per element.  A cluster of KS <= 8 CTAs owns a strip of
// 8 * LANES columns and splits its tokens, so one launch also finishes db: the
// CTAs' column sums meet through distributed shared memory and are added in
// CTA order (the result does not depend on timing).  LANES threads read a row
// of the strip, 16 bytes each; a thread has two rows of both inputs in flight,
// four CTAs an SM (2048 x 14336, tanh GELU: 36.5 us; four rows in flight 40.3,
// where registers spill; six CTAs 47.8).  A thread's sums go through two levels
// (at most 64 rows, then the sums of those), which bounds the rounding for long
// batches.
//
// Measured (176 MB, 27 us at the copy bandwidth): relu 33.1 us, SiLU 35.4, tanh GELU
// 36.8, GELU 40.5; 2048 x 4096 (50 MB) 12.4 / 13.2 / 13.6 / 13.9; 17 x 4096 2.4 to 3.1.
//
// What bounds it: the loads of a pass wait until the pass before is computed and
// stored, so neither memory nor any pipe is busy all the time (GELU: DRAM 36%, special
// functions 39%, ALU 29%, issue slots 49%; relu: DRAM 55%, ALU 36%, issue slots 34%,
// and a warp that waits for its loads in most cycles).
#include "common.cuh"
#include "epilogue.cuh"
#include "tc_ptx.cuh"

namespace slr {
namespace {

constexpr int kThreads = 256;
constexpr int kUnroll = 2;
constexpr int kFold = 64 / kUnroll;   // passes between folds of the first level

// Coherent loads: dZ may be dY or Z itself.
__device__ __forceinline__ uint4 ld_v4(const void *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}

// Z within [-200, 200], NaN kept: the slopes are at their limits, 0 and 1, well
// inside, and no product of a zero and an infinity arises.
__device__ __forceinline__ uint32_t clamp_bf16x2(uint32_t v) {
    uint32_t r;
    asm("{\n\t.reg .b32 t;\n\tmax.NaN.bf16x2 t, %1, %2;\n\tmin.NaN.bf16x2 %0, t, %3;\n\t}"
        : "=r"(r)
        : "r"(v), "r"(0xC348C348u), "r"(0x43484348u));
    return r;
}

template <int LANES, int ACT>
__global__ void __launch_bounds__(kThreads, 4)
    epilogue_backward_kernel(const uint16_t *dY, const uint16_t *Z, int64_t M, int64_t d_out, uint16_t *dZ, float *db) {
    constexpr int kRows = kThreads / LANES;   // rows of one pass
    __shared__ float red[kRows][8 * LANES + 4];
    __shared__ float cols[8 * LANES];
    uint32_t ks_n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks_n));
    const uint32_t ks_q = tc::cluster_ctarank();
    const int64_t strip = blockIdx.x / ks_n;
    const int lane = threadIdx.x % LANES, sub = threadIdx.x / LANES;
    const int64_t col = (strip * LANES + lane) * 8;
    const int64_t m1 = M * (ks_q + 1) / ks_n;
    f32x2 part[4];
    float *own = &red[sub][8 * lane];   // second level of this thread's sums
    auto fold = [&]() {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float a, b;
            unpack2(part[i], a, b);
            own[2 * i] += a;
            own[2 * i + 1] += b;
            part[i] = dup2(0.f);
        }
    };
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        own[2 * i] = own[2 * i + 1] = 0.f;
        part[i] = dup2(0.f);
    }
    if (col < d_out) {
        int pass = 0;
        const int64_t step = (int64_t)kRows * d_out, end = m1 * d_out;
        for (int64_t at = (M * ks_q / ks_n + sub) * d_out + col; at < end; at += kUnroll * step) {
            uint4 g[kUnroll], z[kUnroll];
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (at + u * step < end) {
                    g[u] = ld_v4(dY + at + u * step);
                    if (ACT != SLR_ACT_NONE) z[u] = ld_v4(Z + at + u * step);
                }
            }
#pragma unroll
            for (int u = 0; u < kUnroll; ++u) {
                if (at + u * step >= end) break;
                const uint32_t gw[4] = {g[u].x, g[u].y, g[u].z, g[u].w};
                const uint32_t zw[4] = {z[u].x, z[u].y, z[u].z, z[u].w};
                uint32_t o[4];
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    f32x2 v = pack2(bf16lo_to_f32(gw[i]), bf16hi_to_f32(gw[i]));
                    if constexpr (ACT != SLR_ACT_NONE) {
                        const uint32_t zc = clamp_bf16x2(zw[i]);
                        v = mul2(v, slope2<ACT>(pack2(bf16lo_to_f32(zc), bf16hi_to_f32(zc))));
                    }
                    part[i] = add2(part[i], v);
                    float a, b;
                    unpack2(v, a, b);
                    asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(b), "f"(a));
                }
                if (dZ != nullptr) *reinterpret_cast<uint4 *>(dZ + at + u * step) = make_uint4(o[0], o[1], o[2], o[3]);
            }
            if (++pass == kFold) {
                pass = 0;
                fold();
            }
        }
    }
    if (db == nullptr) return;   // uniform over the grid
    fold();
    __syncthreads();
    for (int c = threadIdx.x; c < 8 * LANES; c += kThreads) {
        float s = 0.f;
#pragma unroll 8
        for (int r = 0; r < kRows; ++r) s += red[r][c];
        cols[c] = s;
    }
    tc::cluster_sync_all();   // every CTA's column sums are in its shared memory
    if (ks_q == 0) {
        const uint32_t base = tc::smem_u32(cols);
        for (int c = threadIdx.x; c < 8 * LANES; c += kThreads) {
            float s = 0.f;
            for (uint32_t q = 0; q < ks_n; ++q) {
                float v;
                asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(tc::mapa_shared(base + 4 * c, q)));
                s += v;
            }
            if (strip * LANES * 8 + c < d_out) db[strip * LANES * 8 + c] = s;
        }
    }
    tc::cluster_sync_all();   // no CTA leaves while its sums may still be read
}

template <int LANES, int ACT>
cudaError_t launch_lanes(const uint16_t *dY, const uint16_t *Z, int64_t M, int64_t d_out, uint16_t *dZ, float *db,
                         cudaStream_t stream) {
    const int64_t strips = (d_out + 8 * LANES - 1) / (8 * LANES);
    unsigned ks = 1;
    while (ks < 8 && M > (int64_t)ks * (kThreads / LANES) * kUnroll) ks *= 2;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(strips * ks));
    cfg.blockDim = dim3(kThreads);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, epilogue_backward_kernel<LANES, ACT>, dY, Z, M, d_out, dZ, db);
}

template <int ACT>
cudaError_t launch_act(const uint16_t *dY, const uint16_t *Z, int64_t M, int64_t d_out, uint16_t *dZ, float *db,
                       cudaStream_t stream) {
    // The widest strip (the longest runs of a row) with which clusters of eight put
    // two and a half CTAs on every SM: 2048 x 14336 takes 36.5 / 39.6 / 45.2 us with
    // 32 / 16 / 8 lanes, 2048 x 4096 23.9 / 17.2 / 13.8.  Batches of up to 64, 128 or
    // 256 tokens (by width) have smaller clusters and fewer CTAs: 16 x 14336 runs 56
    // of them in 2.8 us, 64 x 14336 224 in 4.7.
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t eighths = (d_out + 63) / 64 * 8;   // CTAs with 8 lanes, eight to a cluster
    if (eighths / 4 >= 5 * (int64_t)sms / 2) return launch_lanes<32, ACT>(dY, Z, M, d_out, dZ, db, stream);
    if (eighths / 2 >= 5 * (int64_t)sms / 2) return launch_lanes<16, ACT>(dY, Z, M, d_out, dZ, db, stream);
    return launch_lanes<8, ACT>(dY, Z, M, d_out, dZ, db, stream);
}

}  // namespace

cudaError_t launch_epilogue_backward(const uint16_t *dY, const uint16_t *Z, int64_t M, int64_t d_out, int act,
                                     uint16_t *dZ, float *db, cudaStream_t stream) {
    switch (act) {
        case SLR_ACT_RELU: return launch_act<SLR_ACT_RELU>(dY, Z, M, d_out, dZ, db, stream);
        case SLR_ACT_GELU: return launch_act<SLR_ACT_GELU>(dY, Z, M, d_out, dZ, db, stream);
        case SLR_ACT_GELU_TANH: return launch_act<SLR_ACT_GELU_TANH>(dY, Z, M, d_out, dZ, db, stream);
        case SLR_ACT_SILU: return launch_act<SLR_ACT_SILU>(dY, Z, M, d_out, dZ, db, stream);
        default: return launch_act<SLR_ACT_NONE>(dY, Z, M, d_out, dZ, db, stream);
    }
}

}  // namespace slr
