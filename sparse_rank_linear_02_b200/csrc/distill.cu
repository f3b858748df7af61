// distill.cu -- distillation of a student's logits from a teacher's top logits.
//
// Token m has n_vocab student logits z and up to k teacher entries (column i_j,
// logit t_j); entries whose column lies outside [0, n_vocab) or whose logit is
// -inf are not there.  At temperature tau
//     p_j = exp(t_j / tau) / sum over the entries     q = softmax(z / tau)
//     loss_m = tau^2 sum_j p_j (log p_j - log q_{i_j})
//     dloss_m dL/dz_v = dloss_m tau (q_v - sum of p_j with i_j = v)
// A token without entries has loss 0 and a zero gradient whatever its logits.
//
// Bound by HBM: 2 bytes per logit forward, 4 backward, at least 4 for both in one call.
// A cluster of KS CTAs owns a row, each a slice of its columns.  A thread holds
// NV vectors of eight logits; where the slice fits the CTA's registers it is
// read once and kept from the statistics to the gradient, else it is read again
// (from L2, where it has just been).  A thread's maximum and sum of
// exponentials (online, rescaled once per NV vectors) join by shuffles, shared
// memory and the cluster's distributed shared memory, in a fixed order.  (The
// CTAs of a cluster learn from one barrier that all have started, arrived at
// first and waited for before the first store to a peer, the row's loads in
// between.)  The
// gradient's pass writes tau q dloss everywhere; after a block barrier the k
// listed columns of the slice are written again with their p subtracted.
// Duplicate columns each find the sum of all their p in list order and write
// the same bits.
// The gradient from a given lse takes q = exp(z / tau - lse), except in rows whose
// lse is too large for fp32 to hold it closely (kMaxLse): those read their logits
// twice (4096 x 131072, all rows so: 452 us against 336).
//
// Rows start at any 2-byte boundary: a row is cut into a head up to the first
// 16-byte boundary, vectors, and a tail.
//
// The one call takes the rounds of its gradient backwards: the last one is still in
// the registers, and those just before it are the likeliest to be in L2, which is
// asked to keep a row until its second read.
//
// Measured (a graph of 6 to 96 calls), k = 64, against the copy bandwidth: 4096 x
// 131072 forward 162 us (1.01), backward 336 (0.98), both in one call 413 (0.79);
// 4096 x 32000 49 / 92 / 108 us (0.82 / 0.87 / 0.74); one token of 131072 4.8 / 4.2
// / 6.8 us; 1000 x 50001, k = 20, 23 / 40 / 49 us (0.66 / 0.77 / 0.63: 1000 rows of
// one CTA fill 592 resident ones 1.7 times).  The one call is above its
// 4 bytes a logit by its second reads (three quarters of a row of 131072), of which
// L2 still misses half: by the counters 2.47 GB in all, 4.6 bytes a logit, at 0.91 of
// the copy bandwidth (498 us before L2 was asked to keep rows, 440 forwards; without
// the first pass's exponentials it is 3% faster).  Tried and not kept for it: part of the row in shared memory (459
// us, less of it left to L1), the next round's loads
// among the present one's stores (481 us, and 437 for the backward alone: reads
// in long bursts suit HBM better), a persistent CTA per SM that keeps a row in
// shared memory (502 us: its two passes take turns with HBM), the gradient of one
// row beside the statistics of the next (525 us read from L2, 666 us kept in
// clusters of two), clusters that keep the row in registers (610 to 644 us: two
// cluster barriers a row), and stores that leave L2 first (no gain).
#include "common.cuh"
#include "f32x2.cuh"
#include "tc_ptx.cuh"

namespace slr {
namespace {

constexpr int kNV = 8;
constexpr float kLn2 = 0.6931471805599453f;
// The largest |lse| that the gradient alone takes as given.  Its spacing, and the
// roundings of lse and of 1 / tau, put q off by up to 3 x 2^-24 |lse| relative:
// 1.2e-5 here, but 0.4% at 2^16.  Beyond it (and for an infinite or NaN lse) the
// row's maximum and sum are formed again from its logits, as the one pass forms
// them, to the same bits.
constexpr float kMaxLse = 64.f;

// Coherent loads: the gradient may overwrite the logits.
__device__ __forceinline__ uint4 ld_v4(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
                 : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
                 : "l"(p));
    return v;
}
// The same for a row that is read twice: its lines stay in L2 in preference to
// others until the second read, which gives them up first.
__device__ __forceinline__ uint4 ld_keep_v4(const uint16_t *p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .b64 pol;\n\t"
        "createpolicy.fractional.L2::evict_last.b64 pol, 1.0;\n\t"
        "ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], pol;\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}
__device__ __forceinline__ uint4 ld_last_v4(const uint16_t *p) {
    uint4 v;
    asm volatile(
        "{\n\t.reg .b64 pol;\n\t"
        "createpolicy.fractional.L2::evict_first.b64 pol, 1.0;\n\t"
        "ld.global.L1::no_allocate.L2::cache_hint.v4.u32 {%0,%1,%2,%3}, [%4], pol;\n\t}"
        : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w)
        : "l"(p));
    return v;
}
__device__ __forceinline__ float ld_z(const uint16_t *p) {
    uint16_t v;
    asm volatile("ld.global.u16 %0, [%1];" : "=h"(v) : "l"(p));
    return bf16lo_to_f32(v);
}
__device__ __forceinline__ float ex2(float x) {
    asm("ex2.approx.ftz.f32 %0, %0;" : "+f"(x));
    return x;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b) {
    uint32_t r;
    asm("max.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// A running maximum and the sum of 2^((z - max) c), c = log2(e) / tau.  The
// difference comes first: it is exact or rounded once, and a logit of the type's
// lowest value (a mask) overflows nothing.  With no finite maximum yet the
// reference is 0, so that 2^-inf = 0 and no difference of infinities arises; an
// empty sum stays 0 whatever its factor.
struct MaxSum {
    float m, s;
    __device__ __forceinline__ float ref() const { return m == -INFINITY ? 0.f : m; }
    __device__ __forceinline__ void raise(float to, float c) {
        const float old = ref();
        m = fmaxf(m, to);
        s = s == 0.f ? 0.f : s * ex2((old - ref()) * c);
    }
    __device__ __forceinline__ void add(float z, float c) {
        raise(z, c);
        s += ex2((z - ref()) * c);
    }
};

__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}
__device__ __forceinline__ float warp_sum(float v) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    return v;
}
// The lanes' pairs joined: the maximum first, then each sum rescaled once.
__device__ __forceinline__ void warp_join(MaxSum &r, float c) {
    r.raise(warp_max(r.m), c);
    r.s = warp_sum(r.s);
}

__device__ __forceinline__ void st_cluster_f32(const float *local, uint32_t rank, float v) {
    asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(tc::mapa_shared(tc::smem_u32(local), rank)), "f"(v) : "memory");
}

struct DistillArgs {
    const uint16_t *z;      // bf16 [M, ldz]
    int64_t M, n, ldz;
    const int32_t *idx;     // [M, k]
    const float *t;         // [M, k]
    int32_t k;
    float tau;
    const float *lse_in;    // [M], the gradient alone
    const float *dloss;     // [M], with the gradient
    float *loss, *lse;      // [M], out (lse may be null)
    uint16_t *dz;           // bf16 [M, lddz], out
    int64_t lddz;
};

template <int T, bool kLoss, bool kGrad>
__global__ void __launch_bounds__(T, 1024 / T) distill_kernel(const __grid_constant__ DistillArgs a) {
    constexpr int kWarps = T / 32;
    // The teacher's entries: columns (read four at a time), probabilities, the slice's logits.
    extern __shared__ __align__(16) int32_t sh_i[];
    const int k4 = (a.k + 3) & ~3;
    float *const sh_p = reinterpret_cast<float *>(sh_i + k4), *const sh_z = sh_p + k4;
    __shared__ float row_m[kWarps], row_s[kWarps], tea_m[kWarps], tea_s[kWarps], part_w[kWarps];
    __shared__ float peer_m[8], peer_s[8], peer_l[8];
    uint32_t ks_n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks_n));
    const uint32_t ks_q = tc::cluster_ctarank();
    if (kLoss && ks_n > 1) tc::cluster_arrive_started();
    const int64_t m = blockIdx.x / ks_n;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5, k = a.k;
    const float c = kLog2e / a.tau;

    // This CTA's slice [lo, hi): vectors [v0, v1) of the row, with the head on
    // the first CTA and the tail on the last.
    const uint16_t *z = a.z + m * a.ldz;
    int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / 2;
    if (head > a.n) head = a.n;
    const int64_t nv = (a.n - head) / 8;
    const int64_t v0 = nv * ks_q / ks_n, v1 = nv * (ks_q + 1) / ks_n;
    const int64_t lo = ks_q == 0 ? 0 : head + 8 * v0, hi = ks_q == ks_n - 1 ? a.n : head + 8 * v1;
    const int64_t tail = head + 8 * nv;   // first column of the row's tail
    const bool has_head = ks_q == 0 && tid < head;
    const bool has_tail = ks_q == ks_n - 1 && tid < a.n - tail;

    // The first vectors are requested before anything is waited for: the
    // teacher's entries and their statistics are worked on while they come.
    uint4 x[kNV];
    constexpr bool kBoth = kLoss && kGrad;
    const int nb = (int)((v1 - v0 + T * kNV - 1) / (T * kNV));   // rounds of kNV vectors per thread
    auto load = [&](int i, bool again) {
#pragma unroll
        for (int u = 0; u < kNV; ++u) {
            const int64_t v = v0 + tid + ((int64_t)i * kNV + u) * T;
            const uint16_t *src = z + head + 8 * v;
            x[u] = make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);   // -inf
            if (v < v1) x[u] = again ? ld_last_v4(src) : kBoth && i < nb - 1 ? ld_keep_v4(src) : ld_v4(src);
        }
    };
    load(0, false);
    const float zhead = has_head ? ld_z(z + tid) : 0.f, ztail = has_tail ? ld_z(z + tail + tid) : 0.f;
    const float w = kGrad ? __ldg(a.dloss + m) * a.tau : 0.f;
    // Whether the row's statistics are formed here: the same for the whole cluster.
    const float lse_in = kLoss ? 0.f : __ldg(a.lse_in + m);
    const bool stats = kLoss || !(fabsf(lse_in) <= kMaxLse);

    // Teacher entries, their maximum and sum, and the slice's listed logits.  A
    // NaN logit is kept as the maximum's mark (+inf would give NaN as well).
    MaxSum t{-INFINITY, 0.f};
    if (tid < k4 - k) sh_i[k + tid] = -1;
    for (int j = tid; j < k; j += T) {
        const int32_t i = __ldg(a.idx + m * k + j);
        const bool there = i >= 0 && i < a.n;
        const float v = there ? __ldg(a.t + m * k + j) : -INFINITY;
        sh_i[j] = v == -INFINITY ? -1 : i;
        sh_p[j] = v;
        sh_z[j] = there && i >= lo && i < hi ? ld_z(z + i) : 0.f;
        t.add(v != v ? INFINITY : v, c);
    }
    warp_join(t, c);
    if (lane == 0) {
        tea_m[warp] = t.m;
        tea_s[warp] = t.s;
    }

    // Statistics of the row's slice; kept in registers where it fits.
    MaxSum r{-INFINITY, 0.f};
    if (stats) {
        if (has_head) r.add(zhead, c);
        if (has_tail) r.add(ztail, c);
        for (int i = 0; i < nb; ++i) {
            if (i != 0) load(i, false);
            uint32_t mx = 0xFF80FF80u;
#pragma unroll
            for (int u = 0; u < kNV; ++u)
                mx = max_bf16x2(mx, max_bf16x2(max_bf16x2(x[u].x, x[u].y), max_bf16x2(x[u].z, x[u].w)));
            r.raise(fmaxf(bf16lo_to_f32(mx), bf16hi_to_f32(mx)), c);
            const f32x2 neg = dup2(-r.ref()), c2 = dup2(c);
            f32x2 sum = dup2(0.f);
#pragma unroll
            for (int u = 0; u < kNV; ++u) {
                const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sum = add2(sum, exp2_2(mul2(add2(pack2(bf16lo_to_f32(xw[j]), bf16hi_to_f32(xw[j])), neg), c2)));
            }
            float s0, s1;
            unpack2(sum, s0, s1);
            r.s += s0 + s1;
        }
        warp_join(r, c);
        if (lane == 0) {
            row_m[warp] = r.m;
            row_s[warp] = r.s;
        }
    }
    __syncthreads();
    t = MaxSum{lane < kWarps ? tea_m[lane] : -INFINITY, lane < kWarps ? tea_s[lane] : 0.f};
    warp_join(t, c);
    const bool empty = t.m == -INFINITY;
    const float t_ref = t.ref(), t_log = log2f(t.s);   // log2 p_j = (t_j - t_ref) c - t_log

    uint16_t *dz = kGrad ? a.dz + m * a.lddz : nullptr;
    const bool same_phase = ((reinterpret_cast<uintptr_t>(dz) ^ reinterpret_cast<uintptr_t>(z)) & 15) == 0;
    auto put8 = [&](int64_t v, const uint32_t (&o)[4]) {
        uint16_t *at = dz + head + 8 * v;
        if (same_phase) {
            *reinterpret_cast<uint4 *>(at) = make_uint4(o[0], o[1], o[2], o[3]);
        } else {
#pragma unroll
            for (int i = 0; i < 8; ++i) at[i] = (uint16_t)(o[i / 2] >> (16 * (i & 1)));
        }
    };
    // log2 q = (z scale - ref) fac - logs: with the row's statistics scale is 1,
    // ref the row's maximum and fac c; from a given lse scale is 1 / tau, ref that
    // lse, fac log2(e) and logs 0.
    float scale = 1.f, ref = 0.f, fac = c, logs = 0.f;
    if (stats) {
        r = MaxSum{lane < kWarps ? row_m[lane] : -INFINITY, lane < kWarps ? row_s[lane] : 0.f};
        warp_join(r, c);
        if (ks_n > 1) {
            if constexpr (kLoss)
                tc::cluster_wait_started();
            else
                tc::cluster_sync_all();   // every CTA has started
            if (tid < (int)ks_n) {
                st_cluster_f32(&peer_m[ks_q], tid, r.m);
                st_cluster_f32(&peer_s[ks_q], tid, r.s);
            }
            tc::cluster_sync_all();
            r = MaxSum{lane < (int)ks_n ? peer_m[lane] : -INFINITY, lane < (int)ks_n ? peer_s[lane] : 0.f};
            warp_join(r, c);
        }
        ref = r.ref();
        logs = log2f(r.s);
    } else {
        scale = 1.f / a.tau;
        ref = lse_in;
        fac = kLog2e;
    }
    // The entries' probabilities, and their terms of the loss.
    if (32 * warp < k) {
        float part = 0.f;
        for (int j = tid; j < k; j += T) {
            const int32_t i = sh_i[j];
            const float logp = fmaf(sh_p[j] - t_ref, c, -t_log), p = i < 0 ? 0.f : exp2f(logp);
            sh_p[j] = p;
            if (kLoss && i >= lo && i < hi && !(p == 0.f)) part += p * (logp - fmaf(sh_z[j] - ref, c, -logs));
        }
        if constexpr (kLoss) {
            part = warp_sum(part);
            if (lane == 0) part_w[warp] = part;
        }
    }
    if constexpr (kLoss) {
        __syncthreads();
        float part = 0.f;
        if (warp == 0) {
            part = warp_sum(lane < kWarps && 32 * lane < k ? part_w[lane] : 0.f);
            if (ks_n > 1 && lane == 0) st_cluster_f32(&peer_l[ks_q], 0, part);
        }
        if (ks_n > 1) tc::cluster_sync_all();   // the parts are in the first CTA's shared memory, which alone reads them
        if (ks_q == 0 && warp == 0) {
            if (ks_n > 1) part = warp_sum(lane < (int)ks_n ? peer_l[lane] : 0.f);
            if (lane == 0) {
                a.loss[m] = empty ? 0.f : a.tau * a.tau * kLn2 * part;
                if (a.lse != nullptr) a.lse[m] = empty ? 0.f : fmaf(kLn2, logs, ref / a.tau);
            }
        }
    }
    if constexpr (kGrad) {
        if (empty || w == 0.f) {   // a token without entries or weight: zero whatever its logits
            const uint32_t zero[4] = {0, 0, 0, 0};
            for (int64_t v = v0 + tid; v < v1; v += T) put8(v, zero);
            if (has_head) dz[tid] = 0;
            if (has_tail) dz[tail + tid] = 0;
            return;
        }
        const f32x2 scale2 = dup2(scale), nref2 = dup2(-ref), fac2 = dup2(fac), nlogs2 = dup2(-logs);
        auto q2 = [&](f32x2 zz) {
            return exp2_2(fma2(kLoss ? add2(zz, nref2) : fma2(zz, scale2, nref2), fac2, nlogs2));
        };
        auto q1 = [&](float zz) { return ex2(fmaf(kLoss ? zz - ref : fmaf(zz, scale, -ref), fac, -logs)); };
        // After the statistics the last round is in the registers, and the rounds
        // just before it are the likeliest to be in L2: they go first.
        for (int s = 0; s < nb; ++s) {
            const int i = stats ? nb - 1 - s : s;
            if (s != 0) load(i, kBoth);
#pragma unroll
            for (int u = 0; u < kNV; ++u) {
                const int64_t v = v0 + tid + ((int64_t)i * kNV + u) * T;
                if (v < v1) {
                    const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                    uint32_t o[4];
#pragma unroll
                    for (int j = 0; j < 4; ++j) {
                        float g0, g1;
                        unpack2(mul2(dup2(w), q2(pack2(bf16lo_to_f32(xw[j]), bf16hi_to_f32(xw[j])))), g0, g1);
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[j]) : "f"(g1), "f"(g0));
                    }
                    put8(v, o);
                }
            }
        }
        if (has_head) dz[tid] = f32_to_bf16_bits(w * q1(zhead));
        if (has_tail) dz[tail + tid] = f32_to_bf16_bits(w * q1(ztail));
        __syncthreads();   // the listed columns below overwrite what other threads wrote
        for (int j = tid; j < k; j += T) {
            const int32_t i = sh_i[j];
            if (i < lo || i >= hi) continue;
            float p = 0.f;
#pragma unroll 4
            for (int l = 0; l < k; l += 4) {
                const int4 at = *reinterpret_cast<const int4 *>(sh_i + l);
                if (at.x == i) p += sh_p[l];
                if (at.y == i) p += sh_p[l + 1];
                if (at.z == i) p += sh_p[l + 2];
                if (at.w == i) p += sh_p[l + 3];
            }
            dz[i] = f32_to_bf16_bits(w * (q1(sh_z[j]) - p));
        }
    }
}

template <int T, bool kLoss, bool kGrad>
cudaError_t launch_t(const DistillArgs &a, unsigned ks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.M * ks));
    cfg.blockDim = dim3(T);
    cfg.dynamicSmemBytes = (size_t)((a.k + 3) & ~3) * 12;
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ks > 1 ? 1 : 0;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, kLoss, kGrad>, a);
}

template <bool kLoss, bool kGrad>
cudaError_t launch_distill(const DistillArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t vecs = a.n / 8;   // of eight logits, at most
    if (vecs <= 128 * kNV) return launch_t<128, kLoss, kGrad>(a, 1, stream);
    // Few rows: as many threads on each as a cluster gives (64 x 131072: 9.3 /
    // 11.0 / 14.0 us forward / backward / both with 8 x 256, 21.4 / 28.6 / 44.2
    // with 1 x 128).  Many: small CTAs hide each other's reductions (4096 x
    // 131072 forward: 165 us with 1 x 128, 180 with 1 x 512, 249 with 2 x 512); a
    // gradient wants fewer rows at a time (L2 holds them between the passes) and
    // slices of at most 65536 logits (backward / both: 336 / 413 us with 2 x 256,
    // 356 / 454 with 1 x 256, 374 / 493 with 1 x 128; 4096 x 32000: 93 / 107 with
    // 1 x 256, 114 / 153 with 2 x 256).
    if (a.M * 8 < 5 * (int64_t)sms && vecs > 8 * 256) return launch_t<256, kLoss, kGrad>(a, 8, stream);
    constexpr int T = kGrad ? 256 : 128;
    unsigned ks = 1;
    while (ks < 8 && ((kGrad && a.n > (int64_t)ks * 65536) || (a.M * ks < 5 * (int64_t)sms && vecs > (int64_t)ks * 2 * T)))
        ks *= 2;
    return launch_t<T, kLoss, kGrad>(a, ks, stream);
}

}  // namespace

cudaError_t launch_distill_forward(const uint16_t *z, int64_t M, int64_t n, int64_t ldz, const int32_t *idx,
                                   const float *t, int64_t k, float tau, float *loss, float *lse, cudaStream_t stream) {
    DistillArgs a = {};
    a.z = z, a.M = M, a.n = n, a.ldz = ldz, a.idx = idx, a.t = t, a.k = (int32_t)k, a.tau = tau, a.loss = loss, a.lse = lse;
    return launch_distill<true, false>(a, stream);
}

cudaError_t launch_distill_backward(const uint16_t *z, int64_t M, int64_t n, int64_t ldz, const int32_t *idx,
                                    const float *t, int64_t k, float tau, const float *lse, const float *dloss,
                                    uint16_t *dz, int64_t lddz, cudaStream_t stream) {
    DistillArgs a = {};
    a.z = z, a.M = M, a.n = n, a.ldz = ldz, a.idx = idx, a.t = t, a.k = (int32_t)k, a.tau = tau, a.lse_in = lse;
    a.dloss = dloss, a.dz = dz, a.lddz = lddz;
    return launch_distill<false, true>(a, stream);
}

cudaError_t launch_distill_loss_grad(const uint16_t *z, int64_t M, int64_t n, int64_t ldz, const int32_t *idx,
                                     const float *t, int64_t k, float tau, const float *dloss, float *loss,
                                     uint16_t *dz, int64_t lddz, cudaStream_t stream) {
    DistillArgs a = {};
    a.z = z, a.M = M, a.n = n, a.ldz = ldz, a.idx = idx, a.t = t, a.k = (int32_t)k, a.tau = tau, a.dloss = dloss;
    a.loss = loss, a.dz = dz, a.lddz = lddz;
    return launch_distill<true, true>(a, stream);
}

}  // namespace slr
