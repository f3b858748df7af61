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
// Bound by HBM: 2 bytes per logit forward, 4 backward, 4 for both in one pass.
// A cluster of KS CTAs owns a row, each a slice of its columns.  A thread holds
// NV vectors of eight logits; where the slice fits the CTA's registers it is
// read once and kept from the statistics to the gradient, else it is read again
// (from L2, where it has just been).  A thread's maximum and sum of
// exponentials (online, rescaled once per NV vectors) join by shuffles, shared
// memory and the cluster's distributed shared memory, in a fixed order.  The
// gradient's pass writes tau q dloss everywhere; after a block barrier the k
// listed columns of the slice are written again with their p subtracted.
// Duplicate columns each find the sum of all their p in list order and write
// the same bits.
//
// Rows start at any 2-byte boundary: a row is cut into a head up to the first
// 16-byte boundary, vectors, and a tail.
#include "common.cuh"
#include "tc_ptx.cuh"

namespace slr {
namespace {

constexpr int kMaxK = SLR_DISTILL_MAX_K;
constexpr int kNV = 8;
constexpr float kLog2e = 1.4426950408889634f, kLn2 = 0.6931471805599453f;

// Coherent loads: the gradient may overwrite the logits.
__device__ __forceinline__ uint4 ld_v4(const uint16_t *p) {
    uint4 v;
    asm volatile("ld.global.L1::no_allocate.v4.u32 {%0,%1,%2,%3}, [%4];"
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

// A running maximum and the sum of 2^(z c + b), c = log2(e) / tau, b = -max c as
// rounded: every later use adds the same b, so its rounding drops out of the
// logarithms.  With no finite maximum yet b is 0, so that 2^-inf = 0 and no
// difference of infinities arises; an empty sum stays 0 whatever its factor.
struct MaxSum {
    float m, b, s;
    __device__ __forceinline__ void raise(float to, float c) {
        const float old = b;
        m = fmaxf(m, to);
        b = m == -INFINITY ? 0.f : -m * c;
        s = s == 0.f ? 0.f : s * ex2(b - old);
    }
    __device__ __forceinline__ void add(float z, float c) {
        raise(z, c);
        s += ex2(fmaf(z, c, b));
    }
    __device__ __forceinline__ void join(float om, float os, float c) {
        const float ob = om == -INFINITY ? 0.f : -om * c;
        raise(om, c);
        s += os == 0.f ? 0.f : os * ex2(b - ob);
    }
};

template <int T>
__device__ __forceinline__ float block_sum(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v += __shfl_xor_sync(0xFFFFFFFFu, v, o);
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 32; ++w) v += red[w];
    return v;
}
template <int T>
__device__ __forceinline__ float block_max(float v, float *red) {
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) v = fmaxf(v, __shfl_xor_sync(0xFFFFFFFFu, v, o));
    __syncthreads();
    if ((threadIdx.x & 31) == 0) red[threadIdx.x >> 5] = v;
    __syncthreads();
    v = red[0];
#pragma unroll
    for (int w = 1; w < T / 32; ++w) v = fmaxf(v, red[w]);
    return v;
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
    __shared__ int32_t sh_i[kMaxK];
    __shared__ float sh_p[kMaxK], sh_z[kMaxK];
    __shared__ float red[T / 32], red2[T / 32];
    __shared__ float peer_m[8], peer_s[8], peer_l[8];
    uint32_t ks_n;
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(ks_n));
    const uint32_t ks_q = tc::cluster_ctarank();
    const int64_t m = blockIdx.x / ks_n;
    const int tid = threadIdx.x, k = a.k;
    const float c = kLog2e / a.tau, itau = 1.0f / a.tau;

    // This CTA's slice [lo, hi): vectors [v0, v1) of the row, with the head on
    // the first CTA and the tail on the last.
    const uint16_t *z = a.z + m * a.ldz;
    int64_t head = (int64_t)((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / 2;
    if (head > a.n) head = a.n;
    const int64_t nv = (a.n - head) / 8;
    const int64_t v0 = nv * ks_q / ks_n, v1 = nv * (ks_q + 1) / ks_n;
    const int64_t lo = ks_q == 0 ? 0 : head + 8 * v0, hi = ks_q == ks_n - 1 ? a.n : head + 8 * v1;
    const int64_t tail = head + 8 * nv;   // first column of the row's tail
    const uint16_t *zv = z + head;

    // Teacher entries: probabilities and the slice's listed logits.
    float tmax = -INFINITY;
    for (int j = tid; j < k; j += T) {
        const int32_t i = __ldg(a.idx + m * k + j);
        const bool there = i >= 0 && i < a.n;
        const float t = there ? __ldg(a.t + m * k + j) : -INFINITY;
        sh_i[j] = t == -INFINITY ? -1 : i;
        sh_p[j] = t;
        sh_z[j] = there && i >= lo && i < hi ? ld_z(z + i) : 0.f;
        tmax = t != t ? t : (tmax != tmax ? tmax : fmaxf(tmax, t));
    }
    // NaN teacher logits give a NaN loss; fmaxf alone would drop them.
    const bool tnan = __syncthreads_or(tmax != tmax);
    tmax = block_max<T>(tmax != tmax ? -INFINITY : tmax, red);
    const bool empty = tmax == -INFINITY && !tnan;
    const float w = kGrad ? __ldg(a.dloss + m) * a.tau : 0.f;

    if (empty && kLoss && ks_q == 0 && tid == 0) {
        a.loss[m] = 0.f;
        if (a.lse != nullptr) a.lse[m] = 0.f;
    }
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
    if (empty || (!kLoss && w == 0.f)) {   // uniform over the cluster: nothing of the row is read
        if constexpr (kGrad) {
            const uint32_t zero[4] = {0, 0, 0, 0};
            for (int64_t v = v0 + tid; v < v1; v += T) put8(v, zero);
            if (ks_q == 0 && tid < head) dz[tid] = 0;
            if (ks_q == ks_n - 1 && tid < a.n - tail) dz[tail + tid] = 0;
        }
        return;
    }
    float logsum_t = 0.f;
    {
        float e = 0.f;
        for (int j = tid; j < k; j += T) {
            const float x = sh_i[j] < 0 ? 0.f : expf((sh_p[j] - tmax) * itau);
            e += x;
        }
        e = block_sum<T>(e, red);
        logsum_t = logf(e);
    }

    // Statistics of the row, the slice kept in registers where it fits.
    uint4 x[kNV];
    const bool fits = v1 - v0 <= (int64_t)T * kNV;
    float edge = 0.f;        // this thread's head or tail logit
    const bool has_edge = ks_q == 0 && tid < head;
    const bool has_tail = ks_q == ks_n - 1 && tid < a.n - tail;
    float edge2 = 0.f;
    if (has_edge) edge = ld_z(z + tid);
    if (has_tail) edge2 = ld_z(z + tail + tid);
    auto load = [&](int64_t b) {
#pragma unroll
        for (int u = 0; u < kNV; ++u) {
            const int64_t v = b + tid + (int64_t)u * T;
            x[u] = v < v1 ? ld_v4(zv + 8 * v) : make_uint4(0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u, 0xFF80FF80u);   // -inf
        }
    };
    float shift;   // q = exp2(z c - shift)
    if constexpr (kLoss) {
        MaxSum r{-INFINITY, 0.f, 0.f};
        if (has_edge) r.add(edge, c);
        if (has_tail) r.add(edge2, c);
        for (int64_t b = v0; b < v1; b += (int64_t)T * kNV) {
            load(b);
            uint32_t mx = 0xFF80FF80u;
#pragma unroll
            for (int u = 0; u < kNV; ++u)
                mx = max_bf16x2(mx, max_bf16x2(max_bf16x2(x[u].x, x[u].y), max_bf16x2(x[u].z, x[u].w)));
            r.raise(fmaxf(bf16lo_to_f32(mx), bf16hi_to_f32(mx)), c);
            float s0 = 0.f, s1 = 0.f;
#pragma unroll
            for (int u = 0; u < kNV; ++u) {
                const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    s0 += ex2(fmaf(bf16lo_to_f32(xw[i]), c, r.b));
                    s1 += ex2(fmaf(bf16hi_to_f32(xw[i]), c, r.b));
                }
            }
            r.s += s0 + s1;
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            r.join(__shfl_xor_sync(0xFFFFFFFFu, r.m, o), __shfl_xor_sync(0xFFFFFFFFu, r.s, o), c);
        __syncthreads();
        if ((tid & 31) == 0) {
            red[tid >> 5] = r.m;
            red2[tid >> 5] = r.s;
        }
        __syncthreads();
        r = MaxSum{-INFINITY, 0.f, 0.f};
#pragma unroll
        for (int i = 0; i < T / 32; ++i) r.join(red[i], red2[i], c);
        if (ks_n > 1) {
            if (tid < (int)ks_n) {
                st_cluster_f32(&peer_m[ks_q], tid, r.m);
                st_cluster_f32(&peer_s[ks_q], tid, r.s);
            }
            tc::cluster_sync_all();
            r = MaxSum{-INFINITY, 0.f, 0.f};
            for (uint32_t q = 0; q < ks_n; ++q) r.join(peer_m[q], peer_s[q], c);
        }
        const float logs = log2f(r.s);
        float part = 0.f;
        for (int j = tid; j < k; j += T) {
            const int32_t i = sh_i[j];
            if (i < 0) continue;
            const float logp = (sh_p[j] - tmax) * itau - logsum_t, p = expf(logp);
            if (i >= lo && i < hi && !(p == 0.f)) part += p * (logp - kLn2 * (fmaf(sh_z[j], c, r.b) - logs));
        }
        part = block_sum<T>(part, red);
        if (ks_n > 1) {
            if (tid == 0) st_cluster_f32(&peer_l[ks_q], 0, part);
            tc::cluster_sync_all();   // the parts are in the first CTA's shared memory, which reads its own
            if (ks_q == 0) {
                part = peer_l[0];
                for (uint32_t q = 1; q < ks_n; ++q) part += peer_l[q];
            }
        }
        if (ks_q == 0 && tid == 0) {
            a.loss[m] = a.tau * a.tau * (tnan ? NAN : part);
            if (a.lse != nullptr) a.lse[m] = kLn2 * (logs - r.b);
        }
        shift = logs - r.b;
    } else {
        shift = __ldg(a.lse_in + m) * kLog2e;
    }
    if constexpr (kGrad) {
        if (kLoss && w == 0.f) {   // a token without weight: its row is zero whatever its logits
            const uint32_t zero[4] = {0, 0, 0, 0};
            for (int64_t v = v0 + tid; v < v1; v += T) put8(v, zero);
            if (has_edge) dz[tid] = 0;
            if (has_tail) dz[tail + tid] = 0;
            return;
        }
        for (int64_t b = v0; b < v1; b += (int64_t)T * kNV) {
            if (!kLoss || !fits) load(b);
#pragma unroll
            for (int u = 0; u < kNV; ++u) {
                const int64_t v = b + tid + (int64_t)u * T;
                if (v < v1) {
                    const uint32_t xw[4] = {x[u].x, x[u].y, x[u].z, x[u].w};
                    uint32_t o[4];
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        const float g0 = w * ex2(fmaf(bf16lo_to_f32(xw[i]), c, -shift));
                        const float g1 = w * ex2(fmaf(bf16hi_to_f32(xw[i]), c, -shift));
                        asm("cvt.rn.bf16x2.f32 %0, %1, %2;" : "=r"(o[i]) : "f"(g1), "f"(g0));
                    }
                    put8(v, o);
                }
            }
        }
        if (has_edge) dz[tid] = f32_to_bf16_bits(w * ex2(fmaf(edge, c, -shift)));
        if (has_tail) dz[tail + tid] = f32_to_bf16_bits(w * ex2(fmaf(edge2, c, -shift)));
        __syncthreads();   // the listed columns below overwrite what other threads wrote
        for (int j = tid; j < k; j += T) {
            const int32_t i = sh_i[j];
            if (i < lo || i >= hi) continue;
            float p = 0.f;
            for (int l = 0; l < k; ++l)
                if (sh_i[l] == i) p += expf((sh_p[l] - tmax) * itau - logsum_t);
            dz[i] = f32_to_bf16_bits(w * (ex2(fmaf(sh_z[j], c, -shift)) - (tnan ? NAN : p)));
        }
    }
}

template <int T, bool kLoss, bool kGrad>
cudaError_t launch_t(const DistillArgs &a, unsigned ks, cudaStream_t stream) {
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(a.M * ks));
    cfg.blockDim = dim3(T);
    cfg.stream = stream;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeClusterDimension;
    attr[0].val.clusterDim.x = ks;
    attr[0].val.clusterDim.y = 1;
    attr[0].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, distill_kernel<T, kLoss, kGrad>, a);
}

template <bool kLoss, bool kGrad>
cudaError_t launch_distill(const DistillArgs &a, cudaStream_t stream) {
    int dev = 0, sms = 148;
    if (cudaGetDevice(&dev) == cudaSuccess) cudaDeviceGetAttribute(&sms, cudaDevAttrMultiProcessorCount, dev);
    const int64_t vecs = a.n / 8;   // of eight logits, at most
    if (vecs <= 128 * kNV) return launch_t<128, kLoss, kGrad>(a, 1, stream);
    unsigned ks = 1;
    while (ks < 8 && (vecs > (int64_t)ks * 512 * kNV || a.M * ks < 2 * (int64_t)sms) && vecs > (int64_t)ks * 512) ks *= 2;
    return launch_t<512, kLoss, kGrad>(a, ks, stream);
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
