// Policy loss on the logits of the chosen tokens, its gradient, and token log-probabilities.
#include <cmath>

#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kPiece = 1024;                  // 16-byte vectors of one bulk copy
constexpr int kMaxPieces = 8;
// Row bytes a CTA keeps in shared memory: three CTAs of 512 threads share an SM.
constexpr int kStageBytes = 72 * 1024;

// Running maximum of the logits and sum_i 2^(k (z_i - max)), k = log2(e) / tau. The difference is
// taken first: it is exact for near logits, however large they are. A pair whose maximum is
// -inf has the sum 0.
struct MaxSum {
    float m, s;
};
__device__ __forceinline__ MaxSum join(MaxSum a, MaxSum b, float k) {
    const float m = fmaxf(a.m, b.m);
    if (m == -INFINITY) return {m, a.s + b.s};       // keeps a NaN sum
    return {m, a.s * ex2_approx((a.m - m) * k) + b.s * ex2_approx((b.m - m) * k)};
}

struct PolicyArgs {
    const int32_t* target;
    const float* advantage;
    const float* old_logp;
    const float* ref_logp;
    const float* weight;
    float* logp;
    float* tok_loss;      // [T] weight * l, or null
    int T, V;
    int64_t ld, ld_grad;
    float inv_tau, clip_low, clip_high, kl;
    int* err;
};

// The 16 bytes of a vector as fp32 pairs.
template <typename T> struct Pairs { static constexpr int N = 8 / sizeof(T); };
template <typename T>
__device__ __forceinline__ void to_pairs(const uint4& u, uint64_t (&p)[Pairs<T>::N]) {
    const uint32_t w[4] = {u.x, u.y, u.z, u.w};
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) p[i] = pk2(__uint_as_float(w[i] << 16), __uint_as_float(w[i] & 0xffff0000u));
    } else {
        p[0] = pk2(__uint_as_float(w[0]), __uint_as_float(w[1]));
        p[1] = pk2(__uint_as_float(w[2]), __uint_as_float(w[3]));
    }
}
template <typename T>
__device__ __forceinline__ uint4 from_pairs(const uint64_t (&p)[Pairs<T>::N]) {
    uint32_t w[4];
    if constexpr (sizeof(T) == 2) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float lo, hi;
            upk2(p[i], lo, hi);
            const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
            w[i] = *reinterpret_cast<const uint32_t*>(&h);
        }
    } else {
        float f[4];
        upk2(p[0], f[0], f[1]);
        upk2(p[1], f[2], f[3]);
#pragma unroll
        for (int i = 0; i < 4; ++i) w[i] = __float_as_uint(f[i]);
    }
    return make_uint4(w[0], w[1], w[2], w[3]);
}
template <typename T>
__device__ __forceinline__ float vec_max(const uint4& u) {
    if constexpr (sizeof(T) == 2) {
        const __nv_bfloat162* h = reinterpret_cast<const __nv_bfloat162*>(&u);
        const __nv_bfloat162 t = __hmax2(__hmax2(h[0], h[1]), __hmax2(h[2], h[3]));
        return fmaxf(__low2float(t), __high2float(t));
    } else {
        return fmaxf(fmaxf(__uint_as_float(u.x), __uint_as_float(u.y)), fmaxf(__uint_as_float(u.z), __uint_as_float(u.w)));
    }
}

// A thread's own running maximum, and its sum as a pair.
struct Running {
    float m;
    uint64_t s;
};
template <typename T, int U>
__device__ __forceinline__ void add_vecs(Running& a, const uint4 (&u)[U], float k) {
    float top = vec_max<T>(u[0]);
#pragma unroll
    for (int j = 1; j < U; ++j) top = fmaxf(top, vec_max<T>(u[j]));
    if (top > a.m) {
        const float f = ex2_approx((a.m - top) * k);
        a.s = mul2(a.s, splat2(f));
        a.m = top;
    }
    // a row of -inf so far: measured from 0, so that -inf gives 0 and not NaN
    const uint64_t minus = splat2(a.m == -INFINITY ? 0.f : -a.m), kk = splat2(k);
#pragma unroll
    for (int j = 0; j < U; ++j) {
        uint64_t p[Pairs<T>::N];
        to_pairs<T>(u[j], p);
#pragma unroll
        for (int i = 0; i < Pairs<T>::N; ++i) {
            float x0, x1;
            upk2(mul2(add2(p[i], minus), kk), x0, x1);
            a.s = add2(a.s, pk2(ex2_approx(x0), ex2_approx(x1)));
        }
    }
}

// What one token adds: its log-probability, its term of the loss, and the factor c of its
// gradient row c (1[v = target] - p_v).
__device__ __forceinline__ float token_terms(const PolicyArgs& a, int t, bool put, float w, float zt, MaxSum row,
                                             float k) {
    // a row of -inf alone has no distribution
    const float lp = row.s != 0.f ? ((zt - row.m) * k - log2f(row.s)) * kLn2 : NAN;
    if (a.logp && put) a.logp[t] = lp;
    if (!a.advantage) return 0.f;
    const float A = a.advantage[t];
    const float r = a.old_logp ? expf(lp - a.old_logp[t]) : 1.f;
    const float un = r * A, cl = fminf(fmaxf(r, 1.f - a.clip_low), 1.f + a.clip_high) * A;
    float l = -fminf(un, cl);
    float slope = un <= cl ? -un : 0.f;
    if (lp != lp) l = slope = lp;
    if (a.kl != 0.f) {
        const float u = a.ref_logp[t] - lp, eu = expm1f(u);
        l += a.kl * (u == INFINITY ? u : eu - u);
        slope -= a.kl * eu;
    }
    if (a.tok_loss && put) a.tok_loss[t] = w * l;
    return w * slope * a.inv_tau;
}

// What the gradient of one row needs: dz = c 1[v = target] - q 2^(k (z - top)).
struct RowGrad {
    float c, top, q;
    float lift;        // see grad_vec
};

// Gradient of one vector. Exponentials are computed as 2^(x + lift) with q carrying 2^-lift: the
// fast exponential flushes results below 2^-126, and with lift = 64 what it flushes is below
// the smallest fp32 number once multiplied by q.
template <typename T>
__device__ __forceinline__ uint4 grad_vec(const uint4& u, const RowGrad& g, float k) {
    uint64_t p[Pairs<T>::N];
    to_pairs<T>(u, p);
    const uint64_t minus = splat2(-g.top), kk = splat2(k), lift = splat2(g.lift), q = splat2(-g.q);
#pragma unroll
    for (int i = 0; i < Pairs<T>::N; ++i) {
        float x0, x1;
        upk2(fma2(add2(p[i], minus), kk, lift), x0, x1);
        p[i] = mul2(pk2(ex2_approx(x0), ex2_approx(x1)), q);
    }
    return from_pairs<T>(p);
}

template <typename T>
__device__ __forceinline__ T grad_one(float x, const RowGrad& g, float k, bool hot) {
    const float e = ex2_approx(fmaf(x - g.top, k, g.lift));
    return Elem<T>::from_f(fmaf(-g.q, e, hot ? g.c : 0.f));
}

// One token to a cluster of CTAs (1, 2, 4 or 8), each with its share of the row's 16-byte
// vectors; the first CTA also takes the elements before the first and after the last whole
// vector. Every CTA hands its (max, sum) to all others through distributed shared memory, and
// each computes the token's scalars for itself.
// kStaged: the share stays in shared memory between the sum and the gradient (one reading of
// the logits); else it is read again (log-probabilities alone, or rows past 8 x 72 KB). Both
// take the same vectors in the same order: a token's logp has the same bits from either.
template <typename T, bool kStaged>
__global__ void __launch_bounds__(kThreads, 3) policy_kernel(PolicyArgs a, const T* logits, T* dlogits) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ uint64_t full[kMaxPieces];
    __shared__ MaxSum part[kThreads / 32], peer[kMaxCluster];
    __shared__ RowGrad row;
    const int tid = threadIdx.x, nt = blockDim.x;
    uint32_t rank, cs;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    if (kStaged && tid == 0) {
        for (int i = 0; i < kMaxPieces; ++i) tc::mbar_init(&full[i], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    pdl_wait();
    const int t = blockIdx.x / cs;
    const float w = a.weight ? a.weight[t] : 1.f;
    const int target = a.target[t];
    if (target >= a.V && w != 0.f && rank == 0 && tid == 0) raise_error(a.err, kErrBounds);
    const bool kept = w != 0.f && (uint32_t)target < (uint32_t)a.V;
    const T* z = logits + t * a.ld;
    T* dz = dlogits ? dlogits + t * a.ld_grad : nullptr;
    const int V = a.V;
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(T)));
    const int nvec = (V - head) / N;
    const int share = (nvec + cs - 1) / cs;
    const int v0 = min(nvec, (int)rank * share), nv = min(nvec, v0 + share) - v0;
    const uint4* zv = reinterpret_cast<const uint4*>(z + head) + v0;
    const int rest = rank == 0 ? V - nvec * N : 0;
    const int odd = tid < head ? tid : nvec * N + tid;      // this thread's single element, if tid < rest
    // 16-byte stores need the gradient's row on the same alignment as the logits' row
    const bool wide = ((reinterpret_cast<uintptr_t>(z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
    if (!kept) {
        if (rank == 0 && tid == 0) {
            if (a.logp) a.logp[t] = 0.f;
            if (a.tok_loss) a.tok_loss[t] = 0.f;
        }
        if (dz) {
            const T zero = Elem<T>::from_f(0.f);
            if (wide) {
                uint4* o = reinterpret_cast<uint4*>(dz + head) + v0;
                for (int i = tid; i < nv; i += nt) o[i] = make_uint4(0u, 0u, 0u, 0u);
            } else {
                for (int i = tid; i < nv * N; i += nt) dz[head + v0 * N + i] = zero;
            }
            if (tid < rest) dz[odd] = zero;
        }
        return;      // every CTA of the cluster: none waits for another
    }
    // distributed shared memory may be written once every CTA of the cluster runs
    if (cs > 1) asm volatile("barrier.cluster.arrive.relaxed;" ::: "memory");
    if constexpr (kStaged) {
        if (tid == 0) {
            for (int i = 0, c = 0; i < nv; i += kPiece, ++c) {
                const uint32_t bytes = (uint32_t)min(kPiece, nv - i) * 16u;
                tc::mbar_expect_tx(&full[c], bytes);
                asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                             ::"r"(tc::smem_u32(stage) + i * 16), "l"(zv + i), "r"(bytes), "r"(tc::smem_u32(&full[c]))
                             : "memory");
            }
        }
        __syncthreads();     // the barriers are set up
    }
    const float k = a.inv_tau * kLog2e;
    // read before any CTA of the cluster may write the row (dlogits may be logits)
    const float zt = Elem<T>::to_f(z[target]);
    const float lone = tid < rest ? Elem<T>::to_f(z[odd]) : 0.f;
    const uint4* sv = reinterpret_cast<const uint4*>(stage);
    Running run{-INFINITY, 0};
    bool ok = true;
    if constexpr (kStaged) {
        for (int i0 = 0, c = 0; i0 < nv; i0 += kPiece, ++c) {
            ok = ok && tc::mbar_wait(&full[c], 0, a.err);
            const int end = min(i0 + kPiece, nv);
            int i = i0 + tid;
            for (; i + nt < end; i += 2 * nt) {
                const uint4 u[2] = {sv[i], sv[i + nt]};
                add_vecs<T, 2>(run, u, k);
            }
            if (i < end) {
                const uint4 u[1] = {sv[i]};
                add_vecs<T, 1>(run, u, k);
            }
        }
    } else {
        int i = tid;
        for (; i + 3 * nt < nv; i += 4 * nt) {
            const uint4 u[2] = {zv[i], zv[i + nt]}, v[2] = {zv[i + 2 * nt], zv[i + 3 * nt]};
            add_vecs<T, 2>(run, u, k);
            add_vecs<T, 2>(run, v, k);
        }
        for (; i + nt < nv; i += 2 * nt) {
            const uint4 u[2] = {zv[i], zv[i + nt]};
            add_vecs<T, 2>(run, u, k);
        }
        if (i < nv) {
            const uint4 u[1] = {zv[i]};
            add_vecs<T, 1>(run, u, k);
        }
    }
    float s0, s1;
    upk2(run.s, s0, s1);
    MaxSum acc{run.m, s0 + s1};
    if (tid < rest) acc = join(acc, MaxSum{lone, lone == -INFINITY ? 0.f : 1.f}, k);
#pragma unroll
    for (int o = 16; o > 0; o >>= 1)
        acc = join(acc, MaxSum{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o)}, k);
    if ((tid & 31) == 0) part[tid >> 5] = acc;
    __syncthreads();
    if (tid < 32) {
        acc = tid < nt / 32 ? part[tid] : MaxSum{-INFINITY, 0.f};
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc = join(acc, MaxSum{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o)}, k);
    }
    if (cs > 1) {
        asm volatile("barrier.cluster.wait;" ::: "memory");
        if (tid < (int)cs) {
            uint32_t to;
            asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(&peer[rank])), "r"(tid));
            asm volatile("st.shared::cluster.v2.f32 [%0], {%1, %2};" ::"r"(to), "f"(acc.m), "f"(acc.s) : "memory");
        }
        asm volatile("barrier.cluster.arrive.release;" ::: "memory");
        asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    }
    if (tid == 0) {
        if (cs > 1) {
            acc = peer[0];
            for (uint32_t i = 1; i < cs; ++i) acc = join(acc, peer[i], k);
        }
        RowGrad g;
        g.c = token_terms(a, t, rank == 0, w, zt, acc, k);
        g.top = acc.m;
        const float q = g.c / acc.s;
        g.lift = fabsf(q) > 9.0949470e-13f ? 64.f : 0.f;               // 2^-40
        g.q = g.lift != 0.f ? q * 5.4210109e-20f : q;                   // 2^-64
        row = g;
    }
    if (!dz) return;
    __syncthreads();
    const RowGrad g = row;
    const int hot = target - head - v0 * N;          // the target's place in this CTA's vectors
    const int hot_vec = hot >= 0 && hot < nv * N ? hot / N : -1;
    for (int i = tid; i < nv; i += nt) {
        const uint4 u = kStaged ? sv[i] : zv[i];
        uint4 o = grad_vec<T>(u, g, k);
        if (i == hot_vec) reinterpret_cast<T*>(&o)[hot % N] = grad_one<T>(zt, g, k, true);
        if (wide) {
            (reinterpret_cast<uint4*>(dz + head) + v0)[i] = o;
        } else {
            T* to = dz + head + (int64_t)(v0 + i) * N;
#pragma unroll
            for (int j = 0; j < N; ++j) to[j] = reinterpret_cast<const T*>(&o)[j];
        }
    }
    if (tid < rest) dz[odd] = grad_one<T>(lone, g, k, odd == target);
    (void)ok;            // a wait that ran out has set the error word
}

// loss = sum of the tokens' terms, one block, in a fixed order.
__global__ void __launch_bounds__(1024) policy_sum_kernel(const float* __restrict__ tok, int T, float* __restrict__ loss) {
    __shared__ float part[32];
    pdl_wait();
    float s = 0.f;
    for (int i = threadIdx.x; i < T; i += 1024) s += tok[i];
    s = warp_sum(s);
    if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = s;
    __syncthreads();
    if (threadIdx.x < 32) {
        s = warp_sum(part[threadIdx.x]);
        if (threadIdx.x == 0) *loss = s;
    }
}

template <typename T, bool kStaged>
cudaError_t launch_rows(const PolicyArgs& a, int cs, int threads, size_t smem, const T* z, T* dz, cudaStream_t s) {
    if (kStaged) {
        const cudaError_t e = cudaFuncSetAttribute(policy_kernel<T, kStaged>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                                   kStageBytes);
        if (e != cudaSuccess) return e;
    }
    // grids are numbered in 31 bits: a batch of more CTAs goes in several launches
    const int rows = (1 << 30) / cs;
    for (int64_t t0 = 0; t0 < a.T; t0 += rows) {
        PolicyArgs b = a;
        const int n = (int)std::min<int64_t>(rows, a.T - t0);
        b.target += t0;
        for (const float** p : {&b.advantage, &b.old_logp, &b.ref_logp, &b.weight})
            if (*p) *p += t0;
        if (b.logp) b.logp += t0;
        if (b.tok_loss) b.tok_loss += t0;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3((unsigned)n * cs);
        cfg.blockDim = dim3(threads);
        cfg.dynamicSmemBytes = smem;
        cfg.stream = s;
        cudaLaunchAttribute at[2];
        at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
        at[0].val.programmaticStreamSerializationAllowed = 1;
        at[1].id = cudaLaunchAttributeClusterDimension;
        at[1].val.clusterDim.x = cs;
        at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 2;
        const cudaError_t e = launch_ex(cfg, policy_kernel<T, kStaged>, b, z + t0 * a.ld, dz ? dz + t0 * a.ld_grad : dz);
        count_launch();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_policy(const PolicyArgs& a, const void* logits, void* dlogits, cudaStream_t s) {
    const int64_t vecs = a.V / Vec16<T>::N;
    auto share = [&](int cs) { return (vecs + cs - 1) / cs; };
    int cs = 1;
    while (cs < kMaxCluster && share(cs) * 16 > kStageBytes) cs *= 2;
    // for the gradient, rows that fit the cluster's shared memory are kept there
    const bool staged = dlogits && share(cs) * 16 <= kStageBytes;
    // few rows: a row over more CTAs, while SMs are idle and a share is long
    while (cs < kMaxCluster && (int64_t)a.T * cs * 2 <= num_sms() && share(cs) > 2 * kThreads) cs *= 2;
    const int threads = share(cs) >= 2 * kThreads ? kThreads : 128;
    const T* z = static_cast<const T*>(logits);
    T* dz = static_cast<T*>(dlogits);
    return staged ? launch_rows<T, true>(a, cs, threads, (size_t)share(cs) * 16, z, dz, s)
                  : launch_rows<T, false>(a, cs, threads, 0, z, dz, s);
}

moe_status_t check_policy(const moe_policy_config_t* c) {
    if (!c || c->T < 0 || c->V < 1 || c->ld < c->V || c->ld_grad < c->V) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (!(c->temperature > 0.f) || !std::isfinite(c->temperature) || !std::isfinite(1.f / c->temperature))
        return MOE_ERR_INVALID_ARG;
    if (!(c->clip_low >= 0.f && c->clip_low <= 1.f) || !(c->clip_high >= 0.f) || !std::isfinite(c->clip_high) ||
        !std::isfinite(c->kl_weight))
        return MOE_ERR_INVALID_ARG;
    if (c->V > (1 << 30) || c->ld > ((int64_t)1 << 40) || c->ld_grad > ((int64_t)1 << 40)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

cudaError_t run_policy(const moe_policy_config_t& c, PolicyArgs a, const void* logits, void* dlogits, cudaStream_t s) {
    a.T = c.T;
    a.V = c.V;
    a.ld = c.ld;
    a.ld_grad = c.ld_grad;
    a.inv_tau = 1.f / c.temperature;
    a.clip_low = c.clip_low;
    a.clip_high = c.clip_high;
    a.kl = c.kl_weight;
    a.err = device_error_word();
    return c.dtype == MOE_BF16 ? launch_policy<__nv_bfloat16>(a, logits, dlogits, s)
                               : launch_policy<float>(a, logits, dlogits, s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_policy_workspace_bytes(const moe_policy_config_t* cfg) {
    if (check_policy(cfg) != MOE_OK) return 0;
    return align_up(((size_t)cfg->T + 1) * sizeof(float), 256);
}

extern "C" MOE_API moe_status_t moe_policy_loss(const moe_policy_config_t* cfg, const void* logits,
                                                const int32_t* target, const float* advantage, const float* old_logp,
                                                const float* ref_logp, const float* weight, float* logp, float* loss,
                                                void* dlogits, void* ws, moe_stream_t stream) {
    const moe_status_t st = check_policy(cfg);
    if (st != MOE_OK) return st;
    if (cfg->T > 0 && (!logits || !target || !advantage || (cfg->kl_weight != 0.f && !ref_logp)))
        return MOE_ERR_INVALID_ARG;
    if (loss && !ws) return MOE_ERR_INVALID_ARG;
    if (dlogits && dlogits == logits && cfg->ld != cfg->ld_grad) return MOE_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(dlogits, 16) || misaligned(ws, 16)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {(const void*)target, (const void*)advantage, (const void*)old_logp, (const void*)ref_logp,
                          (const void*)weight, (const void*)logp, (const void*)loss})
        if (misaligned(p, 4)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    PolicyArgs a{};
    a.target = target;
    a.advantage = advantage;
    a.old_logp = old_logp;
    a.ref_logp = ref_logp;
    a.weight = weight;
    a.logp = logp;
    a.tok_loss = loss ? static_cast<float*>(ws) : nullptr;
    if (cfg->T > 0 && run_policy(*cfg, a, logits, dlogits, s) != cudaSuccess) return MOE_ERR_CUDA;
    if (loss) {
        const cudaError_t e = launch_pdl(policy_sum_kernel, dim3(1), dim3(1024), 0, s, static_cast<const float*>(ws),
                                         (int)cfg->T, loss);
        count_launch();
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    }
    return MOE_OK;
}

extern "C" MOE_API moe_status_t moe_token_logp(const moe_policy_config_t* cfg, const void* logits,
                                               const int32_t* target, float* logp, moe_stream_t stream) {
    const moe_status_t st = check_policy(cfg);
    if (st != MOE_OK) return st;
    if (cfg->T > 0 && (!logits || !target || !logp)) return MOE_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(target, 4) || misaligned(logp, 4)) return MOE_ERR_INVALID_ARG;
    if (cfg->T == 0) return MOE_OK;
    PolicyArgs a{};
    a.target = target;
    a.logp = logp;
    return run_policy(*cfg, a, logits, nullptr, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
