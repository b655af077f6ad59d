// Policy loss on the logits of the chosen tokens, its gradient, and token log-probabilities.
#include <cmath>

#include "internal.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kThreads = 512;

// 2^x for the gradient: unlike ex2_approx, results below 2^-126 are not flushed to zero (in the
// sum they are far below its rounding).
__device__ __forceinline__ float ex2_tail(float x) {
    float r;
    asm("ex2.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

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

template <typename T>
__device__ __forceinline__ void add_chunk(MaxSum& a, const float (&x)[Vec16<T>::N], float k) {
    float top = x[0];
#pragma unroll
    for (int i = 1; i < Vec16<T>::N; ++i) top = fmaxf(top, x[i]);
    if (top > a.m) {
        a.s *= ex2_approx((a.m - top) * k);
        a.m = top;
    }
    // a row of -inf so far: measured from 0, so that -inf gives 0 and not NaN
    const float m = a.m == -INFINITY ? 0.f : a.m;
#pragma unroll
    for (int i = 0; i < Vec16<T>::N; ++i) a.s += ex2_approx((x[i] - m) * k);
}

// What one token adds: its log-probability, its term of the loss, and the factor c of its
// gradient row c (1[v = target] - p_v).
__device__ __forceinline__ float token_terms(const PolicyArgs& a, int t, float w, float zt, MaxSum row, float k) {
    // a row of -inf alone has no distribution
    const float lp = row.s != 0.f ? ((zt - row.m) * k - log2f(row.s)) * kLn2 : NAN;
    if (a.logp) a.logp[t] = lp;
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
    if (a.tok_loss) a.tok_loss[t] = w * l;
    return w * slope * a.inv_tau;
}

// One block a token.
template <typename T>
__global__ void __launch_bounds__(kThreads) policy_kernel(PolicyArgs a, const T* logits, T* dlogits) {
    constexpr int N = Vec16<T>::N;
    __shared__ MaxSum part[kThreads / 32];
    __shared__ float sh[3];
    pdl_wait();
    const int t = blockIdx.x;
    const float w = a.weight ? a.weight[t] : 1.f;
    const int target = a.target[t];
    if (target >= a.V && w != 0.f && threadIdx.x == 0) raise_error(a.err, kErrBounds);
    const bool kept = w != 0.f && (uint32_t)target < (uint32_t)a.V;
    const T* z = logits + t * a.ld;
    T* dz = dlogits ? dlogits + t * a.ld_grad : nullptr;
    const int V = a.V;
    const int head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(z) & 15)) & 15) / sizeof(T)));
    const int nvec = (V - head) / N;
    const float k = a.inv_tau * kLog2e;
    float c = 0.f, top = 0.f, q = 0.f;
    if (kept) {
        MaxSum acc{-INFINITY, 0.f};
        for (int i = threadIdx.x; i < nvec; i += kThreads) {
            float x[N];
            const uint4 u = *reinterpret_cast<const uint4*>(z + head + (int64_t)i * N);
            unpack16<T>(u, x);
            add_chunk<T>(acc, x, k);
        }
        const int rest = V - nvec * N;      // the unaligned head and tail
        if ((int)threadIdx.x < rest) {
            const int v = (int)threadIdx.x < head ? (int)threadIdx.x : head + nvec * N + ((int)threadIdx.x - head);
            const float x = Elem<T>::to_f(z[v]);
            acc = join(acc, MaxSum{x, x == -INFINITY ? 0.f : 1.f}, k);
        }
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            acc = join(acc, MaxSum{__shfl_xor_sync(0xffffffffu, acc.m, o), __shfl_xor_sync(0xffffffffu, acc.s, o)}, k);
        if ((threadIdx.x & 31) == 0) part[threadIdx.x >> 5] = acc;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kThreads / 32; ++i) acc = join(acc, part[i], k);
            sh[0] = token_terms(a, t, w, Elem<T>::to_f(z[target]), acc, k);
            sh[1] = acc.m;
            sh[2] = acc.s;
        }
        __syncthreads();
        c = sh[0];
        top = sh[1];
        q = c / sh[2];
    } else if (threadIdx.x == 0) {
        if (a.logp) a.logp[t] = 0.f;
        if (a.tok_loss) a.tok_loss[t] = 0.f;
    }
    if (!dz) return;
    if (kept) {
        for (int v = threadIdx.x; v < V; v += kThreads) {
            const float e = ex2_tail((Elem<T>::to_f(z[v]) - top) * k);
            dz[v] = Elem<T>::from_f(fmaf(-q, e, v == target ? c : 0.f));
        }
    } else {
        for (int v = threadIdx.x; v < V; v += kThreads) dz[v] = Elem<T>::from_f(0.f);
    }
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

template <typename T>
cudaError_t launch_policy(const PolicyArgs& a, const void* logits, void* dlogits, cudaStream_t s) {
    const cudaError_t e = launch_pdl(policy_kernel<T>, dim3(a.T), dim3(kThreads), 0, s, a,
                                     static_cast<const T*>(logits), static_cast<T*>(dlogits));
    count_launch();
    return e;
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
