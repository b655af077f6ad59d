// Policy loss on the logits of the chosen tokens, its gradient, and token log-probabilities.
#include <cmath>

#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2 = 0.6931471805599453f;
constexpr int kWarps = 8;                     // warps that compute; one more warp loads
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
constexpr int kPiece = 1024;                  // 16-byte vectors of one bulk copy: four a thread
constexpr int kEach = kPiece / kThreads;
constexpr int kSlots = 7;                     // pieces in a CTA's ring: 112 KB, two CTAs to an SM
constexpr int kShare = 4;                     // pieces of a row that a CTA takes, while clusters last

// What becomes of a piece of a row after its sum was taken.
enum Reuse : int {
    kFree = 0,      // no gradient wanted: its slot takes the next piece
    kKeep = 1,      // it stays for the gradient: the logits are read once
    kAgain = 2,     // the share is longer than the ring: all of its pieces come a second time
};

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

// All lanes' pairs as one, in every lane.
__device__ __forceinline__ MaxSum warp_join(MaxSum a, float k) {
    float m = a.m;
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) m = fmaxf(m, __shfl_xor_sync(0xffffffffu, m, o));
    return {m, warp_sum(m == -INFINITY ? a.s : a.s * ex2_approx((a.m - m) * k))};
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
__device__ __forceinline__ float token_terms(const PolicyArgs& a, int64_t t, bool put, float w, float zt, MaxSum row,
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

__device__ __forceinline__ void consumers_sync() { asm volatile("bar.sync 1, %0;" ::"n"(kThreads) : "memory"); }

// Phase wait whose acquire covers what the other CTAs of the cluster have written.
__device__ __forceinline__ bool wait_cluster(uint64_t* bar, uint32_t parity, int* err) {
    const long long t0 = clock64();
    for (;;) {
        uint32_t done;
        asm volatile(
            "{\n\t.reg .pred p;\n\t"
            "mbarrier.try_wait.parity.acquire.cluster.shared::cta.b64 p, [%1], %2;\n\t"
            "selp.u32 %0, 1, 0, p;\n\t}"
            : "=r"(done)
            : "r"(tc::smem_u32(bar)), "r"(parity)
            : "memory");
        if (done) return true;
        if (clock64() - t0 > kSpinBudgetCycles) {
            raise_error(err, kErrTimeout);
            return false;
        }
    }
}

// This CTA's part of a row: whole 16-byte vectors, shared out over the cluster; the elements
// before the first and after the last whole vector are the first CTA's.
template <typename T>
struct Share {
    const T* z;
    int head, nvec, v0, nv, rest;
    __device__ __forceinline__ Share(const T* row, int V, uint32_t rank, uint32_t cs) : z(row) {
        constexpr int N = Vec16<T>::N;
        head = min(V, (int)(((16 - (reinterpret_cast<uintptr_t>(row) & 15)) & 15) / sizeof(T)));
        nvec = (V - head) / N;
        const int share = (nvec + (int)cs - 1) / (int)cs;
        v0 = min(nvec, (int)rank * share);
        nv = min(nvec, v0 + share) - v0;
        rest = rank == 0 ? V - nvec * N : 0;
    }
    __device__ __forceinline__ const uint4* vecs() const { return reinterpret_cast<const uint4*>(z + head) + v0; }
};

// Place in the ring: the slot, and the parity of its full barrier's phase.
struct Ring {
    uint32_t slot = 0, phase = 0;
    __device__ __forceinline__ void next() {
        if (++slot == kSlots) {
            slot = 0;
            phase ^= 1;
        }
    }
};

template <typename T>
__device__ __forceinline__ void put_elements(T* to, const uint4& o) {
    const uint32_t w[4] = {o.x, o.y, o.z, o.w};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        if constexpr (sizeof(T) == 2) {
            reinterpret_cast<uint16_t*>(to)[2 * i] = (uint16_t)w[i];
            reinterpret_cast<uint16_t*>(to)[2 * i + 1] = (uint16_t)(w[i] >> 16);
        } else {
            reinterpret_cast<uint32_t*>(to)[i] = w[i];
        }
    }
}

// Rows over clusters of 1, 2, 4 or 8 CTAs, two CTAs to an SM, resident for the whole batch: a
// cluster takes every n-th row. In each CTA one warp keeps a ring of bulk copies running, rows
// ahead of the eight that compute, so that the loads of the next row pass under the
// reductions, the cluster's exchange and the gradient's stores of this one. Each CTA hands its
// (max, sum) to all CTAs of the cluster by asynchronous remote stores that complete on the
// receiver's barrier, and computes the token's scalars for itself.
// All uses (gradient or not) take a row's vectors in the same order: a token's logp has the
// same bits from each.
template <typename T>
__global__ void __launch_bounds__(kThreads + 32, 2)
policy_ring_kernel(PolicyArgs a, const T* logits, T* dlogits, int reuse) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ uint64_t full[kSlots], empty[kSlots], xbar[2];
    __shared__ MaxSum part[kWarps];
    __shared__ __align__(8) MaxSum peer[2][kMaxCluster];
    __shared__ RowGrad row;
    const int tid = threadIdx.x, lane = tid & 31;
    uint32_t rank, cs;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], kWarps);
        }
        tc::mbar_init(&xbar[0], 1);
        tc::mbar_init(&xbar[1], 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
    }
    __syncthreads();
    // remote stores may come once every CTA of the cluster has its barriers
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
    pdl_wait();
    const int first = blockIdx.x / cs, stride = gridDim.x / cs;
    const auto kept_row = [&](float w, int target) { return w != 0.f && (uint32_t)target < (uint32_t)a.V; };

    if (tid >= kThreads) {
        // ---- the loading warp: looks 32 of its rows ahead for the ones that are not left out
        Ring at;
        bool ok = true, reused = false;
        for (int64_t t0 = first; t0 < a.T && ok; t0 += 32LL * stride) {
            const int64_t tl = t0 + (int64_t)lane * stride;
            const uint32_t rows = __ballot_sync(
                0xffffffffu, tl < a.T && kept_row(a.weight ? a.weight[tl] : 1.f, a.target[tl]));
            if (lane == 0)
                for (uint32_t left = rows; left && ok; left &= left - 1) {
                    const Share<T> s(logits + (t0 + (int64_t)(__ffs(left) - 1) * stride) * a.ld, a.V, rank, cs);
                    for (int pass = 0; pass < (reuse == kAgain ? 2 : 1); ++pass)
                        for (int i = 0; i < s.nv && ok; i += kPiece) {
                            const uint32_t slot = at.slot;
                            if (reused && !tc::mbar_wait(&empty[slot], at.phase ^ 1, a.err)) {
                                ok = false;
                                break;
                            }
                            at.next();
                            reused = reused || at.slot == 0;
                            const uint32_t bytes = (uint32_t)min(kPiece, s.nv - i) * 16u;
                            tc::mbar_expect_tx(&full[slot], bytes);
                            asm volatile(
                                "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                                ::"r"(tc::smem_u32(stage) + slot * (kPiece * 16u)), "l"(s.vecs() + i), "r"(bytes),
                                "r"(tc::smem_u32(&full[slot]))
                                : "memory");
                        }
                }
            ok = __shfl_sync(0xffffffffu, (int)ok, 0);
        }
    } else {
        const float k = a.inv_tau * kLog2e;
        Ring at;
        uint32_t turn = 0;                     // kept rows so far
        bool ok = true;
        for (int64_t t = first; t < a.T; t += stride) {
            const float w = a.weight ? a.weight[t] : 1.f;
            const int target = a.target[t];
            const Share<T> s(logits + t * a.ld, a.V, rank, cs);
            T* dz = dlogits ? dlogits + t * a.ld_grad : nullptr;
            // 16-byte stores need the gradient's row on the same alignment as the logits' row
            const bool wide = ((reinterpret_cast<uintptr_t>(s.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
            uint4* out = reinterpret_cast<uint4*>(dz + s.head) + s.v0;
            const int odd = tid < s.head ? tid : s.nvec * N + tid;   // this thread's single element, if tid < rest
            if (!kept_row(w, target)) {
                if (rank == 0 && tid == 0) {
                    if (w != 0.f && target >= a.V) raise_error(a.err, kErrBounds);
                    if (a.logp) a.logp[t] = 0.f;
                    if (a.tok_loss) a.tok_loss[t] = 0.f;
                }
                if (dz) {
                    const T zero = Elem<T>::from_f(0.f);
                    if (wide)
                        for (int i = tid; i < s.nv; i += kThreads) out[i] = make_uint4(0u, 0u, 0u, 0u);
                    else
                        for (int i = tid; i < s.nv * N; i += kThreads) dz[s.head + s.v0 * N + i] = zero;
                    if (tid < s.rest) dz[odd] = zero;
                }
                continue;
            }
            const float zt = tid == 0 ? Elem<T>::to_f(s.z[target]) : 0.f;
            const float lone = tid < s.rest ? Elem<T>::to_f(s.z[odd]) : 0.f;
            // ---- sum
            Running run{-INFINITY, 0};
            const Ring at0 = at;
            for (int i0 = 0; i0 < s.nv; i0 += kPiece, at.next()) {
                ok = ok && tc::mbar_wait(&full[at.slot], at.phase, a.err);
                const uint4* v = reinterpret_cast<const uint4*>(stage + at.slot * (kPiece * 16)) + tid;
                const int left = s.nv - i0 - tid;
                if (left > kPiece - kThreads) {
                    uint4 u[kEach];
#pragma unroll
                    for (int h = 0; h < kEach; ++h) u[h] = v[h * kThreads];
                    add_vecs<T, kEach>(run, u, k);
                } else {
#pragma unroll 1
                    for (int j = 0; j < left; j += kThreads) {
                        const uint4 u[1] = {v[j]};
                        add_vecs<T, 1>(run, u, k);
                    }
                }
                if (reuse != kKeep) {
                    __syncwarp();
                    if (lane == 0) tc::mbar_arrive(&empty[at.slot]);
                }
            }
            float s0, s1;
            upk2(run.s, s0, s1);
            MaxSum acc{run.m, s0 + s1};
            if (tid < s.rest) acc = join(acc, MaxSum{lone, lone == -INFINITY ? 0.f : 1.f}, k);
            acc = warp_join(acc, k);
            if (lane == 0) part[tid >> 5] = acc;
            consumers_sync();
            if (tid < 32) {
                acc = warp_join(lane < kWarps ? part[lane] : MaxSum{-INFINITY, 0.f}, k);
                if (cs > 1) {
                    const uint32_t b = turn & 1;
                    if (lane == 0) tc::mbar_expect_tx(&xbar[b], cs * (uint32_t)sizeof(MaxSum));
                    // the target's logit has arrived before a peer can write over it (dlogits may be logits)
                    asm volatile("" ::"f"(zt), "f"(lone) : "memory");
                    if (lane < (int)cs) {
                        uint32_t to, bar;
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(to) : "r"(tc::smem_u32(&peer[b][rank])), "r"(lane));
                        asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(tc::smem_u32(&xbar[b])), "r"(lane));
                        asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                                     ::"r"(to), "r"(__float_as_uint(acc.m)), "r"(__float_as_uint(acc.s)), "r"(bar)
                                     : "memory");
                    }
                    __syncwarp();
                    ok = wait_cluster(&xbar[b], (turn >> 1) & 1, a.err) && ok;
                    acc = warp_join(lane < (int)cs ? peer[b][lane] : MaxSum{-INFINITY, 0.f}, k);
                }
                if (lane == 0) {
                    RowGrad g;
                    g.c = token_terms(a, t, rank == 0, w, zt, acc, k);
                    g.top = acc.m;
                    const float q = g.c / acc.s;
                    g.lift = fabsf(q) > 9.0949470e-13f ? 64.f : 0.f;               // 2^-40
                    g.q = g.lift != 0.f ? q * 5.4210109e-20f : q;                   // 2^-64
                    row = g;
                }
            }
            ++turn;
            consumers_sync();
            if (!dz) continue;
            // ---- gradient
            const RowGrad g = row;
            const int hot = target - s.head - s.v0 * N;      // the target's place in this CTA's vectors
            const int hot_vec = hot >= 0 && hot < s.nv * N ? hot / N : -1;
            if (reuse == kKeep) at = at0;
            for (int i0 = 0; i0 < s.nv; i0 += kPiece, at.next()) {
                if (reuse == kAgain) ok = ok && tc::mbar_wait(&full[at.slot], at.phase, a.err);
                const uint4* v = reinterpret_cast<const uint4*>(stage + at.slot * (kPiece * 16)) + tid;
                const int left = s.nv - i0 - tid;
                if (wide && left > kPiece - kThreads) {
                    uint4* o = out + i0 + tid;
#pragma unroll
                    for (int h = 0; h < kEach; ++h) o[h * kThreads] = grad_vec<T>(v[h * kThreads], g, k);
                } else {
#pragma unroll 1
                    for (int j = 0; j < min(left, kPiece - tid); j += kThreads) {
                        const uint4 o = grad_vec<T>(v[j], g, k);
                        if (wide) out[i0 + tid + j] = o;
                        else put_elements<T>(dz + s.head + (int64_t)(s.v0 + i0 + tid + j) * N, o);
                    }
                }
                // the target's element again, by the thread that has just written its vector
                const int mine = hot_vec - i0 - tid;
                if (hot_vec >= 0 && mine >= 0 && mine < kPiece - tid && mine % kThreads == 0)
                    dz[target] = grad_one<T>(Elem<T>::to_f(reinterpret_cast<const T*>(v + mine)[hot % N]), g, k, true);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&empty[at.slot]);
            }
            if (tid < s.rest) dz[odd] = grad_one<T>(lone, g, k, odd == target);
        }
        (void)ok;            // a wait that ran out has set the error word
    }
    // no CTA leaves while another of its cluster may still write to it
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
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

// Clusters of `cs` CTAs that are resident at once (asked of the runtime once for each type and
// size on a device).
template <typename T>
cudaError_t resident_clusters(int cs, size_t smem, int* out) {
    constexpr int kMaxDevices = 64;
    static std::mutex mu;
    static int known[kMaxDevices][kMaxCluster + 1];
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess) return e;
    if (dev < 0 || dev >= kMaxDevices) return cudaErrorInvalidDevice;
    std::lock_guard<std::mutex> lk(mu);
    int& n = known[dev][cs];
    if (!n) {
        e = cudaFuncSetAttribute(policy_ring_kernel<T>, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)smem);
        if (e != cudaSuccess) return e;
        cudaLaunchConfig_t cfg{};
        cfg.gridDim = dim3(num_sms() * 2 / cs * cs);
        cfg.blockDim = dim3(kThreads + 32);
        cfg.dynamicSmemBytes = smem;
        cudaLaunchAttribute at[1];
        at[0].id = cudaLaunchAttributeClusterDimension;
        at[0].val.clusterDim.x = cs;
        at[0].val.clusterDim.y = at[0].val.clusterDim.z = 1;
        cfg.attrs = at;
        cfg.numAttrs = 1;
        e = cudaOccupancyMaxActiveClusters(&n, policy_ring_kernel<T>, &cfg);
        if (e != cudaSuccess) {
            n = 0;
            return e;
        }
        n = std::max(n, 1);
    }
    *out = n;
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_policy(const PolicyArgs& a, const void* logits, void* dlogits, cudaStream_t s) {
    constexpr size_t smem = (size_t)kSlots * kPiece * 16;
    const int64_t vecs = a.V / Vec16<T>::N;
    const auto pieces = [&](int cs) { return (vecs + (int64_t)cs * kPiece - 1) / ((int64_t)cs * kPiece); };
    int cs = 1;
    while (cs < kMaxCluster && pieces(cs) > kShare) cs *= 2;
    // few rows: a row over more CTAs, while SMs are idle and a share is longer than a piece
    while (cs < kMaxCluster && (int64_t)a.T * cs * 2 <= num_sms() && pieces(cs) > 1) cs *= 2;
    const int reuse = !dlogits ? kFree : pieces(cs) <= kSlots ? kKeep : kAgain;
    int clusters = 0;
    cudaError_t e = resident_clusters<T>(cs, smem, &clusters);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)std::min(a.T, clusters) * cs);
    cfg.blockDim = dim3(kThreads + 32);
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
    e = launch_ex(cfg, policy_ring_kernel<T>, a, static_cast<const T*>(logits), static_cast<T*>(dlogits), reuse);
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
