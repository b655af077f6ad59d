// Policy loss on the logits of the chosen tokens, its gradient, and token log-probabilities.
#include <cmath>

#include "pairs.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

constexpr float kLog2e = 1.4426950408889634f;
constexpr float kLn2High = 0.693145751953125f, kLn2Low = 1.4286068203094172e-6f;   // 16 bits, and the rest
constexpr int kWarps = 8;                     // warps that compute; one more warp loads
constexpr int kThreads = 32 * kWarps;
constexpr int kMaxCluster = 8;
constexpr int kEach = 4;                      // 16-byte vectors of a piece to a thread
constexpr int kPiece = kEach * kThreads;      // vectors of one bulk copy: 16 KB
constexpr int kSlots = 6;                     // pieces in a CTA's ring: two CTAs to an SM
constexpr int kHeld = 8;                      // vectors a thread holds of a short row
constexpr int kShare = 4;                     // pieces of a row that a CTA takes, while clusters last

// What becomes of a piece of a row after its sum was taken.
enum Reuse : int {
    kFree = 0,      // no gradient wanted: its slot takes the next piece
    kKeep = 1,      // it stays for the gradient: the logits are read once
    kAgain = 2,     // the share is longer than the ring: all of its pieces come a second time
};

// The mathematics. One pass over a row keeps a running maximum m and s = sum_v 2^(k (z_v - m)); two
// such pairs join by scaling both to the larger maximum. Then
//   lp = (z_target - m) / tau - ln s,   dz_v = c (1[v = target] - 2^(k (z_v - m)) / s),
// with the factor c from lp and the token's scalars alone, so the row need not be read from memory
// again if it is still on the chip. Sums and statistics are fp32; dlogits are rounded once.

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
    float tau, inv_tau, clip_low, clip_high, kl;
    int* err;
};

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

// A row, as the loading warp hands it to the computing warps.
struct Row {
    int t;             // token, or -1 past the last
    int target;
    float w;           // 0: left out
};

// A kept row's scalars, loaded when its work begins.
struct Token {
    int t;
    float w, zt, adv, old, ref;
};

// a + b, and what its rounding lost: exact whichever is the larger (Knuth's two-sum).
__device__ __forceinline__ float exact_sum(float a, float b, float& lost) {
    const float s = a + b, of_b = s - a;
    lost = (a - (s - of_b)) + (b - of_b);
    return s;
}

// What one token adds: its log-probability and its term of the loss (written if `put`), and the
// factor c of its gradient row c (1[v = target] - p_v).
__device__ __forceinline__ float token_terms(const PolicyArgs& a, const Token& r, bool put, MaxSum row) {
    // lp = (z - max) / tau - ln(sum), with the sum as 2^e f: the quotient's and the partial sums'
    // roundings are kept in `low`, so that the ratios to other policies, which differ by a little
    // from numbers of ten and more, do not lose them. e times the upper part of ln 2 is exact.
    const float d = r.zt - row.m, q = d * a.inv_tau, q_low = fmaf(-q, a.tau, d) * a.inv_tau;
    const int e = (int)(__float_as_uint(row.s) >> 23) - 127;
    const float f = __uint_as_float((__float_as_uint(row.s) & 0x7fffffu) | 0x3f800000u);
    float hi_low, sum_low;
    const float hi = exact_sum(q, -(float)e * kLn2High, hi_low);
    const float ln_f = fmaf((float)e, kLn2Low, logf(f));
    const float sum = exact_sum(hi, -ln_f, sum_low), low = sum_low + hi_low + q_low;
    float lp = sum, lp_low = low;
    if (!(fabsf(q) <= 3.4028235e38f) || !(row.s >= 1.f && row.s <= 3.4028235e38f)) {
        // a target of -inf has the log-probability -inf; a row of -inf alone, or with a NaN or
        // +inf in it, has no distribution
        lp = row.s >= 1.f && row.s <= 3.4028235e38f ? q : NAN;
        lp_low = 0.f;
    }
    if (a.logp && put) a.logp[r.t] = lp;
    if (!a.advantage) return 0.f;
    // an old log-probability that is this one, rounded as this one is, stands for the same policy: its
    // low part is not known, and the ratio is one
    const float ratio = !a.old_logp || lp == r.old ? 1.f : expf(lp - r.old + lp_low);
    const float un = ratio * r.adv, cl = fminf(fmaxf(ratio, 1.f - a.clip_low), 1.f + a.clip_high) * r.adv;
    float l = -fminf(un, cl);
    float slope = un <= cl ? -un : 0.f;
    if (lp != lp) l = slope = lp;
    if (a.kl != 0.f) {
        const float u = r.ref - lp - lp_low, eu = expm1f(u);
        l += a.kl * (u == INFINITY ? u : eu - u);
        slope -= a.kl * eu;
    }
    if (a.tok_loss && put) a.tok_loss[r.t] = r.w * l;
    return r.w * slope * a.inv_tau;
}

// What the gradient of one row needs: dz = c 1[v = target] - q 2^(k (z - top)). The fast exponential
// flushes results below 2^-126, which a gradient element times q need not be.
//   bf16: 2^(x + lift), with q carrying 2^-lift. With lift = 64 what is flushed is below the smallest
//     fp32 number once multiplied by q. An exponent near 0 loses six bits to the sum: probabilities
//     are off by up to 2e-6, a thousandth of what the rounding to bf16 then adds.
//   fp32: the square of 2^(x / 2), multiplied into q one factor at a time; halving is exact, and what
//     the root flushes is below 2^-252 in the square. One multiplication more a pair, which bf16 rows
//     do not hide (8192 x 131072: 619 us against 606) and fp32 rows do (4096 x 131072: 578 and 578).
template <typename T>
struct RowGrad {
    static constexpr bool kLift = sizeof(T) == 2;
    float c, top, q, k, lift;
    __device__ __forceinline__ RowGrad(float c_, MaxSum row, float k_) : c(c_), top(row.m), q(c_ / row.s), k(k_), lift(0.f) {
        if constexpr (kLift) {
            lift = fabsf(q) > 9.0949470e-13f ? 64.f : 0.f;              // 2^-40
            q = lift != 0.f ? q * 5.4210109e-20f : q;                    // 2^-64
        } else {
            k *= 0.5f;
        }
    }
};

// Gradient of one vector.
template <typename T>
__device__ __forceinline__ uint4 grad_vec(const uint4& u, const RowGrad<T>& g) {
    uint64_t p[Pairs<T>::N];
    to_pairs<T>(u, p);
    const uint64_t minus = splat2(-g.top), k = splat2(g.k), lift = splat2(g.lift), q = splat2(-g.q);
#pragma unroll
    for (int i = 0; i < Pairs<T>::N; ++i) {
        float x0, x1;
        const uint64_t d = add2(p[i], minus);
        if constexpr (RowGrad<T>::kLift) {
            upk2(fma2(d, k, lift), x0, x1);
            p[i] = mul2(pk2(ex2_approx(x0), ex2_approx(x1)), q);
        } else {
            upk2(mul2(d, k), x0, x1);
            const uint64_t e = pk2(ex2_approx(x0), ex2_approx(x1));
            p[i] = mul2(mul2(e, q), e);
        }
    }
    return from_pairs<T>(p);
}

template <typename T>
__device__ __forceinline__ T grad_one(float x, const RowGrad<T>& g, bool hot) {
    const float c = hot ? g.c : 0.f;
    if constexpr (RowGrad<T>::kLift) {
        return Elem<T>::from_f(fmaf(-g.q, ex2_approx(fmaf(x - g.top, g.k, g.lift)), c));
    } else {
        const float e = ex2_approx((x - g.top) * g.k);
        return Elem<T>::from_f(fmaf(-g.q * e, e, c));
    }
}

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

// Place in a ring of SLOTS: the slot, the parity of its barrier's phase, and whether it was used before.
template <int SLOTS>
struct Ring {
    int slot = 0;
    uint32_t phase = 0;
    bool again = false;
    __device__ __forceinline__ void next() {
        if (++slot == SLOTS) {
            slot = 0;
            phase ^= 1;
            again = true;
        }
    }
    __device__ __forceinline__ void from(int src) {      // as lane src has it
        const uint32_t all = __shfl_sync(0xffffffffu, (uint32_t)slot | phase << 8 | (uint32_t)again << 9, src);
        slot = all & 255;
        phase = all >> 8 & 1;
        again = all >> 9;
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

constexpr int kRows = 8;        // rows handed over and not yet taken

// Long rows (over 32 KB): rows over clusters of 1, 2, 4 or 8 CTAs, two CTAs to an SM, resident for
// the whole batch. In
// each CTA one warp keeps a ring of bulk copies running, rows ahead of the eight that compute,
// so that the loads of the next rows pass under this row's reductions, exchange and stores. The
// rows that are not left out are dealt out evenly, and so are the others, whose gradient is
// only zeroed.
// The eight warps of a CTA never meet at a barrier: each sends the (max, sum) of its vectors to
// every CTA of the cluster by an asynchronous remote store that completes on the receiver's
// barrier, waits there for all of them, and works out the token's scalars for itself.
// All uses (gradient or not) take a row's vectors in the same order: a token's logp has the
// same bits from each.
// Bound by memory: a kept row is read once and written once, about 14 instructions and two
// exponentials an element lie beside four bytes of bf16. 8192 x 131072 bf16, a fifth left out:
// 611 us, 6330 GB/s of needed traffic (94 % of the copy rate); log-probabilities of 4096 x 32000
// fp32: 82 us, 6410 GB/s. On the way: one block a row, read again for the gradient, 1890 us; a CTA
// a share without the ring, 818; the ring with barriers in the CTA, 699. Shares of two pieces
// instead of four (clusters twice as large): 760 against 594; 16 warps with two vectors each: 830;
// pieces of 8 KB: 675.
template <typename T>
__global__ void __launch_bounds__(kThreads + 32, 2)
policy_ring_kernel(PolicyArgs a, const T* logits, T* dlogits, int reuse) {
    constexpr int N = Vec16<T>::N;
    extern __shared__ __align__(128) unsigned char stage[];
    __shared__ uint64_t full[kSlots], empty[kSlots], given[kRows], taken[kRows], xbar[2];
    __shared__ __align__(8) MaxSum peer[2][kMaxCluster * kWarps];
    __shared__ Row rows[kRows];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    uint32_t rank, cs;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(rank));
    asm volatile("mov.u32 %0, %%cluster_nctarank;" : "=r"(cs));
    if (tid == 0) {
        for (int i = 0; i < kSlots; ++i) {
            tc::mbar_init(&full[i], 1);
            tc::mbar_init(&empty[i], kWarps);
        }
        for (int i = 0; i < kRows; ++i) {
            tc::mbar_init(&given[i], 1);
            tc::mbar_init(&taken[i], kWarps);
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

    if (warp == kWarps) {
        // ---- the loading warp
        const uint32_t clusters = gridDim.x / cs, mine = blockIdx.x / cs;
        uint32_t skip_kept = mine, skip_out = mine;    // rows of each sort before the next that is dealt here
        Ring<kSlots> at;
        Ring<kRows> to;
        bool ok = true;
        constexpr int kAhead = 4;
        float w[kAhead], w_next[kAhead];
        int target[kAhead], target_next[kAhead];
        const auto look = [&](int64_t t0) {
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                const int64_t t = t0 + 32 * h + lane;
                w_next[h] = t < a.T && a.weight ? a.weight[t] : 1.f;
                target_next[h] = t < a.T ? a.target[t] : -1;
            }
        };
        look(0);
        for (int64_t t0 = 0; t0 < a.T && ok; t0 += 32 * kAhead) {
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                w[h] = w_next[h];
                target[h] = target_next[h];
            }
            look(t0 + 32 * kAhead);      // in flight while these rows are dealt out
#pragma unroll
            for (int h = 0; h < kAhead; ++h) {
                const int64_t t = t0 + 32 * h + lane;
                if (t0 + 32 * h >= a.T) break;
                const bool kept = w[h] != 0.f && (uint32_t)target[h] < (uint32_t)a.V;
                const uint32_t all = __ballot_sync(0xffffffffu, t < a.T), in = __ballot_sync(0xffffffffu, kept);
                const uint32_t kept_here = __popc(in), out_here = __popc(all & ~in);
                if (skip_kept >= kept_here && skip_out >= out_here) {
                    skip_kept -= kept_here;
                    skip_out -= out_here;
                    continue;
                }
                const uint32_t before = __popc((kept ? in : all & ~in) & ((1u << lane) - 1u)), skip = kept ? skip_kept : skip_out;
                const bool me = t < a.T && before >= skip && (before - skip) % clusters == 0;
                while (skip_kept < kept_here) skip_kept += clusters;
                while (skip_out < out_here) skip_out += clusters;
                skip_kept -= kept_here;
                skip_out -= out_here;
                if (me && !kept && w[h] != 0.f && target[h] >= a.V) raise_error(a.err, kErrBounds);
                for (uint32_t left = __ballot_sync(0xffffffffu, me); left && ok; left &= left - 1) {
                    if (lane == __ffs(left) - 1) {
                        ok = !to.again || tc::mbar_wait(&taken[to.slot], to.phase ^ 1, a.err);
                        if (ok) {
                            rows[to.slot] = Row{(int)t, target[h], kept ? w[h] : 0.f};
                            tc::mbar_arrive(&given[to.slot]);
                        }
                        const Share<T> s(logits + t * a.ld, a.V, rank, cs);
                        for (int pass = kept ? reuse == kAgain ? 0 : 1 : 2; pass < 2; ++pass)
                            for (int i = 0; i < s.nv && ok; i += kPiece) {
                                ok = !at.again || tc::mbar_wait(&empty[at.slot], at.phase ^ 1, a.err);
                                if (!ok) break;
                                const uint32_t bytes = (uint32_t)min(kPiece, s.nv - i) * 16u;
                                tc::mbar_expect_tx(&full[at.slot], bytes);
                                asm volatile(
                                    "cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                                    ::"r"(tc::smem_u32(stage) + at.slot * (kPiece * 16u)), "l"(s.vecs() + i), "r"(bytes),
                                    "r"(tc::smem_u32(&full[at.slot]))
                                    : "memory");
                                at.next();
                            }
                    }
                    const int src = __ffs(left) - 1;
                    ok = __shfl_sync(0xffffffffu, (int)ok, src);
                    at.from(src);
                    to.next();
                }
            }
        }
        if (lane == 0 && ok && (!to.again || tc::mbar_wait(&taken[to.slot], to.phase ^ 1, a.err))) {
            rows[to.slot] = Row{-1, 0, 0.f};
            tc::mbar_arrive(&given[to.slot]);
        }
        // No copy is in flight when the CTA leaves, also where a wait ran out and nobody takes the
        // pieces any more: lane i waits for the last copy into slot i.
        __syncwarp();
        if (lane < kSlots && (lane < at.slot || at.again))
            tc::mbar_wait(&full[lane], lane < at.slot ? at.phase : at.phase ^ 1, a.err);
    } else {
        const float k = a.inv_tau * kLog2e;
        Ring<kSlots> at;
        Ring<kRows> from;
        uint32_t turn = 0;                     // kept rows so far
        bool ok = true;
        Token before{};
        // A warp's pair to every CTA of the cluster; all pairs of the cluster as one. The two
        // buffers suffice: whoever sends for a row has received all pairs of the row before it,
        // whose senders have read those of the row before that.
        const auto send = [&](MaxSum acc, uint32_t row) {
            const uint32_t b = row & 1;
            if (tid == 0) tc::mbar_expect_tx(&xbar[b], cs * kWarps * (uint32_t)sizeof(MaxSum));
            if (lane < (int)cs) {
                uint32_t to, bar;
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;"
                             : "=r"(to) : "r"(tc::smem_u32(&peer[b][rank * kWarps + warp])), "r"(lane));
                asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(bar) : "r"(tc::smem_u32(&xbar[b])), "r"(lane));
                asm volatile("st.async.weak.shared::cluster.mbarrier::complete_tx::bytes.v2.b32 [%0], {%1, %2}, [%3];"
                             ::"r"(to), "r"(__float_as_uint(acc.m)), "r"(__float_as_uint(acc.s)), "r"(bar)
                             : "memory");
            }
            __syncwarp();
        };
        const auto receive = [&](uint32_t row) {
            const uint32_t b = row & 1;
            ok = wait_cluster(&xbar[b], (row >> 1) & 1, a.err) && ok;
            const int n = (int)cs * kWarps;
            MaxSum acc = lane < n ? peer[b][lane] : MaxSum{-INFINITY, 0.f};
            if (lane + 32 < n) acc = join(acc, peer[b][lane + 32], k);
            return warp_join(acc, k);
        };
        const auto finish = [&](const Token& x, MaxSum sum) {
            if (rank == 0 && warp == 0) token_terms(a, x, lane == 0, sum);
        };
        while (ok) {
            if (!tc::mbar_wait(&given[from.slot], from.phase, a.err)) break;
            const Row r = rows[from.slot];
            __syncwarp();
            if (lane == 0) tc::mbar_arrive(&taken[from.slot]);
            from.next();
            if (r.t < 0) break;
            const Share<T> s(logits + r.t * a.ld, a.V, rank, cs);
            T* dz = dlogits ? dlogits + r.t * a.ld_grad : nullptr;
            // 16-byte stores need the gradient's row on the same alignment as the logits' row
            const bool wide = ((reinterpret_cast<uintptr_t>(s.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
            uint4* out = reinterpret_cast<uint4*>(dz + s.head) + s.v0;
            const int odd = tid < s.head ? tid : s.nvec * N + tid;   // this thread's single element, if tid < rest
            if (r.w == 0.f) {
                if (rank == 0 && tid == 0) {
                    if (a.logp) a.logp[r.t] = 0.f;
                    if (a.tok_loss) a.tok_loss[r.t] = 0.f;
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
            Token x{r.t, r.w, Elem<T>::to_f(s.z[r.target]), 0.f, 0.f, 0.f};
            if (a.advantage) x.adv = a.advantage[r.t];
            if (a.old_logp) x.old = a.old_logp[r.t];
            if (a.kl != 0.f) x.ref = a.ref_logp[r.t];
            const float lone = tid < s.rest ? Elem<T>::to_f(s.z[odd]) : 0.f;
            // ---- sum
            Running run{-INFINITY, 0};
            const Ring<kSlots> at0 = at;
            for (int i0 = 0; i0 < s.nv; i0 += kPiece, at.next()) {
                ok = ok && tc::mbar_wait(&full[at.slot], at.phase, a.err);
                const uint4* v = reinterpret_cast<const uint4*>(stage + at.slot * (kPiece * 16)) + tid;
                const int left = min(kPiece, s.nv - i0) - tid;
                if (left + lane > 31 + (kEach - 1) * kThreads) {          // all of the warp's vectors
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
            // a NaN goes into the sum, which keeps it: the maximum passes over it
            if (tid < s.rest) acc = join(acc, MaxSum{lone, lone == -INFINITY ? 0.f : lone != lone ? lone : 1.f}, k);
            acc = warp_join(acc, k);
            // ---- exchange. What this warp reads of the row itself has arrived: once all warps have
            // sent, any of them may write over it (dlogits may be logits)
            asm volatile("" ::"f"(x.zt), "f"(lone) : "memory");
            if (reuse == kFree) {
                // nothing of this row waits for its sum: the row before it is finished now, its
                // exchange having passed under this row's work
                if (turn) finish(before, receive(turn - 1));
                before = x;
                send(acc, turn++);
                continue;
            }
            send(acc, turn);
            acc = receive(turn++);
            const RowGrad<T> g(token_terms(a, x, rank == 0 && tid == 0, acc), acc, k);
            // ---- gradient
            const int hot = r.target - s.head - s.v0 * N;    // the target's place in this CTA's vectors
            const int hot_vec = hot >= 0 && hot < s.nv * N ? hot / N : -1;
            if (reuse == kKeep) at = at0;
            for (int i0 = 0; i0 < s.nv; i0 += kPiece, at.next()) {
                if (reuse == kAgain) ok = ok && tc::mbar_wait(&full[at.slot], at.phase, a.err);
                const uint4* v = reinterpret_cast<const uint4*>(stage + at.slot * (kPiece * 16)) + tid;
                const int left = min(kPiece, s.nv - i0) - tid;
                uint4* o = out + i0 + tid;
                if (wide && left + lane > 31 + (kEach - 1) * kThreads) {
#pragma unroll
                    for (int h = 0; h < kEach; ++h) o[h * kThreads] = grad_vec<T>(v[h * kThreads], g);
                } else if (wide) {
#pragma unroll
                    for (int h = 0; h < kEach; ++h)
                        if (h * kThreads < left) o[h * kThreads] = grad_vec<T>(v[h * kThreads], g);
                } else {
#pragma unroll 1
                    for (int j = 0; j < left; j += kThreads) {
                        put_elements<T>(dz + s.head + (int64_t)(s.v0 + i0 + tid + j) * N, grad_vec<T>(v[j], g));
                    }
                }
                // the target's element again, by the thread that has just written its vector
                const int hit = hot_vec - i0 - tid;
                if (hot_vec >= 0 && hit >= 0 && hit < left && hit % kThreads == 0)
                    dz[r.target] = grad_one<T>(x.zt, g, true);
                __syncwarp();
                if (lane == 0) tc::mbar_arrive(&empty[at.slot]);
            }
            if (tid < s.rest) dz[odd] = grad_one<T>(lone, g, odd == r.target);
        }
        // (also where a wait ran out: whoever has sent a row's pairs waits for all of that row's before it
        // leaves, so that none is under way by then)
        if (reuse == kFree && turn) {
            const MaxSum last = receive(turn - 1);
            if (ok) finish(before, last);
        }
    }
    // no CTA leaves while another of its cluster may still write to it
    __syncwarp();
    asm volatile("barrier.cluster.arrive.release;" ::: "memory");
    asm volatile("barrier.cluster.wait.acquire;" ::: "memory");
}

// Short rows: G threads (a warp, or the block) hold a row in registers, up to eight vectors each:
// exact maximum, sum and gradient from them, no shared memory for the row. Many small blocks hide
// the row's chain of latencies, which the long rows' ring cannot where a row is a few KB: with the
// loss, 16384 x 500 bf16 19 us against 130 by the ring, 8192 x 4096 29 against 74, 2048 x 16384 29
// against 36; at 20000 a row the ring's 37 us is what the block would need more registers for.
constexpr int short_block(int G) { return G == 32 ? 256 : G; }
template <typename T, int G>
__global__ void __launch_bounds__(short_block(G), 1024 / short_block(G)) policy_short_kernel(PolicyArgs a, const T* logits, T* dlogits) {
    constexpr int N = Vec16<T>::N;
    __shared__ MaxSum part[8];
    pdl_wait();
    const int tid = threadIdx.x % G, lane = threadIdx.x & 31;
    const int64_t t = (int64_t)blockIdx.x * (short_block(G) / G) + threadIdx.x / G;
    if (t >= a.T) return;                     // a whole warp (G = 32) or block
    const float w = a.weight ? a.weight[t] : 1.f;
    const int target = a.target[t];
    const Share<T> s(logits + t * a.ld, a.V, 0, 1);
    T* dz = dlogits ? dlogits + t * a.ld_grad : nullptr;
    const bool wide = ((reinterpret_cast<uintptr_t>(s.z) ^ reinterpret_cast<uintptr_t>(dz)) & 15) == 0;
    uint4* out = reinterpret_cast<uint4*>(dz + s.head);
    const int odd = tid < s.head ? tid : s.nvec * N + tid;
    if (w == 0.f || (uint32_t)target >= (uint32_t)a.V) {
        if (tid == 0) {
            if (w != 0.f && target >= a.V) raise_error(a.err, kErrBounds);
            if (a.logp) a.logp[t] = 0.f;
            if (a.tok_loss) a.tok_loss[t] = 0.f;
        }
        if (dz) {
            const T zero = Elem<T>::from_f(0.f);
            if (wide)
                for (int i = tid; i < s.nvec; i += G) out[i] = make_uint4(0u, 0u, 0u, 0u);
            else
                for (int i = tid; i < s.nvec * N; i += G) dz[s.head + i] = zero;
            if (tid < s.rest) dz[odd] = zero;
        }
        return;
    }
    const float k = a.inv_tau * kLog2e;
    Token x{(int)t, w, Elem<T>::to_f(s.z[target]), 0.f, 0.f, 0.f};
    if (a.advantage) x.adv = a.advantage[t];
    if (a.old_logp) x.old = a.old_logp[t];
    if (a.kl != 0.f) x.ref = a.ref_logp[t];
    const float lone = tid < s.rest ? Elem<T>::to_f(s.z[odd]) : -INFINITY;
    const uint32_t none = sizeof(T) == 2 ? 0xff80ff80u : 0xff800000u;       // -inf, which adds 0
    uint4 u[kHeld];
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        u[h] = make_uint4(none, none, none, none);
        if (tid + h * G < s.nvec) u[h] = s.vecs()[tid + h * G];
    }
    MaxSum acc{lone, 0.f};
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (h * G < s.nvec) acc.m = fmaxf(acc.m, vec_max<T>(u[h]));
    const float base = acc.m == -INFINITY ? 0.f : acc.m;
    const uint64_t minus = splat2(-base), kk = splat2(k);
    uint64_t sum = 0;
#pragma unroll
    for (int h = 0; h < kHeld; ++h)
        if (h * G < s.nvec) {
            uint64_t p[Pairs<T>::N];
            to_pairs<T>(u[h], p);
#pragma unroll
            for (int i = 0; i < Pairs<T>::N; ++i) {
                float x0, x1;
                upk2(mul2(add2(p[i], minus), kk), x0, x1);
                sum = add2(sum, pk2(ex2_approx(x0), ex2_approx(x1)));
            }
        }
    float s0, s1;
    upk2(sum, s0, s1);
    acc.s = s0 + s1;
    if (tid < s.rest) acc.s += ex2_approx((lone - base) * k);
    acc = warp_join(acc, k);
    // what this thread reads of the row has arrived before any thread writes it (dlogits may be logits)
    asm volatile("" ::"f"(x.zt), "f"(lone) : "memory");
    if constexpr (G > 32) {
        if (lane == 0) part[threadIdx.x >> 5] = acc;
        __syncthreads();
        acc = warp_join(lane < G / 32 ? part[lane] : MaxSum{-INFINITY, 0.f}, k);
    }
    __syncwarp();
    const RowGrad<T> g(token_terms(a, x, tid == 0, acc), acc, k);
    if (!dz) return;
#pragma unroll
    for (int h = 0; h < kHeld; ++h) {
        const int i = tid + h * G;
        if (i >= s.nvec) break;
        const uint4 o = grad_vec<T>(u[h], g);
        if (wide) out[i] = o;
        else put_elements<T>(dz + s.head + i * N, o);
    }
    // the target's element again, by the thread that has just written its vector
    const int hot = target - s.head, hot_vec = hot >= 0 && hot < s.nvec * N ? hot / N : -1;
    if (hot_vec >= 0 && hot_vec % G == tid) dz[target] = grad_one<T>(x.zt, g, true);
    if (tid < s.rest) dz[odd] = grad_one<T>(lone, g, odd == target);
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
    // rows that a warp, or a block, holds in registers
    if (vecs <= 256 * kHeld) {
        const T* z = static_cast<const T*>(logits);
        T* dz = static_cast<T*>(dlogits);
        const cudaError_t e =
            vecs <= 32 * kHeld    ? launch_pdl(policy_short_kernel<T, 32>, dim3(ceil_div(a.T, 8)), dim3(256), 0, s, a, z, dz)
            : vecs <= 64 * kHeld  ? launch_pdl(policy_short_kernel<T, 64>, dim3(a.T), dim3(64), 0, s, a, z, dz)
            : vecs <= 128 * kHeld ? launch_pdl(policy_short_kernel<T, 128>, dim3(a.T), dim3(128), 0, s, a, z, dz)
                                  : launch_pdl(policy_short_kernel<T, 256>, dim3(a.T), dim3(256), 0, s, a, z, dz);
        count_launch();
        return e;
    }
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
    if (!(c->temperature > 0.f) || !std::isfinite(c->temperature) || !std::isfinite(2.f / c->temperature))
        return MOE_ERR_INVALID_ARG;
    if (!(c->clip_low >= 0.f && c->clip_low <= 1.f) || !(c->clip_high >= 0.f) || !std::isfinite(c->clip_high) ||
        !std::isfinite(c->kl_weight))
        return MOE_ERR_INVALID_ARG;
    // a token past the last one that a loop steps to is numbered in 31 bits
    if (c->T > INT32_MAX - 4096 || c->V > (1 << 30) || c->ld > ((int64_t)1 << 40) || c->ld_grad > ((int64_t)1 << 40)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

cudaError_t run_policy(const moe_policy_config_t& c, PolicyArgs a, const void* logits, void* dlogits, cudaStream_t s) {
    a.T = c.T;
    a.V = c.V;
    a.ld = c.ld;
    a.ld_grad = c.ld_grad;
    a.tau = c.temperature;
    a.inv_tau = 1.f / c.temperature;
    a.clip_low = c.clip_low;
    a.clip_high = c.clip_high;
    a.kl = a.advantage ? c.kl_weight : 0.f;      // without an advantage there is no loss, and no ref_logp
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
