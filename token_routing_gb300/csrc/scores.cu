// Choice of experts from scores (softmax over all experts, or sigmoids), with a bias for balance,
// expert groups and renormalised weights, and its gradient in the logits.
#include <cfloat>
#include <cmath>

#include "internal.cuh"

namespace moe {

namespace {

constexpr int kWarps = 8;                 // warps of a block; each takes a token at a time
constexpr int kThreads = 32 * kWarps;
constexpr int kScoreBlocks = 4;           // blocks of the choice on an SM (64 registers)
constexpr int kCand = 32;                 // candidates that a warp ranks at once, one to a lane
constexpr float kTiny = 1e-20f;           // added to the sum of the chosen sigmoids

struct ScoreArgs {
    const float* logits;
    const float* bias;
    int32_t* idx;
    float* w;
    int32_t* part;        // [blocks, 32 V] choices per block, zeros beyond E; or null
    int T, E, k, groups, kept, top, renorm;
    uint32_t group_mul;   // e / group size = e * group_mul >> 16
    int lanes_log;        // log2 of the lanes that read one group
    float inv_hi, inv_lo; // 1 / temperature in two parts
    float to_log2;        // log2(e) / temperature
    float scale;
};

// z / temperature, by a reciprocal in two parts: within one rounding of the quotient. An infinite z
// stays what it is (times a low part of zero it would be NaN).
__device__ __forceinline__ float scaled(float z, float hi, float lo) {
    return fabsf(z) == INFINITY ? z : fmaf(z, hi, z * lo);
}

// The largest of a warp's values (no NaN among them).
__device__ __forceinline__ float warp_max(float v) {
    float r;
    asm volatile("redux.sync.max.f32 %0, %1, 0xffffffff;" : "=f"(r) : "f"(v));
    return r;
}

// What is compared: logits; scores plus bias; or, without a bias but with groups that are worth the sum of two scores,
// scores for the groups and logits for the experts in them (scores that round alike keep the order of their logits).
enum Compare : int { kLogits = 0, kScores = 1, kGroups = 2 };

// One token by a warp, up to its list of chosen experts. FULL: E = 32 V, and a lane has V experts side by side, so that a group is a lane or more and needs no
// exchange but shuffles; else expert lane + 32 i is the lane's i-th. Scores of all experts serve the comparison
// only, by hardware exponential and reciprocal: s (1 - s) times the argument's rounding (0.22 2^-23) and the exponential's
// (0.25 2^-22), the sum's and the reciprocal's are 2.3 2^-23 for a sigmoid; a softmax has the roundings of its sum, too
// (13 additions: 12.4 2^-23 in all). Weights are computed anew, in full precision, from the chosen logits.
//
// Bound by instructions: 32768 tokens of 256 experts in groups are 34 MB, 5 us at the copy rate, and take 22 us,
// 518 warp instructions a token in 75% of the issue slots (700 with every 32nd expert to a lane, groups exchanged
// through shared memory and each token's weights by themselves: 29 us). What keeps them few: the k-th largest of the
// 32 lanes' maxima bounds the k largest from below, so only experts at or above it (8 to 14 of 256 for k = 8) are
// ranked, each by counting those ahead of it; a reduction over the warp is one instruction; weights are left to
// route_weights, for four tokens at once.
template <int V, bool SOFTMAX, int COMPARE, bool FULL>
__device__ __forceinline__ void route_token(const ScoreArgs& a, const float (&z)[V], const float (&bias)[V], int lane,
                                            float* s_row, float* s_val, int* s_id, int* pick, float2* norm) {
    constexpr bool CHOICE = COMPARE != kLogits;
    const int E = a.E, k = a.k;
    const float inf = INFINITY;
    auto id_of = [&](int i) { return FULL ? lane * V + i : lane + 32 * i; };
    // a row that holds NaN or +inf has no softmax: its first experts, with NaN weights
    bool bad = false;
    if (SOFTMAX) {
#pragma unroll
        for (int i = 0; i < V; ++i) bad |= !(z[i] < inf);      // -inf beyond E
        bad = __any_sync(0xffffffffu, bad);
    }
    float c[V];
    float row_max = 0.f, row_inv = 1.f;       // softmax: row maximum and 1 / sum
    if (SOFTMAX && (CHOICE || !a.renorm)) {
        float mx = z[0];
#pragma unroll
        for (int i = 1; i < V; ++i) mx = fmaxf(mx, z[i]);
        mx = warp_max(bad ? 0.f : mx);
        row_max = mx == -inf ? 0.f : mx;
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            c[i] = ex2_approx((z[i] - row_max) * a.to_log2);
            sum += c[i];
        }
        sum = warp_sum(sum);
        if (CHOICE) {
            const float inv = sum > 0.f ? rcp_approx(sum) : 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) c[i] *= inv;
        }
        if (!a.renorm) {
            // the sum that weights are divided by, in full precision
            float exact = 0.f;
#pragma unroll
            for (int i = 0; i < V; ++i) exact += expf(scaled(z[i] - row_max, a.inv_hi, a.inv_lo));
            exact = warp_sum(exact);
            row_inv = exact > 0.f ? 1.0f / exact : 0.f;
        }
    } else if (CHOICE) {
#pragma unroll
        for (int i = 0; i < V; ++i) c[i] = rcp_approx(1.0f + ex2_approx(-z[i] * a.to_log2));
    }
    if (SOFTMAX && lane == 0) *norm = make_float2(row_max, bad ? NAN : row_inv);
#pragma unroll
    for (int i = 0; i < V; ++i) {
        // a logit of -inf, or a NaN, counts as -inf (fmaxf drops a NaN)
        c[i] = CHOICE ? (z[i] > -inf ? COMPARE == kScores ? c[i] + bias[i] : c[i] : -inf) : fmaxf(z[i], -inf);
        if (SOFTMAX && bad) c[i] = -inf;
    }

    uint32_t shut = 0;                        // bit h << log: group h is not kept
    bool out = false;                         // FULL: the lane's group is not
    float top = -inf;                         // the lane's largest that is not shut
    const int log = a.lanes_log;
    if (a.kept < a.groups) {
        // 2^log lanes to a group
        float m1 = -inf, m2 = -inf;
        auto see = [&](float v) {
            m2 = fmaxf(m2, fminf(m1, v));
            m1 = fmaxf(m1, v);
        };
        auto worth_of = [&](int size) { return a.top == 2 && size > 1 ? fmaxf(m1 + m2, -inf) : m1; };
        auto join = [&](int o) {
            const float n1 = __shfl_xor_sync(0xffffffffu, m1, o), n2 = __shfl_xor_sync(0xffffffffu, m2, o);
            m2 = fmaxf(fmaxf(m2, n2), fminf(m1, n1));
            m1 = fmaxf(m1, n1);
        };
        if (FULL) {
#pragma unroll
            for (int i = 0; i < V; ++i) see(c[i]);
            top = m1;
            // a group's rank is counted by its lanes together, each against every 2^log-th group
            auto rank_of = [&](int groups, int lg) {
                const int step = 1 << lg, g = lane >> lg, sub = lane & (step - 1);
#pragma unroll
                for (int o = step >> 1; o > 0; o >>= 1) join(o);
                const float worth = worth_of(V << lg);
                int rank = 0;
#pragma unroll
                for (int first = 0; first < groups; first += step) {
                    const int h = first + sub;
                    const float v = __shfl_sync(0xffffffffu, worth, h << lg);
                    if (h < groups && (v > worth || (v == worth && h < g))) ++rank;
                }
#pragma unroll
                for (int o = step >> 1; o > 0; o >>= 1) rank += __shfl_xor_sync(0xffffffffu, rank, o);
                return rank;
            };
            // (groups of 32 in a full row: with all numbers known)
            const bool mine = (a.groups == V ? rank_of(V, V == 8 ? 2 : V == 4 ? 3 : V == 2 ? 4 : 5)
                                             : rank_of(a.groups, log)) >= a.kept;
            shut = __ballot_sync(0xffffffffu, mine);
            out = mine;
            if (mine) top = -inf;
        } else {
            // a lane reads every 2^log-th of a group's experts; a row of 32 is 33 words apart, so that groups of 32
            // are read from different banks
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (lane + 32 * i < E) s_row[lane + 33 * i] = c[i];
            __syncwarp();
            const int size = E / a.groups, step = 1 << log, g = lane >> log, sub = lane & (step - 1);
            if (g < a.groups)
                for (int e = g * size + sub; e < (g + 1) * size; e += step) see(s_row[e + (e >> 5)]);
            for (int o = step >> 1; o > 0; o >>= 1) join(o);
            const float worth = worth_of(size);
            int rank = 0;
            for (int h = 0; h < a.groups; ++h) {
                const float v = __shfl_sync(0xffffffffu, worth, h << log);
                if (v > worth || (v == worth && h < g)) ++rank;
            }
            shut = __ballot_sync(0xffffffffu, g >= a.groups || rank >= a.kept);
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t h = ((uint32_t)(lane + 32 * i) * a.group_mul) >> 16;
                if (lane + 32 * i < E && ((shut >> (h << log)) & 1u)) c[i] = -inf;
                top = fmaxf(top, c[i]);
            }
        }
    } else {
#pragma unroll
        for (int i = 0; i < V; ++i) top = fmaxf(top, c[i]);
    }
    if (COMPARE == kGroups) {
        top = -inf;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            if (c[i] > -inf) c[i] = z[i];
            if (!out) top = fmaxf(top, c[i]);
        }
    }

    // a lower bound of the k largest (lanes that tie fall out together, which only lowers it)
    float least = -inf;
#pragma unroll
    for (int j = 0; j < MOE_MAX_K; ++j) {
        if (j >= k) break;
        least = warp_max(top);
        if (top == least) top = -inf;
    }
    // experts at or above it, in order of their ids
    int n = kCand + 1;
    if (least > -inf) {
        if (FULL) {
            const float bar = out ? NAN : least;       // (no comparison holds)
            int own = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) own += c[i] >= bar;
            // places of a lane's own: the lanes before it, by the bits of their counts (a scan: 25.2 us for 24.7)
            const uint32_t before = (1u << lane) - 1u;
            const uint32_t b0 = __ballot_sync(0xffffffffu, own & 1), b1 = __ballot_sync(0xffffffffu, own & 2),
                           b2 = __ballot_sync(0xffffffffu, own & 4), b3 = __ballot_sync(0xffffffffu, own & 8);
            int at = __popc(b0 & before) + 2 * __popc(b1 & before);
            n = __popc(b0) + 2 * __popc(b1);
            if (b2 | b3) {
                at += 4 * __popc(b2 & before) + 8 * __popc(b3 & before);
                n += 4 * __popc(b2) + 8 * __popc(b3);
            }
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (c[i] >= bar) {
                    s_val[at] = c[i];
                    s_id[at++] = lane * V + i;
                }
        } else {
            n = 0;
#pragma unroll
            for (int i = 0; i < V; ++i) {
                const uint32_t at = __ballot_sync(0xffffffffu, c[i] >= least);
                if (c[i] >= least) {
                    const int to = n + __popc(at & ((1u << lane) - 1u));
                    s_val[to] = c[i];
                    s_id[to] = lane + 32 * i;
                }
                n += __popc(at);
            }
        }
        if (lane < 4) s_val[n + lane] = -inf;       // ranks are counted in fours
    }
    __syncwarp();
    if (n <= kCand) {
        const float own = s_val[lane];              // (counts for nothing behind the last)
        int rank = 0;
        for (int j = 0; j < n; j += 4) {
            const float4 v = *reinterpret_cast<const float4*>(s_val + j);
            rank += (v.x > own) + (v.y > own) + (v.z > own) + (v.w > own);
        }
        if (__popc(__reduce_or_sync(0xffffffffu, lane < n ? 1u << rank : 0u)) != n)      // equal ones: the first is ahead
            for (int j = 0; j < n; ++j) rank += j < lane && s_val[j] == own;
        if (lane < n && rank < k) pick[rank] = s_id[lane];
    } else {
        // many equal values, or fewer than k above -inf: one expert after another
        uint32_t open = 0;       // bit i: the lane's i-th expert may be taken
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const uint32_t h = ((uint32_t)id_of(i) * a.group_mul) >> 16;
            if ((FULL || lane + 32 * i < E) && !((shut >> (h << log)) & 1u)) open |= 1u << i;
        }
        for (int j = 0; j < k; ++j) {
            float best = -inf;
            uint32_t id = 0xffffffffu;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if (((open >> i) & 1u) && (c[i] > best || id == 0xffffffffu)) {
                    best = c[i];
                    id = (uint32_t)id_of(i);
                }
            const float most = warp_max(best);
            const uint32_t first = __reduce_min_sync(0xffffffffu, best == most ? id : 0xffffffffu);
            if (lane == j) pick[j] = (int)first;
#pragma unroll
            for (int i = 0; i < V; ++i)
                if ((uint32_t)id_of(i) == first) open &= ~(1u << i);
        }
    }
    __syncwarp();
}

// Weights of up to four tokens t, t + step, ..., eight lanes to each.
template <bool SOFTMAX>
__device__ __forceinline__ void route_weights(const ScoreArgs& a, int t, int step, int tokens, int lane, const int* pick,
                                              const float2* norm, int* s_hist) {
    const int j = lane >> 3, slot = lane & 7;
    const bool has = j < tokens && slot < a.k;
    const size_t row = (size_t)t + (size_t)j * step;
    const int mine = has ? pick[lane] : 0;
    const float zc = has ? __ldg(a.logits + row * a.E + mine) : -INFINITY;
    const float2 whole = SOFTMAX && has ? norm[j] : make_float2(0.f, 1.f);      // row maximum, 1 / sum or NaN
    float s = 0.f;
    if (SOFTMAX && a.renorm) {
        float mx = fmaxf(zc, -INFINITY);
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx == -INFINITY) mx = 0.f;
        s = has ? expf(scaled(zc - mx, a.inv_hi, a.inv_lo)) : 0.f;
    } else if (has) {
        s = SOFTMAX ? expf(scaled(zc - whole.x, a.inv_hi, a.inv_lo)) : 1.0f / (1.0f + expf(-scaled(zc, a.inv_hi, a.inv_lo)));
    }
    if (a.renorm) {
        float sum = s;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
        s = SOFTMAX ? (sum > 0.f ? s / sum : 0.f) : s / (sum + kTiny);
    }
    if (SOFTMAX) s *= whole.y;
    if (has) {
        const size_t at = row * a.k + slot;
        a.idx[at] = mine;
        a.w[at] = s * a.scale;
        if (a.part) atomicAdd(s_hist + mine, 1);
    }
    __syncwarp();
}

__device__ __forceinline__ void cluster_barrier() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
// balance_loss = mean_e (counts[e] - T k / E)^2, by the whole block: counts differ from their mean by
// up to T k, whose squares want 64 bits; the sum is of integers (E counts - T k), exact.
__device__ __forceinline__ void block_balance(const int* s_counts, int T, int E, int k, float* out, double* s_red) {
    double sq = 0.0;
    for (int e = threadIdx.x; e < E; e += blockDim.x) {
        const double off = (double)s_counts[e] * E - (double)T * k;
        sq += off * off;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
    if ((threadIdx.x & 31) == 0) s_red[threadIdx.x >> 5] = sq;
    __syncthreads();
    if (threadIdx.x == 0) {
        double all = 0.0;
        for (int w = 0; w < (int)(blockDim.x >> 5); ++w) all += s_red[w];
        *out = (float)(all / ((double)E * E * E));
    }
}

template <int V, bool SOFTMAX, int COMPARE, bool FULL>
__global__ void __launch_bounds__(kThreads, kScoreBlocks) route_scores_kernel(const ScoreArgs a, int32_t* counts,
                                                                             float* balance) {
    __shared__ float s_row[FULL ? 1 : kWarps][FULL ? 1 : 33 * V];
    __shared__ __align__(16) float s_val[kWarps][32 * V + 4];    // (all may tie)
    __shared__ int s_id[kWarps][32 * V];
    __shared__ int s_pick[kWarps][4 * MOE_MAX_K];
    __shared__ float2 s_norm[kWarps][4];
    __shared__ int s_hist[MOE_MAX_EXPERTS];
    __shared__ double s_red[kWarps];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int nwarps = gridDim.x * kWarps;
    for (int e = threadIdx.x; e < a.E; e += kThreads) s_hist[e] = 0;
    __syncthreads();
    pdl_wait();
    float bias[V];
#pragma unroll
    for (int i = 0; i < V; ++i) {
        const int e = FULL ? lane * V + i : lane + 32 * i;
        bias[i] = COMPARE == kScores && e < a.E ? fmaxf(__ldg(a.bias + e), -INFINITY) : 0.f;     // (a NaN: never chosen)
    }
    int t = blockIdx.x * kWarps + warp;
    float z[V], next[V];
    auto fetch = [&](int u, float (&into)[V]) {
        const float* p = a.logits + (size_t)min(u, a.T - 1) * a.E;     // (behind the last token: not used)
        if constexpr (FULL && V >= 4) {
#pragma unroll
            for (int i = 0; i < V; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(p + lane * V + i));
                into[i] = v.x; into[i + 1] = v.y; into[i + 2] = v.z; into[i + 3] = v.w;
            }
        } else if constexpr (FULL && V == 2) {
            const float2 v = __ldg(reinterpret_cast<const float2*>(p + lane * V));
            into[0] = v.x; into[1] = v.y;
        } else {
#pragma unroll
            for (int i = 0; i < V; ++i) into[i] = FULL || lane + 32 * i < a.E ? __ldg(p + lane + 32 * i) : -INFINITY;
        }
    };
    if (t < a.T) fetch(t, z);
    for (int done = 0; t < a.T; t += nwarps) {
        fetch(t + nwarps, next);
        route_token<V, SOFTMAX, COMPARE, FULL>(a, z, bias, lane, s_row[FULL ? 0 : warp], s_val[warp], s_id[warp],
                                              s_pick[warp] + done * MOE_MAX_K, s_norm[warp] + done);
        ++done;
        if (done == 4 || t + nwarps >= a.T) {
            route_weights<SOFTMAX>(a, t - (done - 1) * nwarps, nwarps, done, lane, s_pick[warp], s_norm[warp], s_hist);
            done = 0;
        }
#pragma unroll
        for (int i = 0; i < V; ++i) z[i] = next[i];
    }
    __syncthreads();
    if (a.part)
        for (int e = threadIdx.x; e < 32 * V; e += kThreads) a.part[(size_t)blockIdx.x * (32 * V) + e] = e < a.E ? s_hist[e] : 0;
    if (gridDim.x == 1) {      // few tokens: one block has all of the counts
        if (counts)
            for (int e = threadIdx.x; e < a.E; e += kThreads) counts[e] = s_hist[e];
        if (balance) block_balance(s_hist, a.T, a.E, a.k, balance, s_red);
    }
}

// counts = sum of the blocks' choices, and the balance loss: a cluster of CTAs, 32 experts each. A warp reads four
// rows of the partial counts at once, and all of a thread's rows are in flight together: one latency, not one for
// each of the 600 rows (7 us in that form, of which 3 were the rows).
constexpr int kFinish = 1024;
__global__ void __launch_bounds__(kFinish) route_counts_kernel(const int32_t* __restrict__ part, int parts, int T,
                                                              int E, int k, int32_t* counts, float* balance) {
    __shared__ int s_sum[kFinish / 8][33];
    __shared__ double s_sq[MOE_MAX_EXPERTS / 32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int4* rows = reinterpret_cast<const int4*>(part + blockIdx.x * 32) + (lane & 7);
    const int stride = gridDim.x * 8;      // of a row, in int4
    int4 sum = make_int4(0, 0, 0, 0);
#pragma unroll 8
    for (int b = threadIdx.x >> 3; b < parts; b += kFinish / 8) {
        const int4 v = __ldg(rows + (size_t)b * stride);
        sum.x += v.x; sum.y += v.y; sum.z += v.z; sum.w += v.w;
    }
    int* to = &s_sum[threadIdx.x >> 3][(lane & 7) * 4];
    to[0] = sum.x; to[1] = sum.y; to[2] = sum.z; to[3] = sum.w;
    __syncthreads();
    int all = 0;                           // warp w: rows w, w + 32, w + 64, w + 96 of the sums
#pragma unroll
    for (int r = 0; r < 4; ++r) all += s_sum[warp + 32 * r][lane];
    __syncthreads();
    s_sum[warp][lane] = all;
    cluster_barrier();                     // (all CTAs run, too)
    if (warp == 0) {
        const int e = blockIdx.x * 32 + lane;
        all = 0;
#pragma unroll
        for (int w = 0; w < 32; ++w) all += s_sum[w][lane];
        if (counts && e < E) counts[e] = all;
        double sq = e < E ? (double)all * E - (double)T * k : 0.0;
        sq *= sq;
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) sq += __shfl_xor_sync(0xffffffffu, sq, o);
        if (lane == 0) {
            uint32_t at;
            asm volatile("mapa.shared::cluster.u32 %0, %1, 0;"
                         : "=r"(at) : "r"(static_cast<uint32_t>(__cvta_generic_to_shared(s_sq + blockIdx.x))));
            asm volatile("st.shared::cluster.f64 [%0], %1;" ::"r"(at), "d"(sq) : "memory");
        }
    }
    cluster_barrier();
    if (balance && blockIdx.x == 0 && threadIdx.x == 0) {
        double total = 0.0;
        for (int b = 0; b < (int)gridDim.x; ++b) total += s_sq[b];
        *balance = (float)(total / ((double)E * E * E));
    }
}

// ---------------------------------------------------------------- gradient
struct ScoreGradArgs {
    const float* logits;
    const int32_t* idx;
    const float* dw;
    float* dlogits;
    float* dz;            // [T, k] gradients of the chosen logits (nullable)
    int T, E, k, renorm;
    float inv_hi, inv_lo, scale;
    int* err;
};

// Slot j = lane % 8 of a token: its expert, whether it counts, the weight's gradient.
struct Slot {
    int e;
    bool on;
    float dw;
    __device__ __forceinline__ void load(const ScoreGradArgs& a, int t, int j) {
        on = t < a.T && j < a.k;
        const size_t at = (size_t)t * a.k + j;
        e = on ? __ldg(a.idx + at) : -1;
        dw = on ? __ldg(a.dw + at) : 0.f;
    }
    // Experts out of range, or that an earlier slot of the token holds, are left out.
    __device__ __forceinline__ void check(const ScoreGradArgs& a, int j) {
        bool bad = on && (uint32_t)e >= (uint32_t)a.E;
        for (int i = 0; i < a.k - 1; ++i) {
            const int o = __shfl_sync(0xffffffffu, e, i, 8);
            bad |= on && i < j && o == e;
        }
        if (bad) {
            raise_error(a.err, kErrBounds);
            on = false;
        }
    }
};

// The gradient of the slot's logit z, by lanes of eight to a token. The derivative of a share in its own sum is
// taken by differences of dw, since one share can be nearly all of the sum. A softmax subtracts the largest logit before
// it divides by the temperature, as the forward pass does: quotients far from zero have lost what tells them apart.
template <bool SOFTMAX>
__device__ __forceinline__ float slot_grad(const ScoreGradArgs& a, const Slot& s, float z) {
    float score, slope;             // slope: d score / d x, with x = z / temperature
    if (SOFTMAX) {
        float mx = s.on ? z : -INFINITY;
#pragma unroll
        for (int o = 4; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        if (mx == -INFINITY) mx = 0.f;
        score = s.on ? expf(scaled(z - mx, a.inv_hi, a.inv_lo)) : 0.f;
        slope = score;              // the part through the sum cancels in the shares
    } else {
        const float x = scaled(z, a.inv_hi, a.inv_lo);
        score = s.on ? 1.0f / (1.0f + expf(-x)) : 0.f;
        // s (1 - s), with 1 - s = 1 / (1 + e^x) taken apart so that it does not cancel
        slope = score * (1.0f / (1.0f + expf(x)));
    }
    if (!a.renorm) return s.on ? s.dw * a.scale * slope : 0.f;
    float sum = score;
#pragma unroll
    for (int o = 4; o > 0; o >>= 1) sum += __shfl_xor_sync(0xffffffffu, sum, o);
    const float tiny = SOFTMAX ? 0.f : kTiny;
    const float inv = sum + tiny == 0.f ? 0.f : 1.0f / (sum + tiny);
    const float share = score * inv;
    float g = s.dw * (tiny * inv);
    for (int i = 0; i < a.k; ++i) {
        const float si = __shfl_sync(0xffffffffu, share, i, 8), di = __shfl_sync(0xffffffffu, s.dw, i, 8);
        if (si != 0.f) g = fmaf(si, s.dw - di, g);
    }
    return s.on ? g * (a.scale * inv) * slope : 0.f;
}

// Gradient at the chosen experts, zeros elsewhere, by a warp for four tokens at a time: zeros go out while idx and
// then its logits are on their way, and the chosen entries after them (the lines are still in L2).
constexpr int kGradWarps = 4, kGradBlocks = 12;
template <bool SOFTMAX>
__global__ void __launch_bounds__(32 * kGradWarps, kGradBlocks) scores_grad_kernel(const ScoreGradArgs a) {
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, j = lane & 7;
    pdl_wait();
    const int quads = (a.T + 3) / 4, step = gridDim.x * kGradWarps;
    for (int q = blockIdx.x * kGradWarps + warp; q < quads; q += step) {
        const int t = 4 * q + (lane >> 3);
        Slot s;
        s.load(a, t, j);
        float* out = a.dlogits + (size_t)4 * q * a.E;
        if (4 * q + 4 <= a.T) {
            for (int i = lane; i < a.E; i += 32) reinterpret_cast<float4*>(out)[i] = make_float4(0.f, 0.f, 0.f, 0.f);
        } else {
            for (int i = lane; i < (a.T - 4 * q) * a.E; i += 32) out[i] = 0.f;
        }
        s.check(a, j);
        const float z = s.on ? __ldg(a.logits + (size_t)t * a.E + s.e) : -INFINITY;
        const float dz = scaled(slot_grad<SOFTMAX>(a, s, z), a.inv_hi, a.inv_lo);
        __syncwarp();                    // the zeros come first
        if (s.on) a.dlogits[(size_t)t * a.E + s.e] = dz;
        if (a.dz && t < a.T && j < a.k) a.dz[(size_t)t * a.k + j] = s.on ? dz : 0.f;
    }
}

// Softmax over all experts, weights not renormalised: dz_e = p_e (g_e - sum_chosen p g) / temperature.
template <int V>
__global__ void __launch_bounds__(kThreads) scores_grad_full_kernel(const ScoreGradArgs a) {
    __shared__ float s_g[kWarps][32 * V];
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    float* sg = s_g[warp];
#pragma unroll
    for (int i = 0; i < V; ++i) sg[lane + 32 * i] = 0.f;
    __syncwarp();
    pdl_wait();
    for (int t = blockIdx.x * kWarps + warp; t < a.T; t += gridDim.x * kWarps) {
        float x[V];
        float mx = -INFINITY;
        bool bad = false;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int e = lane + 32 * i;
            x[i] = e < a.E ? __ldg(a.logits + (size_t)t * a.E + e) : -INFINITY;
            bad |= !(x[i] < INFINITY);
            mx = fmaxf(mx, x[i]);
        }
        // all four groups of eight lanes work on the same token; the first one's slots are set
        Slot slot;
        slot.load(a, t, lane & 7);
        slot.check(a, lane & 7);
        const bool on = slot.on && lane < 8;
        const int e = slot.e;
        if (on) sg[e] = slot.dw * a.scale;
        if (a.dz && lane < a.k) a.dz[(size_t)t * a.k + lane] = 0.f;   // all of the gradient is dense
        __syncwarp();
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) mx = fmaxf(mx, __shfl_xor_sync(0xffffffffu, mx, o));
        bad = __any_sync(0xffffffffu, bad);
        if (mx == -INFINITY) mx = 0.f;
        float sum = 0.f, dot = 0.f;
        float gi[V];
#pragma unroll
        for (int i = 0; i < V; ++i) {
            x[i] = expf(scaled(x[i] - mx, a.inv_hi, a.inv_lo));
            sum += x[i];
            gi[i] = sg[lane + 32 * i];
            dot = fmaf(x[i], gi[i], dot);
        }
        sum = warp_sum(sum);
        dot = warp_sum(dot);
        const float inv = bad ? NAN : sum > 0.f ? 1.0f / sum : 0.f;
        dot *= inv;
#pragma unroll
        for (int i = 0; i < V; ++i) {
            const int c = lane + 32 * i;
            if (c < a.E) a.dlogits[(size_t)t * a.E + c] = scaled(x[i] * inv * (gi[i] - dot), a.inv_hi, a.inv_lo);
        }
        __syncwarp();
        if (on) sg[e] = 0.f;
        __syncwarp();
    }
}

// ---------------------------------------------------------------- host
// log2(e) / temperature: what the comparison multiplies logits by. Where fp32 does not hold it the largest logit's
// score would be 0 inf, and no expert the largest.
double to_log2(float temperature) { return 1.4426950408889634 / (double)temperature; }

moe_status_t check_scores(const moe_score_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->T < 0 || c->E < 1 || c->E > MOE_MAX_EXPERTS || c->groups < 1 || c->groups > 32 || c->E % c->groups ||
        c->groups_kept < 1 || c->groups_kept > c->groups || c->k < 1 || c->k > MOE_MAX_K ||
        c->k > c->E / c->groups * c->groups_kept)
        return MOE_ERR_INVALID_ARG;
    if ((c->score != MOE_SCORE_SOFTMAX && c->score != MOE_SCORE_SIGMOID) || (c->group_top != 1 && c->group_top != 2) ||
        (c->renormalise != 0 && c->renormalise != 1))
        return MOE_ERR_INVALID_ARG;
    if (!(c->temperature > 0.0f) || !std::isfinite(c->temperature) || !(to_log2(c->temperature) <= FLT_MAX) ||
        !std::isfinite(c->scale))
        return MOE_ERR_INVALID_ARG;
    if (c->T > (1 << 27)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

void reciprocal(float temperature, float* hi, float* lo) {
    const double inv = 1.0 / (double)temperature;
    *hi = (float)inv;
    *lo = (float)(inv - (double)*hi);
}

// Blocks of the choice: all that the SMs hold at once, or one for few tokens.
int score_blocks(const moe_score_config_t& c) {
    const int need = ceil_div(c.T, kWarps);
    return need <= 4 ? 1 : std::min(need, num_sms() * kScoreBlocks);
}
// Registers to a lane that hold a token's experts (1, 2, 4 or 8).
int score_width(const moe_score_config_t& c) { return c.E > 128 ? 8 : c.E > 64 ? 4 : c.E > 32 ? 2 : 1; }

template <int V, bool FULL>
cudaError_t launch_scores(const ScoreArgs& a, bool softmax, Compare by, int blocks, int32_t* counts, float* balance,
                          cudaStream_t s) {
    auto kern = softmax ? (by == kScores   ? route_scores_kernel<V, true, kScores, FULL>
                           : by == kGroups ? route_scores_kernel<V, true, kGroups, FULL>
                                           : route_scores_kernel<V, true, kLogits, FULL>)
                        : (by == kScores   ? route_scores_kernel<V, false, kScores, FULL>
                           : by == kGroups ? route_scores_kernel<V, false, kGroups, FULL>
                                           : route_scores_kernel<V, false, kLogits, FULL>);
    const cudaError_t e = launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, s, a, counts, balance);
    count_launch();
    return e;
}

cudaError_t launch_counts(const moe_score_config_t& c, const int32_t* part, int parts, int32_t* counts, float* balance,
                          cudaStream_t s) {
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)score_width(c));
    cfg.blockDim = dim3(kFinish);
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = cfg.gridDim.x;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    const cudaError_t e = launch_ex(cfg, route_counts_kernel, part, parts, c.T, c.E, c.k, counts, balance);
    count_launch();
    return e;
}

}  // namespace

cudaError_t launch_scores_grad(const moe_score_config_t& c, const float* logits, const int32_t* idx, const float* dw,
                               float* dlogits, float* dz, cudaStream_t s) {
    if (c.T == 0) return cudaSuccess;
    ScoreGradArgs a{logits, idx, dw, dlogits, dz, c.T, c.E, c.k, c.renormalise, 0.f, 0.f, c.scale, device_error_word()};
    reciprocal(c.temperature, &a.inv_hi, &a.inv_lo);
    cudaError_t e;
    if (c.score == MOE_SCORE_SOFTMAX && !c.renormalise) {
        const int blocks = std::min(ceil_div(c.T, kWarps), num_sms() * 8);
        const int v = ceil_div(c.E, 32);
        auto kern = v <= 1 ? scores_grad_full_kernel<1> : v <= 2 ? scores_grad_full_kernel<2>
                    : v <= 4 ? scores_grad_full_kernel<4> : scores_grad_full_kernel<8>;
        e = launch_pdl(kern, dim3(blocks), dim3(kThreads), 0, s, a);
    } else {
        const int blocks = std::min(ceil_div(c.T, 4 * kGradWarps), num_sms() * kGradBlocks);
        auto kern = c.score == MOE_SCORE_SOFTMAX ? scores_grad_kernel<true> : scores_grad_kernel<false>;
        e = launch_pdl(kern, dim3(blocks), dim3(32 * kGradWarps), 0, s, a);
    }
    count_launch();
    return e;
}

moe_status_t scores_status(const moe_score_config_t* c) { return check_scores(c); }

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_route_scores_workspace_bytes(const moe_score_config_t* cfg) {
    if (check_scores(cfg) != MOE_OK) return 0;
    return align_up((size_t)score_blocks(*cfg) * score_width(*cfg) * 32 * sizeof(int32_t), 256);
}

extern "C" MOE_API moe_status_t moe_route_scores(const moe_score_config_t* cfg, const float* logits, const float* bias,
                                                 int32_t* idx, float* w, int32_t* counts, float* balance_loss,
                                                 void* ws, moe_stream_t stream) {
    const moe_status_t st = check_scores(cfg);
    if (st != MOE_OK) return st;
    const moe_score_config_t& c = *cfg;
    if (c.T > 0 && (!logits || !idx || !w)) return MOE_ERR_INVALID_ARG;
    if ((counts || balance_loss) && !ws) return MOE_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(ws, 16) || misaligned(bias, 4) || misaligned(idx, 4) || misaligned(w, 4) ||
        misaligned(counts, 4) || misaligned(balance_loss, 4))
        return MOE_ERR_INVALID_ARG;
    const bool tally = counts || balance_loss;
    if (c.T == 0 && !tally) return MOE_OK;
    cudaStream_t s = (cudaStream_t)stream;
    const int blocks = score_blocks(c);
    ScoreArgs a{};
    a.logits = logits; a.bias = bias; a.idx = idx; a.w = w;
    a.part = tally ? static_cast<int32_t*>(ws) : nullptr;
    a.T = c.T; a.E = c.E; a.k = c.k; a.groups = c.groups; a.kept = c.groups_kept; a.top = c.group_top;
    a.renorm = c.renormalise; a.scale = c.scale;
    const int size = c.E / c.groups;
    a.group_mul = (uint32_t)((65536 + size - 1) / size);
    while ((c.groups << (a.lanes_log + 1)) <= 32) ++a.lanes_log;
    reciprocal(c.temperature, &a.inv_hi, &a.inv_lo);
    const bool softmax = c.score == MOE_SCORE_SOFTMAX;
    const Compare by = bias ? kScores : c.groups_kept < c.groups && c.group_top == 2 ? kGroups : kLogits;
    a.to_log2 = (float)to_log2(c.temperature);
    auto go = c.E == 256 ? launch_scores<8, true> : c.E == 128 ? launch_scores<4, true>
              : c.E == 64 ? launch_scores<2, true> : c.E == 32 ? launch_scores<1, true>
              : c.E > 128 ? launch_scores<8, false> : c.E > 64 ? launch_scores<4, false>
              : c.E > 32 ? launch_scores<2, false> : launch_scores<1, false>;
    cudaError_t e = go(a, softmax, by, blocks, counts, balance_loss, s);
    if (e == cudaSuccess && tally && blocks > 1) e = launch_counts(c, a.part, blocks, counts, balance_loss, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API moe_status_t moe_route_scores_backward(const moe_score_config_t* cfg, const float* logits,
                                                          const int32_t* idx, const float* dw, float* dlogits,
                                                          moe_stream_t stream) {
    const moe_status_t st = check_scores(cfg);
    if (st != MOE_OK) return st;
    if (cfg->T == 0) return MOE_OK;
    if (!logits || !idx || !dw || !dlogits || logits == dlogits) return MOE_ERR_INVALID_ARG;
    if (misaligned(logits, 16) || misaligned(dlogits, 16) || misaligned(idx, 4) || misaligned(dw, 4))
        return MOE_ERR_INVALID_ARG;
    return launch_scores_grad(*cfg, logits, idx, dw, dlogits, nullptr, (cudaStream_t)stream) == cudaSuccess ? MOE_OK
                                                                                                  : MOE_ERR_CUDA;
}
