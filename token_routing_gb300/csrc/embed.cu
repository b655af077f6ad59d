// Token embedding: the lookup that makes the layer's x, and its gradient by sorted tokens.
#include <cmath>

#include "internal.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- vectors of VE elements
// Rows of an odd length start at every alignment: a row is moved in the widest vectors that
// divide its length (16 bytes when d * es % 16 == 0, down to single elements).
template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = uint16_t; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };

template <typename T, int VE>
struct Vec {
    static constexpr int kBytes = (int)sizeof(T) * VE;
    static __device__ __forceinline__ void load(const T* p, float (&f)[VE]) {
        if constexpr (kBytes > 16) {
            Vec<T, VE / 2>::load(p, reinterpret_cast<float(&)[VE / 2]>(f[0]));
            Vec<T, VE / 2>::load(p + VE / 2, reinterpret_cast<float(&)[VE / 2]>(f[VE / 2]));
        } else {
            const typename Raw<kBytes>::T u = *reinterpret_cast<const typename Raw<kBytes>::T*>(p);
            const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = Elem<T>::to_f(e[i]);
        }
    }
    static __device__ __forceinline__ void store(T* p, const float (&f)[VE]) {
        if constexpr (kBytes > 16) {
            Vec<T, VE / 2>::store(p, reinterpret_cast<const float(&)[VE / 2]>(f[0]));
            Vec<T, VE / 2>::store(p + VE / 2, reinterpret_cast<const float(&)[VE / 2]>(f[VE / 2]));
        } else {
            typename Raw<kBytes>::T u;
            T* e = reinterpret_cast<T*>(&u);
#pragma unroll
            for (int i = 0; i < VE; ++i) e[i] = Elem<T>::from_f(f[i]);
            *reinterpret_cast<typename Raw<kBytes>::T*>(p) = u;
        }
    }
};

// Widest vector (elements) that divides rows of d elements of es bytes.
int row_vec(int d, int es) {
    int v = 16 / es;
    while (v > 1 && d % v) v /= 2;
    return v;
}

// ---------------------------------------------------------------- lookup
// y[t] = scale * W[ids[t]]: U vectors a thread, all loads of a thread in flight together.
template <typename T, int VE, int U>
__global__ void __launch_bounds__(256) embed_kernel(const int32_t* __restrict__ ids, const T* __restrict__ W,
                                                    T* __restrict__ y, uint32_t total, uint32_t nvec, int V,
                                                    float scale, int* err) {
    pdl_wait();
    const uint32_t base = blockIdx.x * (256u * U) + threadIdx.x;
    float f[U][VE];
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = base + u * 256u;
        if (i >= total) break;
        const uint32_t t = i / nvec, c = i - t * nvec;
        const int id = __ldg(ids + t);
        if ((uint32_t)id < (uint32_t)V) {
            Vec<T, VE>::load(W + ((int64_t)id * nvec + c) * VE, f[u]);
        } else {
            if (c == 0) raise_error(err, kErrBounds);
#pragma unroll
            for (int k = 0; k < VE; ++k) f[u][k] = 0.f;
        }
    }
#pragma unroll
    for (int u = 0; u < U; ++u) {
        const uint32_t i = base + u * 256u;
        if (i >= total) break;
#pragma unroll
        for (int k = 0; k < VE; ++k) f[u][k] *= scale;
        Vec<T, VE>::store(y + (int64_t)i * VE, f[u]);
    }
}

template <typename T, int VE>
cudaError_t launch_embed_v(const moe_embed_config_t& c, const int32_t* ids, const void* W, void* y, cudaStream_t s) {
    const int nvec = c.d / VE;
    // vectors of one launch are numbered in 31 bits; more rows go to further launches
    const int rows = (int)std::min<int64_t>(c.T, std::max<int64_t>(1, ((int64_t)1 << 30) / nvec));
    for (int64_t t0 = 0; t0 < c.T; t0 += rows) {
        const uint32_t total = (uint32_t)(std::min<int64_t>(rows, c.T - t0) * nvec);
        const T* w = static_cast<const T*>(W);
        T* out = static_cast<T*>(y) + t0 * c.d;
        cudaError_t e;
        if (total >= 2048u * 4u * (uint32_t)num_sms())
            e = launch_pdl(embed_kernel<T, VE, 4>, dim3(ceil_div(total, 1024)), dim3(256), 0, s, ids + t0, w, out, total,
                           (uint32_t)nvec, (int)c.V, c.scale, device_error_word());
        else
            e = launch_pdl(embed_kernel<T, VE, 1>, dim3(ceil_div(total, 256)), dim3(256), 0, s, ids + t0, w, out, total,
                           (uint32_t)nvec, (int)c.V, c.scale, device_error_word());
        count_launch();
        if (e != cudaSuccess) return e;
    }
    return cudaSuccess;
}

template <typename T>
cudaError_t launch_embed(const moe_embed_config_t& c, const int32_t* ids, const void* W, void* y, cudaStream_t s) {
    switch (row_vec(c.d, (int)sizeof(T))) {
        case 8:
            if constexpr (sizeof(T) == 2) return launch_embed_v<T, 8>(c, ids, W, y, s);
        case 4: return launch_embed_v<T, 4>(c, ids, W, y, s);
        case 2: return launch_embed_v<T, 2>(c, ids, W, y, s);
        default: return launch_embed_v<T, 1>(c, ids, W, y, s);
    }
}

// ---------------------------------------------------------------- gradient: sort by token
// Stable radix sort of (id, token) pairs, least digit first, by ordinary launches: per digit a
// histogram of every chunk of kChunk pairs, then each chunk's ranks and the scatter. Left-out
// tokens (padding, ids out of range) take the key V and end up behind all others.
constexpr int kChunk = 1024;         // pairs a block of 256 threads ranks
constexpr int kWarps = 8;
constexpr int kPerLane = kChunk / 256;
constexpr int kMaxBits = 9;          // bits of a digit
constexpr int kMaxBins = 1 << kMaxBits;

struct SortArgs {
    const int32_t* ids;      // first pass: keys are made from the ids
    const uint2* in;         // later passes: (key, token)
    uint2* out;
    int32_t* hist;           // [chunks, bins]
    int T, V, pad;
    int shift, bits, chunks;
    int* err;
};

__device__ __forceinline__ uint2 sort_pair(const SortArgs& a, int i, bool report) {
    if (a.in) return a.in[i];
    const int id = __ldg(a.ids + i);
    const bool in_range = (uint32_t)id < (uint32_t)a.V;
    if (!in_range && report) raise_error(a.err, kErrBounds);
    return make_uint2(in_range && id != a.pad ? (uint32_t)id : (uint32_t)a.V, (uint32_t)i);
}

__global__ void __launch_bounds__(256) embed_hist_kernel(SortArgs a) {
    __shared__ int h[kMaxBins];
    const int bins = 1 << a.bits;
    for (int b = threadIdx.x; b < bins; b += 256) h[b] = 0;
    pdl_wait();
    __syncthreads();
    const int i0 = blockIdx.x * kChunk;
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const int i = i0 + k * 256 + (int)threadIdx.x;
        if (i < a.T) atomicAdd(&h[(sort_pair(a, i, true).x >> a.shift) & (bins - 1)], 1);
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += 256) a.hist[(int64_t)blockIdx.x * bins + b] = h[b];
}

// Exclusive prefix over `bins` values held two a thread (256 threads).
__device__ __forceinline__ void block_scan2(int& v0, int& v1, int* tmp) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int pair = v0 + v1;
    int x = pair;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int n = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += n;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    int before = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w) before += w < warp ? tmp[w] : 0;
    const int excl = before + x - pair;
    v1 = excl + v0;
    v0 = excl;
}

__global__ void __launch_bounds__(256) embed_scatter_kernel(SortArgs a) {
    __shared__ int cnt[kWarps][kMaxBins];
    __shared__ int base[kMaxBins];
    __shared__ int tmp[kWarps];
    const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = threadIdx.x; b < kWarps * kMaxBins; b += 256) (&cnt[0][0])[b] = 0;
    pdl_wait();
    __syncthreads();
    // ranks within the warp's 128 consecutive pairs: the lanes of one digit, in lane order
    uint2 pr[kPerLane];
    int rank[kPerLane];
    const int i0 = blockIdx.x * kChunk + warp * (32 * kPerLane);
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const int i = i0 + k * 32 + lane;
        pr[k] = i < a.T ? sort_pair(a, i, false) : make_uint2(0u, 0u);
    }
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const bool live = i0 + k * 32 + lane < a.T;
        const int dg = live ? (int)((pr[k].x >> a.shift) & (bins - 1)) : kMaxBins;
        const uint32_t same = __match_any_sync(0xffffffffu, dg);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int had = live ? cnt[warp][dg] : 0;
        __syncwarp();
        if (live && before == 0) cnt[warp][dg] = had + __popc(same);
        __syncwarp();
        rank[k] = had + before;
    }
    // every block reads the whole histogram: totals of all digits, and of the chunks before it
    int tot[2] = {0, 0}, mine[2] = {0, 0};
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int b = 2 * (int)threadIdx.x + q;
        if (b < bins)
            for (int c = 0; c < a.chunks; ++c) {
                const int v = __ldg(a.hist + (int64_t)c * bins + b);
                tot[q] += v;
                if (c < (int)blockIdx.x) mine[q] += v;
            }
    }
    block_scan2(tot[0], tot[1], tmp);
#pragma unroll
    for (int q = 0; q < 2; ++q) {
        const int b = 2 * (int)threadIdx.x + q;
        if (b < bins) base[b] = tot[q] + mine[q];
    }
    __syncthreads();
    for (int b = threadIdx.x; b < bins; b += 256) {
        int run = base[b];
#pragma unroll
        for (int w = 0; w < kWarps; ++w) {
            const int n = cnt[w][b];
            cnt[w][b] = run;
            run += n;
        }
    }
    __syncthreads();
#pragma unroll
    for (int k = 0; k < kPerLane; ++k)
        if (i0 + k * 32 + lane < a.T) a.out[cnt[warp][(pr[k].x >> a.shift) & (bins - 1)] + rank[k]] = pr[k];
}

// ---------------------------------------------------------------- gradient: sums over runs
// The sorted pairs are cut into groups of kGroup. A thread owns VE columns of one group and
// walks its rows in order; a run of one token that lies inside the group is finished there. A
// run that crosses groups leaves one fp32 partial row in each (slot 0: the run the group begins
// with, slot 1: the run it ends with and that begins in it), and embed_join_kernel adds them
// in group order. Every row of dW has one writer and a fixed order of sums.
constexpr int kGroup = 32;

struct SumArgs {
    const uint2* pairs;      // sorted (key, token)
    float* part;             // [groups, 2, d]
    int T, V, d, groups;
    int accumulate;
    float scale;
};

template <typename G, int VE>
__device__ __forceinline__ void put_row(const SumArgs& a, G* dW, uint32_t key, int col, float (&s)[VE]) {
    G* p = dW + (int64_t)key * a.d + col;
#pragma unroll
    for (int i = 0; i < VE; ++i) s[i] *= a.scale;
    if (a.accumulate) {
        float o[VE];
        Vec<G, VE>::load(p, o);
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] += o[i];
    }
    Vec<G, VE>::store(p, s);
}

template <typename T, typename G, int VE>
__global__ void __launch_bounds__(256) embed_sum_kernel(SumArgs a, const T* __restrict__ dy, G* __restrict__ dW) {
    __shared__ uint2 pr[kGroup + 2];   // the group's pairs, with a neighbour on either side
    pdl_wait();
    const int g = blockIdx.x, i0 = g * kGroup, n = min(kGroup, a.T - i0);
    for (int j = threadIdx.x; j < kGroup + 2; j += blockDim.x) {
        const int i = i0 + j - 1;
        pr[j] = i >= 0 && i < a.T ? a.pairs[i] : make_uint2(0xffffffffu, 0u);
    }
    __syncthreads();
    for (int col = (blockIdx.y * blockDim.x + threadIdx.x) * VE; col < a.d; col += gridDim.y * blockDim.x * VE) {
        float s[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] = 0.f;
        bool from_before = pr[0].x == pr[1].x;
        for (int j0 = 0; j0 < n; j0 += 8) {
            float r[8][VE];
#pragma unroll
            for (int j = 0; j < 8; ++j)
                if (j0 + j < n && pr[j0 + j + 1].x < (uint32_t)a.V)
                    Vec<T, VE>::load(dy + (int64_t)pr[j0 + j + 1].y * a.d + col, r[j]);
#pragma unroll
            for (int j = 0; j < 8; ++j) {
                if (j0 + j >= n) break;
                const uint32_t key = pr[j0 + j + 1].x;
                if (key >= (uint32_t)a.V) break;
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] += r[j][i];
                const bool ends = pr[j0 + j + 2].x != key;
                if (ends || j0 + j + 1 == n) {
                    if (ends && !from_before)
                        put_row(a, dW, key, col, s);
                    else
                        Vec<float, VE>::store(a.part + ((int64_t)g * 2 + (from_before ? 0 : 1)) * a.d + col, s);
                    from_before = false;
#pragma unroll
                    for (int i = 0; i < VE; ++i) s[i] = 0.f;
                }
            }
        }
    }
}

// First position whose key is >= key.
__device__ __forceinline__ int lower_bound(const uint2* p, int n, uint32_t key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = (lo + hi) >> 1;
        if (p[mid].x < key) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Runs that begin in group blockIdx.x and go on past it: their partial rows, in order. Eight
// warps take every eighth partial of the same columns; their sums are added in warp order.
template <typename G, int VE>
__global__ void __launch_bounds__(256) embed_join_kernel(SumArgs a, G* __restrict__ dW) {
    __shared__ float part[kWarps][32 * VE];
    pdl_wait();
    const int g = blockIdx.x, last = (g + 1) * kGroup - 1;
    if (last + 1 >= a.T) return;
    const uint32_t key = a.pairs[last].x;
    if (key >= (uint32_t)a.V || a.pairs[last + 1].x != key) return;
    if (g > 0 && a.pairs[g * kGroup - 1].x == key) return;     // it began before this group
    const int end = lower_bound(a.pairs, a.T, key + 1);
    const int parts = (end - 1) / kGroup - g + 1;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int c0 = blockIdx.y * 32 * VE; c0 < a.d; c0 += gridDim.y * 32 * VE) {
        const int col = c0 + lane * VE;
        float s[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] = 0.f;
        if (col < a.d)
#pragma unroll 4
            for (int k = warp; k < parts; k += kWarps) {
                float r[VE];
                Vec<float, VE>::load(a.part + ((int64_t)(g + k) * 2 + (k ? 0 : 1)) * a.d + col, r);
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] += r[i];
            }
#pragma unroll
        for (int i = 0; i < VE; ++i) part[warp][lane * VE + i] = s[i];
        __syncthreads();
        if (warp == 0 && col < a.d) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] += part[w][lane * VE + i];
            put_row(a, dW, key, col, s);
        }
        __syncthreads();
    }
}

// Zero rows of tokens that do not occur. A block owns 64 rows: one search for its first key,
// then the sorted keys of its rows mark the ones that were seen.
constexpr int kZeroRows = 64;
template <typename G, int VE>
__global__ void __launch_bounds__(256) embed_zero_kernel(const uint2* __restrict__ pairs, G* __restrict__ dW, int T, int V, int d) {
    __shared__ int seen[kZeroRows];
    __shared__ int lo, hi;
    for (int i = threadIdx.x; i < kZeroRows; i += 256) seen[i] = 0;
    pdl_wait();
    const int v0 = blockIdx.x * kZeroRows, v1 = min(v0 + kZeroRows, V);
    if (threadIdx.x == 0) lo = lower_bound(pairs, T, (uint32_t)v0);
    if (threadIdx.x == 32) hi = lower_bound(pairs, T, (uint32_t)v1);
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += 256) seen[pairs[i].x - v0] = 1;
    __syncthreads();
    float z[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) z[i] = 0.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int v = v0 + warp; v < v1; v += kWarps)
        if (!seen[v - v0])
            for (int c = lane * VE; c < d; c += 32 * VE) Vec<G, VE>::store(dW + (int64_t)v * d + c, z);
}

struct EmbedScratch {
    uint2* a;
    uint2* b;
    int32_t* hist;
    float* part;
};

int groups_of(const moe_embed_config_t& c) { return ceil_div(c.T, kGroup); }

size_t carve_embed(const moe_embed_config_t& c, void* base, EmbedScratch* s) {
    Workspace ws{static_cast<char*>(base), 0};
    s->a = ws.take<uint2>((size_t)c.T + 1);
    s->b = ws.take<uint2>((size_t)c.T + 1);
    s->hist = ws.take<int32_t>((size_t)ceil_div(c.T, kChunk) * kMaxBins + 1);
    s->part = ws.take<float>((size_t)groups_of(c) * 2 * c.d + 4);
    return align_up(ws.used, 256);
}

template <typename T, typename G, int VE>
cudaError_t launch_embed_bwd_v(const moe_embed_config_t& c, const uint2* pairs, float* part, const void* dy, void* dW,
                               cudaStream_t s) {
    cudaError_t e = cudaSuccess;
    const int nvec = c.d / VE;
    G* out = static_cast<G*>(dW);
    if (c.T > 0) {
        SumArgs a{pairs, part, c.T, c.V, c.d, groups_of(c), c.accumulate, c.scale};
        const int threads = std::min(256, ceil_div(nvec, 32) * 32);
        e = launch_pdl(embed_sum_kernel<T, G, VE>, dim3(a.groups, std::min(ceil_div(nvec, threads), 64)), dim3(threads),
                       0, s, a, static_cast<const T*>(dy), out);
        count_launch();
        if (e != cudaSuccess) return e;
        e = launch_pdl(embed_join_kernel<G, VE>, dim3(a.groups, std::min(ceil_div(nvec, 32), 64)), dim3(256), 0, s, a,
                       out);
        count_launch();
        if (e != cudaSuccess) return e;
    }
    if (!c.accumulate) {
        e = launch_pdl(embed_zero_kernel<G, VE>, dim3(ceil_div(c.V, kZeroRows)), dim3(256), 0, s, pairs, out, c.T, c.V,
                       c.d);
        count_launch();
    }
    return e;
}

template <typename T, typename G>
cudaError_t launch_embed_bwd(const moe_embed_config_t& c, const int32_t* ids, const void* dy, void* dW, void* ws,
                             cudaStream_t s) {
    EmbedScratch w;
    carve_embed(c, ws, &w);
    const uint2* sorted = w.a;
    if (c.T > 0) {
        int bits = 1;
        while (((int64_t)1 << bits) <= c.V) ++bits;          // keys 0 .. V
        const int passes = ceil_div(bits, kMaxBits), digit = ceil_div(bits, passes);
        SortArgs a{ids, nullptr, w.a, w.hist, c.T, c.V, c.padding_id, 0, digit, ceil_div(c.T, kChunk),
                   device_error_word()};
        for (int p = 0; p < passes; ++p) {
            a.shift = p * digit;
            cudaError_t e = launch_pdl(embed_hist_kernel, dim3(a.chunks), dim3(256), 0, s, a);
            if (e != cudaSuccess) return e;
            e = launch_pdl(embed_scatter_kernel, dim3(a.chunks), dim3(256), 0, s, a);
            if (e != cudaSuccess) return e;
            count_launch(2);
            sorted = a.out;
            a.in = a.out;
            a.out = a.out == w.a ? w.b : w.a;
        }
    }
    // the widest vector of the dy rows; a dW of another type moves as many elements at once
    switch (row_vec(c.d, (int)sizeof(T))) {
        case 8:
            if constexpr (sizeof(T) == 2) return launch_embed_bwd_v<T, G, 8>(c, sorted, w.part, dy, dW, s);
        case 4: return launch_embed_bwd_v<T, G, 4>(c, sorted, w.part, dy, dW, s);
        case 2: return launch_embed_bwd_v<T, G, 2>(c, sorted, w.part, dy, dW, s);
        default: return launch_embed_bwd_v<T, G, 1>(c, sorted, w.part, dy, dW, s);
    }
}

moe_status_t check_embed(const moe_embed_config_t* c) {
    if (!c || c->T < 0 || c->V < 1 || c->d < 1 || !std::isfinite(c->scale)) return MOE_ERR_INVALID_ARG;
    if (c->padding_id < -1 || c->padding_id >= c->V) return MOE_ERR_INVALID_ARG;
    if (c->dtype != MOE_F32 && c->dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (c->grad_dtype != MOE_F32 && c->grad_dtype != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (c->accumulate != 0 && c->accumulate != 1) return MOE_ERR_INVALID_ARG;
    // the positions of the sorted tokens, a group past the last one and the key V + 1 are 32-bit,
    // and so is the column a block past the last one starts at
    if (c->T > INT32_MAX - 4096 || c->V > INT32_MAX - 4096 || c->d > (1 << 28)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API moe_status_t moe_embed(const moe_embed_config_t* cfg, const int32_t* ids, const void* W, void* y,
                                          moe_stream_t stream) {
    const moe_status_t st = check_embed(cfg);
    if (st != MOE_OK) return st;
    if (!W || (cfg->T > 0 && (!ids || !y))) return MOE_ERR_INVALID_ARG;
    if (misaligned(W, 16) || misaligned(y, 16) || misaligned(ids, 4)) return MOE_ERR_INVALID_ARG;
    if (cfg->T == 0) return MOE_OK;
    const cudaError_t e = cfg->dtype == MOE_BF16
                              ? launch_embed<__nv_bfloat16>(*cfg, ids, W, y, (cudaStream_t)stream)
                              : launch_embed<float>(*cfg, ids, W, y, (cudaStream_t)stream);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API size_t moe_embed_workspace_bytes(const moe_embed_config_t* cfg) {
    if (check_embed(cfg) != MOE_OK) return 0;
    EmbedScratch s;
    return carve_embed(*cfg, nullptr, &s);
}

extern "C" MOE_API moe_status_t moe_embed_backward(const moe_embed_config_t* cfg, const int32_t* ids, const void* dy,
                                                   void* dW, void* ws, moe_stream_t stream) {
    const moe_status_t st = check_embed(cfg);
    if (st != MOE_OK) return st;
    if (!dW || !ws || (cfg->T > 0 && (!ids || !dy))) return MOE_ERR_INVALID_ARG;
    if (misaligned(dW, 16) || misaligned(dy, 16) || misaligned(ws, 16) || misaligned(ids, 4))
        return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    cudaError_t e;
    if (cfg->dtype == MOE_BF16)
        e = cfg->grad_dtype == MOE_BF16 ? launch_embed_bwd<__nv_bfloat16, __nv_bfloat16>(*cfg, ids, dy, dW, ws, s)
                                        : launch_embed_bwd<__nv_bfloat16, float>(*cfg, ids, dy, dW, ws, s);
    else
        e = cfg->grad_dtype == MOE_BF16 ? launch_embed_bwd<float, __nv_bfloat16>(*cfg, ids, dy, dW, ws, s)
                                        : launch_embed_bwd<float, float>(*cfg, ids, dy, dW, ws, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
