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

// VE elements as they are in memory.
template <typename T, int VE>
struct Bits {
    static constexpr int kBytes = (int)sizeof(T) * VE, kPart = kBytes > 16 ? 16 : kBytes, kParts = kBytes / kPart;
    typename Raw<kPart>::T u[kParts];
    __device__ __forceinline__ void load(const T* p) {
#pragma unroll
        for (int i = 0; i < kParts; ++i) u[i] = reinterpret_cast<const typename Raw<kPart>::T*>(p)[i];
    }
    __device__ __forceinline__ float at(int i) const { return Elem<T>::to_f(reinterpret_cast<const T*>(u)[i]); }
};

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
// y[t] = scale * W[ids[t]]: U vectors a thread, all loads of a thread in flight together. Bound by
// memory and the two latencies (id, then row) a block pays. 16384 x 1024 bf16 tokens: 10.6 us, 4590
// GB/s of needed traffic (68 %); U = 1: 12.1, U = 4: 11.7, U = 8: 16.5. Shorter vectors take more:
// of four elements 4 (16384 x 1020 bf16 13.4 us, 14.8 with 2, 15.7 with 8), of one or two 8 (x 1022
// 19.5, 23.9 with 2; x 1023 31.4, 41.6). Fewer vectors than 4 to each of an SM's 2048 threads take
// U = 1: there latency counts, not bytes.
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
        constexpr int kMany = VE >= 8 ? 2 : VE == 4 ? 4 : 8;
        if (total >= 2048u * 4u * (uint32_t)num_sms())
            e = launch_pdl(embed_kernel<T, VE, kMany>, dim3(ceil_div(total, 256 * kMany)), dim3(256), 0, s,
                           ids + t0, w, out, total, (uint32_t)nvec, (int)c.V, c.scale, device_error_word());
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
// Stable radix sort of (id, token) pairs, least digit first, by ordinary launches: a histogram of
// every chunk of kChunk pairs for the first digit, then for each digit (with many chunks) a scan of
// the histogram, and the chunks' ranks and the scatter, which also counts the next digit's histogram
// by integer atomics. Left-out tokens
// (padding, ids out of range) take the key V and end up behind all others.
// Bound by latency: two digits take three launches of 2, 4 and 4 us at 4096 tokens; at 32768 they
// take five, the scans 5 and the scatters 6 us each (by themselves, caches cold). One block for all
// of it takes 4 us at 777 tokens, 6 at 2048, 10 at 4096 and 45 at 16384 (one SM then ranks and
// scatters everything): it sorts batches of up to 4096.
// The sort needs few of the SMs: the other blocks of its launches zero the first rows of a dW that
// is overwritten, whether or not they get a sum later. (Where dW is added to, bringing dy into the
// L2 cache meanwhile gained nothing: the sums wait for latencies, not for bytes.)
struct ZeroArgs {
    char* p;
    int64_t bytes;                         // a multiple of 16
};
constexpr int kZeroBytes = 16384;          // a block's part

__device__ __forceinline__ void zero_part(const ZeroArgs& z, int block) {
    char* p = z.p + (int64_t)block * kZeroBytes;
    const int n = (int)min((int64_t)kZeroBytes, z.bytes - (int64_t)block * kZeroBytes);
    for (int i = threadIdx.x * 16; i < n; i += blockDim.x * 16) *reinterpret_cast<uint4*>(p + i) = make_uint4(0u, 0u, 0u, 0u);
}

constexpr int kChunk = 1024;         // pairs a block of 256 threads ranks
constexpr int kWarps = 8;
constexpr int kPerLane = kChunk / 256;
constexpr int kMaxBits = 9;          // bits of a digit
constexpr int kMaxBins = 1 << kMaxBits;
constexpr int kMaxPasses = 4;        // 31 bits of keys
// Bytes zeroed beside one launch of the sort: about what the memory takes in its time at 16384 to
// 32768 tokens. A smaller batch's launches are shorter, and the zeros then outlast them; all of the
// bytes have to be written by the end in any case, by these blocks or by the last launch's.
constexpr int64_t kZeroOne = 24 << 20, kZeroHist = 32 << 20, kZeroScatter = 44 << 20;

struct SortArgs {
    const int32_t* ids;      // first pass: keys are made from the ids
    const uint2* in;         // later passes: (key, token)
    uint2* out;
    int32_t* hist;           // [chunks, bins] of this pass
    int32_t* hist_next;      // of the next, or null
    int32_t* total;          // [bins] of the whole batch, where embed_scan_kernel has run; else null
    int64_t later;           // first launch: counts of the later passes' histograms, to zero
    int32_t* crossing;       // counts of crossing runs, zeroed here (see SumArgs)
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

// Lanes whose digit is this lane's, by one ballot a bit (a match instruction takes three times as
// long where a whole SM ranks: 90 cycles a warp).
__device__ __forceinline__ uint32_t same_digit(uint32_t dg, int bits) {
    uint32_t same = 0xffffffffu;
#pragma unroll
    for (int b = 0; b <= kMaxBits; ++b) {
        if (b > bits) break;                         // one bit more than the digit: lanes past the end
        const uint32_t set = __ballot_sync(0xffffffffu, dg >> b & 1);
        same &= dg >> b & 1 ? set : ~set;
    }
    return same;
}

__global__ void __launch_bounds__(256) embed_hist_kernel(SortArgs a, ZeroArgs z) {
    __shared__ int h[kMaxBins];
    const int bins = 1 << a.bits;
    for (int b = threadIdx.x; b < bins; b += 256) h[b] = 0;
    pdl_wait();
    if ((int)blockIdx.x >= a.chunks) {
        zero_part(z, blockIdx.x - a.chunks);
        return;
    }
    for (int64_t i = (int64_t)blockIdx.x * 256 + threadIdx.x; i < a.later; i += (int64_t)a.chunks * 256)
        a.hist_next[i] = 0;
    __syncthreads();
    if (blockIdx.x == 0 && threadIdx.x < 2) a.crossing[threadIdx.x] = 0;
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

// The histogram's counts as counts of the chunks before each, and the totals: one column to 32
// threads, each of which takes a 32nd of the chunks. Without it every block of the scatter reads the
// whole histogram, chunks^2 bins counts in all, 2 GB a digit at a million tokens. That is less than
// this launch takes while chunks are few. The gradient of rows of 64 bf16, added to 131072 rows, with
// the scan and without: 8192 tokens 23.6 and 22.7 us, 16384 24.3 and 25.4, 32768 26.6 and 29.0,
// 1048576 298 and 579.
constexpr int kScanFrom = 16;        // chunks
__global__ void __launch_bounds__(1024) embed_scan_kernel(int32_t* hist, int32_t* total, int chunks, int bins) {
    __shared__ int part[32][33];
    pdl_wait();
    const int col = blockIdx.x * 32 + (threadIdx.x & 31), seg = threadIdx.x >> 5, each = (chunks + 31) / 32;
    const int c0 = min(seg * each, chunks), c1 = min(c0 + each, chunks);
    const bool live = col < bins;
    constexpr int kAtOnce = 8;
    int sum = 0;
    if (live)
#pragma unroll 8
        for (int c = c0; c < c1; ++c) sum += hist[(int64_t)c * bins + col];
    part[seg][threadIdx.x & 31] = sum;
    __syncthreads();
    if (!live) return;
    int run = 0;
    for (int s = 0; s < seg; ++s) run += part[s][threadIdx.x & 31];
    for (int c = c0; c < c1; c += kAtOnce) {
        int n[kAtOnce];
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) n[j] = c + j < c1 ? hist[(int64_t)(c + j) * bins + col] : 0;
#pragma unroll
        for (int j = 0; j < kAtOnce; ++j) {
            if (c + j < c1) hist[(int64_t)(c + j) * bins + col] = run;
            run += n[j];
        }
    }
    if (seg == 31) total[col] = run;
}

__global__ void __launch_bounds__(256) embed_scatter_kernel(SortArgs a, ZeroArgs z) {
    __shared__ int cnt[kWarps][kMaxBins];
    __shared__ int base[kMaxBins];
    __shared__ int tmp[kWarps];
    const int bins = 1 << a.bits, lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    for (int b = threadIdx.x; b < kWarps * kMaxBins; b += 256) (&cnt[0][0])[b] = 0;
    pdl_wait();
    if ((int)blockIdx.x >= a.chunks) {
        zero_part(z, blockIdx.x - a.chunks);
        return;
    }
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
    // totals of all digits, and of the chunks before this one
    int tot[2] = {0, 0}, mine[2] = {0, 0};
    if (2 * (int)threadIdx.x < bins && a.total) {
        const int2 v = reinterpret_cast<const int2*>(a.total)[threadIdx.x];
        const int2 w = reinterpret_cast<const int2*>(a.hist)[(int64_t)blockIdx.x * (bins / 2) + threadIdx.x];
        tot[0] = v.x;
        tot[1] = v.y;
        mine[0] = w.x;
        mine[1] = w.y;
    } else if (2 * (int)threadIdx.x < bins) {
        const int2* h = reinterpret_cast<const int2*>(a.hist) + threadIdx.x;
#pragma unroll 8
        for (int c = 0; c < a.chunks; ++c) {
            const int2 v = h[(int64_t)c * (bins / 2)];
            tot[0] += v.x;
            tot[1] += v.y;
            if (c < (int)blockIdx.x) {
                mine[0] += v.x;
                mine[1] += v.y;
            }
        }
    }
#pragma unroll
    for (int k = 0; k < kPerLane; ++k) {
        const bool live = i0 + k * 32 + lane < a.T;
        const int dg = live ? (int)((pr[k].x >> a.shift) & (bins - 1)) : bins;
        const uint32_t same = same_digit(dg, a.bits);
        const int before = __popc(same & ((1u << lane) - 1u));
        const int had = live ? cnt[warp][dg] : 0;
        __syncwarp();
        if (live && before == 0) cnt[warp][dg] = had + __popc(same);
        __syncwarp();
        rank[k] = had + before;
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
        if (i0 + k * 32 + lane < a.T) {
            const int to = cnt[warp][(pr[k].x >> a.shift) & (bins - 1)] + rank[k];
            a.out[to] = pr[k];
            if (a.hist_next)
                atomicAdd(a.hist_next + (int64_t)(to / kChunk) * bins + (pr[k].x >> (a.shift + a.bits) & (bins - 1)), 1);
        }
}

// A batch of at most kOneBlock tokens is sorted by one block in one launch, in shared memory:
// keys, tokens (16 bits) and the warps' digit counts.
constexpr int kOneBlock = 4096;
constexpr int kOneThreads = 1024;
constexpr int kOneWarps = kOneThreads / 32;
constexpr int kOneEach = kOneBlock / kOneThreads;

__global__ void __launch_bounds__(kOneThreads) embed_sort_kernel(SortArgs a, int passes, ZeroArgs z) {
    extern __shared__ __align__(16) unsigned char smem[];
    uint32_t* keys = reinterpret_cast<uint32_t*>(smem);
    uint16_t* toks = reinterpret_cast<uint16_t*>(keys + kOneBlock);
    uint16_t(*cnt)[kMaxBins] = reinterpret_cast<uint16_t(*)[kMaxBins]>(toks + kOneBlock);
    __shared__ int total[kMaxBins], tmp[kOneWarps];
    pdl_wait();
    if (blockIdx.x > 0) {
        zero_part(z, blockIdx.x - 1);
        return;
    }
    if (threadIdx.x < 2) a.crossing[threadIdx.x] = 0;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, bins = 1 << a.bits;
    // a warp holds consecutive pairs, `each` to a lane; a shorter batch takes fewer
    const int each = (a.T + kOneThreads - 1) / kOneThreads, i0 = warp * each * 32;
    uint32_t key[kOneEach], tok[kOneEach], rank[kOneEach];
#pragma unroll
    for (int k = 0; k < kOneEach; ++k) {
        const int i = i0 + k * 32 + lane;
        key[k] = 0;
        tok[k] = (uint32_t)i;
        if (k < each && i < a.T) key[k] = sort_pair(a, i, true).x;
    }
    for (int p = 0; p < passes; ++p) {
        const int shift = p * a.bits;
        for (int b = threadIdx.x; b < kOneWarps * kMaxBins / 2; b += kOneThreads) reinterpret_cast<uint32_t*>(cnt)[b] = 0;
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kOneEach; ++k) {
            if (k >= each) break;
            const bool live = i0 + k * 32 + lane < a.T;
            const uint32_t dg = live ? key[k] >> shift & (bins - 1) : (uint32_t)bins;
            const uint32_t same = same_digit(dg, a.bits);
            const uint32_t before = __popc(same & ((1u << lane) - 1u));
            const uint32_t had = live ? cnt[warp][dg] : 0u;
            __syncwarp();
            if (live && before == 0) cnt[warp][dg] = (uint16_t)(had + __popc(same));
            __syncwarp();
            rank[k] = had + before;
        }
        __syncthreads();
        // counts before each warp within a digit, then before each digit
        if (threadIdx.x < kMaxBins) {
            int run = 0;
            if ((int)threadIdx.x < bins)
#pragma unroll 8
                for (int w = 0; w < kOneWarps; ++w) {
                    const int n = cnt[w][threadIdx.x];
                    cnt[w][threadIdx.x] = (uint16_t)run;
                    run += n;
                }
            int x = run;
#pragma unroll
            for (int o = 1; o < 32; o <<= 1) {
                const int n = __shfl_up_sync(0xffffffffu, x, o);
                if (lane >= o) x += n;
            }
            if (lane == 31) tmp[warp] = x;
            total[threadIdx.x] = x - run;
        }
        __syncthreads();
        if (threadIdx.x < kMaxBins) {
            int before = 0;
            for (int w = 0; w < warp; ++w) before += tmp[w];
            total[threadIdx.x] += before;
        }
        __syncthreads();
#pragma unroll
        for (int k = 0; k < kOneEach; ++k) {
            if (k >= each) break;
            if (i0 + k * 32 + lane < a.T) {
                const uint32_t dg = key[k] >> shift & (bins - 1);
                const uint32_t to = (uint32_t)total[dg] + cnt[warp][dg] + rank[k];
                keys[to] = key[k];
                toks[to] = (uint16_t)tok[k];
            }
        }
        __syncthreads();
        if (p + 1 < passes)
#pragma unroll
            for (int k = 0; k < kOneEach; ++k) {
                const int i = i0 + k * 32 + lane;
                if (k < each && i < a.T) {
                    key[k] = keys[i];
                    tok[k] = toks[i];
                }
            }
    }
    for (int i = threadIdx.x; i < a.T; i += kOneThreads) a.out[i] = make_uint2(keys[i], toks[i]);
}

// ---------------------------------------------------------------- gradient: sums over runs
// The sorted pairs are cut into groups of kGroup. A thread owns VE columns of one group, loads
// them of several rows (and of the dW rows that it will add to) at once, and walks them in
// order; a run of one token that lies inside the group is finished there. A run that crosses
// groups leaves one fp32 partial row in each (slot 0: the run the group begins with, slot 1: the
// run it ends with and that begins in it) and an entry in a list, and embed_join_kernel adds them
// in group order. Every row of dW has one writer and a fixed order of sums.
// Bound by memory (dy once, the touched rows of dW) and by the latency of gathered rows: 32768 x
// 2048 bf16 into fp32 rows that are added to, 51 us by themselves of 79 in all, 272 MB at 5300 GB/s,
// 54 registers and half of the warps resident. Groups of 8 leave twice the partial rows (88 us in
// all against 81 at the time), groups of 32 half the blocks (86).
constexpr int kGroup = 16;
constexpr int kLong = 16;        // a run over more groups than this is joined by a whole block

struct SumArgs {
    const uint2* pairs;      // sorted (key, token)
    float* part;             // [groups, 2, d]
    int32_t* crossing;       // counts of crossing runs: short ones, long ones
    uint2* heads;            // [2, groups] their keys and the groups they begin in, in any order
    int T, V, d, groups;
    int zero_from;           // first row that is zeroed here if it gets no sum
    int joins;               // blocks of the last launch that join; the others zero rows
    float scale;
};

// First position whose key is >= key.
__device__ __forceinline__ int lower_bound(const uint2* p, int n, uint32_t key) {
    int lo = 0, hi = n;
    while (lo < hi) {
        const int mid = lo + (hi - lo) / 2;              // lo + hi passes 31 bits above 2^30 tokens
        if (p[mid].x < key) lo = mid + 1; else hi = mid;
    }
    return lo;
}

// Zero rows of tokens that do not occur. A block owns 64 rows: one search for its first key,
// then the sorted keys of its rows mark the ones that were seen.
constexpr int kZeroRows = 64;
template <typename G, int VE>
__device__ __forceinline__ void zero_rows(const SumArgs& a, G* dW, int block) {
    __shared__ int seen[kZeroRows];
    __shared__ int lo, hi;
    for (int i = threadIdx.x; i < kZeroRows; i += blockDim.x) seen[i] = 0;
    const int v0 = a.zero_from + block * kZeroRows, v1 = min(v0 + kZeroRows, a.V);
    if (threadIdx.x == 0) lo = lower_bound(a.pairs, a.T, (uint32_t)v0);
    if (threadIdx.x == 32) hi = lower_bound(a.pairs, a.T, (uint32_t)v1);
    __syncthreads();
    for (int i = lo + threadIdx.x; i < hi; i += blockDim.x) seen[a.pairs[i].x - v0] = 1;
    __syncthreads();
    float z[VE];
#pragma unroll
    for (int i = 0; i < VE; ++i) z[i] = 0.f;
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int64_t row = (int64_t)a.d * (int64_t)sizeof(G);
    for (int v = v0 + warp; v < v1; v += blockDim.x >> 5) {
        if (seen[v - v0]) continue;
        char* p = reinterpret_cast<char*>(dW) + v * row;
        if (row % 16 == 0)
            for (int64_t c = lane * 16; c < row; c += 512) *reinterpret_cast<uint4*>(p + c) = make_uint4(0u, 0u, 0u, 0u);
        else
            for (int c = lane * VE; c < a.d; c += 32 * VE) Vec<G, VE>::store(dW + (int64_t)v * a.d + c, z);
    }
}

template <typename T, typename G, int VE, bool kAdd>
__global__ void __launch_bounds__(128, 8) embed_sum_kernel(SumArgs a, const T* __restrict__ dy, G* __restrict__ dW) {
    __shared__ uint2 pr[kGroup + 2];   // the group's pairs, with a neighbour on either side
    pdl_wait();
    const int g = blockIdx.x, i0 = g * kGroup;
    if ((int)threadIdx.x < kGroup + 2) {
        const int i = i0 + (int)threadIdx.x - 1;
        pr[threadIdx.x] = i >= 0 && i < a.T ? a.pairs[i] : make_uint2(0xffffffffu, 0u);
    }
    __syncthreads();
    for (int col = (blockIdx.y * blockDim.x + threadIdx.x) * VE; col < a.d; col += gridDim.y * blockDim.x * VE) {
        float s[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] = 0.f;
        bool from_before = pr[0].x == pr[1].x;
        // Rows in flight: four, or two where dW is added to, whose old rows take registers too: with
        // eight (and four) half as many blocks fit an SM (32768 x 2048 into fp32: 88 against 81 us). All
        // 16 staged in shared memory by asynchronous copies cost residency too: 65 against 53 us.
        // Vectors of one or two elements take few registers, and go 16 at once: 6566 x 1393 bf16 added
        // to fp32 36 us against 51, 32768 x 511 54 against 81.
        constexpr int kAtOnce = VE <= 2 ? kGroup : kAdd ? 2 : 4;
#pragma unroll
        for (int j0 = 0; j0 < kGroup; j0 += kAtOnce) {
            Bits<T, VE> r[kAtOnce];
            Bits<G, kAdd ? VE : 1> old[kAtOnce];
            bool before = from_before;
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const uint2 q = pr[j0 + j + 1];
                if (q.x >= (uint32_t)a.V) continue;
                r[j].load(dy + (int64_t)q.y * a.d + col);
                if constexpr (kAdd) {
                    const bool ends = pr[j0 + j + 2].x != q.x;
                    if (ends && !before) old[j].load(dW + (int64_t)q.x * a.d + col);
                    before = before && !ends;
                }
            }
#pragma unroll
            for (int j = 0; j < kAtOnce; ++j) {
                const uint32_t key = pr[j0 + j + 1].x;
                if (key >= (uint32_t)a.V) break;
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] += r[j].at(i);
                const bool ends = pr[j0 + j + 2].x != key;
                if (!ends && j0 + j + 1 < kGroup) continue;
                if (ends && !from_before) {
#pragma unroll
                    for (int i = 0; i < VE; ++i) s[i] *= a.scale;
                    if constexpr (kAdd)
#pragma unroll
                        for (int i = 0; i < VE; ++i) s[i] += old[j].at(i);
                    Vec<G, VE>::store(dW + (int64_t)key * a.d + col, s);
                } else {
                    Vec<float, VE>::store(a.part + ((int64_t)g * 2 + (from_before ? 0 : 1)) * a.d + col, s);
                    if (!ends && !from_before && col == 0) {
                        const int64_t far = (int64_t)(g + kLong) * kGroup;
                        const int is_long = far < a.T && a.pairs[far].x == key;
                        a.heads[(int64_t)is_long * a.groups + atomicAdd(a.crossing + is_long, 1)] = make_uint2(key, g);
                    }
                }
                from_before = false;
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] = 0.f;
            }
        }
    }
}

// The crossing runs' partial rows (531 runs of 7264 in a batch of 16384 tokens), in order,
// 32 * VE columns at a time: one by a warp, or a long one by a block, whose eight warps take every
// eighth partial and whose sums are added in warp order.
template <typename G, int VE, bool kAdd>
__device__ __forceinline__ void join_row(const SumArgs& a, G* dW, uint32_t key, int col, float (&s)[VE]) {
    G* p = dW + (int64_t)key * a.d + col;
    float old[VE];
    if constexpr (kAdd) Vec<G, VE>::load(p, old);
#pragma unroll
    for (int i = 0; i < VE; ++i) s[i] = kAdd ? fmaf(s[i], a.scale, old[i]) : s[i] * a.scale;
    Vec<G, VE>::store(p, s);
}

// The other blocks zero the rows that get no sum and that the sort's launches have not zeroed: the
// joins' chain of latencies (8 us) passes beside them. The whole gradient of 16384 x 1024 bf16 into
// 131072 rows: 59 us, 5080 GB/s of needed traffic (76 %); zeros after the joins: 87.
template <typename G, int VE, bool kAdd>
__global__ void __launch_bounds__(256) embed_join_kernel(SumArgs a, G* __restrict__ dW) {
    __shared__ float part[kWarps][32 * VE];
    pdl_wait();
    if ((int)blockIdx.x >= a.joins) {
        zero_rows<G, VE>(a, dW, blockIdx.x - a.joins);
        return;
    }
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5;
    const int slabs = (a.d + 32 * VE - 1) / (32 * VE);
    const auto add = [&](float (&s)[VE], int g, int k, int col) {
        float r[VE];
        Vec<float, VE>::load(a.part + ((int64_t)(g + k) * 2 + (k ? 0 : 1)) * a.d + col, r);
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] += r[i];
    };
    const int64_t n_long = (int64_t)a.crossing[1] * slabs, n_short = (int64_t)a.crossing[0] * slabs;
    // While the long ones take less than half of the blocks, each has one and the other blocks take
    // the short ones; else all blocks take both.
    const bool apart = n_long * 2 <= a.joins;
    for (int64_t q = blockIdx.x; q < n_long; q += a.joins) {
        const uint2 head = a.heads[a.groups + q / slabs];
        const int g = (int)head.y, col = ((int)(q % slabs) * 32 + lane) * VE;
        const uint32_t key = head.x;
        // groups that the run reaches into, looked at 256 at a time
        int parts = 1;
        for (int in = 256; in == 256; parts += in) {
            const int64_t i = (int64_t)(g + parts + (int)threadIdx.x) * kGroup;
            in = __syncthreads_count(i < a.T && a.pairs[i].x == key);
        }
        float s[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] = 0.f;
        if (col < a.d)
#pragma unroll 8
            for (int k = warp; k < parts; k += kWarps) add(s, g, k, col);
#pragma unroll
        for (int i = 0; i < VE; ++i) part[warp][lane * VE + i] = s[i];
        __syncthreads();
        if (warp == 0 && col < a.d) {
#pragma unroll
            for (int w = 1; w < kWarps; ++w)
#pragma unroll
                for (int i = 0; i < VE; ++i) s[i] += part[w][lane * VE + i];
            join_row<G, VE, kAdd>(a, dW, key, col, s);
        }
        __syncthreads();
    }
    const int64_t first = (int64_t)blockIdx.x - (apart ? n_long : 0), blocks = a.joins - (apart ? n_long : 0);
    if (first < 0) return;
    for (int64_t q = first * kWarps + warp; q < n_short; q += blocks * kWarps) {
        const uint2 head = a.heads[q / slabs];
        const int g = (int)head.y, col = ((int)(q % slabs) * 32 + lane) * VE;
        const uint32_t key = head.x;
        float s[VE];
#pragma unroll
        for (int i = 0; i < VE; ++i) s[i] = 0.f;
        if (col < a.d) {
            add(s, g, 0, col);                       // there are two parts at least
            add(s, g, 1, col);
        }
        static_assert(kLong <= 32, "one look finds a short run's end");
        const int64_t i = (int64_t)(g + 1 + lane) * kGroup;
        const int parts = 1 + __popc(__ballot_sync(0xffffffffu, i < a.T && a.pairs[i].x == key));
        if (col >= a.d) continue;
#pragma unroll 8
        for (int k = 2; k < parts; ++k) add(s, g, k, col);
        join_row<G, VE, kAdd>(a, dW, key, col, s);
    }
}

struct EmbedScratch {
    uint2* a;
    uint2* b;
    int32_t* hist;
    int32_t* total;
    int32_t* crossing;
    uint2* heads;
    float* part;
};

int groups_of(const moe_embed_config_t& c) { return ceil_div(c.T, kGroup); }

size_t carve_embed(const moe_embed_config_t& c, void* base, EmbedScratch* s) {
    Workspace ws{static_cast<char*>(base), 0};
    s->a = ws.take<uint2>((size_t)c.T + 1);
    s->b = ws.take<uint2>((size_t)c.T + 1);
    s->hist = ws.take<int32_t>((size_t)ceil_div(c.T, kChunk) * kMaxBins * kMaxPasses + 1);
    s->total = ws.take<int32_t>(kMaxBins);
    s->crossing = ws.take<int32_t>(2);
    s->heads = ws.take<uint2>((size_t)groups_of(c) * 2 + 1);
    s->part = ws.take<float>((size_t)groups_of(c) * 2 * c.d + 4);
    return align_up(ws.used, 256);
}

template <typename T, typename G, int VE, bool kAdd>
cudaError_t launch_sums(const moe_embed_config_t& c, SumArgs a, const void* dy, void* dW, cudaStream_t s) {
    const int nvec = c.d / VE;
    G* out = static_cast<G*>(dW);
    const int threads = std::max(64, std::min(128, ceil_div(nvec, 32) * 32));
    cudaError_t e = cudaSuccess;
    if (a.groups > 0) {
        e = launch_pdl(embed_sum_kernel<T, G, VE, kAdd>, dim3(a.groups, std::min(ceil_div(nvec, threads), 64)),
                       dim3(threads), 0, s, a, static_cast<const T*>(dy), out);
        count_launch();
        if (e != cudaSuccess) return e;
    }
    // as many warps as there can be items, up to what the SMs hold; one group has no run that leaves it
    const int64_t items = (int64_t)a.groups * ceil_div(nvec, 32);
    a.joins = a.groups < 2 ? 0 : (int)std::min<int64_t>((items + 7) / 8, num_sms() * 6);
    const int zero = kAdd ? 0 : ceil_div(a.V - a.zero_from, kZeroRows);
    if (a.joins + zero == 0) return e;
    e = launch_pdl(embed_join_kernel<G, VE, kAdd>, dim3(a.joins + zero), dim3(256), 0, s, a, out);
    count_launch();
    return e;
}

template <typename T, typename G, int VE>
cudaError_t launch_embed_bwd_v(const moe_embed_config_t& c, const SumArgs& a, const void* dy, void* dW, cudaStream_t s) {
    return c.accumulate ? launch_sums<T, G, VE, true>(c, a, dy, dW, s) : launch_sums<T, G, VE, false>(c, a, dy, dW, s);
}

template <typename T, typename G>
cudaError_t launch_embed_bwd(const moe_embed_config_t& c, const int32_t* ids, const void* dy, void* dW, void* ws,
                             cudaStream_t s) {
    EmbedScratch w;
    carve_embed(c, ws, &w);
    SumArgs sums{w.a, w.part, w.crossing, w.heads, c.T, c.V, c.d, groups_of(c), 0, 0, c.scale};
    if (c.T > 0) {
        int bits = 1;
        while (((int64_t)1 << bits) <= c.V) ++bits;          // keys 0 .. V
        const int passes = ceil_div(bits, kMaxBits), digit = ceil_div(bits, passes);
        SortArgs a{ids, nullptr, w.a, w.hist, nullptr, nullptr, 0, w.crossing, c.T, c.V, c.padding_id, 0, digit,
                   ceil_div(c.T, kChunk), device_error_word()};
        // the next `wish` bytes of dW, in whole rows whose bytes are a multiple of 16, and their blocks
        const int64_t row = (int64_t)c.d * (int64_t)sizeof(G);
        unsigned blocks = 0;
        const auto zero_next = [&](int64_t wish) {
            const int rows = c.accumulate ? 0 : (int)std::min<int64_t>(c.V - sums.zero_from, wish / row) & ~15;
            const ZeroArgs z{static_cast<char*>(dW) + sums.zero_from * row, rows * row};
            sums.zero_from += rows;
            blocks = (unsigned)((z.bytes + kZeroBytes - 1) / kZeroBytes);
            return z;
        };
        cudaError_t e;
        if (c.T <= kOneBlock) {
            constexpr int smem = kOneBlock * 6 + kOneWarps * kMaxBins * 2;
            e = cudaFuncSetAttribute(embed_sort_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem);
            if (e != cudaSuccess) return e;
            const ZeroArgs z = zero_next(kZeroOne);
            e = launch_pdl(embed_sort_kernel, dim3(1 + blocks), dim3(kOneThreads), (size_t)smem, s, a, passes, z);
            count_launch();
            if (e != cudaSuccess) return e;
        } else {
            const int64_t size = (int64_t)a.chunks << digit;
            a.hist_next = w.hist + size;
            a.later = size * (passes - 1);
            ZeroArgs z = zero_next(kZeroHist);
            e = launch_pdl(embed_hist_kernel, dim3(a.chunks + blocks), dim3(256), 0, s, a, z);
            count_launch();
            if (e != cudaSuccess) return e;
            for (int p = 0; p < passes; ++p) {
                a.shift = p * digit;
                a.hist = w.hist + size * p;
                a.hist_next = p + 1 < passes ? a.hist + size : nullptr;
                if (a.chunks >= kScanFrom) {
                    a.total = w.total;
                    e = launch_pdl(embed_scan_kernel, dim3(ceil_div(1 << digit, 32)), dim3(1024), 0, s, a.hist, a.total,
                                   a.chunks, 1 << digit);
                    count_launch();
                    if (e != cudaSuccess) return e;
                }
                z = zero_next(kZeroScatter);
                e = launch_pdl(embed_scatter_kernel, dim3(a.chunks + blocks), dim3(256), 0, s, a, z);
                count_launch();
                if (e != cudaSuccess) return e;
                sums.pairs = a.out;
                a.in = a.out;
                a.out = a.out == w.a ? w.b : w.a;
            }
        }
    }
    // the widest vector of the dy rows; a dW of another type moves as many elements at once
    switch (row_vec(c.d, (int)sizeof(T))) {
        case 8:
            if constexpr (sizeof(T) == 2) return launch_embed_bwd_v<T, G, 8>(c, sums, dy, dW, s);
        case 4: return launch_embed_bwd_v<T, G, 4>(c, sums, dy, dW, s);
        case 2: return launch_embed_bwd_v<T, G, 2>(c, sums, dy, dW, s);
        default: return launch_embed_bwd_v<T, G, 1>(c, sums, dy, dW, s);
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
