// Layer norm of rows (and of a residual sum), and its gradient.
#include <cmath>

#include "internal.cuh"
#include "tc_ptx.cuh"

namespace moe {

namespace {

// ---------------------------------------------------------------- vectors of VE elements
template <int BYTES> struct Raw;
template <> struct Raw<2> { using T = uint16_t; };
template <> struct Raw<4> { using T = uint32_t; };
template <> struct Raw<8> { using T = uint2; };
template <> struct Raw<16> { using T = uint4; };

// VE elements as they are in memory.
template <typename T, int VE>
struct Chunk {
    using R = typename Raw<(int)sizeof(T) * VE>::T;
    R u;
    __device__ __forceinline__ void load(const T* p) { u = *reinterpret_cast<const R*>(p); }
    __device__ __forceinline__ void zero() { u = R{}; }
    __device__ __forceinline__ void get(float (&f)[VE]) const {
        const T* e = reinterpret_cast<const T*>(&u);
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = Elem<T>::to_f(e[i]);
    }
    static __device__ __forceinline__ void store(T* p, const float (&f)[VE]) {
        R u;
        T* e = reinterpret_cast<T*>(&u);
#pragma unroll
        for (int i = 0; i < VE; ++i) e[i] = Elem<T>::from_f(f[i]);
        *reinterpret_cast<R*>(p) = u;
    }
};

// VE parameters from column c on (fp32 or bf16; null: `none`).
template <int VE>
__device__ __forceinline__ void load_params(const void* p, bool f32, int c, float none, float (&f)[VE]) {
    if (!p) {
#pragma unroll
        for (int i = 0; i < VE; ++i) f[i] = none;
    } else if (f32) {
        if constexpr (VE >= 4) {
#pragma unroll
            for (int i = 0; i < VE; i += 4) {
                const float4 v = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(p) + c + i));
                f[i] = v.x; f[i + 1] = v.y; f[i + 2] = v.z; f[i + 3] = v.w;
            }
        } else {
#pragma unroll
            for (int i = 0; i < VE; ++i) f[i] = __ldg(static_cast<const float*>(p) + c + i);
        }
    } else {
        Chunk<__nv_bfloat16, VE> v;
        v.load(static_cast<const __nv_bfloat16*>(p) + c);
        v.get(f);
    }
}

// NE elements of a row as a thread holds them: chunks `lane`, lane + tpr, ... of the row's nvec; beyond
// them zero. FULL: the row is just that many chunks. Arithmetic is on packed fp32 pairs.
template <typename T, int VE, int NE, bool FULL>
struct Part {
    static constexpr int NC = NE / VE, NP = NE / 2;
    Chunk<T, VE> c[NC];
    __device__ __forceinline__ void load(const T* row, int lane, int tpr, int nvec, bool live = true) {
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int at = lane + i * tpr;
            c[i].zero();
            if (live && (FULL || at < nvec)) c[i].load(row + (int64_t)at * VE);
        }
    }
    __device__ __forceinline__ void pairs(uint64_t (&p)[NP]) const {
        if constexpr (VE == 1) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float a[1], b[1];
                c[2 * i].get(a);
                c[2 * i + 1].get(b);
                p[i] = pk2(a[0], b[0]);
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const uint32_t* w = reinterpret_cast<const uint32_t*>(&c[i].u);
#pragma unroll
                for (int k = 0; k < VE / 2; ++k) {
                    if constexpr (sizeof(T) == 2)
                        p[i * (VE / 2) + k] = pk2(__uint_as_float(w[k] << 16), __uint_as_float(w[k] & 0xffff0000u));
                    else
                        p[i * (VE / 2) + k] = pk2(__uint_as_float(w[2 * k]), __uint_as_float(w[2 * k + 1]));
                }
            }
        }
    }
    static __device__ __forceinline__ void store(T* row, int lane, int tpr, int nvec, const uint64_t (&p)[NP]) {
        if constexpr (VE == 1) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                float f[2];
                upk2(p[i], f[0], f[1]);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const int at = lane + (2 * i + k) * tpr;
                    if (FULL || at < nvec) st_f(row + at, f[k]);
                }
            }
        } else {
#pragma unroll
            for (int i = 0; i < NC; ++i) {
                const int at = lane + i * tpr;
                Chunk<T, VE> o;
                uint32_t* w = reinterpret_cast<uint32_t*>(&o.u);
#pragma unroll
                for (int k = 0; k < VE / 2; ++k) {
                    float lo, hi;
                    upk2(p[i * (VE / 2) + k], lo, hi);
                    if constexpr (sizeof(T) == 2) {
                        const __nv_bfloat162 h = __floats2bfloat162_rn(lo, hi);
                        w[k] = *reinterpret_cast<const uint32_t*>(&h);
                    } else {
                        w[2 * k] = __float_as_uint(lo);
                        w[2 * k + 1] = __float_as_uint(hi);
                    }
                }
                if (FULL || at < nvec) *reinterpret_cast<typename Chunk<T, VE>::R*>(row + (int64_t)at * VE) = o.u;
            }
        }
    }
    // Zeros in the pairs of chunks that the row does not have.
    static __device__ __forceinline__ void cut(int lane, int tpr, int nvec, uint64_t (&p)[NP]) {
        if constexpr (!FULL) {
#pragma unroll
            for (int i = 0; i < NP; ++i) {
                if constexpr (VE == 1) {
                    float lo, hi;
                    upk2(p[i], lo, hi);
                    p[i] = pk2(lane + 2 * i * tpr < nvec ? lo : 0.f, lane + (2 * i + 1) * tpr < nvec ? hi : 0.f);
                } else if (lane + i / (VE / 2) * tpr >= nvec) {
                    p[i] = 0;
                }
            }
        }
    }
    // The parameters of the thread's columns.
    static __device__ __forceinline__ void params(const void* v, bool f32, float none, int lane, int tpr, int nvec,
                                                  uint64_t (&p)[NP]) {
        float f[NE];
#pragma unroll
        for (int i = 0; i < NC; ++i) {
            const int at = lane + i * tpr;
            float one[VE];
#pragma unroll
            for (int k = 0; k < VE; ++k) one[k] = none;
            if (FULL || at < nvec) load_params<VE>(v, f32, at * VE, none, one);
#pragma unroll
            for (int k = 0; k < VE; ++k) f[i * VE + k] = one[k];
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) p[i] = pk2(f[2 * i], f[2 * i + 1]);
    }
};

// Widest vector (elements, up to 16 bytes) that divides rows of d elements of es bytes.
int row_vec(int d, int es) {
    int v = 16 / es;
    while (v > 1 && d % v) v /= 2;
    return v;
}

// Sums over the `tpr` threads of a row (a power of two; a block holds whole rows, `own` is the number of the row, or
// of the warp whose rows are shorter, in it). `red` (a value to each warp) is free again after the next sum on another buffer. The row's
// threads meet.
__device__ __forceinline__ void row_sync(int tpr, int own) {
    asm volatile("bar.sync %0, %1;" ::"r"(own + 1), "r"(tpr) : "memory");
}
template <bool SHORT = false>
__device__ __forceinline__ float row_sum(float v, int tpr, int own, float* red) {
    if (SHORT) {                 // (tpr < 32)
        for (int o = tpr >> 1; o > 0; o >>= 1) v += __shfl_xor_sync(0xffffffffu, v, o);
        __syncwarp();
        return v;
    }
    v = warp_sum(v);
    if (tpr == 32) {
        __syncwarp();
        return v;
    }
    const int warp = threadIdx.x >> 5, n = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    row_sync(tpr, own);
    const float* at = red + own * n;
    float s = at[0];
    for (int i = 1; i < n; ++i) s += at[i];
    return s;
}
template <bool SHORT = false>
__device__ __forceinline__ float2 row_sum2(float2 v, int tpr, int own, float2* red) {
    if (SHORT) {                 // (tpr < 32)
        for (int o = tpr >> 1; o > 0; o >>= 1) {
            v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
            v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
        }
        __syncwarp();
        return v;
    }
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) {
        v.x += __shfl_xor_sync(0xffffffffu, v.x, o);
        v.y += __shfl_xor_sync(0xffffffffu, v.y, o);
    }
    if (tpr == 32) {
        __syncwarp();
        return v;
    }
    const int warp = threadIdx.x >> 5, n = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    row_sync(tpr, own);
    const float2* at = red + own * n;
    float2 s = at[0];
    for (int i = 1; i < n; ++i) { s.x += at[i].x; s.y += at[i].y; }
    return s;
}
template <int N>
__device__ __forceinline__ float pair_sum(const uint64_t (&p)[N]) {
    uint64_t s = p[0];
#pragma unroll
    for (int i = 1; i < N; ++i) s = add2(s, p[i]);
    float lo, hi;
    upk2(s, lo, hi);
    return lo + hi;
}

// ---------------------------------------------------------------- rows through shared memory
// A ring of stages in shared memory, which rows reach by bulk copies: up to 180 KB are in flight to an SM
// whatever the registers hold. A stage holds `per` adjacent rows of each of up to three arrays. A copy starts on
// a 16-byte boundary: it takes in what lies before and behind odd rows, but for the end of the last one, whose
// odd bytes a thread fetches.
//
// The forward pass has a ring to each row's group of threads, which wait for no other row; the gradient one to
// the block, whose rows are one copy. Both ways measured: forward 16384 x 1024 bf16 with a residual 25.1 us and
// 28, gradient 32768 x 2048 98 us and 89, before its sums joined at once (DRAM is read in pieces of 4 KB and 16).
constexpr int kRingThreads = 512;         // threads of a block; one block to an SM
constexpr int kMaxStages = 6;
constexpr int kRingBytes = 180 * 1024;
constexpr int kRingSmem = 200 * 1024;     // two stages of three rows of 32 KB

__device__ __forceinline__ void bulk_load(uint32_t dst, const void* src, uint32_t bytes, uint64_t* bar) {
    asm volatile("cp.async.bulk.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(dst), "l"(src), "r"(bytes), "r"(tc::smem_u32(bar)) : "memory");
}

struct RingArgs {
    int stages, array_bytes, arrays, per;
    int* err;
};

// Arrays are named at each call, so that they stay in constant memory.
template <typename T>
struct Ring {
    uint8_t* base;            // the stages
    uint64_t* full;           // and their barriers
    int tile, step, tiles;    // tiles of `per` rows: the current one, to the next, all
    int row_bytes, stage;
    uint32_t phase;
    bool ok, lead;

    // By all threads, before the first global access: `rings` to a block, this one `own`, filled by thread `lead_`.
    __device__ __forceinline__ void init(const RingArgs& a, int T_, int d, int rings, int own, bool lead_, uint8_t* smem,
                                         uint64_t* bars) {
        row_bytes = d * (int)sizeof(T);
        tiles = (T_ + a.per - 1) / a.per;
        tile = blockIdx.x * rings + own;
        step = gridDim.x * rings;
        base = smem + (size_t)own * a.stages * a.arrays * a.array_bytes;
        full = bars + own * kMaxStages;
        stage = 0;
        phase = 0;
        ok = true;
        lead = lead_;
        if (lead) {
            for (int i = 0; i < a.stages; ++i) tc::mbar_init(full + i, 1);
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
        }
        __syncthreads();
    }
    __device__ __forceinline__ void tail(const char* src, uint32_t dst, int64_t from, int64_t upto, int64_t end) {
        for (int64_t q = upto; q < end; q += sizeof(T)) {
            if constexpr (sizeof(T) == 2)
                asm volatile("st.shared.b16 [%0], %1;" ::"r"(dst + (uint32_t)(q - from)),
                             "h"(*reinterpret_cast<const uint16_t*>(src + q)) : "memory");
            else
                asm volatile("st.shared.b32 [%0], %1;" ::"r"(dst + (uint32_t)(q - from)),
                             "r"(*reinterpret_cast<const uint32_t*>(src + q)) : "memory");
        }
    }
    // Tile `t` into stage `to`, by the leading thread.
    __device__ __forceinline__ void fill(const RingArgs& a, int T_, const void* p0, const void* p1, const void* p2, int t, int to) {
        const int64_t all = (int64_t)T_ * row_bytes, begin = (int64_t)t * a.per * row_bytes, from = begin & ~(int64_t)15;
        const int64_t end = min(begin + (int64_t)a.per * row_bytes, all);
        const int64_t upto = min((end + 15) & ~(int64_t)15, all & ~(int64_t)15);    // not past the array
        const uint32_t bytes = (uint32_t)(upto - from);
        const uint32_t dst = tc::smem_u32(base) + (uint32_t)(to * a.arrays * a.array_bytes);
        const char *src0 = static_cast<const char*>(p0), *src1 = static_cast<const char*>(p1), *src2 = static_cast<const char*>(p2);
        if (upto < end) {
            tail(src0, dst, from, upto, end);
            if (a.arrays > 1) tail(src1, dst + a.array_bytes, from, upto, end);
            if (a.arrays > 2) tail(src2, dst + 2 * a.array_bytes, from, upto, end);
        }
        // (the arrive makes the bytes stored above visible to whom waits)
        tc::mbar_expect_tx(full + to, bytes * a.arrays);
        if (bytes) {
            bulk_load(dst, src0 + from, bytes, full + to);
            if (a.arrays > 1) bulk_load(dst + a.array_bytes, src1 + from, bytes, full + to);
            if (a.arrays > 2) bulk_load(dst + 2 * a.array_bytes, src2 + from, bytes, full + to);
        }
    }
    __device__ __forceinline__ void start(const RingArgs& a, int T_, const void* p0, const void* p1, const void* p2) {
        if (lead)
            for (int i = 0; i < a.stages; ++i)
                if (tile + i * step < tiles) fill(a, T_, p0, p1, p2, tile + i * step, i);
    }
    // The tile's first row in the first array (the others array_bytes apart), once it is there.
    __device__ __forceinline__ const uint8_t* wait(const RingArgs& a) {
        if (ok) ok = tc::mbar_wait(full + stage, phase, a.err);
        return base + stage * a.arrays * a.array_bytes + (((uint32_t)tile * (uint32_t)a.per * (uint32_t)row_bytes) & 15u);
    }
    // All of the ring's threads have read the stage (and met since): it is filled again.
    __device__ __forceinline__ void refill(const RingArgs& a, int T_, const void* p0, const void* p1, const void* p2) {
        if (lead && ok && tile + a.stages * step < tiles) {
            asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
            fill(a, T_, p0, p1, p2, tile + a.stages * step, stage);
        }
    }
    __device__ __forceinline__ void next(const RingArgs& a) {
        tile += step;
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    // After the last tile: no copy may be in flight when the block leaves.
    __device__ __forceinline__ void finish(const RingArgs& a) {
        if (!ok && lead)
            for (int i = 0; i < a.stages; ++i) tc::mbar_wait(full + i, phase, a.err);
    }
};

struct NormArgs {
    const void* x;
    const void* r;
    const void* gain;
    const void* bias;
    void* total;
    void* y;
    float* mean;
    float* rstd;
    int T, d, tpr;
    bool p32;
    float eps, inv_d;
};

// A row to `tpr` threads, in registers between the reading and the writing: the mean, then the squares
// of the differences, then the output; gain and bias stay in registers from row to row. Bound by memory.
constexpr int kMaxRow = kRingThreads;      // threads to a row at most
template <typename T, int VE, int NE, bool FULL, bool RES, bool SHORT>
__global__ void __launch_bounds__(kRingThreads, 1) norm_kernel(const NormArgs a, const RingArgs ra) {
    using P = Part<T, VE, NE, FULL>;
    constexpr int NP = NE / 2;
    __shared__ float s_red[2][kRingThreads / 32];
    __shared__ uint64_t s_full[kRingThreads / 32 * kMaxStages];
    extern __shared__ __align__(128) uint8_t s_ring[];
    // SHORT: a warp takes 32 / tpr rows at once, from one ring
    const int unit = SHORT ? 32 : a.tpr, own = threadIdx.x / unit, in = threadIdx.x - own * unit, nvec = a.d / VE;
    const int lane = SHORT ? in & (a.tpr - 1) : in, sub = SHORT ? in / a.tpr : 0, rows = SHORT ? 32 / a.tpr : 1;
    Ring<T> ring;
    ring.init(ra, a.T, a.d, kRingThreads / unit, own, in == 0, s_ring, s_full);
    pdl_wait();
    ring.start(ra, a.T, a.x, a.r, nullptr);
    uint64_t gain[NP], bias[NP];
    P::params(a.gain, a.p32, 1.f, lane, a.tpr, nvec, gain);
    P::params(a.bias, a.p32, 0.f, lane, a.tpr, nvec, bias);
    for (; ring.tile < ring.tiles; ring.next(ra)) {
        const uint8_t* at = ring.wait(ra);
        const int t0 = ring.tile * ra.per, t1 = min(t0 + ra.per, a.T);
        at += sub * ring.row_bytes;
        for (int first = t0; first < t1; first += rows, at += rows * ring.row_bytes) {
            const int t = first + sub;
            const bool live = !SHORT || t < t1;
            uint64_t v[NP];
            P part;
            part.load(reinterpret_cast<const T*>(at), lane, a.tpr, nvec, live);
            part.pairs(v);
            if (RES) {
                uint64_t w[NP];
                part.load(reinterpret_cast<const T*>(at + ra.array_bytes), lane, a.tpr, nvec, live);
                part.pairs(w);
#pragma unroll
                for (int i = 0; i < NP; ++i) v[i] = add2(v[i], w[i]);
            }
            const float mean = row_sum<SHORT>(pair_sum(v), a.tpr, own, s_red[0]) * a.inv_d;
            if (first + rows >= t1) ring.refill(ra, a.T, a.x, a.r, nullptr);
            if (RES && live) P::store(static_cast<T*>(a.total) + (int64_t)t * a.d, lane, a.tpr, nvec, v);
            uint64_t sq[NP];
#pragma unroll
            for (int i = 0; i < NP; ++i) v[i] = add2(v[i], splat2(-mean));
            P::cut(lane, a.tpr, nvec, v);
#pragma unroll
            for (int i = 0; i < NP; ++i) sq[i] = mul2(v[i], v[i]);
            const float var = row_sum<SHORT>(pair_sum(sq), a.tpr, own, s_red[1]) * a.inv_d;
            const float rstd = 1.0f / sqrtf(var + a.eps);
#pragma unroll
            for (int i = 0; i < NP; ++i) v[i] = fma2(mul2(v[i], splat2(rstd)), gain[i], bias[i]);
            if (live) P::store(static_cast<T*>(a.y) + (int64_t)t * a.d, lane, a.tpr, nvec, v);
            if (lane == 0 && live) {
                if (a.mean) a.mean[t] = mean;
                if (a.rstd) a.rstd[t] = rstd;
            }
        }
    }
    ring.finish(ra);
}

// Rows too long for registers: a block to a row, three passes over it (the later ones from L2).
constexpr int kLong = 1024;
template <typename T, int VE>
__global__ void __launch_bounds__(kLong) norm_long_kernel(const NormArgs a) {
    __shared__ float s_red[2][32];
    pdl_wait();
    const int nvec = a.d / VE;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const T* x = static_cast<const T*>(a.x) + t * a.d;
        const T* r = a.r ? static_cast<const T*>(a.r) + t * a.d : nullptr;
        auto element = [&](int c, float (&v)[VE]) {
            Chunk<T, VE> u;
            u.load(x + (int64_t)c * VE);
            u.get(v);
            if (r) {
                float q[VE];
                u.load(r + (int64_t)c * VE);
                u.get(q);
#pragma unroll
                for (int k = 0; k < VE; ++k) v[k] += q[k];
            }
        };
        float sum = 0.f, v[VE];
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            element(c, v);
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < VE; ++k) part += v[k];
            sum += part;
        }
        const float mean = row_sum(sum, kLong, 0, s_red[0]) * a.inv_d;
        float sq = 0.f;
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            element(c, v);
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < VE; ++k) part = fmaf(v[k] - mean, v[k] - mean, part);
            sq += part;
        }
        const float var = row_sum(sq, kLong, 0, s_red[1]) * a.inv_d;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            element(c, v);                    // read before y or total, which may be x or r, is written
            if (r) Chunk<T, VE>::store(static_cast<T*>(a.total) + t * a.d + (int64_t)c * VE, v);
            float g[VE], b[VE];
            load_params<VE>(a.gain, a.p32, c * VE, 1.f, g);
            load_params<VE>(a.bias, a.p32, c * VE, 0.f, b);
#pragma unroll
            for (int k = 0; k < VE; ++k) v[k] = fmaf((v[k] - mean) * rstd, g[k], b[k]);
            Chunk<T, VE>::store(static_cast<T*>(a.y) + t * a.d + (int64_t)c * VE, v);
        }
        if (threadIdx.x == 0) {
            if (a.mean) a.mean[t] = mean;
            if (a.rstd) a.rstd[t] = rstd;
        }
    }
}

// ---------------------------------------------------------------- gradient
struct NormGradArgs {
    const void* dy;
    const void* s;
    const void* gain;
    const float* mean;
    const float* rstd;
    const void* dtotal;
    void* dx;
    float* part;      // [2, blocks, d] sums of dy h and of dy over the block's rows, or null
    int T, d, tpr;
    bool p32;
    float inv_d;
    int stages, array_bytes;   // of the ring: a stage holds 2 arrays, or 3 with dtotal
    int* err;
};

// A row to `tpr` threads, as in the forward pass. A thread keeps its columns from row to row, so it adds
// up dgain and dbias in registers; a block's rows join in shared memory at the end. One block to an SM: its
// partial sums are what the joining kernel reads.
//
// Bound by memory, with registers full of sums. Rows come through one ring to the block, as in Ring, but written
// out: through that struct this kernel took 95 us where it took 89 (32768 x 2048 bf16).
template <typename T, int VE, int NE, bool FULL, bool SHORT>
__global__ void __launch_bounds__(kRingThreads, 1) norm_grad_kernel(const NormGradArgs a) {
    using P = Part<T, VE, NE, FULL>;
    constexpr int NP = NE / 2;
    __shared__ float2 s_red[2][kRingThreads / 32];
    __shared__ uint64_t s_full[kMaxStages], s_empty[kMaxStages];
    extern __shared__ __align__(128) uint8_t s_ring[];
    const int own = threadIdx.x / a.tpr, lane = threadIdx.x - own * a.tpr, rows = kRingThreads / a.tpr, nvec = a.d / VE;
    const int arrays = a.dtotal && a.dx ? 3 : 2;
    if (threadIdx.x == 0) {
        for (int i = 0; i < a.stages; ++i) {
            tc::mbar_init(s_full + i, 1);
            tc::mbar_init(s_empty + i, kRingThreads / 32);
        }
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    __syncthreads();
    pdl_wait();
    const int64_t row_bytes = (int64_t)a.d * sizeof(T);
    const int64_t sets = ((int64_t)a.T + rows - 1) / rows;
    // Set `set` (rows set * rows on) into a stage; where its bytes start in the stage's arrays.
    auto first_byte = [&](int64_t set) { return set * rows * row_bytes; };
    auto fill = [&](int64_t set, int stage) {
        const int64_t all = (int64_t)a.T * row_bytes, from = first_byte(set) & ~(int64_t)15;
        const int64_t end = min((set + 1) * rows * row_bytes, all);
        const int64_t upto = min((end + 15) & ~(int64_t)15, all & ~(int64_t)15);    // not past the array
        const uint32_t bytes = (uint32_t)(upto - from);
        const char* src[3] = {static_cast<const char*>(a.dy), static_cast<const char*>(a.s), static_cast<const char*>(a.dtotal)};
        uint8_t* dst = s_ring + (size_t)stage * arrays * a.array_bytes;
        for (int i = 0; i < arrays; ++i)
            for (int64_t q = upto; q < end; q += sizeof(T))
                *reinterpret_cast<T*>(dst + i * a.array_bytes + (q - from)) = *reinterpret_cast<const T*>(src[i] + q);
        // (the arrive makes the bytes stored above visible to whom waits)
        tc::mbar_expect_tx(s_full + stage, bytes * arrays);
        if (bytes)
            for (int i = 0; i < arrays; ++i)
                bulk_load(tc::smem_u32(dst + i * a.array_bytes), src[i] + from, bytes, s_full + stage);
    };
    uint64_t gain[NP], dg[NP], db[NP];
    P::params(a.gain, a.p32, 1.f, lane, a.tpr, nvec, gain);
#pragma unroll
    for (int i = 0; i < NP; ++i) dg[i] = db[i] = 0;
    if (threadIdx.x == 0)
        for (int i = 0; i < a.stages; ++i)
            if (blockIdx.x + (int64_t)i * gridDim.x < sets) fill(blockIdx.x + (int64_t)i * gridDim.x, i);
    int flip = 0, stage = 0;
    uint32_t phase = 0;
    bool ok = true;
    float mean = 0.f, rstd = 0.f;
    if ((int64_t)blockIdx.x * rows + own < a.T) {
        mean = __ldg(a.mean + (int64_t)blockIdx.x * rows + own);
        rstd = __ldg(a.rstd + (int64_t)blockIdx.x * rows + own);
    }
    for (int64_t set = blockIdx.x; set < sets; set += gridDim.x) {
        const int64_t t = set * rows + own;
        const bool live = t < a.T;
        if (ok) ok = tc::mbar_wait(s_full + stage, phase, a.err);
        const uint8_t* at = s_ring + (size_t)stage * arrays * a.array_bytes + (first_byte(set) & 15) + own * row_bytes;
        uint64_t g[NP], h[NP];
        {
            P py, ps;
            py.load(reinterpret_cast<const T*>(at), lane, a.tpr, nvec, live);
            ps.load(reinterpret_cast<const T*>(at + a.array_bytes), lane, a.tpr, nvec, live);
            py.pairs(g);
            ps.pairs(h);
        }
        const float rs = rstd;
        const uint64_t off = splat2(-mean);
        const int64_t next = t + (int64_t)gridDim.x * rows;
        if (next < a.T) {
            mean = __ldg(a.mean + next);
            rstd = __ldg(a.rstd + next);
        }
#pragma unroll
        for (int i = 0; i < NP; ++i) h[i] = mul2(add2(h[i], off), splat2(rs));
        P::cut(lane, a.tpr, nvec, h);
        if (!live) {
#pragma unroll
            for (int i = 0; i < NP; ++i) h[i] = 0;      // (g is zero)
        }
        uint64_t s1 = 0, s2 = 0;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            dg[i] = fma2(g[i], h[i], dg[i]);
            db[i] = add2(db[i], g[i]);
            g[i] = mul2(g[i], gain[i]);
            s1 = add2(s1, g[i]);
            s2 = fma2(g[i], h[i], s2);
        }
        if (a.dx) {
            float2 lo, hi;
            upk2(s1, lo.x, hi.x);
            upk2(s2, lo.y, hi.y);
            const float2 all = row_sum2<SHORT>(make_float2(lo.x + hi.x, lo.y + hi.y), a.tpr, own, s_red[flip]);
            flip ^= 1;
            const uint64_t c1 = splat2(-all.x * a.inv_d), c2 = splat2(-all.y * a.inv_d);
#pragma unroll
            for (int i = 0; i < NP; ++i) g[i] = mul2(splat2(rs), add2(g[i], fma2(h[i], c2, c1)));
            if (arrays == 3) {
                P pt;
                uint64_t q[NP];
                pt.load(reinterpret_cast<const T*>(at + 2 * a.array_bytes), lane, a.tpr, nvec, live);
                pt.pairs(q);
#pragma unroll
                for (int i = 0; i < NP; ++i) g[i] = add2(g[i], q[i]);
            }
        }
        // the stage is read: thread 0 fills it again when all warps say so
        __syncwarp();
        if ((threadIdx.x & 31) == 0) tc::mbar_arrive(s_empty + stage);
        if (a.dx && live) P::store(static_cast<T*>(a.dx) + t * a.d, lane, a.tpr, nvec, g);
        if (threadIdx.x == 0 && ok) {
            const int64_t more = set + (int64_t)a.stages * gridDim.x;
            if (more < sets) {
                ok = tc::mbar_wait(s_empty + stage, phase, a.err);
                if (ok) {
                    asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
                    fill(more, stage);
                }
            }
        }
        if (++stage == a.stages) {
            stage = 0;
            phase ^= 1;
        }
    }
    if (!ok && threadIdx.x == 0)      // no copy may be in flight when the block leaves
        for (int i = 0; i < a.stages; ++i) tc::mbar_wait(s_full + i, phase, a.err);
    if (!a.part) return;
    // the block's rows join in their order, through the ring's memory [2, rows, d] (one after another, with a
    // wait for each: 32768 x 2048 bf16 89.1 us, so 84.8; 2047 x 1023 fp32 13.7 us, so 11.8)
    float* s_part = reinterpret_cast<float*>(s_ring);
    __syncthreads();
#pragma unroll
    for (int which = 0; which < 2; ++which) {
        float* out = rows > 1 ? s_part + (which * rows + own) * a.d : a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.d;
#pragma unroll
        for (int i = 0; i < NP; ++i) {
            float f[2];
            upk2(which ? db[i] : dg[i], f[0], f[1]);
            const int at = lane + 2 * i / VE * a.tpr, c = at * VE + 2 * i % VE;
            if constexpr (VE > 1) {
                if (FULL || at < nvec) *reinterpret_cast<float2*>(out + c) = make_float2(f[0], f[1]);
            } else {
                if (FULL || at < nvec) out[c] = f[0];
                if (FULL || at + a.tpr < nvec) out[c + a.tpr] = f[1];
            }
        }
    }
    if (rows == 1) return;
    __syncthreads();
    for (int i = threadIdx.x; i < 2 * a.d; i += kRingThreads) {
        const int which = i >= a.d, c = i - which * a.d;
        const float* in = s_part + which * rows * a.d + c;
        float f = in[0];
        for (int q = 1; q < rows; ++q) f += in[q * a.d];
        a.part[((size_t)which * gridDim.x + blockIdx.x) * a.d + c] = f;
    }
}

// Long rows: dx by a block to a row in two passes; dgain and dbias by norm_columns_kernel.
template <typename T, int VE>
__global__ void __launch_bounds__(kLong) norm_grad_long_kernel(const NormGradArgs a) {
    __shared__ float2 s_red[2][32];
    pdl_wait();
    const int nvec = a.d / VE;
    int flip = 0;
    for (int64_t t = blockIdx.x; t < a.T; t += gridDim.x) {
        const int64_t base = t * a.d;
        const float mean = __ldg(a.mean + t), rstd = __ldg(a.rstd + t);
        auto element = [&](int c, float (&g)[VE], float (&h)[VE]) {
            Chunk<T, VE> u;
            float w[VE];
            u.load(static_cast<const T*>(a.dy) + base + (int64_t)c * VE);
            u.get(g);
            u.load(static_cast<const T*>(a.s) + base + (int64_t)c * VE);
            u.get(h);
            load_params<VE>(a.gain, a.p32, c * VE, 1.f, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                g[k] *= w[k];
                h[k] = (h[k] - mean) * rstd;
            }
        };
        float g[VE], h[VE];
        float2 sum = make_float2(0.f, 0.f);
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            element(c, g, h);
            float2 part = make_float2(0.f, 0.f);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                part.x += g[k];
                part.y = fmaf(g[k], h[k], part.y);
            }
            sum.x += part.x;
            sum.y += part.y;
        }
        const float2 all = row_sum2(sum, kLong, 0, s_red[flip]);
        flip ^= 1;
        const float c1 = all.x * a.inv_d, c2 = all.y * a.inv_d;
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            float q[VE];
            element(c, g, h);
            Chunk<T, VE> u;
            u.zero();
            if (a.dtotal) u.load(static_cast<const T*>(a.dtotal) + base + (int64_t)c * VE);
            u.get(q);
#pragma unroll
            for (int k = 0; k < VE; ++k) q[k] = fmaf(rstd, g[k] - fmaf(h[k], c2, c1), q[k]);
            Chunk<T, VE>::store(static_cast<T*>(a.dx) + base + (int64_t)c * VE, q);
        }
    }
}

// Partial sums of dy h and dy over a slice of the rows, a thread to VE columns (long rows: runs before
// dx is written, which may replace dy or s).
template <typename T, int VE>
__global__ void __launch_bounds__(256) norm_columns_kernel(const NormGradArgs a) {
    pdl_wait();
    const int c = blockIdx.x * 256 + threadIdx.x, nvec = a.d / VE;
    if (c >= nvec) return;
    float dg[VE], db[VE];
#pragma unroll
    for (int k = 0; k < VE; ++k) dg[k] = db[k] = 0.f;
    for (int64_t t = blockIdx.y; t < a.T; t += gridDim.y) {
        Chunk<T, VE> u;
        float g[VE], h[VE];
        u.load(static_cast<const T*>(a.dy) + t * a.d + (int64_t)c * VE);
        u.get(g);
        u.load(static_cast<const T*>(a.s) + t * a.d + (int64_t)c * VE);
        u.get(h);
        const float mean = __ldg(a.mean + t), rstd = __ldg(a.rstd + t);
#pragma unroll
        for (int k = 0; k < VE; ++k) {
            dg[k] = fmaf(g[k], (h[k] - mean) * rstd, dg[k]);
            db[k] += g[k];
        }
    }
    float* out = a.part + (size_t)blockIdx.y * a.d + (int64_t)c * VE;
#pragma unroll
    for (int k = 0; k < VE; ++k) {
        out[k] = dg[k];
        out[(size_t)gridDim.y * a.d + k] = db[k];
    }
}

// dgain and dbias from the blocks' sums: 32 columns to a block, its 32 warps take every 32nd partial row,
// then join in order.
constexpr int kJoinWarps = 32;
__global__ void __launch_bounds__(32 * kJoinWarps) norm_join_kernel(const float* __restrict__ part, int blocks, int d,
                                                                   int accumulate, float* dgain, float* dbias) {
    __shared__ float s_sum[kJoinWarps][32];
    pdl_wait();
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31, c = blockIdx.x * 32 + lane;
    float* out = blockIdx.y ? dbias : dgain;
    if (!out) return;
    const float* in = part + (size_t)blockIdx.y * blocks * d;
    float v = 0.f;
    if (c < d) {
#pragma unroll 8
        for (int b = warp; b < blocks; b += kJoinWarps) v += in[(size_t)b * d + c];
    }
    s_sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d) {
#pragma unroll
        for (int w = 1; w < kJoinWarps; ++w) v += s_sum[w][lane];
        out[c] = accumulate ? out[c] + v : v;
    }
}

// ---------------------------------------------------------------- host
moe_status_t check_norm(const moe_norm_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->T < 0 || c->d < 1 || !std::isfinite(c->eps) || c->eps < 0.f || (c->accumulate != 0 && c->accumulate != 1))
        return MOE_ERR_INVALID_ARG;
    if ((c->dtype != MOE_F32 && c->dtype != MOE_BF16) || (c->param_dtype != MOE_F32 && c->param_dtype != MOE_BF16))
        return MOE_ERR_INVALID_ARG;
    if (c->T > (1 << 30) || c->d > (1 << 20)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

// How a row is shared out: vector, threads to a row and bytes of it to a thread (16, 32 or 64; 0: too long
// for registers). 32 bytes to a thread, and the next row's 32 in flight, keep the registers of a block of 512
// threads; below 256 elements a warp takes 16 or 32 bytes a lane, rows of up to 256 bytes several to a warp (409600
// rows of 64 bf16 101 us, so 38, the gradient 148 and 91), and beyond 512 threads 64 of fp32. Measured with
// 16, 32 and 64 bytes to a thread: forward, 16384 rows of 1024 bf16 with a residual, 38, 25 and 41 us; the gradient
// of 32768 rows of 2048 bf16 123, 89 and 267 us; of 2047 rows of 1023 fp32 13.0, 13.7 and 21.2 us. 64 bytes of bf16
// are 32 elements, which spill: 3198 rows of 8195 forward 152 us and by the kernels for long rows 89, gradient 304
// and 133, 1600 rows of 16384 64 and 58, 95 and 97.
// The forward pass takes rows of single elements (odd ones) 8 to a thread at most: 16 spill, too (25625 rows of
// 1023 bf16 101 us, so 72; 3200 rows of 8191 fp32 121, long rows 93).
struct Shape {
    int ve, tpr, bytes;
};
Shape norm_shape(const moe_norm_config_t& c, bool grad) {
    Shape s;
    const int es = c.dtype == MOE_BF16 ? 2 : 4;
    const int64_t row = (int64_t)c.d * es;
    s.ve = row_vec(c.d, es);
    const bool few = s.ve == 1 && !grad;
    const int each = few ? 8 * es : 32, most = es == 2 || few ? each : 64;
    s.tpr = row <= 256 ? 4 : 32;
    if (s.tpr < 32) {
        while (s.tpr * 16 < row) s.tpr *= 2;
    } else {
        while (s.tpr < kMaxRow && s.tpr * each < row) s.tpr *= 2;
    }
    s.bytes = row <= s.tpr * 16 ? 16 : row <= s.tpr * 32 ? 32 : row <= s.tpr * 64 ? 64 : 0;
    if (s.bytes > most) s.bytes = 0;
    return s;
}

// The forward pass: adjacent rows to a copy, 2 KB of short ones, but not so many that groups of threads have none.
int rows_per_copy(const moe_norm_config_t& c, const Shape& sh) {
    const int row = c.d * (c.dtype == MOE_BF16 ? 2 : 4), groups = num_sms() * (kRingThreads / std::max(32, sh.tpr));
    return std::max(1, std::min(2048 / row, c.T / groups));
}

template <typename T, int VE, int NE, bool FULL>
cudaError_t launch_norm_ne(const moe_norm_config_t& c, const NormArgs& a, const Shape& sh, cudaStream_t s) {
    // as many stages as fit (2 at least)
    const int groups = kRingThreads / std::max(32, sh.tpr);
    RingArgs r;
    r.arrays = a.r ? 2 : 1;
    r.per = rows_per_copy(c, sh);
    r.array_bytes = (int)align_up((size_t)r.per * c.d * sizeof(T) + 32, 128);
    r.stages = std::max(2, std::min(kMaxStages, kRingBytes / (groups * r.arrays * r.array_bytes)));
    r.err = device_error_word();
    const size_t bytes = (size_t)groups * r.stages * r.arrays * r.array_bytes;
    const int blocks = std::min(ceil_div(ceil_div(c.T, r.per), groups), num_sms());
    auto kern = a.r ? norm_kernel<T, VE, NE, FULL, true, false> : norm_kernel<T, VE, NE, FULL, false, false>;
    if constexpr (NE * sizeof(T) == 16)
        if (sh.tpr < 32) kern = a.r ? norm_kernel<T, VE, NE, FULL, true, true> : norm_kernel<T, VE, NE, FULL, false, true>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (e != cudaSuccess) return e;
    return launch_pdl(kern, dim3(blocks), dim3(kRingThreads), bytes, s, a, r);
}

template <typename T, int VE>
cudaError_t launch_norm(const moe_norm_config_t& c, NormArgs a, const Shape& sh, cudaStream_t s) {
    constexpr int ES = (int)sizeof(T);
    a.tpr = sh.tpr;
    cudaError_t e = cudaErrorInvalidValue;
    constexpr bool WIDE = VE * ES == 16;      // (rows of other vectors are never taken as whole)
    const bool full = WIDE && (int64_t)c.d * ES == (int64_t)sh.tpr * sh.bytes;
    if (sh.bytes == 0) e = launch_pdl(norm_long_kernel<T, VE>, dim3(std::min(c.T, num_sms() * 2)), dim3(kLong), 0, s, a);
    else if (sh.bytes == 16) e = full ? launch_norm_ne<T, VE, 16 / ES, WIDE>(c, a, sh, s) : launch_norm_ne<T, VE, 16 / ES, false>(c, a, sh, s);
    if constexpr (VE > 1 || ES == 4)
        if (sh.bytes == 32) e = full ? launch_norm_ne<T, VE, 32 / ES, WIDE>(c, a, sh, s) : launch_norm_ne<T, VE, 32 / ES, false>(c, a, sh, s);
    if constexpr (VE > 1 && ES == 4)
        if (sh.bytes == 64) e = full ? launch_norm_ne<T, VE, 64 / ES, WIDE>(c, a, sh, s) : launch_norm_ne<T, VE, 64 / ES, false>(c, a, sh, s);
    count_launch();
    return e;
}

// Blocks whose partial sums norm_join_kernel adds up; for long rows slices of the rows, four blocks to an SM in all
// (16 slices: 2133 rows of 12288 fp32 172 us, so 137).
int grad_blocks(const moe_norm_config_t& c, const Shape& sh) {
    const int slices = std::max(1, num_sms() * 4 / ceil_div(c.d / sh.ve, 256));
    return std::max(1, sh.bytes == 0 ? std::min(c.T, slices) : std::min(ceil_div(c.T, kRingThreads / sh.tpr), num_sms()));
}

template <typename T, int VE, int NE, bool FULL>
cudaError_t launch_grad_ne(const moe_norm_config_t& c, const NormGradArgs& a, const Shape& sh, cudaStream_t s) {
    auto kern = norm_grad_kernel<T, VE, NE, FULL, false>;
    if constexpr (NE * sizeof(T) == 16)
        if (sh.tpr < 32) kern = norm_grad_kernel<T, VE, NE, FULL, true>;
    const cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, kRingSmem);
    if (e != cudaSuccess) return e;
    const size_t ring = (size_t)a.stages * (a.dtotal && a.dx ? 3 : 2) * a.array_bytes;
    const size_t sums = 2 * (size_t)(kRingThreads / sh.tpr) * c.d * sizeof(float);
    return launch_pdl(kern, dim3(grad_blocks(c, sh)), dim3(kRingThreads), std::max(ring, sums), s, a);
}

template <typename T, int VE>
cudaError_t launch_norm_grad(const moe_norm_config_t& c, NormGradArgs a, const Shape& sh, cudaStream_t s) {
    constexpr int ES = (int)sizeof(T);
    a.tpr = sh.tpr;
    // the rows that a block works on at once with what a copy takes in beside them, and as many stages as fit (2
    // at least: rows are 32 KB at most, arrays 3)
    a.array_bytes = (int)align_up((size_t)(kRingThreads / sh.tpr) * c.d * ES + 32, 128);
    a.stages = std::max(2, std::min(kMaxStages, kRingBytes / ((a.dtotal && a.dx ? 3 : 2) * a.array_bytes)));
    a.err = device_error_word();
    cudaError_t e = cudaSuccess;
    if (sh.bytes == 0) {
        if (a.part) {
            const int blocks = grad_blocks(c, sh);
            e = launch_pdl(norm_columns_kernel<T, VE>, dim3(ceil_div(c.d / VE, 256), blocks), dim3(256), 0, s, a);
            count_launch();
        }
        if (e == cudaSuccess && a.dx) {
            e = launch_pdl(norm_grad_long_kernel<T, VE>, dim3(std::min(c.T, num_sms() * 2)), dim3(kLong), 0, s, a);
            count_launch();
        }
        return e;
    }
    constexpr bool WIDE = VE * ES == 16;      // (rows of other vectors are never taken as whole)
    const bool full = WIDE && (int64_t)c.d * ES == (int64_t)sh.tpr * sh.bytes;
    if (sh.bytes == 16) e = full ? launch_grad_ne<T, VE, 16 / ES, WIDE>(c, a, sh, s) : launch_grad_ne<T, VE, 16 / ES, false>(c, a, sh, s);
    else if (sh.bytes == 32) e = full ? launch_grad_ne<T, VE, 32 / ES, WIDE>(c, a, sh, s) : launch_grad_ne<T, VE, 32 / ES, false>(c, a, sh, s);
    if constexpr (ES == 4)
        if (sh.bytes == 64) e = full ? launch_grad_ne<T, VE, 64 / ES, WIDE>(c, a, sh, s) : launch_grad_ne<T, VE, 64 / ES, false>(c, a, sh, s);
    count_launch();
    return e;
}

}  // namespace

}  // namespace moe

using namespace moe;

#define MOE_NORM_VE(T, fn, ...)                                               \
    (sh.ve == 16 / (int)sizeof(T) ? fn<T, 16 / (int)sizeof(T)>(__VA_ARGS__)   \
     : sh.ve == 2                 ? fn<T, 2>(__VA_ARGS__)                     \
     : sh.ve == 4                 ? fn<T, 4>(__VA_ARGS__)                     \
                                  : fn<T, 1>(__VA_ARGS__))

extern "C" MOE_API moe_status_t moe_layer_norm(const moe_norm_config_t* cfg, const void* x, const void* residual,
                                               const void* gain, const void* bias, void* total, void* y, float* mean,
                                               float* rstd, moe_stream_t stream) {
    const moe_status_t st = check_norm(cfg);
    if (st != MOE_OK) return st;
    const moe_norm_config_t& c = *cfg;
    if ((residual != nullptr) != (total != nullptr) || (c.T > 0 && (!x || !y))) return MOE_ERR_INVALID_ARG;
    for (const void* p : {x, residual, gain, bias, (const void*)total, (const void*)y})
        if (misaligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (misaligned(mean, 4) || misaligned(rstd, 4)) return MOE_ERR_INVALID_ARG;
    if (total && total == y) return MOE_ERR_INVALID_ARG;
    if (c.T == 0) return MOE_OK;
    const Shape sh = norm_shape(c, false);
    const NormArgs a{x, residual, gain, bias, total, y, mean, rstd, c.T, c.d, sh.tpr, c.param_dtype == MOE_F32, c.eps,
                     1.0f / (float)c.d};
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = c.dtype == MOE_BF16 ? MOE_NORM_VE(__nv_bfloat16, launch_norm, c, a, sh, s)
                                              : MOE_NORM_VE(float, launch_norm, c, a, sh, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API size_t moe_norm_workspace_bytes(const moe_norm_config_t* cfg) {
    if (check_norm(cfg) != MOE_OK) return 0;
    return align_up(2 * (size_t)grad_blocks(*cfg, norm_shape(*cfg, true)) * cfg->d * sizeof(float), 256);
}

extern "C" MOE_API moe_status_t moe_layer_norm_backward(const moe_norm_config_t* cfg, const void* dy, const void* x,
                                                        const void* gain, const float* mean, const float* rstd,
                                                        const void* dtotal, void* dx, float* dgain, float* dbias,
                                                        void* ws, moe_stream_t stream) {
    const moe_status_t st = check_norm(cfg);
    if (st != MOE_OK) return st;
    const moe_norm_config_t& c = *cfg;
    const bool sums = dgain || dbias;
    if ((c.T > 0 && (!dy || !x || !mean || !rstd || (!dx && !sums))) || (sums && !ws)) return MOE_ERR_INVALID_ARG;
    for (const void* p : {dy, x, gain, dtotal, (const void*)dx, (const void*)dgain, (const void*)dbias, (const void*)ws})
        if (misaligned(p, 16)) return MOE_ERR_INVALID_ARG;
    if (misaligned(mean, 4) || misaligned(rstd, 4) || (dgain && dgain == dbias)) return MOE_ERR_INVALID_ARG;
    cudaStream_t s = (cudaStream_t)stream;
    if (c.T == 0) {
        if (c.accumulate) return MOE_OK;
        for (float* p : {dgain, dbias})
            if (p && launch_fill(p, (long long)c.d, 0.f, s) != cudaSuccess) return MOE_ERR_CUDA;
        return MOE_OK;
    }
    const Shape sh = norm_shape(c, true);
    const NormGradArgs a{dy, x, gain, mean, rstd, dtotal, dx, sums ? static_cast<float*>(ws) : nullptr, c.T, c.d, sh.tpr,
                         c.param_dtype == MOE_F32, 1.0f / (float)c.d, 0, 0, nullptr};
    cudaError_t e = c.dtype == MOE_BF16 ? MOE_NORM_VE(__nv_bfloat16, launch_norm_grad, c, a, sh, s)
                                        : MOE_NORM_VE(float, launch_norm_grad, c, a, sh, s);
    if (e == cudaSuccess && sums) {
        e = launch_pdl(norm_join_kernel, dim3(ceil_div(c.d, 32), 2), dim3(32 * kJoinWarps), 0, s, (const float*)ws,
                       grad_blocks(c, sh), c.d, c.accumulate, dgain, dbias);
        count_launch();
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
