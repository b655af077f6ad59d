// Layer norm of rows (and of a residual sum), and its gradient.
#include <cmath>

#include "internal.cuh"

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

// Widest vector (elements, up to 16 bytes) that divides rows of d elements of es bytes.
int row_vec(int d, int es) {
    int v = 16 / es;
    while (v > 1 && d % v) v /= 2;
    return v;
}

// Sum over the `tpr` threads of a row (32 or more, a power of two; a block holds whole rows). `red`
// is free again after the next row_sum on another buffer.
__device__ __forceinline__ float row_sum(float v, int tpr, float* red) {
    v = warp_sum(v);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, n = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const float* at = red + warp / n * n;
    float s = at[0];
    for (int i = 1; i < n; ++i) s += at[i];
    return s;
}
__device__ __forceinline__ float2 row_sum2(float2 v, int tpr, float2* red) {
    v.x = warp_sum(v.x);
    v.y = warp_sum(v.y);
    if (tpr == 32) return v;
    const int warp = threadIdx.x >> 5, n = tpr >> 5;
    if ((threadIdx.x & 31) == 0) red[warp] = v;
    __syncthreads();
    const float2* at = red + warp / n * n;
    float2 s = at[0];
    for (int i = 1; i < n; ++i) { s.x += at[i].x; s.y += at[i].y; }
    return s;
}

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
// of the differences, then the output. NV vectors of VE elements a thread.
constexpr int kMaxRow = 512;      // threads to a row at most: 128 registers each
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(kMaxRow) norm_kernel(const NormArgs a) {
    __shared__ float s_red[2][32];
    pdl_wait();
    const int rows = blockDim.x / a.tpr, lane = threadIdx.x & (a.tpr - 1), nvec = a.d / VE;
    const T* x = static_cast<const T*>(a.x);
    const T* r = static_cast<const T*>(a.r);
    for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += (int64_t)gridDim.x * rows) {
        const int64_t t = t0 + threadIdx.x / a.tpr;
        const bool live = t < a.T;
        const int64_t base = t * a.d;
        Chunk<T, VE> cx[NV], cr[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane + i * a.tpr;
            cx[i].zero();
            cr[i].zero();
            if (live && c < nvec) {
                cx[i].load(x + base + (int64_t)c * VE);
                if (r) cr[i].load(r + base + (int64_t)c * VE);
            }
        }
        float v[NV][VE];
        float sum = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            cx[i].get(v[i]);
            if (r) {
                float q[VE];
                cr[i].get(q);
#pragma unroll
                for (int k = 0; k < VE; ++k) v[i][k] += q[k];
                const int c = lane + i * a.tpr;
                if (live && c < nvec) Chunk<T, VE>::store(static_cast<T*>(a.total) + base + (int64_t)c * VE, v[i]);
            }
#pragma unroll
            for (int k = 0; k < VE; ++k) sum += v[i][k];
        }
        const float mean = row_sum(sum, a.tpr, s_red[0]) * a.inv_d;
        float sq = 0.f;
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            if (lane + i * a.tpr < nvec) {
#pragma unroll
                for (int k = 0; k < VE; ++k) {
                    v[i][k] -= mean;
                    sq = fmaf(v[i][k], v[i][k], sq);
                }
            }
        }
        const float var = row_sum(sq, a.tpr, s_red[1]) * a.inv_d;
        const float rstd = 1.0f / sqrtf(var + a.eps);
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = lane + i * a.tpr;
                if (c < nvec) {
                    float g[VE], b[VE];
                    load_params<VE>(a.gain, a.p32, c * VE, 1.f, g);
                    load_params<VE>(a.bias, a.p32, c * VE, 0.f, b);
#pragma unroll
                    for (int k = 0; k < VE; ++k) v[i][k] = fmaf(v[i][k] * rstd, g[k], b[k]);
                    Chunk<T, VE>::store(static_cast<T*>(a.y) + base + (int64_t)c * VE, v[i]);
                }
            }
            if (lane == 0) {
                if (a.mean) a.mean[t] = mean;
                if (a.rstd) a.rstd[t] = rstd;
            }
        }
    }
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
        const float mean = row_sum(sum, kLong, s_red[0]) * a.inv_d;
        float sq = 0.f;
        for (int c = threadIdx.x; c < nvec; c += kLong) {
            element(c, v);
            float part = 0.f;
#pragma unroll
            for (int k = 0; k < VE; ++k) part = fmaf(v[k] - mean, v[k] - mean, part);
            sq += part;
        }
        const float var = row_sum(sq, kLong, s_red[1]) * a.inv_d;
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
};

// A row to `tpr` threads, as in the forward pass. A thread keeps its columns from row to row, so it adds
// up dgain and dbias in registers; a block's rows join in shared memory at the end.
template <typename T, int VE, int NV>
__global__ void __launch_bounds__(kMaxRow) norm_grad_kernel(const NormGradArgs a) {
    __shared__ float2 s_red[2][32];
    extern __shared__ float s_part[];     // [d] (blocks of more than one row)
    pdl_wait();
    const int rows = blockDim.x / a.tpr, lane = threadIdx.x & (a.tpr - 1), nvec = a.d / VE;
    const int own = threadIdx.x / a.tpr;
    float dg[NV][VE], db[NV][VE];
#pragma unroll
    for (int i = 0; i < NV; ++i)
#pragma unroll
        for (int k = 0; k < VE; ++k) dg[i][k] = db[i][k] = 0.f;
    int flip = 0;
    for (int64_t t0 = (int64_t)blockIdx.x * rows; t0 < a.T; t0 += (int64_t)gridDim.x * rows) {
        const int64_t t = t0 + own;
        const bool live = t < a.T;
        const int64_t base = t * a.d;
        Chunk<T, VE> cd[NV], cs[NV], ct[NV];
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane + i * a.tpr;
            cd[i].zero();
            cs[i].zero();
            ct[i].zero();
            if (live && c < nvec) {
                cd[i].load(static_cast<const T*>(a.dy) + base + (int64_t)c * VE);
                cs[i].load(static_cast<const T*>(a.s) + base + (int64_t)c * VE);
                if (a.dtotal) ct[i].load(static_cast<const T*>(a.dtotal) + base + (int64_t)c * VE);
            }
        }
        const float mean = live ? __ldg(a.mean + t) : 0.f, rstd = live ? __ldg(a.rstd + t) : 0.f;
        float g[NV][VE], h[NV][VE];
        float2 sum = make_float2(0.f, 0.f);
#pragma unroll
        for (int i = 0; i < NV; ++i) {
            const int c = lane + i * a.tpr;
            float w[VE];
            cd[i].get(g[i]);
            cs[i].get(h[i]);
            if (c < nvec) load_params<VE>(a.gain, a.p32, c * VE, 1.f, w);
#pragma unroll
            for (int k = 0; k < VE; ++k) {
                if (!live || c >= nvec) {
                    g[i][k] = h[i][k] = 0.f;
                    continue;
                }
                h[i][k] = (h[i][k] - mean) * rstd;
                dg[i][k] = fmaf(g[i][k], h[i][k], dg[i][k]);
                db[i][k] += g[i][k];
                g[i][k] *= w[k];
                sum.x += g[i][k];
                sum.y = fmaf(g[i][k], h[i][k], sum.y);
            }
        }
        if (!a.dx) continue;
        const float2 all = row_sum2(sum, a.tpr, s_red[flip]);
        flip ^= 1;
        const float c1 = all.x * a.inv_d, c2 = all.y * a.inv_d;
        if (live) {
#pragma unroll
            for (int i = 0; i < NV; ++i) {
                const int c = lane + i * a.tpr;
                if (c < nvec) {
                    float q[VE];
                    ct[i].get(q);
#pragma unroll
                    for (int k = 0; k < VE; ++k) q[k] = fmaf(rstd, g[i][k] - fmaf(h[i][k], c2, c1), q[k]);
                    Chunk<T, VE>::store(static_cast<T*>(a.dx) + base + (int64_t)c * VE, q);
                }
            }
        }
    }
    if (!a.part) return;
    // the block's rows one after another, dgain then dbias
    for (int which = 0; which < 2; ++which) {
        float* out = a.part + ((size_t)which * gridDim.x + blockIdx.x) * a.d;
        for (int q = 0; q < rows; ++q) {
            if (own == q) {
#pragma unroll
                for (int i = 0; i < NV; ++i) {
                    const int c = lane + i * a.tpr;
                    if (c >= nvec) continue;
#pragma unroll
                    for (int k = 0; k < VE; ++k) {
                        float v = which ? db[i][k] : dg[i][k];
                        if (rows > 1) {
                            if (q > 0) v += s_part[c * VE + k];
                            s_part[c * VE + k] = v;
                        }
                        if (q + 1 == rows) out[c * VE + k] = v;
                    }
                }
            }
            if (rows > 1) __syncthreads();
        }
    }
}

// Long rows: dx by a block to a row in two passes; dgain and dbias by column_kernel.
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
        const float2 all = row_sum2(sum, kLong, s_red[flip]);
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

// dgain and dbias from the blocks' sums: 32 columns to a block, its warps take every eighth partial
// row, then join in order.
constexpr int kJoinWarps = 8;
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
#pragma unroll 4
        for (int b = warp; b < blocks; b += kJoinWarps) v += in[(size_t)b * d + c];
    }
    s_sum[warp][lane] = v;
    __syncthreads();
    if (warp == 0 && c < d) {
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

// How a row is shared out: vector, threads to a row and elements to a thread (8, 16 or 32; 0: too long for
// registers).
struct Shape {
    int ve, tpr, ne, block;
};
Shape norm_shape(const moe_norm_config_t& c) {
    Shape s;
    s.ve = row_vec(c.d, c.dtype == MOE_BF16 ? 2 : 4);
    s.tpr = 32;
    while (s.tpr < kMaxRow && s.tpr * 16 < c.d) s.tpr *= 2;
    s.ne = c.d <= s.tpr * 8 ? 8 : c.d <= s.tpr * 16 ? 16 : c.d <= s.tpr * 32 ? 32 : 0;
    s.block = std::max(s.tpr, 128);
    return s;
}

template <typename T, int VE>
cudaError_t launch_norm(const moe_norm_config_t& c, NormArgs a, const Shape& sh, cudaStream_t s) {
    a.tpr = sh.tpr;
    cudaError_t e;
    if (sh.ne == 0) {
        e = launch_pdl(norm_long_kernel<T, VE>, dim3(std::min(c.T, num_sms() * 2)), dim3(kLong), 0, s, a);
    } else {
        auto kern = sh.ne == 8 ? norm_kernel<T, VE, 8 / VE> : sh.ne == 16 ? norm_kernel<T, VE, 16 / VE>
                                                            : norm_kernel<T, VE, 32 / VE>;
        const int tiles = ceil_div(c.T, sh.block / sh.tpr);
        e = launch_pdl(kern, dim3(std::min(tiles, num_sms() * 64)), dim3(sh.block), 0, s, a);
    }
    count_launch();
    return e;
}

// Blocks whose partial sums norm_join_kernel adds up.
int grad_blocks(const moe_norm_config_t& c, const Shape& sh) {
    if (sh.ne == 0) return std::max(1, std::min(c.T, 16));
    return std::max(1, std::min(ceil_div(c.T, sh.block / sh.tpr), num_sms() * (sh.block >= 512 ? 1 : 512 / sh.block)));
}

template <typename T, int VE>
cudaError_t launch_norm_grad(const moe_norm_config_t& c, NormGradArgs a, const Shape& sh, cudaStream_t s) {
    a.tpr = sh.tpr;
    const int blocks = grad_blocks(c, sh);
    cudaError_t e = cudaSuccess;
    if (sh.ne == 0) {
        if (a.part) {
            e = launch_pdl(norm_columns_kernel<T, VE>, dim3(ceil_div(c.d / VE, 256), blocks), dim3(256), 0, s, a);
            count_launch();
        }
        if (e == cudaSuccess && a.dx) {
            e = launch_pdl(norm_grad_long_kernel<T, VE>, dim3(std::min(c.T, num_sms() * 2)), dim3(kLong), 0, s, a);
            count_launch();
        }
        return e;
    }
    auto kern = sh.ne == 8 ? norm_grad_kernel<T, VE, 8 / VE> : sh.ne == 16 ? norm_grad_kernel<T, VE, 16 / VE>
                                                             : norm_grad_kernel<T, VE, 32 / VE>;
    const size_t smem = sh.block > sh.tpr ? (size_t)c.d * sizeof(float) : 0;
    e = launch_pdl(kern, dim3(blocks), dim3(sh.block), smem, s, a);
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
    const Shape sh = norm_shape(c);
    const NormArgs a{x, residual, gain, bias, total, y, mean, rstd, c.T, c.d, sh.tpr, c.param_dtype == MOE_F32, c.eps,
                     1.0f / (float)c.d};
    cudaStream_t s = (cudaStream_t)stream;
    const cudaError_t e = c.dtype == MOE_BF16 ? MOE_NORM_VE(__nv_bfloat16, launch_norm, c, a, sh, s)
                                              : MOE_NORM_VE(float, launch_norm, c, a, sh, s);
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API size_t moe_norm_workspace_bytes(const moe_norm_config_t* cfg) {
    if (check_norm(cfg) != MOE_OK) return 0;
    return align_up(2 * (size_t)grad_blocks(*cfg, norm_shape(*cfg)) * cfg->d * sizeof(float), 256);
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
    const Shape sh = norm_shape(c);
    const NormGradArgs a{dy, x, gain, mean, rstd, dtotal, dx, sums ? static_cast<float*>(ws) : nullptr, c.T, c.d, sh.tpr,
                         c.param_dtype == MOE_F32, 1.0f / (float)c.d};
    cudaError_t e = c.dtype == MOE_BF16 ? MOE_NORM_VE(__nv_bfloat16, launch_norm_grad, c, a, sh, s)
                                        : MOE_NORM_VE(float, launch_norm_grad, c, a, sh, s);
    if (e == cudaSuccess && sums) {
        e = launch_pdl(norm_join_kernel, dim3(ceil_div(c.d, 32), 2), dim3(32 * kJoinWarps), 0, s, (const float*)ws,
                       grad_blocks(c, sh), c.d, c.accumulate, dgain, dbias);
        count_launch();
    }
    return e == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
