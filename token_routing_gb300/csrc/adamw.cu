// AdamW over many tensors in one launch, with fp32 or 8-bit states.
#include <cuda_fp8.h>

#include <cmath>

#include "internal.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = MOE_ADAMW_BLOCK;     // elements a warp takes at a time: 8 a lane, one scale block
constexpr int kBatch = 256;                // tensors in one launch's parameters

struct TensorArg {
    void* p;
    const void* g;
    float* w;
    void* m;
    void* v;
    float* ms;
    float* vs;
    int64_t n;
    float decay;
    int32_t kind;      // bit 0: p is bf16, bit 1: g is bf16
};

struct AdamArgs {
    double lr, beta1, beta2;
    float eps;
    int count;
    int advance;                       // this launch is the call's last: it counts the step
    const float* lr_dev;
    const float* grad_scale;
    unsigned char* state;
    int64_t units;
    int64_t first[kBatch];             // first unit of each tensor
    TensorArg t[kBatch];
};
static_assert(sizeof(AdamArgs) <= 32000, "kernel parameters");

struct State {
    double c1, c2;                     // 1 - beta^t
    long long step;
    unsigned ticket, pad;
};
static_assert(sizeof(State) == MOE_ADAMW_STATE_BYTES, "state layout");

// Scalars of one step.
struct Step {
    float b1, ob1, b2, ob2;            // betas and 1 - betas
    float keep;                        // 1 - lr * decay
    float rate;                        // -lr / (1 - beta1^t)
    float rc2;                         // 1 / sqrt(1 - beta2^t)
    float eps, gs;
    uint32_t dither;                   // the step's part of the hash
};

template <typename T>
__device__ __forceinline__ void load8(const T* p, int live, float (&f)[8]) {
    if (live == 8) {
        if constexpr (sizeof(T) == 2) {
            load16(p, f);
        } else {
            load16(p, f);
            load16(p + 4, f + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) f[i] = i < live ? ld_f(p + i) : 0.f;
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, int live, const float (&f)[8]) {
    if (live == 8) {
        if constexpr (sizeof(T) == 2) {
            store16(p, f);
        } else {
            store16(p, f);
            store16(p + 4, f + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) st_f(p + i, f[i]);
    }
}

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028235e38f; }

__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

__device__ __forceinline__ void load_codes(const uint8_t* p, int live, float scale, float (&f)[8]) {
    uint16_t b[4];
    if (live == 8) {
        *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            b[i] = (uint16_t)((2 * i < live ? p[2 * i] : 0) | (2 * i + 1 < live ? p[2 * i + 1] : 0) << 8);
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2(b[i], __NV_E4M3));
        const float2 v = __half22float2(h);
        f[2 * i] = v.x * scale;
        f[2 * i + 1] = v.y * scale;
    }
}

// The grid of e4m3 in fp32: three bits after the leading one, a step of 2^-9 below 2^-6. Adding
// 2^-6 to a number below it puts it where the fp32 mantissa has that step too, so that the 20
// low bits of t are the share of the way to the next grid value everywhere.
constexpr float kTiny = 0.015625f;      // 2^-6

// y on the grid, up with the probability of its share of the way: d is the dither, 20 bits.
__device__ __forceinline__ float to_grid(float y, uint32_t d) {
    const float off = copysignf(fabsf(y) < kTiny ? kTiny : 0.f, y);
    return __uint_as_float((__float_as_uint(y + off) + d) & ~0xfffffu) - off;
}

// A root y >= 0 on the grid, the share of the way taken between the squares, so that the square
// is right on average (rounding the root evenly would raise it: the mean of squares is above the
// square of the mean). A root above zero keeps at least the smallest step.
__device__ __forceinline__ float root_to_grid(float y, uint32_t d) {
    const float off = y < kTiny ? kTiny : 0.f;
    const float t = y + off;
    const float low_t = __uint_as_float(__float_as_uint(t) & ~0xfffffu), low = low_t - off;
    const float unit = __uint_as_float((__float_as_uint(t) & 0x7f800000u) - (3u << 23));
    const float over = (t - low_t) * (y + low);                       // y^2 - low^2
    const float step = unit * fmaf(2.f, low, unit);                   // (low + unit)^2 - low^2
    const float rest = 2.f - __uint_as_float(0x3f800000u | d << 3);   // 1 - dither
    const float q = over >= rest * step ? low + unit : low;
    return fmaxf(q, y > 0.f ? 0.001953125f : 0.f);
}

// Codes and scale of one block of 256, eight elements a lane. The scale is the power of two that
// puts the block's largest finite magnitude (`top`, the same in all lanes) into [128, 256): the
// grid of held values then stays where it is from step to step (a scale that followed the
// largest magnitude would move it, and re-round every value, at each step), scaling is exact,
// and no carry passes 448.
// kRoot: f are roots of second moments. odd: a value of this lane is infinite or NaN, held as NaN.
template <bool kRoot>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int live, const float (&f)[8], float top,
                                            bool odd, const uint32_t (&hash)[8]) {
    const bool some = top >= 7.8886091e-31f;         // 2^-100: a block below it counts as 0
    const uint32_t pow2 = (__float_as_uint(top) & 0x7f800000u) - (7u << 23);
    const float inv = some ? __uint_as_float((254u << 23) - pow2) : 0.f;
    uint16_t b[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float q[2];
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float y = f[2 * i + j] * inv;
            q[j] = kRoot ? root_to_grid(y, (hash[2 * i + j] * 0xC2B2AE35u) >> 12) : to_grid(y, hash[2 * i + j] >> 12);
        }
        b[i] = (uint16_t)__nv_cvt_float2_to_fp8x2(make_float2(q[0], q[1]), __NV_SATFINITE, __NV_E4M3);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (!finite(f[i])) b[i / 2] |= 0x7f << 8 * (i % 2);
    }
    if (live == 8) {
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = (uint8_t)(b[i / 2] >> 8 * (i % 2));
    }
    if ((threadIdx.x & 31) == 0) *scale = some ? __uint_as_float(pow2) : 0.f;
}

// Largest finite magnitude of the warp's 256 values, as bits (which order like the values);
// odd: whether one of this lane's is not finite.
__device__ __forceinline__ float block_top(const float (&f)[8], bool& odd) {
    uint32_t top = 0;
#pragma unroll
    for (int i = 0; i < 8; ++i) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
    odd = top >= 0x7f800000u;
    if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (finite(f[i])) top = max(top, __float_as_uint(f[i]) & 0x7fffffffu);
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

// One unit of one tensor by one warp. live: this lane's elements (0 .. 8). m and v are sums of
// rounded products (no fma): the same bits on any machine, so that a block's scale is too.
template <typename P, typename G>
__device__ __forceinline__ void unit(const TensorArg& t, const Step& s, int64_t u, int lane) {
    const int64_t i0 = u * kUnit + lane * 8;
    const int live = (int)max((int64_t)0, min((int64_t)8, t.n - i0));
    float x[8], g[8], m[8], v[8], root[8];
    P* p = static_cast<P*>(t.p) + i0;
    if (t.w) load8(t.w + i0, live, x);
    else load8(p, live, x);
    load8(static_cast<const G*>(t.g) + i0, live, g);
    const bool narrow = t.ms != nullptr;
    if (narrow) {
        load_codes(static_cast<const uint8_t*>(t.m) + i0, live, t.ms[u], m);
        load_codes(static_cast<const uint8_t*>(t.v) + i0, live, t.vs[u], v);
#pragma unroll
        for (int i = 0; i < 8; ++i) v[i] *= v[i];
    } else {
        load8(static_cast<const float*>(t.m) + i0, live, m);
        load8(static_cast<const float*>(t.v) + i0, live, v);
    }
#pragma unroll
    for (int i = 0; i < 8; i += 2) {
        const uint64_t gg = mul2(pk2(g[i], g[i + 1]), splat2(s.gs));
        const uint64_t mm = add2(mul2(splat2(s.b1), pk2(m[i], m[i + 1])), mul2(splat2(s.ob1), gg));
        const uint64_t vv = add2(mul2(splat2(s.b2), pk2(v[i], v[i + 1])), mul2(splat2(s.ob2), mul2(gg, gg)));
        upk2(mm, m[i], m[i + 1]);
        upk2(vv, v[i], v[i + 1]);
        root[i] = sqrt_approx(v[i]);
        root[i + 1] = sqrt_approx(v[i + 1]);
        float d0, d1;
        upk2(fma2(pk2(root[i], root[i + 1]), splat2(s.rc2), splat2(s.eps)), d0, d1);
        const uint64_t up = mul2(mul2(mm, splat2(s.rate)), pk2(rcp_approx(d0), rcp_approx(d1)));
        upk2(fma2(pk2(x[i], x[i + 1]), splat2(s.keep), up), x[i], x[i + 1]);
    }
    store8(p, live, x);
    if (t.w) store8(t.w + i0, live, x);
    if (narrow) {
        // one hash of element and step: its top bits dither m, those of an odd multiple v
        uint32_t hash[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = ((uint32_t)i0 + i) * 0x9E3779B1u + s.dither;
            hash[i] = (h ^ (h >> 15)) * 0x85EBCA6Bu;
        }
        bool odd;
        const float top_m = block_top(m, odd);
        store_codes<false>(static_cast<uint8_t*>(t.m) + i0, t.ms + u, live, m, top_m, odd, hash);
        const float top_v = block_top(v, odd);
        store_codes<true>(static_cast<uint8_t*>(t.v) + i0, t.vs + u, live, root, __fsqrt_rn(top_v), odd, hash);
    } else {
        store8(static_cast<float*>(t.m) + i0, live, m);
        store8(static_cast<float*>(t.v) + i0, live, v);
    }
}

__global__ void __launch_bounds__(kThreads) adamw_kernel(const __grid_constant__ AdamArgs a) {
    pdl_wait();
    State* st = reinterpret_cast<State*>(a.state);
    // 1 - beta^(t+1) = beta (1 - beta^t) + (1 - beta)
    const double c1 = st->c1 * a.beta1 + (1.0 - a.beta1), c2 = st->c2 * a.beta2 + (1.0 - a.beta2);
    const long long step = st->step + 1;
    const float lr = a.lr_dev ? *a.lr_dev : (float)a.lr;
    Step s;
    s.b1 = (float)a.beta1;
    s.ob1 = (float)(1.0 - a.beta1);
    s.b2 = (float)a.beta2;
    s.ob2 = (float)(1.0 - a.beta2);
    s.rate = -lr / (float)c1;
    s.rc2 = 1.f / sqrtf((float)c2);
    s.eps = a.eps;
    s.gs = a.grad_scale ? *a.grad_scale : 1.f;
    s.dither = (uint32_t)step * 0x61C88647u;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    int lo = 0;
    for (int64_t q = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); q < a.units; q += warps) {
        if (lo + 1 < a.count && a.first[lo + 1] <= q) {
            int hi = a.count;                           // the last tensor whose first unit is <= q
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.first[mid] <= q) lo = mid; else hi = mid;
            }
        }
        const TensorArg& t = a.t[lo];
        s.keep = 1.f - lr * t.decay;
        const int64_t u = q - a.first[lo];
        switch (t.kind) {
            case 0: unit<float, float>(t, s, u, lane); break;
            case 1: unit<__nv_bfloat16, float>(t, s, u, lane); break;
            case 2: unit<float, __nv_bfloat16>(t, s, u, lane); break;
            default: unit<__nv_bfloat16, __nv_bfloat16>(t, s, u, lane); break;
        }
    }
    // the last block to get here counts the step: every block has read the old count by then
    if (a.advance) {
        __syncthreads();
        if (threadIdx.x == 0) {
            __threadfence();
            if (atomicAdd(&st->ticket, 1u) == gridDim.x - 1) {
                st->c1 = c1;
                st->c2 = c2;
                st->step = step;
                st->ticket = 0;
            }
        }
    }
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

moe_status_t check_adamw(const moe_adamw_config_t* c, const moe_adamw_tensor_t* ts, int32_t count) {
    if (!c || count < 0 || (count > 0 && !ts)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->lr) || !(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0) ||
        !(c->eps >= 1e-30 && c->eps <= 1e30))
        return MOE_ERR_INVALID_ARG;
    for (int i = 0; i < count; ++i) {
        const moe_adamw_tensor_t& t = ts[i];
        if (t.n < 0 || t.reserved != 0) return MOE_ERR_INVALID_ARG;
        if ((t.dtype != MOE_F32 && t.dtype != MOE_BF16) || (t.grad_dtype != MOE_F32 && t.grad_dtype != MOE_BF16))
            return MOE_ERR_INVALID_ARG;
        if (!std::isfinite(t.weight_decay) || t.weight_decay < 0.f) return MOE_ERR_INVALID_ARG;
        if (t.n > 0 && ((t.m_scale == nullptr) != (t.v_scale == nullptr) || !t.p || !t.g || !t.m || !t.v))
            return MOE_ERR_INVALID_ARG;
        for (const void* p : {(const void*)t.p, t.g, (const void*)t.master, (const void*)t.m, (const void*)t.v})
            if (misaligned(p, 16)) return MOE_ERR_INVALID_ARG;
        if (misaligned(t.m_scale, 4) || misaligned(t.v_scale, 4)) return MOE_ERR_INVALID_ARG;
        if (t.n > ((int64_t)1 << 38)) return MOE_ERR_UNSUPPORTED;
    }
    return MOE_OK;
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API moe_status_t moe_adamw(const moe_adamw_config_t* cfg, const moe_adamw_tensor_t* tensors,
                                          int32_t count, const float* lr, const float* grad_scale, void* state,
                                          moe_stream_t stream) {
    const moe_status_t st = check_adamw(cfg, tensors, count);
    if (st != MOE_OK) return st;
    if (!state || misaligned(state, 8) || misaligned(lr, 4) || misaligned(grad_scale, 4)) return MOE_ERR_INVALID_ARG;
    AdamArgs a{};
    a.lr = cfg->lr;
    a.beta1 = cfg->beta1;
    a.beta2 = cfg->beta2;
    a.eps = (float)cfg->eps;
    a.lr_dev = lr;
    a.grad_scale = grad_scale;
    a.state = static_cast<unsigned char*>(state);
    int i = 0;
    do {
        a.count = 0;
        a.units = 0;
        for (; i < count && a.count < kBatch; ++i) {
            const moe_adamw_tensor_t& t = tensors[i];
            if (t.n == 0) continue;
            a.first[a.count] = a.units;
            a.t[a.count] = {t.p, t.g, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay,
                            (t.dtype == MOE_BF16 ? 1 : 0) | (t.grad_dtype == MOE_BF16 ? 2 : 0)};
            a.units += (t.n + kUnit - 1) / kUnit;
            ++a.count;
        }
        a.advance = i == count;
        const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((a.units + 7) / 8, (int64_t)num_sms() * 8));
        const cudaError_t e = launch_pdl(adamw_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, (cudaStream_t)stream, a);
        count_launch();
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    } while (i < count);
    return MOE_OK;
}
