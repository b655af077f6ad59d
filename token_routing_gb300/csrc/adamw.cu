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
    float rate;                        // lr / (1 - beta1^t)
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

__device__ __forceinline__ void load_codes(const uint8_t* p, int live, float scale, float (&f)[8]) {
    uint8_t b[8];
    if (live == 8) {
        *reinterpret_cast<uint2*>(b) = *reinterpret_cast<const uint2*>(p);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) b[i] = i < live ? p[i] : 0;
    }
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        __nv_fp8_e4m3 e;
        e.__x = b[i];
        f[i] = __fmul_rn(static_cast<float>(e), scale);
    }
}

// e4m3 code of y (|y| < 256 if finite): one of its two neighbours on the grid, chosen by the
// dither d (20 bits). kRoot false: up with the probability of the share of the way up, so that
// the value is right on average. kRoot true: y is the root of a second moment, and the share is
// taken between the squares, so that the moment is right on average (rounding the root evenly
// would raise it: the mean of squares is above the square of the mean); a root above zero keeps
// at least the smallest code. Above 2^-6 a grid step is 2^-3 of the leading bit, below it 2^-9.
template <bool kRoot>
__device__ __forceinline__ uint8_t encode(float y, uint32_t d) {
    const float a = fabsf(y);
    const uint32_t bits = __float_as_uint(a);
    float q;
    if (kRoot) {
        const bool high = a >= 0.015625f;
        const float low = high ? __uint_as_float(bits & ~0xfffffu) : floorf(a * 512.f) * 0.001953125f;
        const float unit = high ? __uint_as_float((bits & 0x7f800000u) - (3u << 23)) : 0.001953125f;
        const float over = __fmul_rn(__fsub_rn(a, low), __fadd_rn(a, low));
        const float step = __fmul_rn(unit, __fadd_rn(2.f * low, unit));
        q = over >= __fmul_rn((float)(0x100000u - d) * 9.5367431640625e-7f, step) ? low + unit : low;
        if (a > 0.f && q == 0.f) q = 0.001953125f;
    } else {
        q = a >= 0.015625f ? __uint_as_float((bits + d) & ~0xfffffu)
                           : floorf(__fadd_rn(a * 512.f, (float)d * 9.5367431640625e-7f)) * 0.001953125f;
    }
    q = copysignf(q, y);
    if (!finite(y)) q = NAN;                         // infinities and NaN are held as NaN
    return __nv_fp8_e4m3(q).__x;
}

// Scale and codes of one block. The scale is the power of two that puts the largest finite
// magnitude into [128, 256): the grid of held values then stays where it is from step to step
// (a scale that followed the largest magnitude would move it, and re-round every value, at
// each step), scaling is exact, and the dither's carry cannot pass 448.
template <bool kRoot>
__device__ __forceinline__ void store_codes(uint8_t* p, float* scale, int live, const float (&f)[8],
                                            const uint32_t (&hash)[8]) {
    float top = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (i < live && finite(f[i])) top = fmaxf(top, fabsf(f[i]));
#pragma unroll
    for (int o = 16; o > 0; o >>= 1) top = fmaxf(top, __shfl_xor_sync(0xffffffffu, top, o));
    const bool some = top >= 7.8886091e-31f;         // 2^-100: a block below it counts as 0
    const uint32_t pow2 = (__float_as_uint(top) & 0x7f800000u) - (7u << 23);
    const float inv = __uint_as_float((254u << 23) - pow2);
    uint8_t b[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t d = (kRoot ? hash[i] * 0xC2B2AE35u : hash[i]) >> 12;
        b[i] = encode<kRoot>(some ? f[i] * inv : finite(f[i]) ? 0.f : NAN, d);
    }
    if (live == 8) {
        *reinterpret_cast<uint2*>(p) = *reinterpret_cast<const uint2*>(b);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < live) p[i] = b[i];
    }
    if ((threadIdx.x & 31) == 0) *scale = some ? __uint_as_float(pow2) : 0.f;
}

// One unit of one tensor by one warp. live: this lane's elements (0 .. 8).
template <typename P, typename G>
__device__ __forceinline__ void unit(const TensorArg& t, const Step& s, int64_t u, int lane) {
    const int64_t i0 = u * kUnit + lane * 8;
    const int live = (int)max((int64_t)0, min((int64_t)8, t.n - i0));
    float x[8], g[8], m[8], v[8];
    P* p = static_cast<P*>(t.p) + i0;
    if (t.w) load8(t.w + i0, live, x);
    else load8(p, live, x);
    load8(static_cast<const G*>(t.g) + i0, live, g);
    const bool narrow = t.ms != nullptr;
    if (narrow) {
        load_codes(static_cast<const uint8_t*>(t.m) + i0, live, t.ms[u], m);
        load_codes(static_cast<const uint8_t*>(t.v) + i0, live, t.vs[u], v);
    } else {
        load8(static_cast<const float*>(t.m) + i0, live, m);
        load8(static_cast<const float*>(t.v) + i0, live, v);
    }
    float root[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const float gi = g[i] * s.gs;
        if (narrow) v[i] = __fmul_rn(v[i], v[i]);
        m[i] = __fadd_rn(__fmul_rn(s.b1, m[i]), __fmul_rn(s.ob1, gi));
        v[i] = __fadd_rn(__fmul_rn(s.b2, v[i]), __fmul_rn(s.ob2, __fmul_rn(gi, gi)));
        root[i] = __fsqrt_rn(v[i]);
        x[i] = x[i] * s.keep - __fdividef(m[i] * s.rate, fmaf(root[i], s.rc2, s.eps));
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
        store_codes<false>(static_cast<uint8_t*>(t.m) + i0, t.ms + u, live, m, hash);
        store_codes<true>(static_cast<uint8_t*>(t.v) + i0, t.vs + u, live, root, hash);
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
    s.rate = lr / (float)c1;
    s.rc2 = 1.f / sqrtf((float)c2);
    s.eps = a.eps;
    s.gs = a.grad_scale ? *a.grad_scale : 1.f;
    s.dither = (uint32_t)step * 0x61C88647u;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    for (int64_t q = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); q < a.units; q += warps) {
        int lo = 0, hi = a.count;                       // the last tensor whose first unit is <= q
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (a.first[mid] <= q) lo = mid; else hi = mid;
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
        !(c->eps > 0.0) || !std::isfinite(c->eps))
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
