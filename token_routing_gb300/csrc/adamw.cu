// AdamW over many tensors in one launch, with fp32 or 8-bit states.
#include <cuda_fp8.h>

#include <cmath>
#include <type_traits>

#include "internal.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = MOE_ADAMW_BLOCK;     // elements a warp takes at a time: 8 a lane, one scale block
constexpr int kBlocks = 4;                 // blocks to an SM
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
    int32_t kind;      // bit 0: p is bf16, bit 1: g is bf16, bit 2: master, bit 3: 8-bit states
};

struct AdamArgs {
    double beta1, beta2;
    float lr, b1, ob1, b2, ob2, eps;   // b1, b2: betas, ob1, ob2: 1 - betas, each rounded from double
    int count;
    int advance;                       // this launch is the call's last: it counts the step
    const float* lr_dev;
    const float* grad_scale;
    unsigned char* state;
    int run;                           // units of one tensor that a warp takes in a row
    int64_t runs;
    int64_t first[kBatch];             // first run of each tensor
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

__device__ __forceinline__ bool finite(float x) { return fabsf(x) <= 3.4028235e38f; }

__device__ __forceinline__ float sqrt_approx(float x) {
    float r;
    asm("sqrt.approx.f32 %0, %1;" : "=f"(r) : "f"(x));
    return r;
}

// Eight elements as fp32 pairs, from 16 or 32 bytes, and back.
template <typename T>
__device__ __forceinline__ void load8(const T* p, uint64_t (&f)[4]) {
    if constexpr (sizeof(T) == 2) {
        to_pairs<T>(*reinterpret_cast<const uint4*>(p), f);
    } else {
        to_pairs<T>(reinterpret_cast<const uint4*>(p)[0], reinterpret_cast<uint64_t(&)[2]>(f[0]));
        to_pairs<T>(reinterpret_cast<const uint4*>(p)[1], reinterpret_cast<uint64_t(&)[2]>(f[2]));
    }
}
template <typename T>
__device__ __forceinline__ void store8(T* p, const uint64_t (&f)[4]) {
    if constexpr (sizeof(T) == 2) {
        *reinterpret_cast<uint4*>(p) = from_pairs<T>(f);
    } else {
        reinterpret_cast<uint4*>(p)[0] = from_pairs<T>(reinterpret_cast<const uint64_t(&)[2]>(f[0]));
        reinterpret_cast<uint4*>(p)[1] = from_pairs<T>(reinterpret_cast<const uint64_t(&)[2]>(f[2]));
    }
}

// Eight e4m3 codes as fp32 pairs times scale.
__device__ __forceinline__ void decode8(uint2 codes, float scale, uint64_t (&f)[4]) {
    const uint32_t w[2] = {codes.x, codes.y};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const __half2 h = __half2(__nv_cvt_fp8x2_to_halfraw2((uint16_t)(w[i / 2] >> 16 * (i % 2)), __NV_E4M3));
        const float2 v = __half22float2(h);
        f[i] = mul2(pk2(v.x, v.y), splat2(scale));
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

// Eight of the codes of one block. `inv` is one over the block's scale, the power of two that
// puts its largest finite magnitude into [128, 256): the grid of held values then stays where it
// is from step to step (a scale that followed the largest magnitude would move it, and re-round
// every value, at each step), scaling is exact, and no carry passes 448.
// kRoot: f are roots of second moments. odd: one of them is infinite or NaN, held as NaN.
template <bool kRoot>
__device__ __forceinline__ uint2 encode8(const uint64_t (&f)[4], float inv, bool odd, const uint32_t (&hash)[8]) {
    uint32_t w[2] = {0, 0};
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        float y0, y1;
        upk2(mul2(f[i], splat2(inv)), y0, y1);
        if constexpr (kRoot) {
            y0 = root_to_grid(y0, (hash[2 * i] * 0xC2B2AE35u) >> 12);
            y1 = root_to_grid(y1, (hash[2 * i + 1] * 0xC2B2AE35u) >> 12);
        } else {
            y0 = to_grid(y0, hash[2 * i] >> 12);
            y1 = to_grid(y1, hash[2 * i + 1] >> 12);
        }
        w[i / 2] |= (uint32_t)__nv_cvt_float2_to_fp8x2(make_float2(y0, y1), __NV_SATFINITE, __NV_E4M3) << 16 * (i % 2);
    }
    if (odd) {
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            float y0, y1;
            upk2(f[i], y0, y1);
            if (!finite(y0)) w[i / 2] |= 0x7fu << 16 * (i % 2);
            if (!finite(y1)) w[i / 2] |= 0x7f00u << 16 * (i % 2);
        }
    }
    return make_uint2(w[0], w[1]);
}

// Largest finite magnitude of the warp's 256 values, as bits (which order like the values);
// odd: whether one of this lane's is not finite.
__device__ __forceinline__ float block_top(const uint64_t (&f)[4], bool& odd) {
    uint32_t top = 0, b[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        b[2 * i] = (uint32_t)f[i] & 0x7fffffffu;
        b[2 * i + 1] = (uint32_t)(f[i] >> 32) & 0x7fffffffu;
        top = max(top, max(b[2 * i], b[2 * i + 1]));
    }
    odd = top >= 0x7f800000u;
    if (odd) {
        top = 0;
#pragma unroll
        for (int i = 0; i < 8; ++i) top = b[i] < 0x7f800000u ? max(top, b[i]) : top;
    }
    return __uint_as_float(__reduce_max_sync(0xffffffffu, top));
}

// The scale of a block whose largest magnitude is top, and one over it; 0 for a block below 2^-100.
__device__ __forceinline__ float block_scale(float top, float& inv) {
    const bool some = top >= 7.8886091e-31f;
    const uint32_t pow2 = (__float_as_uint(top) & 0x7f800000u) - (7u << 23);
    inv = some ? __uint_as_float((254u << 23) - pow2) : 0.f;
    return some ? __uint_as_float(pow2) : 0.f;
}

// The step on eight elements. m and v are sums of rounded products (no fma): the same bits on any
// machine, so that a block's scale is too.
__device__ __forceinline__ void advance8(const Step& s, const uint64_t (&g)[4], uint64_t (&x)[4], uint64_t (&m)[4],
                                         uint64_t (&v)[4], uint64_t (&root)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t gg = mul2(g[i], splat2(s.gs));
        m[i] = add2(mul2(splat2(s.b1), m[i]), mul2(splat2(s.ob1), gg));
        v[i] = add2(mul2(splat2(s.b2), v[i]), mul2(splat2(s.ob2), mul2(gg, gg)));
        float v0, v1, d0, d1;
        upk2(v[i], v0, v1);
        root[i] = pk2(sqrt_approx(v0), sqrt_approx(v1));
        upk2(fma2(root[i], splat2(s.rc2), splat2(s.eps)), d0, d1);
        x[i] = fma2(x[i], splat2(s.keep), mul2(mul2(m[i], splat2(s.rate)), pk2(rcp_approx(d0), rcp_approx(d1))));
    }
}

// The codes and scales of one block of both states.
__device__ __forceinline__ void hold(const uint64_t (&m)[4], const uint64_t (&v)[4], const uint64_t (&root)[4],
                                     uint32_t h0, uint2& cm, uint2& cv, float& sm, float& sv) {
    // one hash of element and step: its top bits dither m, those of an odd multiple v
    uint32_t hash[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = h0 + i * 0x9E3779B1u;
        hash[i] = (h ^ (h >> 15)) * 0x85EBCA6Bu;
    }
    bool odd;
    float inv;
    sm = block_scale(block_top(m, odd), inv);
    cm = encode8<false>(m, inv, odd, hash);
    sv = block_scale(__fsqrt_rn(block_top(v, odd)), inv);
    cv = encode8<true>(root, inv, odd, hash);
}

// Whole units u0 .. u0 + count - 1 of one tensor by one warp, eight elements a lane and unit.
template <typename P, typename G, bool kMaster, bool kNarrow>
__device__ __forceinline__ void run_units(const TensorArg& t, const Step& s, int64_t u0, int count, int lane) {
    const int64_t i0 = u0 * kUnit + lane * 8;
    P* p = static_cast<P*>(t.p) + i0;
    const G* g = static_cast<const G*>(t.g) + i0;
    float* w = kMaster ? t.w + i0 : nullptr;
    using S = std::conditional_t<kNarrow, uint8_t, float>;
    S* m = static_cast<S*>(t.m) + i0;
    S* v = static_cast<S*>(t.v) + i0;
    float* ms = t.ms + u0;
    float* vs = t.vs + u0;
    uint32_t h0 = (uint32_t)i0 * 0x9E3779B1u + s.dither;
    for (int k = 0; k < count; ++k) {
        uint64_t X[4], Gr[4], M[4], V[4], R[4];
        if constexpr (kMaster) load8(w, X);
        else load8(p, X);
        load8(g, Gr);
        if constexpr (kNarrow) {
            const uint2 cm = *reinterpret_cast<const uint2*>(m), cv = *reinterpret_cast<const uint2*>(v);
            decode8(cm, *ms, M);
            decode8(cv, *vs, V);
#pragma unroll
            for (int i = 0; i < 4; ++i) V[i] = mul2(V[i], V[i]);
        } else {
            load8(m, M);
            load8(v, V);
        }
        advance8(s, Gr, X, M, V, R);
        store8(p, X);
        if constexpr (kMaster) store8(w, X);
        if constexpr (kNarrow) {
            uint2 cm, cv;
            float sm, sv;
            hold(M, V, R, h0, cm, cv, sm, sv);
            *reinterpret_cast<uint2*>(m) = cm;
            *reinterpret_cast<uint2*>(v) = cv;
            if (lane == 0) {
                *ms = sm;
                *vs = sv;
            }
        } else {
            store8(m, M);
            store8(v, V);
        }
        p += kUnit;
        g += kUnit;
        if (kMaster) w += kUnit;
        m += kUnit;
        v += kUnit;
        if (kNarrow) {
            ++ms;
            ++vs;
        }
        h0 += kUnit * 0x9E3779B1u;
    }
}

// The unit that a tensor's end cuts short, element by element.
__device__ __noinline__ void last_unit(const TensorArg& t, const Step& s, int64_t u, int lane) {
    const int64_t i0 = u * kUnit + lane * 8;
    float f[4][8];
    const auto live = [&](int i) { return i0 + i < t.n; };
    const bool narrow = t.ms != nullptr;
    for (int i = 0; i < 8; ++i) {
        f[0][i] = f[1][i] = f[2][i] = f[3][i] = 0.f;
        if (!live(i)) continue;
        f[0][i] = t.w ? t.w[i0 + i] : t.kind & 1 ? ld_f(static_cast<const __nv_bfloat16*>(t.p) + i0 + i)
                                                 : static_cast<const float*>(t.p)[i0 + i];
        f[1][i] = t.kind & 2 ? ld_f(static_cast<const __nv_bfloat16*>(t.g) + i0 + i) : static_cast<const float*>(t.g)[i0 + i];
        if (!narrow) {
            f[2][i] = static_cast<const float*>(t.m)[i0 + i];
            f[3][i] = static_cast<const float*>(t.v)[i0 + i];
        }
    }
    uint64_t X[4], Gr[4], M[4], V[4], R[4];
    for (int i = 0; i < 4; ++i) {
        X[i] = pk2(f[0][2 * i], f[0][2 * i + 1]);
        Gr[i] = pk2(f[1][2 * i], f[1][2 * i + 1]);
        M[i] = pk2(f[2][2 * i], f[2][2 * i + 1]);
        V[i] = pk2(f[3][2 * i], f[3][2 * i + 1]);
    }
    uint8_t* cm = static_cast<uint8_t*>(t.m) + i0;
    uint8_t* cv = static_cast<uint8_t*>(t.v) + i0;
    if (narrow) {
        uint32_t b[4] = {0, 0, 0, 0};
        for (int i = 0; i < 8; ++i)
            if (live(i)) {
                b[i / 4] |= (uint32_t)cm[i] << 8 * (i % 4);
                b[2 + i / 4] |= (uint32_t)cv[i] << 8 * (i % 4);
            }
        decode8(make_uint2(b[0], b[1]), t.ms[u], M);
        decode8(make_uint2(b[2], b[3]), t.vs[u], V);
        for (int i = 0; i < 4; ++i) V[i] = mul2(V[i], V[i]);
    }
    advance8(s, Gr, X, M, V, R);
    uint2 km{}, kv{};
    if (narrow) {
        float sm, sv;
        hold(M, V, R, (uint32_t)i0 * 0x9E3779B1u + s.dither, km, kv, sm, sv);
        if (lane == 0) {
            t.ms[u] = sm;
            t.vs[u] = sv;
        }
    }
    for (int i = 0; i < 8; ++i) {
        if (!live(i)) continue;
        float x0, x1, m0, m1, v0, v1;
        upk2(X[i / 2], x0, x1);
        upk2(M[i / 2], m0, m1);
        upk2(V[i / 2], v0, v1);
        const float x = i % 2 ? x1 : x0;
        if (t.w) t.w[i0 + i] = x;
        if (t.kind & 1) st_f(static_cast<__nv_bfloat16*>(t.p) + i0 + i, x);
        else static_cast<float*>(t.p)[i0 + i] = x;
        if (narrow) {
            cm[i] = (uint8_t)((i < 4 ? km.x : km.y) >> 8 * (i % 4));
            cv[i] = (uint8_t)((i < 4 ? kv.x : kv.y) >> 8 * (i % 4));
        } else {
            static_cast<float*>(t.m)[i0 + i] = i % 2 ? m1 : m0;
            static_cast<float*>(t.v)[i0 + i] = i % 2 ? v1 : v0;
        }
    }
}

__global__ void __launch_bounds__(kThreads, kBlocks) adamw_kernel(const __grid_constant__ AdamArgs a) {
    pdl_wait();
    State* st = reinterpret_cast<State*>(a.state);
    // 1 - beta^(t+1) = beta (1 - beta^t) + (1 - beta)
    const double c1 = st->c1 * a.beta1 + (1.0 - a.beta1), c2 = st->c2 * a.beta2 + (1.0 - a.beta2);
    const long long step = st->step + 1;
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    Step s;
    s.b1 = a.b1;
    s.ob1 = a.ob1;
    s.b2 = a.b2;
    s.ob2 = a.ob2;
    s.rate = -lr / (float)c1;
    s.rc2 = 1.f / sqrtf((float)c2);
    s.eps = a.eps;
    s.gs = a.grad_scale ? *a.grad_scale : 1.f;
    s.dither = (uint32_t)step * 0x61C88647u;
    const int lane = threadIdx.x & 31;
    const int64_t warps = (int64_t)gridDim.x * (kThreads / 32);
    int lo = 0;
    for (int64_t q = (int64_t)blockIdx.x * (kThreads / 32) + (threadIdx.x >> 5); q < a.runs; q += warps) {
        if (lo + 1 < a.count && a.first[lo + 1] <= q) {
            int hi = a.count;                           // the last tensor whose first run is <= q
            while (hi - lo > 1) {
                const int mid = (lo + hi) >> 1;
                if (a.first[mid] <= q) lo = mid; else hi = mid;
            }
        }
        const TensorArg& t = a.t[lo];
        s.keep = 1.f - lr * t.decay;
        const int64_t u = (q - a.first[lo]) * a.run, whole = t.n / kUnit;
        const int count = (int)min((int64_t)a.run, whole - u);
        using B = __nv_bfloat16;
        switch (t.kind) {
            case 0: run_units<float, float, false, false>(t, s, u, count, lane); break;
            case 1: run_units<B, float, false, false>(t, s, u, count, lane); break;
            case 2: run_units<float, B, false, false>(t, s, u, count, lane); break;
            case 3: run_units<B, B, false, false>(t, s, u, count, lane); break;
            case 4: run_units<float, float, true, false>(t, s, u, count, lane); break;
            case 5: run_units<B, float, true, false>(t, s, u, count, lane); break;
            case 6: run_units<float, B, true, false>(t, s, u, count, lane); break;
            case 7: run_units<B, B, true, false>(t, s, u, count, lane); break;
            case 8: run_units<float, float, false, true>(t, s, u, count, lane); break;
            case 9: run_units<B, float, false, true>(t, s, u, count, lane); break;
            case 10: run_units<float, B, false, true>(t, s, u, count, lane); break;
            case 11: run_units<B, B, false, true>(t, s, u, count, lane); break;
            case 12: run_units<float, float, true, true>(t, s, u, count, lane); break;
            case 13: run_units<B, float, true, true>(t, s, u, count, lane); break;
            case 14: run_units<float, B, true, true>(t, s, u, count, lane); break;
            default: run_units<B, B, true, true>(t, s, u, count, lane); break;
        }
        if (count < a.run && whole * kUnit < t.n && u + count == whole) last_unit(t, s, whole, lane);
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
    a.lr = (float)cfg->lr;
    a.beta1 = cfg->beta1;
    a.beta2 = cfg->beta2;
    a.b1 = (float)cfg->beta1;
    a.ob1 = (float)(1.0 - cfg->beta1);
    a.b2 = (float)cfg->beta2;
    a.ob2 = (float)(1.0 - cfg->beta2);
    a.eps = (float)cfg->eps;
    a.lr_dev = lr;
    a.grad_scale = grad_scale;
    a.state = static_cast<unsigned char*>(state);
    // long runs spare a warp the start of a run, short ones spread small tensors over more warps
    int64_t units = 0;
    for (int k = 0; k < count; ++k) units += (tensors[k].n + kUnit - 1) / kUnit;
    const int64_t warps = (int64_t)num_sms() * kBlocks * (kThreads / 32);
    a.run = units >= 16 * warps ? 8 : 1;
    int i = 0;
    do {
        a.count = 0;
        a.runs = 0;
        for (; i < count && a.count < kBatch; ++i) {
            const moe_adamw_tensor_t& t = tensors[i];
            if (t.n == 0) continue;
            a.first[a.count] = a.runs;
            a.t[a.count] = {t.p, t.g, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay,
                            (t.dtype == MOE_BF16 ? 1 : 0) | (t.grad_dtype == MOE_BF16 ? 2 : 0) | (t.master ? 4 : 0) |
                                (t.m_scale ? 8 : 0)};
            a.runs += (t.n + (int64_t)kUnit * a.run - 1) / ((int64_t)kUnit * a.run);
            ++a.count;
        }
        a.advance = i == count;
        const int64_t blocks = std::max<int64_t>(1, std::min<int64_t>((a.runs + 7) / 8, (int64_t)num_sms() * kBlocks));
        const cudaError_t e = launch_pdl(adamw_kernel, dim3((unsigned)blocks), dim3(kThreads), 0, (cudaStream_t)stream, a);
        count_launch();
        if (e != cudaSuccess) return MOE_ERR_CUDA;
    } while (i < count);
    return MOE_OK;
}
