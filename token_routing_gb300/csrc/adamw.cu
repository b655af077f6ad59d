// AdamW over many tensors in one launch, with fp32 or 8-bit states.
//
// Per element: m = b1 m + (1 - b1) g, v = b2 v + (1 - b2) g^2, x = keep x - rate m / (sqrt(v) rc2 + eps),
// with the bias corrections folded into rate and rc2. Bound by memory: 30 bytes an element with
// fp32 states and a master (bf16 weight and gradient), 18 with 8-bit states.
#include <cuda_fp8.h>

#include <climits>
#include <cmath>
#include <type_traits>

#include "pairs.cuh"

namespace moe {

namespace {

constexpr int kThreads = 256;
constexpr int kUnit = MOE_ADAMW_BLOCK;     // elements a warp takes at a time: 8 a lane, one scale block
constexpr uint32_t kTicket = 1024;         // blocks that may take a ticket each
constexpr int kResident[2] = {2, 3};       // blocks to an SM, with fp32 and with 8-bit states
constexpr int kRun[2] = {16, 32};          // longest runs, with fp32 and with 8-bit states
constexpr int kBatch = kThreads;           // tensors in one launch's parameters, one looked at by each thread

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
    int32_t kind;      // bit 0: p is bf16, bit 1: g is bf16, bit 2: master
};

struct AdamArgs {
    double beta1, beta2;
    float lr, b1, ob1, b2, ob2, eps;   // b1, b2: betas, ob1, ob2: 1 - betas, each rounded from double
    int count;
    int advance;                       // this launch is the call's last: it counts the step
    const float* lr_dev;
    const float* grad_scale;
    unsigned char* state;
    int run;                           // eights of units of one tensor that a block takes in a row
    uint32_t runs;
    uint32_t first[kBatch];            // first run of each tensor
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
__device__ __forceinline__ void unpack8(const uint4* u, uint64_t (&f)[4]) {
    if constexpr (sizeof(T) == 2) {
        to_pairs<T>(u[0], f);
    } else {
        to_pairs<T>(u[0], reinterpret_cast<uint64_t(&)[2]>(f[0]));
        to_pairs<T>(u[1], reinterpret_cast<uint64_t(&)[2]>(f[2]));
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

// e4m3 in fp32. A value times 2^-120 has its e4m3 code in bits 26 .. 20 of the fp32 number: e4m3's
// exponent bias is then that of fp32, its numbers below 2^-6 are fp32's own subnormal ones, and
// the 20 bits below are the share of the way to the next code, for all of them alike.
constexpr float kToCode = 7.5231638e-37f;       // 2^-120
constexpr float kFromCode = 1.3292280e+36f;     // 2^120

// Code of y 2^-120 in the top byte, up with the probability of its share of the way: the 20 top
// bits of the hash are added to it.
__device__ __forceinline__ uint32_t value_code(float y, uint32_t hash) {
    const uint32_t t = __float_as_uint(y) + (hash >> 12);
    return (t << 4 & 0x7f000000u) | (t & 0x80000000u);
}

// Both halves of y times 2^-120, cut off where fp32's subnormal numbers end: what is left says for
// every value between which two codes it lies, and its share of the way to 20 bits.
__device__ __forceinline__ uint64_t to_codes(uint64_t y) {
    uint64_t r;
    asm("mul.rz.f32x2 %0, %1, %2;" : "=l"(r) : "l"(y), "l"(splat2(kToCode)));
    return r;
}

// Codes of two roots y >= 0 (and y 2^-120) in the top bytes. The share of the way is taken between
// the squares, so that the square is right on average (rounding the root evenly would raise it:
// the mean of squares is above the square of the mean). A root above zero keeps at least code 1.
__device__ __forceinline__ void root_codes(uint64_t y, uint64_t down, uint32_t hash0, uint32_t hash1, uint32_t& c0,
                                           uint32_t& c1) {
    const uint32_t l0 = (uint32_t)down & ~0xfffffu, l1 = (uint32_t)(down >> 32) & ~0xfffffu;
    const uint32_t n0 = l0 + 0x100000u, n1 = l1 + 0x100000u;
    const uint64_t low = mul2((uint64_t)l1 << 32 | l0, splat2(kFromCode));
    const uint64_t next = mul2((uint64_t)n1 << 32 | n0, splat2(kFromCode));
    const uint64_t minus = splat2(-1.f);
    const uint64_t over = mul2(fma2(low, minus, y), add2(y, low));                   // y^2 - low^2
    const uint64_t step = fma2(mul2(low, low), minus, mul2(next, next));             // next^2 - low^2
    // 1 - the dither, from 1 + the dither
    const uint64_t d = (uint64_t)(0x3f800000u | (hash1 >> 9 & 0x7ffff8u)) << 32 | (0x3f800000u | (hash0 >> 9 & 0x7ffff8u));
    float o0, o1, t0, t1;
    upk2(over, o0, o1);
    upk2(mul2(fma2(d, minus, splat2(2.f)), step), t0, t1);
    c0 = max(o0 >= t0 ? n0 : l0, min((uint32_t)y, 0x100000u)) << 4;
    c1 = max(o1 >= t1 ? n1 : l1, min((uint32_t)(y >> 32), 0x100000u)) << 4;
}

// Top bytes of four words as one word.
__device__ __forceinline__ uint32_t top_bytes(uint32_t a, uint32_t b, uint32_t c, uint32_t d) {
    return __byte_perm(__byte_perm(a, b, 0x0073), __byte_perm(c, d, 0x7300), 0x7610);
}

// Eight of the codes of one block. `inv` is one over the block's scale, the power of two that
// puts its largest finite magnitude into [128, 256): the grid of held values then stays where it
// is from step to step (a scale that followed the largest magnitude would move it, and re-round
// every value, at each step), scaling is exact, and no carry passes 448.
// kRoot: f are roots of second moments. odd: one of them is infinite or NaN, held as NaN.
// kWeyl: the words are a Weyl sequence, and a root's share of the way is taken in the root itself,
// with the top bit of its word turned; a root above zero keeps at least code 1 here too.
template <bool kRoot, bool kWeyl>
__device__ __forceinline__ uint2 encode8(const uint64_t (&f)[4], float inv, bool odd, const uint32_t (&hash)[8]) {
    uint32_t c[8];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t y = mul2(f[i], splat2(inv)), down = to_codes(y);
        if constexpr (kRoot && kWeyl) {
            float y0, y1;
            upk2(down, y0, y1);
            c[2 * i] = max(value_code(y0, hash[2 * i] ^ 0x80000000u), min((uint32_t)y, 0x100000u) << 4);
            c[2 * i + 1] = max(value_code(y1, hash[2 * i + 1] ^ 0x80000000u), min((uint32_t)(y >> 32), 0x100000u) << 4);
        } else if constexpr (kRoot) {
            root_codes(y, down, hash[2 * i] * 0xC2B2AE35u, hash[2 * i + 1] * 0xC2B2AE35u, c[2 * i], c[2 * i + 1]);
        } else {
            float y0, y1;
            upk2(down, y0, y1);
            c[2 * i] = value_code(y0, hash[2 * i]);
            c[2 * i + 1] = value_code(y1, hash[2 * i + 1]);
        }
    }
    uint32_t w[2] = {top_bytes(c[0], c[1], c[2], c[3]), top_bytes(c[4], c[5], c[6], c[7])};
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

// a x + b y, each product rounded by itself (packed products and sums are contracted by the
// compiler, rounding modifier or not: seen in the results).
__device__ __forceinline__ uint64_t rounded_sum(float a, uint64_t x, float b, uint64_t y) {
    float x0, x1, y0, y1;
    upk2(x, x0, x1);
    upk2(y, y0, y1);
    return pk2(__fadd_rn(__fmul_rn(a, x0), __fmul_rn(b, y0)), __fadd_rn(__fmul_rn(a, x1), __fmul_rn(b, y1)));
}

// The step on eight elements. With 8-bit states m and v are sums of rounded products: a mean that
// stays where it is (m = g) is then exactly what it was, and a block whose largest magnitude is a
// power of two keeps its scale, where a fused product and sum would be a rounding off to either
// side.
template <bool kNarrow>
__device__ __forceinline__ void advance8(const Step& s, const uint64_t (&g)[4], uint64_t (&x)[4], uint64_t (&m)[4],
                                         uint64_t (&v)[4], uint64_t (&root)[4]) {
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const uint64_t gg = mul2(g[i], splat2(s.gs));
        if constexpr (kNarrow) {
            m[i] = rounded_sum(s.b1, m[i], s.ob1, gg);
            v[i] = rounded_sum(s.b2, v[i], s.ob2, mul2(gg, gg));
        } else {
            m[i] = fma2(splat2(s.ob1), gg, mul2(splat2(s.b1), m[i]));
            v[i] = fma2(splat2(s.ob2), mul2(gg, gg), mul2(splat2(s.b2), v[i]));
        }
        float v0, v1, d0, d1;
        upk2(v[i], v0, v1);
        root[i] = kNarrow ? pk2(__fsqrt_rn(v0), __fsqrt_rn(v1)) : pk2(sqrt_approx(v0), sqrt_approx(v1));
        upk2(fma2(root[i], splat2(s.rc2), splat2(s.eps)), d0, d1);
        x[i] = fma2(x[i], splat2(s.keep), mul2(mul2(m[i], splat2(s.rate)), pk2(rcp_approx(d0), rcp_approx(d1))));
    }
}

// The codes and scales of one block of both states.
template <bool kWeyl>
__device__ __forceinline__ void hold(const uint64_t (&m)[4], const uint64_t (&v)[4], const uint64_t (&root)[4],
                                     uint32_t h0, uint2& cm, uint2& cv, float& sm, float& sv) {
    // The Weyl word of element and step (2^32 over the golden ratio and over its square), or one hash
    // of it, whose top bits dither m and those of an odd multiple v. The hash is a shift and the two
    // multipliers of Appleby's 32-bit finaliser (MurmurHash3).
    uint32_t hash[8];
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        const uint32_t h = h0 + i * 0x9E3779B1u;
        hash[i] = kWeyl ? h : (h ^ (h >> 15)) * 0x85EBCA6Bu;
    }
    bool odd;
    float inv;
    sm = block_scale(block_top(m, odd), inv);
    cm = encode8<false, kWeyl>(m, inv, odd, hash);
    sv = block_scale(__fsqrt_rn(block_top(v, odd)), inv);
    cv = encode8<true, kWeyl>(root, inv, odd, hash);
}

// What a lane reads of one unit, as it is in memory.
template <typename P, typename G, bool kMaster, bool kNarrow>
struct Raw {
    static constexpr int kX = (kMaster || sizeof(P) == 4) ? 2 : 1, kG = sizeof(G) / 2;
    uint4 x[kX], g[kG], m[kNarrow ? 1 : 2], v[kNarrow ? 1 : 2];     // 8 bits: both states' codes in m[0]
    float ms, vs;
};

// Whole units of one block's run: the block's eight warps take units u0 + 8 k + warp, eight
// elements a lane, while they are whole. Addresses are the run's bases, the same for the block,
// plus a 32-bit place.
template <typename P, typename G, bool kMaster, bool kNarrow, bool kWeyl>
__device__ __forceinline__ void run_units(const TensorArg& t, const Step& s, int64_t u0, int count, int run) {
    __shared__ float scales[2][kNarrow ? kRun[1] * 8 : 1];
    using R = Raw<P, G, kMaster, kNarrow>;
    using S = std::conditional_t<kNarrow, uint8_t, float>;
    const int64_t i0 = u0 * kUnit;
    P* const p = static_cast<P*>(t.p) + i0;
    const G* const g = static_cast<const G*>(t.g) + i0;
    float* const w = kMaster ? t.w + i0 : nullptr;
    S* const m = static_cast<S*>(t.m) + i0;
    S* const v = static_cast<S*>(t.v) + i0;
    float* const ms = kNarrow ? t.ms + u0 : nullptr;
    float* const vs = kNarrow ? t.vs + u0 : nullptr;
    const uint32_t warp = threadIdx.x >> 5;
    const auto fetch = [&](uint32_t u, R& r) {
        const uint32_t i = u * kUnit + (threadIdx.x & 31) * 8;
#pragma unroll
        for (int j = 0; j < R::kX; ++j)
            r.x[j] = kMaster ? reinterpret_cast<const uint4*>(w + i)[j] : reinterpret_cast<const uint4*>(p + i)[j];
#pragma unroll
        for (int j = 0; j < R::kG; ++j) r.g[j] = reinterpret_cast<const uint4*>(g + i)[j];
        if constexpr (kNarrow) {
            const uint2 a = *reinterpret_cast<const uint2*>(m + i), b = *reinterpret_cast<const uint2*>(v + i);
            r.m[0] = make_uint4(a.x, a.y, b.x, b.y);
            r.ms = ms[u];
            r.vs = vs[u];
        } else {
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                r.m[j] = reinterpret_cast<const uint4*>(m + i)[j];
                r.v[j] = reinterpret_cast<const uint4*>(v + i)[j];
            }
        }
    };
    R r;
    if ((int)warp < count) fetch(warp, r);
    for (uint32_t u = warp; (int)u < min(count, run * 8); u += 8) {
        uint64_t X[4], Gr[4], M[4], V[4], root[4];
        if constexpr (kMaster) unpack8<float>(r.x, X);
        else unpack8<P>(r.x, X);
        unpack8<G>(r.g, Gr);
        if constexpr (kNarrow) {
            decode8(make_uint2(r.m[0].x, r.m[0].y), r.ms, M);
            decode8(make_uint2(r.m[0].z, r.m[0].w), r.vs, V);
#pragma unroll
            for (int j = 0; j < 4; ++j) V[j] = mul2(V[j], V[j]);
            // much arithmetic to a byte: the next unit is on its way meanwhile
            if ((int)u + 8 < min(count, run * 8)) fetch(u + 8, r);
        } else {
            unpack8<float>(r.m, M);
            unpack8<float>(r.v, V);
        }
        advance8<kNarrow>(s, Gr, X, M, V, root);
        const uint32_t i = u * kUnit + (threadIdx.x & 31) * 8;
        store8(p + i, X);
        if constexpr (kMaster) store8(w + i, X);
        if constexpr (kNarrow) {
            uint2 cm, cv;
            float sm, sv;
            hold<kWeyl>(M, V, root, ((uint32_t)i0 + i) * 0x9E3779B1u + s.dither, cm, cv, sm, sv);
            *reinterpret_cast<uint2*>(m + i) = cm;
            *reinterpret_cast<uint2*>(v + i) = cv;
            if ((threadIdx.x & 31) == 0) {
                scales[0][u] = sm;
                scales[1][u] = sv;
            }
        } else {
            store8(m + i, M);
            store8(v + i, V);
            if ((int)u + 8 < min(count, run * 8)) fetch(u + 8, r);
        }
    }
    if constexpr (kNarrow) {
        // The scales go out by whole sectors: four bytes at a time from one warp after the other made
        // the memory fill and rewrite sectors (1.1G weights, at the time: 3240 - 3820 us against 2740).
        __syncthreads();
        for (int u = threadIdx.x; u < min(count, run * 8); u += kThreads) {
            ms[u] = scales[0][u];
            vs[u] = scales[1][u];
        }
    }
}

// The unit that a tensor's end cuts short, element by element.
template <bool kNarrow, bool kWeyl>
__device__ __noinline__ void last_unit(const TensorArg& t, const Step& s, int64_t u, int lane) {
    const int64_t i0 = u * kUnit + lane * 8;
    const auto live = [&](int i) { return i0 + i < t.n; };
    // all loads of the lane together
    float x[8], g[8], m[8], v[8];
    uint32_t b[4] = {0, 0, 0, 0};
    const uint8_t* lm = static_cast<const uint8_t*>(t.m) + i0;
    const uint8_t* lv = static_cast<const uint8_t*>(t.v) + i0;
#pragma unroll
    for (int i = 0; i < 8; ++i) x[i] = g[i] = m[i] = v[i] = 0.f;
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (live(i)) {
            if (t.w) x[i] = t.w[i0 + i];
            else if (t.kind & 1) x[i] = ld_f(static_cast<const __nv_bfloat16*>(t.p) + i0 + i);
            else x[i] = static_cast<const float*>(t.p)[i0 + i];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (live(i)) {
            if (t.kind & 2) g[i] = ld_f(static_cast<const __nv_bfloat16*>(t.g) + i0 + i);
            else g[i] = static_cast<const float*>(t.g)[i0 + i];
        }
#pragma unroll
    for (int i = 0; i < 8; ++i)
        if (live(i)) {
            if constexpr (kNarrow) {
                b[i / 4] |= (uint32_t)lm[i] << 8 * (i % 4);
                b[2 + i / 4] |= (uint32_t)lv[i] << 8 * (i % 4);
            } else {
                m[i] = static_cast<const float*>(t.m)[i0 + i];
                v[i] = static_cast<const float*>(t.v)[i0 + i];
            }
        }
    uint64_t X[4], Gr[4], M[4], V[4], R[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        X[i] = pk2(x[2 * i], x[2 * i + 1]);
        Gr[i] = pk2(g[2 * i], g[2 * i + 1]);
        M[i] = pk2(m[2 * i], m[2 * i + 1]);
        V[i] = pk2(v[2 * i], v[2 * i + 1]);
    }
    if constexpr (kNarrow) {
        decode8(make_uint2(b[0], b[1]), t.ms[u], M);
        decode8(make_uint2(b[2], b[3]), t.vs[u], V);
#pragma unroll
        for (int i = 0; i < 4; ++i) V[i] = mul2(V[i], V[i]);
    }
    advance8<kNarrow>(s, Gr, X, M, V, R);
    uint2 km{}, kv{};
    if constexpr (kNarrow) {
        float sm, sv;
        hold<kWeyl>(M, V, R, (uint32_t)i0 * 0x9E3779B1u + s.dither, km, kv, sm, sv);
        if (lane == 0) {
            t.ms[u] = sm;
            t.vs[u] = sv;
        }
    }
    uint8_t* cm = static_cast<uint8_t*>(t.m) + i0;
    uint8_t* cv = static_cast<uint8_t*>(t.v) + i0;
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        if (!live(i)) continue;
        float x0, x1, m0, m1, v0, v1;
        upk2(X[i / 2], x0, x1);
        upk2(M[i / 2], m0, m1);
        upk2(V[i / 2], v0, v1);
        const float y = i % 2 ? x1 : x0;
        if (t.w) t.w[i0 + i] = y;
        if (t.kind & 1) st_f(static_cast<__nv_bfloat16*>(t.p) + i0 + i, y);
        else static_cast<float*>(t.p)[i0 + i] = y;
        if constexpr (kNarrow) {
            cm[i] = (uint8_t)((i < 4 ? km.x : km.y) >> 8 * (i % 4));
            cv[i] = (uint8_t)((i < 4 ? kv.x : kv.y) >> 8 * (i % 4));
        } else {
            static_cast<float*>(t.m)[i0 + i] = i % 2 ? m1 : m0;
            static_cast<float*>(t.v)[i0 + i] = i % 2 ? v1 : v0;
        }
    }
}

// One block, one run: up to 16 (or, with 8-bit states, 32) times 2048 elements of one tensor, a unit
// of 256 to a warp at a time; small batches of tensors take shorter runs over more blocks. The
// tensors come as launch parameters (no table on the device to keep), a block finds its own by one
// vote over all of them.
// fp32 states, 156M weights with masters: 700 us, 6690 GB/s (99 %); 114 registers and two blocks to
// an SM, against 720 us at three and 800 at four, whose loads are cut apart. 8-bit states, 1.1G
// weights: 2800 us, 6350 GB/s (95 %), four fifths of the issue slots taken: the next unit's loads
// pass under the arithmetic of this one (without: 3400), and blocks start seldom (runs of 8: 3000).
// The Weyl rule is less arithmetic: 2705 us, 6580 GB/s (98 %), 70 % of the issue slots; 112M bf16
// weights without masters, bound by issue, 242 us against 285.
template <bool kNarrow, bool kWeyl>
__global__ void __launch_bounds__(kThreads, kResident[kNarrow]) adamw_kernel(const __grid_constant__ AdamArgs a) {
    pdl_wait();
    // The step's scalars, by one thread: double precision is slow here, and every block pays for it.
    __shared__ float corr[2];
    __shared__ uint32_t step_low;
    State* st = reinterpret_cast<State*>(a.state);
    long long step = 0;
    double c1 = 0.0, c2 = 0.0;
    unsigned ticket = 0;
    if (threadIdx.x == 0) {
        // 1 - beta^(t+1) = beta (1 - beta^t) + (1 - beta)
        c1 = st->c1 * a.beta1 + (1.0 - a.beta1);
        c2 = st->c2 * a.beta2 + (1.0 - a.beta2);
        step = st->step + 1;
        corr[0] = (float)c1;
        corr[1] = (float)c2;
        step_low = (uint32_t)step;
        if (a.advance) {
            __threadfence();                   // the state has been read before the ticket is taken
            ticket = atomicAdd(&st->ticket, 1u);
        }
    }
    // the last tensor whose first run is <= this block's
    const int lo = __syncthreads_count((int)threadIdx.x < a.count && a.first[threadIdx.x] <= blockIdx.x) - 1;
    const float lr = a.lr_dev ? *a.lr_dev : a.lr;
    Step s;
    s.b1 = a.b1;
    s.ob1 = a.ob1;
    s.b2 = a.b2;
    s.ob2 = a.ob2;
    s.rate = -lr / corr[0];
    s.rc2 = 1.f / sqrtf(corr[1]);
    s.eps = a.eps;
    s.gs = a.grad_scale ? *a.grad_scale : 1.f;
    s.dither = step_low * 0x61C88647u;
    if (blockIdx.x < a.runs) {
        const TensorArg& t = a.t[lo];
        s.keep = 1.f - lr * t.decay;
        const int64_t u0 = (int64_t)(blockIdx.x - a.first[lo]) * a.run * 8, whole = t.n / kUnit - u0;
        const int count = (int)min((int64_t)a.run * 8, whole);
        using B = __nv_bfloat16;
        switch (t.kind) {
            case 0: run_units<float, float, false, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 1: run_units<B, float, false, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 2: run_units<float, B, false, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 3: run_units<B, B, false, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 4: run_units<float, float, true, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 5: run_units<B, float, true, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            case 6: run_units<float, B, true, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
            default: run_units<B, B, true, kNarrow, kWeyl>(t, s, u0, count, a.run); break;
        }
        // the unit that the tensor's end cuts short
        if (t.n % kUnit && whole < (int64_t)a.run * 8 && (int)(threadIdx.x >> 5) == (int)(whole & 7))
            last_unit<kNarrow, kWeyl>(t, s, u0 + whole, threadIdx.x & 31);
    }
    // the last block to take a ticket counts the step: every block has read the old count by then
    if (threadIdx.x == 0 && a.advance && ticket == gridDim.x - 1) {
        st->c1 = c1;
        st->c2 = c2;
        st->step = step;
        st->ticket = 0;
    }
}

// The step's count as a launch of its own, after all others.
__global__ void adamw_count_kernel(unsigned char* state, double beta1, double beta2) {
    pdl_wait();
    State* st = reinterpret_cast<State*>(state);
    st->c1 = st->c1 * beta1 + (1.0 - beta1);
    st->c2 = st->c2 * beta2 + (1.0 - beta2);
    st->step += 1;
}

bool misaligned(const void* p, unsigned bytes) { return (reinterpret_cast<uintptr_t>(p) & (bytes - 1)) != 0; }

moe_status_t check_adamw(const moe_adamw_config_t* c, const moe_adamw_tensor_t* ts, int32_t count) {
    if (!c || count < 0 || (count > 0 && !ts)) return MOE_ERR_INVALID_ARG;
    if (!std::isfinite(c->lr) || !(c->beta1 >= 0.0 && c->beta1 < 1.0) || !(c->beta2 >= 0.0 && c->beta2 < 1.0) ||
        !(c->eps >= 1e-30 && c->eps <= 1e30) || c->reserved != 0 ||
        (c->rounding != MOE_ADAMW_ROUND_EVEN && c->rounding != MOE_ADAMW_ROUND_WEYL))
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
    // fp32 and 8-bit states go to launches of their own
    int64_t units[2] = {0, 0};
    for (int k = 0; k < count; ++k) units[tensors[k].m_scale != nullptr] += (tensors[k].n + kUnit - 1) / kUnit;
    const int launches[2] = {units[0] > 0 || units[1] == 0, units[1] > 0};
    for (int narrow = 0; narrow < 2; ++narrow) {
        if (!launches[narrow]) continue;
        const auto kernel = !narrow ? adamw_kernel<false, false>
                            : cfg->rounding == MOE_ADAMW_ROUND_WEYL ? adamw_kernel<true, true> : adamw_kernel<true, false>;
        // Runs that fill whole rounds of the SMs, as few as the longest run allows, with a block more to
        // each tensor for its last, short run. A block's start (parameters, state, first loads) costs
        // what several units do: 29M weights with 8-bit states 98 us in 1.3 rounds, 93 in ten.
        const int64_t slots = (int64_t)num_sms() * kResident[narrow], per_slot = (units[narrow] + 8 * slots - 1) / (8 * slots);
        const int64_t rounds = std::max<int64_t>(1, (per_slot + kRun[narrow] - 1) / kRun[narrow]);
        const int64_t blocks = std::max<int64_t>(rounds * slots - std::min<int64_t>(count, slots / 2), 1);
        a.run = (int)std::min<int64_t>(kRun[narrow], std::max<int64_t>(1, (units[narrow] + 8 * blocks - 1) / (8 * blocks)));
        if (units[narrow] / (8 * a.run) + count > INT32_MAX) return MOE_ERR_UNSUPPORTED;
        int i = 0;
        bool last = false;
        while (!last) {
            a.count = 0;
            a.runs = 0;
            for (; i < count && a.count < kBatch; ++i) {
                const moe_adamw_tensor_t& t = tensors[i];
                if (t.n == 0 || (t.m_scale != nullptr) != (narrow != 0)) continue;
                a.first[a.count] = a.runs;
                a.t[a.count] = {t.p, t.g, t.master, t.m, t.v, t.m_scale, t.v_scale, t.n, t.weight_decay,
                                (t.dtype == MOE_BF16 ? 1 : 0) | (t.grad_dtype == MOE_BF16 ? 2 : 0) | (t.master ? 4 : 0)};
                const int64_t per = (int64_t)kUnit * 8 * a.run;
                a.runs += (uint32_t)((t.n + per - 1) / per);
                ++a.count;
            }
            last = i == count;
            // Many blocks would queue at the ticket (20 ns each); few are done sooner with it than a
            // second launch takes.
            const bool ends = last && (narrow || !launches[1]), apart = a.runs > kTicket;
            a.advance = ends && !apart;
            const cudaError_t e = launch_pdl(kernel,
                                             dim3(std::max(1u, a.runs)), dim3(kThreads), 0, (cudaStream_t)stream, a);
            count_launch();
            if (e != cudaSuccess) return MOE_ERR_CUDA;
            if (ends && apart) {
                const cudaError_t f = launch_pdl(adamw_count_kernel, dim3(1), dim3(1), 0, (cudaStream_t)stream,
                                                 a.state, a.beta1, a.beta2);
                count_launch();
                if (f != cudaSuccess) return MOE_ERR_CUDA;
            }
        }
    }
    return MOE_OK;
}
