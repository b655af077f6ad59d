// Orthogonalised updates of stacks of matrices (Muon): momentum, Newton-Schulz products on CTA pairs
// (tcgen05.mma.cta_group::2, tiles of 256 rows, 64 to 256 columns and 64 k of fp16 operands), and the step on the
// weights.
//
// With A = X X^T (X^T X where there are more rows than columns: the smaller side), one step is
//   gram:  A                                   symmetric
//   poly:  B = a I + b A + c A A               symmetric
//   apply: X = B X   (X B)
// Of the symmetric two only the tiles on and below the diagonal are computed; each is stored twice, once
// as it is and once turned. Where both operands of a square tile are the same rows, they are loaded once.
//
// Operands are fp16, not bf16: the tensor cores take both at one rate, and all of the factors are
// bounded (singular values of X are 1 at most and stay near it), so bf16's range buys nothing and fp16's
// three more bits make the rounding of one operand 2^-12 of it. X and A are held times 2^11 and B times
// 2^10, so that what is far smaller than the largest elements keeps its bits too. In MOE_F32 precision an
// operand is two fp16 planes, x = hi + lo, and a product takes hi hi + hi lo + lo hi.
//
// X is kept in two parts in MOE_BF16 precision too. A rounding of X stands in all directions, also in those that u
// does not have, and the steps that follow multiply small singular values by a each: with 11 bits of X a matrix of
// 512 x 1024 is off by 8e-4 of its size at full rank, but by 1.4e-2 at rank 128 and by 0.1 at rank 1 (simulated;
// gradients of experts that few tokens reached are such matrices). So D X takes both parts, and so does the product
// (B - D) X in all steps but the last two, as a second run over K; A and B, whose roundings reach u's own directions
// only, stay in one. That leaves 1e-3 at any rank (simulated, 129 x 129 to 700 x 720: 1.1e-3 at most for products of
// random factors, 1.9e-3 where a few rows alone are not zero, 2.4e-3 for a matrix of ones; with the low part in D X
// only 3.7e-3, 4.5e-2 and 8.6e-3; in the product of the first two steps, too, 2.6e-3, 4e-3 and 3.7e-3; of all five
// 1.1e-3, 1.8e-3 and 3.3e-3). Measured: 16 x 4096 x 1024 a step 1.27 ms and, so, 1.60.
//
// The diagonal of B, which is near a = 3.4 where the rest is small, is not rounded with it: it stays in fp32 and
// multiplies X in the epilogue of the product, B X = (B - D) X + D X. (Rounded, it is off by up to 2^-12 in one
// direction in all rows alike: 2.7e-3 of the result for 35 x 3195 instead of 1.3e-3, simulated. And most of a
// product goes past the tensor cores' sums, which cut off.)
#include <cmath>
#include <type_traits>

#include "tc_gemm_common.cuh"
#include "tc_pair_ptx.cuh"

#include <cuda_fp16.h>

namespace moe {

namespace {

constexpr int kTile = 256, kHalf = 128;              // tile of a pair, rows of a CTA
constexpr int kPartBytes = kHalf * BK * 2;           // 16 KB: a CTA's rows of A
constexpr int kRingBytes = 12 * kPartBytes;          // the stages
// A stage holds a k-block of the CTA's rows of A and of its half of B's nt columns, in one part or two.
constexpr int stage_bytes(int nt, bool split) { return (split ? 2 : 1) * (kPartBytes + nt / 2 * BK * 2); }
constexpr int kEpiWarps = 8;
constexpr int kGemmThreads = 64 + 32 * kEpiWarps;
constexpr int kSegment = 2;                          // k-blocks (of 64) to a partial sum, with SPLIT
constexpr float kXScale = 2048.f, kAScale = 2048.f, kBScale = 1024.f;

enum Op : int { kGram = 0, kPoly = 1, kApply = 2 };

struct MuonGemm {
    int count, M, N, K;           // per matrix: out [M, N], reduction K
    int n_tiles, tiles;           // of a row of tiles; of one matrix
    const uint16_t* side;         // [planes][count][M, ld]: poly: A; apply: X (2 planes)
    int ld;
    int twice;                    // apply, one part: X's low part is multiplied, too (before the high one)
    float* diag;                  // [count][dstride]: poly writes B's diagonal, apply reads it
    int dstride;
    const uint16_t* weights;      // last product with bf16 output: what it steps [count, M, N] (null: o is written)
    float gain;                   // last product: o = gain X
    float alpha, beta, a;         // poly: B = alpha acc + beta side + a I; others: alpha acc (+ D X)
    const float* lr_dev;          // (last product)
    float lr, decay, scale;       // scale includes 1 / kXScale
    int* err;
};

// ---- 3D tensors [planes * count, rows, cols]
__device__ __forceinline__ void tma_load_3d_pair(uint32_t dst, const CUtensorMap* tm, int x, int y, int z,
                                                 uint32_t mbar_cluster) {
    asm volatile(
        "cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes [%0], [%1, {%2, %3, %4}], [%5];"
        ::"r"(dst), "l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(mbar_cluster)
        : "memory");
}
__device__ __forceinline__ void tma_store_3d(const CUtensorMap* tm, uint32_t src, int x, int y, int z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%1, %2, %3}], [%4];"
                 ::"l"(reinterpret_cast<uint64_t>(tm)), "r"(x), "r"(y), "r"(z), "r"(src) : "memory");
}
// kind::f16, fp16 operands, fp32 sums.
__host__ __device__ constexpr uint32_t idesc_fp16(int M, int N, bool a_mn, bool b_mn) {
    return (1u << 4) | ((a_mn ? 1u : 0u) << 15) | ((b_mn ? 1u : 0u) << 16) | ((uint32_t)(N >> 3) << 17) |
           ((uint32_t)(M >> 4) << 24);
}

struct MuonTile {
    int z, m0, n0;
};
// Tile r of a matrix: row-major, or for the symmetric products the tiles on and below the diagonal, one
// row of tiles after another.
template <bool SYM, int NT>
__device__ __forceinline__ MuonTile decode_tile(const MuonGemm& p, int tile) {
    constexpr int R = kTile / NT;      // tiles to a square
    MuonTile t;
    t.z = tile / p.tiles;
    const int r = tile - t.z * p.tiles;
    int i, j;
    if (SYM) {
        const int q = r / R;
        i = (int)((sqrtf(8.0f * (float)q + 1.0f) - 1.0f) * 0.5f);
        while (i * (i + 1) / 2 > q) --i;
        while ((i + 1) * (i + 2) / 2 <= q) ++i;
        j = r - R * (i * (i + 1) / 2);
    } else {
        i = r / p.n_tiles;
        j = r - i * p.n_tiles;
    }
    t.m0 = i * kTile;
    t.n0 = j * NT;
    return t;
}

__device__ __forceinline__ uint32_t pack_half2(float lo, float hi) {
    const __half2 h = __floats2half2_rn(lo, hi);
    return *reinterpret_cast<const uint32_t*>(&h);
}

// One epilogue warp's two staging buffers of 32 rows x 64 bytes (64-byte swizzle).
struct Staging {
    uint32_t base;
    int count;
    __device__ __forceinline__ uint32_t acquire(int lane) {
        if (lane == 0 && count >= 2) bulk_wait_read1();
        __syncwarp();
        return base + (count & 1) * STG_BYTES;
    }
    __device__ __forceinline__ void release(int lane, uint32_t buf, const CUtensorMap* tm, int x, int y, int z) {
        fence_async_smem();
        __syncwarp();
        if (lane == 0) {
            tma_store_3d(tm, buf, x, y, z);
            bulk_commit();
        }
        ++count;
    }
    // 16-byte units that were read in order (lane l: unit l & 3 of rows l / 4 + 8 i) to the lane's own row.
    __device__ __forceinline__ void to_rows(int lane, uint4 (&r)[4]) {
        const uint32_t buf = acquire(lane);
#pragma unroll
        for (int i = 0; i < 4; ++i) sts128(sw64_addr(buf, (lane >> 2) + 8 * i, lane & 3), r[i]);
        __syncwarp();
#pragma unroll
        for (int j = 0; j < 4; ++j) r[j] = lds128(sw64_addr(buf, lane, j));
        __syncwarp();
    }
    // h[i]: columns 2i and 2i + 1 of the lane's row
    __device__ __forceinline__ void store(int lane, const uint32_t (&h)[16], const CUtensorMap* tm, int x, int y, int z) {
        const uint32_t buf = acquire(lane);
#pragma unroll
        for (int j = 0; j < 4; ++j)
            sts128(sw64_addr(buf, lane, j), make_uint4(h[4 * j], h[4 * j + 1], h[4 * j + 2], h[4 * j + 3]));
        release(lane, buf, tm, x, y, z);
    }
    // The box turned: even lanes write the words (rows l, l + 1) of column 2i, odd ones of column 2i + 1.
    __device__ __forceinline__ void store_turned(int lane, const uint32_t (&h)[16], const CUtensorMap* tm, int x, int y,
                                                 int z) {
        const uint32_t buf = acquire(lane);
        const int odd = lane & 1, word = lane >> 1;
#pragma unroll
        for (int i = 0; i < 16; ++i) {
            const uint32_t other = __shfl_xor_sync(0xffffffffu, h[i], 1);
            const uint32_t v = odd ? __byte_perm(other, h[i], 0x7632) : __byte_perm(h[i], other, 0x5410);
            const uint32_t addr = sw64_addr(buf, 2 * i + odd, word >> 2) + (word & 3) * 4;
            asm volatile("st.shared.b32 [%0], %1;" ::"r"(addr), "r"(v) : "memory");
        }
        release(lane, buf, tm, x, y, z);
    }
};

// What the product's epilogue makes of X: fp16 parts for the next step, or, where rows are whole 16-byte units,
// the bf16 result itself, o or stepped weights (apart, 320 us of 7900 for 128 x 1024 x 4096).
enum Out : int { kParts = 0, kResult = 1 };

// out = alpha P Q + beta side + a I on CTA pairs; the pipeline and its barriers are those of the grouped
// expert GEMMs.
//
// SPLIT: the tensor cores cut off their sums at 24 bits with every addition, which over a long K is far more
// than 22-bit operands leave. So K is taken in segments, of kSegment k-blocks in the widest tiles (4 x 2048 x 1024:
// 722 us, with one 892) and of one in the others, which do not fill the tensor cores (416 x 768: 2.2e-6 of the
// result, where segments of two left 3.7e-6; plain fp32 products 2.2e-6). Each segment has a TMEM buffer to itself, lo hi
// and hi lo before hi hi (what is cut off is measured by what the sum holds: one k-block's three products after
// the other's, 4.5e-6), and the epilogue warps add the segments up in registers, rounding to nearest, while the
// next buffer fills. A stage has all four parts of its k-block (loaded for each product anew, 6 in place of 4:
// 1024 x 4096 in tiles of 64 columns 701 us, so 608).
template <int OP, bool A_MN, bool B_MN, bool SPLIT, int OUT, int NT>
__global__ void __cluster_dims__(2, 1, 1) __launch_bounds__(kGemmThreads, 1)
muon_gemm_kernel(const MuonGemm p, const __grid_constant__ CUtensorMap tmA, const __grid_constant__ CUtensorMap tmB,
                 const __grid_constant__ CUtensorMap tmO) {
    constexpr bool SYM = OP != kApply, SIDED = OP != kGram, TALL = OP == kApply && !B_MN;
    constexpr bool TWO = SPLIT || OP == kApply;      // side input and output in two parts
    constexpr int PL = SPLIT ? 2 : 1, B_BYTES = NT / 2 * BK * 2, STAGE = stage_bytes(NT, SPLIT), STAGES = kRingBytes / STAGE;
    constexpr int BUFS = NT == kTile ? 2 : 4;      // sums in TMEM (1024 x 1024 in two parts: 295 us with 2, 263 with 4)
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* stg_smem = smem + kRingBytes;
    uint64_t* full = reinterpret_cast<uint64_t*>(stg_smem + kEpiWarps * 2 * STG_BYTES);
    uint64_t* empty = full + STAGES;
    uint64_t* tfull = empty + STAGES;
    uint64_t* tempty = tfull + BUFS;
    uint64_t* drain = tempty + BUFS;
    uint32_t* tmem_slot = reinterpret_cast<uint32_t*>(drain + 1);
    volatile int* s_fail = reinterpret_cast<volatile int*>(tmem_slot + 1);

    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const uint32_t rank = cluster_rank();
    const bool leader = (rank == 0);
    const int cluster_id = blockIdx.x >> 1, nclusters = gridDim.x >> 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < STAGES; ++s) { mbar_init(full + s, 1); mbar_init(empty + s, 1); }
        for (int b = 0; b < BUFS; ++b) { mbar_init(tfull + b, 1); mbar_init(tempty + b, 2 * 32 * kEpiWarps); }
        mbar_init(drain, 1);
        *s_fail = 0;
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0 && lane == 0) { tma_prefetch_desc(&tmA); tma_prefetch_desc(&tmB); tma_prefetch_desc(&tmO); }
    if (warp == 1) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     ::"r"(smem_u32(tmem_slot)), "r"(TMEM_COLS) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    }
    pdl_wait();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    cluster_sync();   // both CTAs' barriers exist before any remote arrive or complete_tx
    const uint32_t tmem_base = *tmem_slot;
    const int num_tiles = p.count * p.tiles;
    const int kblocks1 = (p.K + BK - 1) / BK;
    const bool twice = OP == kApply && !SPLIT && p.twice;
    const int kblocks = twice ? 2 * kblocks1 : kblocks1;
    const int seg = SPLIT ? (NT == kTile ? kSegment : 1) : kblocks;      // k-blocks to an accumulator

    if (warp == 0) {
        if (lane == 0) {
            uint32_t s = 0, ph = 0;
            long long issued = 0;
            bool ok = true;
            for (int tile = cluster_id; tile < num_tiles && ok; tile += nclusters) {
                const MuonTile t = decode_tile<SYM, NT>(p, tile);
                const int mr = t.m0 + (int)rank * kHalf, nh = t.n0 + (int)rank * (NT / 2);
                const bool same = SYM && !SPLIT && NT == kTile && t.m0 == t.n0;
                for (int kb = 0; kb < kblocks; ++kb) {
                    if (!mbar_wait(empty + s, ph ^ 1, p.err)) { ok = false; break; }
                    const uint32_t sa = smem_u32(smem + s * STAGE), sb = sa + PL * kPartBytes;
                    const uint32_t fb = map_to_rank(smem_u32(full + s), 0);
                    if (leader) mbar_expect_tx(full + s, same ? 2 * kPartBytes : 2 * STAGE);
                    const bool low = twice && kb < kblocks1;       // of X: the left operand of X B, the right one of B X
                    const int k0 = (twice && !low ? kb - kblocks1 : kb) * BK;
#pragma unroll
                    for (int part = 0; part < PL; ++part) {
                        const int za = t.z + (part + (TALL && low)) * p.count, zb = t.z + (part + (!TALL && low)) * p.count;
                        if (!A_MN) {
                            tma_load_3d_pair(sa + part * kPartBytes, &tmA, k0, mr, za, fb);
                        } else {
#pragma unroll
                            for (int j = 0; j < kHalf / 64; ++j)
                                tma_load_3d_pair(sa + part * kPartBytes + j * (BK * 128), &tmA, mr + 64 * j, k0, za, fb);
                        }
                        if (same) {
                        } else if (!B_MN) {
                            tma_load_3d_pair(sb + part * B_BYTES, &tmB, k0, nh, zb, fb);
                        } else {
#pragma unroll
                            for (int j = 0; j < NT / 128; ++j)
                                tma_load_3d_pair(sb + part * B_BYTES + j * (BK * 128), &tmB, nh + 64 * j, k0, zb, fb);
                        }
                    }
                    ++issued;
                    if (++s == STAGES) { s = 0; ph ^= 1; }
                }
            }
            if (!ok) {
                *s_fail = 1;
                // no copy may be in flight when the CTAs leave: the stages issued last, oldest first
                const long long n = issued < STAGES ? issued : STAGES;
                for (long long i = issued - n; i < issued && leader; ++i)
                    if (!mbar_wait(full + (int)(i % STAGES), (uint32_t)(i / STAGES) & 1u, p.err)) break;
            }
        }
    } else if (warp == 1) {
        if (leader && lane == 0) {
            const uint32_t idesc = idesc_fp16(kTile, NT, A_MN, B_MN);
            const uint32_t s0 = smem_u32(smem);
            const uint64_t a_desc0 = A_MN ? make_desc(s0, BK * 128, 1024) : make_desc(s0, 16, 1024);
            const uint32_t b0 = s0 + PL * kPartBytes;
            const uint64_t b_desc0 = B_MN ? make_desc(b0, BK * 128, 1024) : make_desc(b0, 16, 1024);
            constexpr uint32_t A_KSTEP = (A_MN ? UMMA_K * 128 : UMMA_K * 2) >> 4;
            constexpr uint32_t B_KSTEP = (B_MN ? UMMA_K * 128 : UMMA_K * 2) >> 4;
            constexpr uint32_t STAGE_STEP = STAGE >> 4;
            uint32_t s = 0, ph = 0, soff = 0, tl = 0;
            bool ok = true;
            for (int tile = cluster_id; tile < num_tiles && ok; tile += nclusters)
            for (int first = 0; first < kblocks && ok; first += seg) {
                const int buf = tl % BUFS;
                const uint32_t aph = (tl / BUFS) & 1;
                ++tl;
                if (!mbar_wait(tempty + buf, aph ^ 1, p.err)) { ok = false; break; }
                tc_fence_after();
                const uint32_t d_tmem = tmem_base + buf * NT;
                const MuonTile t = decode_tile<SYM, NT>(p, tile);
                const uint64_t b_desc = SYM && !SPLIT && NT == kTile && t.m0 == t.n0 ? a_desc0 : b_desc0;
                const int steps = min(seg, kblocks - first);
                // one part of A times one of B, of the k-block in the stage at `off`
                auto product = [&](uint32_t off, int term, bool add) {      // term: lo hi, hi lo, hi hi
                    const uint64_t ad = a_desc0 + off + (term == 0 ? kPartBytes >> 4 : 0);
                    const uint64_t bd = b_desc + off + (term == 1 ? B_BYTES >> 4 : 0);
#pragma unroll
                    for (int kk = 0; kk < BK / UMMA_K; ++kk)
                        mma_pair(d_tmem, ad + kk * A_KSTEP, bd + kk * B_KSTEP, idesc, add || kk > 0 ? 1u : 0u);
                };
                auto forward = [&]() {
                    if (++s == STAGES) { s = 0; ph ^= 1; soff = 0; } else { soff += STAGE_STEP; }
                };
                if constexpr (SPLIT) {
                    uint32_t back = s, boff = soff;       // the segment's first stage
                    for (int q = 0; q < steps; ++q) {
                        if (!mbar_wait(full + s, ph, p.err)) { ok = false; break; }
                        tc_fence_after();
                        product(soff, 0, q > 0);
                        product(soff, 1, true);
                        forward();
                    }
                    for (int q = 0; q < steps && ok; ++q) {
                        product(boff, 2, true);
                        commit_pair_both(empty + back);
                        if (++back == STAGES) { back = 0; boff = 0; } else { boff += STAGE_STEP; }
                    }
                } else {
                    for (int q = 0; q < steps; ++q) {
                        if (!mbar_wait(full + s, ph, p.err)) { ok = false; break; }
                        tc_fence_after();
                        product(soff, 2, q > 0);
                        commit_pair_both(empty + s);
                        forward();
                    }
                }
                if (!ok) break;
                commit_pair_both(tfull + buf);
            }
            if (!ok) *s_fail = 1;
            commit_pair_local(drain);
            mbar_wait(drain, 0, p.err);
        }
    } else {
        const int quarter = warp & 3, half = (warp - 2) >> 2;
        const float lr = OUT == kResult && p.lr_dev ? __ldg(p.lr_dev) : p.lr, lose = lr * p.decay, move = lr * p.scale;
        Staging st{smem_u32(stg_smem + (warp - 2) * 2 * STG_BYTES), 0};
        const uint32_t tempty_leader = map_to_rank(smem_u32(tempty), 0);
        uint32_t tl = 0;
        for (int tile = cluster_id; tile < num_tiles; tile += nclusters) {
            const MuonTile t = decode_tile<SYM, NT>(p, tile);
            const int y = t.m0 + (int)rank * kHalf + quarter * 32;    // the warp's first row
            const int x0 = t.n0 + half * (NT / 2);                    // its first column
            const bool turn = SYM && t.n0 < t.m0;
            const uint32_t toff = ((uint32_t)(quarter * 32) << 16) + half * (NT / 2);
            bool ok = true;
            // The side input of a box, fetched a box ahead, in whole sectors (a row of it to a lane took a read of
            // 32 lines for every 16 bytes: stepping weights in the last product then took longer than apart from it).
            auto fetch = [&](const uint16_t* from, int ld, int c, int part, uint4 (&to)[4]) {
                const int row = y + (lane >> 2), col = x0 + c + (lane & 3) * 8;
                const uint16_t* src = from + ((size_t)(t.z + part * p.count) * p.M + row) * ld + col;
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    to[i] = make_uint4(0, 0, 0, 0);
                    if (row + 8 * i < p.M && col < ld) to[i] = __ldcg(reinterpret_cast<const uint4*>(src + (size_t)8 * i * ld));
                }
            };
            uint4 ahead[4], low[4], weights[4];
            if (SIDED) fetch(p.side, p.ld, 0, 0, ahead);
            if (TWO && !SPLIT) fetch(p.side, p.ld, 0, 1, low);
            if (OUT == kResult && p.weights) fetch(p.weights, p.N, 0, 0, weights);
            float drow = 0.f;              // D of the lane's row (X times it on the left)
            if (OP == kApply && !TALL && y + lane < p.M) drow = __ldg(p.diag + (size_t)t.z * p.dstride + y + lane);
            // one box of 32 rows x 32 columns from column x0 + c on, out of its sums
            auto box = [&](int c, const uint32_t (&acc)[32], auto ready) {
                const int x = x0 + c;
                if (x >= p.N || y >= p.M) return;
                float v[32];
                uint4 own[4];
                if (SIDED) {
#pragma unroll
                    for (int i = 0; i < 4; ++i) own[i] = ahead[i];
                    if (c + 32 < NT / 2) fetch(p.side, p.ld, c + 32, 0, ahead);
                    st.to_rows(lane, own);
                    auto add = [&](bool first) {
                        const __half2* h = reinterpret_cast<const __half2*>(own);
#pragma unroll
                        for (int i = 0; i < 16; ++i) {
                            const float2 f = __half22float2(h[i]);
                            v[2 * i] = first ? f.x : v[2 * i] + f.x;
                            v[2 * i + 1] = first ? f.y : v[2 * i + 1] + f.y;
                        }
                    };
                    add(true);
                    if (TWO) {
                        if (SPLIT) {
                            fetch(p.side, p.ld, c, 1, own);
                        } else {
#pragma unroll
                            for (int i = 0; i < 4; ++i) own[i] = low[i];
                            if (c + 32 < NT / 2) fetch(p.side, p.ld, c + 32, 1, low);
                        }
                        st.to_rows(lane, own);
                        add(false);
                    }
                }
                ready();
                if (OP == kGram) {
#pragma unroll
                    for (int i = 0; i < 32; ++i) v[i] = p.alpha * __uint_as_float(acc[i]);
                } else if (OP == kPoly) {
                    float d = 0.f;
#pragma unroll
                    for (int i = 0; i < 32; ++i) {
                        v[i] = fmaf(p.beta, v[i], p.alpha * __uint_as_float(acc[i]));
                        if (x == y && i == lane) {       // (a box on the diagonal)
                            d = v[i];
                            v[i] = 0.f;
                        }
                    }
                    if (x == y && y + lane < p.M) p.diag[(size_t)t.z * p.dstride + y + lane] = fmaf(d, 1.f / kBScale, p.a);
                } else {
                    const float4* dcol = reinterpret_cast<const float4*>(p.diag + (size_t)t.z * p.dstride + x);
#pragma unroll
                    for (int i = 0; i < 32; i += 4) {
                        const float4 d = TALL ? __ldg(dcol + i / 4) : make_float4(drow, drow, drow, drow);
                        v[i] = fmaf(d.x, v[i], p.alpha * __uint_as_float(acc[i]));
                        v[i + 1] = fmaf(d.y, v[i + 1], p.alpha * __uint_as_float(acc[i + 1]));
                        v[i + 2] = fmaf(d.z, v[i + 2], p.alpha * __uint_as_float(acc[i + 2]));
                        v[i + 3] = fmaf(d.w, v[i + 3], p.alpha * __uint_as_float(acc[i + 3]));
                    }
                }
                uint32_t h[16];
                if (OUT == kResult) {
                    if (p.weights) {
#pragma unroll
                        for (int i = 0; i < 4; ++i) own[i] = weights[i];
                        if (c + 32 < NT / 2) fetch(p.weights, p.N, c + 32, 0, weights);
                        st.to_rows(lane, own);
                        float w[32];
#pragma unroll
                        for (int j = 0; j < 4; ++j) unpack8(own[j], w + 8 * j);
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] = fmaf(-move, v[i], fmaf(-lose, w[i], w[i]));
                    } else {
#pragma unroll
                        for (int i = 0; i < 32; ++i) v[i] *= p.gain;
                    }
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const __nv_bfloat162 b = __floats2bfloat162_rn(v[2 * i], v[2 * i + 1]);
                        h[i] = *reinterpret_cast<const uint32_t*>(&b);
                    }
                    st.store(lane, h, &tmO, x, y, t.z);
                    return;
                }
#pragma unroll
                for (int i = 0; i < 16; ++i) h[i] = pack_half2(v[2 * i], v[2 * i + 1]);
                st.store(lane, h, &tmO, x, y, t.z);
                if (turn) st.store_turned(lane, h, &tmO, y, x, t.z);
                if (TWO) {
#pragma unroll
                    for (int i = 0; i < 16; ++i) {
                        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
                        h[i] = pack_half2(v[2 * i] - f.x, v[2 * i + 1] - f.y);
                    }
                    st.store(lane, h, &tmO, x, y, t.z + p.count);
                    if (turn) st.store_turned(lane, h, &tmO, y, x, t.z + p.count);
                }
            };
            auto wait_full = [&]() {
                const bool got = mbar_wait(tfull + tl % BUFS, (tl / BUFS) & 1, p.err);
                tc_fence_after();
                return got;
            };
            auto free_buffer = [&]() {
                tc_fence_before();
                if (leader) mbar_arrive(tempty + tl % BUFS);
                else mbar_arrive_cluster(tempty_leader + tl % BUFS * 8);
                ++tl;
            };
            if constexpr (SPLIT) {
                uint32_t sum[NT / 64][32];
#pragma unroll
                for (int c = 0; c < NT / 64; ++c)
#pragma unroll
                    for (int i = 0; i < 32; ++i) sum[c][i] = 0;
                for (int first = 0; first < kblocks; first += seg) {
                    if (!wait_full()) { ok = false; break; }
                    const uint32_t taddr = tmem_base + toff + tl % BUFS * NT;
#pragma unroll
                    for (int c = 0; c < NT / 64; ++c) {
                        uint32_t acc[32];
                        tmem_ld32(taddr + 32 * c, acc);
                        tmem_ld_wait_regs(acc);
#pragma unroll
                        for (int i = 0; i < 32; ++i)
                            sum[c][i] = __float_as_uint(__uint_as_float(sum[c][i]) + __uint_as_float(acc[i]));
                    }
                    free_buffer();
                }
                if (!ok) break;
#pragma unroll
                for (int c = 0; c < NT / 64; ++c) box(32 * c, sum[c], [] {});
            } else {
                if (!wait_full()) break;
                const uint32_t taddr = tmem_base + toff + tl % BUFS * NT;
                for (int c = 0; c < NT / 2; c += 32) {
                    if (x0 + c >= p.N || y >= p.M) break;
                    uint32_t acc[32];
                    tmem_ld32(taddr + c, acc);
                    box(c, acc, [&] { tmem_ld_wait_regs(acc); });
                }
                free_buffer();
            }
            if (*s_fail) break;
        }
        if (lane == 0) bulk_wait_all();
        __syncwarp();
    }

    tc_fence_before();
    __syncthreads();
    cluster_sync();   // all work of both CTAs is done before the pair releases its TMEM
    tc_fence_after();
    if (warp == 1) {
        __syncwarp();
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" ::"r"(tmem_base), "r"(TMEM_COLS)
                     : "memory");
    }
}

constexpr size_t kGemmSmem = 1024 + (size_t)kRingBytes + kEpiWarps * 2 * STG_BYTES + 32 * sizeof(uint64_t);
static_assert(kGemmSmem <= 227 * 1024, "shared memory per CTA");

// ---------------------------------------------------------------- before the products
struct MuonPrep {
    const void* g;
    float* m;                 // momentum, or null (orthogonalize)
    const float* grad_scale;
    float* sums;              // [count, chunks] partial sums of squares
    __half* X;                // [2, count, rows, ld]
    int64_t n, chunk;         // elements of a matrix, of a chunk
    int chunks, count, rows, cols, ld;
    float momentum, eps;
    int nesterov;
};

constexpr int kPrepThreads = 256;

// V elements of the gradient from element i of a matrix on.
template <typename G, int V>
__device__ __forceinline__ void load_v(const G* p, float (&f)[V]) {
    if constexpr (V == 1) {
        f[0] = Elem<G>::to_f(*p);
    } else {
        static_assert(V == 8, "");
        if constexpr (sizeof(G) == 2) {
            load16(p, f);
        } else {
            load16(p, f);
            load16(p + 4, f + 4);
        }
    }
}

// The gradient and momentum of V elements, and u = g (+ momentum); the first pass writes the momentum.
template <typename G, int V, bool MOMENTUM>
struct Update {
    static constexpr int NG = V == 1 ? 1 : V * (int)sizeof(G) / 16;
    G one;                    // V = 1
    uint4 g[NG];              // V = 8, as it is in memory
    float m[MOMENTUM ? V : 1];
    __device__ __forceinline__ void load(const MuonPrep& a, int64_t at) {
        const G* p = static_cast<const G*>(a.g) + at;
        if constexpr (V == 1) {
            one = *p;
            if (MOMENTUM) m[0] = a.m[at];
        } else {
#pragma unroll
            for (int q = 0; q < NG; ++q) g[q] = __ldg(reinterpret_cast<const uint4*>(p) + q);
            if constexpr (MOMENTUM) {
#pragma unroll
                for (int q = 0; q < V; q += 4) *reinterpret_cast<float4*>(m + q) = *reinterpret_cast<const float4*>(a.m + at + q);
            }
        }
    }
    template <bool FIRST>
    __device__ __forceinline__ void step(const MuonPrep& a, int64_t at, float gs, float (&u)[V]) {
        if constexpr (V == 1) {
            u[0] = Elem<G>::to_f(one);
        } else {
#pragma unroll
            for (int q = 0; q < NG; ++q) unpack16<G>(g[q], u + q * (16 / (int)sizeof(G)));
        }
        if constexpr (MOMENTUM) {
#pragma unroll
            for (int q = 0; q < V; ++q) {
                u[q] *= gs;
                if (FIRST) m[q] = fmaf(a.momentum, m[q], u[q]);
            }
            if constexpr (FIRST && V == 1) a.m[at] = m[0];
            if constexpr (FIRST && V > 1) {
#pragma unroll
                for (int q = 0; q < V; q += 4) *reinterpret_cast<float4*>(a.m + at + q) = *reinterpret_cast<float4*>(m + q);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) u[q] = a.nesterov ? fmaf(a.momentum, m[q], u[q]) : m[q];
        }
    }
};
// Vectors that a thread has in flight. (One, with 2048 threads to an SM, read 4 TB/s.)
template <bool MOMENTUM> constexpr int kAhead = MOMENTUM ? 2 : 4;

// First pass: momentum, and the sum of squares of each chunk of a matrix.
template <typename G, int V, bool MOMENTUM>
__global__ void __launch_bounds__(kPrepThreads, 4) muon_sums_kernel(const MuonPrep a) {
    constexpr int U = kAhead<MOMENTUM>;
    __shared__ float s_sum[kPrepThreads / 32];
    pdl_wait();
    const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f;
    for (int64_t w = blockIdx.x; w < (int64_t)a.count * a.chunks; w += gridDim.x) {
        const int64_t z = w / a.chunks, c = w - z * a.chunks;
        const int64_t end = min(a.n, (c + 1) * a.chunk);
        float sum = 0.f;
        for (int64_t i = c * a.chunk + threadIdx.x * V; i < end; i += kPrepThreads * V * U) {
            Update<G, V, MOMENTUM> x[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i + k * kPrepThreads * V < end) x[k].load(a, z * a.n + i + k * kPrepThreads * V);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                if (i + k * kPrepThreads * V >= end) break;
                float u[V];
                x[k].template step<true>(a, z * a.n + i + k * kPrepThreads * V, gs, u);
                float part = 0.f;
#pragma unroll
                for (int q = 0; q < V; ++q) part = fmaf(u[q], u[q], part);
                sum += part;
            }
        }
        sum = warp_sum(sum);
        if ((threadIdx.x & 31) == 0) s_sum[threadIdx.x >> 5] = sum;
        __syncthreads();
        if (threadIdx.x == 0) {
            for (int i = 1; i < kPrepThreads / 32; ++i) sum += s_sum[i];
            a.sums[w] = sum;
        }
        __syncthreads();
    }
}

// Second pass: X = u / (|u| + eps), in fp16 parts.
template <typename G, int V, bool MOMENTUM>
__global__ void __launch_bounds__(kPrepThreads, 4) muon_scale_kernel(const MuonPrep a) {
    constexpr int U = kAhead<MOMENTUM>;
    __shared__ float s_scale;
    pdl_wait();
    const float gs = a.grad_scale ? __ldg(a.grad_scale) : 1.f;
    const size_t plane = (size_t)a.count * a.rows * a.ld;
    for (int64_t w = blockIdx.x; w < (int64_t)a.count * a.chunks; w += gridDim.x) {
        const int64_t z = w / a.chunks, c = w - z * a.chunks;
        if (threadIdx.x < 32) {
            float sum = 0.f;
            for (int i = threadIdx.x; i < a.chunks; i += 32) sum += a.sums[z * a.chunks + i];
            sum = warp_sum(sum);
            const float norm = sqrtf(sum) + a.eps;
            if (threadIdx.x == 0) s_scale = sum < INFINITY ? kXScale / norm : NAN;
        }
        __syncthreads();
        const float scale = s_scale;
        const int64_t end = min(a.n, (c + 1) * a.chunk);
        for (int64_t i0 = c * a.chunk + threadIdx.x * V; i0 < end; i0 += kPrepThreads * V * U) {
            Update<G, V, MOMENTUM> x[U];
#pragma unroll
            for (int k = 0; k < U; ++k)
                if (i0 + k * kPrepThreads * V < end) x[k].load(a, z * a.n + i0 + k * kPrepThreads * V);
#pragma unroll
            for (int k = 0; k < U; ++k) {
                const int64_t i = i0 + k * kPrepThreads * V;
                if (i >= end) break;
                float u[V];
                x[k].template step<false>(a, z * a.n + i, gs, u);
                int64_t at;
                if constexpr (V == 8) {
                    at = z * a.n + i;           // cols % 8 = 0: ld = cols
                } else {
                    const int r = (int)(i / a.cols);
                    at = (z * a.rows + r) * a.ld + (i - (int64_t)r * a.cols);
                }
                __half hi[V], lo[V];
#pragma unroll
                for (int q = 0; q < V; ++q) {
                    const float y = u[q] * scale;
                    hi[q] = __float2half_rn(y);
                    lo[q] = __float2half_rn(y - __half2float(hi[q]));
                }
                if constexpr (V == 8) {
                    *reinterpret_cast<uint4*>(a.X + at) = *reinterpret_cast<uint4*>(hi);
                    *reinterpret_cast<uint4*>(a.X + plane + at) = *reinterpret_cast<uint4*>(lo);
                } else {
                    a.X[at] = hi[0];
                    a.X[plane + at] = lo[0];
                }
            }
        }
        __syncthreads();
    }
}

// ---------------------------------------------------------------- after the products
struct MuonFinish {
    const __half* X;
    void* out;                // o, or p
    float* master;
    const float* lr_dev;
    int64_t n, total;
    int count, rows, cols, ld;
    float lr, decay, scale;
    bool step;                // p is stepped; else o is written
};

template <typename T, int V>
__global__ void __launch_bounds__(256) muon_finish_kernel(const MuonFinish a) {
    pdl_wait();
    const float lr = a.lr_dev ? __ldg(a.lr_dev) : a.lr;
    const float lose = lr * a.decay, move = lr * a.scale * (1.f / kXScale);
    const size_t plane = (size_t)a.count * a.rows * a.ld;
    T* out = static_cast<T*>(a.out);
    for (int64_t i = ((int64_t)blockIdx.x * 256 + threadIdx.x) * V; i < a.total; i += (int64_t)gridDim.x * 256 * V) {
        float x[V];
        if constexpr (V == 8) {
            const uint4 h4 = *reinterpret_cast<const uint4*>(a.X + i);
            const __half* h = reinterpret_cast<const __half*>(&h4);
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] = __half2float(h[q]);
            const uint4 l4 = *reinterpret_cast<const uint4*>(a.X + plane + i);
            const __half* l = reinterpret_cast<const __half*>(&l4);
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] += __half2float(l[q]);
        } else {
            const int64_t row = i / a.cols, at = row * a.ld + (i - row * a.cols);
            x[0] = __half2float(a.X[at]) + __half2float(a.X[plane + at]);
        }
        if (!a.step) {
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] *= 1.f / kXScale;
        } else {
            float p[V];
            if (a.master) {
                if constexpr (V == 8) {
                    *reinterpret_cast<float4*>(p) = *reinterpret_cast<const float4*>(a.master + i);
                    *reinterpret_cast<float4*>(p + 4) = *reinterpret_cast<const float4*>(a.master + i + 4);
                } else {
                    p[0] = a.master[i];
                }
            } else {
                load_v<T, V>(out + i, p);
            }
#pragma unroll
            for (int q = 0; q < V; ++q) x[q] = fmaf(-move, x[q], fmaf(-lose, p[q], p[q]));
            if (a.master) {
                if constexpr (V == 8) {
                    *reinterpret_cast<float4*>(a.master + i) = *reinterpret_cast<float4*>(x);
                    *reinterpret_cast<float4*>(a.master + i + 4) = *reinterpret_cast<float4*>(x + 4);
                } else {
                    a.master[i] = x[0];
                }
            }
        }
        if constexpr (V == 8) {
            if constexpr (sizeof(T) == 2) {
                store16(out + i, x);
            } else {
                store16(out + i, x);
                store16(out + i + 4, x + 4);
            }
        } else {
            st_f(out + i, x[0]);
        }
    }
}

// ---------------------------------------------------------------- small matrices, in one launch
// A matrix of 128 at most on its smaller side and 1024 on the other stays in shared memory from the
// gradient to the update: a cluster of CTAs holds a slice of 128 along the longer side each. Of a step only
// the Gram matrix concerns all of them: each multiplies its slice with itself and sends every CTA its part of
// the rows of the fp32 sums; each adds up its rows over all CTAs, in their order, and sends them, in fp16
// parts, to all. B is then computed by each for itself, and B X is each one's own slice.
//
// Slices and A lie as the tensor cores read 128-byte swizzled tiles: blocks of 64 columns, each of 128 rows
// of 128 bytes. One such block is read along either side: as K-major rows, or as MN-major columns, so the
// products X X^T, X^T X, B X and X B need no copy that is turned. The fp32 sums lie in four such blocks (of 32
// columns), so that the rows of one CTA take the same bytes as fp32 sums and as fp16 parts: a CTA that sends
// its rows of A overwrites only what it has received.
//
// The exchanges wait for no cluster barrier (one that they arrive on is waited for a product later, before B
// takes the place of A, which copies may still read until then). Sums arrive in a buffer of their own, which is read before the rows
// of A that it makes are sent, and no CTA sends sums again before it has all rows of A; rows of A arrive where
// their sums stood, which the sender has.
constexpr int kSide = 128;
constexpr int kPlaneBytes = kSide * kSide * 2;       // one fp16 part of a slice, or of A
constexpr int kBlockBytes = kSide * 128;             // 128 rows of 128 bytes
constexpr int kSmallThreads = 512;
constexpr int kMaxCluster = 8;
constexpr int kUnits = kSide * kSide / 8 / kSmallThreads;   // units of 8 elements to a thread
constexpr int kRecvBytes = 68608;                    // sums of n CTAs' rows: n ceil(128 / n) 512, at most for n = 7

struct MuonSmall {
    MuonPrep pre;
    MuonFinish fin;
    int steps, cluster, side;
    bool g_bf16, p_bf16, vec;     // vec: rows are whole units of 8 elements
    float a, b, c;
    int* err;
};

// Byte of the 16-byte unit u of a row: fp16 parts have 16, fp32 sums 32.
__device__ __forceinline__ uint32_t unit_at(int row, int u) {
    return (uint32_t)((u >> 3) * kBlockBytes + row * 128 + (((u & 7) ^ (row & 7)) << 4));
}
// `bytes` of this CTA's shared memory to another's, counted on a barrier there.
__device__ __forceinline__ void send(uint32_t to, uint32_t from, uint32_t bytes, uint32_t bar) {
    asm volatile("cp.async.bulk.shared::cluster.shared::cta.mbarrier::complete_tx::bytes [%0], [%1], %2, [%3];"
                 ::"r"(to), "r"(from), "r"(bytes), "r"(bar) : "memory");
}
// 8 elements at p (fp32 or bf16) of which the first n exist.
__device__ __forceinline__ void load_unit(const void* p, int64_t at, bool bf16, bool vec, int n, float (&f)[8]) {
    if (vec && n == 8) {
        if (bf16) {
            const uint4 u = *reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(p) + at);
            unpack16<__nv_bfloat16>(u, f);
        } else {
            *reinterpret_cast<float4*>(f) = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at);
            *reinterpret_cast<float4*>(f + 4) = *reinterpret_cast<const float4*>(static_cast<const float*>(p) + at + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            f[i] = i >= n ? 0.f : bf16 ? Elem<__nv_bfloat16>::to_f(static_cast<const __nv_bfloat16*>(p)[at + i])
                                       : static_cast<const float*>(p)[at + i];
    }
}
__device__ __forceinline__ void store_unit(void* p, int64_t at, bool bf16, bool vec, int n, const float (&f)[8]) {
    if (vec && n == 8) {
        if (bf16) {
            store16(static_cast<__nv_bfloat16*>(p) + at, f);
        } else {
            store16(static_cast<float*>(p) + at, f);
            store16(static_cast<float*>(p) + at + 4, f + 4);
        }
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < n) {
                if (bf16) st_f(static_cast<__nv_bfloat16*>(p) + at + i, f[i]);
                else static_cast<float*>(p)[at + i] = f[i];
            }
    }
}
// 8 values in fp16 parts.
__device__ __forceinline__ void split8(const float* v, uint4& hi, uint4& lo) {
    uint32_t h[4], l[4];
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        h[i] = pack_half2(v[2 * i], v[2 * i + 1]);
        const float2 f = __half22float2(*reinterpret_cast<const __half2*>(&h[i]));
        l[i] = pack_half2(v[2 * i] - f.x, v[2 * i + 1] - f.y);
    }
    hi = make_uint4(h[0], h[1], h[2], h[3]);
    lo = make_uint4(l[0], l[1], l[2], l[3]);
}

template <bool SPLIT, bool TALL>
__global__ void __launch_bounds__(kSmallThreads, 1) muon_small_kernel(const MuonSmall a) {
    constexpr int PL = SPLIT ? 2 : 1;
    // With two parts K steps go to four sums in turn, which the epilogue adds up rounding to nearest: the tensor
    // cores cut off with every addition (128 x 1024: 1.3e-6 of the result, as plain fp32 products; with two sums
    // 2.0e-6, with one 3.6e-6, in 1 and 9% less time).
    constexpr int SUMS = SPLIT ? 4 : 1;
    extern __shared__ __align__(16) uint8_t smem_raw[];
    uint8_t* smem = reinterpret_cast<uint8_t*>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t* sX = smem;                           // two parts
    uint8_t* sA = sX + 2 * kPlaneBytes;           // fp32 sums, A, B, and the result
    uint8_t* sR = sA + 4 * kBlockBytes;           // sums of the CTA's rows from the others
    __shared__ uint64_t s_bar, s_sums, s_rows;    // products; sums, rows of A that have arrived
    __shared__ uint32_t s_tmem;
    __shared__ float s_warp[kSmallThreads / 32];
    __shared__ __align__(16) float s_diag[kSide]; // of B
    __shared__ float s_sq[kMaxCluster];
    const int tid = threadIdx.x, warp = tid >> 5, lane = tid & 31;
    const int CS = a.cluster, rank = blockIdx.x % CS, z = blockIdx.x / CS;
    const int rows = a.pre.rows, cols = a.pre.cols;
    // the slice: rows r0 .. r0 + nr and columns c0 .. c0 + nc of the matrix
    const int r0 = TALL ? rank * kSide : 0, c0 = TALL ? 0 : rank * kSide;
    const int nr = min(rows - r0, kSide), nc = min(cols - c0, kSide);
    const int64_t base = (int64_t)z * a.pre.n + (int64_t)r0 * cols + c0;

    if (tid == 0) {
        mbar_init(&s_bar, 1);
        mbar_init(&s_sums, 1);
        mbar_init(&s_rows, 1);
        asm volatile("fence.mbarrier_init.release.cluster;" ::: "memory");
        asm volatile("fence.proxy.async.shared::cta;" ::: "memory");
    }
    if (warp == 0) tmem_alloc(&s_tmem, SUMS * kSide);
    cluster_sync();      // every CTA runs, with its barriers, before one writes into another
    pdl_wait();

    // ---- u = g (+ momentum) in registers, and its sum of squares
    const float gs = a.pre.grad_scale ? __ldg(a.pre.grad_scale) : 1.f;
    const float mu = a.pre.momentum;
    float u[kUnits][8];
    float sum = 0.f;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int e = tid + i * kSmallThreads, r = e >> 4, c = (e & 15) * 8;
        load_unit(a.pre.g, base + (int64_t)r * cols + c, a.g_bf16, a.vec, r < nr ? min(nc - c, 8) : 0, u[i]);
    }
    if (a.pre.m) {
#pragma unroll
        for (int h = 0; h < kUnits; h += kUnits / 2) {
            float m[kUnits / 2][8];
#pragma unroll
            for (int i = 0; i < kUnits / 2; ++i) {
                const int e = tid + (h + i) * kSmallThreads, r = e >> 4, c = (e & 15) * 8;
                load_unit(a.pre.m, base + (int64_t)r * cols + c, false, a.vec, r < nr ? min(nc - c, 8) : 0, m[i]);
            }
#pragma unroll
            for (int i = 0; i < kUnits / 2; ++i) {
                const int e = tid + (h + i) * kSmallThreads, r = e >> 4, c = (e & 15) * 8;
#pragma unroll
                for (int q = 0; q < 8; ++q) {
                    const float g = u[h + i][q] * gs;
                    m[i][q] = fmaf(mu, m[i][q], g);
                    u[h + i][q] = a.pre.nesterov ? fmaf(mu, m[i][q], g) : m[i][q];
                }
                if (r < nr) store_unit(a.pre.m, base + (int64_t)r * cols + c, false, a.vec, min(nc - c, 8), m[i]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < kUnits; ++i)
#pragma unroll
        for (int q = 0; q < 8; ++q) sum = fmaf(u[i][q], u[i][q], sum);
    sum = warp_sum(sum);
    if (lane == 0) s_warp[warp] = sum;
    __syncthreads();
    if (tid < CS) {
        float all = 0.f;
        for (int w = 0; w < kSmallThreads / 32; ++w) all += s_warp[w];
        // every CTA's sum into every CTA
        asm volatile("st.shared::cluster.f32 [%0], %1;" ::"r"(map_to_rank(smem_u32(s_sq + rank), (uint32_t)tid)), "f"(all)
                     : "memory");
    }
    cluster_sync();
    float total = 0.f;
    for (int q = 0; q < CS; ++q) total += s_sq[q];
    const float scale = total < INFINITY ? kXScale / (sqrtf(total) + a.pre.eps) : NAN;
#pragma unroll
    for (int i = 0; i < kUnits; ++i) {
        const int e = tid + i * kSmallThreads, r = e >> 4;
#pragma unroll
        for (int q = 0; q < 8; ++q) u[i][q] *= scale;
        uint4 hi, lo;
        split8(u[i], hi, lo);
        *reinterpret_cast<uint4*>(sX + unit_at(r, e & 15)) = hi;
        *reinterpret_cast<uint4*>(sX + kPlaneBytes + unit_at(r, e & 15)) = lo;
    }
    fence_async_smem();
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = s_tmem;

    // One product of 128 x 128 into TMEM by thread 0, waited for by all. k: length of the reduction; terms (bits):
    // lo hi, hi lo, hi hi. A K step of
    // 16 is 32 bytes of a K-major row (a block holds four), or 16 rows of an MN-major block; both are constants
    // in the unrolled loop, since the issuing thread's own instructions are what a small product waits for.
    bool ok = true;
    uint32_t phase = 0;
    auto product = [&](const uint8_t* pa, auto a_mn, const uint8_t* pb, auto b_mn, int k, int terms) {
        constexpr bool AMN = decltype(a_mn)::value, BMN = decltype(b_mn)::value;
        if (tid == 0 && ok) {
            constexpr uint32_t idesc = idesc_fp16(kSide, kSide, AMN, BMN);
            const uint64_t da = make_desc(smem_u32(pa), AMN ? kBlockBytes : 16, 1024);
            const uint64_t db = make_desc(smem_u32(pb), BMN ? kBlockBytes : 16, 1024);
            const int n = (k + 15) / 16;
#pragma unroll
            for (int term = 0; term < 3; ++term) {
                if (!((terms >> term) & 1)) continue;
                const bool first = !(terms & ((1 << term) - 1));
                const uint64_t ta = da + (term == 0 ? kPlaneBytes >> 4 : 0), tb = db + (term == 1 ? kPlaneBytes >> 4 : 0);
#pragma unroll
                for (int q = 0; q < kSide / 16; ++q) {
                    const uint32_t major = ((q >> 2) * kBlockBytes + (q & 3) * 32) >> 4, minor = (q * 16 * 128) >> 4;
                    if (q < n) tc_mma(tmem + q % SUMS * kSide, ta + (AMN ? minor : major), tb + (BMN ? minor : major), idesc,
                                      first && q < SUMS ? 0u : 1u);
                }
            }
            tc_commit(&s_bar);
        }
        if (ok) ok = mbar_wait(&s_bar, phase, a.err);
        phase ^= 1;
        tc_fence_after();
    };
    constexpr std::integral_constant<bool, TALL> tall{};
    constexpr std::false_type major{};
    constexpr std::true_type minor{};
    constexpr int all = SPLIT ? 7 : 4;
    // Each thread has a row of the product (TMEM lane) and 32 of its columns.
    const int row = (warp & 3) * 32 + lane, part = warp >> 2;
    const uint32_t taddr = tmem + ((uint32_t)((warp & 3) * 32) << 16) + part * 32;
    auto put8 = [&](uint8_t* to, int unit, const float* v, bool two) {
        uint4 hi, lo;
        split8(v, hi, lo);
        *reinterpret_cast<uint4*>(to + unit_at(row, unit)) = hi;
        if (two) *reinterpret_cast<uint4*>(to + kPlaneBytes + unit_at(row, unit)) = lo;
    };
    // The thread's columns of the product; k: the reduction's length.
    auto sums = [&](int k, float (&v)[32]) {
        uint32_t acc[32];
        tmem_ld32(taddr, acc);
        tmem_ld_wait_regs(acc);
#pragma unroll
        for (int i = 0; i < 32; ++i) v[i] = __uint_as_float(acc[i]);
#pragma unroll
        for (int m = 1; m < SUMS; ++m) {
            if (16 * m >= k) break;
            tmem_ld32(taddr + m * kSide, acc);
            tmem_ld_wait_regs(acc);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] += __uint_as_float(acc[i]);
        }
    };
    // 8 fp16 values (in parts) of the thread's row.
    auto get8 = [&](const uint8_t* from, int unit, float* v, bool two) {
        const uint4 q4 = *reinterpret_cast<const uint4*>(from + unit_at(row, unit));
        const __half2* q = reinterpret_cast<const __half2*>(&q4);
        uint4 l4 = make_uint4(0, 0, 0, 0);
        if (two) l4 = *reinterpret_cast<const uint4*>(from + kPlaneBytes + unit_at(row, unit));
        const __half2* l = reinterpret_cast<const __half2*>(&l4);
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 f = __half22float2(q[i]), g = __half22float2(l[i]);
            v[2 * i] = f.x + g.x;
            v[2 * i + 1] = f.y + g.y;
        }
    };
    auto ready = [&]() {     // this CTA's writes are there for the next product or copy, and TMEM is read
        fence_async_smem();
        tc_fence_before();
        __syncthreads();
        tc_fence_after();
    };
    const int per = (kSide + CS - 1) / CS;                               // rows of A that a CTA adds up
    const int own0 = min(rank * per, kSide), own = min(own0 + per, kSide) - own0;

    for (int step = 0; step < a.steps; ++step) {
        // ---- gram
        product(sX, tall, sX, tall, TALL ? nr : nc, all);
        {
            float v[32];
            sums(TALL ? nr : nc, v);
#pragma unroll
            for (int i = 0; i < 32; ++i) v[i] *= kAScale / (kXScale * kXScale);
            if (CS == 1) {
#pragma unroll
                for (int j = 0; j < 4; ++j) put8(sA, part * 4 + j, v + 8 * j, SPLIT);
            } else {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4*>(sA + unit_at(row, part * 8 + j)) =
                        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            }
        }
        ready();
        if (CS > 1) {
            // the others' rows of the sums to them: lane = 4 * CTA + block
            const int q = lane >> 2, k = lane & 3;
            const int q0 = min(q * per, kSide), nq = min(q0 + per, kSide) - q0;
            if (warp == 0 && ok && q < CS && q != rank && nq > 0)
                send(map_to_rank(smem_u32(sR) + (uint32_t)((rank * 4 + k) * nq * 128), (uint32_t)q),
                     smem_u32(sA) + (uint32_t)(k * kBlockBytes + q0 * 128), (uint32_t)nq * 128,
                     map_to_rank(smem_u32(&s_sums), (uint32_t)q));
            if (tid == 0) mbar_expect_tx(&s_sums, (uint32_t)((CS - 1) * own * 512));
            if (ok) ok = mbar_wait(&s_sums, (uint32_t)step & 1u, a.err);
            // a thread adds up one unit of 8 values, or two (two CTAs: 64 rows of 16 units each)
            constexpr int MOST = kSide / 2 * (kSide / 8) / kSmallThreads;
            float v[MOST][8];
#pragma unroll
            for (int i = 0; i < MOST; ++i) {
                const int e = tid + i * kSmallThreads, r = own0 + (e >> 4), c = e & 15;
#pragma unroll
                for (int j = 0; j < 8; ++j) v[i][j] = 0.f;
                for (int o = 0; o < CS && (e >> 4) < own; ++o) {
                    // fp32 units 2 c and 2 c + 1 of the row
#pragma unroll
                    for (int w = 0; w < 2; ++w) {
                        const int unit = 2 * c + w;
                        const uint8_t* from = o == rank ? sA + unit_at(r, unit)
                                                        : sR + (o * 4 + (unit >> 3)) * own * 128 + (r - own0) * 128 +
                                                              (((unit & 7) ^ (r & 7)) << 4);
                        const float4 f = *reinterpret_cast<const float4*>(from);
                        v[i][4 * w] += f.x; v[i][4 * w + 1] += f.y; v[i][4 * w + 2] += f.z; v[i][4 * w + 3] += f.w;
                    }
                }
            }
            __syncthreads();      // the sums of the CTA's own rows are read: its rows of A take their place
#pragma unroll
            for (int i = 0; i < MOST; ++i) {
                const int e = tid + i * kSmallThreads, r = own0 + (e >> 4), c = e & 15;
                if ((e >> 4) < own) {
                    uint4 hi, lo;
                    split8(v[i], hi, lo);
                    *reinterpret_cast<uint4*>(sA + unit_at(r, c)) = hi;
                    if (SPLIT) *reinterpret_cast<uint4*>(sA + kPlaneBytes + unit_at(r, c)) = lo;
                }
            }
            fence_async_smem();
            __syncthreads();
            // the CTA's rows of A to the others
            if (warp == 0 && ok && q < CS && q != rank && k < 2 * PL && own > 0) {
                const uint32_t at = smem_u32(sA) + (uint32_t)(k * kBlockBytes + own0 * 128);
                send(map_to_rank(at, (uint32_t)q), at, (uint32_t)own * 128, map_to_rank(smem_u32(&s_rows), (uint32_t)q));
            }
            if (tid == 0) mbar_expect_tx(&s_rows, (uint32_t)((kSide - own) * 128 * 2 * PL));
            if (ok) ok = mbar_wait(&s_rows, (uint32_t)step & 1u, a.err);
            asm volatile("barrier.cluster.arrive.aligned;" ::: "memory");
        }
        // ---- poly: B = a I + b A + c A A in the place of A
        product(sA, major, sA, major, a.side, all);
        // every CTA has its rows of A, so none of this one's are still being read by a copy
        if (CS > 1) asm volatile("barrier.cluster.wait.aligned;" ::: "memory");
        {
            float v[32], w[32];
            sums(a.side, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) get8(sA, part * 4 + j, w + 8 * j, SPLIT);
#pragma unroll
            for (int i = 0; i < 32; ++i) {
                v[i] = fmaf(a.b * (kBScale / kAScale), w[i], a.c * (kBScale / (kAScale * kAScale)) * v[i]);
                if (part * 32 + i == row) {
                    s_diag[row] = fmaf(v[i], 1.f / kBScale, a.a);
                    v[i] = 0.f;
                }
            }
#pragma unroll
            for (int j = 0; j < 4; ++j) put8(sA, part * 4 + j, v + 8 * j, SPLIT);
        }
        ready();
        // ---- apply
        const int terms = SPLIT || step + 2 < a.steps ? all | (TALL ? 1 : 2) : all;      // (X's low part, too)
        if constexpr (TALL) product(sX, major, sA, major, a.side, terms);
        else product(sA, major, sX, minor, a.side, terms);
        const bool last = step + 1 == a.steps;
        const float drow = s_diag[row];
        {
            float v[32], w[32];
            sums(a.side, v);
#pragma unroll
            for (int j = 0; j < 4; ++j) get8(sX, part * 4 + j, w + 8 * j, true);
#pragma unroll
            for (int i = 0; i < 32; i += 4) {
                float4 d = make_float4(drow, drow, drow, drow);
                if (TALL) d = *reinterpret_cast<const float4*>(s_diag + part * 32 + i);
                v[i] = fmaf(d.x, w[i], v[i] * (1.f / kBScale));
                v[i + 1] = fmaf(d.y, w[i + 1], v[i + 1] * (1.f / kBScale));
                v[i + 2] = fmaf(d.z, w[i + 2], v[i + 2] * (1.f / kBScale));
                v[i + 3] = fmaf(d.w, w[i + 3], v[i + 3] * (1.f / kBScale));
            }
            if (last) {
#pragma unroll
                for (int j = 0; j < 8; ++j)
                    *reinterpret_cast<float4*>(sA + unit_at(row, part * 8 + j)) =
                        make_float4(v[4 * j], v[4 * j + 1], v[4 * j + 2], v[4 * j + 3]);
            } else {
#pragma unroll
                for (int j = 0; j < 4; ++j) put8(sX, part * 4 + j, v + 8 * j, true);
            }
        }
        ready();
    }

    // ---- o, or the step on the weights
    const float lr = a.fin.lr_dev ? __ldg(a.fin.lr_dev) : a.fin.lr;
    const float lose = lr * a.fin.decay, move = lr * a.fin.scale;
#pragma unroll
    for (int h = 0; h < kUnits; h += kUnits / 2) {
        float p[kUnits / 2][8];
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i) {
            const int e = tid + (h + i) * kSmallThreads, r = e >> 4, c = (e & 15) * 8;
            if (a.fin.step)
                load_unit(a.fin.master ? (const void*)a.fin.master : a.fin.out, base + (int64_t)r * cols + c,
                          !a.fin.master && a.p_bf16, a.vec, r < nr ? min(nc - c, 8) : 0, p[i]);
        }
#pragma unroll
        for (int i = 0; i < kUnits / 2; ++i) {
            const int e = tid + (h + i) * kSmallThreads, r = e >> 4, c = (e & 15) * 8, n = min(nc - c, 8);
            if (r >= nr || n <= 0) continue;
            const int64_t at = base + (int64_t)r * cols + c;
            float x[8];
            if (a.steps) {
                *reinterpret_cast<float4*>(x) = *reinterpret_cast<const float4*>(sA + unit_at(r, 2 * (e & 15)));
                *reinterpret_cast<float4*>(x + 4) = *reinterpret_cast<const float4*>(sA + unit_at(r, 2 * (e & 15) + 1));
            } else {
                const __half* hi = reinterpret_cast<const __half*>(sX + unit_at(r, e & 15));
                const __half* lo = reinterpret_cast<const __half*>(sX + kPlaneBytes + unit_at(r, e & 15));
#pragma unroll
                for (int q = 0; q < 8; ++q) x[q] = __half2float(hi[q]) + __half2float(lo[q]);
            }
#pragma unroll
            for (int q = 0; q < 8; ++q) {
                x[q] *= 1.f / kXScale;
                if (a.fin.step) x[q] = fmaf(-move, x[q], fmaf(-lose, p[i][q], p[i][q]));
            }
            if (a.fin.master) store_unit(a.fin.master, at, false, a.vec, n, x);
            store_unit(a.fin.out, at, a.p_bf16, a.vec, n, x);
        }
    }
    tc_fence_before();
    __syncthreads();
    cluster_sync();      // no CTA leaves while another may still write into it
    if (warp == 0) {
        tc_fence_after();
        tmem_dealloc(tmem, SUMS * kSide);
    }
}

constexpr size_t kSmallSmem = 1024 + 2 * (size_t)kPlaneBytes + 4 * kBlockBytes + kRecvBytes;
static_assert(kSmallSmem <= 227 * 1024 - 1024, "shared memory per CTA");

// ---------------------------------------------------------------- host
// Whether fp16 holds, at their scales, all that the steps make of singular values in [0, 1]: the largest of X by the
// maximum of |s (a + b s^2 + c s^4)| from step to step, A's by its square, and of B without its diagonal by that of
// |b A + c A^2|; no element is larger than those. With 2^-9 to spare for roundings.
bool fits_fp16(const moe_muon_config_t& c) {
    constexpr double kMost = 65504.0 * (1.0 - 1.0 / 512), kSlack = 1.0 + 1.0 / 512;
    double s = 1.0;                                    // largest singular value of X
    for (int k = 0; k < c.steps; ++k) {
        const double t = s * s;                        // and of A
        auto poly = [&](double u) { return std::fabs(std::sqrt(u) * (c.a + u * (c.b + u * c.c))); };
        auto rest = [&](double u) { return std::fabs(u * (c.b + u * c.c)); };
        double x = poly(t), b = rest(t);
        if (c.c != 0.0 && -c.b / (2.0 * c.c) > 0.0) b = std::max(b, rest(std::min(t, -c.b / (2.0 * c.c))));
        // zeros of a + 3 b u + 5 c u^2
        const double root = 9.0 * c.b * c.b - 20.0 * c.a * c.c;
        if (c.c != 0.0 && root >= 0.0) {
            for (double sign : {-1.0, 1.0}) {
                const double u = (-3.0 * c.b + sign * std::sqrt(root)) / (10.0 * c.c);
                if (u > 0.0 && u < t) x = std::max(x, poly(u));
            }
        } else if (c.c == 0.0 && c.b != 0.0) {
            const double u = -c.a / (3.0 * c.b);
            if (u > 0.0 && u < t) x = std::max(x, poly(u));
        }
        if (!(t * kAScale <= kMost && b * kBScale <= kMost && x * kXScale <= kMost)) return false;
        s = x * kSlack;
    }
    return true;
}

moe_status_t check_muon(const moe_muon_config_t* c) {
    if (!c) return MOE_ERR_INVALID_ARG;
    if (c->count < 0 || c->rows < 1 || c->cols < 1 || c->steps < 0 || c->steps > 100) return MOE_ERR_INVALID_ARG;
    for (double v : {c->a, c->b, c->c})
        if (!(std::fabs(v) <= 16.0)) return MOE_ERR_INVALID_ARG;
    for (double v : {c->lr, c->weight_decay, c->scale})
        if (!std::isfinite(v) || !std::isfinite((float)v)) return MOE_ERR_INVALID_ARG;
    if (!(c->momentum >= 0.0 && c->momentum < 1.0) || !(c->eps >= 1e-12 && c->eps <= 1.0)) return MOE_ERR_INVALID_ARG;
    if (c->nesterov != 0 && c->nesterov != 1) return MOE_ERR_INVALID_ARG;
    for (int32_t t : {c->dtype, c->grad_dtype, c->precision})
        if (t != MOE_F32 && t != MOE_BF16) return MOE_ERR_INVALID_ARG;
    if (c->count > 65535 || c->rows > 65536 || c->cols > 65536) return MOE_ERR_UNSUPPORTED;
    const int64_t tiles = (int64_t)ceil_div(c->rows, kTile) * ceil_div(c->cols, kTile);
    if (c->count * tiles > (1 << 30) || !fits_fp16(*c)) return MOE_ERR_UNSUPPORTED;
    return MOE_OK;
}

bool misaligned(const void* p, uintptr_t a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1)) != 0; }

constexpr int64_t kChunk = 32768;     // elements whose squares one block adds up
constexpr int kMaxChunks = 1024;      // chunks of a matrix

struct MuonScratch {
    __half* X[2];
    __half* A;
    __half* B;
    float* diag;
    float* sums;
    int planes, ld, lds, side;        // planes: of A and B (X has 2); ld: of X; side, lds: of A and B
    int dstride;
    int64_t chunk;
    int chunks;
};

// Whether a matrix fits a cluster of CTAs (8, the portable most) that keep it in shared memory. At the border: 128 x 1024
// 63 us in fp32 and 47 in bf16, 128 x 1025, by tiled products, 180 and 127; 128 x 2048 216 and 122, 256 x 1024 170 and 112.
bool small_matrix(const moe_muon_config_t& c) {
    return std::min(c.rows, c.cols) <= kSide && std::max(c.rows, c.cols) <= kSide * kMaxCluster;
}

size_t carve_muon(const moe_muon_config_t& c, void* base, MuonScratch* b) {
    Workspace ws{static_cast<char*>(base), 0};
    b->planes = c.precision == MOE_F32 ? 2 : 1;
    b->ld = (int)align_up(c.cols, 8);
    b->side = std::min(c.rows, c.cols);
    b->lds = (int)align_up(b->side, 8);
    const int64_t n = (int64_t)c.rows * c.cols;
    b->chunk = std::max<int64_t>(kChunk, ((n + kMaxChunks - 1) / kMaxChunks + 7) / 8 * 8);
    b->chunks = (int)((n + b->chunk - 1) / b->chunk);
    const size_t all = (size_t)b->planes * c.count;
    b->sums = ws.take<float>((size_t)c.count * b->chunks + 1);
    for (__half*& x : b->X) x = ws.take<__half>((size_t)2 * c.count * c.rows * b->ld + 1);
    b->dstride = (int)align_up(b->side, 32);
    b->diag = ws.take<float>((size_t)c.count * b->dstride + kTile);
    b->A = ws.take<__half>(all * b->side * b->lds + 1);
    b->B = ws.take<__half>(all * b->side * b->lds + 1);
    return align_up(ws.used, 256);
}

// 16-bit elements [outer, rows, cols] with rows ld elements apart.
bool map_3d(CUtensorMap* tm, const void* base, uint64_t cols, uint64_t rows, uint64_t outer, uint64_t ld,
            uint32_t box_cols, uint32_t box_rows, CUtensorMapSwizzle swizzle,
            CUtensorMapDataType type = CU_TENSOR_MAP_DATA_TYPE_FLOAT16) {
    auto fn = encode_fn();
    if (!fn) return false;
    cuuint64_t dims[3] = {cols, rows, outer};
    cuuint64_t strides[2] = {ld * 2, ld * rows * 2};
    cuuint32_t box[3] = {box_cols, box_rows, 1};
    cuuint32_t estr[3] = {1, 1, 1};
    return fn(tm, type, 3, const_cast<void*>(base), dims, strides, box, estr,
              CU_TENSOR_MAP_INTERLEAVE_NONE, swizzle, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
              CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE) == CUDA_SUCCESS;
}

struct Operand {
    const void* base;
    int rows, cols, ld, planes;
};

// K-major operands come in boxes of 64 k x 128 rows (B: half a tile's columns), MN-major ones of 64 columns x 64 k.
template <int OP, bool A_MN, bool B_MN, int NT>
cudaError_t launch_gemm_as(MuonGemm p, bool split, const Operand& a, const Operand& b, const Operand& o, int out,
                           cudaStream_t s) {
    auto outer = [&](const Operand& q) { return (uint64_t)q.planes * p.count; };
    CUtensorMap ta, tb, to;
    if (!map_3d(&ta, a.base, a.cols, a.rows, outer(a), a.ld, 64, A_MN ? BK : kHalf, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map_3d(&tb, b.base, b.cols, b.rows, outer(b), b.ld, 64, B_MN ? BK : NT / 2, CU_TENSOR_MAP_SWIZZLE_128B) ||
        !map_3d(&to, o.base, o.cols, o.rows, outer(o), o.ld, 32, 32, CU_TENSOR_MAP_SWIZZLE_64B,
                out == kResult ? CU_TENSOR_MAP_DATA_TYPE_BFLOAT16 : CU_TENSOR_MAP_DATA_TYPE_FLOAT16))
        return cudaErrorInvalidValue;
    auto kern = split ? muon_gemm_kernel<OP, A_MN, B_MN, true, kParts, NT>
                      : muon_gemm_kernel<OP, A_MN, B_MN, false, kParts, NT>;
    if constexpr (OP == kApply)
        if (out == kResult) kern = muon_gemm_kernel<OP, A_MN, B_MN, false, kResult, NT>;
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kGemmSmem);
    if (e != cudaSuccess) return e;
    const int clusters = (int)std::min<int64_t>((int64_t)p.count * p.tiles, num_sms() / 2);
    e = launch_pdl(kern, dim3(2 * clusters), dim3(kGemmThreads), kGemmSmem, s, p, ta, tb, to);
    count_launch();
    return e;
}

// Tiles of a matrix, nt columns wide.
int tiles_of(const MuonGemm& p, bool sym, int nt) {
    const int m = ceil_div(p.M, kTile), n = ceil_div(p.N, nt);
    return sym ? kTile / nt * (m * (m - 1) / 2) + n : m * n;
}

// Tiles are as narrow as they may be (256, 128 or 64 columns; 128 where B is MN-major, which comes in boxes of 64)
// without a further round of tiles over the pairs: a product of few tiles waits for its longest one (polynomial of
// 1024 x 1024 in two parts: 34.7 us, 26.5 and 20.4), but a tile of half the columns takes 0.6 to 0.85 of the time
// (4 x 2048 x 1024, two rounds for one: gram 42 us and 67, polynomial 37 and 45).
template <int OP, bool A_MN, bool B_MN>
cudaError_t launch_gemm(MuonGemm p, bool split, const Operand& a, const Operand& b, const Operand& o, cudaStream_t s,
                        int out = kParts) {
    constexpr bool SYM = OP != kApply;
    constexpr int LEAST = B_MN ? 128 : 64;
    auto rounds = [&](int w) { return ((int64_t)p.count * tiles_of(p, SYM, w) + num_sms() / 2 - 1) / (num_sms() / 2); };
    int nt = kTile;
    while (nt > LEAST && rounds(nt / 2) <= rounds(nt)) nt /= 2;
    p.n_tiles = ceil_div(p.N, nt);
    p.tiles = tiles_of(p, SYM, nt);
    p.err = device_error_word();
    if (nt == 256) return launch_gemm_as<OP, A_MN, B_MN, 256>(p, split, a, b, o, out, s);
    if (nt == 128) return launch_gemm_as<OP, A_MN, B_MN, 128>(p, split, a, b, o, out, s);
    if constexpr (LEAST == 64) return launch_gemm_as<OP, A_MN, B_MN, 64>(p, split, a, b, o, out, s);
    return cudaErrorInvalidValue;
}

template <typename G, bool MOMENTUM>
cudaError_t launch_prep(const MuonPrep& a, cudaStream_t s) {
    const int64_t work = (int64_t)a.count * a.chunks;
    const int grid = (int)std::min<int64_t>(work, (int64_t)num_sms() * 4);
    cudaError_t e = launch_pdl(a.n % 8 == 0 ? muon_sums_kernel<G, 8, MOMENTUM> : muon_sums_kernel<G, 1, MOMENTUM>,
                               dim3(grid), dim3(kPrepThreads), 0, s, a);
    count_launch();
    if (e != cudaSuccess) return e;
    e = launch_pdl(a.cols % 8 == 0 ? muon_scale_kernel<G, 8, MOMENTUM> : muon_scale_kernel<G, 1, MOMENTUM>, dim3(grid), dim3(kPrepThreads), 0, s, a);
    count_launch();
    return e;
}

template <typename T>
cudaError_t launch_finish(const MuonFinish& a, cudaStream_t s) {
    const int v = a.cols % 8 == 0 ? 8 : 1;
    auto kern = v == 8 ? muon_finish_kernel<T, 8> : muon_finish_kernel<T, 1>;
    const int64_t need = (a.total + 256 * v - 1) / (256 * v);
    const cudaError_t e = launch_pdl(kern, dim3((unsigned)std::min<int64_t>(need, (int64_t)num_sms() * 32)), dim3(256),
                                     0, s, a);
    count_launch();
    return e;
}

cudaError_t launch_small(const moe_muon_config_t& c, const MuonPrep& pre, const MuonFinish& fin, bool split,
                         cudaStream_t s) {
    MuonSmall a{};
    a.pre = pre;
    a.fin = fin;
    a.steps = c.steps;
    a.side = std::min(c.rows, c.cols);
    a.cluster = ceil_div(std::max(c.rows, c.cols), kSide);
    a.g_bf16 = c.grad_dtype == MOE_BF16;
    a.p_bf16 = c.dtype == MOE_BF16;
    a.vec = c.cols % 8 == 0;
    a.a = (float)c.a;
    a.b = (float)c.b;
    a.c = (float)c.c;
    a.err = device_error_word();
    const bool tall = c.rows > c.cols;
    auto kern = split ? (tall ? muon_small_kernel<true, true> : muon_small_kernel<true, false>)
                      : (tall ? muon_small_kernel<false, true> : muon_small_kernel<false, false>);
    cudaError_t e = cudaFuncSetAttribute(kern, cudaFuncAttributeMaxDynamicSharedMemorySize, (int)kSmallSmem);
    if (e != cudaSuccess) return e;
    cudaLaunchConfig_t cfg{};
    cfg.gridDim = dim3((unsigned)(c.count * a.cluster));
    cfg.blockDim = dim3(kSmallThreads);
    cfg.dynamicSmemBytes = kSmallSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[2];
    at[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    at[0].val.programmaticStreamSerializationAllowed = 1;
    at[1].id = cudaLaunchAttributeClusterDimension;
    at[1].val.clusterDim.x = (unsigned)a.cluster;
    at[1].val.clusterDim.y = at[1].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 2;
    e = launch_ex(cfg, kern, a);
    count_launch();
    return e;
}

cudaError_t launch_muon(const moe_muon_config_t& c, const void* g, float* m, const float* grad_scale, MuonFinish f,
                        void* ws, cudaStream_t s) {
    MuonScratch b;
    carve_muon(c, ws, &b);
    const bool split = b.planes == 2, tall = c.rows > c.cols;
    MuonPrep pre{g, m, grad_scale, b.sums, b.X[0], (int64_t)c.rows * c.cols, b.chunk, b.chunks, c.count, c.rows, c.cols,
                 b.ld, (float)c.momentum, (float)c.eps, c.nesterov};
    f.n = pre.n;
    f.total = pre.n * c.count;
    f.count = c.count;
    f.rows = c.rows;
    f.cols = c.cols;
    f.ld = b.ld;
    f.lr = (float)c.lr;
    f.decay = (float)c.weight_decay;
    f.scale = (float)c.scale;
    if (small_matrix(c)) return launch_small(c, pre, f, split, s);
    cudaError_t e = c.grad_dtype == MOE_BF16
                        ? (m ? launch_prep<__nv_bfloat16, true>(pre, s) : launch_prep<__nv_bfloat16, false>(pre, s))
                        : (m ? launch_prep<float, true>(pre, s) : launch_prep<float, false>(pre, s));
    if (e != cudaSuccess) return e;
    const Operand A{b.A, b.side, b.side, b.lds, b.planes}, B{b.B, b.side, b.side, b.lds, b.planes};
    // the last product writes the result where that is bf16, in rows of whole 16-byte units
    const bool direct = !split && c.dtype == MOE_BF16 && !f.master && c.cols % 8 == 0;
    int at = 0;
    for (int k = 0; k < c.steps; ++k, at ^= 1) {
        const bool result = direct && k + 1 == c.steps;
        const Operand X{b.X[at], c.rows, c.cols, b.ld, 2};
        const Operand Y{result ? f.out : b.X[at ^ 1], c.rows, c.cols, result ? c.cols : b.ld, result ? 1 : 2};
        MuonGemm p{};
        p.count = c.count;
        p.M = p.N = b.side;
        p.K = std::max(c.rows, c.cols);
        p.alpha = kAScale / (kXScale * kXScale);
        e = tall ? launch_gemm<kGram, true, true>(p, split, X, X, A, s)
                 : launch_gemm<kGram, false, false>(p, split, X, X, A, s);
        if (e != cudaSuccess) return e;
        p.K = b.side;
        p.side = reinterpret_cast<const uint16_t*>(b.A);
        p.diag = b.diag;
        p.dstride = b.dstride;
        p.ld = b.lds;
        p.alpha = (float)(c.c * kBScale / ((double)kAScale * kAScale));
        p.beta = (float)(c.b * kBScale / kAScale);
        p.a = (float)c.a;
        e = launch_gemm<kPoly, false, false>(p, split, A, A, B, s);
        if (e != cudaSuccess) return e;
        p.M = c.rows;
        p.N = c.cols;
        p.alpha = 1.f / kBScale;
        p.side = reinterpret_cast<const uint16_t*>(b.X[at]);
        p.ld = b.ld;
        p.twice = !split && k + 2 < c.steps;
        if (result) {
            p.weights = f.step ? static_cast<const uint16_t*>(f.out) : nullptr;
            p.gain = 1.f / kXScale;
            p.lr_dev = f.lr_dev;
            p.lr = f.lr;
            p.decay = f.decay;
            p.scale = f.scale / kXScale;
        }
        const int out = result ? kResult : kParts;
        e = tall ? launch_gemm<kApply, false, false>(p, split, X, B, Y, s, out)
                 : launch_gemm<kApply, false, true>(p, split, B, X, Y, s, out);
        if (e != cudaSuccess) return e;
        if (result) return cudaSuccess;
    }
    f.X = b.X[at];
    return c.dtype == MOE_BF16 ? launch_finish<__nv_bfloat16>(f, s) : launch_finish<float>(f, s);
}

}  // namespace

}  // namespace moe

using namespace moe;

extern "C" MOE_API size_t moe_muon_workspace_bytes(const moe_muon_config_t* cfg) {
    if (check_muon(cfg) != MOE_OK || cfg->count == 0) return 0;
    if (small_matrix(*cfg)) return 256;      // (all of it in shared memory)
    MuonScratch b;
    return carve_muon(*cfg, nullptr, &b);
}

extern "C" MOE_API moe_status_t moe_orthogonalize(const moe_muon_config_t* cfg, const void* g, void* o, void* ws,
                                                  moe_stream_t stream) {
    const moe_status_t st = check_muon(cfg);
    if (st != MOE_OK) return st;
    if (cfg->count == 0) return MOE_OK;
    if (!g || !o || !ws || (g == o && cfg->dtype != cfg->grad_dtype)) return MOE_ERR_INVALID_ARG;
    if (misaligned(g, 16) || misaligned(o, 16) || misaligned(ws, 16)) return MOE_ERR_INVALID_ARG;
    MuonFinish f{};
    f.out = o;
    return launch_muon(*cfg, g, nullptr, nullptr, f, ws, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}

extern "C" MOE_API moe_status_t moe_muon(const moe_muon_config_t* cfg, void* p, const void* g, float* master, float* m,
                                         const float* lr, const float* grad_scale, void* ws, moe_stream_t stream) {
    const moe_status_t st = check_muon(cfg);
    if (st != MOE_OK) return st;
    if (cfg->count == 0) return MOE_OK;
    if (!p || !g || !m || !ws) return MOE_ERR_INVALID_ARG;
    if (misaligned(p, 16) || misaligned(g, 16) || misaligned(master, 16) || misaligned(m, 16) || misaligned(ws, 16) ||
        misaligned(lr, 4) || misaligned(grad_scale, 4))
        return MOE_ERR_INVALID_ARG;
    MuonFinish f{};
    f.out = p;
    f.master = master;
    f.lr_dev = lr;
    f.step = true;
    return launch_muon(*cfg, g, m, grad_scale, f, ws, (cudaStream_t)stream) == cudaSuccess ? MOE_OK : MOE_ERR_CUDA;
}
