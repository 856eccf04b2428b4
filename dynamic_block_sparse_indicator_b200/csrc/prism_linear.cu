// prism_linear.cu -- the projections around the attention on sm_100a tensor cores:
//     z = x W^T + b,  y = act(z) + residual            (forward)
//     dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz   (gradients)
// with x, y and their gradients either rows [M][K] or head-major [heads][M][D], so the
// input projection writes what prism_plan reads and the output projection reads what
// prism_attn_fwd writes, without a transposing copy.
//
// All products are one kernel: C[r][c] = sum_k B[r][k] A[c][k], c the contiguous index of
// C.  The tensor core's M dimension (TMEM lanes) runs over c and its N dimension (TMEM
// columns) over r, so an epilogue warp holds 32 consecutive c of one row in its lanes:
// bias is one value per lane, residual and results are consecutive addresses, and few
// tokens are a small N instead of an M tile of padding.  An operand is a 3-D TMA map
// (inner, rows, heads) with the contraction along the inner index (K-major) or along the
// rows (MN-major); head-major inner coordinates split into (channel, head):
//     forward  A = W  [N][K] K-major     B = x  [M][K] K-major
//     dx       A = W  [N][K] MN-major    B = dz [M][N] K-major
//     dW       A = x  [M][K] MN-major    B = dz [M][N] MN-major
// Bound: the tensor cores for many tokens (2 M K N flops), HBM's read of W for few.
//
// Warp roles: 0-7 epilogue (TMEM lane quarter w % 4, column half w / 4), 8 TMA producer and
// TMEM allocator, 9 MMA issuer.  Two TMEM accumulators alternate, so the next products run
// while the epilogue reads the last.
//
// The tensor core's fp32 accumulation truncates: over a contraction of 16,384 the result
// is low by 1.6e-5 of its size, growing linearly (measured with standard normal operands;
// 4.7e-6 at 5,120).  So a contraction is cut into chunks of at most kChunk elements, each
// summed by the tensor core into a fresh accumulator, and the chunks are added in
// registers with round-to-nearest.
//
// Every barrier wait is bounded (PRISM_ERR_TIMEOUT with a site in the status block).
#include <cuda.h>
#include <cuda_bf16.h>
#include <cuda_runtime.h>
#include <cudaTypedefs.h>

#include "prism_dev.cuh"
#include "prism_internal.h"

namespace prism {
namespace lin {

constexpr int kEpiWarps = 8;
constexpr int kThreads = (kEpiWarps + 2) * 32;
constexpr int kKB = 64;                    // contraction elements per stage (128-byte rows)
constexpr int kChunkKB = 32;               // stages per accumulation chunk: 2,048 elements

struct Operand {
    int inner;                             // extent of the inner index of one head
    int mn;                                // 1 = MN-major
};

struct Out {
    void* p;                               // element (r, c): p + head(c) hs + r rs + c in head
    int64_t rs, hs;
    int hd;                                // channels per head; 0 = one head
    int f32;
};

struct Args {
    Operand a, b;
    int64_t R;                             // rows of C
    int C;                                 // columns of C
    int kblocks;                           // stages of the whole contraction
    int split;                             // CTAs of a cluster that share a tile's contraction
    int tiles_c, tiles_r, band;
    Out y, pre, res;
    const void* bias;
    int bias_f32, act;
    int* err;
};

// ---------------------------------------------------------------- PTX
template <int CG>
__device__ __forceinline__ void tma3(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z) {
    if (CG == 2)
        // the barrier may lie in the pair's other CTA
        asm volatile("cp.async.bulk.tensor.3d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5}], [%2];"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5}], [%2];"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z) : "memory");
}
template <int CG>
__device__ __forceinline__ void mma(uint32_t d, uint64_t a, uint64_t b, uint32_t idesc, uint32_t acc) {
    if (CG == 2)
        asm volatile("{\n\t.reg .pred p;\n\tsetp.ne.b32 p, %4, 0;\n\t"
                     "tcgen05.mma.cta_group::2.kind::f16 [%0], %1, %2, %3, p;\n\t}"
                     :: "r"(d), "l"(a), "l"(b), "r"(idesc), "r"(acc) : "memory");
    else
        umma_f16(d, a, b, idesc, acc);
}
// Arrive on `bar` (of both CTAs of a pair) when this thread's MMAs so far are done.
template <int CG>
__device__ __forceinline__ void commit(uint64_t* bar) {
    if (CG == 2)
        asm volatile("tcgen05.commit.cta_group::2.mbarrier::arrive::one.shared::cluster.multicast::cluster.b64 [%0], %1;"
                     :: "r"(smem_u32(bar)), "h"((uint16_t)3) : "memory");
    else
        umma_commit(bar);
}
template <int CG>
__device__ __forceinline__ void alloc_tmem(uint32_t* dst, uint32_t cols) {
    if (CG == 2) {
        asm volatile("tcgen05.alloc.cta_group::2.sync.aligned.shared::cta.b32 [%0], %1;"
                     :: "r"(smem_u32(dst)), "r"(cols) : "memory");
        asm volatile("tcgen05.relinquish_alloc_permit.cta_group::2.sync.aligned;" ::: "memory");
    } else {
        tmem_alloc(dst, cols);
    }
}
template <int CG>
__device__ __forceinline__ void free_tmem(uint32_t addr, uint32_t cols) {
    if (CG == 2)
        asm volatile("tcgen05.dealloc.cta_group::2.sync.aligned.b32 %0, %1;" :: "r"(addr), "r"(cols) : "memory");
    else
        tmem_dealloc(addr, cols);
}
__device__ __forceinline__ uint32_t cluster_rank() {
    uint32_t r;
    asm volatile("mov.u32 %0, %%cluster_ctarank;" : "=r"(r));
    return r;
}
__device__ __forceinline__ uint32_t map_to(uint32_t saddr, uint32_t rank) {
    uint32_t r;
    asm volatile("mapa.shared::cluster.u32 %0, %1, %2;" : "=r"(r) : "r"(saddr), "r"(rank));
    return r;
}
__device__ __forceinline__ void cluster_sync() {
    asm volatile("barrier.cluster.arrive.release.aligned;\n\tbarrier.cluster.wait.acquire.aligned;" ::: "memory");
}
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.release.cluster.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
__device__ __forceinline__ float ld_peer(uint32_t cluster_addr) {
    float v;
    asm volatile("ld.shared::cluster.f32 %0, [%1];" : "=f"(v) : "r"(cluster_addr) : "memory");
    return v;
}

// mbar_wait with its loop in line: the epilogue waits with a tile's sums in registers, which
// a call would have to save.
__device__ __forceinline__ bool mbar_wait_inline(uint64_t* bar, uint32_t parity, int* err, int where) {
    if (mbar_try(bar, parity)) return true;
    const uint64_t t0 = globaltimer_ns();
    for (;;) {
        if (mbar_try_suspend(bar, parity, 20000)) return true;
        if (*(volatile int*)err != 0) return false;
        if (globaltimer_ns() - t0 > kWaitNs) break;
    }
    if (atomicCAS(err, 0, PRISM_ERR_TIMEOUT) == 0) {
        err[1] = where;
        err[2] = (int)blockIdx.x;
        err[3] = (int)threadIdx.x;
    }
    return false;
}

// Accumulator columns of this thread's lane.
template <int N> struct Cols;
#define PRISM_U(x) __float_as_uint(x)
template <> struct Cols<8> {
    static __device__ __forceinline__ void load(uint32_t t, uint32_t* r) {
        asm volatile("tcgen05.ld.sync.aligned.32x32b.x8.b32 {%0,%1,%2,%3,%4,%5,%6,%7}, [%8];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3]), "=r"(r[4]), "=r"(r[5]), "=r"(r[6]), "=r"(r[7])
                     : "r"(t));
    }
    static __device__ __forceinline__ void store(uint32_t t, const float* v) {
        asm volatile("tcgen05.st.sync.aligned.32x32b.x8.b32 [%0], {%1,%2,%3,%4,%5,%6,%7,%8};"
                     :: "r"(t), "r"(PRISM_U(v[0])), "r"(PRISM_U(v[1])), "r"(PRISM_U(v[2])), "r"(PRISM_U(v[3])),
                        "r"(PRISM_U(v[4])), "r"(PRISM_U(v[5])), "r"(PRISM_U(v[6])), "r"(PRISM_U(v[7])) : "memory");
    }
};
#undef PRISM_U
template <int N> struct Cols {
    static __device__ __forceinline__ void load(uint32_t t, uint32_t* r) {
        #pragma unroll
        for (int i = 0; i < N; i += 8) Cols<8>::load(t + i, r + i);
    }
    static __device__ __forceinline__ void store(uint32_t t, const float* v) {
        #pragma unroll
        for (int i = 0; i < N; i += 8) Cols<8>::store(t + i, v + i);
    }
};

// Instruction descriptor, kind::f16 with bf16 A and B, fp32 accumulate.
__host__ __device__ constexpr uint32_t idesc_bf16(int M, int N, int a_mn, int b_mn) {
    return (1u << 4) | (1u << 7) | (1u << 10) | ((uint32_t)a_mn << 15) | ((uint32_t)b_mn << 16) |
           ((uint32_t)(N >> 3) << 17) | ((uint32_t)(M >> 4) << 24);
}

// ---------------------------------------------------------------- activations
__device__ __forceinline__ float act_of(float z, int act) {
    switch (act) {
        case PRISM_ACT_GELU: return 0.5f * z * (1.f + erff(z * 0.70710678118654752f));
        case PRISM_ACT_GELU_TANH: {
            const float u = 0.79788456080286536f * (z + 0.044715f * z * z * z);
            return 0.5f * z * (1.f + tanhf(u));
        }
        case PRISM_ACT_SILU: return z / (1.f + expf(-z));
        default: return z;
    }
}
__device__ __forceinline__ float act_grad(float z, int act) {
    switch (act) {
        case PRISM_ACT_GELU:
            return 0.5f * (1.f + erff(z * 0.70710678118654752f)) + z * expf(-0.5f * z * z) * 0.39894228040143268f;
        case PRISM_ACT_GELU_TANH: {
            const float t = tanhf(0.79788456080286536f * (z + 0.044715f * z * z * z));
            return 0.5f * (1.f + t) + 0.5f * z * (1.f - t * t) * 0.79788456080286536f * (1.f + 0.134145f * z * z);
        }
        case PRISM_ACT_SILU: {
            const float s = 1.f / (1.f + expf(-z));
            return s * (1.f + z * (1.f - s));
        }
        default: return 1.f;
    }
}

// One lane's column c of C: where its elements lie.
struct Lane {
    char* y;
    const char* res;
    char* pre;
    int64_t ys, rs, ps;                    // bytes per row
    float bias;
    bool on;
};
__device__ __forceinline__ int64_t at(const Out& o, int c) {
    return o.hd ? (int64_t)(c / o.hd) * o.hs + c % o.hd : (int64_t)c;
}
__device__ __forceinline__ Lane lane_of(const Args& a, int c) {
    Lane l;
    l.on = c < a.C;
    c = l.on ? c : 0;
    const int yb = a.y.f32 ? 4 : 2, rb = a.res.f32 ? 4 : 2;
    l.y = static_cast<char*>(a.y.p) + at(a.y, c) * yb;
    l.ys = a.y.rs * yb;
    l.res = a.res.p ? static_cast<const char*>(a.res.p) + at(a.res, c) * rb : nullptr;
    l.rs = a.res.rs * rb;
    l.pre = a.pre.p ? static_cast<char*>(a.pre.p) + at(a.pre, c) * 2 : nullptr;
    l.ps = a.pre.rs * 2;
    l.bias = !a.bias ? 0.f : a.bias_f32 ? static_cast<const float*>(a.bias)[c]
                                        : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[c]);
    return l;
}
// Rows r0 .. r0 + n - 1 of the lane's column, n <= NC: bias, kept pre-activation, activation,
// residual, one rounding.  The rows' residuals are read before any of them is used (the
// result may be the residual's own memory: each element is read before it is written).
template <int NC>
__device__ __forceinline__ void emit(const Args& a, const Lane& l, int64_t r0, int n, const uint32_t* v) {
    if (!l.on) return;
    float res[NC];
    if (l.res) {
        #pragma unroll
        for (int j = 0; j < NC; ++j) {
            res[j] = 0.f;
            if (j < n) {
                const char* p = l.res + (r0 + j) * l.rs;
                res[j] = a.res.f32 ? *reinterpret_cast<const float*>(p)
                                   : __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p));
            }
        }
    }
    #pragma unroll
    for (int j = 0; j < NC; ++j) {
        if (j < n) {
            const int64_t r = r0 + j;
            float z = __uint_as_float(v[j]) + l.bias;
            // the kept z has the operands' 16 bits: the backward forms dz from it for 16-bit products
            if (l.pre) *reinterpret_cast<__nv_bfloat16*>(l.pre + r * l.ps) = __float2bfloat16_rn(z);
            if (a.act != PRISM_ACT_NONE) z = act_of(z, a.act);
            if (l.res) z += res[j];
            char* p = l.y + r * l.ys;
            if (a.y.f32) *reinterpret_cast<float*>(p) = z;
            else *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(z);
        }
    }
}

template <int CG, int BR>
struct Cfg {
    static constexpr int kA = 128 * kKB * 2;                 // bytes of a stage: A, then B
    static constexpr int kB = (BR / CG) * kKB * 2;
    static constexpr int kStage = kA + kB;
    // CG 2: one CTA per SM; CG 1: two per SM (TMEM 2 x 2 BR <= 512 columns)
    static constexpr int kStages = (CG == 2 ? 196608 : 98304) / kStage;
    static constexpr int kCols = 2 * BR;
    static constexpr int kHalf = BR / 2;                     // columns per epilogue warp
    static constexpr int kSmem = kStages * kStage + 1024;
};

// Grid: clusters of CG (a pair on one tile) or split CTAs (one tile, each a part of the
// contraction); clusters walk the tiles.
template <int CG, int BR>
__global__ void __launch_bounds__(kThreads, CG == 2 ? 1 : 2)
k_gemm(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Args a) {
    using F = Cfg<CG, BR>;
    constexpr int ST = F::kStages;
    extern __shared__ uint8_t smem_raw[];
    __shared__ uint64_t full[ST], empty[ST], acc_full[2], acc_empty[2];
    __shared__ uint32_t tmem_base;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const bool clustered = CG == 2 || a.split > 1;
    const uint32_t rank = clustered ? cluster_rank() : 0;
    const int group = CG == 2 ? 2 : a.split;
    const int first = blockIdx.x / group, step = gridDim.x / group;
    const int ntiles = a.tiles_c * a.tiles_r;
    // this CTA's part of the contraction
    const int kb0 = CG == 2 ? 0 : (int)((int64_t)a.kblocks * rank / a.split);
    const int kb1 = CG == 2 ? a.kblocks : (int)((int64_t)a.kblocks * (rank + 1) / a.split);
    const int nk = kb1 - kb0, nch = (nk + kChunkKB - 1) / kChunkKB;
    constexpr int W_PROD = kEpiWarps, W_MMA = kEpiWarps + 1;

    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&full[s], 1);
            mbar_init(&empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&acc_full[i], 1);
            mbar_init(&acc_empty[i], kEpiWarps * CG);
        }
        mbar_fence_init();
    }
    if (warp == W_PROD) {
        __syncwarp();
        alloc_tmem<CG>(&tmem_base, F::kCols);
    }
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    const uint32_t tmem = tmem_base;

    // tile t: bands of `band` row tiles, the columns of a band one after the other, so the
    // tiles that run at one time share their operands' rows in L2
    auto tile_at = [&](int t, int& tc, int& tr) {
        const int per = a.band * a.tiles_c, b = t / per, q = t - b * per;
        const int rows = min(a.band, a.tiles_r - b * a.band);
        tc = q / rows;
        tr = b * a.band + q - tc * rows;
    };

    if (warp == W_PROD) {
        if (lane == 0) {
            tma_prefetch_desc(&tm_a);
            tma_prefetch_desc(&tm_b);
            int it = 0;
            bool ok = true;
            for (int t = first; ok && t < ntiles; t += step) {
                int tc, tr;
                tile_at(t, tc, tr);
                const int c0 = tc * 128 * CG + (CG == 2 ? 128 * (int)rank : 0);
                const int64_t r0 = (int64_t)tr * BR + (CG == 2 ? (BR / 2) * (int)rank : 0);
                for (int kb = kb0; kb < kb1; ++kb, ++it) {
                    const int s = it % ST;
                    if (it >= ST && !mbar_wait(&empty[s], (it / ST - 1) & 1, a.err, 3101)) { ok = false; break; }
                    uint32_t bar = smem_u32(&full[s]);
                    if (CG == 2) bar = map_to(bar, 0);
                    // the pair's first CTA expects the bytes of both
                    if (CG == 1 || rank == 0) mbar_expect_tx(&full[s], CG * F::kStage);
                    const uint32_t da = ring + s * F::kStage, db = da + F::kA;
                    const int k = kb * kKB;
                    if (a.a.mn) {
                        #pragma unroll
                        for (int i = 0; i < 2; ++i) {
                            const int c = c0 + 64 * i;
                            tma3<CG>(da + i * 8192, &tm_a, bar, c % a.a.inner, k, c / a.a.inner);
                        }
                    } else {
                        tma3<CG>(da, &tm_a, bar, k % a.a.inner, c0, k / a.a.inner);
                    }
                    if (a.b.mn) {
                        #pragma unroll
                        for (int i = 0; i < (BR / CG + 63) / 64; ++i) {
                            const int r = (int)r0 + 64 * i;
                            tma3<CG>(db + i * 8192, &tm_b, bar, r % a.b.inner, k, r / a.b.inner);
                        }
                    } else {
                        tma3<CG>(db, &tm_b, bar, k % a.b.inner, (int)r0, k / a.b.inner);
                    }
                }
            }
            // every copy has landed before the block may end (an MMA issuer that gave up waits for none)
            if (CG == 1 || rank == 0)
                for (int i = it > ST ? it - ST : 0; i < it; ++i)
                    if (!mbar_try(&full[i % ST], (i / ST) & 1) && !mbar_wait(&full[i % ST], (i / ST) & 1, a.err, 3102)) break;
        }
    } else if (warp == W_MMA) {
        if (lane == 0 && (CG == 1 || rank == 0)) {
            const uint32_t idesc = idesc_bf16(128 * CG, BR, a.a.mn, a.b.mn);
            const uint32_t sa = a.a.mn ? 128 : 2, sb = a.b.mn ? 128 : 2;        // 16-byte units per 16 of k
            const uint32_t la = a.a.mn ? 8192 : 16, lb = a.b.mn ? 8192 : 16;
            int it = 0, ac = 0;
            bool ok = true;
            for (int t = first; ok && t < ntiles; t += step) {
                for (int ch = 0; ok && ch < nch; ++ch, ++ac) {
                    const int n = (int)((int64_t)nk * (ch + 1) / nch - (int64_t)nk * ch / nch), buf = ac & 1;
                    if (ac >= 2 && !mbar_wait(&acc_empty[buf], (ac / 2 - 1) & 1, a.err, 3201)) { ok = false; break; }
                    tc_fence_after();
                    for (int i = 0; i < n; ++i, ++it) {
                        const int s = it % ST;
                        if (!mbar_wait(&full[s], (it / ST) & 1, a.err, 3202)) { ok = false; break; }
                        tc_fence_after();
                        const uint32_t da = desc_lo(ring + s * F::kStage, la);
                        const uint32_t db = desc_lo(ring + s * F::kStage + F::kA, lb);
                        #pragma unroll
                        for (int kk = 0; kk < kKB / 16; ++kk)
                            mma<CG>(tmem + buf * BR, desc_from_lo(da + kk * sa), desc_from_lo(db + kk * sb), idesc,
                                    i > 0 || kk > 0 ? 1u : 0u);
                        commit<CG>(&empty[s]);
                    }
                    if (ok) commit<CG>(&acc_full[buf]);
                }
            }
        }
    } else {
        // ------------------------------------------------ epilogue
        // One chunk: straight from the accumulator, E columns at a time in a rolled loop (the
        // activations' code stays small).  Several: all but the last are added up in registers,
        // the sum goes back to the accumulator's columns and takes the same loop.
        constexpr int H = F::kHalf, CH = H < 16 ? H : 16, E = H < 16 ? H : 16;
        const int q = warp & 3, half = warp >> 2;
        const uint32_t at0 = tmem + ((uint32_t)(q * 32) << 16) + half * H;
        int ac = 0;
        bool ok = true;
        for (int t = first; ok && t < ntiles; t += step) {
            int tc, tr;
            tile_at(t, tc, tr);
            float v[H];
            for (int ch = 0; ch < nch; ++ch, ++ac) {
                const int buf = ac & 1;
                const bool last = ch == nch - 1;
                if (!__all_sync(0xffffffffu, mbar_wait_inline(&acc_full[buf], (ac / 2) & 1, a.err, 3301))) { ok = false; break; }
                tc_fence_after();
                if (nch > 1 || (CG == 1 && a.split > 1)) {
                    #pragma unroll
                    for (int i = 0; i < H / CH; ++i) {
                        uint32_t u[CH];
                        Cols<CH>::load(at0 + buf * BR + i * CH, u);
                        tmem_wait_ld();
                        #pragma unroll
                        for (int e = 0; e < CH; ++e)
                            v[i * CH + e] = ch == 0 ? __uint_as_float(u[e]) : v[i * CH + e] + __uint_as_float(u[e]);
                    }
                }
                if (last) {
                    if (CG == 1 && a.split > 1) {
                        // the parts meet in shared memory, column j of the tile at part[j][c].  The stages'
                        // memory is free: this tile is the block's only one and its last product is done.
                        float* part = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
                        #pragma unroll
                        for (int e = 0; e < H; ++e) part[(half * H + e) * 128 + q * 32 + lane] = v[e];
                    } else {
                        if (nch > 1) {
                            #pragma unroll
                            for (int i = 0; i < H / CH; ++i) Cols<CH>::store(at0 + buf * BR + i * CH, v + i * CH);
                            tmem_wait_st();
                        }
                        const Lane l = lane_of(a, tc * 128 * CG + (CG == 2 ? 128 * (int)rank : 0) + q * 32 + lane);
                        const int64_t r0 = (int64_t)tr * BR + half * H;
                        #pragma unroll 1
                        for (int e = 0; e < H; e += E) {
                            const int64_t left = a.R - (r0 + e);
                            if (left <= 0) break;
                            uint32_t u[E];
                            Cols<E>::load(at0 + buf * BR + e, u);
                            tmem_wait_ld();
                            emit<E>(a, l, r0 + e, left < E ? (int)left : E, u);
                            __syncwarp();
                        }
                    }
                }
                tc_fence_before();
                __syncwarp();
                if (lane == 0) {
                    if (CG == 2) arrive_at(map_to(smem_u32(&acc_empty[buf]), 0));
                    else mbar_arrive(&acc_empty[buf]);
                }
            }
        }
    }
    if (CG == 1 && a.split > 1) {
        __syncwarp();
        cluster_sync();
        // each CTA of the cluster sums its share of the columns over the parts, in rank order
        if (warp < kEpiWarps) {
            int tc, tr;
            tile_at(first, tc, tr);
            const int c = threadIdx.x & 127;
            const Lane l = lane_of(a, tc * 128 + c);
            const int j0 = BR * (int)rank / a.split, j1 = BR * ((int)rank + 1) / a.split;
            for (int j = j0 + (threadIdx.x >> 7); j < j1; j += 2) {
                const uint32_t my = ring + (uint32_t)(j * 128 + c) * 4;
                float s = 0.f;
                for (int p = 0; p < a.split; ++p) s += ld_peer(map_to(my, p));
                const int64_t r = (int64_t)tr * BR + j;
                const uint32_t u = __float_as_uint(s);
                if (r < a.R) emit<1>(a, l, r, 1, &u);
            }
        }
        __syncwarp();
        cluster_sync();                      // no CTA's memory goes while another reads it
    }
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    if (warp == W_PROD) {
        __syncwarp();
        free_tmem<CG>(tmem, F::kCols);
    }
}

// ------------------------------------------------- elementwise passes
// Rows [M][K] whose address or stride a TMA map cannot take (K or the stride not a multiple
// of 8 elements), copied to a padded stride in the workspace.
__global__ void __launch_bounds__(256) k_pack(const __nv_bfloat16* src, int64_t stride, int64_t rows, int K,
                                              __nv_bfloat16* dst, int64_t dstride) {
    for (int64_t r = blockIdx.x; r < rows; r += gridDim.x)
        for (int c = threadIdx.x; c < K; c += blockDim.x) dst[r * dstride + c] = src[r * stride + c];
}

struct DzArgs {
    Out dy, pre;                           // pre.p null: no activation
    int64_t M;
    int N, act;
    __nv_bfloat16* dz;                     // [M][dzs], or null (dy itself feeds the products)
    int64_t dzs;
    float* part;                           // [row chunks][N] column sums, or null
    int64_t rows;                          // rows of a chunk
};

// dz = dy act'(z) rounded to the products' 16 bits, and its column sums (of the unrounded
// values): a block takes 32 V columns of a chunk of rows, 8 rows at a time, and adds its
// sums in a fixed order.  HBM-bound: one read of dy (and z), one write of dz.
template <int V>
__global__ void __launch_bounds__(256) k_dz(const DzArgs a) {
    __shared__ float sm[8][32 * V + 1];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + cl) * V;
    const int64_t r1 = min(a.M, (int64_t)(blockIdx.y + 1) * a.rows);
    float sum[V];
    #pragma unroll
    for (int e = 0; e < V; ++e) sum[e] = 0.f;
    if (c < a.N) {
        const int64_t dyo = at(a.dy, c), preo = a.pre.p ? at(a.pre, c) : 0;
        #pragma unroll 4
        for (int64_t r = (int64_t)blockIdx.y * a.rows + rl; r < r1; r += 8) {
            float g[V], z[V];
            if (V == 8) {
                if (a.dy.f32) {
                    const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(a.dy.p) + dyo + r * a.dy.rs);
                    const float4 x = __ldcs(p), y = __ldcs(p + 1);
                    g[0] = x.x; g[1 % V] = x.y; g[2 % V] = x.z; g[3 % V] = x.w;
                    g[4 % V] = y.x; g[5 % V] = y.y; g[6 % V] = y.z; g[7 % V] = y.w;
                } else {
                    const uint4 x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.dy.p) + dyo + r * a.dy.rs));
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        g[(2 * e) % V] = __uint_as_float(u[e] << 16);
                        g[(2 * e + 1) % V] = __uint_as_float(u[e] & 0xffff0000u);
                    }
                }
                if (a.pre.p) {
                    const uint4 x = __ldcs(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(a.pre.p) + preo + r * a.pre.rs));
                    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
                    #pragma unroll
                    for (int e = 0; e < 4; ++e) {
                        z[(2 * e) % V] = __uint_as_float(u[e] << 16);
                        z[(2 * e + 1) % V] = __uint_as_float(u[e] & 0xffff0000u);
                    }
                }
            } else {
                g[0] = a.dy.f32 ? static_cast<const float*>(a.dy.p)[dyo + r * a.dy.rs]
                                : __bfloat162float(static_cast<const __nv_bfloat16*>(a.dy.p)[dyo + r * a.dy.rs]);
                if (a.pre.p) z[0] = __bfloat162float(static_cast<const __nv_bfloat16*>(a.pre.p)[preo + r * a.pre.rs]);
            }
            #pragma unroll
            for (int e = 0; e < V; ++e) {
                if (a.pre.p) g[e] *= act_grad(z[e], a.act);
                sum[e] += g[e];
            }
            if (a.dz) {
                if (V == 8)
                    *reinterpret_cast<uint4*>(a.dz + r * a.dzs + c) =
                        make_uint4(pack_bf16(g[0], g[1 % V]), pack_bf16(g[2 % V], g[3 % V]), pack_bf16(g[4 % V], g[5 % V]),
                                   pack_bf16(g[6 % V], g[7 % V]));
                else
                    a.dz[r * a.dzs + c] = __float2bfloat16_rn(g[0]);
            }
        }
    }
    if (!a.part) return;
    #pragma unroll
    for (int e = 0; e < V; ++e) sm[rl][cl * V + e] = sum[e];
    __syncthreads();
    for (int i = threadIdx.x; i < 32 * V; i += 256) {
        const int col = blockIdx.x * 32 * V + i;
        if (col >= a.N) break;
        float s = 0.f;
        #pragma unroll
        for (int k = 0; k < 8; ++k) s += sm[k][i];
        a.part[(int64_t)blockIdx.y * a.N + col] = s;
    }
}

// db: the chunks' sums in a fixed order, in 64 bits (a sum over every token: its parts cancel).
__global__ void __launch_bounds__(256) k_db(const float* part, int chunks, int N, float* db) {
    const int c = blockIdx.x * 32 + (threadIdx.x & 31), g = threadIdx.x >> 5;
    __shared__ double sm[8][32];
    double s = 0.0;
    if (c < N)
        for (int i = g; i < chunks; i += 8) s += part[(int64_t)i * N + c];
    sm[g][threadIdx.x & 31] = s;
    __syncthreads();
    if (g == 0 && c < N) {
        for (int i = 1; i < 8; ++i) s += sm[i][threadIdx.x];
        db[c] = (float)s;
    }
}

// ------------------------------------------------------------- host side
static PFN_cuTensorMapEncodeTiled_v12000 encode_fn() {
    static PFN_cuTensorMapEncodeTiled_v12000 fn = [] {
        void* f = nullptr;
        cudaDriverEntryPointQueryResult q;
        if (cudaGetDriverEntryPoint("cuTensorMapEncodeTiled", &f, cudaEnableDefault, &q) != cudaSuccess ||
            q != cudaDriverEntryPointSuccess)
            f = nullptr;
        return reinterpret_cast<PFN_cuTensorMapEncodeTiled_v12000>(f);
    }();
    return fn;
}

// An operand in memory: `heads` times [rows][inner], `ld` elements between rows (head-major
// tensors are contiguous: ld = inner).
struct Matrix {
    const void* p;
    int64_t rows, inner, ld;
    int heads;
};

// Boxes of 64 inner elements (128-byte swizzle) by `box` rows; what lies outside reads as zeros.
static int make_map(CUtensorMap* m, const Matrix& x, int box) {
    auto enc = encode_fn();
    if (!enc) return PRISM_ERR_CUDA;
    cuuint64_t dims[3] = {(cuuint64_t)x.inner, (cuuint64_t)x.rows, (cuuint64_t)x.heads};
    cuuint64_t strides[2] = {(cuuint64_t)x.ld * 2, (cuuint64_t)(x.rows * x.ld) * 2};
    cuuint32_t boxd[3] = {64, (cuuint32_t)box, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, const_cast<void*>(x.p), dims, strides, boxd, es,
                     CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PRISM_OK : PRISM_ERR_CUDA;
}

struct Shape {
    int cg, br, split;
};

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

// The tile of a product of R rows, C columns and kb stages.
static Shape shape_of(int64_t R, int64_t C, int kb, bool b_mn) {
    const int64_t pairs = ceil_div(R, 256) * ceil_div(C, 256);
    if (R > 128 && pairs >= 74) return Shape{2, 256, 1};
    Shape s{1, 128, 1};
    for (int br : {16, 32, 64})
        if (R <= br && !(b_mn && br < 64)) { s.br = br; break; }
    const int64_t tiles = ceil_div(R, s.br) * ceil_div(C, 128);
    while (s.split < 8 && tiles * s.split * 2 <= 2 * 148 && kb >= 8 * s.split) s.split *= 2;
    return s;
}

template <int CG, int BR>
static int launch(const CUtensorMap& ta, const CUtensorMap& tb, Args& a, int split, cudaStream_t s) {
    using F = Cfg<CG, BR>;
    a.split = split;
    a.tiles_c = (int)ceil_div(a.C, 128 * CG);
    const int64_t tr = ceil_div(a.R, BR);
    if (tr * a.tiles_c > 0x3fffffff) return PRISM_ERR_INVALID_ARG;
    a.tiles_r = (int)tr;
    a.band = 8;
    const int64_t tiles = tr * a.tiles_c;
    if (cudaFuncSetAttribute(k_gemm<CG, BR>, cudaFuncAttributeMaxDynamicSharedMemorySize, F::kSmem) != cudaSuccess)
        return PRISM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    const int group = CG == 2 ? 2 : split;
    cfg.gridDim = dim3((unsigned)(CG == 2 ? 2 * (tiles < 74 ? tiles : 74) : tiles * split));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = F::kSmem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)group;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, k_gemm<CG, BR>, ta, tb, a) == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA;
}

// C[r][c] = sum_k B[r][k] A[c][k]; K the contraction's length, a_mn / b_mn: the matrix's rows are k.
static int product(const Matrix& A, bool a_mn, const Matrix& B, bool b_mn, int64_t R, int C, int64_t K, Args& a,
                   cudaStream_t s) {
    a.R = R;
    a.C = C;
    a.kblocks = (int)ceil_div(K, kKB);
    a.a.mn = a_mn;
    a.b.mn = b_mn;
    a.a.inner = A.heads > 1 ? (int)A.inner : 0x7fffffff;
    a.b.inner = B.heads > 1 ? (int)B.inner : 0x7fffffff;
    const Shape sh = shape_of(R, C, a.kblocks, b_mn);
    CUtensorMap ta, tb;
    int st = make_map(&ta, A, a_mn ? kKB : 128);
    if (!st) st = make_map(&tb, B, b_mn ? kKB : sh.br / sh.cg);
    if (st) return st;
    if (sh.cg == 2) return launch<2, 256>(ta, tb, a, 1, s);
    switch (sh.br) {
        case 16: return launch<1, 16>(ta, tb, a, sh.split, s);
        case 32: return launch<1, 32>(ta, tb, a, sh.split, s);
        case 64: return launch<1, 64>(ta, tb, a, sh.split, s);
        default: return launch<1, 128>(ta, tb, a, sh.split, s);
    }
}

static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }
static bool bad_heads(int heads, int n) {
    if (heads == 0) return false;
    return heads < 0 || n % heads || (n / heads != 64 && n / heads != 128);
}

static bool bad_params(const prism_linear_params* p) {
    if (!p || p->M < 0 || p->M > 0x7fffffffLL - 255 || p->K < 1 || p->K > (1 << 24) || p->N < 1 || p->N > (1 << 24))
        return true;
    if (bad_heads(p->in_heads, p->K) || bad_heads(p->out_heads, p->N)) return true;
    if (p->activation < PRISM_ACT_NONE || p->activation > PRISM_ACT_SILU) return true;
    for (int d : {p->out_dtype, p->bias_dtype, p->dw_dtype})
        if (d != PRISM_BF16 && d != PRISM_F32) return true;
    const int64_t most = 1LL << 38;        // a tensor map's stride is below 2^40 bytes
    if (p->x_stride < p->K || p->w_stride < p->K || p->y_stride < p->N || p->r_stride < p->N) return true;
    for (int64_t t : {p->x_stride, p->w_stride, p->y_stride, p->r_stride})
        if (t > most / (p->M > p->N ? p->M + 1 : p->N + 1)) return true;
    if ((p->in_heads && p->x_stride != p->K) || (p->out_heads && (p->y_stride != p->N || p->r_stride != p->N)))
        return true;
    return false;
}

static int64_t pad8(int64_t n) { return (n + 7) / 8 * 8; }
static size_t up256(size_t n) { return (n + 255) / 256 * 256; }
static bool pack_x(const prism_linear_params* p) { return !p->in_heads && p->x_stride % 8; }
static bool pack_w(const prism_linear_params* p) { return p->w_stride % 8; }
static size_t x_bytes(const prism_linear_params* p) { return pack_x(p) ? up256((size_t)p->M * pad8(p->K) * 2) : 0; }
static size_t w_bytes(const prism_linear_params* p) { return pack_w(p) ? up256((size_t)p->N * pad8(p->K) * 2) : 0; }
// whether dz is formed in memory: through an activation, from fp32, or because dy's rows cannot feed a map
static bool forms_dz(const prism_linear_params* p) {
    return p->activation != PRISM_ACT_NONE || p->out_dtype == PRISM_F32 || (!p->out_heads && p->y_stride % 8);
}
static size_t dz_bytes(const prism_linear_params* p) { return forms_dz(p) ? up256((size_t)p->M * pad8(p->N) * 2) : 0; }

struct DzGrid {
    int v, x, y;
    int64_t rows;
};
// Row chunks so that about eight blocks per SM run; a chunk has at least 64 rows.
static DzGrid dz_grid(const prism_linear_params* p) {
    DzGrid g;
    g.v = p->N % 8 == 0 && p->y_stride % 8 == 0 ? 8 : 1;
    g.x = (int)ceil_div(p->N, 32 * g.v);
    int64_t y = ceil_div(8 * 148, g.x);
    if (y > ceil_div(p->M, 64)) y = ceil_div(p->M, 64);
    if (y < 1) y = 1;
    g.rows = ceil_div(p->M > 0 ? p->M : 1, y);
    g.y = (int)ceil_div(p->M > 0 ? p->M : 1, g.rows);
    return g;
}

static Out out_rows(const void* p, int64_t M, int N, int heads, int64_t stride, int f32) {
    Out o;
    o.p = const_cast<void*>(p);
    o.f32 = f32;
    o.hd = heads ? N / heads : 0;
    o.rs = heads ? o.hd : stride;
    o.hs = heads ? M * (int64_t)o.hd : 0;
    return o;
}

static Matrix matrix(const void* p, int64_t rows, int cols, int heads, int64_t stride) {
    if (heads) return Matrix{p, rows, cols / heads, cols / heads, heads};
    return Matrix{p, rows, cols, stride, 1};
}

// Bytes of a tensor of rows, to see whether two calls' arguments share any.
struct Span {
    uintptr_t lo;
    int64_t row, stride, rows;             // bytes
};
static Span span(const void* p, int64_t rows, int64_t cols, int heads, int64_t stride, int elt) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    if (heads || rows <= 1 || stride == cols) return Span{lo, (rows ? ((rows - 1) * (heads ? cols : stride) + cols) : 0) * elt, 0, 1};
    return Span{lo, cols * elt, stride * elt, rows};
}
static bool apart(const Span& x, const Span& y) {
    if (!x.lo || !y.lo) return true;
    const uintptr_t xe = x.lo + (uintptr_t)(x.stride * (x.rows - 1) + x.row), ye = y.lo + (uintptr_t)(y.stride * (y.rows - 1) + y.row);
    if (xe <= y.lo || ye <= x.lo) return true;
    if (x.stride != y.stride || !x.stride) return false;
    // columns of one buffer
    const uintptr_t d = y.lo >= x.lo ? y.lo - x.lo : x.lo - y.lo;
    const int64_t m = (int64_t)(d % (uintptr_t)x.stride);
    const int64_t lead = y.lo >= x.lo ? x.row : y.row, back = y.lo >= x.lo ? y.row : x.row;
    return m >= lead && x.stride - m >= back;
}

static int device_ok() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PRISM_ERR_UNSUPPORTED;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    return major == 10 && minor == 0 ? PRISM_OK : PRISM_ERR_UNSUPPORTED;
}

// A matrix of rows as the products read it: itself, or packed at `ws`.
static int operand(Matrix* m, const void* p, int64_t rows, int cols, int heads, int64_t stride, bool pack, char*& ws,
                   cudaStream_t s) {
    if (!pack) {
        *m = matrix(p, rows, cols, heads, stride);
        return PRISM_OK;
    }
    const int64_t ld = pad8(cols);
    auto* dst = reinterpret_cast<__nv_bfloat16*>(ws);
    ws += up256((size_t)rows * ld * 2);
    k_pack<<<(unsigned)(rows < 148 * 8 ? rows : 148 * 8), 256, 0, s>>>(static_cast<const __nv_bfloat16*>(p), stride, rows, cols,
                                                                       dst, ld);
    *m = Matrix{dst, rows, cols, ld, 1};
    return cudaGetLastError() == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA;
}

static int forward(const prism_linear_params* p, const void* x, const void* W, const void* bias, const void* residual,
                   void* y, void* pre, char* ws, int* err, cudaStream_t s) {
    Matrix mx, mw;
    int st = operand(&mx, x, p->M, p->K, p->in_heads, p->x_stride, pack_x(p), ws, s);
    if (!st) st = operand(&mw, W, p->N, p->K, 0, p->w_stride, pack_w(p), ws, s);
    if (st) return st;
    Args a{};
    const int f32 = p->out_dtype == PRISM_F32;
    a.y = out_rows(y, p->M, p->N, p->out_heads, p->y_stride, f32);
    if (residual) a.res = out_rows(residual, p->M, p->N, p->out_heads, p->r_stride, f32);
    if (pre) a.pre = out_rows(pre, p->M, p->N, p->out_heads, p->N, 0);
    a.bias = bias;
    a.bias_f32 = p->bias_dtype == PRISM_F32;
    a.act = p->activation;
    a.err = err;
    return product(mw, false, mx, false, p->M, p->N, p->K, a, s);
}

static int backward(const prism_linear_params* p, const void* dy, const void* x, const void* W, const void* pre, void* dx,
                    void* dW, float* db, char* ws, int* err, cudaStream_t s) {
    Matrix mx{}, mw{}, mz = matrix(dy, p->M, p->N, p->out_heads, p->y_stride);
    int st = PRISM_OK;
    const bool dz = forms_dz(p) && (dx || dW);
    if (dz || db) {
        DzArgs d{};
        d.dy = out_rows(dy, p->M, p->N, p->out_heads, p->y_stride, p->out_dtype == PRISM_F32);
        if (p->activation != PRISM_ACT_NONE) d.pre = out_rows(pre, p->M, p->N, p->out_heads, p->N, 0);
        d.M = p->M;
        d.N = p->N;
        d.act = p->activation;
        if (dz) {
            d.dz = reinterpret_cast<__nv_bfloat16*>(ws);
            d.dzs = pad8(p->N);
            mz = Matrix{d.dz, p->M, p->N, d.dzs, 1};
        }
        ws += dz_bytes(p);
        const DzGrid g = dz_grid(p);
        d.rows = g.rows;
        if (db) d.part = reinterpret_cast<float*>(ws);
        ws += up256((size_t)g.y * p->N * 4);
        if (g.v == 8) k_dz<8><<<dim3(g.x, g.y), 256, 0, s>>>(d);
        else k_dz<1><<<dim3(g.x, g.y), 256, 0, s>>>(d);
        if (db) k_db<<<(unsigned)ceil_div(p->N, 32), 256, 0, s>>>(d.part, g.y, p->N, db);
        if (cudaGetLastError() != cudaSuccess) return PRISM_ERR_CUDA;
    }
    if (dx) {
        st = operand(&mw, W, p->N, p->K, 0, p->w_stride, pack_w(p), ws, s);
        if (st) return st;
        Args a{};
        a.y = out_rows(dx, p->M, p->K, p->in_heads, p->K, 0);
        a.err = err;
        st = product(mw, true, mz, false, p->M, p->K, p->N, a, s);
        if (st) return st;
    }
    if (dW) {
        st = operand(&mx, x, p->M, p->K, p->in_heads, p->x_stride, pack_x(p), ws, s);
        if (st) return st;
        Args a{};
        a.y = out_rows(dW, p->N, p->K, 0, p->K, p->dw_dtype == PRISM_F32);
        a.err = err;
        st = product(mx, true, mz, true, p->N, p->K, p->M, a, s);
    }
    return st;
}

}  // namespace lin
}  // namespace prism

extern "C" size_t prism_linear_workspace_bytes(const prism_linear_params* p) {
    using namespace prism::lin;
    return bad_params(p) ? 0 : x_bytes(p) + w_bytes(p) + 256;
}

extern "C" int prism_linear(const prism_linear_params* p, const void* x, const void* W, const void* bias,
                            const void* residual, void* y, void* pre, void* workspace, size_t ws_bytes,
                            int32_t* dev_status, void* stream) {
    using namespace prism::lin;
    if (bad_params(p)) return PRISM_ERR_INVALID_ARG;
    if (p->M == 0) return PRISM_OK;
    if (!x || !W || !y || !dev_status) return PRISM_ERR_INVALID_ARG;
    for (const void* q : {x, W, bias, residual, (const void*)y, (const void*)pre, (const void*)workspace, (const void*)dev_status})
        if (!aligned16(q)) return PRISM_ERR_INVALID_ARG;
    const int e = p->out_dtype == PRISM_F32 ? 4 : 2;
    const Span sy = span(y, p->M, p->N, p->out_heads, p->y_stride, e);
    const Span sp = span(pre, p->M, p->N, p->out_heads, p->N, 2);
    const Span in[3] = {span(x, p->M, p->K, p->in_heads, p->x_stride, 2), span(W, p->N, p->K, 0, p->w_stride, 2),
                        span(bias, 1, p->N, 0, p->N, p->bias_dtype == PRISM_F32 ? 4 : 2)};
    for (const Span& i : in)
        if (!apart(sy, i) || !apart(sp, i)) return PRISM_ERR_INVALID_ARG;
    const Span sr = span(residual, p->M, p->N, p->out_heads, p->r_stride, e);
    if (!apart(sy, sp) || !apart(sp, sr)) return PRISM_ERR_INVALID_ARG;
    if (!apart(sy, sr) && !(y == residual && (p->y_stride == p->r_stride || p->M == 1))) return PRISM_ERR_INVALID_ARG;
    const size_t need = x_bytes(p) + w_bytes(p);
    if (need && !workspace) return PRISM_ERR_INVALID_ARG;
    if (need > ws_bytes) return PRISM_ERR_WORKSPACE;
    if (int st = device_ok()) return st;
    nvtxRangePushA("prism linear");
    const int st = forward(p, x, W, bias, residual, y, pre, static_cast<char*>(workspace), dev_status,
                           static_cast<cudaStream_t>(stream));
    nvtxRangePop();
    return st;
}

extern "C" size_t prism_linear_bwd_workspace_bytes(const prism_linear_params* p) {
    using namespace prism::lin;
    if (bad_params(p)) return 0;
    return x_bytes(p) + w_bytes(p) + dz_bytes(p) + up256((size_t)dz_grid(p).y * p->N * 4) + 256;
}

extern "C" int prism_linear_bwd(const prism_linear_params* p, const void* dy, const void* x, const void* W,
                                const void* pre, void* dx, void* dW, float* db, void* workspace, size_t ws_bytes,
                                int32_t* dev_status, void* stream) {
    using namespace prism::lin;
    if (bad_params(p)) return PRISM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    for (const void* q : {dy, x, W, pre, (const void*)dx, (const void*)dW, (const void*)db, (const void*)workspace,
                          (const void*)dev_status})
        if (!aligned16(q)) return PRISM_ERR_INVALID_ARG;
    if (p->M == 0) {         // no rows: the gradients by the weights are zero
        if (dW && cudaMemsetAsync(dW, 0, (size_t)p->N * p->K * (p->dw_dtype == PRISM_F32 ? 4 : 2), s) != cudaSuccess)
            return PRISM_ERR_CUDA;
        if (db && cudaMemsetAsync(db, 0, (size_t)p->N * 4, s) != cudaSuccess) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    if (!dy || !dev_status || (dx && !W) || (dW && !x) || (p->activation != PRISM_ACT_NONE && !pre))
        return PRISM_ERR_INVALID_ARG;
    const int e = p->out_dtype == PRISM_F32 ? 4 : 2;
    const Span in[4] = {span(dy, p->M, p->N, p->out_heads, p->y_stride, e), span(x, p->M, p->K, p->in_heads, p->x_stride, 2),
                        span(W, p->N, p->K, 0, p->w_stride, 2), span(pre, p->M, p->N, p->out_heads, p->N, 2)};
    const Span out[3] = {span(dx, p->M, p->K, p->in_heads, p->K, 2),
                         span(dW, p->N, p->K, 0, p->K, p->dw_dtype == PRISM_F32 ? 4 : 2), span(db, 1, p->N, 0, p->N, 4)};
    for (int i = 0; i < 3; ++i) {
        for (const Span& q : in)
            if (!apart(out[i], q)) return PRISM_ERR_INVALID_ARG;
        for (int j = 0; j < i; ++j)
            if (!apart(out[i], out[j])) return PRISM_ERR_INVALID_ARG;
    }
    if (!dx && !dW && !db) return PRISM_OK;
    const size_t need = prism_linear_bwd_workspace_bytes(p) - 256;
    if (need && !workspace) return PRISM_ERR_INVALID_ARG;
    if (need > ws_bytes) return PRISM_ERR_WORKSPACE;
    if (int st = device_ok()) return st;
    nvtxRangePushA("prism linear bwd");
    const int st = backward(p, dy, x, W, pre, dx, dW, db, static_cast<char*>(workspace), dev_status, s);
    nvtxRangePop();
    return st;
}
