// prism_linear.cu -- the projections around the attention on sm_100a tensor cores:
//     z = x W^T + b,  y = act(z) + residual            (forward)
//     dz = dy act'(z),  dx = dz W,  dW = dz^T x,  db = sum_m dz   (gradients)
// with x, y and their gradients either rows [M][K] or head-major [heads][M][D], so the
// input projection writes what prism_plan reads and the output projection reads what
// prism_attn_fwd writes, without a transposing copy.
//
// Every product is C[r][c] = sum_k X[r][k] Y[c][k], c the contiguous index of C.  An operand
// is a TMA map (inner, rows, heads) with the contraction along the inner index (K-major) or
// along the rows (MN-major); head-major inner coordinates split into (channel, head):
//     forward  X = x  [M][K] K-major     Y = W [N][K] K-major
//     dx       X = dz [M][N] K-major     Y = W [N][K] MN-major
//     dW       X = dz [M][N] MN-major    Y = x [M][K] MN-major
// Two kernels:
//   k_tile  many rows: TMEM lanes are rows, columns are c.  A pair of CTAs (cta_group::2)
//           shares a 256 x BN tile, or one CTA has 128 x 128, whose contraction a cluster may
//           split.  A warp's results leave through a 4 KB stage and TMA stores.  Bound by the
//           tensor cores: 522 to 530 cycles per stage of 512 at BN 256 (92,160 x 5,120 x 5,120
//           in 3.1 ms, 1,530 TFLOP/s, while the card is below its power cap; 1,250 to 1,370 over
//           seconds).
//   k_few   up to 64 rows: TMEM lanes are c and columns are rows, so few tokens are a small
//           N of the instruction instead of an M tile of padding.  Bound by HBM's read of W
//           (one token against 30,720 x 5,120: 54 us, 5.8 TB/s); a cluster splits the contraction
//           (13 tokens, 5,120 x 5,120: 10.7 us).
//
// Warp roles: epilogue warps (TMEM lane quarter w % 4, columns by w / 4), then a TMA producer that
// also allocates TMEM, then the MMA issuer.  Two TMEM accumulators alternate, so the next products run
// while the epilogue reads the last.
//
// The tensor core's fp32 accumulation truncates: over a contraction of 16,384 the result
// is low by 1.6e-5 of its size, growing linearly (measured with standard normal operands;
// 4.7e-6 at 5,120).  So a contraction is cut into chunks, each summed by the tensor core into
// a fresh accumulator, and the chunks are added in registers with round-to-nearest: chunks of
// 768 elements where the result is fp32 (7e-7 low; 20,000 x 5,120 x 5,120 takes 1 to 3% longer
// than with 2,048, 1.7e-6 low), of 16,384 where it is rounded to bf16 (a hundredth of half a step).
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

constexpr int kKB = 64;                    // contraction elements per stage (128-byte rows)
constexpr int kChunkF32 = 12;              // stages per accumulation chunk (see above): 768 elements
constexpr int kChunkBF16 = 256;            // and 16,384 where the result keeps 16 bits

struct Operand {
    int mn;                                // MN-major
    int shift;                             // K-major: k >> shift is the head, the rest the channel (31: one head)
    int slabs;                             // MN-major: slabs of 64 before the next head; 0: no whole slabs
};

struct Out {
    void* p;                               // element (r, c): p + head(c) hs + r rs + c in head
    int64_t rs, hs;
    int hd;                                // channels per head; 0 = one head
    int f32;
    int vec;                               // 16-byte accesses at multiples of 16 bytes of a row
};

struct Args {
    Operand a, b;                          // the operand along the tensor core's M, and along its N
    int64_t R;                             // rows of C
    int C;                                 // columns of C
    int kblocks;                           // stages of the whole contraction
    int split;                             // CTAs of a cluster that share a tile's contraction
    int chunk;                             // stages per accumulation chunk
    int tiles_c, tiles_r, band;
    Out y, pre, res;
    int fast;                              // results leave by TMA; residual and kept z in 16-byte accesses
    const void* bias;
    int bias_f32, act;
    int* err;
};

// ---------------------------------------------------------------- PTX
template <int CG>
__device__ __forceinline__ void tma4(uint32_t dst, const void* tmap, uint32_t bar, int32_t x, int32_t y, int32_t z, int32_t v) {
    if (CG == 2)
        // the barrier may lie in the pair's other CTA
        asm volatile("cp.async.bulk.tensor.4d.cta_group::2.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5, %6}], [%2];"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(v) : "memory");
    else
        asm volatile("cp.async.bulk.tensor.4d.shared::cluster.global.mbarrier::complete_tx::bytes"
                     " [%0], [%1, {%3, %4, %5, %6}], [%2];"
                     :: "r"(dst), "l"(reinterpret_cast<uint64_t>(tmap)), "r"(bar), "r"(x), "r"(y), "r"(z), "r"(v) : "memory");
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
// An arrival at another CTA's barrier that says only that TMEM has been read (the tcgen05 fence
// before it orders that): no memory of this thread is published, so it need not wait for the
// thread's stores in flight, as a release at cluster scope did (2,000 to 4,000 cycles per tile).
__device__ __forceinline__ void arrive_at(uint32_t cluster_addr) {
    asm volatile("mbarrier.arrive.shared::cluster.b64 _, [%0];" :: "r"(cluster_addr) : "memory");
}
// One lane of a converged warp, the same one every time.
__device__ __forceinline__ bool elect() {
    uint32_t p;
    asm volatile("{\n\t.reg .pred p;\n\telect.sync _|p, 0xffffffff;\n\tselp.u32 %0, 1, 0, p;\n\t}" : "=r"(p));
    return p != 0;
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

// The same for a whole warp: true in every lane, or false in every lane.
__device__ __forceinline__ bool warp_wait(uint64_t* bar, uint32_t parity, int* err, int where) {
    return __all_sync(0xffffffffu, mbar_wait_inline(bar, parity, err, where));
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
// tanh(u) = 2 / (1 + e^-2u) - 1, so the tanh form is z / (1 + e^-2u), like SiLU's z / (1 + e^-z):
// one __expf (its error grows with |argument|, where the quotient no longer depends on it) and
// one quotient.
__device__ __forceinline__ float logistic(float t) { return __fdividef(1.f, 1.f + __expf(-t)); }
__device__ __forceinline__ float tanh_arg(float z) { return 1.5957691216057308f * (z + 0.044715f * z * z * z); }
// The normal distribution's Phi(z): Abramowitz and Stegun's formula 7.1.26 for erfc(x),
// x = |z| / sqrt 2, t = 1 / (1 + p x), a polynomial of degree 5 in t times e^(-x^2), within 1.5e-7.
__device__ __forceinline__ float normal_cdf(float z) {
    const float x = fabsf(z) * 0.70710678118654752f;
    const float t = __fdividef(1.f, fmaf(0.3275911f, x, 1.f));
    const float e = __expf(-x * x);
    const float q = t * fmaf(t, fmaf(t, fmaf(t, fmaf(t, 1.061405429f, -1.453152027f), 1.421413741f), -0.284496736f),
                             0.254829592f);
    const float tail = 0.5f * q * e;
    return z > 0.f ? 1.f - tail : tail;
}
__device__ __forceinline__ float act_of(float z, int act) {
    switch (act) {
        case PRISM_ACT_GELU: return z * normal_cdf(z);
        case PRISM_ACT_GELU_TANH: return z * logistic(tanh_arg(z));
        case PRISM_ACT_SILU: return z * logistic(z);
        default: return z;
    }
}
__device__ __forceinline__ float rcp(float x) {
    float y;
    asm("rcp.approx.ftz.f32 %0, %1;" : "=f"(y) : "f"(x));
    return y;
}
// g0 act'(z0), g1 act'(z1): the derivatives of the same forms, two at a time (packed products and
// sums; k_dz's instructions are what bounds it once its loads are in flight: 36,342 x 5,492 with GELU
// 427 us, one at a time 492 us; 32,760 x 8,960 with GELU 305 us, was 336).
template <int ACT>
__device__ __forceinline__ void times_grad(float& g0, float& g1, float z0, float z1) {
    constexpr float kLog2e = 1.4426950408889634f;
    float a0, a1, q0, q1, s0, s1, u0, u1, w0, w1;            // z^2, ...
    if (ACT == PRISM_ACT_GELU) {
        // Phi(z) + z phi(z), by normal_cdf's formula
        fmul2(a0, a1, z0, z1, z0, z1);
        fmul2(w0, w1, a0, a1, -0.5f * kLog2e, -0.5f * kLog2e);
        const float e0 = ex2(w0), e1 = ex2(w1);
        constexpr float p = 0.3275911f * 0.70710678118654752f;
        ffma2(u0, u1, fabsf(z0), fabsf(z1), p, p, 1.f, 1.f);
        const float t0 = rcp(u0), t1 = rcp(u1);
        ffma2(q0, q1, t0, t1, 1.061405429f, 1.061405429f, -1.453152027f, -1.453152027f);
        ffma2(q0, q1, t0, t1, q0, q1, 1.421413741f, 1.421413741f);
        ffma2(q0, q1, t0, t1, q0, q1, -0.284496736f, -0.284496736f);
        ffma2(q0, q1, t0, t1, q0, q1, 0.254829592f, 0.254829592f);
        fmul2(s0, s1, t0, t1, 0.5f * e0, 0.5f * e1);
        fmul2(q0, q1, q0, q1, s0, s1);                       // Phi(-|z|)
        s0 = z0 > 0.f ? 1.f - q0 : q0;
        s1 = z1 > 0.f ? 1.f - q1 : q1;
        fmul2(w0, w1, z0, z1, e0, e1);
        ffma2(s0, s1, w0, w1, 0.39894228040143268f, 0.39894228040143268f, s0, s1);
    } else if (ACT == PRISM_ACT_GELU_TANH) {
        // s + z s (1 - s) t', t = 1.596 (z + 0.0447 z^3), s = 1 / (1 + e^-t)
        fmul2(a0, a1, z0, z1, z0, z1);
        constexpr float c = 1.5957691216057308f, d = c * 0.044715f;
        ffma2(q0, q1, a0, a1, -d * kLog2e, -d * kLog2e, -c * kLog2e, -c * kLog2e);
        fmul2(q0, q1, q0, q1, z0, z1);
        s0 = rcp(1.f + ex2(q0));
        s1 = rcp(1.f + ex2(q1));
        ffma2(q0, q1, a0, a1, 3.f * d, 3.f * d, c, c);       // t'
        q0 = fminf(q0, 3e38f);                               // (s (1 - s) is 0 where z^2 overflows)
        q1 = fminf(q1, 3e38f);
        ffma2(u0, u1, s0, s1, -1.f, -1.f, 1.f, 1.f);
        fmul2(w0, w1, z0, z1, s0, s1);
        fmul2(w0, w1, w0, w1, u0, u1);
        ffma2(s0, s1, w0, w1, q0, q1, s0, s1);
    } else {
        // s (1 + z (1 - s))
        fmul2(q0, q1, z0, z1, -kLog2e, -kLog2e);
        s0 = rcp(1.f + ex2(q0));
        s1 = rcp(1.f + ex2(q1));
        ffma2(u0, u1, s0, s1, -1.f, -1.f, 1.f, 1.f);
        ffma2(u0, u1, z0, z1, u0, u1, 1.f, 1.f);
        fmul2(s0, s1, s0, s1, u0, u1);
    }
    fmul2(g0, g1, g0, g1, s0, s1);
}

template <int NC>
__device__ __forceinline__ void activate(float* z, int act) {
    switch (act) {
        case PRISM_ACT_GELU:
            #pragma unroll
            for (int i = 0; i < NC; ++i) z[i] = act_of(z[i], PRISM_ACT_GELU);
            break;
        case PRISM_ACT_GELU_TANH:
            #pragma unroll
            for (int i = 0; i < NC; ++i) z[i] = act_of(z[i], PRISM_ACT_GELU_TANH);
            break;
        case PRISM_ACT_SILU:
            #pragma unroll
            for (int i = 0; i < NC; ++i) z[i] = act_of(z[i], PRISM_ACT_SILU);
            break;
        default: break;
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
__device__ __forceinline__ void emit(const Args& a, const Lane& l, int64_t r0, int n, const float* v) {
    if (!l.on) return;
    float res[NC], z[NC];
    if (l.res) {
        const char* p = l.res + r0 * l.rs;
        if (a.res.f32) {
            #pragma unroll
            for (int j = 0; j < NC; ++j, p += l.rs) res[j] = j < n ? *reinterpret_cast<const float*>(p) : 0.f;
        } else {
            #pragma unroll
            for (int j = 0; j < NC; ++j, p += l.rs)
                res[j] = j < n ? __bfloat162float(*reinterpret_cast<const __nv_bfloat16*>(p)) : 0.f;
        }
    }
    #pragma unroll
    for (int j = 0; j < NC; ++j) z[j] = v[j] + l.bias;
    if (l.pre) {
        // the kept z has the operands' 16 bits: the backward forms dz from it for 16-bit products
        char* p = l.pre + r0 * l.ps;
        #pragma unroll
        for (int j = 0; j < NC; ++j, p += l.ps)
            if (j < n) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(z[j]);
    }
    activate<NC>(z, a.act);
    if (l.res) {
        #pragma unroll
        for (int j = 0; j < NC; ++j) z[j] += res[j];
    }
    char* p = l.y + r0 * l.ys;
    if (a.y.f32) {
        #pragma unroll
        for (int j = 0; j < NC; ++j, p += l.ys)
            if (j < n) *reinterpret_cast<float*>(p) = z[j];
    } else {
        #pragma unroll
        for (int j = 0; j < NC; ++j, p += l.ys)
            if (j < n) *reinterpret_cast<__nv_bfloat16*>(p) = __float2bfloat16_rn(z[j]);
    }
}

// The roles that both kernels share.  BM x BN: the tile along the tensor core's M (of all CTAs
// of the group) and N.
template <int CG, int BN>
struct Cfg {
    static constexpr int kM = 128 * CG;
    static constexpr int kA = 128 * kKB * 2;                 // bytes of a stage: A, then B
    static constexpr int kB = (BN / CG) * kKB * 2;
    static constexpr int kStage = kA + kB;
    // the pair's CTAs and the single one have an SM to themselves; k_few's run two per SM
    static constexpr int kStages = (CG == 2 ? 163840 : BN >= 128 ? 196608 : 98304) / kStage;
    static constexpr int kCols = BN > 128 ? 512 : BN > 64 ? 256 : BN > 32 ? 128 : BN > 16 ? 64 : 32;   // 2 BN, a power of two
    // epilogue: a warpgroup per 64 columns of a wide tile (the sums of 64 columns fit a thread's
    // registers beside the rest: with 128, and half the warps, they spilled), two on a narrow one
    static constexpr int kCol = BN >= 128 ? 64 : BN / 2;     // columns per epilogue warp
    static constexpr int kEpi = 4 * (BN / kCol);             // epilogue warps
    static constexpr int kThreads = (kEpi + 2) * 32;
    static constexpr int kRing = kStages * kStage;
};

template <int ST>
struct Bars {
    uint64_t full[ST], empty[ST], acc_full[2], acc_empty[2];
    uint32_t tmem_base;
};

// What a CTA works on.
struct Work {
    uint32_t rank;                         // in its cluster
    int first, step, ntiles;               // tiles first, first + step, ...
    int kb0, kb1, nk, nch;                 // stages of the contraction, accumulation chunks
};
template <int CG>
__device__ __forceinline__ Work work_of(const Args& a) {
    Work w;
    w.rank = CG == 2 || a.split > 1 ? cluster_rank() : 0;
    const int group = CG == 2 ? 2 : a.split;
    w.first = blockIdx.x / group;
    w.step = gridDim.x / group;
    w.ntiles = a.tiles_c * a.tiles_r;
    w.kb0 = CG == 2 ? 0 : (int)((int64_t)a.kblocks * w.rank / a.split);
    w.kb1 = CG == 2 ? a.kblocks : (int)((int64_t)a.kblocks * (w.rank + 1) / a.split);
    w.nk = w.kb1 - w.kb0;
    w.nch = (w.nk + a.chunk - 1) / a.chunk;
    return w;
}
// Tile t: bands of `band` row tiles, the columns of a band one after the other, so the tiles
// that run at one time share their operands' rows in L2.
__device__ __forceinline__ void tile_at(const Args& a, int t, int& tc, int& tr) {
    const int per = a.band * a.tiles_c, b = t / per, q = t - b * per;
    const int rows = min(a.band, a.tiles_r - b * a.band);
    tc = q / rows;
    tr = b * a.band + q - tc * rows;
}

// Barriers and TMEM; returns the TMEM address.
template <int CG, int BN, int ST>
__device__ __forceinline__ uint32_t start(Bars<ST>& sm, int warp) {
    if (threadIdx.x == 0) {
        for (int s = 0; s < ST; ++s) {
            mbar_init(&sm.full[s], 1);
            mbar_init(&sm.empty[s], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&sm.acc_full[i], 1);
            mbar_init(&sm.acc_empty[i], Cfg<CG, BN>::kEpi * CG);
        }
        mbar_fence_init();
    }
    if (warp == Cfg<CG, BN>::kEpi) {
        __syncwarp();
        alloc_tmem<CG>(&sm.tmem_base, Cfg<CG, BN>::kCols);
    }
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();
    else __syncthreads();
    tc_fence_after();
    return sm.tmem_base;
}
template <int CG, int BN>
__device__ __forceinline__ void finish_cta(uint32_t tmem, int warp) {
    tc_fence_before();
    __syncwarp();
    if (CG == 2) cluster_sync();           // the pair's other CTA may still signal this one's barriers
    else __syncthreads();
    tc_fence_after();
    if (warp == Cfg<CG, BN>::kEpi) {
        __syncwarp();
        free_tmem<CG>(tmem, Cfg<CG, BN>::kCols);
    }
}

// One operand's tile at the producer: the fixed coordinates of its copies.  K-major: one box of
// ROWS rows by 64 k.  MN-major: 64 k by slabs of 64 columns, one box of every slab where the
// map has a slab dimension, else a box each.
template <int CG, int ROWS>
struct Feed {
    const void* tm;
    int mn, shift, mask, two, x0, y0, z0, v0;
    __device__ __forceinline__ Feed(const void* tm, const Operand& o) : tm(tm), mn(o.mn), shift(o.shift) {
        mask = o.shift == 31 ? 0x7fffffff : (1 << o.shift) - 1;
        two = o.mn && !o.slabs && ROWS > 64;
        x0 = y0 = z0 = v0 = 0;
    }
    __device__ __forceinline__ void tile(const Operand& o, int o0) {
        if (!mn) {
            y0 = o0;
        } else if (o.slabs) {
            const int sl = o0 >> 6;
            v0 = sl / o.slabs;
            z0 = sl - v0 * o.slabs;
        } else {
            x0 = o0;
        }
    }
    __device__ __forceinline__ void load(uint32_t dst, uint32_t bar, int k) const {
        const int x = mn ? x0 : k & mask, y = mn ? k : y0, z = mn ? z0 : k >> shift;
        tma4<CG>(dst, tm, bar, x, y, z, v0);
        if (two) tma4<CG>(dst + 8192, tm, bar, x + 64, y, z, v0);
    }
};

// The two issuing loops run once per 64 of k, beside products of 256 to 512 cycles, and their
// instructions are a latency chain: with divisions, address maps and constants reloaded in the
// loop the producer took 626 to 780 cycles per stage and bound the products.  So what is fixed
// is in registers before the loop, and the whole warp runs it on values that are the same in
// every lane, one elected lane only issuing: copies and products take their operands from the
// warp's uniform registers, which a branch of one lane has to fill one by one.

// The TMA producer (one warp).  ROWS_ARE_M: C's rows lie along the tensor core's M.
template <int CG, int BN, bool ROWS_ARE_M, int ST>
__device__ __forceinline__ void produce(const void* tm_a, const void* tm_b, const Args& a, const Work& w, Bars<ST>& sm,
                                        uint32_t ring) {
    using F = Cfg<CG, BN>;
    if (elect()) {
        tma_prefetch_desc(tm_a);
        tma_prefetch_desc(tm_b);
    }
    __syncwarp();
    Feed<CG, 128> fa(tm_a, a.a);
    Feed<CG, BN / CG> fb(tm_b, a.b);
    // the pair's first CTA has the barrier of both CTAs' copies and expects their bytes
    const uint32_t bars = CG == 2 ? map_to(smem_u32(sm.full), 0) : smem_u32(sm.full);
    const bool expects = CG == 1 || w.rank == 0;
    int* const err = a.err;
    int s = 0, round = 0;
    bool ok = true;
    for (int t = w.first; ok && t < w.ntiles; t += w.step) {
        int tc, tr;
        tile_at(a, t, tc, tr);
        fa.tile(a.a, (ROWS_ARE_M ? tr : tc) * F::kM + (CG == 2 ? 128 * (int)w.rank : 0));
        fb.tile(a.b, (ROWS_ARE_M ? tc : tr) * BN + (CG == 2 ? (BN / 2) * (int)w.rank : 0));
        const int k1 = w.kb1 * kKB;
        for (int k = w.kb0 * kKB; k < k1; k += kKB) {
            if (round && !warp_wait(&sm.empty[s], (round - 1) & 1, err, 3101)) { ok = false; break; }
            const uint32_t da = ring + s * F::kStage, bar = bars + s * 8;
            if (elect()) {
                if (expects) mbar_expect_tx(&sm.full[s], CG * F::kStage);
                fa.load(da, bar, k);
                fb.load(da + F::kA, bar, k);
            }
            __syncwarp();
            if (++s == ST) { s = 0; ++round; }
        }
    }
    // Before the block may end, every copy has landed and every product's arrival at this CTA's `empty`
    // has come: the arrivals of the last stages have no other wait, and in a pair they come from the
    // other CTA.  (After a wait that gave up, too: then for at most a tenth of a second.)
    const bool lands = CG == 1 || w.rank == 0;
    const uint64_t t0 = globaltimer_ns();
    for (int i = 0; i < ST; ++i) {
        const int uses = round + (i < s ? 1 : 0);
        if (!uses) continue;
        const uint32_t par = (uses - 1) & 1;
        if (lands)
            while (!mbar_try(&sm.full[i], par) && globaltimer_ns() - t0 < kWaitNs / 10) {}
        while (!mbar_try(&sm.empty[i], par) && globaltimer_ns() - t0 < kWaitNs / 10) {}
    }
    __syncwarp();
}

// The MMA issuer (one warp; of a pair, the first CTA's).
template <int CG, int BN, int ST>
__device__ __forceinline__ void issue(const Args& a, const Work& w, Bars<ST>& sm, uint32_t ring, uint32_t tmem) {
    using F = Cfg<CG, BN>;
    const uint32_t idesc = idesc_bf16(128 * CG, BN, a.a.mn, a.b.mn);
    const uint32_t sa = a.a.mn ? 128 : 2, sb = a.b.mn ? 128 : 2;        // 16-byte units per 16 of k
    const uint32_t da0 = desc_lo(ring, a.a.mn ? 8192 : 16), db0 = desc_lo(ring + F::kA, a.b.mn ? 8192 : 16);
    int* const err = a.err;
    int s = 0, par = 0, ac = 0;
    bool ok = true;
    for (int t = w.first; ok && t < w.ntiles; t += w.step) {
        for (int ch = 0; ok && ch < w.nch; ++ch, ++ac) {
            const int n = (int)((int64_t)w.nk * (ch + 1) / w.nch - (int64_t)w.nk * ch / w.nch), buf = ac & 1;
            if (ac >= 2 && !warp_wait(&sm.acc_empty[buf], (ac / 2 - 1) & 1, err, 3201)) { ok = false; break; }
            tc_fence_after();
            const uint32_t acc = tmem + buf * BN;
            for (int i = 0; i < n; ++i) {
                if (!warp_wait(&sm.full[s], par, err, 3202)) { ok = false; break; }
                tc_fence_after();
                const uint32_t da = da0 + s * (F::kStage >> 4), db = db0 + s * (F::kStage >> 4);
                if (elect()) {
                    mma<CG>(acc, desc_from_lo(da), desc_from_lo(db), idesc, i > 0 ? 1u : 0u);
                    #pragma unroll
                    for (int kk = 1; kk < kKB / 16; ++kk)
                        mma<CG>(acc, desc_from_lo(da + kk * sa), desc_from_lo(db + kk * sb), idesc, 1u);
                    commit<CG>(&sm.empty[s]);
                    if (i == n - 1) commit<CG>(&sm.acc_full[buf]);
                }
                __syncwarp();
                if (++s == ST) { s = 0; par ^= 1; }
            }
        }
    }
}

// An epilogue warp's columns of an accumulator added to v (or taken, from the first chunk).
template <int H>
__device__ __forceinline__ void add_columns(uint32_t t, float* v, bool take) {
    constexpr int CH = 8;
    #pragma unroll
    for (int i = 0; i < H / CH; ++i) {
        uint32_t u[CH];
        Cols<CH>::load(t + i * CH, u);
        tmem_wait_ld();
        #pragma unroll
        for (int e = 0; e < CH; ++e) v[i * CH + e] = take ? __uint_as_float(u[e]) : v[i * CH + e] + __uint_as_float(u[e]);
    }
}
template <int CG, int ST>
__device__ __forceinline__ void release(Bars<ST>& sm, int buf, int lane) {
    tc_fence_before();
    __syncwarp();
    if (lane == 0) {
        if (CG == 2) arrive_at(map_to(smem_u32(&sm.acc_empty[buf]), 0));
        else mbar_arrive(&sm.acc_empty[buf]);
    }
}

// ---------------------------------------------------------------- rows of results
// NC results of row r from column c on (bias, kept z, activation, residual), n of them inside C.
// ACT false: bias and residual alone; RES false: no residual.
template <int NC, bool ACT = true, bool RES = true>
__device__ __forceinline__ void finish(const Args& a, float* z, int64_t r, int c, int n) {
    if (a.bias) {
        if (n == NC) {
            if (a.bias_f32) {
                #pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const float4 b = __ldg(reinterpret_cast<const float4*>(static_cast<const float*>(a.bias) + c + i));
                    z[i] += b.x; z[i + 1] += b.y; z[i + 2] += b.z; z[i + 3] += b.w;
                }
            } else {
                #pragma unroll
                for (int i = 0; i < NC; i += 4) {
                    const uint2 b = __ldg(reinterpret_cast<const uint2*>(static_cast<const __nv_bfloat16*>(a.bias) + c + i));
                    z[i] += __uint_as_float(b.x << 16); z[i + 1] += __uint_as_float(b.x & 0xffff0000u);
                    z[i + 2] += __uint_as_float(b.y << 16); z[i + 3] += __uint_as_float(b.y & 0xffff0000u);
                }
            }
        } else {
            #pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i < n) z[i] += a.bias_f32 ? static_cast<const float*>(a.bias)[c + i]
                                              : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[c + i]);
        }
    }
    if (ACT && a.pre.p && r < a.R) {
        // the kept z has the operands' 16 bits: the backward forms dz from it for 16-bit products
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.pre.p) + at(a.pre, c) + r * a.pre.rs;
        if (a.pre.vec && n == NC) {
            #pragma unroll
            for (int i = 0; i < NC; i += 4)
                *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16(z[i], z[i + 1]), pack_bf16(z[i + 2], z[i + 3]));
        } else {
            #pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i < n) p[i] = __float2bfloat16_rn(z[i]);
        }
    }
    if (ACT) activate<NC>(z, a.act);
    if (RES && a.res.p && r < a.R) {
        if (a.res.f32) {
            const float* p = static_cast<const float*>(a.res.p) + at(a.res, c) + r * a.res.rs;
            if (a.res.vec && n == NC) {
                float4 x[NC / 4];
                #pragma unroll
                for (int i = 0; i < NC / 4; ++i) x[i] = reinterpret_cast<const float4*>(p)[i];
                #pragma unroll
                for (int i = 0; i < NC / 4; ++i) {
                    z[4 * i] += x[i].x; z[4 * i + 1] += x[i].y; z[4 * i + 2] += x[i].z; z[4 * i + 3] += x[i].w;
                }
            } else {
                #pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (i < n) z[i] += p[i];
            }
        } else {
            const __nv_bfloat16* p = static_cast<const __nv_bfloat16*>(a.res.p) + at(a.res, c) + r * a.res.rs;
            if (a.res.vec && n == NC) {
                uint2 x[NC / 4];
                #pragma unroll
                for (int i = 0; i < NC / 4; ++i) x[i] = reinterpret_cast<const uint2*>(p)[i];
                #pragma unroll
                for (int i = 0; i < NC / 4; ++i) {
                    z[4 * i] += __uint_as_float(x[i].x << 16); z[4 * i + 1] += __uint_as_float(x[i].x & 0xffff0000u);
                    z[4 * i + 2] += __uint_as_float(x[i].y << 16); z[4 * i + 3] += __uint_as_float(x[i].y & 0xffff0000u);
                }
            } else {
                #pragma unroll
                for (int i = 0; i < NC; ++i)
                    if (i < n) z[i] += __bfloat162float(p[i]);
            }
        }
    }
}
// The same results stored by the thread itself.
template <int NC>
__device__ __forceinline__ void store_row(const Args& a, const float* z, int64_t r, int c, int n) {
    if (r >= a.R) return;
    if (a.y.f32) {
        float* p = static_cast<float*>(a.y.p) + at(a.y, c) + r * a.y.rs;
        if (a.y.vec && n == NC) {
            #pragma unroll
            for (int i = 0; i < NC; i += 4) *reinterpret_cast<float4*>(p + i) = make_float4(z[i], z[i + 1], z[i + 2], z[i + 3]);
        } else {
            #pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i < n) p[i] = z[i];
        }
    } else {
        __nv_bfloat16* p = static_cast<__nv_bfloat16*>(a.y.p) + at(a.y, c) + r * a.y.rs;
        if (a.y.vec && n == NC) {
            #pragma unroll
            for (int i = 0; i < NC; i += 4)
                *reinterpret_cast<uint2*>(p + i) = make_uint2(pack_bf16(z[i], z[i + 1]), pack_bf16(z[i + 2], z[i + 3]));
        } else {
            #pragma unroll
            for (int i = 0; i < NC; ++i)
                if (i < n) p[i] = __float2bfloat16_rn(z[i]);
        }
    }
}
__device__ __forceinline__ float ld_shared_f32(uint32_t a) {
    float v;
    asm volatile("ld.shared.f32 %0, [%1];" : "=f"(v) : "r"(a) : "memory");
    return v;
}
__device__ __forceinline__ void tma_store_3d(const void* tmap, uint32_t src, int32_t x, int32_t y, int32_t z) {
    asm volatile("cp.async.bulk.tensor.3d.global.shared::cta.bulk_group [%0, {%2, %3, %4}], [%1];"
                 :: "l"(reinterpret_cast<uint64_t>(tmap)), "r"(src), "r"(x), "r"(y), "r"(z) : "memory");
}
__device__ __forceinline__ float4 ld_peer4(uint32_t cluster_addr) {
    float4 v;
    asm volatile("ld.shared::cluster.v4.f32 {%0, %1, %2, %3}, [%4];"
                 : "=f"(v.x), "=f"(v.y), "=f"(v.z), "=f"(v.w) : "r"(cluster_addr) : "memory");
    return v;
}


// The parts of a tile's sum, ROWS rows of 128 results at pitch PITCH in the ring of each CTA of
// the cluster: each CTA takes its share of the rows, adds the parts in rank order and finishes
// them.  U rows per warp at a time: their loads from the other CTAs are in flight together.
constexpr int kJoinWarps = 8;              // the epilogue warps of the kernels that split
template <int ROWS, int PITCH>
__device__ __forceinline__ void join(const Args& a, const Work& w, uint32_t ring, int warp, int lane, int tc, int tr) {
    constexpr int U = ROWS >= 64 ? 4 : ROWS / 16;
    const int j0 = ROWS * (int)w.rank / a.split, j1 = ROWS * ((int)w.rank + 1) / a.split;
    const int c = tc * 128 + lane * 4, n = min(4, a.C - c);
    for (int j = j0 + warp; j < j1; j += kJoinWarps * U) {
        float z[U][4];
        #pragma unroll
        for (int u = 0; u < U; ++u) z[u][0] = z[u][1] = z[u][2] = z[u][3] = 0.f;
        #pragma unroll 2
        for (int p = 0; p < a.split; ++p) {
            const uint32_t from = map_to(ring + (uint32_t)(j * PITCH + lane * 4) * 4, p);
            float4 x[U];
            #pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u * kJoinWarps < j1) x[u] = ld_peer4(from + u * kJoinWarps * PITCH * 4);
            #pragma unroll
            for (int u = 0; u < U; ++u)
                if (j + u * kJoinWarps < j1) {
                    z[u][0] += x[u].x; z[u][1] += x[u].y; z[u][2] += x[u].z; z[u][3] += x[u].w;
                }
        }
        #pragma unroll
        for (int u = 0; u < U; ++u) {
            const int64_t r = (int64_t)tr * ROWS + j + u * kJoinWarps;
            if (j + u * kJoinWarps < j1 && r < a.R && n > 0) {
                finish<4>(a, z[u], r, c, n);
                store_row<4>(a, z[u], r, c, n);
            }
        }
    }
}

// ---------------------------------------------------------------- few rows
// Lanes are columns c of C, accumulator columns its rows.  Grid: a cluster of `split` CTAs per
// tile of 128 c; the parts of the sum meet in shared memory and are added in rank order.
template <int BN>
__global__ void __launch_bounds__(Cfg<1, BN>::kThreads, 2)
k_few(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b, const Args a) {
    using F = Cfg<1, BN>;
    constexpr int ST = F::kStages, H = F::kCol, E = H < 16 ? H : 16;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<ST> sm;
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const Work w = work_of<1>(a);
    const uint32_t tmem = start<1, BN, ST>(sm, warp);
    int tc, tr;
    tile_at(a, w.first, tc, tr);
    if (warp == F::kEpi) {
        produce<1, BN, false, ST>(&tm_a, &tm_b, a, w, sm, ring);
    } else if (warp == F::kEpi + 1) {
        issue<1, BN, ST>(a, w, sm, ring, tmem);
    } else {
        const int q = warp & 3, half = warp >> 2;
        const uint32_t at0 = tmem + ((uint32_t)(q * 32) << 16) + half * H;
        float v[H];
        bool ok = true;
        for (int ch = 0; ch < w.nch; ++ch) {
            const int buf = ch & 1;
            if (!warp_wait(&sm.acc_full[buf], (ch / 2) & 1, a.err, 3301)) { ok = false; break; }
            tc_fence_after();
            add_columns<H>(at0 + buf * BN, v, ch == 0);
            release<1>(sm, buf, lane);
        }
        if (!ok) {
            // the status block says so; the results are not complete
        } else if (a.split > 1) {
            // column j of the tile at part[j][c].  The stages' memory is free: this tile is the
            // block's only one and its last product is done.
            float* part = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
            #pragma unroll
            for (int e = 0; e < H; ++e) part[(half * H + e) * 128 + q * 32 + lane] = v[e];
        } else {
            const Lane l = lane_of(a, tc * 128 + q * 32 + lane);
            const int64_t r0 = (int64_t)tr * BN + half * H;
            #pragma unroll
            for (int e = 0; e < H; e += E) {
                const int64_t left = a.R - (r0 + e);
                if (left > 0) emit<E>(a, l, r0 + e, left < E ? (int)left : E, v + e);
            }
        }
    }
    if (a.split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < F::kEpi) join<BN, 128>(a, w, ring, warp, lane, tc, tr);
        __syncwarp();
        cluster_sync();                    // no CTA's memory goes while another reads it
    }
    finish_cta<1, BN>(tmem, warp);
}

constexpr int kStageOut = 4096;            // an epilogue warp's outgoing 32 rows of 128 bytes
template <int CG, int BN>
constexpr int tile_smem() { return Cfg<CG, BN>::kRing + Cfg<CG, BN>::kEpi * kStageOut + 1024; }
constexpr int kPartPitch = 132;            // floats per row of a part (CG 1): rows start 4 banks apart

__device__ __forceinline__ uint4 ld_shared_v4(uint32_t a) {
    uint4 v;
    asm volatile("ld.shared.v4.b32 {%0, %1, %2, %3}, [%4];" : "=r"(v.x), "=r"(v.y), "=r"(v.z), "=r"(v.w) : "r"(a) : "memory");
    return v;
}
// The stage's rows of 8 `chunks` bf16 to the kept z, `chunks` lanes to a row (an access touches four
// lines or eight; a lane writing along its own row touched thirty-two).
__device__ __forceinline__ void pre_out(const Args& a, uint32_t stage, int64_t r0, int c, int lane, int chunks) {
    const Out& o = a.pre;
    __nv_bfloat16* base = static_cast<__nv_bfloat16*>(o.p) + at(o, c);
    const int sh = chunks == 8 ? 3 : 2;
    for (int i = 0; i < chunks; ++i) {
        const int row = (lane + 32 * i) >> sh, k = lane & (chunks - 1), cols = a.C - c - k * 8;
        const uint4 x = ld_shared_v4(stage + swz128(row, k));
        if (r0 + row >= a.R || cols <= 0) continue;
        __nv_bfloat16* p = base + (r0 + row) * o.rs + k * 8;
        if (cols >= 8) {
            *reinterpret_cast<uint4*>(p) = x;
        } else {
            const uint32_t w[4] = {x.x, x.y, x.z, x.w};
            #pragma unroll
            for (int j = 0; j < 7; ++j)
                if (j < cols) reinterpret_cast<uint16_t*>(p)[j] = (uint16_t)(w[j / 2] >> (16 * (j & 1)));
        }
    }
}
// The lane's own row of the stage, 32 columns from column `from` of the piece on, added to z.
__device__ __forceinline__ void add_own(bool f32, uint32_t stage, int lane, int from, float* z) {
    if (f32) {
        #pragma unroll
        for (int k = 0; k < 8; ++k) {
            const uint4 x = ld_shared_v4(stage + swz128(lane, from / 4 + k));
            z[4 * k] += __uint_as_float(x.x); z[4 * k + 1] += __uint_as_float(x.y);
            z[4 * k + 2] += __uint_as_float(x.z); z[4 * k + 3] += __uint_as_float(x.w);
        }
    } else {
        #pragma unroll
        for (int k = 0; k < 4; ++k) {
            const uint4 x = ld_shared_v4(stage + swz128(lane, from / 8 + k));
            const uint32_t u[4] = {x.x, x.y, x.z, x.w};
            #pragma unroll
            for (int e = 0; e < 4; ++e) {
                z[8 * k + 2 * e] += __uint_as_float(u[e] << 16);
                z[8 * k + 2 * e + 1] += __uint_as_float(u[e] & 0xffff0000u);
            }
        }
    }
}
__device__ __forceinline__ void put_bf16(uint32_t stage, int lane, int from, const float* z) {
    #pragma unroll
    for (int k = 0; k < 4; ++k)
        st_shared_v4(stage + swz128(lane, from / 8 + k), pack_bf16(z[8 * k], z[8 * k + 1]), pack_bf16(z[8 * k + 2], z[8 * k + 3]),
                     pack_bf16(z[8 * k + 4], z[8 * k + 5]), pack_bf16(z[8 * k + 6], z[8 * k + 7]));
}
__device__ __forceinline__ void put_own(bool f32, uint32_t stage, int lane, int from, const float* z) {
    if (f32) {
        #pragma unroll
        for (int k = 0; k < 8; ++k)
            st_shared_v4(stage + swz128(lane, from / 4 + k), __float_as_uint(z[4 * k]), __float_as_uint(z[4 * k + 1]),
                         __float_as_uint(z[4 * k + 2]), __float_as_uint(z[4 * k + 3]));
    } else {
        put_bf16(stage, lane, from, z);
    }
}
// A warp's residual pieces, brought into its stage by TMA (plain loads of them were limited by the
// little L1 that the ring leaves: 38,701 x 504 x 17,056 in fp32 takes 1.5 ms, took 2.1).  One load
// at a time.
struct Residual {
    const void* tm;
    uint64_t* bar;
    int issued = 0, waited = 0;
    // to 4 KB that must be free; every lane's accesses to them come first
    __device__ __forceinline__ void issue(const Args& a, uint32_t to, int64_t r0, int c, int lane) {
        fence_proxy_async_smem();
        __syncwarp();
        if (lane == 0) {
            const int zh = a.res.hd ? c / a.res.hd : 0;
            mbar_expect_tx(bar, 4096);
            asm volatile("cp.async.bulk.tensor.3d.shared::cluster.global.mbarrier::complete_tx::bytes"
                         " [%0], [%1, {%3, %4, %5}], [%2];"
                         :: "r"(to), "l"(reinterpret_cast<uint64_t>(tm)), "r"(smem_u32(bar)), "r"(c - zh * a.res.hd),
                            "r"((int)r0), "r"(zh) : "memory");
        }
        ++issued;
    }
    __device__ __forceinline__ bool wait(const Args& a) {
        const bool ok = warp_wait(bar, waited & 1, a.err, 3302);
        waited += ok;
        return ok;
    }
    // a load that a warp which gave up has not waited for
    __device__ __forceinline__ void drain() {
        const uint64_t t0 = globaltimer_ns();
        if (issued != waited)
            while (!mbar_try(bar, waited & 1) && globaltimer_ns() - t0 < kWaitNs / 10) {}
        __syncwarp();
    }
};

__device__ __forceinline__ float bias_at(const Args& a, int c) {
    if (c >= a.C) return 0.f;
    return a.bias_f32 ? __ldg(static_cast<const float*>(a.bias) + c)
                      : __bfloat162float(static_cast<const __nv_bfloat16*>(a.bias)[c]);
}

// Lanes are rows of C.  Grid: pairs (CG 2) walk the tiles; or a cluster of `split` CTAs per tile.
// Four epilogues for pairs, so that each keeps its registers, and one that has all for single CTAs:
//   kSingle  one chunk, rows at 16-byte alignment: straight from the accumulator's columns.
//   kDirect  several chunks, no activation, no kept z, the same alignment.  The registers' sums leave
//            from the registers, and the last accumulator is handed back as soon as it is added; only
//            then come bias and residual, whose first piece is in the stage since before the chunks and
//            whose second takes the first's place (behind a block's last product, where nothing else
//            runs, a place in the ring: 2,600 x 5,000 x 2,000 65 us, 67 in the first's place).  Sums that
//            started from the residual were rounded at its size every chunk, and took longer: 92,160 x
//            5,120 x 5,120 of zeros with an fp32 residual 2.75 ms, 2.69 now; 9,472 x 800 x 5,120 100 us,
//            92 now.
//   kSums    several chunks, the same alignment: their sum goes back to the last one's columns and
//            leaves from there like a single chunk's.
//   kRows    rows of any alignment.
constexpr int kSingle = 0, kDirect = 1, kSums = 2, kRows = 3, kAll = 4;
template <int CG, int BN, int MODE>
__global__ void __launch_bounds__(Cfg<CG, BN>::kThreads, 1)
k_tile(const __grid_constant__ CUtensorMap tm_a, const __grid_constant__ CUtensorMap tm_b,
       const __grid_constant__ CUtensorMap tm_y, const __grid_constant__ CUtensorMap tm_r, const Args a) {
    using F = Cfg<CG, BN>;
    constexpr int ST = F::kStages, H = F::kCol;
    extern __shared__ uint8_t smem_raw[];
    __shared__ Bars<ST> sm;
    __shared__ uint64_t res_full[F::kEpi];
    const uint32_t ring = (smem_u32(smem_raw) + 1023u) & ~1023u;
    const int warp = __shfl_sync(0xffffffffu, (int)(threadIdx.x >> 5), 0), lane = threadIdx.x & 31;
    const Work w = work_of<CG>(a);
    if (threadIdx.x == 0)
        for (int i = 0; i < F::kEpi; ++i) mbar_init(&res_full[i], 1);
    const uint32_t tmem = start<CG, BN, ST>(sm, warp);
    if (warp == F::kEpi) {
        produce<CG, BN, true, ST>(&tm_a, &tm_b, a, w, sm, ring);
    } else if (warp == F::kEpi + 1) {
        if (CG == 1 || w.rank == 0) issue<CG, BN, ST>(a, w, sm, ring, tmem);
    } else {
        const int q = warp & 3, half = warp >> 2;
        const uint32_t at0 = tmem + ((uint32_t)(q * 32) << 16) + half * H;
        const uint32_t stage = ring + F::kRing + warp * kStageOut;
        constexpr bool DIRECT = MODE == kDirect;
        const bool parts = CG == 1 && a.split > 1;
        int ac = 0;
        bool ok = true;
        // the 32 rows at `from`, from column c on, leave; what lies outside C is not written
        auto leave = [&](uint32_t from, int c, int64_t r0) {
            fence_proxy_async_smem();
            __syncwarp();
            if (lane == 0) {
                const int zh = a.y.hd ? c / a.y.hd : 0;
                tma_store_3d(&tm_y, from, c - zh * a.y.hd, (int)r0, zh);
                bulk_commit();
            }
        };
        auto stage_free = [&]() {
            if (lane == 0) bulk_wait_read0();                  // its last store has read it
            __syncwarp();
        };
        const int piece = a.y.f32 ? 32 : 64;                   // columns of a stage's row
        Residual res{&tm_r, &res_full[warp]};
        for (int t = w.first; ok && t < w.ntiles; t += w.step) {
            int tc, tr;
            tile_at(a, t, tc, tr);
            const int64_t r0 = (int64_t)tr * F::kM + (CG == 2 ? 128 * (int)w.rank : 0) + q * 32;
            const int c0 = tc * BN + half * H;
            int buf = ac & 1;
            if ((DIRECT || (MODE == kSingle && !a.pre.p)) && a.res.p && c0 < a.C) {        // while the products run
                stage_free();
                res.issue(a, stage, r0, c0, lane);
            }
            if (DIRECT || (MODE != kSingle && (w.nch > 1 || parts))) {
                // the chunks add up in registers
                float v[H], b0 = 0.f, b1 = 0.f;
                const bool last = t + w.step >= w.ntiles;
                auto take_bias = [&]() {                       // a column's bias in its lane
                    b0 = bias_at(a, c0 + lane);
                    b1 = bias_at(a, c0 + 32 + lane);
                };
                for (int ch = 0; ch < w.nch; ++ch, ++ac) {
                    buf = ac & 1;
                    if (DIRECT && a.bias && last && ch == w.nch - 1) take_bias();
                    if (!warp_wait(&sm.acc_full[buf], (ac / 2) & 1, a.err, 3301)) { ok = false; break; }
                    tc_fence_after();
                    add_columns<H>(at0 + buf * BN, v, ch == 0);
                    if (DIRECT || ch < w.nch - 1) release<CG>(sm, buf, lane);
                }
                if (!ok) break;
                if (DIRECT) {
                    if (c0 >= a.C) continue;
                    // behind a block's last product the ring is free, and a second piece has a place of its own there
                    const bool two = a.y.f32 && c0 + 32 < a.C;
                    const uint32_t second = last ? ring + warp * kStageOut : stage;
                    if (a.res.p) {
                        if (!res.wait(a)) { ok = false; break; }
                        if (two && last) res.issue(a, second, r0, c0 + 32, lane);
                    } else {
                        stage_free();
                    }
                    if (a.bias) {
                        if (!last) take_bias();
                        #pragma unroll
                        for (int e = 0; e < H; ++e) v[e] += __shfl_sync(0xffffffffu, e < 32 ? b0 : b1, e & 31);
                    }
                    if (a.res.p) {
                        add_own(a.y.f32, stage, lane, 0, v);
                        if (!a.y.f32) add_own(false, stage, lane, 32, v + 32);
                    }
                    put_own(a.y.f32, stage, lane, 0, v);
                    if (!a.y.f32) put_bf16(stage, lane, 32, v + 32);
                    leave(stage, c0, r0);
                    if (two) {
                        if (!last) stage_free();
                        if (a.res.p) {
                            if (!last) res.issue(a, second, r0, c0 + 32, lane);
                            if (!res.wait(a)) { ok = false; break; }
                            add_own(true, second, lane, 0, v + 32);
                        }
                        put_own(true, second, lane, 0, v + 32);
                        leave(second, c0 + 32, r0);
                    }
                    continue;
                }
                if (parts) {
                    // row by row into the stages' memory, free since this tile is the block's only one
                    float* part = reinterpret_cast<float*>(smem_raw + (ring - smem_u32(smem_raw)));
                    #pragma unroll
                    for (int e = 0; e < H; e += 4)
                        *reinterpret_cast<float4*>(part + (q * 32 + lane) * kPartPitch + half * H + e) =
                            make_float4(v[e], v[e + 1], v[e + 2], v[e + 3]);
                    release<CG>(sm, buf, lane);
                    break;
                }
                // the sum goes back to the last chunk's columns
                #pragma unroll
                for (int i = 0; i < H / 8; ++i) Cols<8>::store(at0 + buf * BN + i * 8, v + i * 8);
                tmem_wait_st();
            } else {
                if (!warp_wait(&sm.acc_full[buf], (ac / 2) & 1, a.err, 3301)) { ok = false; break; }
                tc_fence_after();
                ++ac;
            }
            auto load32 = [&](int e, float* z) {
                uint32_t u[32];
                PRISM_TMEM_LD32(at0 + buf * BN + e, u);
                tmem_wait_ld();
                #pragma unroll
                for (int i = 0; i < 32; ++i) z[i] = __uint_as_float(u[i]);
            };
            if (MODE != kRows && (MODE != kAll || a.fast)) {
                #pragma unroll 1
                for (int e = 0; e < H; e += piece) {
                    const int c = c0 + e;
                    if (c >= a.C) break;
                    if (res.issued == res.waited) stage_free();
                    if (a.pre.p) {
                        // the kept z has the operands' 16 bits: the backward forms dz from it for 16-bit products
                        #pragma unroll 1
                        for (int k = 0; k < piece && c + k < a.C; k += 32) {
                            float z[32];
                            load32(e + k, z);
                            finish<32, false, false>(a, z, r0 + lane, c + k, min(32, a.C - c - k));
                            put_bf16(stage, lane, k, z);
                        }
                        __syncwarp();
                        pre_out(a, stage, r0, c, lane, piece / 8);
                        __syncwarp();
                    }
                    if (a.res.p) {
                        if (res.issued == res.waited) res.issue(a, stage, r0, c, lane);
                        if (!res.wait(a)) { ok = false; break; }
                    }
                    #pragma unroll 1
                    for (int k = 0; k < piece && c + k < a.C; k += 32) {
                        float z[32];
                        load32(e + k, z);
                        // the accumulator is free once its last columns are in registers
                        if (e + k + 32 >= H || c + k + 32 >= a.C) release<CG>(sm, buf, lane);
                        finish<32, false, false>(a, z, r0 + lane, c + k, min(32, a.C - c - k));
                        activate<32>(z, a.act);
                        if (a.res.p) add_own(a.y.f32, stage, lane, k, z);
                        put_own(a.y.f32, stage, lane, k, z);
                    }
                    leave(stage, c, r0);
                }
            } else {
                // rows at any alignment: turned in the stage, so that a row's columns lie in the lanes
                // (a lane writing along its own row took 7.1 ms where this takes 2.1, 24,743 rows of
                // 1,904 by 13,119)
                #pragma unroll 1
                for (int e = 0; e < H && c0 + e < a.C; e += 32) {
                    const int c = c0 + e;
                    float z[32];
                    load32(e, z);
                    if (e + 32 >= H || c + 32 >= a.C) release<CG>(sm, buf, lane);
                    #pragma unroll
                    for (int k = 0; k < 8; ++k)
                        st_shared_v4(stage + swz128(lane, k), __float_as_uint(z[4 * k]), __float_as_uint(z[4 * k + 1]),
                                     __float_as_uint(z[4 * k + 2]), __float_as_uint(z[4 * k + 3]));
                    __syncwarp();
                    const Lane l = lane_of(a, c + lane);
                    #pragma unroll 1
                    for (int j = 0; j < 32; j += 16) {
                        const int64_t left = a.R - (r0 + j);
                        if (left <= 0) break;
                        float x[16];
                        #pragma unroll
                        for (int i = 0; i < 16; ++i) x[i] = ld_shared_f32(stage + swz128(j + i, lane >> 2) + (lane & 3) * 4);
                        emit<16>(a, l, r0 + j, left < 16 ? (int)left : 16, x);
                    }
                    __syncwarp();
                }
            }
            if (c0 >= a.C) release<CG>(sm, buf, lane);         // (a tile's half without columns)
        }
        res.drain();
        if (lane == 0) bulk_wait0();
    }
    if (CG == 1 && a.split > 1) {
        __syncwarp();
        cluster_sync();
        if (warp < F::kEpi) {
            int tc, tr;
            tile_at(a, w.first, tc, tr);
            join<128, kPartPitch>(a, w, ring, warp, lane, tc, tr);
        }
        __syncwarp();
        cluster_sync();                    // no CTA's memory goes while another reads it
    }
    finish_cta<CG, BN>(tmem, warp);
}

// ------------------------------------------------- elementwise passes
// Eight bf16 from element `at` on of a tensor of `total` elements at a 16-byte aligned address,
// at any offset: the one or two aligned 16-byte words that hold them, shifted together.  (The
// second word is read only where all of it lies in the tensor.)
__device__ __forceinline__ uint4 load8(const __nv_bfloat16* base, int64_t at, int64_t total) {
    const int64_t a = at & ~int64_t(7);
    const int o = (int)(at & 7);
    const uint4 lo = __ldg(reinterpret_cast<const uint4*>(base + a));
    if (o == 0) return lo;
    uint32_t w[8] = {lo.x, lo.y, lo.z, lo.w, 0, 0, 0, 0};
    if (a + 16 <= total) {
        const uint4 hi = __ldg(reinterpret_cast<const uint4*>(base + a + 8));
        w[4] = hi.x; w[5] = hi.y; w[6] = hi.z; w[7] = hi.w;
    } else {
        const uint16_t* p = reinterpret_cast<const uint16_t*>(base + a + 8);
        #pragma unroll
        for (int i = 0; i < 8; ++i)
            if (i < o) w[4 + i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
    }
    // the first of the words, and half a word more where o is odd
    const uint32_t h = (o & 1) * 16;
    switch (o >> 1) {
        case 0: return make_uint4(__funnelshift_r(w[0], w[1], h), __funnelshift_r(w[1], w[2], h),
                                  __funnelshift_r(w[2], w[3], h), __funnelshift_r(w[3], w[4], h));
        case 1: return make_uint4(__funnelshift_r(w[1], w[2], h), __funnelshift_r(w[2], w[3], h),
                                  __funnelshift_r(w[3], w[4], h), __funnelshift_r(w[4], w[5], h));
        case 2: return make_uint4(__funnelshift_r(w[2], w[3], h), __funnelshift_r(w[3], w[4], h),
                                  __funnelshift_r(w[4], w[5], h), __funnelshift_r(w[5], w[6], h));
        default: return make_uint4(__funnelshift_r(w[3], w[4], h), __funnelshift_r(w[4], w[5], h),
                                   __funnelshift_r(w[5], w[6], h), __funnelshift_r(w[6], w[7], h));
    }
}
__device__ __forceinline__ void unpack8(const uint4& x, float* f) {
    const uint32_t u[4] = {x.x, x.y, x.z, x.w};
    #pragma unroll
    for (int e = 0; e < 4; ++e) {
        f[2 * e] = __uint_as_float(u[e] << 16);
        f[2 * e + 1] = __uint_as_float(u[e] & 0xffff0000u);
    }
}
// Row r's columns c .. c + 7 of a tensor as fp32; columns from N on read as zeros.
__device__ __forceinline__ void read8(const Out& o, int64_t off, int64_t r, int c, int N, int64_t total, float* f) {
    const int64_t at0 = off + r * o.rs;
    const int n = min(8, N - c);
    if (o.f32) {
        const float* p = static_cast<const float*>(o.p) + at0;
        if (o.vec && n == 8) {
            const float4 x = __ldg(reinterpret_cast<const float4*>(p)), y = __ldg(reinterpret_cast<const float4*>(p) + 1);
            f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
            f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < n ? __ldg(p + e) : 0.f;
        }
    } else {
        const __nv_bfloat16* b = static_cast<const __nv_bfloat16*>(o.p);
        if (n == 8) {
            unpack8(load8(b, at0, total), f);
        } else {
            #pragma unroll
            for (int e = 0; e < 8; ++e) f[e] = e < n ? __bfloat162float(b[at0 + e]) : 0.f;
        }
    }
}

// Rows [rows][K] whose stride a TMA map cannot take (no multiple of 8 elements), copied to a
// padded stride in the workspace (the padding is zero); and copied again to `dst2`, where given.
__global__ void __launch_bounds__(256) k_pack(const __nv_bfloat16* src, int64_t stride, int64_t rows, int K,
                                              __nv_bfloat16* dst, __nv_bfloat16* dst2, int groups) {
    const int64_t total = (rows - 1) * stride + K;
    // a block takes one row's groups at a time, or several short rows
    const int per = groups < 256 ? 256 / groups : 1;
    const int sub = groups < 256 ? threadIdx.x / groups : 0, g0 = groups < 256 ? threadIdx.x - sub * groups : threadIdx.x;
    if (sub >= per) return;
    for (int64_t r = (int64_t)blockIdx.x * per + sub; r < rows; r += (int64_t)gridDim.x * per)
        for (int g = g0; g < groups; g += 256) {
            const int c = g * 8;
            uint4 x;
            if (c + 8 <= K) {
                x = load8(src, r * stride + c, total);
            } else {
                const uint16_t* p = reinterpret_cast<const uint16_t*>(src + r * stride + c);
                uint32_t w[4] = {0, 0, 0, 0};
                #pragma unroll
                for (int i = 0; i < 8; ++i)
                    if (c + i < K) w[i / 2] |= (uint32_t)p[i] << (16 * (i & 1));
                x = make_uint4(w[0], w[1], w[2], w[3]);
            }
            reinterpret_cast<uint4*>(dst)[r * groups + g] = x;
            if (dst2) reinterpret_cast<uint4*>(dst2)[r * groups + g] = x;
        }
}

struct DzArgs {
    Out dy, pre;                           // pre.p null: no activation
    int64_t M, dy_total, pre_total;        // elements of the tensors
    int N, act;
    __nv_bfloat16* dz;                     // [M][dzs], or null (dy itself feeds the products)
    __nv_bfloat16* lo;                     // [M][dzs], what dz's rounding leaves, or null
    int64_t dzs;
    float* part;                           // [row chunks][N] column sums, or null
    int64_t rows;                          // rows of a chunk
};

// A row's eight values as they are loaded, so that several rows' loads are in flight before the
// first is used.  VEC: the tensor's rows lie at 16-byte alignment.
template <bool VEC, bool F32> struct Raw8;
template <> struct Raw8<true, false> {
    uint4 x;
    __device__ __forceinline__ void load(const Out& o, int64_t at, int64_t) {
        x = __ldg(reinterpret_cast<const uint4*>(static_cast<const __nv_bfloat16*>(o.p) + at));
    }
    __device__ __forceinline__ void get(float* f) const { unpack8(x, f); }
};
template <> struct Raw8<false, false> {
    uint4 x;
    __device__ __forceinline__ void load(const Out& o, int64_t at, int64_t total) {
        x = load8(static_cast<const __nv_bfloat16*>(o.p), at, total);
    }
    __device__ __forceinline__ void get(float* f) const { unpack8(x, f); }
};
template <> struct Raw8<true, true> {
    float4 x, y;
    __device__ __forceinline__ void load(const Out& o, int64_t at, int64_t) {
        const float4* p = reinterpret_cast<const float4*>(static_cast<const float*>(o.p) + at);
        x = __ldg(p);
        y = __ldg(p + 1);
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = x.x; f[1] = x.y; f[2] = x.z; f[3] = x.w;
        f[4] = y.x; f[5] = y.y; f[6] = y.z; f[7] = y.w;
    }
};
template <> struct Raw8<false, true> {
    float x[8];
    __device__ __forceinline__ void load(const Out& o, int64_t at, int64_t) {
        const float* p = static_cast<const float*>(o.p) + at;
        #pragma unroll
        for (int e = 0; e < 8; ++e) x[e] = __ldg(p + e);
    }
    __device__ __forceinline__ void get(float* f) const {
        #pragma unroll
        for (int e = 0; e < 8; ++e) f[e] = x[e];
    }
};

// What a bf16 of the pair u leaves of (a, b), as bf16 itself (0 where it is not finite).
__device__ __forceinline__ uint32_t left_bf16(uint32_t u, float a, float b) {
    const float x = __uint_as_float(u << 16), y = __uint_as_float(u & 0xffff0000u);
    return pack_bf16(fabsf(x) < INFINITY ? a - x : 0.f, fabsf(y) < INFINITY ? b - y : 0.f);
}

// dz = dy act'(z) rounded to the products' 16 bits (and, for an fp32 dW, what that rounding left, in
// 16 bits again: together 2^-18 of it is lost), and its column sums (of the unrounded values): a block
// takes 256 columns of a chunk of rows, 8 rows at a time and U of those loaded
// ahead, and adds its sums in a fixed order.  HBM-bound: one read of dy (and z), one write of dz.
template <bool VEC, bool F32, int ACT, bool LO>
__global__ void __launch_bounds__(256, LO ? 3 : 4) k_dz(const DzArgs a) {
    constexpr int U = ACT ? 2 : 4;             // rows loaded ahead
    __shared__ float sm[8][256 + 8];
    const int cl = threadIdx.x & 31, rl = threadIdx.x >> 5;
    const int c = (blockIdx.x * 32 + cl) * 8;
    const int64_t r1 = min(a.M, (int64_t)(blockIdx.y + 1) * a.rows);
    float sum[8];
    #pragma unroll
    for (int e = 0; e < 8; ++e) sum[e] = 0.f;
    if (c < a.N) {
        const int64_t dyo = at(a.dy, c), preo = ACT ? at(a.pre, c) : 0;
        auto take = [&](float* g, const float* z, int64_t r) {
            if (ACT) {
                #pragma unroll
                for (int e = 0; e < 8; e += 2) times_grad<ACT>(g[e], g[e + 1], z[e], z[e + 1]);
            }
            #pragma unroll
            for (int e = 0; e < 8; ++e) sum[e] += g[e];
            if (a.dz) {    // (the padding behind N is zero)
                const uint4 u = make_uint4(pack_bf16(g[0], g[1]), pack_bf16(g[2], g[3]), pack_bf16(g[4], g[5]), pack_bf16(g[6], g[7]));
                *reinterpret_cast<uint4*>(a.dz + r * a.dzs + c) = u;
                if (LO)
                    *reinterpret_cast<uint4*>(a.lo + r * a.dzs + c) =
                        make_uint4(left_bf16(u.x, g[0], g[1]), left_bf16(u.y, g[2], g[3]), left_bf16(u.z, g[4], g[5]),
                                   left_bf16(u.w, g[6], g[7]));
            }
        };
        int64_t r = (int64_t)blockIdx.y * a.rows + rl;
        if (c + 8 <= a.N)
            for (; r + 8 * (U - 1) < r1; r += 8 * U) {
                Raw8<VEC, F32> g[U];
                Raw8<VEC, false> z[U];
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    g[i].load(a.dy, dyo + (r + 8 * i) * a.dy.rs, a.dy_total);
                    if (ACT) z[i].load(a.pre, preo + (r + 8 * i) * a.pre.rs, a.pre_total);
                }
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    float x[8], y[8];
                    g[i].get(x);
                    if (ACT) z[i].get(y);
                    take(x, y, r + 8 * i);
                }
            }
        for (; r < r1; r += 8) {
            float x[8], y[8];
            read8(a.dy, dyo, r, c, a.N, a.dy_total, x);
            if (ACT) read8(a.pre, preo, r, c, a.N, a.pre_total, y);
            take(x, y, r);
        }
    }
    if (!a.part) return;
    #pragma unroll
    for (int e = 0; e < 8; ++e) sm[rl][cl * 8 + e] = sum[e];
    __syncthreads();
    const int col = blockIdx.x * 256 + threadIdx.x;
    if (col >= a.N) return;
    float s = 0.f;
    #pragma unroll
    for (int k = 0; k < 8; ++k) s += sm[k][threadIdx.x];
    a.part[(int64_t)blockIdx.y * a.N + col] = s;
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

// The map of an operand's tiles of `rows` rows (what lies outside the matrix reads as zeros,
// 128-byte swizzle), and how the producer addresses it.  K-major: boxes of 64 inner elements by
// `rows` rows.  MN-major: 64 k by `rows` inner elements in slabs of 64.
static int make_operand(CUtensorMap* m, Operand* o, const Matrix& x, bool mn, int rows) {
    auto enc = encode_fn();
    if (!enc) return PRISM_ERR_CUDA;
    o->mn = mn;
    o->shift = x.heads == 1 ? 31 : x.inner == 64 ? 6 : 7;
    o->slabs = 0;
    const cuuint64_t row = (cuuint64_t)x.ld * 2, head = (cuuint64_t)(x.rows * x.ld) * 2;
    cuuint64_t dims[4] = {(cuuint64_t)x.inner, (cuuint64_t)x.rows, (cuuint64_t)x.heads, 1};
    cuuint64_t strides[3] = {row, head, head};
    cuuint32_t box[4] = {64, (cuuint32_t)(mn ? kKB : rows), 1, 1};
    cuuint32_t es[4] = {1, 1, 1, 1};
    if (mn && x.inner % 64 == 0) {
        // (64, rows, slabs, heads); a head of 64 channels is a slab itself
        const bool flat = x.heads == 1, one = !flat && x.inner == 64;
        o->slabs = one ? x.heads : (int)(x.inner / 64);
        dims[0] = 64;
        dims[2] = (cuuint64_t)o->slabs;
        dims[3] = (cuuint64_t)(flat || one ? 1 : x.heads);
        strides[1] = one ? head : 128;
        box[2] = (cuuint32_t)(rows / 64);
    }
    const CUresult r = enc(m, CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 4, const_cast<void*>(x.p), dims, strides, box, es,
                           CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_L2_256B,
                           CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PRISM_OK : PRISM_ERR_CUDA;
}

// C, or a residual of its shape, as boxes of 32 rows by 128 bytes.
static int make_out_map(CUtensorMap* m, const Out& y, int64_t R, int C) {
    auto enc = encode_fn();
    if (!enc) return PRISM_ERR_CUDA;
    const int e = y.f32 ? 4 : 2;
    cuuint64_t dims[3] = {(cuuint64_t)(y.hd ? y.hd : C), (cuuint64_t)R, (cuuint64_t)(y.hd ? C / y.hd : 1)};
    cuuint64_t strides[2] = {(cuuint64_t)y.rs * e, (cuuint64_t)(y.hd ? y.hs : R * y.rs) * e};
    cuuint32_t boxd[3] = {(cuuint32_t)(128 / e), 32, 1};
    cuuint32_t es[3] = {1, 1, 1};
    CUresult r = enc(m, y.f32 ? CU_TENSOR_MAP_DATA_TYPE_FLOAT32 : CU_TENSOR_MAP_DATA_TYPE_BFLOAT16, 3, y.p, dims, strides,
                     boxd, es, CU_TENSOR_MAP_INTERLEAVE_NONE, CU_TENSOR_MAP_SWIZZLE_128B, CU_TENSOR_MAP_L2_PROMOTION_NONE,
                     CU_TENSOR_MAP_FLOAT_OOB_FILL_NONE);
    return r == CUDA_SUCCESS ? PRISM_OK : PRISM_ERR_CUDA;
}

static int64_t ceil_div(int64_t a, int64_t b) { return (a + b - 1) / b; }

struct Shape {
    int few;                               // k_few, else k_tile
    int cg, bn, split;
};

// The tile of a product of R rows, C columns and kb stages.
//   up to 64 rows: k_few, its contraction split until two CTAs run on every SM.
//   else the least of the estimates, in cycles of one SM:
//     pairs on 256 x bn tiles: their waves over 74 pairs, each kb stages of 522, 430 or 310 cycles
//       (measured; the instructions' own 512, 384 and 256: narrower tiles load more bytes per
//       product) and 2,500 to fill and drain; 8,000 to start;
//     single CTAs on 128 x 128 tiles, `split` to a tile: all at once, kb / split stages of 460 cycles
//       (32 KB each to one SM), 10,000 to start and 4,000 to join the parts.
//   A tile width that fits the waves counts most: 512 rows of 5,120 by 5,120 are 80 tiles at bn = 128
//   (two waves, 31.8 us), 40 at 256 (half of the pairs idle, 30.6 us), 54 at 192.
static Shape shape_of(int64_t R, int64_t C, int kb, bool x_mn, bool y_mn) {
    if (R <= 64) {
        Shape s{1, 1, 64, 1};
        if (!x_mn) s.bn = R <= 16 ? 16 : R <= 32 ? 32 : 64;      // an MN-major slab has 64 rows
        const int64_t tiles = ceil_div(C, 128);
        while (s.split < 8 && tiles * s.split * 2 <= 2 * 148 && kb >= 8 * s.split) s.split *= 2;
        return s;
    }
    Shape best{0, 2, 256, 1};
    int64_t least = INT64_MAX;
    for (int bn : {256, 192, 128}) {
        if (bn == 192 && y_mn) continue;                         // a CTA's half is no whole slabs
        const int64_t waves = ceil_div(ceil_div(R, 256) * ceil_div(C, bn), 74);
        const int64_t t = 8000 + waves * ((int64_t)kb * (bn == 256 ? 522 : bn == 192 ? 430 : 310) + 2500);
        if (t < least) { least = t; best = Shape{0, 2, bn, 1}; }
    }
    const int64_t tiles = ceil_div(R, 128) * ceil_div(C, 128);
    for (int split : {1, 2, 4, 8}) {
        if (tiles * split > 148 || (split > 1 && kb < 4 * split)) break;
        const int64_t t = 10000 + ceil_div(kb, split) * 460 + (split > 1 ? 4000 : 0);
        if (t < least) { least = t; best = Shape{0, 1, 128, split}; }
    }
    return best;
}

// Starts `kernel` as clusters of `group` CTAs.  The shared-memory opt-in is made for every call:
// it belongs to the device that is current.
template <typename... P, typename... A>
static int start_kernel(void (*kernel)(P...), int64_t ctas, int group, int threads, int smem, cudaStream_t s, const A&... args) {
    if (cudaFuncSetAttribute(kernel, cudaFuncAttributeMaxDynamicSharedMemorySize, smem) != cudaSuccess) return PRISM_ERR_CUDA;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas);
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = s;
    cudaLaunchAttribute at[1];
    at[0].id = cudaLaunchAttributeClusterDimension;
    at[0].val.clusterDim.x = (unsigned)group;
    at[0].val.clusterDim.y = 1;
    at[0].val.clusterDim.z = 1;
    cfg.attrs = at;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, args...) == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA;
}

template <int CG, int BN>
static int launch_tile(const CUtensorMap& ta, const CUtensorMap& tb, const CUtensorMap& ty, const CUtensorMap& tr,
                       const Args& a, cudaStream_t s) {
    const int64_t tiles = (int64_t)a.tiles_c * a.tiles_r;
    void (*kernel)(CUtensorMap, CUtensorMap, CUtensorMap, CUtensorMap, Args);
    if constexpr (CG == 2) {
        if (!a.fast) kernel = k_tile<CG, BN, kRows>;
        else if (a.kblocks <= a.chunk) kernel = k_tile<CG, BN, kSingle>;
        else if (a.act == PRISM_ACT_NONE && !a.pre.p) kernel = k_tile<CG, BN, kDirect>;
        else kernel = k_tile<CG, BN, kSums>;
    } else {
        kernel = k_tile<CG, BN, kAll>;
    }
    return start_kernel(kernel, CG == 2 ? 2 * (tiles < 74 ? tiles : 74) : tiles * a.split, CG == 2 ? 2 : a.split,
                        Cfg<CG, BN>::kThreads, tile_smem<CG, BN>(), s, ta, tb, ty, tr, a);
}
template <int BN>
static int launch_few(const CUtensorMap& ta, const CUtensorMap& tb, const Args& a, cudaStream_t s) {
    return start_kernel(k_few<BN>, (int64_t)a.tiles_c * a.tiles_r * a.split, a.split, Cfg<1, BN>::kThreads,
                        Cfg<1, BN>::kRing + 1024, s, ta, tb, a);
}

// C[r][c] = sum_k X[r][k] Y[c][k]; K the contraction's length, x_mn / y_mn: the matrix's rows are k.
static int product(const Matrix& X, bool x_mn, const Matrix& Y, bool y_mn, int64_t R, int C, int64_t K, Args& a,
                   cudaStream_t s) {
    a.R = R;
    a.C = C;
    a.kblocks = (int)ceil_div(K, kKB);
    const Shape sh = shape_of(R, C, a.kblocks, x_mn, y_mn);
    a.split = sh.split;
    a.chunk = a.y.f32 ? kChunkF32 : kChunkBF16;
    a.band = 8;
    const int rows = sh.few ? sh.bn : 128 * sh.cg, cols = sh.few ? 128 : sh.bn;
    const int64_t tr = ceil_div(R, rows), tc = ceil_div(C, cols);
    if (tr * tc > 0x0fffffff) return PRISM_ERR_INVALID_ARG;
    a.tiles_r = (int)tr;
    a.tiles_c = (int)tc;
    CUtensorMap tx, ty;
    Operand ox, oy;
    int st = make_operand(&tx, &ox, X, x_mn, sh.few ? sh.bn : 128);
    if (!st) st = make_operand(&ty, &oy, Y, y_mn, sh.few ? 128 : sh.bn / sh.cg);
    if (st) return st;
    a.a = sh.few ? oy : ox;                // along the tensor core's M
    a.b = sh.few ? ox : oy;
    if (sh.few)
        return sh.bn == 16 ? launch_few<16>(ty, tx, a, s) : sh.bn == 32 ? launch_few<32>(ty, tx, a, s) : launch_few<64>(ty, tx, a, s);
    // a map of C wants its address and row stride in whole 16 bytes
    CUtensorMap to{}, tr2{};
    a.fast = a.y.vec && (!a.res.p || a.res.vec) && (!a.pre.p || a.pre.vec);
    if (a.fast) st = make_out_map(&to, a.y, R, C);
    if (!st && a.fast && a.res.p) st = make_out_map(&tr2, a.res, R, C);
    if (st) return st;
    if (sh.cg == 1) return launch_tile<1, 128>(tx, ty, to, tr2, a, s);
    return sh.bn == 256   ? launch_tile<2, 256>(tx, ty, to, tr2, a, s)
           : sh.bn == 192 ? launch_tile<2, 192>(tx, ty, to, tr2, a, s)
                          : launch_tile<2, 128>(tx, ty, to, tr2, a, s);
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
    // a tensor map's stride is below 2^40 bytes: a tensor's rows (M, of W and dW N) times its stride,
    // dx and dW (no wider than x and W) among them
    const int64_t most = 1LL << 38;
    if (p->x_stride < p->K || p->w_stride < p->K || p->y_stride < p->N || p->r_stride < p->N) return true;
    for (int64_t t : {p->x_stride, p->y_stride, p->r_stride})
        if (t > most / (p->M + 1)) return true;
    if (p->w_stride > most / ((int64_t)p->N + 1)) return true;
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
// whether dW is the sum of two products: an fp32 dW from a dz that has more than 16 bits.  One bf16 part
// alone leaves 1.7e-3 of it, two leave 2.6e-6 (the sums' own truncation 7e-7); dx and a bf16 dW hold no
// more than 16 bits themselves and take one.
static bool two_parts(const prism_linear_params* p) {
    return p->dw_dtype == PRISM_F32 && (p->activation != PRISM_ACT_NONE || p->out_dtype == PRISM_F32);
}
// The parts lie one behind the other.  With fewer rows than features they are one contraction of 2 M
// rows against x twice (x copied: dW, the largest tensor then, is written once; one token, 30,720 x 5,120
// through SiLU with dx 212 us, as two products 419; 2,477 x 5,120 x 20,480 1,186 and 1,260), else two
// products, the second added onto the first.
static bool stacked(const prism_linear_params* p) { return two_parts(p) && !p->in_heads && p->M < p->N; }
static size_t parts_bytes(const prism_linear_params* p) {
    return forms_dz(p) ? up256((size_t)p->M * pad8(p->N) * (two_parts(p) ? 4 : 2)) : 0;
}
static size_t x_twice_bytes(const prism_linear_params* p) {
    return stacked(p) ? up256((size_t)p->M * pad8(p->K) * 4) : x_bytes(p);
}

struct DzGrid {
    int x, y;
    int64_t rows;
};
// Row chunks: two full rounds of four blocks per SM at most; a chunk has at least 64 rows.
static DzGrid dz_grid(const prism_linear_params* p) {
    DzGrid g;
    g.x = (int)ceil_div(p->N, 256);
    int64_t y = 8 * 148 / g.x;
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
    o.vec = o.rs * (f32 ? 4 : 2) % 16 == 0;
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

// A matrix of rows as the products read it: itself, or packed at `ws` (`twice`: and once more behind it).
static int operand(Matrix* m, const void* p, int64_t rows, int cols, int heads, int64_t stride, bool pack, char*& ws,
                   cudaStream_t s, bool twice = false) {
    if (!pack && !twice) {
        *m = matrix(p, rows, cols, heads, stride);
        return PRISM_OK;
    }
    const int64_t ld = pad8(cols);
    auto* dst = reinterpret_cast<__nv_bfloat16*>(ws);
    ws += up256((size_t)rows * ld * (twice ? 4 : 2));
    const int groups = (int)(ld / 8), per = groups < 256 ? 256 / groups : 1;
    const int64_t blocks = ceil_div(rows, per);
    k_pack<<<(unsigned)(blocks < 148 * 32 ? blocks : 148 * 32), 256, 0, s>>>(static_cast<const __nv_bfloat16*>(p), stride, rows,
                                                                            cols, dst, twice ? dst + rows * ld : nullptr, groups);
    *m = Matrix{dst, twice ? 2 * rows : rows, cols, ld, 1};
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
    return product(mx, false, mw, false, p->M, p->N, p->K, a, s);
}

template <bool VEC, bool F32, int ACT>
static void launch_dz_act(const DzArgs& d, dim3 grid, cudaStream_t s) {
    if constexpr (F32 || ACT != PRISM_ACT_NONE) {
        if (d.lo) {
            k_dz<VEC, F32, ACT, true><<<grid, 256, 0, s>>>(d);
            return;
        }
    }
    k_dz<VEC, F32, ACT, false><<<grid, 256, 0, s>>>(d);
}
template <bool VEC, bool F32>
static void launch_dz_of(const DzArgs& d, dim3 grid, cudaStream_t s) {
    switch (d.pre.p ? d.act : PRISM_ACT_NONE) {
        case PRISM_ACT_GELU: launch_dz_act<VEC, F32, PRISM_ACT_GELU>(d, grid, s); break;
        case PRISM_ACT_GELU_TANH: launch_dz_act<VEC, F32, PRISM_ACT_GELU_TANH>(d, grid, s); break;
        case PRISM_ACT_SILU: launch_dz_act<VEC, F32, PRISM_ACT_SILU>(d, grid, s); break;
        default: launch_dz_act<VEC, F32, PRISM_ACT_NONE>(d, grid, s); break;
    }
}
static void launch_dz(const DzArgs& d, dim3 grid, cudaStream_t s) {
    const bool vec = d.dy.vec && d.N % 8 == 0;
    if (vec) d.dy.f32 ? launch_dz_of<true, true>(d, grid, s) : launch_dz_of<true, false>(d, grid, s);
    else d.dy.f32 ? launch_dz_of<false, true>(d, grid, s) : launch_dz_of<false, false>(d, grid, s);
}

static int backward(const prism_linear_params* p, const void* dy, const void* x, const void* W, const void* pre, void* dx,
                    void* dW, float* db, char* ws, int* err, cudaStream_t s) {
    Matrix mx{}, mw{}, mlo{}, mz = matrix(dy, p->M, p->N, p->out_heads, p->y_stride);
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
        if (dW && two_parts(p)) {
            d.lo = d.dz + p->M * d.dzs;
            mlo = Matrix{d.lo, p->M, p->N, d.dzs, 1};
        }
        ws += parts_bytes(p);
        const DzGrid g = dz_grid(p);
        d.rows = g.rows;
        if (db) d.part = reinterpret_cast<float*>(ws);
        ws += up256((size_t)g.y * p->N * 4);
        d.dy_total = p->out_heads ? p->M * p->N : (p->M - 1) * p->y_stride + p->N;
        d.pre_total = p->M * p->N;
        launch_dz(d, dim3(g.x, g.y), s);
        if (db) k_db<<<(unsigned)ceil_div(p->N, 32), 256, 0, s>>>(d.part, g.y, p->N, db);
        if (cudaGetLastError() != cudaSuccess) return PRISM_ERR_CUDA;
    }
    if (dx) {
        st = operand(&mw, W, p->N, p->K, 0, p->w_stride, pack_w(p), ws, s);
        if (st) return st;
        Args a{};
        a.y = out_rows(dx, p->M, p->K, p->in_heads, p->K, 0);
        a.err = err;
        st = product(mz, false, mw, true, p->M, p->K, p->N, a, s);
        if (st) return st;
    }
    if (dW) {
        const bool twice = stacked(p);
        st = operand(&mx, x, p->M, p->K, p->in_heads, p->x_stride, pack_x(p), ws, s, twice);
        if (st) return st;
        Args a{};
        a.y = out_rows(dW, p->N, p->K, 0, p->K, p->dw_dtype == PRISM_F32);
        a.err = err;
        if (twice) {
            mz.rows = 2 * p->M;
        } else if (mlo.p) {  // the small part first, the other added onto it
            st = product(mlo, true, mx, true, p->N, p->K, p->M, a, s);
            if (st) return st;
            a.res = a.y;
        }
        st = product(mz, true, mx, true, p->N, p->K, mz.rows, a, s);
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
    const Span sw = span(need ? workspace : nullptr, 1, (int64_t)need, 0, (int64_t)need, 1);
    const Span ss = span(dev_status, 1, 4, 0, 4, 4);
    for (const Span& i : {in[0], in[1], in[2], sr, sy, sp, ss})
        if (!apart(sw, i)) return PRISM_ERR_INVALID_ARG;
    if (!apart(ss, sy) || !apart(ss, sp)) return PRISM_ERR_INVALID_ARG;
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
    return x_twice_bytes(p) + w_bytes(p) + parts_bytes(p) + up256((size_t)dz_grid(p).y * p->N * 4) + 256;
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
    const Span sw = span(workspace, 1, (int64_t)need, 0, (int64_t)need, 1), ss = span(dev_status, 1, 4, 0, 4, 4);
    for (const Span& i : {in[0], in[1], in[2], in[3], out[0], out[1], out[2], ss})
        if (!apart(sw, i)) return PRISM_ERR_INVALID_ARG;
    for (const Span& o : out)
        if (!apart(ss, o)) return PRISM_ERR_INVALID_ARG;
    if (int st = device_ok()) return st;
    nvtxRangePushA("prism linear bwd");
    const int st = backward(p, dy, x, W, pre, dx, dW, db, static_cast<char*>(workspace), dev_status, s);
    nvtxRangePop();
    return st;
}
