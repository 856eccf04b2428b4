// prism_norm_rope.cu -- RMS norm of every head's query and key rows with the
// rotation by grid position in the same pass, and its gradients.
//
// Row x (one token of one head, D channels), weight w, pair (a, b) of channels
// turned by the angle of the token's position on the pair's axis (cos c, sin s):
//     r = 1 / sqrt(mean_d x_d^2 + eps),  u = x r w,
//     y_a = u_a c - u_b s,  y_b = u_a s + u_b c.
// Gradients, with g = dy and v = R^T g (v_a = g_a c + g_b s, v_b = g_b c - g_a s):
//     dw = sum over rows of v x r,   dx = r (w v - x r mean_d(w v x r)).
//
// Bound: HBM.  The forward moves each element twice (one read, one write), the
// backward three times; the arithmetic is a few operations per element.  Nothing
// but the inputs is kept for the backward: x has to be read again anyway, and r
// follows from it.
//
// Layout: a row is D / 8 lanes of 8 channels (16-byte accesses for bf16), a warp
// holds 32 / (D / 8) consecutive tokens of one head, and a block walks heads with
// its tokens fixed, so a lane's cos and sin are read once for all the heads of its
// token (they are gathered from three small per-axis tables: [T], [H], [W] rows
// instead of one table of T H W rows).  Consecutive tokens of one head make the
// head-major side of the pass contiguous; on a token-major side each row is still
// whole 128-byte lines, and the following heads of the loop continue them.
#include <cuda_bf16.h>
#include <cuda_runtime.h>

#include "prism_dev.cuh"
#include "prism_internal.h"

namespace prism {
namespace nr {

constexpr int kThreads = 256;

struct Rows {
    void* p;
    int64_t hs, ts;          // head and token strides in elements
};

struct Rope {
    const float2* tab;       // (cos, sin): [T][dt/2], [H][dh/2], [W][dw/2]; null = no rotation
    int T, H, W;
    int dt, dh, dw;
};

struct Args {
    Rows in[2], out[2], grad[2];   // forward: in -> out; backward: in = x, grad = dy, out = dx
    const void* w[2];
    int w_f32;
    Rope rope;
    int64_t N;
    int heads, hpc, tensors;       // heads, heads per block, 2 with a key
    float eps;
    float* part;                   // backward: [2][blocks of a tensor][D] partial weight gradients, or null
};

// ---------------------------------------------------------- 8-channel accesses
template <typename T> struct Vec8;
template <> struct Vec8<__nv_bfloat16> {
    uint4 r;
    __device__ __forceinline__ void load(const __nv_bfloat16* p) { r = __ldcs(reinterpret_cast<const uint4*>(p)); }
    __device__ __forceinline__ void get(float* f) const {
        const uint32_t u[4] = {r.x, r.y, r.z, r.w};
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            f[2 * i] = __uint_as_float(u[i] << 16);
            f[2 * i + 1] = __uint_as_float(u[i] & 0xffff0000u);
        }
    }
    // the values that lane `from` holds
    __device__ __forceinline__ Vec8 of(int from) const {
        Vec8 o;
        o.r.x = __shfl_sync(0xffffffffu, r.x, from);
        o.r.y = __shfl_sync(0xffffffffu, r.y, from);
        o.r.z = __shfl_sync(0xffffffffu, r.z, from);
        o.r.w = __shfl_sync(0xffffffffu, r.w, from);
        return o;
    }
    static __device__ __forceinline__ void store(__nv_bfloat16* p, const float* f) {
        __stcs(reinterpret_cast<uint4*>(p), make_uint4(pack_bf16(f[0], f[1]), pack_bf16(f[2], f[3]),
                                                       pack_bf16(f[4], f[5]), pack_bf16(f[6], f[7])));
    }
};
template <> struct Vec8<float> {
    float4 a, b;
    __device__ __forceinline__ void load(const float* p) {
        a = __ldcs(reinterpret_cast<const float4*>(p));
        b = __ldcs(reinterpret_cast<const float4*>(p) + 1);
    }
    __device__ __forceinline__ void get(float* f) const {
        f[0] = a.x; f[1] = a.y; f[2] = a.z; f[3] = a.w;
        f[4] = b.x; f[5] = b.y; f[6] = b.z; f[7] = b.w;
    }
    __device__ __forceinline__ Vec8 of(int from) const {
        Vec8 o;
        o.a.x = __shfl_sync(0xffffffffu, a.x, from);
        o.a.y = __shfl_sync(0xffffffffu, a.y, from);
        o.a.z = __shfl_sync(0xffffffffu, a.z, from);
        o.a.w = __shfl_sync(0xffffffffu, a.w, from);
        o.b.x = __shfl_sync(0xffffffffu, b.x, from);
        o.b.y = __shfl_sync(0xffffffffu, b.y, from);
        o.b.z = __shfl_sync(0xffffffffu, b.z, from);
        o.b.w = __shfl_sync(0xffffffffu, b.w, from);
        return o;
    }
    static __device__ __forceinline__ void store(float* p, const float* f) {
        __stcs(reinterpret_cast<float4*>(p), make_float4(f[0], f[1], f[2], f[3]));
        __stcs(reinterpret_cast<float4*>(p) + 1, make_float4(f[4], f[5], f[6], f[7]));
    }
};

// Sums of U rows' values over the LANES lanes that hold a row: s[i] is this lane's part of row
// i.  Each exchange halves the rows a lane still carries, so U rows cost U - 1 + log2(LANES / U)
// shuffles instead of U log2(LANES); what follows from a row's sum is computed by the lanes that
// own the row (lane & (U - 1) is its number) and handed to all by from_owner().
template <int LANES, int U>
__device__ __forceinline__ float owned_sum(const float* s, int lane) {
    static_assert(U == 1 || U == 2 || U == 4, "rows of a group");
    float k;
    int o = 1;
    if (U == 4) {
        const bool hi = lane & 1, hi2 = lane & 2;
        float k0 = hi ? s[1 % U] : s[0], k1 = hi ? s[3 % U] : s[2 % U];
        k0 += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[1 % U], 1);
        k1 += __shfl_xor_sync(0xffffffffu, hi ? s[2 % U] : s[3 % U], 1);
        k = hi2 ? k1 : k0;
        k += __shfl_xor_sync(0xffffffffu, hi2 ? k0 : k1, 2);
        o = 4;
    } else if (U == 2) {
        const bool hi = lane & 1;
        k = hi ? s[1 % U] : s[0];
        k += __shfl_xor_sync(0xffffffffu, hi ? s[0] : s[1 % U], 1);
        o = 2;
    } else {
        k = s[0];
    }
    #pragma unroll
    for (int i = 0; i < 4; ++i, o <<= 1)
        if (o < LANES) k += __shfl_xor_sync(0xffffffffu, k, o);
    return k;
}
template <int U>
__device__ __forceinline__ float from_owner(float v, int lane, int i) {
    return __shfl_sync(0xffffffffu, v, (lane & ~(U - 1)) | i);
}

__device__ __forceinline__ float weight_at(const void* w, int f32, int ch) {
    return !w ? 1.f : f32 ? static_cast<const float*>(w)[ch] : __bfloat162float(static_cast<const __nv_bfloat16*>(w)[ch]);
}
// A lane's eight weights from their copy in shared memory (read again for every group of
// rows: two loads instead of eight registers held over the loop).
__device__ __forceinline__ void read_w(const float4* sw, int ch, float* w) {
    const float4 a = sw[ch / 4], b = sw[ch / 4 + 1];
    w[0] = a.x; w[1] = a.y; w[2] = a.z; w[3] = a.w;
    w[4] = b.x; w[5] = b.y; w[6] = b.z; w[7] = b.w;
}

// A lane's part of the rotation at one token, by how the pairs lie.
//   kAdjacent  (2p, 2p + 1), in one lane: four (cos, sin).
//   kHalves    channel p of an axis of d channels pairs with p + d / 2, in general in another lane at
//              no alignment (d / 2 may be odd): the row passes through shared memory and the lane
//              keeps its eight channels' cos, sin (the sign of the channel's own side folded in)
//              and the places of their partners.
//   kLanes     halves of axes whose d / 2 is a multiple of 8: the partners of a lane's channels are
//              the channels of one other lane, brought by shuffles of the loaded words (40 heads of
//              92,160 tokens, bf16: forward 5.7 TB/s and backward 5.3, through shared memory 5.2 and 4.6).
// Channels behind the last axis are not rotated: cos 1, sin 0.
constexpr int kAdjacent = 0, kHalves = 1, kLanes = 2;
template <int PAIRS> struct Turn;

__device__ __forceinline__ float2 rope_at(const Rope& r, int pair, int t, int h, int w) {
    const int pt = r.dt >> 1, ph = r.dh >> 1, pw = r.dw >> 1;
    if (pair < pt) return __ldg(r.tab + (int64_t)t * pt + pair);
    pair -= pt;
    if (pair < ph) return __ldg(r.tab + (int64_t)r.T * pt + (int64_t)h * ph + pair);
    pair -= ph;
    if (pair < pw) return __ldg(r.tab + (int64_t)r.T * pt + (int64_t)r.H * ph + (int64_t)w * pw + pair);
    return make_float2(1.f, 0.f);
}

template <> struct Turn<kAdjacent> {
    float2 cs[4];
    __device__ __forceinline__ void init(const Rope& r, int ch, int t, int h, int w) {
        #pragma unroll
        for (int i = 0; i < 4; ++i) cs[i] = rope_at(r, (ch >> 1) + i, t, h, w);
    }
    // u -> R u (DIR = 1) or R^T u (DIR = -1)
    template <int DIR>
    __device__ __forceinline__ void take(float* u, const float*) const {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = u[2 * i], b = u[2 * i + 1], c = cs[i].x, s = DIR * cs[i].y;
            u[2 * i] = a * c - b * s;
            u[2 * i + 1] = a * s + b * c;
        }
    }
};

template <> struct Turn<kHalves> {
    float c[8], s[8];
    int at[8];               // the partners' places in the row's shared-memory copy
    // one pad word per 8 channels: the lanes of a row write and read at an odd stride
    static __device__ __forceinline__ int place(int ch) { return ch + (ch >> 3); }
    __device__ __forceinline__ void init(const Rope& r, int ch, int t, int h, int w) {
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const int e = ch + i;
            int base = 0, d = r.dt;
            if (e >= r.dt) { base = r.dt; d = r.dh; }
            if (e >= r.dt + r.dh) { base = r.dt + r.dh; d = r.dw; }
            const int l = e - base, half = d >> 1;
            if (l >= d) {
                c[i] = 1.f; s[i] = 0.f; at[i] = place(e);
            } else {
                const bool lo = l < half;
                const float2 v = rope_at(r, (base >> 1) + (lo ? l : l - half), t, h, w);
                c[i] = v.x;
                s[i] = lo ? -v.y : v.y;
                at[i] = place(lo ? e + half : e - half);
            }
        }
    }
    static __device__ __forceinline__ void put(const float* u, float* row, int ch) {
        #pragma unroll
        for (int i = 0; i < 8; ++i) row[place(ch) + i] = u[i];
    }
    template <int DIR>
    __device__ __forceinline__ void take(float* u, const float* row) const {
        #pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float p0, p1;
            fmul2(p0, p1, row[at[i]], row[at[i + 1]], DIR * s[i], DIR * s[i + 1]);
            ffma2(u[i], u[i + 1], u[i], u[i + 1], c[i], c[i + 1], p0, p1);
        }
    }
};

template <> struct Turn<kLanes> {
    float c[8], s[8];
    int partner;             // the partners' first channel
    __device__ __forceinline__ void init(const Rope& r, int ch, int t, int h, int w) {
        int base = 0, d = r.dt;
        if (ch >= r.dt) { base = r.dt; d = r.dh; }
        if (ch >= r.dt + r.dh) { base = r.dt + r.dh; d = r.dw; }
        const int l = ch - base, half = d >> 1;
        const bool turns = l < d, lo = l < half;
        partner = !turns ? ch : lo ? ch + half : ch - half;
        #pragma unroll
        for (int i = 0; i < 8; ++i) {
            const float2 v = turns ? rope_at(r, (base >> 1) + (lo ? l : l - half) + i, t, h, w) : make_float2(1.f, 0.f);
            c[i] = v.x;
            s[i] = lo ? -v.y : v.y;
        }
    }
    __device__ __forceinline__ int from(int lane, int lanes) const { return (lane & ~(lanes - 1)) | (partner >> 3); }
    template <int DIR>
    __device__ __forceinline__ void take(float* u, const float* p) const {
        #pragma unroll
        for (int i = 0; i < 8; i += 2) {
            float p0, p1;
            fmul2(p0, p1, p[i], p[i + 1], DIR * s[i], DIR * s[i + 1]);
            ffma2(u[i], u[i + 1], u[i], u[i + 1], c[i], c[i + 1], p0, p1);
        }
    }
};

// The rotation with a tensor's weights in it, x -> R (w x) (`w` laid out by place()).
__device__ __forceinline__ int place(int ch) { return Turn<kHalves>::place(ch); }
template <int PAIRS> struct Fold;
template <> struct Fold<kAdjacent> {
    float a0[4], b0[4], a1[4], b1[4];        // y_a = x_a a0 + x_b b0, y_b = x_a a1 + x_b b1
    __device__ __forceinline__ void init(const Rope& r, const float* w, int ch, int t, int h, int g) {
        const float* own = w + Turn<kHalves>::place(ch);
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float2 cs = r.tab ? rope_at(r, (ch >> 1) + i, t, h, g) : make_float2(1.f, 0.f);
            a0[i] = own[2 * i] * cs.x; b0[i] = -own[2 * i + 1] * cs.y;
            a1[i] = own[2 * i] * cs.y; b1[i] = own[2 * i + 1] * cs.x;
        }
    }
    __device__ __forceinline__ void apply(float* x, const float*) const {
        #pragma unroll
        for (int i = 0; i < 4; ++i) {
            const float a = x[2 * i], b = x[2 * i + 1];
            float p0, p1;
            fmul2(p0, p1, b, a, b0[i], a1[i]);
            ffma2(x[2 * i], x[2 * i + 1], a, b, a0[i], b1[i], p0, p1);
        }
    }
};
template <> struct Fold<kHalves> {
    Turn<kHalves> turn;
    __device__ __forceinline__ void init(const Rope& r, const float* w, int ch, int t, int h, int g) {
        turn.init(r, ch, t, h, g);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            turn.c[e] *= w[Turn<kHalves>::place(ch) + e];
            turn.s[e] *= w[turn.at[e]];
        }
    }
    __device__ __forceinline__ void apply(float* x, const float* row) const { turn.take<1>(x, row); }
};
template <> struct Fold<kLanes> {
    Turn<kLanes> turn;
    __device__ __forceinline__ void init(const Rope& r, const float* w, int ch, int t, int h, int g) {
        turn.init(r, ch, t, h, g);
        #pragma unroll
        for (int e = 0; e < 8; ++e) {
            turn.c[e] *= w[place(ch) + e];
            turn.s[e] *= w[place(turn.partner) + e];
        }
    }
    __device__ __forceinline__ void apply(float* x, const float* p) const { turn.take<1>(x, p); }
};

// Rows of a group, and shared memory for their exchange (kHalves only).
template <typename T, int D, int PAIRS, int U>
struct Group {
    static constexpr int kRows = kThreads / (D / 8);      // rows of one head in a block
    static constexpr int kPitch = D + D / 8;
    static constexpr int kFloats = PAIRS == kHalves ? U * kRows * kPitch : 1;
};

__device__ __forceinline__ void grid_at(const Rope& r, int64_t n, int& t, int& h, int& w) {
    const uint32_t hw = (uint32_t)r.H * (uint32_t)r.W, m = (uint32_t)n;     // N < 2^31
    t = (int)(m / hw);
    const uint32_t q = m - (uint32_t)t * hw;
    h = (int)(q / (uint32_t)r.W);
    w = (int)(q - (uint32_t)h * (uint32_t)r.W);
}

// Sum of squares of a lane's eight channels, and eight products by one factor (two at a time).
__device__ __forceinline__ float squares(const float* x) {
    float a0, a1;
    fmul2(a0, a1, x[0], x[1], x[0], x[1]);
    #pragma unroll
    for (int e = 2; e < 8; e += 2) ffma2(a0, a1, x[e], x[e + 1], x[e], x[e + 1], a0, a1);
    return a0 + a1;
}
__device__ __forceinline__ void scale8(float* x, float r) {
    #pragma unroll
    for (int e = 0; e < 8; e += 2) fmul2(x[e], x[e + 1], x[e], x[e + 1], r, r);
}

// The forward.  Grid: x = token tiles (strided), y = head groups.  A block takes its tokens'
// rows of both tensors, U heads at a time: U loads in flight per lane.
// The weights are folded into the rotation, y_a = r (x_a w_a c - x_b w_b s): the factors are made
// once per token and tensor, and with halves the rows pass through shared memory as they were
// read, so a group's exchange does not wait for its norms.  At 40 heads of 92,160 tokens adjacent
// pairs move 6.2 TB/s (64 registers for 4 blocks per SM; 3 blocks 6.2, 6 blocks with U = 2 5.5) and
// halves 5.2: there shared memory is 82% busy, eight words written and eight read per lane and row
// (unfolded, every row summed by itself: 4.3).  At 5 heads, 1,013,760 tokens, 5.0: a token's factors
// and addresses serve ten rows only, and five heads are a group of four and one of a single row, for
// each tensor, so 2.5 loads of 4 are in flight on average.
template <typename TI, typename TO, int D, int PAIRS>
__global__ void __launch_bounds__(kThreads, PAIRS == kAdjacent ? 4 : 3) k_norm_rope(const Args a) {
    constexpr int U = sizeof(TI) == 2 ? 4 : 2;
    constexpr bool HALVES = PAIRS == kHalves;
    using G = Group<TI, D, PAIRS, U>;
    constexpr int LANES = D / 8, RPB = G::kRows;
    __shared__ float sx[G::kFloats];
    __shared__ float sw[2][D + D / 8];
    const int lane = threadIdx.x & 31, ch = (threadIdx.x % LANES) * 8, sub = threadIdx.x / LANES;
    float* row = HALVES ? sx + sub * G::kPitch : sx;
    const int h0 = blockIdx.y * a.hpc, h1 = min(h0 + a.hpc, a.heads);
    for (int i = threadIdx.x; i < a.tensors * D; i += kThreads)
        sw[i / D][Turn<kHalves>::place(i % D)] = weight_at(a.w[i / D], a.w_f32, i % D);
    __syncthreads();
    for (int64_t n0 = (int64_t)blockIdx.x * RPB; n0 < a.N; n0 += (int64_t)gridDim.x * RPB) {
        const int64_t n = n0 + sub;
        const bool ok = n < a.N;
        int gt = 0, gh = 0, gw = 0;
        if (a.rope.tab) grid_at(a.rope, ok ? n : 0, gt, gh, gw);
        for (int z = 0; z < a.tensors; ++z) {
            Fold<PAIRS> fold;
            fold.init(a.rope, sw[z], ch, gt, gh, gw);
            const TI* src = static_cast<const TI*>(a.in[z].p) + n * a.in[z].ts + h0 * a.in[z].hs + ch;
            TO* dst = static_cast<TO*>(a.out[z].p) + n * a.out[z].ts + h0 * a.out[z].hs + ch;
            for (int h = h0; h < h1; h += U, src += U * a.in[z].hs, dst += U * a.out[z].hs) {
                Vec8<TI> v[U];
                float r[U];
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    v[i] = Vec8<TI>{};
                    if (ok && h + i < h1) v[i].load(src + i * a.in[z].hs);
                }
                if (HALVES) __syncwarp();            // the previous group's reads are done
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    float x[8];
                    v[i].get(x);
                    if (HALVES) Turn<kHalves>::put(x, row + i * RPB * G::kPitch, ch);
                    r[i] = squares(x);
                }
                if (HALVES) __syncwarp();
                const float own = rsqrtf(owned_sum<LANES, U>(r, lane) * (1.f / D) + a.eps);
                #pragma unroll
                for (int i = 0; i < U; ++i) r[i] = from_owner<U>(own, lane, i);
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    if (h + i >= h1) break;          // the same for the whole block
                    float x[8];
                    v[i].get(x);
                    if constexpr (PAIRS == kLanes) {
                        float p[8];
                        v[i].of(fold.turn.from(lane, LANES)).get(p);
                        fold.apply(x, p);
                    } else {
                        fold.apply(x, row + i * RPB * G::kPitch);
                    }
                    scale8(x, r[i]);
                    if (ok) Vec8<TO>::store(dst + i * a.out[z].hs, x);
                }
            }
        }
    }
}

// The gradients.  TI: type of x and dx; TG: type of dy.  Grid: z = query or key (a block
// then holds one weight's sums).  A block sums its rows' part of dw in registers (in the
// order of its loop), then over its rows through shared memory, and writes one row of
// partial sums: no atomics, the same bits every time.
template <typename TI, typename TG, int D, int PAIRS>
__global__ void __launch_bounds__(kThreads, 2) k_norm_rope_bwd(const Args a) {
    // rows at a time: four, but two where four rows' fp32 gradients and their exchange do not fit the
    // registers (40 heads of 92,160 tokens, halves: fp32 4.7 TB/s with two and 4.0 with four, bf16 4.0
    // and 4.6; adjacent 5.6 and 6.4, 3.6 and 5.5)
    constexpr int U = PAIRS == kHalves && sizeof(TG) == 4 ? 2 : 4;
    constexpr bool HALVES = PAIRS == kHalves, KEEP = PAIRS != kAdjacent;
    using G = Group<TG, D, PAIRS, U>;
    constexpr int LANES = D / 8, RPB = G::kRows;
    constexpr int kSum = RPB * D;
    __shared__ float sx[kSum > G::kFloats ? kSum : G::kFloats];
    __shared__ float4 sw[1][D / 4];
    const int lane = threadIdx.x & 31, z = blockIdx.z, ch = (threadIdx.x % LANES) * 8, sub = threadIdx.x / LANES;
    float* row = HALVES ? sx + sub * G::kPitch : sx;
    const int h0 = blockIdx.y * a.hpc, h1 = min(h0 + a.hpc, a.heads);
    float dw[8];
    #pragma unroll
    for (int e = 0; e < 8; ++e) dw[e] = 0.f;
    if (threadIdx.x < D) reinterpret_cast<float*>(sw)[threadIdx.x] = weight_at(a.w[z], a.w_f32, threadIdx.x);
    __syncthreads();
    for (int64_t n0 = (int64_t)blockIdx.x * RPB; n0 < a.N; n0 += (int64_t)gridDim.x * RPB) {
        const int64_t n = n0 + sub;
        const bool ok = n < a.N;
        Turn<PAIRS> turn;
        if (a.rope.tab) {
            int t, h, w;
            grid_at(a.rope, ok ? n : 0, t, h, w);
            turn.init(a.rope, ch, t, h, w);
        }
        const TI* src = static_cast<const TI*>(a.in[z].p) + n * a.in[z].ts + ch;
        const TG* gsr = static_cast<const TG*>(a.grad[z].p) + n * a.grad[z].ts + ch;
        TI* dst = static_cast<TI*>(a.out[z].p) + n * a.out[z].ts + ch;
        for (int h = h0; h < h1; h += U) {
            Vec8<TI> v[U];
            Vec8<TG> q[U];
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                v[i] = Vec8<TI>{};
                q[i] = Vec8<TG>{};
                if (ok && h + i < h1) {
                    v[i].load(src + (h + i) * a.in[z].hs);
                    q[i].load(gsr + (h + i) * a.grad[z].hs);
                }
            }
            if (HALVES && a.rope.tab) {
                __syncwarp();                        // the previous group's reads are done
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    float g[8];
                    q[i].get(g);
                    Turn<kHalves>::put(g, row + i * RPB * G::kPitch, ch);
                }
                __syncwarp();
            }
            // (with halves the rotated rows stay in registers: reading the exchange twice cost 13% of the
            // bandwidth; adjacent pairs are rotated again, from fewer registers)
            float w[8], r[U], k[U], kept[KEEP ? U : 1][8];
            read_w(sw[0], ch, w);
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                float x[8], g[8], d0 = 0.f, d1 = 0.f;
                v[i].get(x);
                q[i].get(g);
                if constexpr (PAIRS == kLanes) {
                    float p[8];
                    q[i].of(turn.from(lane, LANES)).get(p);
                    turn.template take<-1>(g, p);
                } else {
                    if (a.rope.tab) turn.template take<-1>(g, row + i * RPB * G::kPitch);
                }
                if (KEEP) {
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) kept[KEEP ? i : 0][e] = g[e];
                }
                r[i] = squares(x);
                #pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    float p0, p1;
                    fmul2(p0, p1, g[e], g[e + 1], w[e], w[e + 1]);
                    ffma2(d0, d1, p0, p1, x[e], x[e + 1], d0, d1);
                }
                k[i] = d0 + d1;
            }
            {
                const float ro = rsqrtf(owned_sum<LANES, U>(r, lane) * (1.f / D) + a.eps);
                const float ko = owned_sum<LANES, U>(k, lane) * ro * ro * ro * (-1.f / D);   // -r^3 mean(w v x)
                #pragma unroll
                for (int i = 0; i < U; ++i) {
                    r[i] = from_owner<U>(ro, lane, i);
                    k[i] = from_owner<U>(ko, lane, i);
                }
            }
            #pragma unroll
            for (int i = 0; i < U; ++i) {
                if (h + i >= h1) break;              // the same for the whole block
                float x[8], g[8];
                v[i].get(x);
                if constexpr (KEEP) {
                    #pragma unroll
                    for (int e = 0; e < 8; ++e) g[e] = kept[i][e];
                } else {
                    q[i].get(g);
                    if (a.rope.tab) turn.template take<-1>(g, nullptr);
                }
                scale8(g, r[i]);                     // r v
                #pragma unroll
                for (int e = 0; e < 8; e += 2) {
                    // a token behind the last one has x = g = 0 and adds nothing
                    ffma2(dw[e], dw[e + 1], g[e], g[e + 1], x[e], x[e + 1], dw[e], dw[e + 1]);
                    fmul2(x[e], x[e + 1], x[e], x[e + 1], k[i], k[i]);
                    ffma2(x[e], x[e + 1], g[e], g[e + 1], w[e], w[e + 1], x[e], x[e + 1]);
                }
                if (ok) Vec8<TI>::store(dst + (h + i) * a.out[z].hs, x);
            }
        }
    }
    if (a.part) {
        __syncthreads();                             // the exchange rows are free
        #pragma unroll
        for (int e = 0; e < 8; ++e) sx[sub * D + ch + e] = dw[e];
        __syncthreads();
        if (threadIdx.x < D) {
            float s = 0.f;
            for (int i = 0; i < RPB; ++i) s += sx[i * D + threadIdx.x];
            const int64_t blk = ((int64_t)z * gridDim.y + blockIdx.y) * gridDim.x + blockIdx.x;
            a.part[blk * D + threadIdx.x] = s;
        }
    }
}

// dw of tensor blockIdx.x: the `blocks` rows of partial sums in a fixed order, in 64 bits
// (a sum over every token and head: its parts cancel).
template <int D>
__global__ void __launch_bounds__(1024) k_norm_rope_dw(const float* part, int blocks, float* dwq, float* dwk) {
    constexpr int G = 1024 / D;
    __shared__ double sm[1024];
    const int c = threadIdx.x % D, g = threadIdx.x / D;
    const float* p = part + (int64_t)blockIdx.x * blocks * D;
    double s = 0.0;
    for (int i = g; i < blocks; i += G) s += p[(int64_t)i * D + c];
    sm[threadIdx.x] = s;
    __syncthreads();
    if (g == 0) {
        for (int i = 1; i < G; ++i) s += sm[i * D + c];
        float* dw = blockIdx.x ? dwk : dwq;
        if (dw) dw[c] = (float)s;
    }
}

// cos and sin of position * theta^(-2 p / d) in 64 bits, rounded once.
__global__ void k_rope_table(int L, int d, int64_t first, double theta, float2* out) {
    const int half = d >> 1, i = blockIdx.x * blockDim.x + threadIdx.x;
    if (i >= L * half) return;
    const int l = i / half, p = i - l * half;
    double s, c;
    sincos((double)(first + l) * pow(theta, -2.0 * p / d), &s, &c);
    out[i] = make_float2((float)c, (float)s);
}

// ------------------------------------------------------------- host side
static bool aligned16(const void* p) { return (reinterpret_cast<uintptr_t>(p) & 15u) == 0; }

static int elt(int dtype) { return dtype == PRISM_F32 ? 4 : 2; }

static bool bad_params(const prism_norm_rope_params* p) {
    if (!p || p->N < 0 || p->N > 0x7fffffffLL || p->heads < 1 || p->heads > 65535 ||
        (p->head_dim != 64 && p->head_dim != 128))
        return true;
    for (int d : {p->dtype, p->out_dtype, p->w_dtype})
        if (d != PRISM_BF16 && d != PRISM_F32) return true;
    return !(p->eps > 0.f) || !(p->eps < 3.0e38f);
}

static bool bad_rope(const prism_norm_rope_params* p) {
    if (p->T < 1 || p->H < 1 || p->W < 1 || (int64_t)p->H * p->W > 0x7fffffffLL ||
        (int64_t)p->T * ((int64_t)p->H * p->W) != p->N)
        return true;
    for (int d : {p->dim_t, p->dim_h, p->dim_w})
        if (d < 0 || (d & 1) || d > p->head_dim) return true;
    return p->dim_t + p->dim_h + p->dim_w > p->head_dim ||
           (p->pairing != PRISM_PAIR_ADJACENT && p->pairing != PRISM_PAIR_HALVES);
}

// Rows must start on 16 bytes; a stride is free when its extent is one.
static bool bad_rows(const prism_rows* r, int dtype, int64_t N, int heads) {
    const int64_t q = 16 / elt(dtype);
    return !r->data || !aligned16(r->data) || (heads > 1 && (r->head_stride % q || r->head_stride < 0)) ||
           (N > 1 && (r->token_stride % q || r->token_stride < 0));
}

// The byte layout of a tensor of rows, for the check that what is written shares no
// element with what else the call reads or writes.
struct Span {
    uintptr_t lo, hi;        // first and one past the last byte
    int64_t hs, ts;          // strides in bytes (0 where the extent is one)
    int heads;
    int64_t N, row;          // row bytes
};

static Span span_of(const prism_rows* r, int dtype, int64_t N, int heads, int D) {
    Span s;
    const int e = elt(dtype);
    s.hs = heads > 1 ? r->head_stride * e : 0;
    s.ts = N > 1 ? r->token_stride * e : 0;
    s.heads = heads;
    s.N = N;
    s.row = (int64_t)D * e;
    s.lo = reinterpret_cast<uintptr_t>(r->data);
    s.hi = s.lo + (uintptr_t)(s.hs * (heads - 1) + s.ts * (N - 1) + s.row);
    return s;
}

// A tensor's rows do not overlap one another (else two rows would be written to one place).
static bool rows_apart(const Span& s) {
    const int64_t a = s.hs, b = s.ts;
    if (s.heads > 1 && a < s.row) return false;
    if (s.N > 1 && b < s.row) return false;
    if (s.heads <= 1 || s.N <= 1) return true;
    return a >= b ? a >= b * (s.N - 1) + s.row : b >= a * (s.heads - 1) + s.row;
}

// Whether two tensors certainly share no byte: apart as ranges, or of the same strides with
// rows that fall between each other's (slices of one fused buffer).
static bool apart(const Span& x, const Span& y) {
    if (x.hi <= y.lo || y.hi <= x.lo) return true;
    if (x.ts != y.ts || x.hs != y.hs || x.N != y.N || x.heads != y.heads) return false;
    // the inner extent of one step of the outer stride
    const bool tok_out = x.ts >= x.hs;
    const int64_t outer = tok_out ? x.ts : x.hs;
    const int64_t xin = (tok_out ? x.hs * (x.heads - 1) : x.ts * (x.N - 1)) + x.row;
    const int64_t yin = (tok_out ? y.hs * (y.heads - 1) : y.ts * (y.N - 1)) + y.row;
    if (outer <= 0) return false;
    const uintptr_t d = y.lo >= x.lo ? y.lo - x.lo : x.lo - y.lo;
    const int64_t m = (int64_t)(d % (uintptr_t)outer);
    return y.lo >= x.lo ? m >= xin && outer - m >= yin : m >= yin && outer - m >= xin;
}

// Consecutive bytes at `p` (none where it is null).
static Span flat(const void* p, size_t bytes) {
    const uintptr_t lo = reinterpret_cast<uintptr_t>(p);
    return Span{lo, p ? lo + bytes : lo, 0, 0, 1, 1, p ? (int64_t)bytes : 0};
}
static bool clear_of(const Span& x, const Span* others, int n) {
    for (int i = 0; i < n; ++i)
        if (others[i].lo != others[i].hi && !apart(x, others[i])) return false;
    return true;
}
static size_t table_bytes(const prism_norm_rope_params* p) {
    return ((size_t)p->T * p->dim_t + (size_t)p->H * p->dim_h + (size_t)p->W * p->dim_w) * sizeof(float);
}

static bool same(const Span& x, const Span& y) {
    return x.lo == y.lo && x.hs == y.hs && x.ts == y.ts && x.row == y.row;
}

static int device_ok() {
    int dev = 0, major = 0, minor = 0;
    if (cudaGetDevice(&dev) != cudaSuccess) return PRISM_ERR_UNSUPPORTED;
    cudaDeviceGetAttribute(&major, cudaDevAttrComputeCapabilityMajor, dev);
    cudaDeviceGetAttribute(&minor, cudaDevAttrComputeCapabilityMinor, dev);
    return major == 10 && minor == 0 ? PRISM_OK : PRISM_ERR_UNSUPPORTED;
}

struct Grid {
    int x, y, z, hpc;
};
constexpr int kFwdPerSM = 32, kBwdPerSM = 8;

// Blocks of a call.  One block takes every head of its tokens (its cos and sin are then
// read once) unless that leaves fewer blocks than two per SM: then the heads are split.
// Token tiles beyond `per_sm` blocks per SM are walked: 8 in the backward, whose blocks each leave
// a row of partial sums, 32 in the forward (2% faster there than 8).
static Grid grid_of(int64_t N, int heads, int D, int z, int per_sm) {
    const int64_t rpb = kThreads / (D / 8), tiles = (N + rpb - 1) / rpb;
    Grid g;
    g.z = z;
    g.hpc = heads;
    while (g.hpc > 1 && tiles * ((heads + g.hpc - 1) / g.hpc) * z < 2 * 148) g.hpc = (g.hpc + 1) / 2;
    g.y = (heads + g.hpc - 1) / g.hpc;
    const int64_t most = (int64_t)per_sm * 148 / ((int64_t)g.y * z), cap = most > 1 ? most : 1;
    g.x = (int)(tiles < cap ? tiles : cap);
    return g;
}

static Rope rope_of(const prism_norm_rope_params* p, const float* table) {
    Rope r;
    r.tab = reinterpret_cast<const float2*>(table);
    r.T = p->T; r.H = p->H; r.W = p->W;
    r.dt = p->dim_t; r.dh = p->dim_h; r.dw = p->dim_w;
    return r;
}

template <typename TI, typename TO, bool BWD, int D>
static void launch(const Args& a, const Grid& g, int pairs, cudaStream_t s) {
    const dim3 grid(g.x, g.y, g.z);
    if constexpr (BWD) {
        pairs == kAdjacent ? k_norm_rope_bwd<TI, TO, D, kAdjacent><<<grid, kThreads, 0, s>>>(a)
        : pairs == kLanes  ? k_norm_rope_bwd<TI, TO, D, kLanes><<<grid, kThreads, 0, s>>>(a)
                           : k_norm_rope_bwd<TI, TO, D, kHalves><<<grid, kThreads, 0, s>>>(a);
    } else {
        pairs == kAdjacent ? k_norm_rope<TI, TO, D, kAdjacent><<<grid, kThreads, 0, s>>>(a)
        : pairs == kLanes  ? k_norm_rope<TI, TO, D, kLanes><<<grid, kThreads, 0, s>>>(a)
                           : k_norm_rope<TI, TO, D, kHalves><<<grid, kThreads, 0, s>>>(a);
    }
}

template <bool BWD, int D>
static void by_type(const prism_norm_rope_params* p, const Args& a, const Grid& g, int pairs, cudaStream_t s) {
    using bf = __nv_bfloat16;
    const bool in32 = p->dtype == PRISM_F32, out32 = p->out_dtype == PRISM_F32;
    if (in32) out32 ? launch<float, float, BWD, D>(a, g, pairs, s) : launch<float, bf, BWD, D>(a, g, pairs, s);
    else out32 ? launch<bf, float, BWD, D>(a, g, pairs, s) : launch<bf, bf, BWD, D>(a, g, pairs, s);
}
template <bool BWD>
static int dispatch(const prism_norm_rope_params* p, const Args& a, const Grid& g, cudaStream_t s) {
    int pairs = kAdjacent;
    if (a.rope.tab && p->pairing == PRISM_PAIR_HALVES)
        pairs = (p->dim_t | p->dim_h | p->dim_w) % 16 == 0 ? kLanes : kHalves;
    p->head_dim == 128 ? by_type<BWD, 128>(p, a, g, pairs, s) : by_type<BWD, 64>(p, a, g, pairs, s);
    return cudaGetLastError() == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA;
}

static Rows rows_of(const prism_rows* r) { return Rows{r->data, r->head_stride, r->token_stride}; }

static int64_t part_rows(int64_t N, int heads, int D, int z) {
    const Grid g = grid_of(N, heads, D, z, kBwdPerSM);
    return (int64_t)g.x * g.y * g.z;
}

}  // namespace nr
}  // namespace prism

extern "C" int prism_rope_table(const prism_norm_rope_params* p, float theta, int64_t first_frame, float* table,
                                void* stream) {
    using namespace prism::nr;
    if (bad_params(p) || p->N < 1 || bad_rope(p) || !table || !aligned16(table) || !(theta > 0.f) || !(theta < 3.0e38f) ||
        first_frame < 0 || first_frame > (1LL << 40))
        return PRISM_ERR_INVALID_ARG;
    if (int st = device_ok()) return st;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    float2* out = reinterpret_cast<float2*>(table);
    const int L[3] = {p->T, p->H, p->W}, d[3] = {p->dim_t, p->dim_h, p->dim_w};
    for (int i = 0; i < 3; ++i) {
        const int64_t n = (int64_t)L[i] * (d[i] / 2);
        if (n > 0x7fffffffLL - 256) return PRISM_ERR_INVALID_ARG;
        if (n == 0) continue;
        k_rope_table<<<(unsigned)((n + 255) / 256), 256, 0, s>>>(L[i], d[i], i == 0 ? first_frame : 0, (double)theta, out);
        out += n;
    }
    return cudaGetLastError() == cudaSuccess ? PRISM_OK : PRISM_ERR_CUDA;
}

extern "C" int prism_qk_norm_rope(const prism_norm_rope_params* p, const prism_rows* q, const prism_rows* k,
                                  const void* wq, const void* wk, const float* rope, const prism_rows* q_out,
                                  const prism_rows* k_out, void* stream) {
    using namespace prism::nr;
    if (bad_params(p) || !q || !q_out || !k != !k_out) return PRISM_ERR_INVALID_ARG;
    if (p->N == 0) return PRISM_OK;
    if (rope && (!aligned16(rope) || bad_rope(p))) return PRISM_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wk) || (wk && !k)) return PRISM_ERR_INVALID_ARG;
    const int D = p->head_dim, z = k ? 2 : 1;
    const prism_rows* in[2] = {q, k};
    const prism_rows* out[2] = {q_out, k_out};
    Span si[2], so[2];
    for (int i = 0; i < z; ++i) {
        if (bad_rows(in[i], p->dtype, p->N, p->heads) || bad_rows(out[i], p->out_dtype, p->N, p->heads))
            return PRISM_ERR_INVALID_ARG;
        si[i] = span_of(in[i], p->dtype, p->N, p->heads, D);
        so[i] = span_of(out[i], p->out_dtype, p->N, p->heads, D);
        if (!rows_apart(so[i])) return PRISM_ERR_INVALID_ARG;
    }
    for (int i = 0; i < z; ++i)
        for (int j = 0; j < z; ++j)
            if (!apart(so[i], si[j]) && !(i == j && same(so[i], si[j]))) return PRISM_ERR_INVALID_ARG;
    if (z == 2 && !apart(so[0], so[1])) return PRISM_ERR_INVALID_ARG;
    const Span read[3] = {flat(wq, (size_t)D * elt(p->w_dtype)), flat(wk, (size_t)D * elt(p->w_dtype)),
                          flat(rope, rope ? table_bytes(p) : 0)};
    for (int i = 0; i < z; ++i)
        if (!clear_of(so[i], read, 3)) return PRISM_ERR_INVALID_ARG;
    if (int st = device_ok()) return st;
    Args a{};
    for (int i = 0; i < z; ++i) {
        a.in[i] = rows_of(in[i]);
        a.out[i] = rows_of(out[i]);
    }
    a.w[0] = wq;
    a.w[1] = wk;
    a.w_f32 = p->w_dtype == PRISM_F32;
    a.tensors = z;
    a.rope = rope_of(p, rope);
    a.N = p->N;
    a.heads = p->heads;
    a.eps = p->eps;
    const Grid g = grid_of(p->N, p->heads, D, 1, kFwdPerSM);
    a.hpc = g.hpc;
    nvtxRangePushA("prism qk norm rope");
    const int st = dispatch<false>(p, a, g, static_cast<cudaStream_t>(stream));
    nvtxRangePop();
    return st;
}

extern "C" size_t prism_qk_norm_rope_bwd_workspace_bytes(const prism_norm_rope_params* p) {
    using namespace prism::nr;
    if (bad_params(p)) return 0;
    if (p->N == 0) return 16;
    const int64_t one = part_rows(p->N, p->heads, p->head_dim, 1), two = part_rows(p->N, p->heads, p->head_dim, 2);
    return (size_t)(one > two ? one : two) * p->head_dim * sizeof(float);
}

extern "C" int prism_qk_norm_rope_bwd(const prism_norm_rope_params* p, const prism_rows* dq_out,
                                      const prism_rows* dk_out, const prism_rows* q, const prism_rows* k,
                                      const void* wq, const void* wk, const float* rope, const prism_rows* dq,
                                      const prism_rows* dk, float* dwq, float* dwk, void* workspace, size_t ws_bytes,
                                      void* stream) {
    using namespace prism::nr;
    if (bad_params(p) || !q || !dq_out || !dq || !k != !dk_out || !k != !dk) return PRISM_ERR_INVALID_ARG;
    if ((dwk || wk) && !k) return PRISM_ERR_INVALID_ARG;
    if (!aligned16(wq) || !aligned16(wk) || !aligned16(dwq) || !aligned16(dwk)) return PRISM_ERR_INVALID_ARG;
    const int D = p->head_dim, z = k ? 2 : 1;
    const Span both[1] = {flat(dwk, D * sizeof(float))};
    if (dwq && !clear_of(flat(dwq, D * sizeof(float)), both, 1)) return PRISM_ERR_INVALID_ARG;
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (p->N == 0) {         // no rows: the weights' gradients are zero
        for (float* dw : {dwq, dwk})
            if (dw && cudaMemsetAsync(dw, 0, D * sizeof(float), s) != cudaSuccess) return PRISM_ERR_CUDA;
        return PRISM_OK;
    }
    if (rope && (!aligned16(rope) || bad_rope(p))) return PRISM_ERR_INVALID_ARG;
    const prism_rows* in[2] = {q, k};
    const prism_rows* gr[2] = {dq_out, dk_out};
    const prism_rows* out[2] = {dq, dk};
    Span si[2], sg[2], so[2];
    for (int i = 0; i < z; ++i) {
        if (bad_rows(in[i], p->dtype, p->N, p->heads) || bad_rows(gr[i], p->out_dtype, p->N, p->heads) ||
            bad_rows(out[i], p->dtype, p->N, p->heads))
            return PRISM_ERR_INVALID_ARG;
        si[i] = span_of(in[i], p->dtype, p->N, p->heads, D);
        sg[i] = span_of(gr[i], p->out_dtype, p->N, p->heads, D);
        so[i] = span_of(out[i], p->dtype, p->N, p->heads, D);
        if (!rows_apart(so[i])) return PRISM_ERR_INVALID_ARG;
    }
    for (int i = 0; i < z; ++i)
        for (int j = 0; j < z; ++j) {
            if (!apart(so[i], si[j]) && !(i == j && same(so[i], si[j]))) return PRISM_ERR_INVALID_ARG;
            if (!apart(so[i], sg[j]) && !(i == j && same(so[i], sg[j]))) return PRISM_ERR_INVALID_ARG;
        }
    if (z == 2 && !apart(so[0], so[1])) return PRISM_ERR_INVALID_ARG;
    const bool want = dwq || dwk;
    if (want && (!workspace || !aligned16(workspace))) return PRISM_ERR_INVALID_ARG;
    const size_t need = want ? prism_qk_norm_rope_bwd_workspace_bytes(p) : 0;
    if (want && ws_bytes < need) return PRISM_ERR_WORKSPACE;
    // the vectors, the table and the workspace: what is written of them is apart from all else, what
    // is read from what is written
    const Span vec[6] = {flat(dwq, D * sizeof(float)), flat(dwk, D * sizeof(float)), flat(want ? workspace : nullptr, need),
                         flat(wq, (size_t)D * elt(p->w_dtype)), flat(wk, (size_t)D * elt(p->w_dtype)),
                         flat(rope, rope ? table_bytes(p) : 0)};
    for (int i = 0; i < z; ++i)
        if (!clear_of(so[i], vec, 6) || !clear_of(si[i], vec, 3) || !clear_of(sg[i], vec, 3)) return PRISM_ERR_INVALID_ARG;
    for (int i = 0; i < 3; ++i)
        if (vec[i].lo != vec[i].hi && !clear_of(vec[i], vec + i + 1, 5 - i)) return PRISM_ERR_INVALID_ARG;
    if (int st = device_ok()) return st;
    Args a{};
    for (int i = 0; i < z; ++i) {
        a.in[i] = rows_of(in[i]);
        a.grad[i] = rows_of(gr[i]);
        a.out[i] = rows_of(out[i]);
    }
    a.w[0] = wq;
    a.w[1] = wk;
    a.w_f32 = p->w_dtype == PRISM_F32;
    a.tensors = z;
    a.rope = rope_of(p, rope);
    a.N = p->N;
    a.heads = p->heads;
    a.eps = p->eps;
    const Grid g = grid_of(p->N, p->heads, D, z, kBwdPerSM);
    a.hpc = g.hpc;
    a.part = want ? static_cast<float*>(workspace) : nullptr;
    nvtxRangePushA("prism qk norm rope bwd");
    int st = dispatch<true>(p, a, g, s);
    if (!st && want) {
        if (D == 128) k_norm_rope_dw<128><<<z, 1024, 0, s>>>(a.part, g.x * g.y, dwq, dwk);
        else k_norm_rope_dw<64><<<z, 1024, 0, s>>>(a.part, g.x * g.y, dwq, dwk);
        if (cudaGetLastError() != cudaSuccess) st = PRISM_ERR_CUDA;
    }
    nvtxRangePop();
    return st;
}
