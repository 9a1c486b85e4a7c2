// Decode step and read-only attend over an E2M1 cache (D = 64 or 128, G <= 8).
//
// A cached vector is D / 2 bytes of codes and D / 16 bytes of E4M3 scales
// (gqa_fp4.cuh), 0.5625 bytes an element, so the step is bound by what the
// SMs spend on unpacking about as much as by memory; the kernel is laid out to
// unpack with few instructions and to need no shared memory for the cache:
//  * the schedule, the split of a unit between CTAs and its merge are those of
//    the other decode kernels (gqa_common.cuh). A CTA is four warps, a tile
//    4 x 16 x kSub slots; each warp takes its 16 x kSub slots of every tile
//    straight from global memory into registers, in the layout of the matrix
//    instructions' operands, one tile ahead.
//  * S^T = K Q^T (m16n8k16, f16 in, float32 sums): the M side is 16 slots, the
//    N side the G <= 8 query rows. Lane (g, t) of a warp holds slots g and
//    g + 8, and of each the D / 4 contiguous dims from D / 4 * t: one 16-byte
//    load (D = 128) a slot. Which dims make up a product step does not matter
//    to a dot product as long as the query fragments are taken in the same
//    order.
//  * O^T += V^T P^T: the M side is 16 dims, the N side the query rows, the
//    contraction 16 slots. Lane (g, t) holds slots 2t, 2t + 1, 2t + 8, 2t + 9
//    and of each the D / 8 contiguous dims from D / 8 * g, the rows of the M
//    side being interleaved to match; a pair of slots is put together while it
//    is multiplied by its scales.
//  * codes become f16 by the hardware's conversion and every E2M1 x E4M3
//    product is an f16 exactly, so K and V enter the products unrounded. A
//    bfloat16 query is scaled by a power of two into f16's range (exact but
//    for elements 2^-38 below the row's largest); a float32 query is an f16
//    and an f16 remainder (22 bits). The weights P are an f16 and a remainder
//    too: in f16 alone the output would be off by 1e-4.
//  * the softmax keeps a reference below the running maximum: weights are
//    2^(s - m) with m set to max - 7 and raised only when a score passes
//    m + 15, so they stay within f16's range and a tile costs a vote instead
//    of a reduction.
//  * the new token (decode step): the warp whose tile holds slot L quantises
//    k_new and v_new, writes them to the cache, and then loads the tile; no
//    other warp touches slot L.
#define GQA_MULTI_TOKEN 0   // single-token steps only
#include <cuda_fp16.h>

#include "gqa_common.cuh"
#include "gqa_fp4.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 2;                       // 16-slot parts of a warp's share of a tile
constexpr int kTile4 = kWarps * 16 * kSub;    // slots a tile
constexpr int kRows = 8;                      // query rows (G <= 8)
constexpr float kLift = 7.f;                  // a reference is set this far below the maximum ...
constexpr float kRoom = 15.f;                 // ... and holds until a score is this far above it

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm volatile("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
                 "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
                 : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
                 : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }

// Two float32 as an f16 pair and the f16 pair of what it leaves.
__device__ __forceinline__ void split2(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = u32(h);
    lo = u32(__floats2half2_rn(x - f.x, y - f.y));
}

// Loads that see this SM's own earlier stores (the append).
__device__ __forceinline__ uint4 ld16(const void *p) { return __ldcg(static_cast<const uint4 *>(p)); }
__device__ __forceinline__ uint2 ld8(const void *p) { return __ldcg(static_cast<const uint2 *>(p)); }
__device__ __forceinline__ uint32_t ld4(const void *p) { return __ldcg(static_cast<const uint32_t *>(p)); }
__device__ __forceinline__ uint32_t ld2(const void *p) { return __ldcg(static_cast<const unsigned short *>(p)); }
__device__ __forceinline__ uint32_t ld1(const void *p) { return __ldcg(static_cast<const uint8_t *>(p)); }

// A warp's 16 slots of a tile, as loaded.
template <int D>
struct Frag {
    uint32_t k[2][D / 32];   // slots g, g + 8: the lane's D / 4 dims
    uint32_t v[4][D / 64];   // slots 2t, 2t + 1, 2t + 8, 2t + 9: the lane's D / 8 dims
    uint32_t ks;             // K scales: slot g's in the low half (D = 128: two bytes, 64: one)
    uint32_t vs;             // V scales: one byte a slot
};

template <int D>
__device__ __forceinline__ void load_k(const DecodeParams &p, long long off, int t, uint32_t (&k)[D / 32], uint32_t &s)
{
    const uint8_t *c = static_cast<const uint8_t *>(p.k_cache) + (off >> 1) + (D / 8) * t;
    const uint8_t *gs = static_cast<const uint8_t *>(p.k_group) + (off >> 4) + (D / 64) * t;
    if constexpr (D == 128) {
        const uint4 w = ld16(c);
        k[0] = w.x; k[1] = w.y; k[2] = w.z; k[3] = w.w;
        s = ld2(gs);
    } else {
        const uint2 w = ld8(c);
        k[0] = w.x; k[1] = w.y;
        s = ld1(gs);
    }
}

template <int D>
__device__ __forceinline__ void load_v(const DecodeParams &p, long long off, int g, uint32_t (&v)[D / 64], uint32_t &s)
{
    const uint8_t *c = static_cast<const uint8_t *>(p.v_cache) + (off >> 1) + (D / 16) * g;
    s = ld1(static_cast<const uint8_t *>(p.v_group) + (off >> 4) + (D == 128 ? g : g >> 1));
    if constexpr (D == 128) {
        const uint2 w = ld8(c);
        v[0] = w.x; v[1] = w.y;
    } else {
        v[0] = ld4(c);
    }
}

// The slots s0 .. s0 + 15 of the cursor's unit. Slots outside the softmax
// read as zeros. `bad` is set where the block table holds no usable block.
template <int D>
__device__ __forceinline__ void load_frag(const DecodeParams &p, const TileCursor &c, bool good, int s0, int lane,
                                          Frag<D> &f, int &bad)
{
    const int g = lane >> 2, t = lane & 3;
    f.ks = f.vs = 0;
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int s = s0 + g + 8 * i;
#pragma unroll
        for (int w = 0; w < D / 32; ++w)
            f.k[i][w] = 0;
        if (good && attended(c.L, c.lo, c.P, s)) {
            const long long off = slot_offset(p, c.b, c.kvh, s);
            if (off < 0) {
                bad = 1;
            } else {
                uint32_t sc;
                load_k<D>(p, off, t, f.k[i], sc);
                f.ks |= sc << (16 * i);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i) {
        const int s = s0 + 2 * t + (i & 1) + 8 * (i >> 1);
#pragma unroll
        for (int w = 0; w < D / 64; ++w)
            f.v[i][w] = 0;
        if (good && attended(c.L, c.lo, c.P, s)) {
            const long long off = slot_offset(p, c.b, c.kvh, s);
            if (off < 0) {
                bad = 1;
            } else {
                uint32_t sc;
                load_v<D>(p, off, g, f.v[i], sc);
                f.vs |= sc << (8 * i);
            }
        }
    }
}

// The new token's vector x (bfloat16, D of them) quantised into the cache at
// element offset off, by one warp: D / 32 dims a lane.
template <int D>
__device__ __forceinline__ void append_vec(const __nv_bfloat16 *x, void *cache, void *groups, long long off, float g,
                                           int lane)
{
    constexpr int N = D / 32;          // 2 or 4 dims
    constexpr int LG = kGroup / N;     // lanes of a group
    float v[N];
    const uint32_t *w = reinterpret_cast<const uint32_t *>(x + lane * N);
#pragma unroll
    for (int i = 0; i < N / 2; ++i) {
        const uint32_t u = __ldg(w + i);
        v[2 * i] = bf16_lo(u);
        v[2 * i + 1] = bf16_hi(u);
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        amax = max_nan(amax, fabsf(v[i]));
#pragma unroll
    for (int o = 1; o < LG; o <<= 1)
        amax = max_nan(amax, __shfl_xor_sync(0xffffffffu, amax, o));
    float t;
    const uint32_t s = group_scale(amax, g, t);
    uint8_t *c = static_cast<uint8_t *>(cache) + (off >> 1) + lane * (N / 2);
#pragma unroll
    for (int i = 0; i < N / 2; ++i)
        c[i] = (uint8_t)to_e2m1x2(over_t(v[2 * i], t), over_t(v[2 * i + 1], t));
    if (lane % LG == 0)
        static_cast<uint8_t *>(groups)[(off >> 4) + lane / LG] = (uint8_t)s;
}

__device__ __forceinline__ int scale_head(const DecodeParams &p, const TileCursor &c)
{
    return p.scale_heads ? c.b % p.scale_heads : c.kvh;
}

// A warp's share of the cursor's tile: the append, then the loads.
template <int D>
__device__ __forceinline__ void load_part(const DecodeParams &p, const TileCursor &c, bool good, int warp, int u,
                                          int lane, Frag<D> &f, int &bad)
{
    const int s0 = tile_slot0(c, kTile4) + warp * 16 * kSub + u * 16;
    if (!p.attend && good && c.L >= s0 && c.L < s0 + 16) {
        const long long off = slot_offset(p, c.b, c.kvh, c.L);
        if (off >= 0) {
            const int h = scale_head(p, c);
            const long long src = ((long long)c.b * p.Hkv + c.kvh) * D;
            append_vec<D>(static_cast<const __nv_bfloat16 *>(p.k_new) + src, p.k_cache, p.k_group, off,
                          __ldg(p.k_scale + h), lane);
            append_vec<D>(static_cast<const __nv_bfloat16 *>(p.v_new) + src, p.v_cache, p.v_group, off,
                          __ldg(p.v_scale + h), lane);
            __syncwarp();              // the loads below see the whole vector
        }
    }
    load_frag<D>(p, c, good, s0, lane, f, bad);
}

// The unit's query fragments: lane (g, t) holds row g's D / 4 dims from
// D / 4 * t, scaled by a power of two into f16's range; `mul` is the factor
// that takes a product to a base-2 score for row g.
template <int D, bool QF32>
__device__ __forceinline__ void load_query(const DecodeParams &p, const TileCursor &c, int lane,
                                           uint32_t (&qh)[D / 16][2], uint32_t (&ql)[QF32 ? D / 16 : 1][2], float &mul)
{
    constexpr int N = D / 4;
    const int g = lane >> 2, t = lane & 3;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = 0.f;
    if (g < p.G) {
        const long long at = ((long long)c.b * p.Hq + (long long)c.kvh * p.G + g) * D + N * t;
        if constexpr (QF32) {
            const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(p.q) + at);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v = __ldg(s + i);
                x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
            }
        } else {
            const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.q) + at);
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const uint4 v = __ldg(s + i);
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = bf16_lo(w[j]);
                    x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
                }
            }
        }
    }
    float amax = 0.f;
#pragma unroll
    for (int i = 0; i < N; ++i)
        amax = fmaxf(amax, fabsf(x[i]));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 1));
    amax = fmaxf(amax, __shfl_xor_sync(0xffffffffu, amax, 2));
    // 2^(14 - exponent of amax), within float32's normal range both ways
    const int e = min(max((int)(__float_as_uint(amax) >> 23) - 127, -110), 127);
    const float up = __uint_as_float((uint32_t)(127 + 14 - e) << 23);
    mul = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * p.scale_log2;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float a = x[4 * i + 2 * j] * up, b = x[4 * i + 2 * j + 1] * up;
            if constexpr (QF32)
                split2(a, b, qh[i][j], ql[i][j]);
            else
                qh[i][j] = u32(__floats2half2_rn(a, b));
        }
}

// Scores of a part's 16 slots: s[0], s[1] slot g and query rows 2t, 2t + 1;
// s[2], s[3] slot g + 8.
template <int D, bool QF32>
__device__ __forceinline__ void scores(const Frag<D> &f, const uint32_t (&qh)[D / 16][2],
                                       const uint32_t (&ql)[QF32 ? D / 16 : 1][2], float (&s)[4])
{
    float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = 0.f;
    const __half2 sa = h2(e4m3x2_f16(f.ks & 0xffffu)), sb = h2(e4m3x2_f16(f.ks >> 16));
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint32_t a[4], b[4];           // four pairs of slot g, of slot g + 8
        e2m1x8_f16(f.k[0][w], a);
        e2m1x8_f16(f.k[1][w], b);
        // D = 128: the lane's first two words are one group, the others the next
        const __half2 ma = (D == 128 && w >= 2) ? __high2half2(sa) : __low2half2(sa);
        const __half2 mb = (D == 128 && w >= 2) ? __high2half2(sb) : __low2half2(sb);
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            a[j] = u32(__hmul2(h2(a[j]), ma));
            b[j] = u32(__hmul2(h2(b[j]), mb));
        }
        mma_f16(s, a[0], b[0], a[1], b[1], qh[2 * w][0], qh[2 * w][1]);
        mma_f16(s2, a[2], b[2], a[3], b[3], qh[2 * w + 1][0], qh[2 * w + 1][1]);
        if constexpr (QF32) {
            mma_f16(s, a[0], b[0], a[1], b[1], ql[2 * w][0], ql[2 * w][1]);
            mma_f16(s2, a[2], b[2], a[3], b[3], ql[2 * w + 1][0], ql[2 * w + 1][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] += s2[i];
}

// O^T += V^T P^T for a part's 16 slots; w[0..3] are the weights in the
// positions of the scores.
template <int D>
__device__ __forceinline__ void weigh(const Frag<D> &f, const float (&w)[4], float (&o)[D / 16][4])
{
    uint32_t h0, l0, h1, l1;
    split2(w[0], w[1], h0, l0);
    split2(w[2], w[3], h1, l1);
    h0 = movmatrix_t(h0);
    h1 = movmatrix_t(h1);
    l0 = movmatrix_t(l0);
    l1 = movmatrix_t(l1);
    const __half2 s01 = h2(e4m3x2_f16(f.vs & 0xffffu)), s23 = h2(e4m3x2_f16(f.vs >> 16));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        uint32_t x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            e2m1x8_f16(f.v[j][i], x[j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const __half2 a0 = __hmul2(__lows2half2(h2(x[0][q]), h2(x[1][q])), s01);
            const __half2 a1 = __hmul2(__highs2half2(h2(x[0][q]), h2(x[1][q])), s01);
            const __half2 a2 = __hmul2(__lows2half2(h2(x[2][q]), h2(x[3][q])), s23);
            const __half2 a3 = __hmul2(__highs2half2(h2(x[2][q]), h2(x[3][q])), s23);
            mma_f16(o[4 * i + q], u32(a0), u32(a1), u32(a2), u32(a3), h0, h1);
            mma_f16(o[4 * i + q], u32(a0), u32(a1), u32(a2), u32(a3), l0, l1);
        }
    }
}

template <int D, bool QF32>
__global__ void __launch_bounds__(kThreads) q4_decode_kernel(const DecodeParams p)
{
    __shared__ long long sched[kThreads / 32 + 8];
    __shared__ TileWalk walk;
    __shared__ int sm_flag;
    __shared__ MergeBuf sm_merge;
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ __align__(16) float sm_o[kWarps][kRows][D + 4];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t = lane & 3;

    // programmatic dependent of the previous kernel: read no input before it is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    schedule_walk(p, sched, &walk);
    TileCursor cur;
    bool in_b = false;
    bool more = walk_first(p, cur, walk, in_b);
    if (!more)
        return;

    Frag<D> f[kSub];
    int bad = 0, bad_next = 0;                  // of the current segment, of the tile loaded ahead
    bool good = row_ok(p, cur.b, cur.L);
#pragma unroll
    for (int u = 0; u < kSub; ++u)
        load_part<D>(p, cur, good, warp, u, lane, f[u], bad);

    uint32_t qh[D / 16][2], ql[QF32 ? D / 16 : 1][2];
    float mul0 = 0.f, mul1 = 0.f;               // product to base-2 score, rows 2t and 2t + 1
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 16][4];
    bool start = true;
    int seg_first_t = 0;

    while (more) {
        if (start) {
            seg_first_t = cur.t;
            if (!good && tid == 0 && cur.t == 0 && cur.kvh == 0)
                report(p, row_error_bits(p, cur.b, cur.L));
            float mul;
            load_query<D, QF32>(p, cur, lane, qh, ql, mul);
            const float ks = __ldg(p.k_scale + scale_head(p, cur));
            mul0 = __shfl_sync(0xffffffffu, mul, 8 * t) * ks;
            mul1 = __shfl_sync(0xffffffffu, mul, 8 * t + 4) * ks;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[i][j] = 0.f;
            start = false;
        }
        TileCursor nxt = cur;
        bool nxt_in_b = in_b;
        const bool more_n = walk_next(p, nxt, walk, nxt_in_b);
        const bool good_n = more_n && (nxt.b == cur.b ? good : row_ok(p, nxt.b, nxt.L));
        const int s0 = tile_slot0(cur, kTile4) + warp * 16 * kSub;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            float s[4];
            scores<D, QF32>(f[u], qh, ql, s);
            const int j0 = s0 + 16 * u + g;
            const bool v0 = good && attended(cur.L, cur.lo, cur.P, j0);
            const bool v1 = good && attended(cur.L, cur.lo, cur.P, j0 + 8);
            s[0] = v0 ? s[0] * mul0 : -INFINITY;
            s[1] = v0 ? s[1] * mul1 : -INFINITY;
            s[2] = v1 ? s[2] * mul0 : -INFINITY;
            s[3] = v1 ? s[3] * mul1 : -INFINITY;
            float c0 = fmaxf(s[0], s[2]), c1 = fmaxf(s[1], s[3]);
            if (__any_sync(0xffffffffu, c0 > m0 + kRoom || c1 > m1 + kRoom)) {
#pragma unroll
                for (int q = 4; q < 32; q <<= 1) {
                    c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, q));
                    c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, q));
                }
                // raised only where a score passed the room left
                const float n0 = c0 > m0 + kRoom ? c0 - kLift : m0, n1 = c1 > m1 + kRoom ? c1 - kLift : m1;
                const float r0 = m0 == -INFINITY ? 0.f : fast_ex2(m0 - n0);
                const float r1 = m1 == -INFINITY ? 0.f : fast_ex2(m1 - n1);
                m0 = n0;
                m1 = n1;
                l0 *= r0;
                l1 *= r1;
#pragma unroll
                for (int i = 0; i < D / 16; ++i) {
                    o[i][0] *= r0;
                    o[i][1] *= r1;
                    o[i][2] *= r0;
                    o[i][3] *= r1;
                }
            }
            s[0] = v0 ? fast_ex2(s[0] - m0) : 0.f;
            s[1] = v0 ? fast_ex2(s[1] - m1) : 0.f;
            s[2] = v1 ? fast_ex2(s[2] - m0) : 0.f;
            s[3] = v1 ? fast_ex2(s[3] - m1) : 0.f;
            l0 += s[0] + s[2];
            l1 += s[1] + s[3];
            weigh<D>(f[u], s, o);
            if (more_n)
                load_part<D>(p, nxt, good_n, warp, u, lane, f[u], bad_next);
        }

        const bool unit_done = (cur.t == cur.nr - 1);
        const bool cta_done = (cur.g + 1 == cur.end);
        if (unit_done || cta_done) {
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) {
                l0 += __shfl_xor_sync(0xffffffffu, l0, q);
                l1 += __shfl_xor_sync(0xffffffffu, l1, q);
            }
            // a NaN score raises no reference: keep the NaN sum in the merge
            m0 = (l0 != l0 && m0 == -INFINITY) ? 0.f : m0;
            m1 = (l1 != l1 && m1 == -INFINITY) ? 0.f : m1;
            if (g == 0) {
                sm_m[warp][2 * t] = m0;
                sm_m[warp][2 * t + 1] = m1;
                sm_l[warp][2 * t] = l0;
                sm_l[warp][2 * t + 1] = l1;
            }
            const float vs = __ldg(p.v_scale + scale_head(p, cur));
#pragma unroll
            for (int i = 0; i < D / 16; i += 2) {
                // rows 2t, 2t + 1: dims D / 8 * g + 2i .. + 3
                *reinterpret_cast<float4 *>(&sm_o[warp][2 * t][D / 8 * g + 2 * i]) =
                    make_float4(o[i][0] * vs, o[i][2] * vs, o[i + 1][0] * vs, o[i + 1][2] * vs);
                *reinterpret_cast<float4 *>(&sm_o[warp][2 * t + 1][D / 8 * g + 2 * i]) =
                    make_float4(o[i][1] * vs, o[i][3] * vs, o[i + 1][1] * vs, o[i + 1][3] * vs);
            }
            const bool seg_bad = __syncthreads_or(bad) != 0;
            bad = 0;
            if (seg_bad && good && tid == 0)
                report(p, kBadBlock);
            finish_segment<kWarps, kRows, D, D + 4, false>(p, cur, walk, seg_first_t, !good || seg_bad, sm_m, sm_l,
                                                          sm_o, &sm_flag, sm_merge, tid, kThreads,
                                                          [] { __syncthreads(); });
            start = true;
        }
        bad |= bad_next;
        bad_next = 0;
        cur = nxt;
        in_b = nxt_in_b;
        good = good_n;
        more = more_n;
    }
}

template <int D, bool QF32>
cudaError_t launch_one(const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    if (!p)
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, q4_decode_kernel<D, QF32>, kThreads, 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p->grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q4_decode_kernel<D, QF32>, *p);
}

}  // namespace

bool q4_supports(int D, int G) { return (D == 64 || D == 128) && G >= 1 && G <= kRows; }

int q4_tile() { return kTile4; }

// The smaller of the two query types' CTAs on an SM: one grid (and one
// workspace size) for both.
int q4_ctas_per_sm(int D)
{
    int a = 0, b = 0;
    const cudaError_t e = D == 128 ? launch_one<128, false>(nullptr, nullptr, &a) : launch_one<64, false>(nullptr, nullptr, &a);
    const cudaError_t h = D == 128 ? launch_one<128, true>(nullptr, nullptr, &b) : launch_one<64, true>(nullptr, nullptr, &b);
    const int n = a < b ? a : b;
    return (e == cudaSuccess && h == cudaSuccess && n > 0) ? n : 1;
}

cudaError_t q4_launch(const DecodeParams &p, cudaStream_t st)
{
    if (p.D == 128)
        return p.q_bf16 ? launch_one<128, false>(&p, st, nullptr) : launch_one<128, true>(&p, st, nullptr);
    return p.q_bf16 ? launch_one<64, false>(&p, st, nullptr) : launch_one<64, true>(&p, st, nullptr);
}

}  // namespace gqa
