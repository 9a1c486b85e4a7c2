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
constexpr int kFlush = 8;                     // tiles between additions to the state in shared memory
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

// A warp's 16 slots of a tile, as loaded.
template <int D>
struct Frag {
    uint32_t k[2][D / 32];   // slots g, g + 8: the lane's D / 4 dims
    uint32_t v[4][D / 64];   // slots 2t, 2t + 1, 2t + 8, 2t + 9: the lane's D / 8 dims
    uint32_t ks, vs;         // four scale bytes of K, of V: the 16 slots' D scales in memory order,
                             // lane by lane (D = 64: lanes 16 .. 31 repeat lanes 0 .. 15)
};

// The lane's places in a cached vector, at vector 0 of the cache.
struct Bases {
    const uint8_t *k, *v, *ks, *vs;
};

template <int D>
__device__ __forceinline__ Bases bases(const DecodeParams &p, int lane)
{
    const int g = lane >> 2, t = lane & 3;
    Bases r;
    r.k = static_cast<const uint8_t *>(p.k_cache) + (D / 2) * g + (D / 8) * t;
    r.v = static_cast<const uint8_t *>(p.v_cache) + (D / 2) * 2 * t + (D / 16) * g;
    r.ks = static_cast<const uint8_t *>(p.k_group) + 4 * (lane % (D / 4));
    r.vs = static_cast<const uint8_t *>(p.v_group) + 4 * (lane % (D / 4));
    return r;
}

__device__ __forceinline__ uint32_t ld4(const uint8_t *p) { return *reinterpret_cast<const uint32_t *>(p); }

template <int D>
__device__ __forceinline__ void ld_k(const uint8_t *p, uint32_t (&k)[D / 32])
{
    if constexpr (D == 128) {
        const uint4 w = *reinterpret_cast<const uint4 *>(p);
        k[0] = w.x; k[1] = w.y; k[2] = w.z; k[3] = w.w;
    } else {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        k[0] = w.x; k[1] = w.y;
    }
}

template <int D>
__device__ __forceinline__ void ld_v(const uint8_t *p, uint32_t (&v)[D / 64])
{
    if constexpr (D == 128) {
        const uint2 w = *reinterpret_cast<const uint2 *>(p);
        v[0] = w.x; v[1] = w.y;
    } else {
        v[0] = ld4(p);
    }
}

// Sixteen slots that are vectors `row` .. row + 15 of the cache.
template <int D>
__device__ __forceinline__ void load_k(const Bases &r, uint32_t row, Frag<D> &f)
{
    const uint8_t *c = r.k + (uint64_t)row * (D / 2);
    ld_k<D>(c, f.k[0]);
    ld_k<D>(c + 8 * (D / 2), f.k[1]);
    f.ks = ld4(r.ks + (uint64_t)row * (D / 16));
}

template <int D>
__device__ __forceinline__ void load_v(const Bases &r, uint32_t row, Frag<D> &f)
{
    const uint8_t *c = r.v + (uint64_t)row * (D / 2);
#pragma unroll
    for (int i = 0; i < 4; ++i)
        ld_v<D>(c + (D / 2) * ((i & 1) + 8 * (i >> 1)), f.v[i]);
    f.vs = ld4(r.vs + (uint64_t)row * (D / 16));
}

// The segment of a unit that tiles are being loaded from.
struct Source {
    int b, kvh, L, lo, P;
    int t_last;        // its last tile here
    int tp, gap;       // tile t sits at position t (t < tp) or t + gap
    uint32_t line;     // dense: vector of slot 0
    bool good;         // the row's content is in order
};

// Vector index of slot s of the source's unit in a paged cache, or -1.
__device__ __noinline__ int paged_row(const int32_t *table, int block_size, int num_blocks, int Hkv, int kvh, int s)
{
    const int blk = __ldg(table + s / block_size);
    if (blk < 0 || blk >= num_blocks)
        return -1;
    return (int)(((uint32_t)blk * Hkv + kvh) * (uint32_t)block_size + (uint32_t)(s % block_size));
}

// Sixteen slots from s0, each vector looked up by itself: any block size, and
// a slot outside the softmax reads slot L instead (it gets weight 0, which
// only a finite value survives). `bad` is set where the block table holds no
// usable block (its output is NaN, whatever is read).
template <int D, bool V, bool PAGED>
__device__ __forceinline__ void load_masked(const DecodeParams &p, const Source &c, const Bases &r, int s0, int lane,
                                            Frag<D> &f, int &bad)
{
    const int g = lane >> 2, t = lane & 3;
    auto row = [&](int j) {
        const int s = attended(c.L, c.lo, c.P, s0 + j) ? s0 + j : c.L;
        if constexpr (PAGED) {
            const int x = paged_row(p.block_table + (long long)c.b * p.max_blocks, p.block_size, p.num_blocks, p.Hkv,
                                    c.kvh, s);
            bad |= x == -1;
            return x == -1 ? 0u : (uint32_t)x;
        } else {
            return c.line + (uint32_t)s;
        }
    };
    // the lane's vectors, from the lane's place in vector 0; then its scales
    if constexpr (V) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            ld_v<D>(r.v - (D / 2) * 2 * t + (uint64_t)row(2 * t + (i & 1) + 8 * (i >> 1)) * (D / 2), f.v[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 2; ++i)
            ld_k<D>(r.k - (D / 2) * g + (uint64_t)row(g + 8 * i) * (D / 2), f.k[i]);
    }
    constexpr int W = D / 64;              // words of a vector's scales
    const int w = lane % (D / 4);
    const uint32_t at = row(w / W);
    if constexpr (V)
        f.vs = ld4(r.vs - 4 * w + 4 * (w % W) + (uint64_t)at * (D / 16));
    else
        f.ks = ld4(r.ks - 4 * w + 4 * (w % W) + (uint64_t)at * (D / 16));
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

__device__ __forceinline__ int scale_head(const DecodeParams &p, int b, int kvh)
{
    return p.scale_heads ? b % p.scale_heads : kvh;
}

// The new token of the source's row into slot L.
template <int D>
__device__ __noinline__ void append_token(const DecodeParams &p, int b, int kvh, int L, int lane)
{
    const long long off = slot_offset(p, b, kvh, L);
    if (off >= 0) {
        const int h = scale_head(p, b, kvh);
        const long long src = ((long long)b * p.Hkv + kvh) * D;
        append_vec<D>(static_cast<const __nv_bfloat16 *>(p.k_new) + src, p.k_cache, p.k_group, off,
                      __ldg(p.k_scale + h), lane);
        append_vec<D>(static_cast<const __nv_bfloat16 *>(p.v_new) + src, p.v_cache, p.v_group, off,
                      __ldg(p.v_scale + h), lane);
        __syncwarp();              // the warp's loads see the whole vector
    }
}

// Where a warp's share of a tile lies.
struct Place {
    int s;                 // first slot
    bool full;             // every slot is in the softmax and the vectors lie as loaded by load_k / load_v
    uint32_t row[kSub];    // full: the parts' first vectors
};

// The unit's query fragments: lane (g, t) holds row g's D / 4 dims from
// D / 4 * t, scaled by a power of two into f16's range; `mul` is the factor
// that takes a product to a base-2 score for row g.
template <int D, bool QF32>
__device__ __forceinline__ void load_query(const DecodeParams &p, int b, int kvh, int lane,
                                           uint32_t (&qh)[D / 16][2], uint32_t (&ql)[QF32 ? D / 16 : 1][2], float &mul)
{
    constexpr int N = D / 4;
    const int g = lane >> 2, t = lane & 3;
    float x[N];
#pragma unroll
    for (int i = 0; i < N; ++i)
        x[i] = 0.f;
    if (g < p.G) {
        const long long at = ((long long)b * p.Hq + (long long)kvh * p.G + g) * D + N * t;
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

// Scores of a part's 16 slots before their scale: s[0], s[1] slot g and query
// rows 2t, 2t + 1; s[2], s[3] slot g + 8.
template <int D, bool QF32>
__device__ __forceinline__ void scores(const Frag<D> &f, int lane, const uint32_t (&qh)[D / 16][2],
                                       const uint32_t (&ql)[QF32 ? D / 16 : 1][2], float (&s)[4])
{
    const int g = lane >> 2, t = lane & 3;
    float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = 0.f;
    // the scales of slots g and g + 8: two groups a lane (D = 64: one)
    constexpr int W = D / 64;              // words of a vector's scales
    const int at = D == 128 ? 2 * g + (t >> 1) : g;
    const int sh = D == 128 ? 16 * (t & 1) : 8 * t;
    const uint32_t ka = __shfl_sync(0xffffffffu, f.ks, at) >> sh;
    const uint32_t kb = __shfl_sync(0xffffffffu, f.ks, at + 8 * W) >> sh;
    const __half2 sa = h2(e4m3x2_f16(ka)), sb = h2(e4m3x2_f16(kb));
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        uint32_t a[4], b[4];           // four pairs of slot g, of slot g + 8
        e2m1x8_f16(f.k[0][w], a);
        e2m1x8_f16(f.k[1][w], b);
        // D = 128: the lane's first two words are one group, the others the next
        const __half2 ma = w >= 2 ? __high2half2(sa) : __low2half2(sa);
        const __half2 mb = w >= 2 ? __high2half2(sb) : __low2half2(sb);
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
__device__ __forceinline__ void weigh(const Frag<D> &f, int lane, const float (&w)[4], float (&o)[D / 16][4])
{
    const int g = lane >> 2, t = lane & 3;
    uint32_t h0, l0, h1, l1;
    split2(w[0], w[1], h0, l0);
    split2(w[2], w[3], h1, l1);
    h0 = movmatrix_t(h0);
    h1 = movmatrix_t(h1);
    l0 = movmatrix_t(l0);
    l1 = movmatrix_t(l1);
    constexpr int W = D / 64;
    const int at = 2 * t * W + (D == 128 ? g >> 2 : 0);
    const int by = D == 128 ? g & 3 : g >> 1;
    const uint32_t w0 = __shfl_sync(0xffffffffu, f.vs, at), w1 = __shfl_sync(0xffffffffu, f.vs, at + W);
    const uint32_t w2 = __shfl_sync(0xffffffffu, f.vs, at + 8 * W), w3 = __shfl_sync(0xffffffffu, f.vs, at + 9 * W);
    const uint32_t sel = by | ((4 + by) << 4);
    const __half2 s01 = h2(e4m3x2_f16(__byte_perm(w0, w1, sel))), s23 = h2(e4m3x2_f16(__byte_perm(w2, w3, sel)));
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        uint32_t x[4][4];
#pragma unroll
        for (int j = 0; j < 4; ++j)
            e2m1x8_f16(f.v[j][i], x[j]);
#pragma unroll
        for (int q = 0; q < 4; ++q) {
            const uint32_t a0 = u32(__hmul2(__lows2half2(h2(x[0][q]), h2(x[1][q])), s01));
            const uint32_t a1 = u32(__hmul2(__highs2half2(h2(x[0][q]), h2(x[1][q])), s01));
            const uint32_t a2 = u32(__hmul2(__lows2half2(h2(x[2][q]), h2(x[3][q])), s23));
            const uint32_t a3 = u32(__hmul2(__highs2half2(h2(x[2][q]), h2(x[3][q])), s23));
            mma_f16(o[4 * i + q], a0, a1, a2, a3, l0, l1);
            mma_f16(o[4 * i + q], a0, a1, a2, a3, h0, h1);
        }
    }
}

// The lane's part of the output state in shared memory: rows 2t, 2t + 1, dims
// D / 8 * g ..
template <int D>
__device__ __forceinline__ float4 *out_at(float (&so)[kRows][D + 4], int lane, int row, int i)
{
    return reinterpret_cast<float4 *>(&so[2 * (lane & 3) + row][D / 8 * (lane >> 2) + 2 * i]);
}

// Adds the accumulators to the state in shared memory (ADD: there is one) and
// clears them; the state is first scaled by r0, r1.
template <int D, bool SCALE>
__device__ __forceinline__ void flush(float (&so)[kRows][D + 4], int lane, float (&o)[D / 16][4], bool add, float r0,
                                      float r1)
{
#pragma unroll
    for (int i = 0; i < D / 16; i += 2) {
        float4 *a = out_at<D>(so, lane, 0, i), *b = out_at<D>(so, lane, 1, i);
        float4 x = make_float4(o[i][0], o[i][2], o[i + 1][0], o[i + 1][2]);
        float4 y = make_float4(o[i][1], o[i][3], o[i + 1][1], o[i + 1][3]);
        if (add) {
            const float4 u = *a, v = *b;
            x = make_float4(x.x + u.x, x.y + u.y, x.z + u.z, x.w + u.w);
            y = make_float4(y.x + v.x, y.y + v.y, y.z + v.z, y.w + v.w);
        }
        if constexpr (SCALE) {
            x = make_float4(x.x * r0, x.y * r0, x.z * r0, x.w * r0);
            y = make_float4(y.x * r1, y.y * r1, y.z * r1, y.w * r1);
        }
        *a = x;
        *b = y;
#pragma unroll
        for (int j = 0; j < 4; ++j)
            o[i][j] = o[i + 1][j] = 0.f;
    }
}

template <int D, bool QF32, bool PAGED>
__global__ void __launch_bounds__(kThreads, 3) q4_decode_kernel(const DecodeParams p)
{
    __shared__ long long sched[kThreads / 32 + 8];
    __shared__ TileWalk walk;
    __shared__ TileCursor sm_cur[kWarps][2];   // the segments being computed and loaded, by parity
    __shared__ int sm_flag;
    __shared__ MergeBuf sm_merge;
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];
    __shared__ __align__(16) float sm_o[kWarps][kRows][D + 4];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t4 = lane & 3;

    // programmatic dependent of the previous kernel: read no input before it is done
    asm volatile("griddepcontrol.wait;" ::: "memory");
    schedule_walk(p, sched, &walk);
    bool in_b = false;
    int par = 0;
    {
        TileCursor c;
        if (!walk_first(p, c, walk, in_b))
            return;
        if (lane == 0)
            sm_cur[warp][0] = c;
        __syncwarp();
    }

    const Bases base = bases<D>(p, lane);
    // whole pages of 16 slots: one vector index a part; else slot by slot
    const int shift = PAGED ? __ffs(p.block_size) - 1 : 0;
    const bool pages = !PAGED || (p.block_size >= 16 && (p.block_size & (p.block_size - 1)) == 0);
    Frag<D> f[kSub] = {};
    Source src = {};
    Place at = {};
    unsigned valid = 0;                        // bits 2 u, 2 u + 1: slots g, g + 8 of part u are in the softmax
    int bad = 0;                               // of the tile loaded
    int t = 0;
    // PAGED: the block of part lane & 1 of the tile (t & ~15) + lane / 2, and of 16 tiles on
    int page = 0, page_next = 0;

    auto load_pages = [&](int tile) {
        const int x = tile + (lane >> 1);
        const int s = (x < src.tp ? x : x + src.gap) * kTile4 + warp * 16 * kSub + 16 * (lane & 1);
        return x <= src.t_last && s <= src.L ? __ldg(p.block_table + (long long)src.b * p.max_blocks + (s >> shift))
                                             : 0;
    };
    // the segment of cursor nxt becomes the source
    auto enter = [&](const TileCursor &nxt) {
        src.b = nxt.b;
        src.kvh = nxt.kvh;
        src.L = nxt.L;
        src.lo = nxt.lo;
        src.P = nxt.P;
        src.tp = nxt.tp;
        src.gap = nxt.gap;
        src.good = row_ok(p, nxt.b, nxt.L);
        t = nxt.t;
        src.t_last = (int)min((long long)nxt.nr - 1, nxt.t + (nxt.end - nxt.g) - 1);
        if constexpr (PAGED) {
            if (src.good && pages) {
                page = load_pages(t & ~15);
                page_next = load_pages((t & ~15) + 16);
            }
        } else if (src.good) {
            const int r = p.slot_ids ? __ldg(p.slot_ids + src.b) : src.b;
            src.line = ((uint32_t)r * p.Hkv + src.kvh) * (uint32_t)p.Smax;
        }
    };
    // finds tile t of the source, appends the new token if it is there
    auto place = [&] {
        at.s = (t < src.tp ? t : t + src.gap) * kTile4 + warp * 16 * kSub;
        const int e = at.s + 16 * kSub - 1;
        at.full = src.good && pages && e <= src.L && (at.s >= src.lo || e < src.P);
        if (!p.attend && src.good && (unsigned)(src.L - at.s) < 16u * kSub)
            append_token<D>(p, src.b, src.kvh, src.L, lane);
        valid = ~0u;
        bad = 0;
        if (at.full) {
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
                if constexpr (PAGED) {
                    int blk = __shfl_sync(0xffffffffu, page, 2 * (t & 15) + u);
                    if (blk < 0 || blk >= p.num_blocks) {
                        bad = 1;
                        blk = 0;           // read something: the unit's output is NaN
                    }
                    at.row[u] = (((uint32_t)blk * p.Hkv + src.kvh) << shift) +
                                ((uint32_t)(at.s + 16 * u) & ((1u << shift) - 1u));
                } else {
                    at.row[u] = src.line + (uint32_t)(at.s + 16 * u);
                }
            }
        } else {
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if (!(src.good && attended(src.L, src.lo, src.P, at.s + 16 * u + 8 * i + g)))
                        valid &= ~(1u << (2 * u + i));
        }
    };
    auto load_keys = [&](int u) {
        if (at.full)
            load_k<D>(base, at.row[u], f[u]);
        else if (src.good)
            load_masked<D, false, PAGED>(p, src, base, at.s + 16 * u, lane, f[u], bad);
    };
    auto load_values = [&](int u) {
        if (at.full)
            load_v<D>(base, at.row[u], f[u]);
        else if (src.good)
            load_masked<D, true, PAGED>(p, src, base, at.s + 16 * u, lane, f[u], bad);
    };

    enter(sm_cur[warp][0]);
    place();
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
        load_keys(u);
        load_values(u);
    }

    uint32_t qh[D / 16][2], ql[QF32 ? D / 16 : 1][2];
    float mul0 = 0.f, mul1 = 0.f;              // product to base-2 score, rows 2t4 and 2t4 + 1
    float m0 = -INFINITY, m1 = -INFINITY, l0 = 0.f, l1 = 0.f;
    float o[D / 16][4];
    int seg_bad = 0;
    bool start = true;
    int flushed = 0, since = 0;                // the state in shared memory, tiles since it was added to
    int first_t = 0;

    for (;;) {
        if (start) {
            first_t = t;
            if (!src.good && tid == 0 && t == 0 && src.kvh == 0)
                report(p, row_error_bits(p, src.b, src.L));
            float mul;
            load_query<D, QF32>(p, src.b, src.kvh, lane, qh, ql, mul);
            const float ks = __ldg(p.k_scale + scale_head(p, src.b, src.kvh));
            mul0 = __shfl_sync(0xffffffffu, mul, 8 * t4) * ks;
            mul1 = __shfl_sync(0xffffffffu, mul, 8 * t4 + 4) * ks;
            m0 = m1 = -INFINITY;
            l0 = l1 = 0.f;
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    o[i][j] = 0.f;
            seg_bad = 0;
            flushed = since = 0;
            start = false;
        }
        float s[kSub][4];
#pragma unroll
        for (int u = 0; u < kSub; ++u)
            scores<D, QF32>(f[u], lane, qh, ql, s[u]);
        seg_bad |= bad;
        const unsigned ok = valid;
        // the next tile: its keys replace these now, its values below
        const bool last = t == src.t_last;
        bool more = true, good = src.good;
        if (!last) {
            ++t;
            if constexpr (PAGED) {
                if ((t & 15) == 0) {
                    page = page_next;
                    page_next = load_pages(t + 16);
                }
            }
        } else {
            TileCursor c = sm_cur[warp][par];
            c.g += t - c.t;
            c.t = t;
            TileCursor n = c;
            more = walk_next(p, n, walk, in_b);
            __syncwarp();
            if (lane == 0) {
                sm_cur[warp][par] = c;
                sm_cur[warp][par ^ 1] = n;
            }
            __syncwarp();
            if (more)
                enter(n);
        }
        if (more) {
            place();
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                load_keys(u);
        }

        // weights: x = base-2 score - reference
        float x[kSub][4];
        float top0 = -INFINITY, top1 = -INFINITY;
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i) {
                x[u][i] = fmaf(s[u][i], i & 1 ? mul1 : mul0, i & 1 ? -m1 : -m0);
                x[u][i] = (ok >> (2 * u + (i >> 1))) & 1u ? x[u][i] : -INFINITY;
            }
            top0 = fmaxf(top0, fmaxf(x[u][0], x[u][2]));
            top1 = fmaxf(top1, fmaxf(x[u][1], x[u][3]));
        }
        if (__any_sync(0xffffffffu, top0 > kRoom || top1 > kRoom)) {
            float c0 = -INFINITY, c1 = -INFINITY;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 2; ++i)
                    if ((ok >> (2 * u + i)) & 1u) {
                        c0 = fmaxf(c0, s[u][2 * i] * mul0);
                        c1 = fmaxf(c1, s[u][2 * i + 1] * mul1);
                    }
#pragma unroll
            for (int q = 4; q < 32; q <<= 1) {
                c0 = fmaxf(c0, __shfl_xor_sync(0xffffffffu, c0, q));
                c1 = fmaxf(c1, __shfl_xor_sync(0xffffffffu, c1, q));
            }
            const float n0 = c0 - m0 > kRoom ? c0 - kLift : m0, n1 = c1 - m1 > kRoom ? c1 - kLift : m1;
            const float r0 = m0 == -INFINITY ? 0.f : fast_ex2(m0 - n0);
            const float r1 = m1 == -INFINITY ? 0.f : fast_ex2(m1 - n1);
            m0 = n0;
            m1 = n1;
            l0 *= r0;
            l1 *= r1;
            flush<D, true>(sm_o[warp], lane, o, flushed, r0, r1);
            flushed = 1;
            since = 0;
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 4; ++i) {
                    x[u][i] = fmaf(s[u][i], i & 1 ? mul1 : mul0, i & 1 ? -m1 : -m0);
                    x[u][i] = (ok >> (2 * u + (i >> 1))) & 1u ? x[u][i] : -INFINITY;
                }
        }
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
#pragma unroll
            for (int i = 0; i < 4; ++i)
                x[u][i] = fast_ex2(x[u][i]);
            l0 += x[u][0] + x[u][2];
            l1 += x[u][1] + x[u][3];
            weigh<D>(f[u], lane, x[u], o);
            if (more)
                load_values(u);
        }
        if (++since == kFlush) {
            flush<D, false>(sm_o[warp], lane, o, flushed, 1.f, 1.f);
            flushed = 1;
            since = 0;
        }
        if (!last)
            continue;

        // the end of the segment
#pragma unroll
        for (int q = 4; q < 32; q <<= 1) {
            l0 += __shfl_xor_sync(0xffffffffu, l0, q);
            l1 += __shfl_xor_sync(0xffffffffu, l1, q);
        }
        // a NaN score raises no reference: keep the NaN sum in the merge
        m0 = (l0 != l0 && m0 == -INFINITY) ? 0.f : m0;
        m1 = (l1 != l1 && m1 == -INFINITY) ? 0.f : m1;
        if (g == 0) {
            sm_m[warp][2 * t4] = m0;
            sm_m[warp][2 * t4 + 1] = m1;
            sm_l[warp][2 * t4] = l0;
            sm_l[warp][2 * t4 + 1] = l1;
        }
        const TileCursor cur = sm_cur[warp][par];
        par ^= 1;
        const float vs = __ldg(p.v_scale + scale_head(p, cur.b, cur.kvh));
        flush<D, true>(sm_o[warp], lane, o, flushed, vs, vs);
        const bool any_bad = __syncthreads_or(seg_bad) != 0;
        if (any_bad && good && tid == 0)
            report(p, kBadBlock);
        finish_segment<kWarps, kRows, D, D + 4, false>(p, cur, walk, first_t, !good || any_bad, sm_m, sm_l, sm_o,
                                                      &sm_flag, sm_merge, tid, kThreads, [] { __syncthreads(); });
        if (!more)
            break;
        start = true;
    }
}

template <int D, bool QF32, bool PAGED>
cudaError_t launch_one(const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    if (!p)
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, q4_decode_kernel<D, QF32, PAGED>, kThreads, 0);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p->grid);
    cfg.blockDim = dim3(kThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q4_decode_kernel<D, QF32, PAGED>, *p);
}

template <int D>
cudaError_t launch_d(bool q_bf16, bool paged, const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    if (q_bf16)
        return paged ? launch_one<D, false, true>(p, st, per_sm) : launch_one<D, false, false>(p, st, per_sm);
    return paged ? launch_one<D, true, true>(p, st, per_sm) : launch_one<D, true, false>(p, st, per_sm);
}

cudaError_t launch(int D, bool q_bf16, bool paged, const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    return D == 128 ? launch_d<128>(q_bf16, paged, p, st, per_sm) : launch_d<64>(q_bf16, paged, p, st, per_sm);
}

}  // namespace

bool q4_supports(int D, int G) { return (D == 64 || D == 128) && G >= 1 && G <= kRows; }

int q4_tile() { return kTile4; }

int q4_ctas_per_sm(int D, bool q_bf16)
{
    int a = 0, b = 0;
    if (launch(D, q_bf16, false, nullptr, nullptr, &a) != cudaSuccess ||
        launch(D, q_bf16, true, nullptr, nullptr, &b) != cudaSuccess)
        return 1;
    const int n = a < b ? a : b;
    return n > 0 ? n : 1;
}

cudaError_t q4_launch(const DecodeParams &p, cudaStream_t st) { return launch(p.D, p.q_bf16, p.paged, &p, st, nullptr); }

}  // namespace gqa
