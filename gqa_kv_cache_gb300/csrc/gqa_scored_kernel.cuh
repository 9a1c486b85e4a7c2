// Attend over an 8-bit cache with a scale for each (block of slots, cache
// head), and attend with capped or distance-biased scores or with the slots'
// weights counted, over that cache or a bfloat16 one (D = 64 or 128, G <= 8).
//
// A base-2 score of slot j and query head h (query position L) is
//   y = log2(e) (cap tanh(s / cap) + slope_h (j - L)),  s = t_j q.c_j / sqrt(D)
// (t_j: the key scale of the slot's block, 1 over a bfloat16 cache; without a
// cap s itself), the output sum_j 2^(y_j - m) u_j v_j / sum_j 2^(y_j - m) with
// the value scales u_j. The schedule, the split of a unit between CTAs and its
// merge are those of the other decode kernels (gqa_common.cuh). A CTA is four
// warps; a tile is 16 kSub slots a warp, copied into a ring of the warp's own in
// shared memory by 16-byte asynchronous copies, with no barrier between warps.
//
//  * S^T = K Q^T (m16n8k16, float32 sums): 16 slots by the query rows. Over an
//    8-bit cache lane (g, t) takes slots g, g + 8 and of each the D / 4
//    contiguous dims from D / 4 * t (the order of the contraction is free);
//    codes become f16 by a byte permute under 0x64 (1024 + 128 + c) and one
//    subtraction, exactly; a bfloat16 query is scaled by a power of two into
//    f16's range (exact but for elements 2^-31 below the row's largest), a
//    float32 one is an f16 and an f16 remainder (22 bits). Over a bfloat16 cache
//    the fragments come by ldmatrix, a float32 query as three bfloat16 (24 bits),
//    the second and third with sums of their own: infinite keys meet the first
//    alone (so it is with values and the weights' parts: with_rest; four long
//    counted rows 241 -> 243 us).
//  * O^T += V^T P^T: 16 dims by the query rows, 16 slots a step, V unrounded.
//    8 bits: lane (g, t) takes D / 8 contiguous dims of slots 2t, 2t + 1, 2t + 8,
//    2t + 9, neighbours paired by a byte permute. P is an f16 and an f16
//    remainder 2^12 times as large with sums of its own (a weight's error: 2^-23
//    of it and 2^-37 - 12 bits of the largest weight). bfloat16: P in three parts.
//  * up to four query rows over an 8-bit cache (FEW): every row has two of the
//    eight columns: in S^T the same query (float32: f16 and remainder), in O^T
//    the weight's two parts: half the matrix products and half the softmax.
//  * value scales: a weight is multiplied by u / ref with ref a power of two of
//    the warp, raised when a scale passes 8 ref, so that products stay within
//    f16's range; the running sum takes the weight before.
//  * the softmax keeps a reference below the running maximum, raised only when
//    a score passes it by kRoom; sums of a tile start from zero and are added to
//    the output in float32 (the matrix unit truncates its sums).
//  * with slopes a segment's tiles go backwards: the largest biased scores stand
//    at the row's end, and forwards steep heads raised their reference at every
//    tile (256 rows of 16 .. 8191 slots, float32 query: 93 -> 86 us).
//  * counted weights: the scores go to a scratch array as they come (float32,
//    without the bias, G padded to 4 or 8 a slot), each row's maximum and
//    denominator at the end of its unit, and a second kernel adds sum_g 2^(y_g -
//    M_g) / den_g to the slot's count. (A second pass over the keys would read D or 2 D bytes a slot
//    instead of 8 G.) The scores ask to stay in L2, the vectors to leave it: four
//    bfloat16 rows of 32768 .. 131071 slots, G = 8, 259 -> 247 us (now 243).
// What bounds it. Over a bfloat16 cache the memory (64 rows of 512 .. 16383 slots
// in 16-slot blocks, G = 6, capped: 329 us, 0.99 of the measured copy rate). Over
// an 8-bit cache of D = 128 nearly so: four rows of 32768 .. 131071 slots, G = 4
// 107 us (0.92), G = 8 110 (0.90; with a cap 124). There a warp issues 785
// instructions for 32 slots (160 byte permutes, 136 f16 sums, 64 sign flips, 48
// products), 0.52 a cycle with two warps a scheduler: dependent instructions
// ("wait" 0.90 of an issue) and little else. D = 64 has the same instructions
// around half the bytes (80 us for half the cache, 0.62). Short units are bound by
// starts and ends: a segment's end costs a CTA about 2.5 us (256 rows of 16 ..
// 8191 slots, 4 heads, G = 8: 78 us, of which the slots would take 56; a float32
// query 82, with slopes 86).
#pragma once

#define GQA_MULTI_TOKEN 0   // single-token steps only
#include <cuda_fp16.h>

#include <atomic>
#include <cfloat>

#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace scored {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kRows = 8;                      // query rows (G <= 8)
constexpr int kFew = 4;                       // and of the form for few
constexpr int kSegs = 4;                      // segments a warp's copies and products are in at once
constexpr float kLift = 10.f;                 // a reference is set this far below the maximum ...
constexpr float kRoom = 12.f;                 // ... and holds until a score is this far above it
constexpr float kNone = -FLT_MAX;             // the first one: a score equals it or is 2^100 above, or is -inf, whose weight is 0
constexpr float kOver = 8.f;                  // value scales reach this times their reference
constexpr float kRest = 4096.f;               // a weight's remainder enters the products this much larger

template <int KIND, int D>
struct Form {
    static constexpr bool I8 = KIND == kI8;
    static constexpr int VB = I8 ? D : 2 * D;             // bytes a vector
    static constexpr int SUB = VB == 256 ? 1 : 2;         // 16-slot parts of a warp's share of a tile
    static constexpr int SHARE = 16 * SUB;                // a warp's slots of a tile
    static constexpr int TILE = kWarps * SHARE;           // slots a tile
    static constexpr int LV = VB / 16;                    // lanes (16-byte pieces) a vector
    static constexpr int VI = 32 / LV;                    // vectors a copy instruction
    static constexpr int NI = 16 / VI;                    // copy instructions a part
};

// Resident CTAs per SM, and tiles of a warp's ring. Measured on four rows of
// 32768 .. 131071 slots: 8 bits, D = 128, G = 8 two CTAs of three tiles 109.9
// us, three of two 114.5 (168 registers are too few); D = 64 three of three 80.0,
// four of three 82.3, two of five 85.2. Three places for query rows are enough
// for the four segments, as a segment's rows are in registers before the copies
// take their place: a fourth left a float32 query of a bfloat16 cache one CTA an
// SM (64 paged rows, capped: 406 us for 331) and one of an 8-bit cache two tiles.
template <int KIND, int D>
constexpr int ctas()
{
    return KIND == kI8 && D == 64 ? 3 : 2;
}
constexpr int kStages = 3;
constexpr int kQueries = kSegs - 1;

// One tile's share of a warp in shared memory: vectors in slot order, their
// 16-byte pieces permuted so that the operand loads below have no bank
// conflicts, and (8 bits) the slots' scales.
template <int KIND, int D>
struct alignas(128) Stage {
    uint8_t k[Form<KIND, D>::SHARE * Form<KIND, D>::VB], v[Form<KIND, D>::SHARE * Form<KIND, D>::VB];
    float ks[KIND == kI8 ? Form<KIND, D>::SHARE : 1], vs[KIND == kI8 ? Form<KIND, D>::SHARE : 1];
};

// Offset of 16-byte piece c of the share's vector r.
template <int VB>
__device__ __forceinline__ int piece(int r, int c)
{
    if constexpr (VB == 64)
        return (r >> 1) * 128 + (((((r & 1) << 2) + c) ^ (2 * ((r >> 1) & 3))) << 4);
    else
        return r * VB + ((c ^ (r & 7)) << 4);
}

__device__ __forceinline__ uint32_t smem_at(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Asynchronous copies to shared memory (DO, SO: byte offsets; HINT: with a
// cache policy), and those of which `n` bytes come from src (all or none of
// them) and the others are zeros.
template <int DO, int SO, bool HINT>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, uint64_t policy)
{
    if constexpr (HINT)
        asm volatile("cp.async.cg.shared.global.L2::cache_hint [%0 + %2], [%1 + %3], 16, %4;" ::"r"(dst), "l"(src), "n"(DO),
                     "n"(SO), "l"(policy)
                     : "memory");
    else
        asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DO), "n"(SO) : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy4(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], 4, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// d += a b, or (first) d = a b: the sum's zeros then take no registers.
template <bool F16>
__device__ __forceinline__ void mma(bool first, float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3, uint32_t b0,
                                    uint32_t b1)
{
    const float c0 = first ? 0.f : d[0], c1 = first ? 0.f : d[1], c2 = first ? 0.f : d[2], c3 = first ? 0.f : d[3];
    if constexpr (F16)
        asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
    else
        asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 {%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, "
            "{%10, %11, %12, %13};"
            : "=f"(d[0]), "=f"(d[1]), "=f"(d[2]), "=f"(d[3])
            : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1), "f"(c0), "f"(c1), "f"(c2), "f"(c3));
}

__device__ __forceinline__ uint32_t movmatrix_t(uint32_t a)
{
    uint32_t d;
    asm("movmatrix.sync.aligned.m8n8.trans.b16 %0, %1;" : "=r"(d) : "r"(a));
    return d;
}

template <bool TRANS>
__device__ __forceinline__ void ldmatrix4(uint32_t (&r)[4], uint32_t at)
{
    if constexpr (TRANS)
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.trans.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
    else
        asm volatile("ldmatrix.sync.aligned.m8n8.x4.shared.b16 {%0, %1, %2, %3}, [%4];"
                     : "=r"(r[0]), "=r"(r[1]), "=r"(r[2]), "=r"(r[3])
                     : "r"(at)
                     : "memory");
}

__device__ __forceinline__ __half2 h2(uint32_t v) { return *reinterpret_cast<__half2 *>(&v); }
__device__ __forceinline__ uint32_t u32(__half2 v) { return *reinterpret_cast<uint32_t *>(&v); }
__device__ __forceinline__ uint32_t u32(__nv_bfloat162 v) { return *reinterpret_cast<uint32_t *>(&v); }

// Bytes SEL of w (codes with the sign bit flipped: c + 128) as an f16 pair: the
// byte under 0x64 is the f16 1024 + 128 + c; exact.
// over: 0x64646464 in a register of its own (magic_bytes).
template <int SEL>
__device__ __forceinline__ uint32_t code_pair(uint32_t w, uint32_t over)
{
    return u32(__hsub2(h2(__byte_perm(w, over, SEL)), h2(0x64806480u)));
}

// 0x64646464 that the compiler cannot see through: as a constant it was moved
// to a register again before most of its 128 uses a tile.
__device__ __forceinline__ uint32_t magic_bytes() { return __shfl_sync(0xffffffffu, 0x64646464u, 0); }

// Two float32 as an f16 pair and the f16 pair of MUL times what it leaves.
__device__ __forceinline__ void split2(float x, float y, float times, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = u32(h);
    lo = u32(__floats2half2_rn((x - f.x) * times, (y - f.y) * times));
}

// Two float32 as three bfloat16 pairs.
__device__ __forceinline__ void split3(float x, float y, uint32_t (&p)[3])
{
#pragma unroll
    for (int i = 0; i < 3; ++i) {
        p[i] = u32(__floats2bfloat162_rn(x, y));
        x -= bf16_lo(p[i]);
        y -= bf16_hi(p[i]);
    }
}

// The unit's query fragments. 8 bits: lane (g, t) holds row g's D / 4 dims from
// D / 4 * t, scaled by a power of two into f16's range, and `mul` is the factor
// that takes a product to a score over `scale`. bfloat16: the fragments of the
// product as they are, PARTS of them. q: the rows in shared memory.
template <int KIND, int D, bool QF32, bool FEW, int PARTS>
__device__ __forceinline__ void load_query(float scale, const void *q, int lane, uint32_t (&qf)[PARTS][D / 16][2], float &mul)
{
    if constexpr (KIND == kI8) {
        constexpr int N = D / 4;
        const int g = FEW ? lane >> 3 : lane >> 2, t = lane & 3;   // query row of column lane / 4
        float x[N];
        if constexpr (QF32) {
            const float4 *s = reinterpret_cast<const float4 *>(static_cast<const float *>(q) + g * D + N * t);
#pragma unroll
            for (int i = 0; i < N / 4; ++i) {
                const float4 v = s[i];
                x[4 * i] = v.x; x[4 * i + 1] = v.y; x[4 * i + 2] = v.z; x[4 * i + 3] = v.w;
            }
        } else {
            const uint4 *s = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(q) + g * D + N * t);
#pragma unroll
            for (int i = 0; i < N / 8; ++i) {
                const uint4 v = s[i];
                const uint32_t w[4] = {v.x, v.y, v.z, v.w};
#pragma unroll
                for (int j = 0; j < 4; ++j) {
                    x[8 * i + 2 * j] = bf16_lo(w[j]);
                    x[8 * i + 2 * j + 1] = bf16_hi(w[j]);
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
        mul = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * scale;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const float a = x[4 * i + 2 * j] * up, b = x[4 * i + 2 * j + 1] * up;
                if constexpr (QF32 && FEW) {
                    // the row's first column takes the f16, its second the remainder
                    uint32_t h, l;
                    split2(a, b, 1.f, h, l);
                    qf[0][i][j] = lane & 4 ? l : h;
                } else if constexpr (QF32) {
                    split2(a, b, 1.f, qf[0][i][j], qf[PARTS - 1][i][j]);
                } else {
                    qf[0][i][j] = u32(__floats2half2_rn(a, b));
                }
            }
    } else {
        const int g = lane >> 2, t = lane & 3;
        mul = scale;
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const int d = g * D + 16 * i + 8 * j + 2 * t;
                if constexpr (QF32) {
                    const float2 v = *reinterpret_cast<const float2 *>(static_cast<const float *>(q) + d);
                    uint32_t part[3];
                    split3(v.x, v.y, part);
#pragma unroll
                    for (int k = 0; k < PARTS; ++k)
                        qf[k][i][j] = part[k];
                } else {
                    qf[0][i][j] = *reinterpret_cast<const uint32_t *>(static_cast<const __nv_bfloat16 *>(q) + d);
                }
            }
    }
}

// A segment of a unit: consecutive tiles that this CTA computes. Kept in a
// small ring in shared memory: the copies run ahead of the products.
struct Segment {
    TileCursor c;      // at its first tile
    int t_last;        // its last tile
    int good;          // the row's content is in order
};

template <int D, bool QF32, bool FEW>
constexpr int query_bytes()
{
    return (FEW ? kFew : kRows) * D * (QF32 ? 4 : 2);
}

// What a warp's copies are taken from.
struct Fetch {
    int t, t_last;     // (the rest of its segment is read from shared memory)
    int turn;          // tiles backwards (see kernel): the sum of a tile's place and its number, else -1
    bool good;
    uint32_t line;     // dense: vector of slot 0
    uint32_t block0;   // dense, 8 bits: block of slot 0
    uint64_t policy;   // cache policy of the vectors
    // paged, whole pages of 16 slots: the block of part lane % SUB of a tile, 32 /
    // SUB tiles, and of the tiles behind them; else the block of slot lane of tile t
    int page, page_next;
};

template <class F>
__device__ __forceinline__ int share_slot(int t, int tp, int gap, int warp)
{
    return (t < tp ? t : t + gap) * F::TILE + warp * F::SHARE;
}

// The number of the segment's tile at place t.
__device__ __forceinline__ int tile_at(int turn, int t) { return turn < 0 ? t : turn - t; }

// lane's page of the 32 / SUB tiles from `tile`
template <class F>
__device__ __forceinline__ int load_page(const ScoredParams &p, const Fetch &f, const TileCursor &c, int shift, int tile,
                                         int warp, int lane)
{
    const int x = tile + lane / F::SUB;
    const int s = share_slot<F>(x, c.tp, c.gap, warp) + 16 * (lane % F::SUB);
    return x >= 0 && x <= f.t_last && s <= c.L ? __ldg(p.block_table + (long long)c.b * p.max_blocks + (s >> shift)) : 0;
}

// the block of the lane's slot of tile f.t
template <class F>
__device__ __forceinline__ int load_slot_page(const ScoredParams &p, const Fetch &f, const TileCursor &c, int warp, int lane)
{
    const int s = share_slot<F>(tile_at(f.turn, f.t), c.tp, c.gap, warp) + lane % F::SHARE;
    return s <= c.L ? __ldg(p.block_table + (long long)c.b * p.max_blocks + s / p.block_size) : 0;
}

// The copies' segment becomes that of cursor c. The segment's query rows (rows
// behind the G are zeros) are copied too, a part by each warp, in the group of
// the copies that comes next.
template <class F, int D, bool QF32, bool PAGED, bool FEW, bool BACK>
__device__ __forceinline__ void enter(const ScoredParams &p, const TileCursor &c, Fetch &f, Segment *seg, int *bad, void *q,
                                      int shift, bool pages, int warp, int lane)
{
    constexpr int B = QF32 ? 4 : 2;                // bytes an element
    constexpr int C = D * B / 16;                  // 16-byte pieces a row
    constexpr int R = FEW ? kFew : kRows;
    constexpr int PER = 32 / F::SUB;
    const char *src = static_cast<const char *>(p.q) + ((long long)c.b * p.Hq + (long long)c.kvh * p.G) * D * B;
#pragma unroll
    for (int i = 0; i < (R * C + kThreads - 1) / kThreads; ++i) {
        const int x = i * kThreads + warp * 32 + lane;
        if (R * C % kThreads == 0 || x < R * C)
            copy16(smem_at(q) + x * 16, x / C < p.G ? src + x * 16 : src, x / C < p.G ? 16 : 0);
    }
    f.t = c.t;
    f.t_last = (int)min((long long)c.nr - 1, c.t + (c.end - c.g) - 1);
    f.turn = BACK && p.slopes ? f.t + f.t_last : -1;
    f.good = row_ok(p, c.b, c.L);
    if constexpr (PAGED) {
        if (f.good && pages) {
            const int group = tile_at(f.turn, f.t) & ~(PER - 1);
            f.page = load_page<F>(p, f, c, shift, group, warp, lane);
            f.page_next = load_page<F>(p, f, c, shift, f.turn < 0 ? group + PER : group - PER, warp, lane);
        } else if (f.good) {
            f.page = load_slot_page<F>(p, f, c, warp, lane);
        }
    } else if (f.good) {
        const int r = p.slot_ids ? __ldg(p.slot_ids + c.b) : c.b;
        f.line = ((uint32_t)r * p.Hkv + c.kvh) * (uint32_t)p.Smax;
        if constexpr (F::I8)
            f.block0 = ((uint32_t)r * p.Hkv + c.kvh) * (uint32_t)(p.Smax / p.scale_block);
    }
    if (lane == 0) {
        seg->c = c;
        seg->t_last = f.t_last;
        seg->good = f.good;
        *bad = 0;
    }
}

// The copies of part U's vectors, which follow each other: instruction j takes
// vectors VI j + lane / LV, whose pieces are permuted as those of vector lane /
// LV but for bits of the piece's number that VI j brings (constants here; the
// stage lies on 128 bytes).
template <class F, int U, bool MORE, int J = 0>
__device__ __forceinline__ void copy_part(uint32_t dk, uint32_t dv, const uint8_t *k, const uint8_t *v, uint64_t policy)
{
    constexpr int FLIP = F::VB == 64 ? 0 : ((F::VI * J) & 7) << 4;
    constexpr int DO = (16 * U + F::VI * J) * F::VB, SO = F::VI * J * F::VB;
    copy16<DO, SO, MORE>(dk ^ FLIP, k, policy);
    copy16<DO, SO, MORE>(dv ^ FLIP, v, policy);
    if constexpr (J + 1 < F::NI)
        copy_part<F, U, MORE, J + 1>(dk, dv, k, v, policy);
}

// Starts the copies of the warp's share of tile f.t.
template <int KIND, int D, bool PAGED, bool MORE>
__device__ __forceinline__ void fetch_tile(const ScoredParams &p, const Fetch &f, const TileCursor &c, Stage<KIND, D> &st,
                                           int *bad, int shift, bool pages, int warp, int lane)
{
    using F = Form<KIND, D>;
    if (!f.good)
        return;                            // its output is NaN, whatever is in the stage
    const int tile = tile_at(f.turn, f.t), s = share_slot<F>(tile, c.tp, c.gap, warp);
    const uint32_t dk = smem_at(st.k), dv = smem_at(st.v);
    [[maybe_unused]] const uint32_t dks = smem_at(st.ks), dvs = smem_at(st.vs);
    const uint8_t *kc = static_cast<const uint8_t *>(p.k_cache), *vc = static_cast<const uint8_t *>(p.v_cache);
    const int e = s + F::SHARE - 1;
    const int r0 = lane / F::LV, c0 = lane % F::LV;
    if (pages && e <= c.L && (s >= c.lo || e < c.P)) {
        // every slot is in the softmax, 16 vectors in a row at least
        const uint32_t to = (uint32_t)piece<F::VB>(r0, c0);
#pragma unroll
        for (int u = 0; u < F::SUB; ++u) {
            uint32_t row;
            [[maybe_unused]] uint32_t block = 0;
            if constexpr (PAGED) {
                int blk = __shfl_sync(0xffffffffu, f.page, F::SUB * (tile & (32 / F::SUB - 1)) + u);
                if (blk < 0 || blk >= p.num_blocks) {
                    *bad = 1;
                    blk = 0;               // read something: the unit's output is NaN
                }
                block = (uint32_t)blk * p.Hkv + c.kvh;
                row = (block << shift) + ((uint32_t)(s + 16 * u) & ((1u << shift) - 1u));
            } else {
                row = f.line + (uint32_t)(s + 16 * u);
            }
            const uint64_t in = (uint64_t)row * F::VB + lane * 16;
            if (u == 0)
                copy_part<F, 0, MORE>(dk + to, dv + to, kc + in, vc + in, f.policy);
            else
                copy_part<F, F::SUB - 1, MORE>(dk + to, dv + to, kc + in, vc + in, f.policy);
            if constexpr (F::I8) {
                // lanes 0 .. 15 the key scales of the part's slots, 16 .. 31 the value scales
                const int i = 16 * u + (lane & 15);
                if constexpr (!PAGED)
                    block = f.block0 + ((uint32_t)(s + i) >> p.scale_shift);
                copy4((lane < 16 ? dks : dvs) + 4 * i, (lane < 16 ? p.k_block_scale : p.v_block_scale) + block, 4);
            }
        }
        return;
    }
    // any block size, and slots outside the softmax, which become zeros: a lane
    // finds the vector of one slot, the copies take it from there
    const int x = s + lane % F::SHARE;
    uint32_t row = ~0u;
    [[maybe_unused]] uint32_t block = 0;
    if (attended(c.L, c.lo, c.P, x)) {
        if constexpr (PAGED) {
            const int blk = pages ? __ldg(p.block_table + (long long)c.b * p.max_blocks + (x >> shift)) : f.page;
            if (blk < 0 || blk >= p.num_blocks) {
                *bad = 1;
            } else {
                block = (uint32_t)blk * p.Hkv + c.kvh;
                row = block * (uint32_t)p.block_size + (uint32_t)x % (uint32_t)p.block_size;
            }
        } else {
            row = f.line + (uint32_t)x;
            if constexpr (F::I8)
                block = f.block0 + (uint32_t)x / (uint32_t)p.scale_block;
        }
    }
#pragma unroll
    for (int j = 0; j < F::SHARE / F::VI; ++j) {
        const int r = F::VI * j + r0;
        const uint32_t v = __shfl_sync(0xffffffffu, row, r);
        const uint64_t at = v == ~0u ? 0 : (uint64_t)v * F::VB + c0 * 16;
        copy16(dk + piece<F::VB>(r, c0), kc + at, v == ~0u ? 0 : 16);
        copy16(dv + piece<F::VB>(r, c0), vc + at, v == ~0u ? 0 : 16);
    }
    if constexpr (F::I8) {                 // SHARE = 32 slots
        const int n = row == ~0u ? 0 : 4;
        copy4(dks + 4 * lane, p.k_block_scale + block, n);
        copy4(dvs + 4 * lane, p.v_block_scale + block, n);
    }
}

// The product of a number's first part and that of its remainders, together.
// Where an operand is infinite the first is the whole product: a remainder's
// would be the other infinity, or 0 times infinity.
__device__ __forceinline__ float with_rest(float first, float rest)
{
    return fabsf(first) <= FLT_MAX ? first + rest : first;
}

// Products of part u: s[0], s[1] slot g and query rows 2t, 2t + 1 (FEW: both
// row t); s[2], s[3] slot g + 8. 8 bits: times the slot's key scale.
template <int KIND, int D, bool QF32, bool FEW, int PARTS>
__device__ __forceinline__ void scores(const Stage<KIND, D> &st, int u, int lane, const uint32_t (&qf)[PARTS][D / 16][2],
                                       float (&s)[4], [[maybe_unused]] uint32_t over)
{
    using F = Form<KIND, D>;
    const int g = lane >> 2, t = lane & 3;
    float s2[4];
    if constexpr (KIND == kI8) {
        uint32_t k[2][D / 16];
#pragma unroll
        for (int i = 0; i < 2; ++i)
#pragma unroll
            for (int j = 0; j < D / 64; ++j) {
                const uint4 w = *reinterpret_cast<const uint4 *>(st.k + piece<F::VB>(16 * u + g + 8 * i, D / 64 * t + j));
                k[i][4 * j] = w.x; k[i][4 * j + 1] = w.y; k[i][4 * j + 2] = w.z; k[i][4 * j + 3] = w.w;
            }
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
            const uint32_t x = k[0][w] ^ 0x80808080u, y = k[1][w] ^ 0x80808080u;
            const uint32_t a0 = code_pair<0x4140>(x, over), a1 = code_pair<0x4140>(y, over);
            const uint32_t a2 = code_pair<0x4342>(x, over), a3 = code_pair<0x4342>(y, over);
            float(&d)[4] = w & 1 ? s2 : s;
            mma<true>(w < 2, d, a0, a1, a2, a3, qf[0][w][0], qf[0][w][1]);
            if constexpr (PARTS == 2)
                mma<true>(false, d, a0, a1, a2, a3, qf[1][w][0], qf[1][w][1]);
        }
    } else {
#pragma unroll
        for (int w = 0; w < D / 16; ++w) {
            uint32_t a[4];
            ldmatrix4<false>(a, smem_at(st.k) + piece<F::VB>(16 * u + (lane & 15), 2 * w + (lane >> 4)));
            if constexpr (PARTS == 1) {
                float(&d)[4] = w & 1 ? s2 : s;
                mma<false>(w < 2, d, a[0], a[1], a[2], a[3], qf[0][w][0], qf[0][w][1]);
            } else {
                // the remainders' products on their own
                mma<false>(w == 0, s, a[0], a[1], a[2], a[3], qf[0][w][0], qf[0][w][1]);
#pragma unroll
                for (int k = 1; k < PARTS; ++k)
                    mma<false>(w == 0 && k == 1, s2, a[0], a[1], a[2], a[3], qf[k][w][0], qf[k][w][1]);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = KIND != kI8 && PARTS > 1 ? with_rest(s[i], s2[i]) : s[i] + s2[i];
    if constexpr (KIND == kI8) {
        if constexpr (QF32 && FEW) {
            s[0] += s[1];
            s[2] += s[3];
        }
        const float a = st.ks[16 * u + g], b = st.ks[16 * u + g + 8];
        s[0] *= a;
        s[2] *= b;
        if constexpr (!FEW) {
            s[1] *= a;
            s[3] *= b;
        }
    }
}

// O^T += V^T P^T over a warp's slots of a tile; w[u] are the weights in the
// positions of the scores. The products of a tile are summed from zero and then
// added to o (the matrix unit truncates its sums). Where o's elements lie:
// out_dim.
template <int KIND, int D, bool FEW>
__device__ __forceinline__ void weigh(const Stage<KIND, D> &st, int lane, const float (&w)[Form<KIND, D>::SUB][FEW ? 2 : 4],
                                      float (&o)[D / 16][FEW ? 2 : 4], [[maybe_unused]] uint32_t over)
{
    using F = Form<KIND, D>;
    constexpr int SUB = F::SUB;
    const int g = lane >> 2, t = lane & 3;
    if constexpr (KIND == kI8) {
        // FEW: a row's two columns take the weight's f16 and its remainder
        uint32_t bh[SUB][2], bl[FEW ? 1 : SUB][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                if constexpr (FEW) {
                    const __half h = __float2half_rn(w[u][i]);
                    bh[u][i] = movmatrix_t(u32(__halves2half2(h, __float2half_rn((w[u][i] - __half2float(h)) * kRest))));
                } else {
                    uint32_t h, l;
                    split2(w[u][2 * i], w[u][2 * i + 1], kRest, h, l);
                    bh[u][i] = movmatrix_t(h);
                    bl[u][i] = movmatrix_t(l);
                }
            }
        constexpr int W = D / 32;          // words of a slot's share: dims D / 8 * g + 4 i
        uint32_t v[SUB][4][W];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const int r = 16 * u + 2 * t + (j & 1) + 8 * (j >> 1);
                if constexpr (D == 128) {
                    const uint4 x = *reinterpret_cast<const uint4 *>(st.v + piece<F::VB>(r, g));
                    v[u][j][0] = x.x; v[u][j][1] = x.y; v[u][j][2] = x.z; v[u][j][3] = x.w;
                } else {
                    const uint2 x = *reinterpret_cast<const uint2 *>(st.v + piece<F::VB>(r, g >> 1) + 8 * (g & 1));
                    v[u][j][0] = x.x; v[u][j][1] = x.y;
                }
            }
#pragma unroll
        for (int i = 0; i < W; ++i) {
            float d[2][4];
            [[maybe_unused]] float r[FEW ? 1 : 2][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                // bytes: dims 4 i, 4 i + 1 (then + 2, + 3) of two neighbouring slots
                const uint32_t x0 = v[u][0][i] ^ 0x80808080u, x1 = v[u][1][i] ^ 0x80808080u;
                const uint32_t x2 = v[u][2][i] ^ 0x80808080u, x3 = v[u][3][i] ^ 0x80808080u;
#pragma unroll
                for (int q = 0; q < 2; ++q) {
                    const uint32_t a = __byte_perm(x0, x1, q ? 0x7362 : 0x5140), b = __byte_perm(x2, x3, q ? 0x7362 : 0x5140);
                    const uint32_t a0 = code_pair<0x4140>(a, over), a1 = code_pair<0x4342>(a, over);
                    const uint32_t a2 = code_pair<0x4140>(b, over), a3 = code_pair<0x4342>(b, over);
                    mma<true>(u == 0, d[q], a0, a1, a2, a3, bh[u][0], bh[u][1]);
                    if constexpr (!FEW)
                        mma<true>(u == 0, r[q], a0, a1, a2, a3, bl[u][0], bl[u][1]);
                }
            }
#pragma unroll
            for (int q = 0; q < 2; ++q) {
                float(&y)[FEW ? 2 : 4] = o[2 * i + q];
                if constexpr (FEW) {
                    y[0] += fmaf(d[q][1], 1.f / kRest, d[q][0]);
                    y[1] += fmaf(d[q][3], 1.f / kRest, d[q][2]);
                } else {
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        y[j] += fmaf(r[q][j], 1.f / kRest, d[q][j]);
                }
            }
        }
    } else {
        uint32_t b[SUB][3][2];
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                uint32_t part[3];
                split3(w[u][2 * i], w[u][2 * i + 1], part);
#pragma unroll
                for (int k = 0; k < 3; ++k)
                    b[u][k][i] = movmatrix_t(part[k]);
            }
#pragma unroll
        for (int i = 0; i < D / 16; ++i) {
            float d[4], r[4];
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
                uint32_t a[4];
                ldmatrix4<true>(a, smem_at(st.v) + piece<F::VB>(16 * u + (lane & 7) + 8 * (lane >> 4), 2 * i + ((lane >> 3) & 1)));
                mma<false>(u == 0, d, a[0], a[1], a[2], a[3], b[u][0][0], b[u][0][1]);
                mma<false>(u == 0, r, a[0], a[1], a[2], a[3], b[u][1][0], b[u][1][1]);
                mma<false>(false, r, a[0], a[1], a[2], a[3], b[u][2][0], b[u][2][1]);
            }
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[i][j] += with_rest(d[j], r[j]);
        }
    }
}

// s -> cap tanh(s) of the lane's scores (s over the cap, cap in base-2 units).
// While every score of the warp is within the cap tanh is Lambert's continued
// fraction cut at the 7th partial quotient (off by 2.2e-12 of it at 1, less
// below), in all four steps of 2^-24, in tanhf's place, which takes
// about three times as long.
template <int SUB, int C>
__device__ __forceinline__ void cap_scores(float (&s)[SUB][4], float cap)
{
    float top = 0.f;
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 2 * C; ++i)
            top = fmaxf(top, fabsf(s[u][i / C * 2 + i % C]));
    if (__any_sync(0xffffffffu, top > 1.f)) {
#pragma unroll
        for (int u = 0; u < SUB; ++u)
#pragma unroll
            for (int i = 0; i < 2 * C; ++i) {
                float &y = s[u][i / C * 2 + i % C];
                y = tanhf(y) * cap;
            }
        return;
    }
#pragma unroll
    for (int u = 0; u < SUB; ++u)
#pragma unroll
        for (int i = 0; i < 2 * C; ++i) {
            float &y = s[u][i / C * 2 + i % C];
            const float z = y * y;
            // z (378 + z) .. over 135135: both sides of the fraction divided by it
            const float num = fmaf(fmaf(fmaf(z, 1.f / 135135.f, 378.f / 135135.f), z, 17325.f / 135135.f), z, 1.f);
            const float den = fmaf(fmaf(fmaf(z, 28.f / 135135.f, 3150.f / 135135.f), z, 62370.f / 135135.f), z, 1.f);
            y = __fdividef(y * cap * num, den);
        }
}

// A lane's scores of a slot into the array of counted scores (C = 1: the first),
// to stay in L2 until they are read.
template <int C>
__device__ __forceinline__ void store_scores(float *to, float x, float y, uint64_t keep)
{
    if constexpr (C == 1)
        asm volatile("st.global.L2::cache_hint.f32 [%0], %1, %2;" ::"l"(to), "f"(x), "l"(keep) : "memory");
    else
        asm volatile("st.global.L2::cache_hint.v2.f32 [%0], {%1, %2}, %3;" ::"l"(to), "f"(x), "f"(y), "l"(keep) : "memory");
}

// Scratch of the merge (segment_out, unit_ticket_merge): as many partials at a
// time as the spare slot has room for.
template <int KIND, int D>
using Merge = MergeBufT<kRows, D == 128 ? 28 : 12>;

template <int KIND, int D, bool QF32, bool PAGED, bool FEW, bool MORE>
__global__ void __launch_bounds__(kThreads, ctas<KIND, D>()) scored_kernel(const ScoredParams p)
{
    using F = Form<KIND, D>;
    using St = Stage<KIND, D>;
    constexpr bool I8 = F::I8;
    constexpr int SUB = F::SUB, STAGES = kStages, SHARE = F::SHARE;
    constexpr int C = FEW ? 1 : 2;             // query rows of a lane: t4, or 2t4 and 2t4 + 1
    constexpr int PARTS = !QF32 ? 1 : !I8 ? 3 : FEW ? 1 : 2;
    extern __shared__ __align__(128) unsigned char dyn[];
    St(*ring)[kWarps] = reinterpret_cast<St(*)[kWarps]>(dyn);      // [STAGES]
    auto sm_q = reinterpret_cast<uint8_t(*)[query_bytes<D, QF32, FEW>()]>(dyn + STAGES * kWarps * sizeof(St));   // [kQueries]
    __shared__ long long sched[kThreads / 32 + 8];
    __shared__ TileWalk walk;
    __shared__ Segment segs[kSegs];            // every warp writes the same
    __shared__ int sm_bad[kWarps][kSegs];      // a block that the segment needs is not usable
    __shared__ int sm_flag;
    __shared__ float sm_m[kWarps][kRows], sm_l[kWarps][kRows];

    const int tid = threadIdx.x, warp = tid / 32, lane = tid % 32;
    const int g = lane >> 2, t4 = lane & 3;

    // the next kernel may be set up meanwhile (it waits for this one's end);
    // programmatic dependent of the previous kernel: read no input before it is done
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (!p.whole_units)
        schedule_walk(p, sched, &walk);
    // whole pages of 16 slots: one vector index a part; else slot by slot (a
    // dense 8-bit cache: where a block of scales is not a power of two)
    const int shift = PAGED ? __ffs(p.block_size) - 1 : 0;
    const bool pages = PAGED ? p.block_size >= 16 && (p.block_size & (p.block_size - 1)) == 0 : !I8 || p.scale_shift >= 0;

    // the copies: tile f.t of segment sf is the next to fetch
    Fetch f = {};
    if constexpr (MORE) {
        if (p.xs)                          // the vectors leave the L2 to the scores
            asm("createpolicy.fractional.L2::evict_first.b64 %0, 1.0;" : "=l"(f.policy));
        else
            asm("createpolicy.fractional.L2::evict_normal.b64 %0, 1.0;" : "=l"(f.policy));
    }
    int sf = 0, qf_at = 0;                 // and its query rows' place
    bool in_b = false, left;
    {
        TileCursor c;
        if (p.whole_units) {
            // this CTA's tiles are those of its unit, one segment
            c = cursor_at(p, blockIdx.x / p.Hkv, 0, 0, 0);
            c.kvh = blockIdx.x % p.Hkv;
            c.end = c.nr;
            left = true;
        } else {
            left = walk_first(p, c, walk, in_b);
            if (!left)
                return;
        }
        enter<F, D, QF32, PAGED, FEW, MORE>(p, c, f, &segs[0], &sm_bad[warp][0], sm_q[0], shift, pages, warp, lane);
        __syncwarp();
    }
    auto fetch = [&](int slot) {
        if (left) {
            fetch_tile<KIND, D, PAGED, MORE>(p, f, segs[sf].c, ring[slot][warp], &sm_bad[warp][sf], shift, pages, warp, lane);
            if (f.t < f.t_last) {
                ++f.t;
                if constexpr (PAGED) {
                    constexpr int PER = 32 / SUB;
                    const int tile = tile_at(f.turn, f.t);
                    if (f.good && !pages) {
                        f.page = load_slot_page<F>(p, f, segs[sf].c, warp, lane);
                    } else if ((tile & (PER - 1)) == (f.turn < 0 ? 0 : PER - 1) && f.good) {
                        f.page = f.page_next;
                        f.page_next = load_page<F>(p, f, segs[sf].c, shift, f.turn < 0 ? tile + PER : tile - 2 * PER + 1, warp, lane);
                    }
                }
            } else {
                TileCursor c = segs[sf].c;
                c.g += f.t - c.t;
                c.t = f.t;
                left = !p.whole_units && walk_next(p, c, walk, in_b);
                if (left) {
                    sf = (sf + 1) % kSegs;
                    qf_at = qf_at == kQueries - 1 ? 0 : qf_at + 1;
                    enter<F, D, QF32, PAGED, FEW, MORE>(p, c, f, &segs[sf], &sm_bad[warp][sf], sm_q[qf_at], shift, pages, warp, lane);
                    __syncwarp();
                }
            }
        }
        copy_commit();                     // an empty group behind the last tile
    };
    int slot = 0;                          // ring slot of the tile to compute
#pragma unroll
    for (int i = 0; i < STAGES - 1; ++i)
        fetch(i);

    const uint32_t over = I8 ? magic_bytes() : 0u;
    // the first segment's query rows, every warp's part (those of a later one
    // came with the last tile of the segment before it, whose end the warps
    // meet at)
    copy_wait<STAGES - 2>();
    __syncthreads();
    [[maybe_unused]] uint64_t keep;        // cache policy of the counted scores
    if constexpr (MORE)
        asm("createpolicy.fractional.L2::evict_last.b64 %0, 1.0;" : "=l"(keep));
    uint32_t qf[PARTS][D / 16][2];
    // product to (base-2) score, base-2 bias a slot. MORE: scores that are capped,
    // biased or counted are formed in place
    float mul[C];
    [[maybe_unused]] float slope[C];
    float m[C], l[C];                      // reference and sum of the lane's rows
    float o[D / 16][FEW ? 2 : 4];
    for (int sc = 0, q_at = 0;; sc = (sc + 1) % kSegs, q_at = q_at == kQueries - 1 ? 0 : q_at + 1) {
        // the next segment
        const Segment *seg = &segs[sc];
        const bool good = seg->good;
        if (!good && tid == 0 && seg->c.t == 0 && seg->c.kvh == 0)
            report(p, row_error_bits(p, seg->c.b, seg->c.L));
        float mine;
        load_query<KIND, D, QF32, FEW, PARTS>(MORE && p.cap > 0.f ? p.scale_cap : p.scale_log2, sm_q[q_at], lane, qf, mine);
        __syncthreads();                   // the copies that run ahead may take the rows' place
#pragma unroll
        for (int c = 0; c < C; ++c) {
            [[maybe_unused]] const int row = C * t4 + c;
            mul[c] = I8 ? __shfl_sync(0xffffffffu, mine, 8 * t4 + 4 * c) : mine;
            if constexpr (MORE)
                slope[c] = p.slopes && row < p.G ? __ldg(p.slopes + seg->c.kvh * p.G + row) * 1.4426950408889634f : 0.f;
            m[c] = kNone;
            l[c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / 16; ++i)
#pragma unroll
            for (int j = 0; j < (FEW ? 2 : 4); ++j)
                o[i][j] = 0.f;
        [[maybe_unused]] float vref = 0.f;     // 8 bits: 1 / the reference of the value scales (0: none yet)

        int arrived = -1;                  // thread 0: the unit's arrival count before the last tile
        for (int t = seg->c.t; t <= seg->t_last; ++t) {
            if (t == seg->t_last && tid == 0 && (seg->c.t != 0 || t != seg->c.nr - 1))
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];"
                             : "=r"(arrived)
                             : "l"(p.ws_cnt + seg->c.b * p.Hkv + seg->c.kvh)
                             : "memory");
            copy_wait<STAGES - 2>();       // this lane's copies of the tile, then the other lanes'
            __syncwarp();
            fetch(slot == 0 ? STAGES - 1 : slot - 1);
            const St &st = ring[slot][warp];
            slot = slot + 1 == STAGES ? 0 : slot + 1;
            float s[SUB][4];
#pragma unroll
            for (int u = 0; u < SUB; ++u)
                scores<KIND, D, QF32, FEW, PARTS>(st, u, lane, qf, s[u], over);
            // bits 2 u + i: slot 16 u + g + 8 i is in the softmax
            unsigned ok = good ? ~0u : 0u;
            const int tile = tile_at(MORE && p.slopes ? seg->c.t + seg->t_last : -1, t);
            const int s0 = share_slot<F>(tile, seg->c.tp, seg->c.gap, warp), L = seg->c.L, lo = seg->c.lo, P = seg->c.P;
            if (s0 + SHARE - 1 > L || (s0 < lo && s0 + SHARE - 1 >= P)) {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!attended(L, lo, P, s0 + 16 * u + g + 8 * i))
                            ok &= ~(1u << (2 * u + i));
            }
            if constexpr (MORE) {
                // base-2 scores (but for the bias) in place
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2 * C; ++i)
                        s[u][i / C * 2 + i % C] *= mul[i % C];
                if (p.cap > 0.f)
                    cap_scores<SUB, C>(s, p.cap);
                if (p.xs && C * t4 < p.gp) {
                    float *to = p.xs + (((unsigned long long)seg->c.b * p.Hkv + seg->c.kvh) * p.xs_cap + s0 + g) * p.gp + C * t4;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if ((ok >> (2 * u + i)) & 1u)
                                store_scores<C>(to + (16 * u + 8 * i) * p.gp, s[u][2 * i], s[u][2 * i + 1], keep);
                }
            }
            // distance of slots u, i from the query
            [[maybe_unused]] const float far0 = (float)(s0 + g - L);
            [[maybe_unused]] auto far = [&](int u, int i) { return far0 + (float)(16 * u + 8 * i); };
            // x = base-2 score - reference, of slots u, i and rows c. A bias and the
            // reference may be large and near each other (a negative slope's, in a long
            // row): they meet in one rounding, before the score
            float x[SUB][2 * C], top = -INFINITY;
            auto shifted = [&] {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2 * C; ++i)
                        x[u][i] = MORE ? s[u][i / C * 2 + i % C] - m[i % C] : fmaf(s[u][i / C * 2 + i % C], mul[i % C], -m[i % C]);
                if (MORE && p.slopes)
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2 * C; ++i)
                            x[u][i] = s[u][i / C * 2 + i % C] + fmaf(slope[i % C], far(u, i / C), -m[i % C]);
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2 * C; ++i)
                        x[u][i] = (ok >> (2 * u + i / C)) & 1u ? x[u][i] : -INFINITY;
            };
            shifted();
#pragma unroll
            for (int u = 0; u < SUB; ++u)
#pragma unroll
                for (int i = 0; i < 2 * C; ++i)
                    top = fmaxf(top, x[u][i]);
            bool raise = top > kRoom;
            [[maybe_unused]] float vs[SUB][2];
            if constexpr (I8) {
#pragma unroll
                for (int u = 0; u < SUB; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i) {
                        vs[u][i] = st.vs[16 * u + g + 8 * i];
                        raise |= vs[u][i] * vref > kOver;
                    }
            }
            if (__any_sync(0xffffffffu, raise)) {
                float r[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float most = -INFINITY;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if ((ok >> (2 * u + i)) & 1u)
                                most = fmaxf(most, MORE ? fmaf(slope[c], far(u, i), s[u][2 * i + c]) : s[u][2 * i + c] * mul[c]);
#pragma unroll
                    for (int q = 4; q < 32; q <<= 1)
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, q));
                    const float n = most - m[c] > kRoom ? most - kLift : m[c];
                    r[c] = fast_ex2(m[c] - n);
                    m[c] = n;
                    l[c] *= r[c];
                }
                if constexpr (I8) {
                    float most = 0.f;
#pragma unroll
                    for (int u = 0; u < SUB; ++u)
                        most = fmaxf(most, fmaxf(vs[u][0], vs[u][1]));
#pragma unroll
                    for (int q = 4; q < 32; q <<= 1)
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, q));
                    if (vref == 0.f || most * vref > kOver) {
                        // the power of two above the largest scale, within 2^-100 .. 2^100
                        const int e = min(max((int)(__float_as_uint(most) >> 23) - 126, -100), 100);
                        const float next = __uint_as_float((uint32_t)(127 - e) << 23);
                        const float less = vref == 0.f ? 0.f : next / vref;
#pragma unroll
                        for (int c = 0; c < C; ++c)
                            r[c] *= less;
                        vref = next;
                    }
                }
#pragma unroll
                for (int i = 0; i < D / 16; ++i)
#pragma unroll
                    for (int j = 0; j < (FEW ? 2 : 4); ++j)
                        o[i][j] *= r[j % C];
                shifted();
            }
#pragma unroll
            for (int u = 0; u < SUB; ++u) {
#pragma unroll
                for (int i = 0; i < 2 * C; ++i)
                    x[u][i] = fast_ex2(x[u][i]);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    l[c] += x[u][c] + x[u][C + c];
                if constexpr (I8)
#pragma unroll
                    for (int i = 0; i < 2 * C; ++i)
                        x[u][i] *= vs[u][i / C] * vref;
            }
            weigh<KIND, D, FEW>(st, lane, x, o, over);
        }

        // the end of the segment
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int q = 4; q < 32; q <<= 1)
                l[c] += __shfl_xor_sync(0xffffffffu, l[c], q);
            // a NaN score raises no reference: keep the NaN sum in the merge
            m[c] = l[c] == 0.f ? -INFINITY : l[c] != l[c] && m[c] == kNone ? 0.f : m[c];
            if (g == 0) {
                sm_m[warp][C * t4 + c] = m[c];
                sm_l[warp][C * t4 + c] = l[c];
            }
        }
        // the ring's slot of the last tile is free until the next segment's
        // first fetch: the warps' outputs and the merge's scratch go there
        St *spare = ring[slot == 0 ? STAGES - 1 : slot - 1];
        auto &sm_o = *reinterpret_cast<float(*)[kWarps][kRows][D]>(spare);
        auto &sm_merge = *reinterpret_cast<Merge<KIND, D> *>(reinterpret_cast<unsigned char *>(spare) + sizeof sm_o);
        static_assert(sizeof sm_o + sizeof(Merge<KIND, D>) <= kWarps * sizeof(St), "the slot holds both");
        __syncthreads();                   // every warp has read its part of the slot
        if constexpr (I8) {
            const float f = vref == 0.f ? 0.f : 1.f / vref;
            // dims D / 8 * g + 2 i, + 1 in o[i][0 ..] and o[i][C ..]
#pragma unroll
            for (int i = 0; i < D / 16; i += 2)
#pragma unroll
                for (int c = 0; c < C; ++c)
                    *reinterpret_cast<float4 *>(&sm_o[warp][C * t4 + c][D / 8 * g + 2 * i]) =
                        make_float4(o[i][c] * f, o[i][C + c] * f, o[i + 1][c] * f, o[i + 1][C + c] * f);
        } else {
            // dims 16 i + g and 16 i + g + 8
#pragma unroll
            for (int i = 0; i < D / 16; ++i)
#pragma unroll
                for (int j = 0; j < 4; ++j)
                    sm_o[warp][2 * t4 + (j & 1)][16 * i + g + 8 * (j >> 1)] = o[i][j % (FEW ? 2 : 4)];
        }
        __syncwarp();
        TileCursor cur = seg->c;
        const int first_t = cur.t;
        cur.g += seg->t_last - cur.t;
        cur.t = seg->t_last;
        const bool any_bad = __syncthreads_or(sm_bad[warp][sc]) != 0;
        if (any_bad && good && tid == 0)
            report(p, kBadBlock);
        const bool end = !left && sc == sf;
        finish_segment<kWarps, kRows, D, D, false, true>(
            p, cur, walk, first_t, !good || any_bad, sm_m, sm_l, sm_o, &sm_flag, sm_merge, tid, kThreads,
            [] { __syncthreads(); }, arrived, [&](int row, float M, float den) {
                if (MORE && p.row_end)     // a NaN denominator: a bad row
                    p.row_end[(long long)cur.b * p.Hq + cur.kvh * p.G + row] = make_float2(M, 1.f / den);
            });
        if (end)
            break;
    }
}

template <int KIND, int D, bool QF32, bool FEW>
constexpr int dyn_bytes()
{
    return kWarps * kStages * (int)sizeof(Stage<KIND, D>) + kQueries * query_bytes<D, QF32, FEW>();
}

template <int KIND, int D, bool QF32, bool PAGED, bool FEW, bool MORE>
cudaError_t launch_one(const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    // the ring's size is set once a device
    static std::atomic<uint64_t> ready;
    constexpr int bytes = dyn_bytes<KIND, D, QF32, FEW>();
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(scored_kernel<KIND, D, QF32, PAGED, FEW, MORE>, cudaFuncAttributeMaxDynamicSharedMemorySize, bytes);
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    if (!p)
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, scored_kernel<KIND, D, QF32, PAGED, FEW, MORE>, kThreads, bytes);
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p->grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = bytes;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, scored_kernel<KIND, D, QF32, PAGED, FEW, MORE>, *p);
}

template <int KIND, int D, bool FEW, bool MORE>
cudaError_t launch_d(bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    if (q_bf16)
        return paged ? launch_one<KIND, D, false, true, FEW, MORE>(p, st, per_sm)
                     : launch_one<KIND, D, false, false, FEW, MORE>(p, st, per_sm);
    return paged ? launch_one<KIND, D, true, true, FEW, MORE>(p, st, per_sm)
                 : launch_one<KIND, D, true, false, FEW, MORE>(p, st, per_sm);
}

}  // namespace scored
}  // namespace gqa
