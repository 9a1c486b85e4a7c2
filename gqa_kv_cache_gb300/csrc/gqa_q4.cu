// Decode step and read-only attend over an E2M1 cache (D = 64 or 128, G <= 8).
//
// A cached vector is D / 2 bytes of codes and D / 16 bytes of E4M3 scales
// (gqa_fp4.cuh), 0.5625 bytes an element. Reading them takes the HBM less time
// than unpacking takes the SMs (below), so the kernel is laid out to unpack
// with few instructions:
//  * the schedule, the split of a unit between CTAs and its merge are those of
//    the other decode kernels (gqa_common.cuh); short units get a CTA each
//    (q4_whole_units). A CTA is four warps, a tile 4 x 32 slots. Each warp
//    copies its 32 slots of every tile into a ring of its own in shared memory
//    (16-byte asynchronous copies, kStages tiles deep: no barrier between the
//    warps, no registers for data in flight), and runs on to the CTA's next
//    segment, whose query rows and scales come the same way. Registers as the
//    stage instead (one tile ahead, 8 warps an SM) took 146 us where the ring
//    takes 94 (four rows of 32768 .. 131071 slots, G = 8).
//  * S^T = K Q^T (m16n8k16, f16 in, float32 sums): the M side is 16 slots, the
//    N side the G <= 8 query rows. Lane (g, t) of a warp takes slots g and
//    g + 8, and of each the D / 4 contiguous dims from D / 4 * t: one 16-byte
//    load (D = 128) a slot. Which dims make up a product step does not matter
//    to a dot product as long as the query fragments are taken in the same
//    order.
//  * O^T += V^T P^T: the M side is 16 dims, the N side the query rows, the
//    contraction 8 slots, each twice: the weight P is an f16 and an f16
//    remainder, neighbours in the contraction, and the value stands beside
//    both, as the doubled half of a register that its scale multiplies anyway.
//    The remainder enters 2^12 times as large, beside the value over 2^12 (both
//    exact), so that small weights keep their bits: a weight's error is at most
//    2^-23 of it and 2^-37, 2^-49 of the largest weight. (With one range for
//    both parts it was 2^-25, and 131072 slots of 2^-32.5 of the largest weight
//    counted as nothing; G > 4 took 105.0 us for 108.5, four rows of 32768 ..
//    131071 slots, float32 query.)
//    (Pairing two slots' values in a register took a byte permute each: 155 us
//    for 148 on 64 rows of 512 .. 16383 slots, G = 6.) Lane (g, t) takes D / 8
//    contiguous dims from D / 8 * g of four slots.
//  * up to four query rows (FEW) leave half the N side free: every row has two
//    columns there. In S^T they are the same (a float32 query: its f16 and its
//    remainder); in O^T one takes the first element of a code pair, the other
//    the second (the weight stands beside a zero), so the pairs enter the
//    product as the conversion gives them: half the f16 products, sums and
//    softmax steps (32 rows of 1024 .. 4095 slots: G = 4 37.7 -> 34.8 us,
//    G = 1 38.5 -> 34.8; float32 query, 64 rows of 512 .. 16383: 147 -> 139).
//    The remainders have sums of their own there (141 us for 139).
//  * codes become f16 by the hardware's conversion and every E2M1 x E4M3
//    product is an f16 exactly, so K and V enter the products unrounded. A
//    bfloat16 query is scaled by a power of two into f16's range (exact but
//    for elements 2^-38 below the row's largest); a float32 query is an f16
//    and an f16 remainder (22 bits). With P in f16 alone the output would be
//    off by 1e-4; so it is within 4e-7 of the 64-bit result on the sizes above.
//  * the softmax keeps a reference below the running maximum: weights are
//    2^(s - m) with m set to max - 12 and raised only when a score passes
//    m + 15, so they stay within f16's range and a tile costs a vote instead
//    of a reduction. (max - 14, raised at every octave: 110.6 us for 108.5 on
//    the rows above.)
//  * the matrix unit truncates its sums: the products of a tile are summed
//    from zero and added to the output in float32 (truncated on, a long cache's
//    output drifted by 3.5e-6).
//  * the new token (decode step): the warp whose tile holds slot L quantises
//    k_new and v_new, writes them to the cache, and then copies the tile; no
//    other warp touches slot L.
// What bounds it. Per 16 slots a warp issues about 358 instructions (D = 128,
// G > 4): 64 conversions and 47 others on the ALU, 104 f16 and 62 float32 on
// the FMA pipes, 24 matrix products. Each of these pipes takes a warp's
// instruction in two cycles, a product in 8.3, and conversions and f16 products
// overlap only in part (alone 7.9 cycles for four, together 12.2). The kernel
// issues 0.58 instructions a cycle (16 rows of 20000 .. 24000 slots, G = 8: 102
// us), 620 cycles per 16 slots and SM quarter, 4.0 TB/s of cache, 0.59 of the
// measured HBM copy rate; it hardly waits for memory (long scoreboard 0.12 of an
// issue). The bare conversions and products run at 0.71, which would be 500
// cycles and 5 TB/s; what keeps the kernel from that is not divided into parts.
// More warps (four CTAs of 128 registers) or scores of one tile beside the
// values of the one before changed nothing.
#define GQA_MULTI_TOKEN 0   // single-token steps only
#include <cuda_fp16.h>

#include <atomic>

#include "gqa_common.cuh"
#include "gqa_fp4.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr int kWarps = 4;
constexpr int kThreads = kWarps * 32;
constexpr int kSub = 2;                       // 16-slot parts of a warp's share of a tile (the code has two)
constexpr int kShare = 16 * kSub;              // a warp's slots of a tile
constexpr int kTile4 = kWarps * kShare;       // slots a tile
constexpr int kStages = 3;                    // tiles of a warp's ring (2: paged 160 us for 154)
constexpr int kCtas = 3;                      // resident CTAs per SM: 168 registers a thread (4 of 128: 167 us)
constexpr int kSegs = 4;                      // segments a warp's copies and products are in at once (< kStages + 1)
constexpr int kRows = 8;                      // query rows (G <= 8)
constexpr int kFew = 4;                       // and of the form for few
constexpr float kLift = 12.f;                 // a reference is set this far below the maximum ...
constexpr float kRoom = 15.f;                 // ... and holds until a score is this far above it
constexpr float kRest = 4096.f;               // a weight's remainder enters the products this much larger

__device__ __forceinline__ void mma_f16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                        uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.f16.f16.f32 "
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

// Two weights (at most 2^15) as an f16 pair and the f16 pair of kRest times what
// it leaves: a remainder of its own range, at most 2^15 like the weight.
__device__ __forceinline__ void split_weights(float x, float y, uint32_t &hi, uint32_t &lo)
{
    const __half2 h = __floats2half2_rn(x, y);
    const float2 f = __half22float2(h);
    hi = u32(h);
    lo = u32(__floats2half2_rn((x - f.x) * kRest, (y - f.y) * kRest));
}

// One tile's share of a warp in shared memory: its slots' codes of K and V
// and their scales, vectors in slot order. With D = 128 a vector's four
// 16-byte pieces and the two vectors of a 128-byte line are permuted so that
// the operand loads below have no bank conflicts.
template <int D>
struct Stage {
    uint8_t k[kShare * D / 2], v[kShare * D / 2];
    uint8_t ks[kShare * D / 16], vs[kShare * D / 16];
};

// Offset of 16-byte piece c of the share's vector r.
template <int D>
__device__ __forceinline__ int piece(int r, int c)
{
    if constexpr (D == 128)
        return (r >> 1) * 128 + (((r ^ (r >> 2)) & 1) << 6) + ((c ^ (r & 2)) << 4);
    else
        return r * 32 + c * 16;
}

__device__ __forceinline__ uint32_t smem_at(const void *p)
{
    return static_cast<uint32_t>(__cvta_generic_to_shared(p));
}

// Asynchronous copies to shared memory (DO, SO: byte offsets), and those of
// which `n` bytes come from src (all or none of them) and the others are zeros.
template <int DO, int SO>
__device__ __forceinline__ void copy16(uint32_t dst, const void *src)
{
    asm volatile("cp.async.cg.shared.global [%0 + %2], [%1 + %3], 16;" ::"r"(dst), "l"(src), "n"(DO), "n"(SO)
                 : "memory");
}
__device__ __forceinline__ void copy16(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.cg.shared.global [%0], [%1], 16, %2;" ::"r"(dst), "l"(src), "r"(n) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2;" ::"r"(dst), "l"(src), "n"(N) : "memory");
}
template <int N>
__device__ __forceinline__ void copy_small(uint32_t dst, const void *src, int n)
{
    asm volatile("cp.async.ca.shared.global [%0], [%1], %2, %3;" ::"r"(dst), "l"(src), "n"(N), "r"(n) : "memory");
}
__device__ __forceinline__ void copy_commit() { asm volatile("cp.async.commit_group;" ::: "memory"); }
template <int N>
__device__ __forceinline__ void copy_wait()
{
    asm volatile("cp.async.wait_group %0;" ::"n"(N) : "memory");
}

// Vector index of slot s of a unit of a paged cache, or -1.
__device__ __noinline__ long long paged_row(const int32_t *table, int block_size, int num_blocks, int Hkv, int kvh,
                                            int s)
{
    const int blk = __ldg(table + s / block_size);
    if (blk < 0 || blk >= num_blocks)
        return -1;
    return ((long long)blk * Hkv + kvh) * block_size + s % block_size;
}

__device__ __forceinline__ int scale_head(const DecodeParams &p, int b, int kvh)
{
    return p.scale_heads ? b % p.scale_heads : kvh;
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

// The unit's query fragments: lane (g, t) holds row g's D / 4 dims from
// D / 4 * t, scaled by a power of two into f16's range; `mul` is the factor
// that takes a product to a base-2 score for row g. q: the rows in shared memory.
template <int D, bool QF32, bool FEW>
__device__ __forceinline__ void load_query(const DecodeParams &p, const void *q, int lane,
                                           uint32_t (&qh)[D / 16][2], uint32_t (&ql)[QF32 && !FEW ? D / 16 : 1][2], float &mul)
{
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
    mul = __uint_as_float((uint32_t)(127 - 14 + e) << 23) * p.scale_log2;
#pragma unroll
    for (int i = 0; i < D / 16; ++i)
#pragma unroll
        for (int j = 0; j < 2; ++j) {
            const float a = x[4 * i + 2 * j] * up, b = x[4 * i + 2 * j + 1] * up;
            if constexpr (QF32 && FEW) {
                // the row's first column takes the f16, its second the remainder
                uint32_t h, l;
                split2(a, b, h, l);
                qh[i][j] = lane & 4 ? l : h;
            } else if constexpr (QF32)
                split2(a, b, qh[i][j], ql[i][j]);
            else
                qh[i][j] = u32(__floats2half2_rn(a, b));
        }
}

// A segment of a unit: consecutive tiles that this CTA computes. Kept in a
// small ring in shared memory: the copies run ahead of the products.
struct Segment {
    TileCursor c;      // at its first tile
    int t_last;        // its last tile
    int good;          // the row's content is in order
    float ks, vs;      // its head's scales
};

template <int D, bool QF32, bool FEW>
constexpr int query_bytes()
{
    return (FEW ? kFew : kRows) * D * (QF32 ? 4 : 2);
}

// What a warp's copies are taken from.
template <int D, bool PAGED>
struct Fetch {
    int t, t_last;     // (the rest of its segment is read from shared memory)
    bool good;
    uint32_t line;     // dense: vector of slot 0
    int page, page_next;   // paged: the block of part lane & 1 of tile (t & ~15) + lane / 2; of 16 tiles on
};

__device__ __forceinline__ int share_slot(int t, int tp, int gap, int warp)
{
    return (t < tp ? t : t + gap) * kTile4 + warp * kShare;
}

template <int D, bool PAGED>
__device__ __forceinline__ int load_page(const DecodeParams &p, const Fetch<D, PAGED> &f, const TileCursor &c, int shift,
                                         int tile, int warp, int lane)
{
    const int x = tile + (lane >> 1);
    const int s = share_slot(x, c.tp, c.gap, warp) + 16 * (lane & 1);
    return x <= f.t_last && s <= c.L ? __ldg(p.block_table + (long long)c.b * p.max_blocks + (s >> shift)) : 0;
}

// The copies' segment becomes that of cursor c. The segment's query rows (rows
// behind the G are zeros) and scales are copied too, a part by each warp, in
// the group of the copies that comes next.
template <int D, bool QF32, bool PAGED, bool FEW>
__device__ __forceinline__ void enter(const DecodeParams &p, const TileCursor &c, Fetch<D, PAGED> &f, Segment *seg, int *bad,
                                      void *q, int shift, bool pages, int warp, int lane)
{
    constexpr int B = QF32 ? 4 : 2;                // bytes an element
    constexpr int C = D * B / 16;                  // 16-byte pieces a row
    constexpr int R = FEW ? kFew : kRows;
    const char *src = static_cast<const char *>(p.q) + ((long long)c.b * p.Hq + (long long)c.kvh * p.G) * D * B;
#pragma unroll
    for (int i = 0; i < (R * C + kThreads - 1) / kThreads; ++i) {
        const int x = i * kThreads + warp * 32 + lane;
        if (R * C % kThreads == 0 || x < R * C)
            copy16(smem_at(q) + x * 16, x / C < p.G ? src + x * 16 : src, x / C < p.G ? 16 : 0);
    }
    if (lane < 2) {
        const float *sc = (lane ? p.v_scale : p.k_scale) + scale_head(p, c.b, c.kvh);
        copy_small<4>(smem_at(lane ? &seg->vs : &seg->ks), sc);
    }
    f.t = c.t;
    f.t_last = (int)min((long long)c.nr - 1, c.t + (c.end - c.g) - 1);
    f.good = row_ok(p, c.b, c.L);
    if constexpr (PAGED) {
        if (f.good && pages) {
            f.page = load_page(p, f, c, shift, f.t & ~15, warp, lane);
            f.page_next = load_page(p, f, c, shift, (f.t & ~15) + 16, warp, lane);
        }
    } else if (f.good) {
        const int r = p.slot_ids ? __ldg(p.slot_ids + c.b) : c.b;
        f.line = ((uint32_t)r * p.Hkv + c.kvh) * (uint32_t)p.Smax;
    }
    if (lane == 0) {
        seg->c = c;
        seg->t_last = f.t_last;
        seg->good = f.good;
        *bad = 0;
    }
}

// Starts the copies of the warp's share of tile f.t.
template <int D, bool PAGED>
__device__ __forceinline__ void fetch_tile(const DecodeParams &p, Fetch<D, PAGED> &f, const TileCursor &c, Stage<D> &st, int *bad,
                                           int shift, bool pages, int warp, int lane)
{
    if (!f.good)
        return;                            // its output is NaN, whatever is in the stage
    const int s = share_slot(f.t, c.tp, c.gap, warp);
    if (!p.attend && (unsigned)(c.L - s) < (unsigned)kShare)
        append_token<D>(p, c.b, c.kvh, c.L, lane);
    constexpr int LV = D / 32;             // lanes (16-byte pieces) a vector
    constexpr int VI = 32 / LV;            // vectors an instruction
    constexpr int SB = D / 16;             // scale bytes a vector
    const uint32_t dk = smem_at(st.k), dv = smem_at(st.v), dks = smem_at(st.ks), dvs = smem_at(st.vs);
    const uint8_t *kc = static_cast<const uint8_t *>(p.k_cache), *vc = static_cast<const uint8_t *>(p.v_cache);
    const uint8_t *kg = static_cast<const uint8_t *>(p.k_group), *vg = static_cast<const uint8_t *>(p.v_group);
    const int e = s + kShare - 1;
    if (pages && e <= c.L && (s >= c.lo || e < c.P)) {
        // every slot is in the softmax, 16 vectors in a row at least
        uint32_t row[kSub];
#pragma unroll
        for (int u = 0; u < kSub; ++u) {
            if constexpr (PAGED) {
                int blk = __shfl_sync(0xffffffffu, f.page, 2 * (f.t & 15) + u);
                if (blk < 0 || blk >= p.num_blocks) {
                    *bad = 1;
                    blk = 0;               // read something: the unit's output is NaN
                }
                row[u] = (((uint32_t)blk * p.Hkv + c.kvh) << shift) + ((uint32_t)(s + 16 * u) & ((1u << shift) - 1u));
            } else {
                row[u] = f.line + (uint32_t)(s + 16 * u);
            }
        }
        // part u, instruction j: vectors 16 u + VI j + lane / LV. piece() of
        // those is a constant past that of vector lane / LV
        const int r0 = lane / LV, c0 = lane % LV;
        const uint32_t to = (uint32_t)piece<D>(r0, c0);
        const uint64_t in = (uint64_t)(r0 * (D / 2) + c0 * 16);
        const uint8_t *k0 = kc + ((uint64_t)row[0] * (D / 2) + in), *v0 = vc + ((uint64_t)row[0] * (D / 2) + in);
        const uint8_t *k1 = kc + ((uint64_t)row[1] * (D / 2) + in), *v1 = vc + ((uint64_t)row[1] * (D / 2) + in);
        constexpr int S = VI * (D / 2);    // bytes between an instruction's vectors and the next one's
        copy16<0, 0>(dk + to, k0);
        copy16<0, 0>(dv + to, v0);
        if constexpr (VI == 8) {
            copy16<S, S>(dk + to, k0);
            copy16<S, S>(dv + to, v0);
            copy16<3 * S, S>(dk + to, k1);
            copy16<3 * S, S>(dv + to, v1);
        }
        copy16<16 * (D / 2), 0>(dk + to, k1);
        copy16<16 * (D / 2), 0>(dv + to, v1);
        const uint64_t at = (uint64_t)((lane < 16 ? row[0] : row[1]) + (lane & 15)) * SB;
        copy_small<SB>(dks + lane * SB, kg + at);
        copy_small<SB>(dvs + lane * SB, vg + at);
        return;
    }
    // slot by slot: any block size; a slot outside the softmax becomes zeros
    auto vector = [&](int j) -> long long {
        if (!attended(c.L, c.lo, c.P, s + j))
            return -1;
        if constexpr (PAGED) {
            const long long r = paged_row(p.block_table + (long long)c.b * p.max_blocks, p.block_size, p.num_blocks,
                                          p.Hkv, c.kvh, s + j);
            if (r < 0)
                *bad = 1;
            return r;
        } else {
            return (long long)f.line + s + j;
        }
    };
#pragma unroll
    for (int j = 0; j < kShare / VI; ++j) {
        const int r = VI * j + lane / LV, q = lane % LV;
        const long long x = vector(r);
        const uint64_t at = x < 0 ? 0 : (uint64_t)x * (D / 2) + q * 16;
        copy16(dk + piece<D>(r, q), kc + at, x < 0 ? 0 : 16);
        copy16(dv + piece<D>(r, q), vc + at, x < 0 ? 0 : 16);
    }
    const long long x = vector(lane);
    const uint64_t at = x < 0 ? 0 : (uint64_t)x * SB;
    copy_small<SB>(dks + lane * SB, kg + at, x < 0 ? 0 : SB);
    copy_small<SB>(dvs + lane * SB, vg + at, x < 0 ? 0 : SB);
}

// The slot (of a part's 16) at row i of the products' slot side, i = 0 .. 7
// (row i + 8: eight more). With it the value loads' four vectors at a time
// are neighbours.
__device__ __forceinline__ int slot_of(int i) { return (i >> 1) + 4 * (i & 1); }

// Scores of part u before their scale: s[0], s[1] slot slot_of(g) and query
// rows 2t, 2t + 1; s[2], s[3] eight slots on.
template <int D, bool QF32, bool FEW>
__device__ __forceinline__ void scores(const Stage<D> &st, int u, int lane, const uint32_t (&qh)[D / 16][2],
                                       const uint32_t (&ql)[QF32 && !FEW ? D / 16 : 1][2], float (&s)[4])
{
    const int g = lane >> 2, t = lane & 3;
    float s2[4] = {0.f, 0.f, 0.f, 0.f};
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] = 0.f;
    const int r = slot_of(g);
    uint32_t k[2][D / 32];
    __half2 sc[2];                         // the lane's group scales: two a vector (D = 64: one)
#pragma unroll
    for (int i = 0; i < 2; ++i) {
        const int v = 16 * u + r + 8 * i;
        if constexpr (D == 128) {
            const uint4 w = *reinterpret_cast<const uint4 *>(st.k + piece<D>(v, t));
            k[i][0] = w.x; k[i][1] = w.y; k[i][2] = w.z; k[i][3] = w.w;
            sc[i] = h2(e4m3x2_f16(*reinterpret_cast<const uint16_t *>(st.ks + v * 8 + 2 * t)));
        } else {
            const uint2 w = *reinterpret_cast<const uint2 *>(st.k + piece<D>(v, t >> 1) + 8 * (t & 1));
            k[i][0] = w.x; k[i][1] = w.y;
            sc[i] = h2(e4m3x2_f16(st.ks[v * 4 + t]));
        }
    }
#pragma unroll
    for (int w = 0; w < D / 32; ++w) {
        // D = 128: the lane's first two words are one group, the others the next
        const __half2 ma = w >= 2 ? __high2half2(sc[0]) : __low2half2(sc[0]);
        const __half2 mb = w >= 2 ? __high2half2(sc[1]) : __low2half2(sc[1]);
        const uint32_t a0 = u32(__hmul2(h2(e2m1x2_f16<0>(k[0][w])), ma)), b0 = u32(__hmul2(h2(e2m1x2_f16<0>(k[1][w])), mb));
        const uint32_t a1 = u32(__hmul2(h2(e2m1x2_f16<1>(k[0][w])), ma)), b1 = u32(__hmul2(h2(e2m1x2_f16<1>(k[1][w])), mb));
        const uint32_t a2 = u32(__hmul2(h2(e2m1x2_f16<2>(k[0][w])), ma)), b2 = u32(__hmul2(h2(e2m1x2_f16<2>(k[1][w])), mb));
        const uint32_t a3 = u32(__hmul2(h2(e2m1x2_f16<3>(k[0][w])), ma)), b3 = u32(__hmul2(h2(e2m1x2_f16<3>(k[1][w])), mb));
        mma_f16(s, a0, b0, a1, b1, qh[2 * w][0], qh[2 * w][1]);
        mma_f16(s2, a2, b2, a3, b3, qh[2 * w + 1][0], qh[2 * w + 1][1]);
        if constexpr (QF32 && !FEW) {
            mma_f16(s, a0, b0, a1, b1, ql[2 * w][0], ql[2 * w][1]);
            mma_f16(s2, a2, b2, a3, b3, ql[2 * w + 1][0], ql[2 * w + 1][1]);
        }
    }
#pragma unroll
    for (int i = 0; i < 4; ++i)
        s[i] += s2[i];
    if constexpr (QF32 && FEW) {
        s[0] += s[1];
        s[2] += s[3];
    }
}

// One product of the sum below: the pair of dims in byte Q of the words x, y
// of two slots, their scales sx, sy as (s, s / kRest) pairs, and the weights
// b0, b1 of the two slots as (f16, remainder) pairs. The contraction runs over
// (slot, part of the weight), so a value enters twice in a row -- the halves of
// a register, the second over kRest -- and is never paired with another slot's.
template <int Q>
__device__ __forceinline__ void weigh_pair(uint32_t x, uint32_t y, __half2 sx, __half2 sy, uint32_t b0, uint32_t b1,
                                           float (&d)[4])
{
    const __half2 p = h2(e2m1x2_f16<Q>(x)), q = h2(e2m1x2_f16<Q>(y));
    mma_f16(d, u32(__hmul2(__low2half2(p), sx)), u32(__hmul2(__high2half2(p), sx)), u32(__hmul2(__low2half2(q), sy)),
            u32(__hmul2(__high2half2(q), sy)), b0, b1);
}

// Two code pairs of slots x and y (scales sc) for few query rows: rows g and
// g + 8 are the pairs of bytes 2 Q and 2 Q + 1, a column one element of the
// pairs for one query; the weights' f16 (bh) are summed in d, their remainders
// (bl, kRest times as large) in r.
template <int Q>
__device__ __forceinline__ void weigh_few(uint32_t x, uint32_t y, __half2 sc, const uint32_t (&bh)[2], const uint32_t (&bl)[2],
                                          float (&d)[4], float (&r)[4])
{
    const __half2 sx = __low2half2(sc), sy = __high2half2(sc);
    const uint32_t a0 = u32(__hmul2(h2(e2m1x2_f16<2 * Q>(x)), sx)), a1 = u32(__hmul2(h2(e2m1x2_f16<2 * Q + 1>(x)), sx));
    const uint32_t a2 = u32(__hmul2(h2(e2m1x2_f16<2 * Q>(y)), sy)), a3 = u32(__hmul2(h2(e2m1x2_f16<2 * Q + 1>(y)), sy));
    mma_f16(d, a0, a1, a2, a3, bh[0], bh[1]);
    mma_f16(r, a0, a1, a2, a3, bl[0], bl[1]);
}

// O^T += V^T P^T over a warp's slots of a tile; w[u] are the weights in the
// positions of the scores. The products of a tile are summed from zero and then
// added to o (the matrix unit truncates its sums). FEW: o[i] are dims 4 i .. + 3
// (from D / 8 * g) of query t; else dims 2 i, 2 i + 1 of queries 2t, 2t + 1.
template <int D, bool FEW>
__device__ __forceinline__ void weigh(const Stage<D> &st, int lane, const float (&w)[kSub][FEW ? 2 : 4],
                                      float (&o)[D / (FEW ? 32 : 16)][4])
{
    const int g = lane >> 2, t = lane & 3;
    // rows 2t, 2t + 1, 2t + 8, 2t + 9 of the slot side: (f16, remainder) of a
    // slot; FEW: (f16, 0) of a slot where the column is the pair's first
    // element, (0, f16) where its second, and the remainders likewise
    uint32_t b[kSub][4], br[FEW ? kSub : 1][4];
    __half2 sc[kSub][2];                   // their scales
    [[maybe_unused]] __half2 sp[FEW ? 1 : kSub][4];   // as (s, s / kRest) (both exact: an E4M3 and one over 2^12)
    uint32_t v[kSub][4][D / 64];
#pragma unroll
    for (int u = 0; u < kSub; ++u) {
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h, l;
            if constexpr (FEW)
                split_weights(w[u][i], w[u][i], h, l);
            else
                split_weights(w[u][2 * i], w[u][2 * i + 1], h, l);
            h = movmatrix_t(h);
            l = movmatrix_t(l);
            if constexpr (FEW) {
                const uint32_t first = g & 1 ? 0x1044u : 0x4410u, second = g & 1 ? 0x3244u : 0x4432u;
                b[u][2 * i] = __byte_perm(h, 0u, first);
                b[u][2 * i + 1] = __byte_perm(h, 0u, second);
                br[u][2 * i] = __byte_perm(l, 0u, first);
                br[u][2 * i + 1] = __byte_perm(l, 0u, second);
            } else {
                b[u][2 * i] = __byte_perm(h, l, 0x5410);
                b[u][2 * i + 1] = __byte_perm(h, l, 0x7632);
            }
        }
        uint32_t e[4];
#pragma unroll
        for (int j = 0; j < 4; ++j) {
            const int x = 16 * u + t + 4 * j;
            if constexpr (D == 128) {
                const uint2 y = *reinterpret_cast<const uint2 *>(st.v + piece<D>(x, g >> 1) + 8 * (g & 1));
                v[u][j][0] = y.x;
                v[u][j][1] = y.y;
                e[j] = st.vs[x * 8 + g];
            } else {
                v[u][j][0] = *reinterpret_cast<const uint32_t *>(st.v + piece<D>(x, g >> 2) + 4 * (g & 3));
                e[j] = st.vs[x * 4 + (g >> 1)];
            }
        }
        sc[u][0] = h2(e4m3x2_f16(e[0] | (e[1] << 8)));
        sc[u][1] = h2(e4m3x2_f16(e[2] | (e[3] << 8)));
        if constexpr (!FEW) {
            const __half2 parts = __floats2half2_rn(1.f, 1.f / kRest);
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                sp[u][2 * j] = __hmul2(__low2half2(sc[u][j]), parts);
                sp[u][2 * j + 1] = __hmul2(__high2half2(sc[u][j]), parts);
            }
        }
    }
#pragma unroll
    for (int i = 0; i < D / 64; ++i) {
        constexpr int N = FEW ? 2 : 4;
        float d[N][4] = {};
        [[maybe_unused]] float r[N][4] = {};   // FEW: the remainders' products
#pragma unroll
        for (int u = 0; u < kSub; ++u)
#pragma unroll
            for (int j = 0; j < 2; ++j) {
                const uint32_t x = v[u][2 * j][i], y = v[u][2 * j + 1][i];
                if constexpr (FEW) {
                    const uint32_t bh[2] = {b[u][2 * j], b[u][2 * j + 1]}, bl[2] = {br[u][2 * j], br[u][2 * j + 1]};
                    weigh_few<0>(x, y, sc[u][j], bh, bl, d[0], r[0]);
                    weigh_few<1>(x, y, sc[u][j], bh, bl, d[1], r[1]);
                } else {
                    weigh_pair<0>(x, y, sp[u][2 * j], sp[u][2 * j + 1], b[u][2 * j], b[u][2 * j + 1], d[0]);
                    weigh_pair<1>(x, y, sp[u][2 * j], sp[u][2 * j + 1], b[u][2 * j], b[u][2 * j + 1], d[1]);
                    weigh_pair<2>(x, y, sp[u][2 * j], sp[u][2 * j + 1], b[u][2 * j], b[u][2 * j + 1], d[2 % N]);
                    weigh_pair<3>(x, y, sp[u][2 * j], sp[u][2 * j + 1], b[u][2 * j], b[u][2 * j + 1], d[3 % N]);
                }
            }
#pragma unroll
        for (int q = 0; q < N; ++q)
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                o[N * i + q][j] += d[q][j];
                if constexpr (FEW)
                    o[N * i + q][j] = fmaf(r[q][j], 1.f / kRest, o[N * i + q][j]);
            }
    }
}

// Scratch of the merge (segment_out, unit_ticket_merge): as many partials at a
// time as the spare slot has room for.
template <int D>
using Merge = MergeBufT<kRows, D == 128 ? 28 : 12>;

template <int D, bool QF32, bool PAGED, bool FEW>
__global__ void __launch_bounds__(kThreads, kCtas) q4_decode_kernel(const DecodeParams p)
{
    constexpr int C = FEW ? 1 : 2;             // query rows of a lane: t4, or 2t4 and 2t4 + 1
    extern __shared__ __align__(128) unsigned char dyn[];
    Stage<D>(*ring)[kWarps] = reinterpret_cast<Stage<D>(*)[kWarps]>(dyn);      // [kStages]
    auto sm_q = reinterpret_cast<uint8_t(*)[query_bytes<D, QF32, FEW>()]>(dyn + kStages * kWarps * sizeof(Stage<D>));   // [kSegs]
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
    // whole pages of 16 slots: one vector index a part; else slot by slot
    const int shift = PAGED ? __ffs(p.block_size) - 1 : 0;
    const bool pages = !PAGED || (p.block_size >= 16 && (p.block_size & (p.block_size - 1)) == 0);

    // the copies: tile f.t of segment sf is the next to fetch
    Fetch<D, PAGED> f = {};
    int sf = 0;
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
        enter<D, QF32, PAGED, FEW>(p, c, f, &segs[0], &sm_bad[warp][0], sm_q[0], shift, pages, warp, lane);
        __syncwarp();
    }
    auto fetch = [&](int slot) {
        if (left) {
            fetch_tile(p, f, segs[sf].c, ring[slot][warp], &sm_bad[warp][sf], shift, pages, warp, lane);
            if (f.t < f.t_last) {
                ++f.t;
                if constexpr (PAGED) {
                    if ((f.t & 15) == 0 && f.good && pages) {
                        f.page = f.page_next;
                        f.page_next = load_page(p, f, segs[sf].c, shift, f.t + 16, warp, lane);
                    }
                }
            } else {
                TileCursor c = segs[sf].c;
                c.g += f.t - c.t;
                c.t = f.t;
                left = !p.whole_units && walk_next(p, c, walk, in_b);
                if (left) {
                    sf = (sf + 1) % kSegs;
                    enter<D, QF32, PAGED, FEW>(p, c, f, &segs[sf], &sm_bad[warp][sf], sm_q[sf], shift, pages, warp, lane);
                    __syncwarp();
                }
            }
        }
        copy_commit();                     // an empty group behind the last tile
    };
    int slot = 0;                          // ring slot of the tile to compute
#pragma unroll
    for (int i = 0; i < kStages - 1; ++i)
        fetch(i);

    // the first segment's query rows and scales, every warp's part (those of
    // a later one came with the last tile of the segment before it, whose end
    // the warps meet at)
    copy_wait<kStages - 2>();
    __syncthreads();
    uint32_t qh[D / 16][2], ql[QF32 && !FEW ? D / 16 : 1][2];
    float mul[C], m[C], l[C];              // product to base-2 score, reference and sum of the lane's rows
    float o[D / (FEW ? 32 : 16)][4];
    for (int sc = 0;; sc = (sc + 1) % kSegs) {
        // the next segment
        const Segment *seg = &segs[sc];
        const bool good = seg->good;
        if (!good && tid == 0 && seg->c.t == 0 && seg->c.kvh == 0)
            report(p, row_error_bits(p, seg->c.b, seg->c.L));
        float mine;
        load_query<D, QF32, FEW>(p, sm_q[sc], lane, qh, ql, mine);
        const float ks = seg->ks;
#pragma unroll
        for (int c = 0; c < C; ++c) {
            mul[c] = __shfl_sync(0xffffffffu, mine, 8 * t4 + 4 * c) * ks;
            m[c] = -INFINITY;
            l[c] = 0.f;
        }
#pragma unroll
        for (int i = 0; i < D / (FEW ? 32 : 16); ++i)
#pragma unroll
            for (int j = 0; j < 4; ++j)
                o[i][j] = 0.f;

        int arrived = -1;                  // thread 0: the unit's arrival count before the last tile
        for (int t = seg->c.t; t <= seg->t_last; ++t) {
            if (t == seg->t_last && tid == 0 && (seg->c.t != 0 || t != seg->c.nr - 1))
                asm volatile("ld.acquire.gpu.global.s32 %0, [%1];"
                             : "=r"(arrived)
                             : "l"(p.ws_cnt + seg->c.b * p.Hkv + seg->c.kvh)
                             : "memory");
            copy_wait<kStages - 2>();      // this lane's copies of the tile, then the other lanes'
            __syncwarp();
            fetch(slot == 0 ? kStages - 1 : slot - 1);
            const Stage<D> &st = ring[slot][warp];
            slot = slot + 1 == kStages ? 0 : slot + 1;
            float s[kSub][4];
#pragma unroll
            for (int u = 0; u < kSub; ++u)
                scores<D, QF32, FEW>(st, u, lane, qh, ql, s[u]);
            // bits 2 u + i: slot 16 u + slot_of(g) + 8 i is in the softmax
            unsigned ok = good ? ~0u : 0u;
            const int s0 = share_slot(t, seg->c.tp, seg->c.gap, warp), L = seg->c.L, lo = seg->c.lo, P = seg->c.P;
            if (s0 + kShare - 1 > L || (s0 < lo && s0 + kShare - 1 >= P)) {
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
                        if (!attended(L, lo, P, s0 + 16 * u + slot_of(g) + 8 * i))
                            ok &= ~(1u << (2 * u + i));
            }
            // x = base-2 score - reference, of slots u, i and rows c
            float x[kSub][2 * C], top = -INFINITY;
            auto shifted = [&] {
#pragma unroll
                for (int u = 0; u < kSub; ++u)
#pragma unroll
                    for (int i = 0; i < 2; ++i)
#pragma unroll
                        for (int c = 0; c < C; ++c) {
                            float &y = x[u][C * i + c];
                            y = fmaf(s[u][2 * i + c], mul[c], -m[c]);
                            y = (ok >> (2 * u + i)) & 1u ? y : -INFINITY;
                        }
            };
            shifted();
#pragma unroll
            for (int u = 0; u < kSub; ++u)
#pragma unroll
                for (int i = 0; i < 2 * C; ++i)
                    top = fmaxf(top, x[u][i]);
            if (__any_sync(0xffffffffu, top > kRoom)) {
                float r[C];
#pragma unroll
                for (int c = 0; c < C; ++c) {
                    float most = -INFINITY;
#pragma unroll
                    for (int u = 0; u < kSub; ++u)
#pragma unroll
                        for (int i = 0; i < 2; ++i)
                            if ((ok >> (2 * u + i)) & 1u)
                                most = fmaxf(most, s[u][2 * i + c] * mul[c]);
#pragma unroll
                    for (int q = 4; q < 32; q <<= 1)
                        most = fmaxf(most, __shfl_xor_sync(0xffffffffu, most, q));
                    const float n = most - m[c] > kRoom ? most - kLift : m[c];
                    r[c] = m[c] == -INFINITY ? 0.f : fast_ex2(m[c] - n);
                    m[c] = n;
                    l[c] *= r[c];
                }
#pragma unroll
                for (int i = 0; i < D / (FEW ? 32 : 16); ++i)
#pragma unroll
                    for (int j = 0; j < 4; ++j)
                        o[i][j] *= r[j % C];
                shifted();
            }
#pragma unroll
            for (int u = 0; u < kSub; ++u) {
#pragma unroll
                for (int i = 0; i < 2 * C; ++i)
                    x[u][i] = fast_ex2(x[u][i]);
#pragma unroll
                for (int c = 0; c < C; ++c)
                    l[c] += x[u][c] + x[u][C + c];
            }
            weigh<D, FEW>(st, lane, x, o);
        }

        // the end of the segment
#pragma unroll
        for (int c = 0; c < C; ++c) {
#pragma unroll
            for (int q = 4; q < 32; q <<= 1)
                l[c] += __shfl_xor_sync(0xffffffffu, l[c], q);
            // a NaN score raises no reference: keep the NaN sum in the merge
            m[c] = (l[c] != l[c] && m[c] == -INFINITY) ? 0.f : m[c];
            if (g == 0) {
                sm_m[warp][C * t4 + c] = m[c];
                sm_l[warp][C * t4 + c] = l[c];
            }
        }
        // the ring's slot of the last tile is free until the next segment's
        // first fetch: the warps' outputs and the merge's scratch go there
        Stage<D> *spare = ring[slot == 0 ? kStages - 1 : slot - 1];
        auto &sm_o = *reinterpret_cast<float(*)[kWarps][kRows][D]>(spare);
        auto &sm_merge = *reinterpret_cast<Merge<D> *>(reinterpret_cast<unsigned char *>(spare) + sizeof sm_o);
        static_assert(sizeof sm_o + sizeof(Merge<D>) <= kWarps * sizeof(Stage<D>), "the slot holds both");
        __syncthreads();                   // every warp has read its part of the slot
        const float vs = seg->vs;
        if constexpr (FEW) {
            // row t4: dims D / 8 * g + 4 i .. + 3
#pragma unroll
            for (int i = 0; i < D / 32; ++i)
                *reinterpret_cast<float4 *>(&sm_o[warp][t4][D / 8 * g + 4 * i]) =
                    make_float4(o[i][0] * vs, o[i][1] * vs, o[i][2] * vs, o[i][3] * vs);
        } else {
#pragma unroll
            for (int i = 0; i < D / 16; i += 2) {
                // rows 2t4, 2t4 + 1: dims D / 8 * g + 2 i .. + 3
                *reinterpret_cast<float4 *>(&sm_o[warp][2 * t4][D / 8 * g + 2 * i]) =
                    make_float4(o[i][0] * vs, o[i][2] * vs, o[i + 1][0] * vs, o[i + 1][2] * vs);
                *reinterpret_cast<float4 *>(&sm_o[warp][2 * t4 + 1][D / 8 * g + 2 * i]) =
                    make_float4(o[i][1] * vs, o[i][3] * vs, o[i + 1][1] * vs, o[i + 1][3] * vs);
            }
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
        finish_segment<kWarps, kRows, D, D, false, true>(p, cur, walk, first_t, !good || any_bad, sm_m, sm_l, sm_o,
                                                         &sm_flag, sm_merge, tid, kThreads,
                                                         [] { __syncthreads(); }, arrived);
        if (end)
            break;
    }
}

template <int D, bool QF32, bool FEW>
constexpr int dyn_bytes()
{
    return kWarps * kStages * (int)sizeof(Stage<D>) + kSegs * query_bytes<D, QF32, FEW>();
}

template <int D, bool QF32, bool PAGED, bool FEW>
cudaError_t launch_one(const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    // the ring's size is set once a device
    static std::atomic<uint64_t> ready;
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(q4_decode_kernel<D, QF32, PAGED, FEW>, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 dyn_bytes<D, QF32, FEW>());
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    if (!p)
        return cudaOccupancyMaxActiveBlocksPerMultiprocessor(per_sm, q4_decode_kernel<D, QF32, PAGED, FEW>, kThreads,
                                                             dyn_bytes<D, QF32, FEW>());
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p->grid);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = dyn_bytes<D, QF32, FEW>();
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, q4_decode_kernel<D, QF32, PAGED, FEW>, *p);
}

template <int D, bool FEW>
cudaError_t launch_d(bool q_bf16, bool paged, const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    if (q_bf16)
        return paged ? launch_one<D, false, true, FEW>(p, st, per_sm) : launch_one<D, false, false, FEW>(p, st, per_sm);
    return paged ? launch_one<D, true, true, FEW>(p, st, per_sm) : launch_one<D, true, false, FEW>(p, st, per_sm);
}

cudaError_t launch(int D, int G, bool q_bf16, bool paged, const DecodeParams *p, cudaStream_t st, int *per_sm)
{
    if (G <= kFew)
        return D == 128 ? launch_d<128, true>(q_bf16, paged, p, st, per_sm) : launch_d<64, true>(q_bf16, paged, p, st, per_sm);
    return D == 128 ? launch_d<128, false>(q_bf16, paged, p, st, per_sm) : launch_d<64, false>(q_bf16, paged, p, st, per_sm);
}

}  // namespace

bool q4_supports(int D, int G) { return (D == 64 || D == 128) && G >= 1 && G <= kRows; }

int q4_tile() { return kTile4; }

// One CTA a unit, whole, where units are short: no schedule to assemble, no
// partial states to merge. Measured back to back (G = 4, D = 128, bfloat16
// query; one CTA a unit / the schedule, us): capacity 256: 8 units 5.4 / 8.8,
// 512 units 12.2 / 15.1, 2048 units 30.2 / 31.6; 512: 6.8 / 9.7, 16.3 / 18.8,
// 46.6 / 47.2; 1024: 9.9 / 10.5, 23.8 / 25.6, 70.9 / 74.3, but 512 units with
// cold caches 32.8 / 30.7; 2048: 15.7 / 12.0, 41.5 / 40.7. So: up to four
// tiles, or eight where all units run at once.
bool q4_whole_units(long long capacity, long long units, int grid)
{
    return capacity <= 4 * kTile4 || (capacity <= 8 * kTile4 && units <= grid);
}

int q4_ctas_per_sm(int D, bool q_bf16)
{
    int least = 1 << 30;
    for (int G : {kFew, kRows})
        for (bool paged : {false, true}) {
            int n = 0;
            if (launch(D, G, q_bf16, paged, nullptr, nullptr, &n) != cudaSuccess)
                return 1;
            least = n < least ? n : least;
        }
    return least > 0 ? least : 1;
}

cudaError_t q4_launch(const DecodeParams &p, cudaStream_t st)
{
    return launch(p.D, p.G, p.q_bf16, p.paged, &p, st, nullptr);
}

}  // namespace gqa
