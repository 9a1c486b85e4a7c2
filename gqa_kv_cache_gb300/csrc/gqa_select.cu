// Block selection: the blocks of slots whose key bounds promise the highest
// scores, for every (row, cache head).
//
// Block j of a row holds the keys of its slots within the box [lo_j, hi_j]
// (element-wise). For the G query heads of a cache head
//   score_j = sum_g max over the box of q_g . k = sum_d P_d hi_jd + N_d lo_jd,
//   P_d = sum_g max(q_gd, 0),  N_d = sum_g min(q_gd, 0),
// so one dot product of 2 D terms scores a block for the whole group. Kept are
// the first n_first and the last n_last valid blocks and the best of the rest,
// equal scores by the lowest index; a NaN score counts as the highest.
//
// The kernel reads 4 D bytes a (block, head) and writes n_select indexes, so
// it is bound by memory when there are many units and by latency when there
// are few: a unit, one (row, cache head), is a cluster of 1 to 8 CTAs, each
// scoring a share of the unit's blocks into the shared memory of the cluster's
// first CTA, which then selects.
//
// Scores are summed in float32, which cannot order two scores that differ by
// less than its rounding. Every score is within E of its exact value, E =
// (a count of roundings, derived below) 2^-24 sum_d |w_d| max |x| over the unit's
// blocks (512 units of up to 1024 blocks: 57 us; 55 with half the count, which
// the terms that a matrix step drops could pass); with T the n-th largest
// float32 score, a score above T + 2 E is kept and one below T - 2 E is not,
// whatever the rounding. The few in between, when they do not all fit, are
// summed again in 64 bits and ordered by that.
#include <cooperative_groups.h>

#include <atomic>

#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kFew = 64;            // candidates ordered by comparing each with each
constexpr int kBins = 256;          // bins of the first cut of the scores
constexpr int kMaxCluster = 8;
constexpr int kMaxBlocks = 16384;   // blocks a row: the leader's shared memory (12 bytes each)
constexpr uint32_t kForced = 0xffffffffu;

// Order-preserving map of floats to unsigned integers; NaN above all.
__device__ __forceinline__ uint32_t key32(float x)
{
    const uint32_t u = __float_as_uint(x);
    if (x != x)
        return kForced - 1;
    return (u & 0x80000000u) ? ~u : u | 0x80000000u;
}
__device__ __forceinline__ unsigned long long key64_of(double x)
{
    const unsigned long long u = (unsigned long long)__double_as_longlong(x);
    if (x != x)
        return ~0ull;
    return (u >> 63) ? ~u : u | (1ull << 63);
}
__device__ __forceinline__ float unkey32(uint32_t k)
{
    if (k >= kForced - 1)
        return __int_as_float(0x7fc00000);
    return __uint_as_float((k & 0x80000000u) ? k & 0x7fffffffu : ~k);
}

// Sums over a block of NT threads, one after the other, each with one barrier
// (two sets of cells in turn: the next sum's writes meet no reader of the last).
// Two counts below 2^16 can share a sum.
template <int NT>
struct Sums {
    int (*cell)[NT / 32];
    int turn;
    __device__ __forceinline__ int operator()(int v)
    {
        v = __reduce_add_sync(0xffffffffu, v);
        turn ^= 1;
        if ((threadIdx.x & 31) == 0)
            cell[turn][threadIdx.x >> 5] = v;
        __syncthreads();
        int s = 0;
#pragma unroll
        for (int i = 0; i < NT / 32; ++i)
            s += cell[turn][i];
        return s;
    }
};

// The n-th largest (n >= 1) of the keys key[0 .. m - 1] (in shared memory) is
// the smallest key that reaches the value returned: the value is found bit by
// bit from the top, and its low bits are left at zero once exactly n keys
// reach it.
template <int NT, typename K>
__device__ __noinline__ K nth_largest(const K *key, int m, int n, Sums<NT> &sum)
{
    K at = 0;
    for (int bit = 8 * (int)sizeof(K) - 1; bit >= 0; --bit) {
        const K cand = at | ((K)1 << bit);
        int c = 0;
        for (int j = threadIdx.x; j < m; j += NT)
            c += key[j] >= cand;
        c = sum(c);
        if (c >= n)
            at = cand;
        if (c == n)
            break;
    }
    return at;
}

// Index of block j of (row b, head h) in the flattened pool of (block, head)
// pairs, or -1.
__device__ __forceinline__ int pool_block(const SelectParams &p, int b, int h, int r, int j)
{
    if (!p.paged)
        return (int)(((long long)r * p.Hkv + h) * p.NB + j);
    const int blk = __ldg(p.block_table + (long long)b * p.NB + j);
    return blk < 0 || blk >= p.num_blocks ? -1 : blk * p.Hkv + h;
}

__device__ __forceinline__ void mma_bf16(float (&d)[4], uint32_t a0, uint32_t a1, uint32_t a2, uint32_t a3,
                                         uint32_t b0, uint32_t b1)
{
    asm("mma.sync.aligned.m16n8k16.row.col.f32.bf16.bf16.f32 "
        "{%0, %1, %2, %3}, {%4, %5, %6, %7}, {%8, %9}, {%0, %1, %2, %3};"
        : "+f"(d[0]), "+f"(d[1]), "+f"(d[2]), "+f"(d[3])
        : "r"(a0), "r"(a1), "r"(a2), "r"(a3), "r"(b0), "r"(b1));
}

// The larger magnitude of each of two bfloat16 (signs xored; NaN ignored).
__device__ __forceinline__ void raise(uint32_t &top, uint32_t x)
{
    asm("max.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(top) : "r"(x));
}

// Element d of query head g of the unit, as loaded, and its value.
__device__ __forceinline__ uint32_t query_raw(const SelectParams &p, long long head0, int g, int D, int d)
{
    const long long at = (head0 + g) * D + d;
    return p.q_bf16 ? (uint32_t)__ldg(static_cast<const unsigned short *>(p.q) + at)
                    : __ldg(static_cast<const uint32_t *>(p.q) + at);
}
__device__ __forceinline__ float query(const SelectParams &p, uint32_t raw)
{
    return __uint_as_float(p.q_bf16 ? raw << 16 : raw);
}

// NT threads a CTA: 256 where a unit has few CTAs, 128 where the units fill
// the GPU (more of them at once, so that one's selection runs beside others'
// loads).
template <int D, int NT>
__global__ void __launch_bounds__(NT, NT == 128 ? 4 : 2) select_kernel(const SelectParams p)
{
    constexpr int NW = NT / 32;
    constexpr int E = 2 * D;               // elements of a block's bounds: lo, then hi
    constexpr int LOADS = E / 32;          // 16-byte loads a lane and block
    constexpr int H = LOADS < 8 ? LOADS : 8;   // those in flight at once
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned long long *key64 = reinterpret_cast<unsigned long long *>(smem);   // [NB]: keys of the 64-bit scores
    uint32_t *key = reinterpret_cast<uint32_t *>(key64 + p.NB);                 // [NB] (leader)
    __shared__ __align__(16) uint16_t wt[3][E];    // the weights N_d, then P_d, as sums of three bfloat16
    __shared__ double wt64[E];             // and in 64 bits, where they are needed
    __shared__ float warp_w[NW];           // sums of |weight|
    __shared__ int cells[2][NW];
    __shared__ float warp_top[NW];
    __shared__ uint32_t warp_key[2][NW];
    __shared__ float err[kMaxCluster];
    __shared__ int any_bad[kMaxCluster];
    __shared__ float range[kMaxCluster][2];   // lowest and highest score that is not forced
    __shared__ int scan[NW];
    __shared__ int bins[kBins];
    __shared__ int few[kFew], n_few, found[2];

    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / ranks;
    const int b = unit / p.Hkv, h = unit % p.Hkv;
    const int G = p.Hq / p.Hkv;
    const long long head0 = (long long)b * p.Hq + (long long)h * G;

    // the next kernel may be set up meanwhile (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int len = __ldg(p.lengths + b);
    // the first query heads' elements, asked for before the bounds (behind
    // every CTA's first bounds they came 4 us later)
    constexpr int DS = (D + NT - 1) / NT, GS = 8;
    uint32_t raw[DS][GS];
#pragma unroll
    for (int i = 0; i < DS; ++i)
#pragma unroll
        for (int q = 0; q < GS; ++q)
            raw[i][q] = q < G && tid + i * NT < D ? query_raw(p, head0, q, D, tid + i * NT) : 0u;
    const int r = p.paged ? 0 : (p.slot_ids ? __ldg(p.slot_ids + b) : b);
    int bits = 0;
    if (len < 1 || (long long)len > (long long)p.NB * p.block_size)
        bits = kBadLength;
    else if (!p.paged && (r < 0 || r >= p.R))
        bits = kBadSlotId;
    const int n = bits ? 0 : (len + p.block_size - 1) / p.block_size;   // valid blocks
    const bool all = n <= p.n_select;
    for (int i = tid; i < kBins; i += NT)
        bins[i] = 0;
    if (tid == 0)
        n_few = 0;
    // the leader's shared memory is written to below: every CTA must have started
    if (ranks > 1)
        cl.sync();

    if (!all) {
        // Scores of 16 blocks at a time on the tensor cores: the blocks are
        // the M side, the weights' three parts columns 0 .. 2 of the N side.
        // Lane (g, t) holds blocks g and g + 8, eight elements a load from
        // 32 i + 8 t; a load makes two product steps, whose weights are taken
        // in the same order. Four sums of each run side by side. The loads
        // of a warp's next blocks are issued as soon as these are used; the
        // blocks' places (one lane each) are known one step ahead of that.
        const int g = lane >> 2, t = lane & 3;
        uint32_t *out = cl.map_shared_rank(key, 0);
        const int j0 = (int)((long long)n * rank / ranks), j1 = (int)((long long)n * (rank + 1) / ranks);
        bool bad = false;
        // (past the share's end its last block again, whose score is not used)
        auto place = [&](int base) {
            return lane < 16 ? pool_block(p, b, h, r, max(0, min(base + lane, j1 - 1))) : 0;
        };
        uint4 xa[H], xb[H];
        // a bad block reads the first of the pool: its score is not used
        auto load = [&](int at, int i0) {
            const int a = max(0, __shfl_sync(0xffffffffu, at, g)), c = max(0, __shfl_sync(0xffffffffu, at, g + 8));
            const uint4 *x0 = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.bounds) + (long long)a * E);
            const uint4 *x1 = reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(p.bounds) + (long long)c * E);
#pragma unroll
            for (int i = 0; i < H; ++i) {
                xa[i] = __ldg(x0 + t + 4 * (i0 + i));
                xb[i] = __ldg(x1 + t + 4 * (i0 + i));
            }
        };
        constexpr int STEP = 16 * NW;
        int at = place(j0 + 16 * warp), at_next = place(j0 + 16 * warp + STEP);

        float mag = 0.f;
#pragma unroll
        for (int k = 0; k < DS; ++k) {
            const int d = tid + k * NT;
            if (d >= D)
                break;
            float dn = 0.f, up = 0.f;      // N_d, P_d
            auto add = [&](float v) {
                dn += v != v ? v : fminf(v, 0.f);
                up += v != v ? v : fmaxf(v, 0.f);
            };
#pragma unroll
            for (int q = 0; q < GS; ++q)
                add(query(p, raw[k][q]));  // (0 past the last head)
            for (int q = GS; q < G; ++q)
                add(query(p, query_raw(p, head0, q, D, d)));
            mag += fabsf(dn) + fabsf(up);
#pragma unroll
            for (int i = 0; i < 3; ++i) {
                const __nv_bfloat16 x = __float2bfloat16_rn(dn), y = __float2bfloat16_rn(up);
                wt[i][d] = __bfloat16_as_ushort(x);
                wt[i][D + d] = __bfloat16_as_ushort(y);
                dn -= __bfloat162float(x);
                up -= __bfloat162float(y);
            }
        }
        bad |= at < 0;
        load(at, 0);
#pragma unroll
        for (int o = 16; o > 0; o >>= 1)
            mag += __shfl_xor_sync(0xffffffffu, mag, o);
        if (lane == 0)
            warp_w[warp] = mag;
        __syncthreads();

        uint32_t top[4] = {0u, 0u, 0u, 0u};   // largest magnitudes, bfloat16 pairs (signs mixed up)
        float low = INFINITY, high = -INFINITY;   // of the scores that are not forced
        for (int base = j0 + 16 * warp; base < j1; base += STEP) {
            float d[4][4] = {};
#pragma unroll
            for (int i0 = 0; i0 < LOADS; i0 += H) {
#pragma unroll
                for (int i = 0; i < H; ++i) {
                    uint4 w = make_uint4(0u, 0u, 0u, 0u);
                    if (g < 3)
                        w = *reinterpret_cast<const uint4 *>(&wt[g][32 * (i0 + i) + 8 * t]);
                    const uint4 a = xa[i], c = xb[i];
                    mma_bf16(d[(2 * i) & 3], a.x, c.x, a.y, c.y, w.x, w.y);
                    mma_bf16(d[(2 * i + 1) & 3], a.z, c.z, a.w, c.w, w.z, w.w);
                    raise(top[0], a.x); raise(top[1], a.y); raise(top[2], a.z); raise(top[3], a.w);
                    raise(top[0], c.x); raise(top[1], c.y); raise(top[2], c.z); raise(top[3], c.w);
                }
                if (i0 + H < LOADS) {
                    load(at, i0 + H);
                } else if (base + STEP < j1) {
                    at = at_next;
                    bad |= at < 0;
                    at_next = place(base + 2 * STEP);
                    load(at, 0);
                }
            }
            // columns 0, 1 are in lanes t = 0, column 2 in lanes t = 1
            float s[2];
#pragma unroll
            for (int i = 0; i < 2; ++i) {
                s[i] = (d[0][2 * i] + d[1][2 * i]) + (d[2][2 * i] + d[3][2 * i]);
                const float m = (d[0][2 * i + 1] + d[1][2 * i + 1]) + (d[2][2 * i + 1] + d[3][2 * i + 1]);
                s[i] += m + __shfl_down_sync(0xffffffffu, s[i], 1);
                const int j = base + g + 8 * i;
                if (t == 0 && j < j1) {
                    const bool f = j < p.n_first || j >= n - p.n_last;
                    out[j] = f ? kForced : key32(s[i]);
                    if (!f) {
                        low = fminf(low, s[i]);
                        high = fmaxf(high, s[i]);
                    }
                }
            }
        }
        raise(top[0], top[1]);
        raise(top[2], top[3]);
        raise(top[0], top[2]);
        float a = fmaxf(fabsf(bf16_lo(top[0])), fabsf(bf16_hi(top[0])));
#pragma unroll
        for (int o = 16; o > 0; o >>= 1) {
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
            low = fminf(low, __shfl_xor_sync(0xffffffffu, low, o));
            high = fmaxf(high, __shfl_xor_sync(0xffffffffu, high, o));
        }
        if (lane == 0) {
            warp_top[warp] = a;
            warp_key[0][warp] = __float_as_uint(low);
            warp_key[1][warp] = __float_as_uint(high);
        }
        const int bad_any = __syncthreads_or(bad);
        if (tid == 0) {
            for (int i = 1; i < NW; ++i) {
                a = fmaxf(a, warp_top[i]);
                low = fminf(low, __uint_as_float(warp_key[0][i]));
                high = fmaxf(high, __uint_as_float(warp_key[1][i]));
            }
            *cl.map_shared_rank(&err[rank], 0) = a;
            *cl.map_shared_rank(&any_bad[rank], 0) = bad_any;
            *cl.map_shared_rank(&range[rank][0], 0) = low;
            *cl.map_shared_rank(&range[rank][1], 0) = high;
        }
    }
    // the scores are in the leader's shared memory
    if (ranks > 1)
        cl.sync();
    else
        __syncthreads();
    if (rank != 0)
        return;

    Sums<NT> sum = {cells, 0};
    float lo = -INFINITY, hi = INFINITY;
    int mode = 0;                          // 0: all; 1: score >= lo; 2: and those between by their 64-bit keys
    unsigned long long thr64 = 0;
    int take = 0;                          // mode 2: how many of those equal to thr64 are kept
    if (all) {
        // every valid block; a bad block is found here
        bool bad = false;
        for (int j = tid; j < n; j += NT)
            bad |= pool_block(p, b, h, r, j) < 0;
        if (__syncthreads_or(bad))
            bits |= kBadBlock;
    } else {
        float amax = err[0], low = range[0][0], high = range[0][1];
        bits |= any_bad[0] ? kBadBlock : 0;
        for (int i = 1; i < ranks; ++i) {
            amax = fmaxf(amax, err[i]);
            low = fminf(low, range[i][0]);
            high = fmaxf(high, range[i][1]);
            bits |= any_bad[i] ? kBadBlock : 0;
        }
        const int need = p.n_select;       // more than the forced blocks?
        const int forced = min(n, p.n_first) + p.n_last;
        mode = 1;
        if (need <= forced) {
            lo = hi = INFINITY;            // only those
        } else {
            // The need-th largest score T: a cut into bins, equal steps of
            // the scores' range (any map that keeps their order does), finds
            // the bin that T is in; its few members are ranked. A bin with
            // many of them, or scores that are not finite: bit by bit.
            const float step = (float)kBins / (high - low);
            auto bin = [&](float s) { return min(kBins - 1, (int)((s - low) * step)); };
            const bool finite = high - low < INFINITY && step < INFINITY;
            int odd = 0;                   // NaN scores (low and high do not show them)
            if (finite)
                for (int j = tid; j < n; j += NT) {
                    const uint32_t k = key[j];
                    if (k == kForced - 1)
                        odd = 1;
                    else if (k != kForced)
                        atomicAdd(&bins[bin(unkey32(k))], 1);
                }
            odd = __syncthreads_or(odd);
            float T = 0.f;
            bool have = false;
            if (finite && !odd) {
                // scores in the bins above this thread's (from the top: 0, 1, ..)
                constexpr int PER = kBins / NT;
                int mine[PER], own = 0;
#pragma unroll
                for (int i = 0; i < PER; ++i)
                    own += mine[i] = bins[kBins - 1 - (tid * PER + i)];
                int incl = own;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int x = __shfl_up_sync(0xffffffffu, incl, o);
                    if (lane >= o)
                        incl += x;
                }
                if (lane == 31)
                    scan[warp] = incl;
                __syncthreads();
                int before = forced + incl - own;
                for (int i = 0; i < warp; ++i)
                    before += scan[i];
#pragma unroll
                for (int i = 0; i < PER; ++i) {
                    if (before < need && before + mine[i] >= need) {
                        found[0] = kBins - 1 - (tid * PER + i);
                        found[1] = before;
                    }
                    before += mine[i];
                }
                __syncthreads();
                const int at_bin = found[0], rest = need - found[1];   // T is the rest-th of its bin
                const int members = bins[at_bin];
                if (members <= kFew) {
                    for (int j = tid; j < n; j += NT) {
                        const uint32_t k = key[j];
                        if (k != kForced && bin(unkey32(k)) == at_bin)
                            few[atomicAdd(&n_few, 1)] = j;
                    }
                    __syncthreads();
                    if (tid == 0)
                        n_few = 0;         // for the next list (behind the barrier below)
                    for (int i = tid; i < members; i += NT) {
                        const uint32_t k = key[few[i]];
                        int above = 0, same = 0;
                        for (int q = 0; q < members; ++q) {
                            const uint32_t x = key[few[q]];
                            above += x > k;
                            same += x == k;
                        }
                        if (above < rest && above + same >= rest)
                            warp_key[0][0] = k;    // (equal keys write the same)
                    }
                    __syncthreads();
                    T = unkey32(warp_key[0][0]);
                    have = true;
                }
            }
            if (!have) {
                const uint32_t thr = nth_largest(key, n, need, sum);
                uint32_t least = kForced;  // the smallest key that reaches it
                for (int j = tid; j < n; j += NT)
                    if (key[j] >= thr)
                        least = min(least, key[j]);
                least = __reduce_min_sync(0xffffffffu, least);
                if (lane == 0)
                    warp_key[1][warp] = least;
                __syncthreads();
                for (int i = 0; i < NW; ++i)
                    least = min(least, warp_key[1][i]);
                T = unkey32(least);
            }
            // sum_d |w_d| |x_d| of any block is at most M, the sum of |w| times
            // the largest |x|. In units of 2^-24 of M: a matrix step aligns its
            // 16 products and the sum so far to the largest of them and cuts
            // each below 2^-25 of its power of two (as measured: 16 products of
            // 0.498 units beside 1 add nothing, 16 of 0.996 add 8), 17 halves,
            // and cuts its result to 24 bits, 2 more: 10.5. A sum takes E / 64
            // steps, and the four sums side by side share M. Joining the sums,
            // the weights' third parts and the group's queries: 8 + G. 1.1
            // covers higher orders (the second parts' sums, 2^-8 of these); a
            // weight near float32's smallest loses its low parts
            float wsum = 0.f;
            for (int i = 0; i < NW; ++i)
                wsum += warp_w[i];
            // where a part of a sum may have left float32's range (or a NaN is
            // met), the 64-bit sums of all of them decide
            const float most = wsum * amax;
            const float e = most < 1e38f ? 1.1f * (float)(21 * E / 128 + 8 + G) * 5.9604645e-8f * most + 2e-37f * amax : INFINITY;
            lo = T - 2.f * e;
            hi = T + 2.f * e;
            // one rounding of each border outwards
            lo -= fabsf(lo) * 1.2e-7f;
            hi += fabsf(hi) * 1.2e-7f;
            int above = 0, between = 0;
            for (int j = tid; j < n; j += NT) {
                const uint32_t k = key[j];
                const float s = unkey32(k);
                if (k == kForced || s > hi) {
                    ++above;
                } else if (!(s < lo)) {
                    ++between;
                    const int i = atomicAdd(&n_few, 1);
                    if (i < kFew)
                        few[i] = j;
                }
            }
            const int both = sum(above | (between << 16));
            above = both & 0xffff;
            between = (int)((unsigned)both >> 16);
            if (above + between != need) {
                mode = 2;
                take = need - above;
                // the elements of a block that this lane sums, and the sum of all
                using Part = __nv_bfloat16[E / 32];
                auto fetch = [&](int a, Part &x) {
                    const __nv_bfloat16 *v = static_cast<const __nv_bfloat16 *>(p.bounds) + (long long)max(0, a) * E;
#pragma unroll
                    for (int d = 0; d < E / 32; ++d)
                        x[d] = v[32 * d + lane];
                };
                auto total = [&](const Part &x) {
                    double acc = 0.0;
#pragma unroll
                    for (int d = 0; d < E / 32; ++d)
                        acc += wt64[32 * d + lane] * (double)__bfloat162float(x[d]);
#pragma unroll
                    for (int o = 16; o > 0; o >>= 1)
                        acc += __shfl_xor_sync(0xffffffffu, acc, o);
                    return key64_of(acc + 0.0);
                };
                // dealt out to the warps, their places looked up at once and
                // the next one's elements loaded beside a sum
                Part x;
                const int c = warp + NW * lane;
                const int a = c < min(between, kFew) ? pool_block(p, b, h, r, few[c]) : 0;
                fetch(__shfl_sync(0xffffffffu, a, 0), x);
                // the weights in 64 bits
                for (int d = tid; d < D; d += NT) {
                    double dn = 0.0, up = 0.0;
#pragma unroll 8
                    for (int q = 0; q < G; ++q) {
                        const float v = query(p, query_raw(p, head0, q, D, d));
                        dn += v != v ? (double)v : (double)fminf(v, 0.f);
                        up += v != v ? (double)v : (double)fmaxf(v, 0.f);
                    }
                    wt64[d] = dn;
                    wt64[D + d] = up;
                }
                __syncthreads();
                if (between <= kFew) {
                    for (int i = warp, l = 1; i < between; i += NW, ++l) {
                        Part y;
                        fetch(__shfl_sync(0xffffffffu, a, l & 31), y);
                        const unsigned long long k = total(x);
                        if (lane == 0)
                            key64[few[i]] = k;
#pragma unroll
                        for (int d = 0; d < E / 32; ++d)
                            x[d] = y[d];
                    }
                } else {
                    for (int base = warp * 32; base < n; base += NT) {
                        const int j = base + lane;
                        const float s = j < n ? unkey32(key[j]) : 0.f;
                        const bool is = j < n && key[j] != kForced && !(s > hi) && !(s < lo);
                        const int a = is ? pool_block(p, b, h, r, j) : 0;
                        if (j < n)
                            key64[j] = 0;  // not in between (no score has this key)
                        __syncwarp();
                        for (unsigned left = __ballot_sync(0xffffffffu, is); left; left &= left - 1) {
                            const int l = __ffs(left) - 1;
                            fetch(__shfl_sync(0xffffffffu, a, l), x);
                            const unsigned long long k = total(x);
                            if (lane == 0)
                                key64[base + l] = k;
                        }
                    }
                }
                __syncthreads();
                if (between <= kFew) {
                    // each one's rank by comparing it with the others (the
                    // list's order does not matter); the last one kept sets
                    // the threshold
                    for (int i = tid; i < between; i += NT) {
                        const int j = few[i];
                        const unsigned long long y = key64[j];
                        int before = 0, equal = 0;
                        for (int q = 0; q < between; ++q) {
                            const unsigned long long x = key64[few[q]];
                            before += x > y || (x == y && few[q] < j);
                            equal += x == y && few[q] <= j;
                        }
                        if (before == take - 1) {
                            found[0] = j;
                            found[1] = equal;
                        }
                    }
                    __syncthreads();
                    thr64 = key64[found[0]];
                    take = found[1];
                } else {
                    thr64 = nth_largest(key64, n, take, sum);
                    int over = 0;
                    for (int j = tid; j < n; j += NT)
                        over += key64[j] > thr64;
                    take -= sum(over);
                }
            }
        }
    }
    const long long row = (long long)unit * p.n_select;
    if (bits) {
        if (tid == 0) {
            if (p.status && h == 0)
                atomicOr(p.status, bits);
            p.sel_lengths[unit] = 0;
        }
        for (int i = tid; i < p.n_select; i += NT)
            p.ids[row + i] = p.table[row + i] = -1;
        return;
    }
    const int total = min(n, p.n_select);
    int *list = reinterpret_cast<int *>(key64);
    if (!all) {
        // the kept blocks in ascending order: each thread a stretch of the
        // blocks (an odd number: its words lie in different banks)
        const int per = (n + NT - 1) / NT | 1;
        const int c0 = min(n, tid * per), c1 = min(n, c0 + per);
        // 2: kept, 1: kept if among the first `take` of its equals, 0: not
        auto state = [&](int j) {
            if (key[j] == kForced)
                return 2;
            const float s = unkey32(key[j]);
            if (mode == 1)
                return !(s < lo) && lo < INFINITY ? 2 : 0;
            if (s > hi || s < lo)
                return s > hi ? 2 : 0;
            return key64[j] > thr64 ? 2 : key64[j] == thr64 ? 1 : 0;
        };
        int mine = 0;                      // kept | ties << 16
        for (int j = c0; j < c1; ++j) {
            const int k = state(j);
            key[j] = k;
            mine += k == 2 ? 1 : k << 16;
        }
        int incl = mine;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
        __syncthreads();                   // (the bins' use of scan, and key64, are over)
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int before = incl - mine;
        for (int i = 0; i < warp; ++i)
            before += scan[i];
        int ties = (int)((unsigned)before >> 16), at = (before & 0xffff) + min(ties, take);
        for (int j = c0; j < c1; ++j) {
            const int k = (int)key[j];
            if ((k == 2 || (k == 1 && ties < take)) && at < total)
                list[at++] = j;
            ties += k == 1;
        }
        __syncthreads();
    }
    for (int i = tid; i < p.n_select; i += NT) {
        const int j = i >= total ? -1 : all ? i : list[i];
        p.ids[row + i] = j;
        p.table[row + i] = j < 0 ? -1 : pool_block(p, b, h, r, j);
    }
    if (tid == 0)
        p.sel_lengths[unit] = (total - 1) * p.block_size + (len - (n - 1) * p.block_size);
}

template <int D, int NT>
cudaError_t launch_one(const SelectParams &p, int c, cudaStream_t st)
{
    static std::atomic<uint64_t> ready;    // devices whose attribute is set, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(select_kernel<D, NT>, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kMaxBlocks);
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(p.B * p.Hkv * c);
    cfg.blockDim = dim3(NT);
    cfg.dynamicSmemBytes = 12 * (size_t)p.NB;
    cfg.stream = st;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = c;
    attr[1].val.clusterDim.y = 1;
    attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 2;
    return cudaLaunchKernelEx(&cfg, select_kernel<D, NT>, p);
}

template <int D>
cudaError_t launch_d(const SelectParams &p, int sms, cudaStream_t st)
{
    const int units = p.B * p.Hkv;
    if (units > 2 * sms)
        return launch_one<D, 128>(p, 1, st);
    // CTAs a unit: enough to give every SM two, each with 16 blocks for its warps
    int c = 1;
    while (c < kMaxCluster && (long long)units * c * 2 <= 2LL * sms && p.NB >= 2 * 16 * 8 * c)
        c *= 2;
    return launch_one<D, 256>(p, c, st);
}

}  // namespace

bool select_supports(int D, int NB) { return (D == 64 || D == 128 || D == 256) && NB >= 1 && NB <= kMaxBlocks; }

cudaError_t select_launch(const SelectParams &p, int sms, cudaStream_t st)
{
    if (p.D == 64)
        return launch_d<64>(p, sms, st);
    if (p.D == 128)
        return launch_d<128>(p, sms, st);
    return launch_d<256>(p, sms, st);
}

}  // namespace gqa
