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
// (adds in a row) 2^-24 sum_d |w_d| max_j |x_jd| over the unit's blocks; with T
// the n-th largest float32 score, a score above T + 2 E is kept and one below
// T - 2 E is not, whatever the rounding. The few in between, when they do not
// all fit, are summed again in 64 bits and ordered by that.
#include <cooperative_groups.h>

#include <atomic>

#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 256;
constexpr int kWarps = kThreads / 32;
constexpr int kFew = 64;            // candidates ordered by comparing each with each
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

// Sums over the block, one after the other: each takes a counter of its own
// (zero before), so a sum costs one barrier.
struct Sums {
    int *cell;
    __device__ __forceinline__ int operator()(int v)
    {
        v = __reduce_add_sync(0xffffffffu, v);
        if ((threadIdx.x & 31) == 0)
            atomicAdd(cell, v);
        __syncthreads();
        return *cell++;
    }
};
constexpr int kSums = 32 + 64 + 8;

// The n-th largest (n >= 1) of the keys key[0 .. m - 1] (in shared memory) is
// the smallest key that reaches the value returned: the value is found bit by
// bit from the top, and its low bits are left at zero once exactly n keys
// reach it. `at`, with all bits from `bit` up decided, is where to start.
template <typename K>
__device__ K nth_largest(const K *key, int m, int n, K at, int bit, Sums &sum)
{
    for (; bit >= 0; --bit) {
        const K cand = at | ((K)1 << bit);
        int c = 0;
        for (int j = threadIdx.x; j < m; j += kThreads)
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

__device__ __forceinline__ uint4 load8(const void *bounds, long long off)
{
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(bounds) + off));
}

// Element d of query head g of the unit.
__device__ __forceinline__ float query(const SelectParams &p, long long head0, int g, int D, int d)
{
    const long long at = (head0 + g) * D + d;
    return p.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at])
                    : static_cast<const float *>(p.q)[at];
}

template <int D>
__global__ void __launch_bounds__(kThreads, 4) select_kernel(const SelectParams p)
{
    constexpr int E = 2 * D;               // elements of a block's bounds: lo, then hi
    constexpr int LPB = E / 8 > 32 ? 32 : E / 8;   // lanes that share a block
    constexpr int V = E / 8 / LPB;         // 16-byte loads a lane
    constexpr int BPW = 32 / LPB;          // blocks a warp takes at once
    constexpr int U = 8 / V;               // and this many times before it sums
    constexpr int STEP = BPW * U;          // blocks of a warp's step: 8 (D = 64: 16, D = 256: 4)
    extern __shared__ __align__(16) unsigned char smem[];
    unsigned long long *key64 = reinterpret_cast<unsigned long long *>(smem);   // [NB]: keys of the 64-bit scores
    uint32_t *key = reinterpret_cast<uint32_t *>(key64 + p.NB);                 // [NB] (leader)
    __shared__ __align__(16) float wt[E];  // N_d, then P_d
    __shared__ int cells[kSums];
    __shared__ float warp_top[kWarps];
    __shared__ uint32_t warp_key[2][kWarps];
    __shared__ float err[kMaxCluster];
    __shared__ int any_bad[kMaxCluster];
    __shared__ int scan[kWarps];
    __shared__ int few[kFew], n_few;

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
    const int r = p.paged ? 0 : (p.slot_ids ? __ldg(p.slot_ids + b) : b);
    int bits = 0;
    if (len < 1 || (long long)len > (long long)p.NB * p.block_size)
        bits = kBadLength;
    else if (!p.paged && (r < 0 || r >= p.R))
        bits = kBadSlotId;
    const int n = bits ? 0 : (len + p.block_size - 1) / p.block_size;   // valid blocks
    const bool all = n <= p.n_select;
    if (rank == 0) {
        for (int i = tid; i < kSums; i += kThreads)
            cells[i] = 0;
        if (tid == 0)
            n_few = 0;
    }
    // the leader's shared memory is written to below: every CTA must have started
    if (ranks > 1)
        cl.sync();

    if (!all) {
        for (int d = tid; d < D; d += kThreads) {
            float up = 0.f, dn = 0.f;
#pragma unroll 8
            for (int g = 0; g < G; ++g) {
                const float x = query(p, head0, g, D, d);
                up += x != x ? x : fmaxf(x, 0.f);
                dn += x != x ? x : fminf(x, 0.f);
            }
            wt[d] = dn;
            wt[D + d] = up;
        }
        __syncthreads();
        const int li = lane % LPB, lb = lane / LPB;
        float w[V][8];
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 8; ++i)
                w[v][i] = wt[(v * LPB + li) * 8 + i];
        uint32_t top[V][4];                // largest |x| of the lane's elements, bfloat16 pairs
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                top[v][i] = 0u;
        uint32_t *out = cl.map_shared_rank(key, 0);
        const int j0 = (int)((long long)n * rank / ranks), j1 = (int)((long long)n * (rank + 1) / ranks);
        bool bad = false;
        // a warp takes 32 blocks at a time: their places first (one lane
        // each, those of the next 32 while these are scored)
        int at_next = j0 + 32 * warp + lane < j1 ? pool_block(p, b, h, r, j0 + 32 * warp + lane) : 0;
        for (int base = j0 + 32 * warp; base < j1; base += 32 * kWarps) {
            const int at = at_next;
            bad |= at < 0;
            const int jn = base + 32 * kWarps + lane;
            at_next = jn < j1 ? pool_block(p, b, h, r, jn) : 0;
#pragma unroll 1
            for (int sub = 0; sub < 32 && base + sub < j1; sub += STEP) {
                uint4 x[U][V];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    // block lb * U + u of the step
                    const int a = __shfl_sync(0xffffffffu, at, sub + lb * U + u);
                    const bool in = a >= 0 && base + sub + lb * U + u < j1;
#pragma unroll
                    for (int v = 0; v < V; ++v)
                        x[u][v] = in ? load8(p.bounds, (long long)a * E + (v * LPB + li) * 8) : make_uint4(0u, 0u, 0u, 0u);
                }
                float s[U];
#pragma unroll
                for (int u = 0; u < U; ++u) {
                    s[u] = 0.f;
#pragma unroll
                    for (int v = 0; v < V; ++v) {
                        const uint32_t q[4] = {x[u][v].x, x[u][v].y, x[u][v].z, x[u][v].w};
#pragma unroll
                        for (int i = 0; i < 4; ++i) {
                            s[u] = fmaf(w[v][2 * i], bf16_lo(q[i]), s[u]);
                            s[u] = fmaf(w[v][2 * i + 1], bf16_hi(q[i]), s[u]);
                            asm("max.bf16x2 %0, %1, %2;" : "=r"(top[v][i]) : "r"(top[v][i]), "r"(q[i] & 0x7fff7fffu));
                        }
                    }
                }
                // sums over the block's lanes: while there are several
                // blocks, half of the lanes go on with half of them
                int o = LPB / 2, mine = 0;
#pragma unroll
                for (int m = U; m > 1; m /= 2) {
                    const bool up = lane & o;
#pragma unroll
                    for (int u = 0; u < m / 2; ++u) {
                        const float keep = up ? s[u + m / 2] : s[u], send = up ? s[u] : s[u + m / 2];
                        s[u] = keep + __shfl_xor_sync(0xffffffffu, send, o);
                    }
                    mine = 2 * mine + (up ? 1 : 0);
                    o /= 2;
                }
                const bool writes = (lane & (2 * o - 1)) == 0;
#pragma unroll
                for (int q = LPB / 2 / U; q > 0; q /= 2)
                    s[0] += __shfl_xor_sync(0xffffffffu, s[0], q);
                const int jj = base + sub + lb * U + mine;
                if (writes && jj < j1)
                    out[jj] = (jj < p.n_first || jj >= n - p.n_last) ? kForced : key32(s[0]);
            }
        }
        // sum_d |w_d| max |x_d| over this CTA's blocks: no block's sum of
        // magnitudes is larger
        float a = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a += fabsf(w[v][2 * i]) * bf16_lo(top[v][i]) + fabsf(w[v][2 * i + 1]) * bf16_hi(top[v][i]);
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1)
            a += __shfl_xor_sync(0xffffffffu, a, o);
#pragma unroll
        for (int o = LPB; o < 32; o <<= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        if (lane == 0)
            warp_top[warp] = a;
        const int bad_any = __syncthreads_or(bad);
        if (tid == 0) {
            for (int i = 1; i < kWarps; ++i)
                a = fmaxf(a, warp_top[i]);
            *cl.map_shared_rank(&err[rank], 0) = a;
            *cl.map_shared_rank(&any_bad[rank], 0) = bad_any;
        }
    }
    // the scores are in the leader's shared memory
    if (ranks > 1)
        cl.sync();
    else
        __syncthreads();
    if (rank != 0)
        return;

    Sums sum = {cells};
    float lo = -INFINITY, hi = INFINITY;
    int mode = 0;                          // 0: all; 1: score >= lo; 2: and those between by their 64-bit keys
    unsigned long long thr64 = 0;
    int take = 0;                          // mode 2: how many of those equal to thr64 are kept
    if (all) {
        // every valid block; a bad block is found here
        bool bad = false;
        for (int j = tid; j < n; j += kThreads)
            bad |= pool_block(p, b, h, r, j) < 0;
        if (__syncthreads_or(bad))
            bits |= kBadBlock;
    } else {
        float amax = err[0];
        for (int i = 0; i < ranks; ++i) {
            amax = fmaxf(amax, err[i]);
            if (any_bad[i])
                bits |= kBadBlock;
        }
        // the bits in which the keys (but the forced ones) differ
        uint32_t low = kForced, high = 0;
        for (int j = tid; j < n; j += kThreads) {
            const uint32_t k = key[j];
            if (k != kForced) {
                low = min(low, k);
                high = max(high, k);
            }
        }
        low = __reduce_min_sync(0xffffffffu, low);
        high = __reduce_max_sync(0xffffffffu, high);
        if (lane == 0) {
            warp_key[0][warp] = low;
            warp_key[1][warp] = high;
        }
        __syncthreads();
        for (int i = 0; i < kWarps; ++i) {
            low = min(low, warp_key[0][i]);
            high = max(high, warp_key[1][i]);
        }
        const int need = p.n_select;       // more than the forced blocks?
        const int forced = min(n, p.n_first) + p.n_last;
        mode = 1;
        if (need <= forced) {
            lo = hi = INFINITY;            // only those
        } else {
            // all of them share the bits above the first that low and high differ in
            const int bit = low == high ? -1 : 31 - __clz(low ^ high);
            const uint32_t start = bit < 0 ? low : bit == 31 ? 0u : low & ~((2u << bit) - 1u);
            const uint32_t thr = nth_largest(key, n, need, start, bit, sum);
            uint32_t least = kForced;      // the smallest key that reaches it
            for (int j = tid; j < n; j += kThreads)
                if (key[j] >= thr)
                    least = min(least, key[j]);
            least = __reduce_min_sync(0xffffffffu, least);
            __syncthreads();
            if (lane == 0)
                warp_key[0][warp] = least;
            __syncthreads();
            for (int i = 0; i < kWarps; ++i)
                least = min(least, warp_key[0][i]);
            // adds in a row: a lane's products, the lanes of a block, the
            // group's queries; 1.1 covers the higher orders and amax's rounding
            const float e = 1.1f * (float)(8 * V + 8 + G) * 5.9604645e-8f * amax;
            const float T = unkey32(least);
            lo = T - 2.f * e;
            hi = T + 2.f * e;
            // one rounding of each border outwards
            lo -= fabsf(lo) * 1.2e-7f;
            hi += fabsf(hi) * 1.2e-7f;
            int above = 0, between = 0;
            for (int j = tid; j < n; j += kThreads) {
                const uint32_t k = key[j];
                const float s = unkey32(k);
                const bool f = k == kForced;
                above += f || s > hi;
                between += !f && !(s > hi) && !(s < lo);
            }
            above = sum(above);
            between = sum(between);
            if (above + between != need) {
                mode = 2;
                take = need - above;
                // 64-bit sums of the blocks in between, a warp each
                for (int j0 = warp * 32; j0 < n; j0 += kThreads) {
                    const int j = j0 + lane;
                    const float s = j < n ? unkey32(key[j]) : 0.f;
                    const bool is = j < n && key[j] != kForced && !(s > hi) && !(s < lo);
                    if (j < n)
                        key64[j] = 0;      // not in between (no score has this key)
                    __syncwarp();
                    for (unsigned left = __ballot_sync(0xffffffffu, is); left; left &= left - 1) {
                        const int jj = j0 + __ffs(left) - 1;
                        const int at = pool_block(p, b, h, r, jj);
                        double acc = 0.0;
                        if (at >= 0) {
                            const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.bounds) + (long long)at * E;
                            for (int d = lane; d < D; d += 32) {
                                double up = 0.0, dn = 0.0;
                                for (int g = 0; g < G; ++g) {
                                    const float v = query(p, head0, g, D, d);
                                    up += v != v ? (double)v : (double)fmaxf(v, 0.f);
                                    dn += v != v ? (double)v : (double)fminf(v, 0.f);
                                }
                                acc += dn * (double)__bfloat162float(x[d]) + up * (double)__bfloat162float(x[D + d]);
                            }
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            acc += __shfl_xor_sync(0xffffffffu, acc, o);
                        if (lane == 0) {
                            key64[jj] = key64_of(acc + 0.0);
                            const int at_few = atomicAdd(&n_few, 1);
                            if (at_few < kFew)
                                few[at_few] = jj;
                        }
                    }
                }
                __syncthreads();
                if (between <= kFew) {
                    // few: each one's rank by comparing it with the others
                    // (the list's order does not matter). The last one kept
                    // sets the threshold
                    for (int i = tid; i < between; i += kThreads) {
                        const int j = few[i];
                        int before = 0, equal = 0;
                        for (int k = 0; k < between; ++k) {
                            const unsigned long long x = key64[few[k]], y = key64[j];
                            before += x > y || (x == y && few[k] < j);
                            equal += x == y && few[k] <= j;
                        }
                        if (before == take - 1) {
                            scan[0] = j;
                            scan[1] = equal;
                        }
                    }
                    __syncthreads();
                    thr64 = key64[scan[0]];
                    take = scan[1];
                    __syncthreads();
                } else {
                    thr64 = nth_largest(key64, n, take, 0ull, 63, sum);
                    int over = 0;
                    for (int j = tid; j < n; j += kThreads)
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
        for (int i = tid; i < p.n_select; i += kThreads)
            p.ids[row + i] = p.table[row + i] = -1;
        return;
    }
    // the kept blocks in ascending order, kThreads blocks at a time
    int kept = 0, ties = 0;                // of the blocks before
    for (int j0 = 0; j0 < n; j0 += kThreads) {
        const int j = j0 + tid;
        bool over = false, tie = false;
        if (j < n) {
            if (mode == 0) {
                over = true;
            } else if (key[j] == kForced) {
                over = true;
            } else {
                const float s = unkey32(key[j]);
                if (mode == 1) {
                    over = !(s < lo) && lo < INFINITY;
                } else {
                    over = s > hi || key64[j] > thr64;
                    tie = !over && key64[j] == thr64;
                }
            }
        }
        // places among the kept: those over, and the first `take` ties
        const unsigned mo = __ballot_sync(0xffffffffu, over), mt = __ballot_sync(0xffffffffu, tie);
        __syncthreads();
        if (lane == 0)
            scan[warp] = __popc(mo) | (__popc(mt) << 16);
        __syncthreads();
        int before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < kWarps; ++i) {
            const int c = scan[i];
            before += i < warp ? c : 0;
            total += c;
        }
        const unsigned below = (1u << lane) - 1u;
        const int nt = ties + (before >> 16) + __popc(mt & below);    // ties before this block
        const int at = kept + (before & 0xffff) + __popc(mo & below) + min(max(0, take - ties), nt - ties);
        if ((over || (tie && nt < take)) && at < p.n_select) {
            p.ids[row + at] = j;
            p.table[row + at] = pool_block(p, b, h, r, j);
        }
        kept += (total & 0xffff) + min(max(0, take - ties), total >> 16);
        ties += total >> 16;
    }
    const int total = min(n, p.n_select);
    for (int i = total + tid; i < p.n_select; i += kThreads)
        p.ids[row + i] = p.table[row + i] = -1;
    if (tid == 0)
        p.sel_lengths[unit] = (total - 1) * p.block_size + (len - (n - 1) * p.block_size);
}

template <int D>
cudaError_t launch_d(const SelectParams &p, int sms, cudaStream_t st)
{
    const int units = p.B * p.Hkv;
    // CTAs a unit: enough to give every SM two, each with work for its warps
    int c = 1;
    while (c < kMaxCluster && (long long)units * c * 2 <= 2LL * sms && p.NB >= 64 * c)
        c *= 2;
    const size_t smem = 12 * (size_t)p.NB;
    static std::atomic<uint64_t> ready;    // devices whose attribute is set, a bit each
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(select_kernel<D>, cudaFuncAttributeMaxDynamicSharedMemorySize, 12 * kMaxBlocks);
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(units * c);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
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
    return cudaLaunchKernelEx(&cfg, select_kernel<D>, p);
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
