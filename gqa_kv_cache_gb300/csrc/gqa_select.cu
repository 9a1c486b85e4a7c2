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

constexpr int kThreads = 512;
constexpr int kWarps = kThreads / 32;
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
__device__ __forceinline__ unsigned long long key64(double x)
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

// Sum of v over the block; every thread gets it. `part`: kWarps + 1 ints.
__device__ __forceinline__ int block_sum(int v, int *part)
{
    v = __reduce_add_sync(0xffffffffu, v);
    __syncthreads();
    if ((threadIdx.x & 31) == 0)
        part[threadIdx.x >> 5] = v;
    __syncthreads();
    int s = 0;
#pragma unroll
    for (int w = 0; w < kWarps; ++w)
        s += part[w];
    return s;
}

// The n-th largest (n >= 1) of the keys key[0 .. m - 1] (in shared memory): the
// largest value that at least n keys reach, bit by bit from the top.
template <typename K>
__device__ K nth_largest(const K *key, int m, int n, int *part)
{
    K at = 0;
    for (int bit = 8 * (int)sizeof(K) - 1; bit >= 0; --bit) {
        const K cand = at | ((K)1 << bit);
        int c = 0;
        for (int j = threadIdx.x; j < m; j += kThreads)
            c += key[j] >= cand;
        c = block_sum(c, part);
        if (c >= n)
            at = cand;
        if (c == n)
            break;                     // cand splits the keys: no need of its low bits
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

// Eight bfloat16 pairs' worth of one lane: 8 elements at x.
__device__ __forceinline__ uint4 load8(const void *bounds, long long off)
{
    return __ldg(reinterpret_cast<const uint4 *>(static_cast<const __nv_bfloat16 *>(bounds) + off));
}

template <int D>
__global__ void __launch_bounds__(kThreads) select_kernel(const SelectParams p)
{
    constexpr int E = 2 * D;               // elements of a block's bounds: lo, then hi
    constexpr int LPB = E / 8 > 32 ? 32 : E / 8;   // lanes that share a block
    constexpr int V = E / 8 / LPB;         // 16-byte loads a lane
    constexpr int BPW = 32 / LPB;          // blocks a warp takes at once
    extern __shared__ __align__(16) unsigned char smem[];
    double *exact = reinterpret_cast<double *>(smem);                 // [NB]: scores in 64 bits, then their keys
    uint32_t *key = reinterpret_cast<uint32_t *>(exact + p.NB);       // [NB] (leader)
    __shared__ __align__(16) float wt[E];  // N_d, then P_d
    __shared__ int part[kWarps + 1];
    __shared__ float err[kMaxCluster];
    __shared__ int any_bad[kMaxCluster];
    __shared__ int scan[kWarps];

    cg::cluster_group cl = cg::this_cluster();
    const int rank = (int)cl.block_rank(), ranks = (int)cl.num_blocks();
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int unit = blockIdx.x / ranks;
    const int b = unit / p.Hkv, h = unit % p.Hkv;
    const int G = p.Hq / p.Hkv;

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
    // the leader's shared memory is written to below: every CTA must have started
    cl.sync();

    if (!all) {
        for (int d = tid; d < D; d += kThreads) {
            float up = 0.f, dn = 0.f;
            for (int g = 0; g < G; ++g) {
                const long long at = ((long long)b * p.Hq + (long long)h * G + g) * D + d;
                const float x = p.q_bf16 ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[at])
                                         : static_cast<const float *>(p.q)[at];
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
        constexpr int U = 4;               // blocks in flight per lane group
        for (int j = j0 + warp * BPW * U; j < j1; j += kWarps * BPW * U) {
            uint4 x[U][V];
#pragma unroll
            for (int u = 0; u < U; ++u) {
                const int jj = j + u * BPW + lb;
                const int at = jj < j1 ? pool_block(p, b, h, r, jj) : -1;
                if (jj < j1 && at < 0)
                    bad = true;
#pragma unroll
                for (int v = 0; v < V; ++v)
                    x[u][v] = at >= 0 ? load8(p.bounds, (long long)at * E + (v * LPB + li) * 8)
                                      : make_uint4(0u, 0u, 0u, 0u);
            }
#pragma unroll
            for (int u = 0; u < U; ++u) {
                float s = 0.f;
#pragma unroll
                for (int v = 0; v < V; ++v) {
                    const uint32_t q[4] = {x[u][v].x, x[u][v].y, x[u][v].z, x[u][v].w};
#pragma unroll
                    for (int i = 0; i < 4; ++i) {
                        s = fmaf(w[v][2 * i], bf16_lo(q[i]), s);
                        s = fmaf(w[v][2 * i + 1], bf16_hi(q[i]), s);
                        asm("max.bf16x2 %0, %1, %2;" : "=r"(top[v][i]) : "r"(top[v][i]), "r"(q[i] & 0x7fff7fffu));
                    }
                }
#pragma unroll
                for (int o = LPB / 2; o > 0; o >>= 1)
                    s += __shfl_xor_sync(0xffffffffu, s, o);
                const int jj = j + u * BPW + lb;
                if (li == 0 && jj < j1)
                    out[jj] = (jj < p.n_first || jj >= n - p.n_last) ? kForced : key32(s);
            }
        }
        // sum_d |w_d| max |x_d| over this CTA's blocks (the largest of its warps' sums
        // of products is below the sum over the largest elements)
        float a = 0.f;
#pragma unroll
        for (int v = 0; v < V; ++v)
#pragma unroll
            for (int i = 0; i < 4; ++i)
                a += fabsf(w[v][2 * i]) * bf16_lo(top[v][i]) + fabsf(w[v][2 * i + 1]) * bf16_hi(top[v][i]);
#pragma unroll
        for (int o = LPB / 2; o > 0; o >>= 1)
            a += __shfl_xor_sync(0xffffffffu, a, o);
        float *ws = reinterpret_cast<float *>(part);
#pragma unroll
        for (int o = LPB; o < 32; o <<= 1)
            a = fmaxf(a, __shfl_xor_sync(0xffffffffu, a, o));
        const int bad_any = __syncthreads_or(bad);
        if (lane == 0)
            ws[warp] = a;
        __syncthreads();
        if (tid == 0) {
            for (int i = 1; i < kWarps; ++i)
                a = fmaxf(a, ws[i]);
            *cl.map_shared_rank(&err[rank], 0) = a;
            *cl.map_shared_rank(&any_bad[rank], 0) = bad_any;
        }
    }
    cl.sync();                             // the scores are in the leader's shared memory
    if (rank != 0)
        return;

    int need = p.n_select;                 // blocks to keep
    uint32_t thr = 0;                      // keep: key > thr, and of key == thr those below `ties`
    float lo = -INFINITY, hi = INFINITY;
    int mode = 0;                          // 0: all; 1: score >= lo; 2: and those between by their 64-bit keys
    unsigned long long thr64 = 0;
    int take = 0;                          // mode 2: how many equal to thr64 are kept
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
        thr = nth_largest(key, n, need, part);
        // adds in a row: a lane's products, the lanes of a block, the group's
        // queries; 1.1 covers the higher orders and the rounding of amax
        const float e = 1.1f * (float)(8 * V + 8 + G) * 5.9604645e-8f * amax;
        // (nth_largest may stop above the smallest kept key's low bits: the
        // threshold is the smallest key that reaches it)
        uint32_t least = kForced;
        for (int j = tid; j < n; j += kThreads)
            if (key[j] >= thr)
                least = min(least, key[j]);
        least = __reduce_min_sync(0xffffffffu, least);
        __syncthreads();
        if (lane == 0)
            part[warp] = (int)least;
        __syncthreads();
        for (int i = 0; i < kWarps; ++i)
            least = min(least, (uint32_t)part[i]);
        if (least == kForced) {            // only forced blocks fit
            lo = hi = INFINITY;
            mode = 1;
        } else {
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
            above = block_sum(above, part);
            between = block_sum(between, part);
            mode = 1;
            if (above + between != need) {
                mode = 2;
                take = need - above;
                // 64-bit sums of the blocks in between, a warp each
                for (int j = warp; j < n; j += kWarps) {
                    const float s = unkey32(key[j]);
                    unsigned long long k64 = 0;      // 0: not in between
                    if (key[j] != kForced && !(s > hi) && !(s < lo)) {
                        const int at = pool_block(p, b, h, r, j);
                        double acc = 0.0;
                        if (at >= 0) {
                            const __nv_bfloat16 *x = static_cast<const __nv_bfloat16 *>(p.bounds) + (long long)at * E;
                            for (int d = lane; d < D; d += 32) {
                                double up = 0.0, dn = 0.0;
                                for (int g = 0; g < G; ++g) {
                                    const long long qa = ((long long)b * p.Hq + (long long)h * G + g) * D + d;
                                    const float v = p.q_bf16
                                                        ? __bfloat162float(static_cast<const __nv_bfloat16 *>(p.q)[qa])
                                                        : static_cast<const float *>(p.q)[qa];
                                    up += v != v ? (double)v : (double)fmaxf(v, 0.f);
                                    dn += v != v ? (double)v : (double)fminf(v, 0.f);
                                }
                                acc += dn * (double)__bfloat162float(x[d]) + up * (double)__bfloat162float(x[D + d]);
                            }
                        }
#pragma unroll
                        for (int o = 16; o > 0; o >>= 1)
                            acc += __shfl_xor_sync(0xffffffffu, acc, o);
                        k64 = key64(acc + 0.0);
                    }
                    if (lane == 0)
                        reinterpret_cast<unsigned long long *>(exact)[j] = k64;
                }
                __syncthreads();
                thr64 = nth_largest(reinterpret_cast<unsigned long long *>(exact), n, take, part);
                // how many of the keys equal to the threshold are kept
                int over = 0;
                for (int j = tid; j < n; j += kThreads)
                    over += reinterpret_cast<unsigned long long *>(exact)[j] > thr64;
                take -= block_sum(over, part);
            }
        }
    }
    if (bits) {
        if (tid == 0) {
            if (p.status && h == 0)
                atomicOr(p.status, bits);
            p.sel_lengths[unit] = 0;
        }
        for (int i = tid; i < p.n_select; i += kThreads)
            p.ids[(long long)unit * p.n_select + i] = p.table[(long long)unit * p.n_select + i] = -1;
        return;
    }
    // the kept blocks in ascending order: each thread a stretch of them
    const int per = (n + kThreads - 1) / kThreads;
    const int c0 = min(n, tid * per), c1 = min(n, c0 + per);
    const unsigned long long *k64 = reinterpret_cast<const unsigned long long *>(exact);
    auto over = [&](int j) {               // kept whatever the ties
        if (mode == 0)
            return true;
        if (key[j] == kForced)
            return true;
        const float s = unkey32(key[j]);
        if (mode == 1)
            return !(s < lo) && lo < INFINITY;
        return s > hi || k64[j] > thr64;
    };
    auto tie = [&](int j) { return mode == 2 && key[j] != kForced && k64[j] == thr64; };
    int mine = 0, equal = 0;
    for (int j = c0; j < c1; ++j) {
        const bool o = over(j);
        mine += o;
        equal += !o && tie(j);
    }
    // exclusive prefix of (equal, kept) over the threads: equal first, since
    // how many of a thread's ties are kept depends on those before it
    auto prefix = [&](int v) {
        int incl = v;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int x = __shfl_up_sync(0xffffffffu, incl, o);
            if (lane >= o)
                incl += x;
        }
        __syncthreads();
        if (lane == 31)
            scan[warp] = incl;
        __syncthreads();
        int before = 0;
        for (int i = 0; i < warp; ++i)
            before += scan[i];
        return before + incl - v;
    };
    const int eq0 = prefix(equal);
    const int kept = mine + max(0, min(equal, take - eq0));
    int at = prefix(kept);
    int left = max(0, min(equal, take - eq0));
    const long long row = (long long)unit * p.n_select;
    for (int j = c0; j < c1; ++j) {
        bool k = over(j);
        if (!k && tie(j) && left > 0) {
            k = true;
            --left;
        }
        if (k && at < p.n_select) {
            p.ids[row + at] = j;
            p.table[row + at] = pool_block(p, b, h, r, j);
            ++at;
        }
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
