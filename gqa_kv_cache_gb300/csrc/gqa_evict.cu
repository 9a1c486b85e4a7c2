// Eviction: a row longer than n_keep slots keeps, for every cache head, its
// first n_first slots, its last n_last, and of the others those with the largest
// counts (ties to the lowest slot, NaN counts highest), in ascending order.
//
// evict_select_kernel, a CTA a (row, head): the counts as integers in order
// (sign folded, -0 as 0), the first kCached of them kept in shared memory; the
// smallest kept count by histograms of its first 11 bits, then of the next 11
// and 10 over the few that share the first (a list; all slots again where many
// do); then every warp counts and places the kept slots of its run. Bound by
// the instructions of these sweeps; a count is read from memory once where the
// row fits. The counts move in the same kernel.
//
// Kept vectors are copied elsewhere by evict_gather_kernel, every 16 bytes on
// their own, or within the cache by evict_compact_kernel. In place, kept slot i
// comes from a slot >= i; a CTA takes a column of 64 bytes of the vectors of
// a (row, head), chunk by chunk of kBytes: the sources of a later
// chunk lie behind the destinations of an earlier one, so copies into shared
// memory may run kDeep chunks ahead of the stores as long as a chunk is stored
// after it and those before it have come. Both are bound by memory: 2 rows of
// bytes a kept vector.
#include <cooperative_groups.h>

#include <atomic>

#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

namespace cg = cooperative_groups;

constexpr int kThreads = 512, kWarps = kThreads / 32;
constexpr int kCached = 15360;     // counts kept in shared memory (60 KB: three CTAs an SM)
constexpr int kCachedWide = 49152; // and by each CTA of a cluster (192 KB)
constexpr int kBins = 2048;
constexpr int kList = 1024;        // counts that share their first digit with the smallest kept one
constexpr int kEach = 4;           // counts a thread loads at once

__device__ __forceinline__ uint32_t order_of(float w)
{
    uint32_t u = __float_as_uint(w);
    if (w != w)
        return 0xffffffffu;
    u = u == 0x80000000u ? 0u : u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Where the vectors of a (row, head) lie (its blocks are known to be usable).
struct Line {
    const int32_t *table;
    long long first;   // dense: vector of slot 0
    int Hkv, h, block_size, shift;
    __device__ __forceinline__ Line(const EvictParams &p, int b, int head)
    {
        table = p.paged ? p.block_table + (long long)b * p.max_blocks : nullptr;
        Hkv = p.Hkv;
        h = head;
        block_size = p.block_size;
        shift = p.block_shift;
        first = 0;
        if (!p.paged)
            first = ((long long)(p.slot_ids ? __ldg(p.slot_ids + b) : b) * Hkv + h) * p.Smax;
    }
    __device__ __forceinline__ long long at(int j) const
    {
        if (!table)
            return first + j;
        if (shift >= 0)
            return (((long long)__ldg(table + (j >> shift)) * Hkv + h) << shift) + (j & ((1 << shift) - 1));
        return ((long long)__ldg(table + j / block_size) * Hkv + h) * block_size + j % block_size;
    }
    // N of them: the blocks are looked up side by side, ahead of their use
    template <int N>
    __device__ __forceinline__ void look_up(const int (&j)[N], int (&blk)[N]) const
    {
        if (!table)
            return;
#pragma unroll
        for (int e = 0; e < N; ++e)
            blk[e] = __ldg(table + (shift >= 0 ? j[e] >> shift : j[e] / block_size));
    }
    template <int N>
    __device__ __forceinline__ void place(const int (&j)[N], const int (&blk)[N], long long (&to)[N]) const
    {
#pragma unroll
        for (int e = 0; e < N; ++e)
            to[e] = !table       ? first + j[e]
                    : shift >= 0 ? (((long long)blk[e] * Hkv + h) << shift) + (j[e] & ((1 << shift) - 1))
                                 : ((long long)blk[e] * Hkv + h) * block_size + j[e] % block_size;
    }
};

// The digit of the k-th largest among the counted ones: hist[] is summed from
// the top. Every thread of the CTA calls it; returns the digit, k less the
// number above it, and the number that share it.
__device__ __forceinline__ int find_digit(const int *hist, int bins, int &k, int &equal, int *scan, int *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = bins / kThreads;   // bins a thread, from the top
    int mine = 0;
    for (int i = 0; i < per; ++i)
        mine += hist[bins - 1 - (tid * per + i)];
    int incl = mine;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int v = __shfl_up_sync(0xffffffffu, incl, o);
        if (lane >= o)
            incl += v;
    }
    if (lane == 31)
        scan[warp] = incl;
    __syncthreads();
    if (warp == 0) {
        int v = lane < kWarps ? scan[lane] : 0;
#pragma unroll
        for (int o = 1; o < kWarps; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += y;
        }
        if (lane < kWarps)
            scan[lane] = v;
    }
    __syncthreads();
    int above = incl - mine + (warp ? scan[warp - 1] : 0);
    if (above < k && above + mine >= k) {
        for (int i = 0; i < per; ++i) {
            const int bin = bins - 1 - (tid * per + i), c = hist[bin];
            if (above + c >= k) {
                found[0] = bin;
                found[1] = k - above;
                found[2] = c;
                break;
            }
            above += c;
        }
    }
    __syncthreads();
    k = found[1];
    equal = found[2];
    const int digit = found[0];
    __syncthreads();                           // before the next call's
    return digit;
}

constexpr int kMove = 256;         // threads of the moving kernels
constexpr int kPieces = 4;         // 16-byte pieces of K, and as many of V, a thread and step
constexpr int kSteps = 4;          // steps a CTA of the gathering kernel

// Pieces x0 .. end - 1 of a unit's kept vectors into the outputs, by THREADS
// threads. The places of the next step's vectors (ids, then blocks) are looked up
// while the vectors of this one are on their way.
template <int THREADS>
__device__ __forceinline__ void gather(const EvictParams &p, const Line &line, int unit, long long x0, long long end)
{
    const unsigned per = p.row_bytes / 16;     // pieces a vector
    const int shift = (per & (per - 1)) == 0 ? __ffs(per) - 1 : -1;
    const uint4 *ks = static_cast<const uint4 *>(p.k_cache), *vs = static_cast<const uint4 *>(p.v_cache);
    uint4 *kd = static_cast<uint4 *>(p.k_out) + (long long)unit * p.out_slots * per;
    uint4 *vd = static_cast<uint4 *>(p.v_out) + (long long)unit * p.out_slots * per;
    const int32_t *ids = p.ids + (long long)unit * p.n_keep;
    long long from[kPieces];
    auto find = [&](long long x) {
        int id[kPieces], blk[kPieces] = {};
        unsigned c[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; ++e) {
            const unsigned y = (unsigned)(x + e * THREADS), i = shift >= 0 ? y >> shift : y / per;
            c[e] = y - i * per;
            id[e] = x + e * THREADS < end ? ids[i] : 0;
        }
        line.look_up(id, blk);
        line.place(id, blk, from);
#pragma unroll
        for (int e = 0; e < kPieces; ++e)
            from[e] = from[e] * per + c[e];
    };
    x0 += threadIdx.x;
    if (x0 >= end)
        return;
    find(x0);
    for (long long x = x0; x < end; x += THREADS * kPieces) {
        uint4 k[kPieces], v[kPieces];
#pragma unroll
        for (int e = 0; e < kPieces; ++e)
            if (x + e * THREADS < end) {
                k[e] = __ldg(ks + from[e]);
                v[e] = __ldg(vs + from[e]);
            }
        find(x + THREADS * kPieces);
#pragma unroll
        for (int e = 0; e < kPieces; ++e)
            if (x + e * THREADS < end) {
                kd[x + e * THREADS] = k[e];
                vd[x + e * THREADS] = v[e];
            }
    }
}

// MOVE: the CTA also moves its unit's vectors into the outputs. WIDE: a unit is a
// cluster of p.cluster CTAs, each with a part of the row's slots; histograms and
// counts are summed over the cluster's shared memory.
template <bool MOVE, bool WIDE>
__global__ void __launch_bounds__(kThreads, MOVE ? 2 : WIDE ? 1 : 3) evict_select_kernel(const EvictParams p)
{
    extern __shared__ uint32_t keys[];         // [p.cached]
    __shared__ int hist[kBins], scan[kWarps], tied[kWarps], found[3], part[2], bad, listed;
    __shared__ int sum[WIDE ? kBins : 1];
    __shared__ uint32_t list[kList];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const cg::cluster_group cluster = cg::this_cluster();
    const int CL = WIDE ? p.cluster : 1, rank = WIDE ? (int)cluster.block_rank() : 0;
    const int unit = blockIdx.x / CL, b = unit / p.Hkv, h = unit % p.Hkv;
    // the next kernel may be set up meanwhile (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int L = __ldg(p.lengths + b);
    const long long cap = p.paged ? (long long)p.max_blocks * p.block_size : (long long)p.Smax;
    int bits = L < 0 || L > cap ? kBadLength : 0;
    if (!bits && !p.paged && p.slot_ids) {
        const int r = __ldg(p.slot_ids + b);
        bits = r < 0 || r >= p.R ? kBadSlotId : 0;
    }
    if (tid == 0)
        bad = bits;
    __syncthreads();
    if (!bits && p.paged)
        for (int i = tid; i < (int)(((long long)L + p.block_size - 1) / p.block_size); i += kThreads) {
            const int blk = __ldg(p.block_table + (long long)b * p.max_blocks + i);
            if (blk < 0 || blk >= p.num_blocks)
                bad = kBadBlock;
        }
    __syncthreads();
    bits = bad;                                // the same in every CTA of the cluster
    const Line line(p, bits ? 0 : b, h);
    int32_t *ids = p.ids + (long long)unit * p.n_keep;
    const int n = bits ? 0 : min(L, p.n_keep);
    if (tid == 0 && h == 0 && rank == 0) {
        p.new_lengths[b] = n;
        if (bits && p.status)
            atomicOr(p.status, bits);
    }
    float *to = nullptr;                       // where the counts go
    if (p.k_out)
        to = p.weights_out ? p.weights_out + (long long)unit * p.out_slots : nullptr;
    if (bits || L <= p.n_keep) {
        for (int i = rank * kThreads + tid; i < p.n_keep; i += kThreads * CL)
            ids[i] = i < n ? i : -1;
        if (to && !bits)
            for (int i = rank * kThreads + tid; i < p.out_slots; i += kThreads * CL)
                to[i] = i < n ? p.weights[line.at(i)] : 0.f;
        if constexpr (MOVE) {
            __syncthreads();                   // the ids are there
            gather<kThreads>(p, line, unit, 0, (long long)n * (p.row_bytes / 16));
        }
        return;
    }
    const int lo = p.n_first, hi = L - p.n_last;       // the slots that compete
    // this CTA's slots, the counts of the first `held` of them in shared memory
    const int mine = WIDE ? (L / CL / 32 + 1) * 32 : L;
    const int a0 = min((long long)L, (long long)rank * mine), a1 = min((long long)L, (long long)a0 + mine);
    const int held = min(a1 - a0, p.cached);
    int k = p.n_keep - p.n_first - p.n_last;           // how many of them are kept
    for (int i = tid; i < kBins; i += kThreads)
        hist[i] = 0;
    if (tid == 0)
        listed = 0;
    __syncthreads();
    // the counts, and a histogram of their first 11 bits
    if (a0 < a1) {
        int j[kEach], blk[kEach] = {};
        auto look = [&](int j0) {
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                j[e] = min(j0 + e * kThreads, a1 - 1);
            line.look_up(j, blk);
        };
        look(a0 + tid);
        for (int j0 = a0 + tid; j0 < a1; j0 += kThreads * kEach) {
            long long at[kEach];
            float w[kEach];
            line.place(j, blk, at);
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                w[e] = p.weights[at[e]];
            look(j0 + kThreads * kEach);
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int x = j0 + e * kThreads;
                const uint32_t u = order_of(w[e]);
                if (x < a0 + held)
                    keys[x - a0] = u;
                if (x >= lo && x < min(hi, a1))
                    atomicAdd(&hist[u >> 21], 1);
            }
        }
    }
    __syncthreads();
    auto key = [&](int j) { return j < a0 + held ? keys[j - a0] : order_of(p.weights[line.at(j)]); };
    // the unit's histogram
    auto whole = [&](int bins) -> const int * {
        if constexpr (WIDE) {
            cluster.sync();
            for (int i = tid; i < bins; i += kThreads) {
                int v = 0;
                for (int r = 0; r < CL; ++r)
                    v += cluster.map_shared_rank(hist, r)[i];
                sum[i] = v;
            }
            cluster.sync();
            return sum;
        } else {
            return hist;
        }
    };

    // the smallest kept count `least`, how many equal it (`equal`), and how many of those are kept (k)
    uint32_t least = 0xffffffffu;
    int equal = 0;
    if (k > 0) {
        least = (uint32_t)find_digit(whole(kBins), kBins, k, equal, scan, found) << 21;
        // the others' digits are found among the counts that share the first: a list of them where it holds them
        const bool few = equal <= kList;
        if (few) {
            for (int j = max(lo, a0) + tid; j < min(hi, a1); j += kThreads) {
                const uint32_t u = key(j);
                if (u >> 21 == least >> 21)
                    list[atomicAdd(&listed, 1)] = u;
            }
        }
        uint32_t mask = 0xffe00000u;
#pragma unroll
        for (int pass = 0; pass < 2; ++pass) {
            const int shift = pass == 0 ? 10 : 0, bins = pass == 0 ? 2048 : 1024;
            for (int i = tid; i < bins; i += kThreads)
                hist[i] = 0;
            __syncthreads();                   // (also: the list is there)
            const int n0 = few ? 0 : max(lo, a0), n1 = few ? listed : min(hi, a1);
            for (int j = n0 + tid; j < n1; j += kThreads) {
                const uint32_t u = few ? list[j] : key(j);
                if ((u & mask) == least)
                    atomicAdd(&hist[(u >> shift) & (bins - 1)], 1);
            }
            __syncthreads();
            least |= (uint32_t)find_digit(whole(bins), bins, k, equal, scan, found) << shift;
            mask |= (uint32_t)(bins - 1) << shift;
        }
    }
    // A warp takes a run of slots: it counts its kept ones, the warps' counts are
    // added up, then every kept slot has its place. Of those that equal `least`
    // the first k are kept, all of them where there are no more.
    const bool all = equal == k;
    const int share = ((a1 - a0) / (32 * kWarps) + 1) * 32, j0 = min((long long)a1, (long long)a0 + (long long)warp * share);
    const int j1 = min((long long)a1, (long long)j0 + share);
    auto look = [&](int j, unsigned &more, unsigned &tie) {
        const bool in = j < j1 && j >= lo && j < hi;
        const uint32_t u = in ? key(j) : 0u;
        more = __ballot_sync(0xffffffffu, j < j1 && (!in || (k > 0 && (u > least || (all && u == least)))));
        tie = all ? 0u : __ballot_sync(0xffffffffu, in && u == least);
    };
    int kept = 0, ties = 0;
    for (int j = j0 + lane; j - lane < j1; j += 32) {
        unsigned more, tie;
        look(j, more, tie);
        kept += __popc(more);
        ties += __popc(tie);
    }
    if (lane == 0) {
        scan[warp] = kept;
        tied[warp] = ties;
    }
    __syncthreads();
    int before = 0, same = 0;                  // kept slots (but ties), ties of the warps before
    for (int w = 0; w < warp; ++w) {
        before += scan[w];
        same += tied[w];
    }
    if constexpr (WIDE) {
        if (warp == kWarps - 1 && lane == 0) {
            part[0] = before + kept;
            part[1] = same + ties;
        }
        cluster.sync();
        for (int r = 0; r < rank; ++r) {       // and of the CTAs before
            const int *q = cluster.map_shared_rank(part, r);
            before += q[0];
            same += q[1];
        }
    }
    for (int j = j0 + lane; j - lane < j1; j += 32) {
        unsigned more, tie;
        look(j, more, tie);
        const unsigned below = (1u << lane) - 1u;
        const int m = before + __popc(more & below), s = same + __popc(tie & below);
        if ((more >> lane & 1u) || ((tie >> lane & 1u) && s < k))
            ids[m + min(s, k)] = j;
        before += __popc(more);
        same += __popc(tie);
    }
    if constexpr (WIDE)
        cluster.sync();                        // every CTA's ids are there (and nobody's shared memory is read any more)
    else
        __syncthreads();
    // the counts: kept ones in order, zeros behind them
    if (p.k_out) {
        for (int i0 = rank * kEach * kThreads + tid; to && i0 < p.out_slots; i0 += kThreads * kEach * CL) {
            int j[kEach], blk[kEach] = {};
            long long at[kEach];
            float w[kEach];
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                j[e] = ids[min(i0 + e * kThreads, n - 1)];
            line.look_up(j, blk);
            line.place(j, blk, at);
#pragma unroll
            for (int e = 0; e < kEach; ++e)
                w[e] = p.weights[at[e]];
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int i = i0 + e * kThreads;
                if (i < p.out_slots)
                    to[i] = i < n ? w[e] : 0.f;
            }
        }
        if constexpr (MOVE)
            gather<kThreads>(p, line, unit, 0, (long long)n * (p.row_bytes / 16));
        return;
    }
    for (int i0 = 0; rank == 0 && i0 < n; i0 += kThreads * kEach) {
        float w[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = i0 + e * kThreads + tid;
            w[e] = i < n ? p.weights[line.at(ids[i])] : 0.f;
        }
        __syncthreads();                       // later counts come from behind these places
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = i0 + e * kThreads + tid;
            if (i < n)
                p.weights[line.at(i)] = w[e];
        }
        __syncthreads();
    }
    if constexpr (WIDE)
        cluster.sync();                        // the kept counts have been read
    for (int j0 = n + rank * kEach * kThreads + tid; j0 < L; j0 += kThreads * kEach * CL) {
        int j[kEach], blk[kEach] = {};
        long long at[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            j[e] = min(j0 + e * kThreads, L - 1);
        line.look_up(j, blk);
        line.place(j, blk, at);
#pragma unroll
        for (int e = 0; e < kEach; ++e)
            p.weights[at[e]] = 0.f;            // (the last slot more than once)
    }
}

// Kept vectors into other buffers (B, Hkv, out_slots, row): a CTA takes a share
// of a unit's pieces.
__global__ void __launch_bounds__(kMove, 4) evict_gather_kernel(const EvictParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr long long share = kMove * kPieces * kSteps;
    const int unit = blockIdx.x / p.shares, b = unit / p.Hkv, h = unit % p.Hkv;
    const long long x0 = blockIdx.x % p.shares * share;
    gather<kMove>(p, Line(p, b, h), unit, x0, min((long long)p.new_lengths[b] * (p.row_bytes / 16), x0 + share));
}

constexpr int kDeep = 4;           // chunks on their way
constexpr int kBytes = 16384;      // of a chunk

// Kept vectors within the cache: blockIdx.x a (unit, column of SLICE bytes), blockIdx.y K or V.
template <int SLICE>
__global__ void __launch_bounds__(kMove) evict_compact_kernel(const EvictParams p)
{
    constexpr int PER = SLICE / 16;            // pieces a slot
    constexpr int CHUNK = kBytes / SLICE;      // kept slots a chunk
    constexpr int N = kBytes / 16 / kMove;     // pieces a thread and chunk
    extern __shared__ uint4 ring[];            // [kDeep][kBytes / 16]
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int columns = p.row_bytes / SLICE;
    const int unit = blockIdx.x / columns, b = unit / p.Hkv, h = unit % p.Hkv;
    const int n = p.new_lengths[b], tid = threadIdx.x;
    const Line line(p, b, h);
    const int32_t *ids = p.ids + (long long)unit * p.n_keep;
    char *cache = static_cast<char *>(blockIdx.y ? p.v_cache : p.k_cache) + (blockIdx.x % columns) * SLICE + tid % PER * 16;
    // the kept slots that stay where they are come first: chunks of them alone need no copy
    int c0 = 0;
    {
        int lo = 0, hi = n;                    // the first i with ids[i] != i
        while (lo < hi) {
            const int mid = (lo + hi) >> 1;
            if (__ldg(ids + mid) == mid)
                lo = mid + 1;
            else
                hi = mid;
        }
        c0 = lo / CHUNK;
    }
    const int chunks = (n + CHUNK - 1) / CHUNK;
    if (c0 >= chunks)
        return;
    // where this thread's pieces of a chunk come from and go to, looked up a chunk ahead
    const int first = tid / PER;               // its slot of a chunk; the others are kMove / PER apart
    long long from[N], to[N];
    auto sources = [&](int c) {
        int j[N], blk[N] = {};
#pragma unroll
        for (int e = 0; e < N; ++e)
            j[e] = __ldg(ids + min(c * CHUNK + first + e * (kMove / PER), n - 1));
        line.look_up(j, blk);
        line.place(j, blk, from);
    };
    auto places = [&](int c) {
        int j[N], blk[N] = {};
#pragma unroll
        for (int e = 0; e < N; ++e)
            j[e] = min(c * CHUNK + first + e * (kMove / PER), n - 1);
        line.look_up(j, blk);
        line.place(j, blk, to);
    };
    auto fetch = [&](int c) {
        if (c < chunks) {
#pragma unroll
            for (int e = 0; e < N; ++e)
                if (c * CHUNK + first + e * (kMove / PER) < n)
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(static_cast<uint32_t>(
                                     __cvta_generic_to_shared(ring + (c % kDeep) * (kBytes / 16) + e * kMove + tid))),
                                 "l"(cache + from[e] * p.row_bytes)
                                 : "memory");
            sources(min(c + 1, chunks - 1));
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    sources(c0);
    places(c0);
    for (int c = c0; c < c0 + kDeep - 1; ++c)
        fetch(c);
    for (int c = c0; c < chunks; ++c) {
        fetch(c + kDeep - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
        __syncthreads();                       // every thread's copies of the chunk (and of those before) have come
#pragma unroll
        for (int e = 0; e < N; ++e)
            if (c * CHUNK + first + e * (kMove / PER) < n)
                *reinterpret_cast<uint4 *>(cache + to[e] * p.row_bytes) = ring[(c % kDeep) * (kBytes / 16) + e * kMove + tid];
        places(min(c + 1, chunks - 1));
        // a thread reads back what it copied itself, so the slot is free for its next copies
    }
}

cudaLaunchConfig_t config(dim3 grid, int threads, size_t smem, cudaStream_t st, cudaLaunchAttribute *attr)
{
    attr->id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr->val.programmaticStreamSerializationAllowed = 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = grid;
    cfg.blockDim = dim3(threads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cfg;
}

}  // namespace

cudaError_t evict_launch(EvictParams p, int sms, cudaStream_t st)
{
    cudaLaunchAttribute attr[2];
    const long long cap = p.paged ? (long long)p.max_blocks * p.block_size : (long long)p.Smax;
    p.block_shift = -1;
    for (int i = 0; i < 31; ++i)
        if (p.paged && 1 << i == p.block_size)
            p.block_shift = i;
    static std::atomic<uint64_t> ready;        // the sizes are set once a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        constexpr int one = kCached * (int)sizeof(uint32_t), wide = kCachedWide * (int)sizeof(uint32_t);
        e = cudaFuncSetAttribute(evict_select_kernel<false, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, one);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(evict_select_kernel<true, false>, cudaFuncAttributeMaxDynamicSharedMemorySize, one);
        if (e == cudaSuccess)
            e = cudaFuncSetAttribute(evict_select_kernel<false, true>, cudaFuncAttributeMaxDynamicSharedMemorySize, wide);
        for (auto *f : {evict_compact_kernel<16>, evict_compact_kernel<32>, evict_compact_kernel<64>})
            if (e == cudaSuccess)
                e = cudaFuncSetAttribute(f, cudaFuncAttributeMaxDynamicSharedMemorySize, kDeep * kBytes);
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned units = (unsigned)(p.B * p.Hkv);
    // where units fill half the GPU each moves its own vectors once its slots are
    // chosen, beside others' choosing: of up to 16384 slots to 2048 (moved by the
    // same / another kernel) 40 units 60.6 / 43.7 us, 80 71.3 / 81.6, 160 98.0 /
    // 105.4, 240 118 / 143, 320 183 / 179
    const bool move = p.k_out && 2LL * units >= sms;
    // few units of long rows: clusters of CTAs, as many as the GPU has SMs for and
    // 4096 slots each are left to (8 units, one CTA / a cluster: 8192 slots to 512
    // 23.1 / 24.2 us, 16384 to 1024 40.9 / 25.7, 131072 to 4096 470 / 48.2)
    p.cluster = 1;
    while (!move && cap > 8192 && p.cluster < 8 && (long long)units * p.cluster * 2 <= sms && cap / (p.cluster * 2) >= 4096)
        p.cluster *= 2;
    const long long most = p.cluster > 1 ? kCachedWide : kCached, held = (cap / p.cluster / 32 + 1) * 32;
    p.cached = (int)(held < most ? held : most);
    cudaLaunchConfig_t cfg = config(dim3(units * p.cluster), kThreads, (size_t)p.cached * sizeof(uint32_t), st, attr);
    if (p.cluster > 1) {
        attr[1].id = cudaLaunchAttributeClusterDimension;
        attr[1].val.clusterDim.x = p.cluster;
        attr[1].val.clusterDim.y = 1;
        attr[1].val.clusterDim.z = 1;
        cfg.numAttrs = 2;
    }
    e = p.cluster > 1 ? cudaLaunchKernelEx(&cfg, evict_select_kernel<false, true>, p)
        : move        ? cudaLaunchKernelEx(&cfg, evict_select_kernel<true, false>, p)
                      : cudaLaunchKernelEx(&cfg, evict_select_kernel<false, false>, p);
    if (e != cudaSuccess || move)
        return e;
    if (p.k_out) {
        const long long pieces = (long long)(p.n_keep < cap ? p.n_keep : cap) * (p.row_bytes / 16);
        constexpr int share = kMove * kPieces * kSteps;
        p.shares = (int)((pieces + share - 1) / share);
        cfg = config(dim3(units * (unsigned)p.shares), kMove, 0, st, attr);
        return cudaLaunchKernelEx(&cfg, evict_gather_kernel, p);
    }
    // columns of 64 bytes (in place, 64 rows of up to 16384 slots of 8 x 256 bytes
    // to 2048: 32 bytes 336 us, 64 288, 128 283; 4 rows of up to 131072 to 16384:
    // 227, 178, 236), or of what divides the rows
    const int slice = p.row_bytes % 64 == 0 ? 64 : p.row_bytes % 32 == 0 ? 32 : 16;
    cfg = config(dim3(units * (unsigned)(p.row_bytes / slice), 2), kMove, kDeep * kBytes, st, attr);
    return slice == 64   ? cudaLaunchKernelEx(&cfg, evict_compact_kernel<64>, p)
           : slice == 32 ? cudaLaunchKernelEx(&cfg, evict_compact_kernel<32>, p)
                         : cudaLaunchKernelEx(&cfg, evict_compact_kernel<16>, p);
}

}  // namespace gqa
