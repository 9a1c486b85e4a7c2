// Eviction: a row longer than n_keep slots keeps, for every cache head, its
// first n_first slots, its last n_last, and of the others those with the largest
// counts (ties to the lowest slot, NaN counts highest), in ascending order.
//
// evict_select_kernel, a CTA a (row, head): the counts as integers in order
// (sign folded, -0 as 0), the first kCached of them kept in shared memory; the
// smallest kept count by three histograms of 11, 11 and 10 bits, each over the
// slots that agree in the bits before; then one pass in slot order that gives
// every kept slot its place (ballots, a scan of the warps' totals). Bound by
// the latency of these passes; a count is read from memory once where the row
// fits. The counts move in the same kernel.
//
// Kept vectors are copied elsewhere by evict_gather_kernel, every 16 bytes on
// their own, or within the cache by evict_compact_kernel. In place, kept slot i
// comes from a slot >= i; a CTA takes a column of kSlice bytes of the vectors of
// a (row, head), chunk by chunk of kChunk kept slots: the sources of a later
// chunk lie behind the destinations of an earlier one, so copies into shared
// memory may run kDeep chunks ahead of the stores as long as a chunk is stored
// after it and those before it have come. Both are bound by memory: 2 rows of
// bytes a kept vector.
#include <atomic>

#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr int kThreads = 1024, kWarps = kThreads / 32;
constexpr int kCached = 16384;     // counts kept in shared memory (64 KB: two CTAs an SM)
constexpr int kBins = 2048;
constexpr int kEach = 4;           // slots a thread per step of the last pass

__device__ __forceinline__ uint32_t order_of(float w)
{
    uint32_t u = __float_as_uint(w);
    if (w != w)
        return 0xffffffffu;
    u = u == 0x80000000u ? 0u : u;
    return u & 0x80000000u ? ~u : u | 0x80000000u;
}

// Index of slot j's vector of the unit (a paged block is known to be usable).
__device__ __forceinline__ long long vector_at(const EvictParams &p, int b, int h, int j)
{
    if (p.paged) {
        const int blk = __ldg(p.block_table + (long long)b * p.max_blocks + j / p.block_size);
        return ((long long)blk * p.Hkv + h) * p.block_size + j % p.block_size;
    }
    const long long r = p.slot_ids ? __ldg(p.slot_ids + b) : b;
    return (r * p.Hkv + h) * p.Smax + j;
}

// The digit of the k-th largest among the counted ones: hist[] is summed from
// the top. Every thread of the CTA calls it; returns the digit, and k less the
// number above it.
__device__ __forceinline__ int find_digit(const int *hist, int bins, int &k, int *scan, int *found)
{
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = bins / kThreads;   // 1 or 2 bins a thread, from the top
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
        int v = scan[lane];
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int y = __shfl_up_sync(0xffffffffu, v, o);
            if (lane >= o)
                v += y;
        }
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
                break;
            }
            above += c;
        }
    }
    __syncthreads();
    k = found[1];
    return found[0];
}

__global__ void __launch_bounds__(kThreads) evict_select_kernel(const EvictParams p)
{
    extern __shared__ uint32_t keys[];         // [min(capacity, kCached)]
    __shared__ int hist[kBins], scan[kWarps], found[2], bad;
    __shared__ int totals[kEach * kWarps];     // kept slots, then their places
    __shared__ int ties[kEach * kWarps];
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int b = blockIdx.x / p.Hkv, h = blockIdx.x % p.Hkv;
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
        for (int i = tid; i < (L + p.block_size - 1) / p.block_size; i += kThreads) {
            const int blk = __ldg(p.block_table + (long long)b * p.max_blocks + i);
            if (blk < 0 || blk >= p.num_blocks)
                bad = kBadBlock;
        }
    __syncthreads();
    bits = bad;
    int32_t *ids = p.ids + (long long)blockIdx.x * p.n_keep;
    const int n = bits ? 0 : min(L, p.n_keep);
    if (tid == 0 && h == 0) {
        p.new_lengths[b] = n;
        if (bits && p.status)
            atomicOr(p.status, bits);
    }
    float *to = nullptr;                       // where the counts go
    if (p.k_out)
        to = p.weights_out ? p.weights_out + (long long)blockIdx.x * p.out_slots : nullptr;
    if (bits || L <= p.n_keep) {
        for (int i = tid; i < p.n_keep; i += kThreads)
            ids[i] = i < n ? i : -1;
        if (to && !bits)
            for (int i = tid; i < p.out_slots; i += kThreads)
                to[i] = i < n ? p.weights[vector_at(p, b, h, i)] : 0.f;
        return;
    }
    const int lo = p.n_first, hi = L - p.n_last;       // the slots that compete
    const int held = min(L, p.cached);
    for (int j = tid; j < held; j += kThreads)
        keys[j] = order_of(p.weights[vector_at(p, b, h, j)]);
    auto key = [&](int j) { return j < held ? keys[j] : order_of(p.weights[vector_at(p, b, h, j)]); };

    // the smallest kept count `least`, and how many that equal it are kept
    int k = p.n_keep - p.n_first - p.n_last;
    uint32_t least = 0xffffffffu, mask = 0;
    if (k > 0) {
        least = 0;
#pragma unroll
        for (int pass = 0; pass < 3; ++pass) {
            const int shift = pass == 0 ? 21 : pass == 1 ? 10 : 0, bins = pass == 2 ? 1024 : 2048;
            for (int i = tid; i < bins; i += kThreads)
                hist[i] = 0;
            __syncthreads();                   // (also: the keys are there)
            // a thread adds up the slots in a row of one digit (many slots may never have been attended)
            int bin = -1, count = 0;
            for (int j = lo + tid; j < hi; j += kThreads) {
                const uint32_t u = key(j);
                if ((u & mask) == least) {
                    const int d = (u >> shift) & (bins - 1);
                    if (d != bin && count) {
                        atomicAdd(&hist[bin], count);
                        count = 0;
                    }
                    bin = d;
                    ++count;
                }
            }
            if (count)
                atomicAdd(&hist[bin], count);
            __syncthreads();
            const int digit = find_digit(hist, bins, k, scan, found);
            least |= (uint32_t)digit << shift;
            mask |= (uint32_t)(bins - 1) << shift;
            __syncthreads();
        }
    } else {
        __syncthreads();
    }
    // k: kept slots among those that equal `least` (0: none competes)
    int before = 0, same = 0;                  // kept slots (but ties), ties so far
    for (int j0 = 0; j0 < L; j0 += kThreads * kEach) {
        unsigned more[kEach], tie[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int j = j0 + e * kThreads + tid;
            const bool in = j >= lo && j < hi;
            const uint32_t u = in ? key(j) : 0u;
            more[e] = __ballot_sync(0xffffffffu, j < L && (!in || (k > 0 && u > least)));
            tie[e] = __ballot_sync(0xffffffffu, in && k > 0 && u == least);
            if (lane == 0) {
                totals[e * kWarps + warp] = __popc(more[e]);
                ties[e * kWarps + warp] = __popc(tie[e]);
            }
        }
        __syncthreads();
        if (warp < 2) {                        // warp 0 scans the totals, warp 1 the ties
            int *a = warp ? ties : totals;
            int carry = 0;
#pragma unroll
            for (int e = 0; e < kEach; ++e) {
                const int x = a[e * kWarps + lane];
                int v = x;
#pragma unroll
                for (int o = 1; o < 32; o <<= 1) {
                    const int y = __shfl_up_sync(0xffffffffu, v, o);
                    if (lane >= o)
                        v += y;
                }
                a[e * kWarps + lane] = carry + v - x;
                carry += __shfl_sync(0xffffffffu, v, 31);
            }
            if (lane == 0)
                found[warp] = carry;
        }
        __syncthreads();
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const unsigned below = (1u << lane) - 1u;
            const int m = before + totals[e * kWarps + warp] + __popc(more[e] & below);
            const int s = same + ties[e * kWarps + warp] + __popc(tie[e] & below);
            const bool is_tie = tie[e] >> lane & 1u;
            if ((more[e] >> lane & 1u) || (is_tie && s < k))
                ids[m + min(s, k)] = j0 + e * kThreads + tid;
        }
        before += found[0];
        same += found[1];
        __syncthreads();
    }
    // the counts: kept ones in order, zeros behind them
    if (p.k_out) {
        if (to)
            for (int i = tid; i < p.out_slots; i += kThreads)
                to[i] = i < n ? p.weights[vector_at(p, b, h, ids[i])] : 0.f;
        return;
    }
    for (int i0 = 0; i0 < n; i0 += kThreads * kEach) {
        float w[kEach];
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = i0 + e * kThreads + tid;
            w[e] = i < n ? p.weights[vector_at(p, b, h, ids[i])] : 0.f;
        }
        __syncthreads();                       // later counts come from behind these places
#pragma unroll
        for (int e = 0; e < kEach; ++e) {
            const int i = i0 + e * kThreads + tid;
            if (i < n)
                p.weights[vector_at(p, b, h, i)] = w[e];
        }
        __syncthreads();
    }
    for (int j = n + tid; j < L; j += kThreads)
        p.weights[vector_at(p, b, h, j)] = 0.f;
}

constexpr int kMove = 256;         // threads of the moving kernels
constexpr int kPieces = 8;         // 16-byte pieces a thread

// Kept vectors into other buffers (B, Hkv, out_slots, row): blockIdx.x a share
// of a unit's pieces of K (blockIdx.y = 0) or V.
__global__ void __launch_bounds__(kMove) evict_gather_kernel(const EvictParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int unit = blockIdx.x / p.shares, b = unit / p.Hkv, h = unit % p.Hkv;
    const int per = p.row_bytes / 16;          // pieces a vector
    const long long x0 = (long long)(blockIdx.x % p.shares) * kMove * kPieces, n = (long long)p.new_lengths[b] * per;
    if (x0 >= n)
        return;
    const uint4 *src = static_cast<const uint4 *>(blockIdx.y ? p.v_cache : p.k_cache);
    uint4 *dst = static_cast<uint4 *>(blockIdx.y ? p.v_out : p.k_out) + (long long)unit * p.out_slots * per;
    const int32_t *ids = p.ids + (long long)unit * p.n_keep;
    uint4 w[kPieces];
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
        const long long x = x0 + e * kMove + threadIdx.x;
        if (x < n) {
            const int i = (int)(x / per);
            w[e] = __ldg(src + vector_at(p, b, h, __ldg(ids + i)) * per + (x - (long long)i * per));
        }
    }
#pragma unroll
    for (int e = 0; e < kPieces; ++e) {
        const long long x = x0 + e * kMove + threadIdx.x;
        if (x < n)
            dst[x] = w[e];
    }
}

constexpr int kDeep = 4;           // chunks on their way
constexpr int kChunk = 256;        // kept slots a chunk

// Kept vectors within the cache: blockIdx.x a (unit, column of SLICE bytes), blockIdx.y K or V.
template <int SLICE>
__global__ void __launch_bounds__(kMove) evict_compact_kernel(const EvictParams p)
{
    constexpr int PER = SLICE / 16;            // pieces a slot
    constexpr int N = kChunk * PER / kMove;    // pieces a thread and chunk
    __shared__ uint4 ring[kDeep][kChunk * PER];
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    const int columns = p.row_bytes / SLICE;
    const int unit = blockIdx.x / columns, b = unit / p.Hkv, h = unit % p.Hkv;
    const int n = p.new_lengths[b], tid = threadIdx.x;
    const int32_t *ids = p.ids + (long long)unit * p.n_keep;
    char *cache = static_cast<char *>(blockIdx.y ? p.v_cache : p.k_cache) + (blockIdx.x % columns) * SLICE;
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
        c0 = lo / kChunk;
    }
    const int chunks = (n + kChunk - 1) / kChunk;
    auto fetch = [&](int c) {
        if (c < chunks) {
#pragma unroll
            for (int e = 0; e < N; ++e) {
                const int x = e * kMove + tid, i = c * kChunk + x / PER;
                if (i < n) {
                    const char *src = cache + vector_at(p, b, h, __ldg(ids + i)) * p.row_bytes + x % PER * 16;
                    asm volatile("cp.async.cg.shared.global [%0], [%1], 16;" ::"r"(
                                     static_cast<uint32_t>(__cvta_generic_to_shared(&ring[c % kDeep][x]))),
                                 "l"(src)
                                 : "memory");
                }
            }
        }
        asm volatile("cp.async.commit_group;" ::: "memory");
    };
    for (int c = c0; c < c0 + kDeep - 1; ++c)
        fetch(c);
    for (int c = c0; c < chunks; ++c) {
        fetch(c + kDeep - 1);
        asm volatile("cp.async.wait_group %0;" ::"n"(kDeep - 1) : "memory");
        __syncthreads();                       // every thread's copies of the chunk (and of those before) have come
#pragma unroll
        for (int e = 0; e < N; ++e) {
            const int x = e * kMove + tid, i = c * kChunk + x / PER;
            if (i < n)
                *reinterpret_cast<uint4 *>(cache + vector_at(p, b, h, i) * p.row_bytes + x % PER * 16) = ring[c % kDeep][x];
        }
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

cudaError_t evict_launch(EvictParams p, cudaStream_t st)
{
    cudaLaunchAttribute attr[1];
    const long long cap = p.paged ? (long long)p.max_blocks * p.block_size : (long long)p.Smax;
    p.cached = (int)(cap < kCached ? cap : kCached);
    const int smem = p.cached * (int)sizeof(uint32_t);
    static std::atomic<uint64_t> ready;        // the size is set once a device
    int dev = 0;
    cudaError_t e = cudaGetDevice(&dev);
    if (e != cudaSuccess)
        return e;
    const uint64_t bit = 1ull << (dev & 63);
    if (!(ready.load(std::memory_order_relaxed) & bit)) {
        e = cudaFuncSetAttribute(evict_select_kernel, cudaFuncAttributeMaxDynamicSharedMemorySize,
                                 kCached * (int)sizeof(uint32_t));
        if (e != cudaSuccess)
            return e;
        ready.fetch_or(bit, std::memory_order_relaxed);
    }
    const unsigned units = (unsigned)(p.B * p.Hkv);
    cudaLaunchConfig_t cfg = config(dim3(units), kThreads, smem, st, attr);
    e = cudaLaunchKernelEx(&cfg, evict_select_kernel, p);
    if (e != cudaSuccess)
        return e;
    if (p.k_out) {
        const long long pieces = (long long)(p.n_keep < cap ? p.n_keep : cap) * (p.row_bytes / 16);
        p.shares = (int)((pieces + kMove * kPieces - 1) / (kMove * kPieces));
        cfg = config(dim3(units * (unsigned)p.shares, 2), kMove, 0, st, attr);
        return cudaLaunchKernelEx(&cfg, evict_gather_kernel, p);
    }
    // columns of 64 bytes, or of the largest power of two that divides the rows
    const int slice = p.row_bytes % 64 == 0 ? 64 : p.row_bytes % 32 == 0 ? 32 : 16;
    cfg = config(dim3(units * (unsigned)(p.row_bytes / slice), 2), kMove, 0, st, attr);
    return slice == 64   ? cudaLaunchKernelEx(&cfg, evict_compact_kernel<64>, p)
           : slice == 32 ? cudaLaunchKernelEx(&cfg, evict_compact_kernel<32>, p)
                         : cudaLaunchKernelEx(&cfg, evict_compact_kernel<16>, p);
}

}  // namespace gqa
