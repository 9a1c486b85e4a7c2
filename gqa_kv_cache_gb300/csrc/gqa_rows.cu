// Writing packed tokens into a cache (append) and reading slots back (read):
// float32, bfloat16, E4M3 and E2M1 caches; dense, slot-id and paged addressing.
//
// Token t of the packed batch belongs to the row b with cu_q[b] <= t <
// cu_q[b + 1] and to slot lengths[b] + t - cu_q[b] of that row. A CTA takes a
// few consecutive tokens: its first threads find each token's row (a binary
// search of cu_q), check it and leave the element offset of its slot in
// shared memory; then every thread takes 16 consecutive elements -- one scale
// group of an E2M1 cache -- of a (token, head) vector of K and of V: 16-byte
// loads, the whole group's maximum and division in one thread, no shuffles.
// Both kernels are bound by memory: 4 D + 2 row bytes a (token, head) to
// append (row = 0.5625 D for E2M1).
//
// Key bounds: the element-wise smallest and largest key of every block of
// slots, kept as the tokens arrive. The tokens of one block that a call brings
// form a run; one CTA owns the run (the one whose share of the tokens holds
// its first token), so the block's bounds have a single writer and the result
// does not depend on any order. A run that begins at the block's first slot
// replaces the bounds, any other widens them.
#include "gqa_common.cuh"
#include "gqa_decode.h"
#include "gqa_fp4.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;
constexpr long long kSkip = -1;   // a token of no row, or of a bad one

struct Token {
    long long off;   // element offset of the slot's vector of head 0, or kSkip
    int b, slot;     // its row (-1: of no row) and slot
};

// The row of packed token t and its slot's offset. Reports what is wrong with
// the token's row (the row's first token only, a bad block each time).
__device__ inline Token find_token(const RowsParams &p, int t)
{
    Token k;
    k.off = kSkip;
    k.b = k.slot = -1;
    int lo = 0, hi = p.B;              // the last b with cu_q[b] <= t
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (__ldg(p.cu_q + mid) <= t)
            lo = mid;
        else
            hi = mid;
    }
    const int t0 = __ldg(p.cu_q + lo), t1 = __ldg(p.cu_q + lo + 1);
    if (t < t0 || t >= t1)
        return k;                      // padding behind (or before) the rows' tokens
    k.b = lo;
    if (t0 < 0 || t1 > p.T) {
        rows_report(p, kBadQLen);
        return k;
    }
    const long long L = __ldg(p.lengths + lo);
    const long long cap = p.paged ? (long long)p.max_blocks * p.block_size : (long long)p.Smax;
    if (L < 0 || L + (t1 - t0) > cap) {
        rows_report(p, kBadLength);
        return k;
    }
    k.slot = (int)(L + (t - t0));
    if (p.paged) {
        const int blk = __ldg(p.block_table + (long long)lo * p.max_blocks + k.slot / p.block_size);
        if (blk < 0 || blk >= p.num_blocks) {
            rows_report(p, kBadBlock);
            return k;
        }
        k.off = ((long long)blk * p.Hkv * p.block_size + k.slot % p.block_size) * p.D;
    } else {
        const int r = p.slot_ids ? __ldg(p.slot_ids + lo) : lo;
        if (r < 0 || r >= p.R) {
            rows_report(p, kBadSlotId);
            return k;
        }
        k.off = ((long long)r * p.Hkv * p.Smax + k.slot) * p.D;
    }
    return k;
}

// Sixteen elements of type T as loaded. 32 bytes at a time where the vectors
// lie on 32-byte boundaries (WIDE; half as many requests, and a store fills
// whole sectors: reading back 131071 tokens of 8 x 128 to bfloat16 took 133 us
// with 16-byte stores), else 16.
template <typename T>
struct Raw {
    uint32_t u[4 * sizeof(T)];
};

__device__ __forceinline__ void ld32(const void *src, uint32_t *u)
{
    asm("ld.global.nc.v8.b32 {%0, %1, %2, %3, %4, %5, %6, %7}, [%8];"
        : "=r"(u[0]), "=r"(u[1]), "=r"(u[2]), "=r"(u[3]), "=r"(u[4]), "=r"(u[5]), "=r"(u[6]), "=r"(u[7])
        : "l"(src));
}
__device__ __forceinline__ void st32(void *dst, const uint32_t *u)
{
    asm volatile("st.global.v8.b32 [%0], {%1, %2, %3, %4, %5, %6, %7, %8};" ::"l"(dst), "r"(u[0]), "r"(u[1]), "r"(u[2]),
                 "r"(u[3]), "r"(u[4]), "r"(u[5]), "r"(u[6]), "r"(u[7])
                 : "memory");
}

template <typename T>
__device__ __forceinline__ Raw<T> load_raw(const T *src, bool wide)
{
    Raw<T> w;
    constexpr int N = 4 * sizeof(T);
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        const uint4 *p = reinterpret_cast<const uint4 *>(src) + i / 4;
        if (wide) {
            ld32(p, w.u + i);
        } else {
            const uint4 a = __ldg(p), b = __ldg(p + 1);
            w.u[i] = a.x; w.u[i + 1] = a.y; w.u[i + 2] = a.z; w.u[i + 3] = a.w;
            w.u[i + 4] = b.x; w.u[i + 5] = b.y; w.u[i + 6] = b.z; w.u[i + 7] = b.w;
        }
    }
    return w;
}

template <typename T>
__device__ __forceinline__ void store_raw(T *dst, const Raw<T> &w, bool wide)
{
    constexpr int N = 4 * sizeof(T);
#pragma unroll
    for (int i = 0; i < N; i += 8) {
        uint4 *p = reinterpret_cast<uint4 *>(dst) + i / 4;
        if (wide) {
            st32(p, w.u + i);
        } else {
            p[0] = make_uint4(w.u[i], w.u[i + 1], w.u[i + 2], w.u[i + 3]);
            p[1] = make_uint4(w.u[i + 4], w.u[i + 5], w.u[i + 6], w.u[i + 7]);
        }
    }
}

// Widened to float32, and rounded from it.
template <typename T>
__device__ __forceinline__ void widen16(const Raw<T> &w, float (&x)[16])
{
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (sizeof(T) == 4)
            x[i] = __uint_as_float(w.u[i]);
        else
            x[i] = (i & 1) ? bf16_hi(w.u[i / 2]) : bf16_lo(w.u[i / 2]);
    }
}
template <typename T>
__device__ __forceinline__ Raw<T> round16(const float (&x)[16])
{
    Raw<T> w;
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 16; ++i)
            w.u[i] = __float_as_uint(x[i]);
    } else {
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            w.u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
    }
    return w;
}

// One group of 16 elements into the cache at element offset `off`.
template <int KIND, typename T>
__device__ __forceinline__ void put16(void *cache, void *groups, long long off, float g, const Raw<T> &w, bool wide)
{
    float x[16];
    widen16(w, x);
    if constexpr (KIND == GQA_DTYPE_F32) {
        store_raw(static_cast<float *>(cache) + off, round16<float>(x), wide);
    } else if constexpr (KIND == GQA_DTYPE_BF16) {
        store_raw(static_cast<__nv_bfloat16 *>(cache) + off, round16<__nv_bfloat16>(x), wide);
    } else if constexpr (KIND == GQA_DTYPE_E4M3) {
        uint32_t u[4] = {0u, 0u, 0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            unsigned short q;
            asm("cvt.rn.satfinite.e4m3x2.f32 %0, %1, %2;"
                : "=h"(q)
                : "f"(__fdiv_rn(x[2 * i + 1], g)), "f"(__fdiv_rn(x[2 * i], g)));
            u[i >> 1] |= (uint32_t)q << (16 * (i & 1));
        }
        *reinterpret_cast<uint4 *>(static_cast<uint8_t *>(cache) + off) = make_uint4(u[0], u[1], u[2], u[3]);
    } else {
        float amax = 0.f;
        if constexpr (sizeof(T) == 2) {
            // two at a time as they came (the signs get mixed up)
            uint32_t m = w.u[0];
#pragma unroll
            for (int i = 1; i < 8; ++i)
                asm("max.NaN.xorsign.abs.bf16x2 %0, %0, %1;" : "+r"(m) : "r"(w.u[i]));
            amax = max_nan(fabsf(bf16_lo(m)), fabsf(bf16_hi(m)));
        } else {
#pragma unroll
            for (int i = 0; i < 16; ++i)
                amax = max_nan(amax, fabsf(x[i]));
        }
        float t;
        const uint32_t s = group_scale(amax, g, t);
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + (off >> 1)) = e2m1_codes16(x, s, t);
        static_cast<uint8_t *>(groups)[off >> 4] = (uint8_t)s;
    }
}

// The group at element offset `off` of the cache.
template <int KIND>
__device__ __forceinline__ void get16(const void *cache, const void *groups, long long off, float g, float (&x)[16],
                                      bool wide)
{
    if constexpr (KIND == GQA_DTYPE_F32) {
        widen16(load_raw(static_cast<const float *>(cache) + off, wide), x);
    } else if constexpr (KIND == GQA_DTYPE_BF16) {
        widen16(load_raw(static_cast<const __nv_bfloat16 *>(cache) + off, wide), x);
    } else if constexpr (KIND == GQA_DTYPE_E4M3) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(static_cast<const uint8_t *>(cache) + off));
        const uint32_t u[4] = {w.x, w.y, w.z, w.w};
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const uint32_t h = e4m3x2_f16((u[i >> 1] >> (16 * (i & 1))) & 0xffffu);
            const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h));
            x[2 * i] = __fmul_rn(f.x, g);
            x[2 * i + 1] = __fmul_rn(f.y, g);
        }
    } else {
        const uint2 w = __ldg(reinterpret_cast<const uint2 *>(static_cast<const uint8_t *>(cache) + (off >> 1)));
        const float t = __fmul_rn(e4m3_f32(__ldg(static_cast<const uint8_t *>(groups) + (off >> 4))), g);
        const uint32_t u[2] = {w.x, w.y};
#pragma unroll
        for (int i = 0; i < 2; ++i) {
            uint32_t h[4];
            e2m1x8_f16(u[i], h);
#pragma unroll
            for (int j = 0; j < 4; ++j) {
                const float2 f = __half22float2(*reinterpret_cast<const __half2 *>(&h[j]));
                x[8 * i + 2 * j] = __fmul_rn(f.x, t);
                x[8 * i + 2 * j + 1] = __fmul_rn(f.y, t);
            }
        }
    }
}

// min or max of bfloat16 pairs; NaN where either is.
__device__ __forceinline__ uint32_t min_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("min.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}
__device__ __forceinline__ uint32_t max_bf16x2(uint32_t a, uint32_t b)
{
    uint32_t r;
    asm("max.NaN.bf16x2 %0, %1, %2;" : "=r"(r) : "r"(a), "r"(b));
    return r;
}

// Bounds of sixteen keys' elements as bfloat16 pairs.
struct Bounds {
    uint32_t lo[8], hi[8];
};

// Widens the bounds of the run by one key (its first: replaces them). A
// float32 key's lower bound is rounded down and its upper bound up, so that the
// bounds hold (bfloat16 keys: exact).
template <typename T>
__device__ __forceinline__ void take(Bounds &r, const Raw<T> &w, bool first)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        uint32_t lo, hi;
        if constexpr (sizeof(T) == 2) {
            lo = hi = w.u[i];
        } else {
            const float x = __uint_as_float(w.u[2 * i]), y = __uint_as_float(w.u[2 * i + 1]);
            lo = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(x)) |
                 ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_rd(y)) << 16);
            hi = (uint32_t)__bfloat16_as_ushort(__float2bfloat16_ru(x)) |
                 ((uint32_t)__bfloat16_as_ushort(__float2bfloat16_ru(y)) << 16);
        }
        r.lo[i] = first ? lo : min_bf16x2(r.lo[i], lo);
        r.hi[i] = first ? hi : max_bf16x2(r.hi[i], hi);
    }
}

__device__ __forceinline__ void widen(Bounds &a, const Bounds &b)
{
#pragma unroll
    for (int i = 0; i < 8; ++i) {
        a.lo[i] = min_bf16x2(a.lo[i], b.lo[i]);
        a.hi[i] = max_bf16x2(a.hi[i], b.hi[i]);
    }
}

// The threads of a CTA over (group, token): group c of the Hkv * D / 16 groups
// of a token's vectors, every `lanes`-th token. A token's groups are
// neighbouring threads (and addresses).
struct Share {
    int per;       // groups of a token
    int lanes;     // tokens at once
    int c, lane;   // this thread's first group and token (lane >= lanes: none)
    __device__ __forceinline__ Share(const RowsParams &p)
    {
        per = p.Hkv * (p.D / kGroup);
        lanes = per >= kThreads ? 1 : kThreads / per;
        c = per >= kThreads ? threadIdx.x : threadIdx.x % per;
        lane = per >= kThreads ? 0 : threadIdx.x / per;
    }
};

// Rows whose offsets decrease (or begin outside the tokens) have no token that
// could tell: the CTAs look at the rows' offsets too.
__device__ __forceinline__ void check_rows(const RowsParams &p)
{
    for (long long b = (long long)blockIdx.x * kThreads + threadIdx.x; b < p.B; b += (long long)gridDim.x * kThreads) {
        const int t0 = __ldg(p.cu_q + b), t1 = __ldg(p.cu_q + b + 1);
        if (t0 < 0 || t1 < t0 || t1 > p.T)
            rows_report(p, kBadQLen);
    }
}

// One CTA: `chunk` tokens and, with bounds, the rest of the last run that
// begins among them. Shared memory: the tokens' slots, then (bounds) one
// Bounds a thread.
template <typename T, int KIND, bool BOUNDS>
__global__ void __launch_bounds__(kThreads, sizeof(T) == 2 ? 4 : 2) append_kernel(const RowsParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    const int run = BOUNDS ? p.bounds_block : 1;
    Token *tok = reinterpret_cast<Token *>(smem);      // [chunk + run - 1]
    Bounds *part = reinterpret_cast<Bounds *>(smem + sizeof(Token) * (p.chunk + run - 1));
    __shared__ int first, last;        // the CTA's tokens: tok[first .. last - 1]
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.chunk;
    const int n = min(p.chunk + run - 1, p.T - t0);   // tokens looked at
    // the next kernel may be set up meanwhile (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        first = BOUNDS ? n : 0;
        last = n;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const Token k = find_token(p, t0 + i);
        tok[i] = k;
        if constexpr (BOUNDS) {
            // the token begins a run: its block's first slot, or its row's
            // first token (a skipped token is a run of its own)
            if (k.off == kSkip || k.slot % run == 0 || t0 + i == __ldg(p.cu_q + k.b))
                atomicMin(i < p.chunk ? &first : &last, i);
        }
    }
    check_rows(p);
    __syncthreads();
    const int a = first, e = max(a, last);
    const Share s(p);
    const long long head = (long long)(p.paged ? p.block_size : p.Smax) * p.D;   // elements between heads
    const T *kn = static_cast<const T *>(p.k_new), *vn = static_cast<const T *>(p.v_new);
    constexpr bool kScaled = KIND == GQA_DTYPE_E4M3 || KIND == GQA_DTYPE_E2M1;
    for (int c0 = 0; c0 < s.per; c0 += kThreads) {     // once, but for very wide tokens
        const int c = c0 + s.c;
        const bool mine = c < s.per && s.lane < s.lanes;
        const int h = c / (p.D / kGroup), d = (c % (p.D / kGroup)) * kGroup;
        const float ks = kScaled && mine ? __ldg(p.k_scale + h) : 1.f, vs = kScaled && mine ? __ldg(p.v_scale + h) : 1.f;
        const long long to = h * head + d;
        const long long row = (long long)p.Hkv * p.D, from = (long long)t0 * row + (long long)c * kGroup;
        int i = a;
        while (i < e) {
            int j = e;                                 // one past the run (without bounds: all tokens)
            if constexpr (BOUNDS) {
                j = i + 1;
                if (tok[i].off != kSkip) {
                    // a run's tokens follow each other and share their block
                    const int left = run - tok[i].slot % run;
                    j = min(min(e, i + left), __ldg(p.cu_q + tok[i].b + 1) - t0);
                }
            }
            Bounds box;
            bool any = false;
            for (int m = i + s.lane; mine && m < j; m += s.lanes) {
                const long long off = tok[m].off;
                if (off == kSkip)
                    continue;
                const Raw<T> x = load_raw(kn + from + m * row, p.wide), y = load_raw(vn + from + m * row, p.wide);
                if constexpr (BOUNDS) {
                    take(box, x, !any);
                    any = true;
                }
                put16<KIND>(p.k_cache, p.k_group, off + to, ks, x, p.wide);
                put16<KIND>(p.v_cache, p.v_group, off + to, vs, y, p.wide);
            }
            if constexpr (BOUNDS) {
                // the lanes' bounds, and what the block had before
                const int held = min(s.lanes, j - i);  // lanes with a token
                if (held > 1) {
                    if (any)
                        part[tid] = box;
                    __syncthreads();
                    if (any && s.lane == 0)
                        for (int l = 1; l < held; ++l)
                            widen(box, part[tid + l * s.per]);
                    __syncthreads();
                }
                if (any && s.lane == 0) {
                    const Token k = tok[i];
                    long long at;                      // (block of the row or of the pool, head)
                    if (p.paged) {
                        at = k.off / ((long long)p.D * p.block_size) + h;   // off is in head 0 of its block
                    } else {
                        const long long r = p.slot_ids ? __ldg(p.slot_ids + k.b) : k.b;
                        at = (r * p.Hkv + h) * (p.Smax / run) + k.slot / run;
                    }
                    uint4 *bl = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.bounds) + at * 2 * p.D + d);
                    uint4 *bh = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.bounds) + (at * 2 + 1) * p.D + d);
                    if (k.slot % run) {
                        const uint4 l0 = bl[0], l1 = bl[1], h0 = bh[0], h1 = bh[1];
                        const Bounds old = {{l0.x, l0.y, l0.z, l0.w, l1.x, l1.y, l1.z, l1.w},
                                            {h0.x, h0.y, h0.z, h0.w, h1.x, h1.y, h1.z, h1.w}};
                        widen(box, old);
                    }
                    bl[0] = make_uint4(box.lo[0], box.lo[1], box.lo[2], box.lo[3]);
                    bl[1] = make_uint4(box.lo[4], box.lo[5], box.lo[6], box.lo[7]);
                    bh[0] = make_uint4(box.hi[0], box.hi[1], box.hi[2], box.hi[3]);
                    bh[1] = make_uint4(box.hi[4], box.hi[5], box.hi[6], box.hi[7]);
                }
            }
            i = j;
        }
    }
}

// One CTA reads `chunk` tokens' slots back.
template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads) read_kernel(const RowsParams p)
{
    extern __shared__ __align__(16) unsigned char smem[];
    Token *tok = reinterpret_cast<Token *>(smem);      // [chunk]
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.chunk;
    const int n = min(p.chunk, p.T - t0);
    // the next kernel may be set up meanwhile (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < n; i += kThreads)
        tok[i] = find_token(p, t0 + i);
    check_rows(p);
    __syncthreads();
    const Share s(p);
    const long long head = (long long)(p.paged ? p.block_size : p.Smax) * p.D;
    constexpr bool kScaled = KIND == GQA_DTYPE_E4M3 || KIND == GQA_DTYPE_E2M1;
    for (int c0 = 0; c0 < s.per; c0 += kThreads) {
        const int c = c0 + s.c;
        if (c >= s.per || s.lane >= s.lanes)
            break;
        const int h = c / (p.D / kGroup), d = (c % (p.D / kGroup)) * kGroup;
        const float ks = kScaled ? __ldg(p.k_scale + h) : 1.f, vs = kScaled ? __ldg(p.v_scale + h) : 1.f;
        const long long row = (long long)p.Hkv * p.D, to = (long long)t0 * row + (long long)c * kGroup;
        for (int m = s.lane; m < n; m += s.lanes) {
            const Token k = tok[m];
            if (k.b < 0)
                continue;                  // of no row: left as it was
            float x[16], y[16];
            if (k.off == kSkip) {
#pragma unroll
                for (int q = 0; q < 16; ++q)
                    x[q] = y[q] = __int_as_float(0x7fc00000);
            } else {
                const long long src = k.off + h * head + d;
                get16<KIND>(p.k_cache, p.k_group, src, ks, x, p.wide);
                get16<KIND>(p.v_cache, p.v_group, src, vs, y, p.wide);
            }
            store_raw(static_cast<T *>(p.k_out) + to + m * row, round16<T>(x), p.wide);
            store_raw(static_cast<T *>(p.v_out) + to + m * row, round16<T>(y), p.wide);
        }
    }
}

template <typename K>
cudaError_t launch(K kernel, const RowsParams &p, size_t smem, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(((long long)p.T + p.chunk - 1) / p.chunk));
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <typename T, int KIND>
cudaError_t launch_append(const RowsParams &p, cudaStream_t st)
{
    if (p.bounds)
        return launch(append_kernel<T, KIND, true>, p,
                      sizeof(Token) * (size_t)(p.chunk + p.bounds_block - 1) + sizeof(Bounds) * kThreads, st);
    return launch(append_kernel<T, KIND, false>, p, sizeof(Token) * (size_t)p.chunk, st);
}

template <int KIND>
cudaError_t launch_kind(const RowsParams &p, bool write, cudaStream_t st)
{
    if (write)
        return p.vec_bf16 ? launch_append<__nv_bfloat16, KIND>(p, st) : launch_append<float, KIND>(p, st);
    const size_t smem = sizeof(Token) * (size_t)p.chunk;
    return p.vec_bf16 ? launch(read_kernel<__nv_bfloat16, KIND>, p, smem, st) : launch(read_kernel<float, KIND>, p, smem, st);
}

}  // namespace

cudaError_t rows_launch(RowsParams p, int kv_dtype, bool write, int sms, cudaStream_t st)
{
    // tokens a CTA: as many as give every SM eight CTAs, at most 64 to append
    // (131071 tokens of 8 x 128 with bounds of 64 slots: 16 tokens 156 us, 32
    // 147, 64 139), 32 to read (113 us; 64: 115)
    const int ctas = sms * 8, most = write ? 64 : 32;
    const long long share = ((long long)p.T + ctas - 1) / ctas;
    p.chunk = share < 1 ? 1 : share > most ? most : (int)share;
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.k_new) | reinterpret_cast<uintptr_t>(p.v_new) |
                         reinterpret_cast<uintptr_t>(p.k_out) | reinterpret_cast<uintptr_t>(p.v_out) |
                         reinterpret_cast<uintptr_t>(p.k_cache) | reinterpret_cast<uintptr_t>(p.v_cache);
    p.wide = (at & 31u) == 0;
    switch (kv_dtype) {
    case GQA_DTYPE_F32: return launch_kind<GQA_DTYPE_F32>(p, write, st);
    case GQA_DTYPE_BF16: return launch_kind<GQA_DTYPE_BF16>(p, write, st);
    case GQA_DTYPE_E4M3: return launch_kind<GQA_DTYPE_E4M3>(p, write, st);
    default: return launch_kind<GQA_DTYPE_E2M1>(p, write, st);
    }
}

}  // namespace gqa
