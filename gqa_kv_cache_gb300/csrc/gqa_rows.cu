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
    if (t0 < 0 || t1 > p.T) {
        rows_report(p, kBadQLen);
        return k;
    }
    k.b = lo;
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

// Sixteen elements at src (element type T) widened to float32.
template <typename T>
__device__ __forceinline__ void load16(const T *src, float (&x)[16])
{
    constexpr int V = sizeof(T) == 4 ? 4 : 2;   // 16-byte loads
    uint4 w[V];
#pragma unroll
    for (int i = 0; i < V; ++i)
        w[i] = __ldg(reinterpret_cast<const uint4 *>(src) + i);
    const uint32_t *u = reinterpret_cast<const uint32_t *>(w);
#pragma unroll
    for (int i = 0; i < 16; ++i) {
        if constexpr (sizeof(T) == 4)
            x[i] = __uint_as_float(u[i]);
        else
            x[i] = (i & 1) ? bf16_hi(u[i / 2]) : bf16_lo(u[i / 2]);
    }
}

template <typename T>
__device__ __forceinline__ void store16(T *dst, const float (&x)[16])
{
    if constexpr (sizeof(T) == 4) {
#pragma unroll
        for (int i = 0; i < 4; ++i)
            reinterpret_cast<float4 *>(dst)[i] = make_float4(x[4 * i], x[4 * i + 1], x[4 * i + 2], x[4 * i + 3]);
    } else {
        uint32_t u[8];
#pragma unroll
        for (int i = 0; i < 8; ++i) {
            const __nv_bfloat162 v = __floats2bfloat162_rn(x[2 * i], x[2 * i + 1]);
            u[i] = *reinterpret_cast<const uint32_t *>(&v);
        }
        reinterpret_cast<uint4 *>(dst)[0] = make_uint4(u[0], u[1], u[2], u[3]);
        reinterpret_cast<uint4 *>(dst)[1] = make_uint4(u[4], u[5], u[6], u[7]);
    }
}

// One group of 16 elements into the cache at element offset `off`.
template <int KIND>
__device__ __forceinline__ void put16(void *cache, void *groups, long long off, float g, const float (&x)[16])
{
    if constexpr (KIND == GQA_DTYPE_F32) {
        store16(static_cast<float *>(cache) + off, x);
    } else if constexpr (KIND == GQA_DTYPE_BF16) {
        store16(static_cast<__nv_bfloat16 *>(cache) + off, x);
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
#pragma unroll
        for (int i = 0; i < 16; ++i)
            amax = max_nan(amax, fabsf(x[i]));
        float t;
        const uint32_t s = group_scale(amax, g, t);
        uint32_t u[2] = {0u, 0u};
#pragma unroll
        for (int i = 0; i < 8; ++i)
            u[i >> 2] |= to_e2m1x2(over_t(x[2 * i], t), over_t(x[2 * i + 1], t)) << (8 * (i & 3));
        *reinterpret_cast<uint2 *>(static_cast<uint8_t *>(cache) + (off >> 1)) = make_uint2(u[0], u[1]);
        static_cast<uint8_t *>(groups)[off >> 4] = (uint8_t)s;
    }
}

// The group at element offset `off` of the cache.
template <int KIND>
__device__ __forceinline__ void get16(const void *cache, const void *groups, long long off, float g, float (&x)[16])
{
    if constexpr (KIND == GQA_DTYPE_F32) {
        load16(static_cast<const float *>(cache) + off, x);
    } else if constexpr (KIND == GQA_DTYPE_BF16) {
        load16(static_cast<const __nv_bfloat16 *>(cache) + off, x);
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

// min (lo) or max of bfloat16 pairs; NaN where either is.
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

// Eight keys at src as bfloat16 pairs: a float32 key's lower bound is rounded
// down and its upper bound up, so that the bounds hold (bfloat16 keys: exact).
template <typename T>
__device__ __forceinline__ void load_bounds8(const T *src, uint32_t (&lo)[4], uint32_t (&hi)[4])
{
    if constexpr (sizeof(T) == 2) {
        const uint4 w = __ldg(reinterpret_cast<const uint4 *>(src));
        lo[0] = hi[0] = w.x;
        lo[1] = hi[1] = w.y;
        lo[2] = hi[2] = w.z;
        lo[3] = hi[3] = w.w;
    } else {
        const float4 a = __ldg(reinterpret_cast<const float4 *>(src));
        const float4 b = __ldg(reinterpret_cast<const float4 *>(src) + 1);
        const float x[8] = {a.x, a.y, a.z, a.w, b.x, b.y, b.z, b.w};
#pragma unroll
        for (int i = 0; i < 4; ++i) {
            const __nv_bfloat16 l0 = __float2bfloat16_rd(x[2 * i]), l1 = __float2bfloat16_rd(x[2 * i + 1]);
            const __nv_bfloat16 h0 = __float2bfloat16_ru(x[2 * i]), h1 = __float2bfloat16_ru(x[2 * i + 1]);
            lo[i] = (uint32_t)__bfloat16_as_ushort(l0) | ((uint32_t)__bfloat16_as_ushort(l1) << 16);
            hi[i] = (uint32_t)__bfloat16_as_ushort(h0) | ((uint32_t)__bfloat16_as_ushort(h1) << 16);
        }
    }
}

// One CTA: `chunk` tokens and, with bounds, the rest of the last run that
// begins among them. Shared memory: the tokens' slots.
template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads) append_kernel(const RowsParams p)
{
    extern __shared__ Token tok[];     // [chunk + run - 1]
    __shared__ int first, last;        // the CTA's tokens: tok[first .. last - 1]
    const int tid = threadIdx.x;
    const int run = p.bounds ? p.bounds_block : 1;
    const int t0 = blockIdx.x * p.chunk;
    const int n = min(p.chunk + run - 1, p.T - t0);   // tokens looked at
    asm volatile("griddepcontrol.wait;" ::: "memory");
    if (tid == 0) {
        first = n;
        last = n;
    }
    __syncthreads();
    for (int i = tid; i < n; i += kThreads) {
        const Token k = find_token(p, t0 + i);
        tok[i] = k;
        // the token begins a run: its block's first slot, or its row's first
        // token (a skipped token is a run of its own)
        const bool begins = run == 1 || k.off == kSkip || k.slot % run == 0 || t0 + i == __ldg(p.cu_q + k.b);
        if (begins) {
            if (i < p.chunk)
                atomicMin(&first, i);
            else
                atomicMin(&last, i);
        }
    }
    __syncthreads();
    const int a = first, e = max(a, last);
    const int per = p.Hkv * (p.D / kGroup);            // groups of a token
    const long long head = (long long)(p.paged ? p.block_size : p.Smax) * p.D;   // elements between heads
    const T *kn = static_cast<const T *>(p.k_new), *vn = static_cast<const T *>(p.v_new);
    const int work = (e - a) * per;
    for (int w = tid; w < work; w += kThreads) {
        const int i = a + w / per, c = w % per;
        const Token k = tok[i];
        if (k.off == kSkip)
            continue;
        const int h = c / (p.D / kGroup), d = (c % (p.D / kGroup)) * kGroup;
        const long long src = ((long long)(t0 + i) * p.Hkv + h) * p.D + d;
        const long long dst = k.off + h * head + d;
        float x[16], y[16];
        load16(kn + src, x);
        load16(vn + src, y);
        const bool scaled = KIND == GQA_DTYPE_E4M3 || KIND == GQA_DTYPE_E2M1;
        put16<KIND>(p.k_cache, p.k_group, dst, scaled ? __ldg(p.k_scale + h) : 1.f, x);
        put16<KIND>(p.v_cache, p.v_group, dst, scaled ? __ldg(p.v_scale + h) : 1.f, y);
    }
    if (!p.bounds)
        return;
    // eight dims of one head a thread, the CTA's runs one after the other (the
    // keys were read above and come from a cache now)
    const int lanes = p.Hkv * (p.D / 8);
    for (int w = tid; w < lanes; w += kThreads) {
        const int h = w / (p.D / 8), d = (w % (p.D / 8)) * 8;
        int i = a;
        while (i < e) {
            const Token k = tok[i];
            if (k.off == kSkip) {
                ++i;
                continue;
            }
            const int block = k.slot / run;
            int j = i + 1;             // one past the run
            while (j < e && tok[j].off != kSkip && tok[j].b == k.b && tok[j].slot / run == block)
                ++j;
            uint32_t lo[4], hi[4];
            load_bounds8(kn + ((long long)(t0 + i) * p.Hkv + h) * p.D + d, lo, hi);
#pragma unroll 4
            for (int m = i + 1; m < j; ++m) {
                uint32_t l[4], u[4];
                load_bounds8(kn + ((long long)(t0 + m) * p.Hkv + h) * p.D + d, l, u);
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    lo[q] = min_bf16x2(lo[q], l[q]);
                    hi[q] = max_bf16x2(hi[q], u[q]);
                }
            }
            // bounds of (block of the row or of the pool, head)
            long long at;
            if (p.paged) {
                at = k.off / ((long long)p.D * p.block_size) + h;   // off is in head 0 of its block
            } else {
                const long long r = p.slot_ids ? __ldg(p.slot_ids + k.b) : k.b;
                at = (r * p.Hkv + h) * (p.Smax / run) + block;
            }
            uint4 *bl = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.bounds) + at * 2 * p.D + d);
            uint4 *bh = reinterpret_cast<uint4 *>(static_cast<__nv_bfloat16 *>(p.bounds) + (at * 2 + 1) * p.D + d);
            if (k.slot % run) {
                const uint4 l = *bl, u = *bh;
                const uint32_t lv[4] = {l.x, l.y, l.z, l.w}, uv[4] = {u.x, u.y, u.z, u.w};
#pragma unroll
                for (int q = 0; q < 4; ++q) {
                    lo[q] = min_bf16x2(lo[q], lv[q]);
                    hi[q] = max_bf16x2(hi[q], uv[q]);
                }
            }
            *bl = make_uint4(lo[0], lo[1], lo[2], lo[3]);
            *bh = make_uint4(hi[0], hi[1], hi[2], hi[3]);
            i = j;
        }
    }
}

// One CTA reads `chunk` tokens' slots back.
template <typename T, int KIND>
__global__ void __launch_bounds__(kThreads) read_kernel(const RowsParams p)
{
    extern __shared__ Token tok[];     // [chunk]
    const int tid = threadIdx.x;
    const int t0 = blockIdx.x * p.chunk;
    const int n = min(p.chunk, p.T - t0);
    asm volatile("griddepcontrol.wait;" ::: "memory");
    for (int i = tid; i < n; i += kThreads)
        tok[i] = find_token(p, t0 + i);
    __syncthreads();
    const int per = p.Hkv * (p.D / kGroup);
    const long long head = (long long)(p.paged ? p.block_size : p.Smax) * p.D;
    for (int w = tid; w < n * per; w += kThreads) {
        const int i = w / per, c = w % per;
        const Token k = tok[i];
        if (k.b < 0)
            continue;                  // of no row: left as it was
        const int h = c / (p.D / kGroup), d = (c % (p.D / kGroup)) * kGroup;
        const long long dst = ((long long)(t0 + i) * p.Hkv + h) * p.D + d;
        float x[16], y[16];
        if (k.off == kSkip) {
#pragma unroll
            for (int q = 0; q < 16; ++q)
                x[q] = y[q] = __int_as_float(0x7fc00000);
        } else {
            const long long src = k.off + h * head + d;
            const bool scaled = KIND == GQA_DTYPE_E4M3 || KIND == GQA_DTYPE_E2M1;
            get16<KIND>(p.k_cache, p.k_group, src, scaled ? __ldg(p.k_scale + h) : 1.f, x);
            get16<KIND>(p.v_cache, p.v_group, src, scaled ? __ldg(p.v_scale + h) : 1.f, y);
        }
        store16(static_cast<T *>(p.k_out) + dst, x);
        store16(static_cast<T *>(p.v_out) + dst, y);
    }
}

template <typename K>
cudaError_t launch(K kernel, const RowsParams &p, int smem_tokens, cudaStream_t st)
{
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((p.T + p.chunk - 1) / p.chunk);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = sizeof(Token) * (size_t)smem_tokens;
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, kernel, p);
}

template <int KIND>
cudaError_t launch_kind(const RowsParams &p, bool write, cudaStream_t st)
{
    if (write) {
        const int tokens = p.chunk + (p.bounds ? p.bounds_block - 1 : 0);
        return p.vec_bf16 ? launch(append_kernel<__nv_bfloat16, KIND>, p, tokens, st)
                          : launch(append_kernel<float, KIND>, p, tokens, st);
    }
    return p.vec_bf16 ? launch(read_kernel<__nv_bfloat16, KIND>, p, p.chunk, st)
                      : launch(read_kernel<float, KIND>, p, p.chunk, st);
}

}  // namespace

cudaError_t rows_launch(RowsParams p, int kv_dtype, bool write, int sms, cudaStream_t st)
{
    // tokens a CTA: as many as give every SM a few CTAs, at most 32 (a run of
    // 64 in the bounds form costs that CTA two shares)
    const int ctas = sms * 8;
    p.chunk = (p.T + ctas - 1) / ctas;
    p.chunk = p.chunk < 1 ? 1 : p.chunk > 32 ? 32 : p.chunk;
    switch (kv_dtype) {
    case GQA_DTYPE_F32: return launch_kind<GQA_DTYPE_F32>(p, write, st);
    case GQA_DTYPE_BF16: return launch_kind<GQA_DTYPE_BF16>(p, write, st);
    case GQA_DTYPE_E4M3: return launch_kind<GQA_DTYPE_E4M3>(p, write, st);
    default: return launch_kind<GQA_DTYPE_E2M1>(p, write, st);
    }
}

}  // namespace gqa
