// Rotary positions: over the first `dim` elements of a head, pair i of a token
// at position pos becomes m (x cos a - y sin a, x sin a + y cos a), a = pos f_i;
// the elements behind `dim` stay as they are. Pair i is (i, i + dim / 2) or
// (2 i, 2 i + 1).
//
// Angles. f_i is given as a fraction of a turn in 64-bit fixed point
// (f_i / 2 pi 2^64, rounded once), so pos f_i mod a turn is the wrapped integer
// product: within 2^-34 of a turn for every int32 position, without 64-bit
// floating point (which this GPU has little of). Its first 32 bits are used
// (another 2^-32 of a turn, 1.5e-9 radians): the nearest quarter turn is taken
// off in integers, and cos and sin of the rest (|a| <= pi / 4, a 30-bit integer
// rounded to float32: 2.4e-8) come from sincospif (one step, 6e-8): both are off
// by less than 2^-23 (1.19e-7).
//
// A CTA takes a few tokens (or a part of one's heads): the angles of a token,
// shared by all heads of q and k, go through shared memory while the first
// vectors are on their way. A thread keeps its place in the heads from token to
// token. Bound by memory: every vector is read and written once, 16 bytes a
// thread at a time (65521 tokens of 56 heads of 128 in bfloat16, half of each
// turned: 289 us, 0.96 of the measured copy rate); sizes and strides that 16 bytes
// do not fit go by 8, 4 or single elements.
#include "gqa_common.cuh"
#include "gqa_launch.h"

namespace gqa {
namespace {

constexpr int kThreads = 256;

__device__ __forceinline__ float2 turn(uint64_t x, float m)
{
    const uint32_t h = (uint32_t)(x >> 32);
    const uint32_t q = (h + 0x20000000u) >> 30;         // nearest quarter
    const float f = (float)(int)(h - (q << 30)) * 0x1p-31f;   // the rest in half turns
    float s, c;
    sincospif(f, &s, &c);
    const float a = q & 1 ? -s : c, b = q & 1 ? c : s;
    return q & 2 ? make_float2(-a * m, -b * m) : make_float2(a * m, b * m);
}

// N elements of type T, 16 bytes of them or fewer.
template <typename T, int N>
struct alignas(sizeof(T) * N) Vec {
    T x[N];
};

__device__ __forceinline__ float wide(float v) { return v; }
__device__ __forceinline__ float wide(__nv_bfloat16 v) { return __bfloat162float(v); }
template <typename T>
__device__ __forceinline__ T narrow(float v);
template <>
__device__ __forceinline__ float narrow<float>(float v) { return v; }
template <>
__device__ __forceinline__ __nv_bfloat16 narrow<__nv_bfloat16>(float v) { return __float2bfloat16_rn(v); }

// Position of token t; false: a token of no row.
__device__ __forceinline__ bool position(const RotateParams &p, int t, int &pos)
{
    if (p.positions) {
        pos = __ldg(p.positions + t);
        return true;
    }
    if (p.B == 0)
        return false;
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
        return false;
    if (t0 < 0 || t1 > p.T) {
        if (p.status)
            atomicOr(p.status, kBadQLen);
        return false;
    }
    pos = (int)((unsigned)__ldg(p.lengths + lo) + (unsigned)(t - t0));
    return true;
}

// What a thread turns in every token it takes: N elements (HALF: of each half of
// the turned elements, or of those behind them) of one head.
template <typename T>
struct Place {
    const T *src;      // in token 0
    T *dst;
    long long from, to;   // elements between tokens
    int i;             // first pair, or -1: elements behind `dim`
    int gap;           // elements to the second N (0: there are none)
};

template <typename T, int N, bool HALF>
__device__ __forceinline__ Place<T> find(const RotateParams &p, int x)
{
    Place<T> w;
    const int head = x / p.units, c = x - head * p.units;
    const bool key = head >= p.Hq;
    const int h = key ? head - p.Hq : head;
    w.from = key ? p.k_token : p.q_token;
    w.to = key ? p.ko_token : p.qo_token;
    w.src = static_cast<const T *>(key ? p.k : p.q) + h * (key ? p.k_head : p.q_head);
    w.dst = static_cast<T *>(key ? p.k_out : p.q_out) + h * (key ? p.ko_head : p.qo_head);
    // units of turned elements: dim / (2 N) pairs of pieces; N = 1 (2 elements) else N / 2 pairs
    const int turned = HALF || N == 1 ? p.dim / 2 / N : p.dim / N;
    const int d = c >= turned ? p.dim + (c - turned) * N : HALF ? c * N : N == 1 ? 2 * c : c * N;
    w.i = c >= turned ? -1 : HALF ? c * N : N == 1 ? c : c * (N / 2);
    // (HALF: elements behind `dim` go by two pieces too where they are even)
    w.gap = c >= turned ? p.rest_gap : HALF ? p.dim / 2 : N == 1 ? 1 : 0;
    w.src += d;
    w.dst += d;
    return w;
}

template <typename T, int N, bool HALF>
struct Unit {
    Vec<T, N> a, b;
};

template <typename T, int N, bool HALF>
__device__ __forceinline__ void load(const RotateParams &p, const Place<T> &at, int t, Unit<T, N, HALF> &w)
{
    const T *src = at.src + t * at.from;
    w.a = *reinterpret_cast<const Vec<T, N> *>(src);
    if ((HALF || N == 1) && at.gap)
        w.b = *reinterpret_cast<const Vec<T, N> *>(src + at.gap);
}

template <typename T, int N, bool HALF>
__device__ __forceinline__ void store(const RotateParams &p, const Place<T> &at, int t, Unit<T, N, HALF> &w, const float2 *cs,
                                      bool known)
{
    T *dst = at.dst + t * at.to;
    if (at.i >= 0 && known) {
        if constexpr (HALF || N == 1) {
#pragma unroll
            for (int j = 0; j < N; ++j) {
                const float2 e = cs[at.i + j];
                const float x = wide(w.a.x[j]), y = wide(w.b.x[j]);
                w.a.x[j] = narrow<T>(x * e.x - y * e.y);
                w.b.x[j] = narrow<T>(x * e.y + y * e.x);
            }
        } else {
#pragma unroll
            for (int j = 0; j < N / 2; ++j) {
                const float2 e = cs[at.i + j];
                const float x = wide(w.a.x[2 * j]), y = wide(w.a.x[2 * j + 1]);
                w.a.x[2 * j] = narrow<T>(x * e.x - y * e.y);
                w.a.x[2 * j + 1] = narrow<T>(x * e.y + y * e.x);
            }
        }
    }
    *reinterpret_cast<Vec<T, N> *>(dst) = w.a;
    if ((HALF || N == 1) && at.gap)
        *reinterpret_cast<Vec<T, N> *>(dst + at.gap) = w.b;
}


// blockIdx.x: `tokens` tokens; blockIdx.y: a part of their units. A thread keeps
// its place in the heads from token to token.
template <typename T, int N, bool HALF>
__global__ void __launch_bounds__(kThreads, 3) rotate_kernel(const RotateParams p)
{
    extern __shared__ float2 cs[];             // [tokens][dim / 2]
    __shared__ int known[32];                  // whether the token has a position
    const int tid = threadIdx.x, pairs = p.dim / 2;
    const int t0 = blockIdx.x * p.tokens, n = min(p.tokens, p.T - t0);
    const int all = (p.Hq + p.Hkv) * p.units;  // units a token
    const int u0 = (int)((long long)all * blockIdx.y / gridDim.y), u1 = (int)((long long)all * (blockIdx.y + 1) / gridDim.y);
    const int per = u1 - u0;
    const int lanes = per >= kThreads ? 1 : kThreads / per;         // tokens at once
    const int lane = per >= kThreads ? 0 : tid / per, c = per >= kThreads ? tid : tid % per;
    // the next kernel may be set up meanwhile (it waits for this one's end)
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int M = (HALF ? 2 : 4) * (16 / (N * (int)sizeof(T))), A = M < 8 ? M : 8;   // tokens of a thread on their way at once
    Place<T> at, next;
    Unit<T, N, HALF> w[A], v[A];
    const bool mine = c < per && lane < lanes;
    auto fetch = [&](const Place<T> &from, int t, Unit<T, N, HALF> (&to)[A]) {
#pragma unroll
        for (int a = 0; a < A; ++a)
            if (t + a * lanes < n)
                load(p, from, t0 + t + a * lanes, to[a]);
    };
    if (mine) {
        next = at = find<T, N, HALF>(p, u0 + c);
        fetch(at, lane, w);                    // before the angles
    }
    for (int i = tid; i < n * pairs; i += kThreads) {
        const int t = i / pairs, j = i - t * pairs;
        int pos = 0;
        const bool ok = position(p, t0 + t, pos);
        if (j == 0)
            known[t] = ok;
        cs[i] = turn((uint64_t)(int64_t)pos * __ldg(p.freqs + j), p.factor);
    }
    if (p.cu_q && blockIdx.y == 0)
        for (long long b = (long long)blockIdx.x * kThreads + tid; b < p.B; b += (long long)gridDim.x * kThreads) {
            const int a = __ldg(p.cu_q + b), e = __ldg(p.cu_q + b + 1);
            if ((a < 0 || e < a || e > p.T) && p.status)
                atomicOr(p.status, kBadQLen);
        }
    __syncthreads();
    if (!mine)
        return;
    int x = c, t = lane;
    while (true) {
        // the next tokens (or the next place's first) are on their way while these are turned
        int s = t + A * lanes;
        if (s >= n) {
            s = lane;
            x += kThreads;                     // (per < kThreads: there is none)
            if (x < per)
                next = find<T, N, HALF>(p, u0 + x);
        }
        if (x < per)
            fetch(next, s, v);
#pragma unroll
        for (int a = 0; a < A; ++a) {
            const int k = t + a * lanes;
            if (k < n)
                store(p, at, t0 + k, w[a], cs + k * pairs, known[k]);
        }
        if (x >= per)
            break;
        at = next;
        t = s;
#pragma unroll
        for (int a = 0; a < A; ++a)
            w[a] = v[a];
    }
}

template <typename T, int N, bool HALF>
cudaError_t launch(RotateParams &p, int sms, cudaStream_t st)
{
    const int turned = HALF || N == 1 ? p.dim / 2 / N : p.dim / N;
    const int pieces = (p.D - p.dim) / N;
    p.rest_gap = HALF && pieces && pieces % 2 == 0 ? (p.D - p.dim) / 2 : 0;
    p.units = turned + (p.rest ? p.rest_gap ? pieces / 2 : pieces : 0);
    const long long all = (long long)(p.Hq + p.Hkv) * p.units;
    // tokens a CTA: as many as leave every SM eight CTAs, at most 16 (65521 tokens
    // of 56 heads: 8 304 us, 16 289, 32 302) and 32 KB of angles; parts of a
    // token's heads where there are few tokens
    const long long share = p.T / ((long long)sms * 8), most = p.dim <= 512 ? 16 : 8192 / p.dim;
    p.tokens = share < 1 ? 1 : share > most ? (int)most : (int)share;
    const long long ctas = ((long long)p.T + p.tokens - 1) / p.tokens;
    long long parts = (all * p.tokens + kThreads - 1) / kThreads, room = (long long)sms * 4 / ctas;
    parts = parts > room ? room : parts;
    parts = parts < 1 ? 1 : parts > 64 ? 64 : parts;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)ctas, (unsigned)parts);
    cfg.blockDim = dim3(kThreads);
    cfg.dynamicSmemBytes = (size_t)p.tokens * (p.dim / 2) * sizeof(float2);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return cudaLaunchKernelEx(&cfg, rotate_kernel<T, N, HALF>, p);
}

// The widest pieces (at most 16 bytes) that addresses, strides and the parts of
// a head fit.
template <typename T, int N>
cudaError_t launch_type(RotateParams &p, int sms, cudaStream_t st)
{
    const uintptr_t at = reinterpret_cast<uintptr_t>(p.q) | reinterpret_cast<uintptr_t>(p.k) |
                         reinterpret_cast<uintptr_t>(p.q_out) | reinterpret_cast<uintptr_t>(p.k_out);
    const long long strides = p.q_token | p.q_head | p.k_token | p.k_head | p.qo_token | p.qo_head | p.ko_token | p.ko_head;
    if constexpr (N > 1) {
        if (at % (N * sizeof(T)) || strides % N || (p.D - p.dim) % N || (p.half ? p.dim / 2 : p.dim) % N)
            return launch_type<T, N / 2>(p, sms, st);
    }
    return p.half ? launch<T, N, true>(p, sms, st) : launch<T, N, false>(p, sms, st);
}

}  // namespace

cudaError_t rotate_launch(RotateParams p, int sms, cudaStream_t st)
{
    // in place the elements behind `dim` need no copy
    p.rest = p.q_out != p.q || p.k_out != p.k || p.qo_token != p.q_token || p.qo_head != p.q_head ||
             p.ko_token != p.k_token || p.ko_head != p.k_head;
    return p.bf16 ? launch_type<__nv_bfloat16, 8>(p, sms, st) : launch_type<float, 4>(p, sms, st);
}

}  // namespace gqa
