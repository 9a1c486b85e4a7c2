// Host side of the scored attend (gqa_scored_kernel.cuh) and the kernel that
// adds a step's attention weights to the slots' counts.
#include "gqa_scored_kernel.cuh"

namespace gqa {

using Launch = cudaError_t(bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm);
Launch scored_i8_128_few_more, scored_i8_128_few, scored_i8_128_rows_more, scored_i8_128_rows,
    scored_i8_64_few_more, scored_i8_64_few, scored_i8_64_rows_more, scored_i8_64_rows,
    scored_bf16_128, scored_bf16_64;

namespace {

using scored::kFew;
using scored::kRows;

// more: capped, biased or counted scores (over a bfloat16 cache always)
cudaError_t launch(int kind, int D, int G, bool more, bool q_bf16, bool paged, const ScoredParams *p, cudaStream_t st, int *per_sm)
{
    Launch *const of[2][2][2] = {{{scored_i8_64_rows, scored_i8_64_rows_more}, {scored_i8_64_few, scored_i8_64_few_more}},
                                 {{scored_i8_128_rows, scored_i8_128_rows_more}, {scored_i8_128_few, scored_i8_128_few_more}}};
    Launch *f = kind == kI8 ? of[D == 128][G <= kFew][more] : D == 128 ? scored_bf16_128 : scored_bf16_64;
    return f(q_bf16, paged, p, st, per_sm);
}

constexpr int kCountThreads = 256, kCountSlots = 4;   // slots a thread

// weights[slot] += sum over the rows of 2^(y - M) / den (the bias, which may be
// as large as M, meets M in one rounding): the scores of a slot are neighbours, 16
// or 32 bytes. Bound by memory: 4 G + 8 bytes a slot (327k
// slots of 8 heads, G = 8: 105 MB, part of it from L2). Added in L2, which lets
// rows share blocks and spares a load (attend and counts 244 -> 239 us).
template <int GP, bool SLOPES>
__global__ void __launch_bounds__(kCountThreads) count_kernel(const ScoredParams p)
{
    asm volatile("griddepcontrol.launch_dependents;" ::: "memory");
    asm volatile("griddepcontrol.wait;" ::: "memory");
    constexpr int share = kCountThreads * kCountSlots;
    const unsigned parts = (unsigned)((p.xs_cap + share - 1) / share);
    const int unit = blockIdx.x / parts, b = unit / p.Hkv, kvh = unit % p.Hkv;
    const RowGeom r = row_geom_inl(p, b);
    const int j0 = (int)(blockIdx.x % parts) * share;
    if (j0 > r.L || !row_ok(p, b, r.L))
        return;
    float M[GP], inv[GP];
    [[maybe_unused]] float slope[SLOPES ? GP : 1];
#pragma unroll
    for (int g = 0; g < GP; ++g) {
        const float2 e = g < p.G ? p.row_end[(long long)b * p.Hq + kvh * p.G + g] : make_float2(0.f, 0.f);
        M[g] = e.x;
        inv[g] = e.y;
        if constexpr (SLOPES)
            slope[g] = g < p.G ? __ldg(p.slopes + kvh * p.G + g) * 1.4426950408889634f : 0.f;
    }
    long long line = 0;
    if (!p.paged)
        line = ((long long)(p.slot_ids ? __ldg(p.slot_ids + b) : b) * p.Hkv + kvh) * p.Smax;
    const float4 *xs = reinterpret_cast<const float4 *>(p.xs + (long long)unit * p.xs_cap * GP);
#pragma unroll
    for (int i = 0; i < kCountSlots; ++i) {
        const int j = j0 + i * kCountThreads + (int)threadIdx.x;
        if (!attended(r.L, r.lo, r.P, j))
            continue;
        long long at = line + j;
        if (p.paged) {
            const int blk = __ldg(p.block_table + (long long)b * p.max_blocks + j / p.block_size);
            if (blk < 0 || blk >= p.num_blocks)
                continue;
            at = ((long long)blk * p.Hkv + kvh) * p.block_size + j % p.block_size;
        }
        [[maybe_unused]] const float far = (float)(j - r.L);
        float sum = 0.f;
#pragma unroll
        for (int k = 0; k < GP / 4; ++k) {
            const float4 x = xs[(long long)j * (GP / 4) + k];
            const float y[4] = {x.x, x.y, x.z, x.w};
#pragma unroll
            for (int g = 0; g < 4; ++g)
                if (4 * k + g < p.G) {
                    if constexpr (SLOPES)
                        sum += fast_ex2(y[g] + fmaf(slope[4 * k + g], far, -M[4 * k + g])) * inv[4 * k + g];
                    else
                        sum += fast_ex2(y[g] - M[4 * k + g]) * inv[4 * k + g];
                }
        }
        atomicAdd(p.weights + at, sum);        // rows may share a block; a slot of one row has one writer
    }
}

template <int GP>
cudaError_t launch_count(const ScoredParams &p, cudaStream_t st)
{
    constexpr int share = kCountThreads * kCountSlots;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3((unsigned)(p.B * p.Hkv * ((p.xs_cap + share - 1) / share)));
    cfg.blockDim = dim3(kCountThreads);
    cfg.stream = st;
    cudaLaunchAttribute attr[1];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    cfg.attrs = attr;
    cfg.numAttrs = 1;
    return p.slopes ? cudaLaunchKernelEx(&cfg, count_kernel<GP, true>, p) : cudaLaunchKernelEx(&cfg, count_kernel<GP, false>, p);
}

}  // namespace

bool scored_supports(int kind, int D, int G)
{
    return (kind == kBf16 || kind == kI8) && (D == 64 || D == 128) && G >= 1 && G <= kRows;
}

int scored_tile(int kind, int D)
{
    if (kind == kI8)
        return D == 128 ? scored::Form<kI8, 128>::TILE : scored::Form<kI8, 64>::TILE;
    return D == 128 ? scored::Form<kBf16, 128>::TILE : scored::Form<kBf16, 64>::TILE;
}

// One CTA a unit, whole, where units are short: no schedule to assemble, no
// partial states to merge.
bool scored_whole_units(int kind, int D, long long capacity, long long units, int grid)
{
    const int tile = scored_tile(kind, D);
    return capacity <= 4 * tile || (capacity <= 8 * tile && units <= grid);
}

int scored_ctas_per_sm(int kind, int D, int G, bool more, bool q_bf16)
{
    int least = 1 << 30;
    for (bool paged : {false, true}) {
        int n = 0;
        if (launch(kind, D, G, more, q_bf16, paged, nullptr, nullptr, &n) != cudaSuccess)
            return 1;
        least = n < least ? n : least;
    }
    return least > 0 ? least : 1;
}

long long scored_count_ctas(int B, int Hkv, long long capacity)
{
    constexpr int share = kCountThreads * kCountSlots;
    return (long long)B * Hkv * ((capacity + share - 1) / share);
}

size_t scored_scratch_bytes(int B, int Hq, int Hkv, long long capacity)
{
    const size_t gp = Hq / Hkv <= kFew ? 4 : 8;
    return align_up((size_t)B * Hkv * (size_t)capacity * gp * sizeof(float), 256) + (size_t)B * Hq * sizeof(float2);
}

cudaError_t scored_launch(const ScoredParams &p, cudaStream_t st)
{
    const cudaError_t e = launch(p.kind, p.D, p.G, p.cap > 0.f || p.slopes || p.weights, p.q_bf16, p.paged, &p, st, nullptr);
    if (e != cudaSuccess || !p.weights)
        return e;
    return p.gp == 4 ? launch_count<4>(p, st) : launch_count<8>(p, st);
}

}  // namespace gqa
