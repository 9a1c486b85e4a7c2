// C ABI of the calls around the decode step (include/gqa_decode.h): append,
// read and block selection. Host-side argument checks and launches.
#include <atomic>
#include <climits>

#include "gqa_decode.h"
#include "gqa_launch.h"

using namespace gqa;

namespace {

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }

bool vec_dtype(gqa_dtype d) { return d == GQA_DTYPE_F32 || d == GQA_DTYPE_BF16; }

// Streaming multiprocessors of the current device (0: a CUDA error).
int current_sms()
{
    constexpr int kDevices = 64;
    static std::atomic<int> cache[kDevices];
    int dev = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0)
        return 0;
    int n = dev < kDevices ? cache[dev].load(std::memory_order_relaxed) : 0;
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        if (dev < kDevices)
            cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

gqa_status run_rows(RowsParams p, gqa_dtype vec, gqa_dtype kv, bool write, void *stream, const gqa_options *opt)
{
    if (p.B < 0 || p.T < 0 || p.Hkv < 1 || p.D < 1 || !vec_dtype(vec) || kv < GQA_DTYPE_F32 || kv > GQA_DTYPE_I8)
        return GQA_ERR_INVALID_ARGUMENT;
    if (p.paged) {
        if (p.num_blocks < 1 || p.block_size < 1 || p.max_blocks < 1 ||
            (long long)p.max_blocks * p.block_size > INT_MAX)
            return GQA_ERR_INVALID_ARGUMENT;
    } else if (p.R < 0 || p.Smax < 1) {
        return GQA_ERR_INVALID_ARGUMENT;
    }
    if (p.D % 16 || (long long)p.Hkv * p.D > (1 << 24))
        return GQA_ERR_UNSUPPORTED;
    if (p.bounds) {
        if (p.bounds_block < 1 || (!p.paged && p.Smax % p.bounds_block))
            return GQA_ERR_INVALID_ARGUMENT;
        if (p.bounds_block > 1024)
            return GQA_ERR_UNSUPPORTED;
    }
    if (kv == GQA_DTYPE_I8) {
        if (p.bounds)
            return GQA_ERR_UNSUPPORTED;
        if (!opt || !opt->k_block_scale || !opt->v_block_scale || !aligned(opt->k_block_scale, 4) ||
            !aligned(opt->v_block_scale, 4))
            return GQA_ERR_INVALID_ARGUMENT;
        p.scale_block = p.paged ? p.block_size : opt->scale_block;
        if (p.scale_block < 1 || (!p.paged && p.Smax % p.scale_block))
            return GQA_ERR_INVALID_ARGUMENT;
        if (write && !append8_supports(p.scale_block, p.Hkv, p.D))
            return GQA_ERR_UNSUPPORTED;
        p.k_block_scale = opt->k_block_scale;
        p.v_block_scale = opt->v_block_scale;
    } else if (kv >= GQA_DTYPE_E4M3) {
        if (!opt || !opt->k_scale || !opt->v_scale || !aligned(opt->k_scale, 4) || !aligned(opt->v_scale, 4))
            return GQA_ERR_INVALID_ARGUMENT;
        p.k_scale = opt->k_scale;
        p.v_scale = opt->v_scale;
    }
    if (p.B == 0 || p.T == 0)
        return GQA_OK;
    if (kv == GQA_DTYPE_E2M1) {
        if (!opt->k_group_scale || !opt->v_group_scale || !aligned(opt->k_group_scale, 16) ||
            !aligned(opt->v_group_scale, 16))
            return GQA_ERR_INVALID_ARGUMENT;
        p.k_group = opt->k_group_scale;
        p.v_group = opt->v_group_scale;
    }
    const void *a = write ? p.k_new : p.k_out, *b = write ? p.v_new : p.v_out;
    if (!a || !b || !p.k_cache || !p.v_cache || !p.lengths || !p.cu_q || (p.paged && !p.block_table) ||
        (!p.paged && !p.slot_ids && p.R < p.B))
        return GQA_ERR_INVALID_ARGUMENT;
    if (!aligned(a, 16) || !aligned(b, 16) || !aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) ||
        !aligned(p.bounds, 16))
        return GQA_ERR_INVALID_ARGUMENT;
    const int sms = current_sms();
    if (!sms)
        return GQA_ERR_CUDA;
    p.vec_bf16 = vec == GQA_DTYPE_BF16;
    return rows_launch(p, kv, write, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status run_select(const SelectParams &p, gqa_dtype q_dtype, void *stream)
{
    if (p.B < 0 || p.Hq < 1 || p.Hkv < 1 || p.Hq % p.Hkv || p.D < 1 || !vec_dtype(q_dtype) || p.NB < 1 ||
        p.block_size < 1 || (long long)p.NB * p.block_size > INT_MAX)
        return GQA_ERR_INVALID_ARGUMENT;
    if (p.paged ? p.num_blocks < 1 : p.R < 0)
        return GQA_ERR_INVALID_ARGUMENT;
    if (p.n_first < 0 || p.n_last < 1 || p.n_select < 1 || (long long)p.n_first + p.n_last > p.n_select)
        return GQA_ERR_INVALID_ARGUMENT;
    const long long pool = p.paged ? (long long)p.num_blocks * p.Hkv : (long long)p.R * p.Hkv * p.NB;
    if (!select_supports(p.D, p.NB) || pool > INT_MAX || (long long)p.n_select * p.block_size > INT_MAX ||
        (long long)p.B * p.Hkv > (1 << 24))
        return GQA_ERR_UNSUPPORTED;
    if (p.B == 0)
        return GQA_OK;
    if (!p.q || !p.bounds || !p.lengths || !p.ids || !p.table || !p.sel_lengths || (p.paged && !p.block_table) ||
        (!p.paged && !p.slot_ids && p.R < p.B))
        return GQA_ERR_INVALID_ARGUMENT;
    if (!aligned(p.q, 16) || !aligned(p.bounds, 16))
        return GQA_ERR_INVALID_ARGUMENT;
    const int sms = current_sms();
    if (!sms)
        return GQA_ERR_CUDA;
    return select_launch(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

extern "C" {

gqa_status gqa_append(const void *k_new, const void *v_new, gqa_dtype new_dtype, void *k_cache, void *v_cache,
                      const int32_t *lengths, const int32_t *cu_q, const int32_t *slot_ids, void *k_bounds,
                      int bounds_block, int B, int T, int Hkv, int D, int R, int Smax, gqa_dtype kv_dtype,
                      int32_t *d_status, void *stream, const gqa_options *opt)
{
    RowsParams p = {};
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.bounds = k_bounds;
    p.bounds_block = bounds_block;
    p.lengths = lengths;
    p.cu_q = cu_q;
    p.slot_ids = slot_ids;
    p.status = d_status;
    p.B = B;
    p.T = T;
    p.Hkv = Hkv;
    p.D = D;
    p.R = R;
    p.Smax = Smax;
    return run_rows(p, new_dtype, kv_dtype, true, stream, opt);
}

gqa_status gqa_append_paged(const void *k_new, const void *v_new, gqa_dtype new_dtype, void *k_blocks,
                            void *v_blocks, const int32_t *block_table, const int32_t *lengths,
                            const int32_t *cu_q, void *k_bounds, int B, int T, int Hkv, int D, int num_blocks,
                            int block_size, int max_blocks, gqa_dtype kv_dtype, int32_t *d_status, void *stream,
                            const gqa_options *opt)
{
    RowsParams p = {};
    p.k_new = k_new;
    p.v_new = v_new;
    p.k_cache = k_blocks;
    p.v_cache = v_blocks;
    p.bounds = k_bounds;
    p.bounds_block = block_size;
    p.lengths = lengths;
    p.cu_q = cu_q;
    p.block_table = block_table;
    p.status = d_status;
    p.B = B;
    p.T = T;
    p.Hkv = Hkv;
    p.D = D;
    p.paged = 1;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks = max_blocks;
    return run_rows(p, new_dtype, kv_dtype, true, stream, opt);
}

gqa_status gqa_read(const void *k_cache, const void *v_cache, const int32_t *lengths, const int32_t *cu_q,
                    const int32_t *slot_ids, void *k_out, void *v_out, gqa_dtype out_dtype, int B, int T, int Hkv,
                    int D, int R, int Smax, gqa_dtype kv_dtype, int32_t *d_status, void *stream,
                    const gqa_options *opt)
{
    RowsParams p = {};
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_cache = const_cast<void *>(k_cache);   // only read
    p.v_cache = const_cast<void *>(v_cache);
    p.lengths = lengths;
    p.cu_q = cu_q;
    p.slot_ids = slot_ids;
    p.status = d_status;
    p.B = B;
    p.T = T;
    p.Hkv = Hkv;
    p.D = D;
    p.R = R;
    p.Smax = Smax;
    return run_rows(p, out_dtype, kv_dtype, false, stream, opt);
}

gqa_status gqa_read_paged(const void *k_blocks, const void *v_blocks, const int32_t *block_table,
                          const int32_t *lengths, const int32_t *cu_q, void *k_out, void *v_out, gqa_dtype out_dtype,
                          int B, int T, int Hkv, int D, int num_blocks, int block_size, int max_blocks,
                          gqa_dtype kv_dtype, int32_t *d_status, void *stream, const gqa_options *opt)
{
    RowsParams p = {};
    p.k_out = k_out;
    p.v_out = v_out;
    p.k_cache = const_cast<void *>(k_blocks);
    p.v_cache = const_cast<void *>(v_blocks);
    p.lengths = lengths;
    p.cu_q = cu_q;
    p.block_table = block_table;
    p.status = d_status;
    p.B = B;
    p.T = T;
    p.Hkv = Hkv;
    p.D = D;
    p.paged = 1;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks = max_blocks;
    return run_rows(p, out_dtype, kv_dtype, false, stream, opt);
}

gqa_status gqa_select_blocks(const void *q, gqa_dtype q_dtype, const void *k_bounds, const int32_t *lengths,
                             const int32_t *slot_ids, int32_t *ids, int32_t *table, int32_t *sel_lengths, int B,
                             int Hq, int Hkv, int D, int R, int NB, int block_size, int n_select, int n_first,
                             int n_last, int32_t *d_status, void *stream)
{
    SelectParams p = {};
    p.q = q;
    p.q_bf16 = q_dtype == GQA_DTYPE_BF16;
    p.bounds = k_bounds;
    p.lengths = lengths;
    p.slot_ids = slot_ids;
    p.ids = ids;
    p.table = table;
    p.sel_lengths = sel_lengths;
    p.status = d_status;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.R = R;
    p.NB = NB;
    p.block_size = block_size;
    p.n_select = n_select;
    p.n_first = n_first;
    p.n_last = n_last;
    return run_select(p, q_dtype, stream);
}

gqa_status gqa_select_blocks_paged(const void *q, gqa_dtype q_dtype, const void *k_bounds,
                                   const int32_t *block_table, const int32_t *lengths, int32_t *ids,
                                   int32_t *table, int32_t *sel_lengths, int B, int Hq, int Hkv, int D,
                                   int num_blocks, int block_size, int max_blocks, int n_select, int n_first,
                                   int n_last, int32_t *d_status, void *stream)
{
    SelectParams p = {};
    p.q = q;
    p.q_bf16 = q_dtype == GQA_DTYPE_BF16;
    p.bounds = k_bounds;
    p.lengths = lengths;
    p.block_table = block_table;
    p.ids = ids;
    p.table = table;
    p.sel_lengths = sel_lengths;
    p.status = d_status;
    p.B = B;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.NB = max_blocks;
    p.paged = 1;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.n_select = n_select;
    p.n_first = n_first;
    p.n_last = n_last;
    return run_select(p, q_dtype, stream);
}

}  // extern "C"
