// C ABI of rotary positions and eviction (include/gqa_decode.h): host-side
// argument checks and launches.
#include <atomic>
#include <climits>

#include "gqa_decode.h"
#include "gqa_launch.h"

using namespace gqa;

namespace {

// Streaming multiprocessors of the current device (0: a CUDA error).
int current_sms()
{
    constexpr int kDevices = 64;
    static std::atomic<int> cache[kDevices];
    int dev = 0, n = 0;
    if (cudaGetDevice(&dev) != cudaSuccess || dev < 0)
        return 0;
    if (dev < kDevices)
        n = cache[dev].load(std::memory_order_relaxed);
    if (!n) {
        if (cudaDeviceGetAttribute(&n, cudaDevAttrMultiProcessorCount, dev) != cudaSuccess)
            return 0;
        if (dev < kDevices)
            cache[dev].store(n, std::memory_order_relaxed);
    }
    return n;
}

bool aligned(const void *p, unsigned a) { return (reinterpret_cast<uintptr_t>(p) & (a - 1u)) == 0; }

bool apart(const void *a, double na, const void *b, double nb)
{
    const double x = (double)reinterpret_cast<uintptr_t>(a), y = (double)reinterpret_cast<uintptr_t>(b);
    return x + na <= y || y + nb <= x;
}

gqa_status run_evict(EvictParams p, int D, gqa_dtype kv, void *stream)
{
    if (p.B < 0 || p.Hkv < 1 || D < 1 || kv < GQA_DTYPE_F32 || kv > GQA_DTYPE_I8)
        return GQA_ERR_INVALID_ARGUMENT;
    if (p.paged) {
        if (p.num_blocks < 1 || p.block_size < 1 || p.max_blocks < 1 ||
            (long long)p.max_blocks * p.block_size > INT_MAX)
            return GQA_ERR_INVALID_ARGUMENT;
    } else if (p.R < 0 || p.Smax < 1) {
        return GQA_ERR_INVALID_ARGUMENT;
    }
    if (p.n_keep < 1 || p.n_first < 0 || p.n_last < 0 || (long long)p.n_first + p.n_last > p.n_keep)
        return GQA_ERR_INVALID_ARGUMENT;
    if (!p.k_out != !p.v_out || (p.weights_out && !p.k_out) || (p.k_out && p.out_slots < p.n_keep))
        return GQA_ERR_INVALID_ARGUMENT;
    if (kv > GQA_DTYPE_E4M3)
        return GQA_ERR_UNSUPPORTED;      // vectors that share scales with their neighbours, or keep them elsewhere
    const long long row = (long long)D * (kv == GQA_DTYPE_F32 ? 4 : kv == GQA_DTYPE_BF16 ? 2 : 1);
    const long long cap = p.paged ? (long long)p.max_blocks * p.block_size : (long long)p.Smax;
    const long long moved = p.n_keep < cap ? p.n_keep : cap;
    // (the kernels step over slots, kept slots and places of the outputs in 32 bits)
    if (row % 16 || row > (1 << 20) || cap > (1 << 30) || p.n_keep > (1 << 30) || p.out_slots > (1 << 30) ||
        (long long)p.B * p.Hkv > (1 << 24) ||
        (double)p.B * p.Hkv * ((double)moved * row / (1 << 15) + row / 16.0 + 1.0) > INT_MAX ||
        (double)moved * row / 16 > INT_MAX)
        return GQA_ERR_UNSUPPORTED;
    if (p.B == 0)
        return GQA_OK;
    if (!p.k_cache || !p.v_cache || !p.weights || !p.lengths || !p.ids || !p.new_lengths || (p.paged && !p.block_table) ||
        (!p.paged && !p.slot_ids && p.R < p.B) || p.lengths == p.new_lengths)
        return GQA_ERR_INVALID_ARGUMENT;
    if (!aligned(p.k_cache, 16) || !aligned(p.v_cache, 16) || !aligned(p.k_out, 16) || !aligned(p.v_out, 16) ||
        !aligned(p.weights, 4) || !aligned(p.weights_out, 4))
        return GQA_ERR_INVALID_ARGUMENT;
    if (p.k_out) {
        const double vectors = p.paged ? (double)p.num_blocks * p.Hkv * p.block_size : (double)p.R * p.Hkv * p.Smax;
        const double out = (double)p.B * p.Hkv * p.out_slots, in = vectors * row;
        if (!apart(p.k_out, out * row, p.v_out, out * row) || (p.weights_out && !apart(p.weights, vectors * 4, p.weights_out, out * 4)))
            return GQA_ERR_INVALID_ARGUMENT;
        for (const void *o : {p.k_out, p.v_out})
            if (!apart(p.k_cache, in, o, out * row) || !apart(p.v_cache, in, o, out * row))
                return GQA_ERR_INVALID_ARGUMENT;
    }
    p.row_bytes = (int)row;
    const int sms = current_sms();
    if (!sms)
        return GQA_ERR_CUDA;
    return evict_launch(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

}  // namespace

extern "C" {

gqa_status gqa_rotate(const void *q, const void *k, void *q_out, void *k_out, gqa_dtype dt, const int64_t *strides,
                      const int32_t *positions, const int32_t *lengths, const int32_t *cu_q, const uint64_t *freqs,
                      float factor, int interleaved, int B, int T, int Hq, int Hkv, int D, int dim, int32_t *d_status,
                      void *stream)
{
    if ((dt != GQA_DTYPE_F32 && dt != GQA_DTYPE_BF16) || T < 0 || Hq < 0 || Hkv < 0 || (long long)Hq + Hkv < 1 ||
        D < 1 || dim < 2 || dim % 2 || dim > D)
        return GQA_ERR_INVALID_ARGUMENT;
    if (T == 0)
        return GQA_OK;
    if (!positions && (B < 0 || !cu_q || (B && !lengths)))
        return GQA_ERR_INVALID_ARGUMENT;
    if (D > 1024 || ((long long)Hq + Hkv) * D > (1 << 24))
        return GQA_ERR_UNSUPPORTED;
    if (!freqs || !strides || (Hq && (!q || !q_out)) || (Hkv && (!k || !k_out)))
        return GQA_ERR_INVALID_ARGUMENT;
    const unsigned es = dt == GQA_DTYPE_F32 ? 4 : 2;
    if (!aligned(q, es) || !aligned(k, es) || !aligned(q_out, es) || !aligned(k_out, es) || !aligned(freqs, 8))
        return GQA_ERR_INVALID_ARGUMENT;
    const int sms = current_sms();
    if (!sms)
        return GQA_ERR_CUDA;
    RotateParams p = {};
    p.q = q;
    p.k = k;
    p.q_out = q_out;
    p.k_out = k_out;
    if (Hq) {
        p.q_token = strides[0];
        p.q_head = strides[1];
        p.qo_token = strides[4];
        p.qo_head = strides[5];
    }
    if (Hkv) {
        p.k_token = strides[2];
        p.k_head = strides[3];
        p.ko_token = strides[6];
        p.ko_head = strides[7];
    }
    p.positions = positions;
    p.lengths = positions ? nullptr : lengths;
    p.cu_q = positions ? nullptr : cu_q;
    p.freqs = freqs;
    p.status = d_status;
    p.factor = factor;
    p.bf16 = dt == GQA_DTYPE_BF16;
    p.half = !interleaved;
    p.B = B;
    p.T = T;
    p.Hq = Hq;
    p.Hkv = Hkv;
    p.D = D;
    p.dim = dim;
    return rotate_launch(p, sms, static_cast<cudaStream_t>(stream)) == cudaSuccess ? GQA_OK : GQA_ERR_CUDA;
}

gqa_status gqa_evict(void *k_cache, void *v_cache, float *weights, const int32_t *lengths, const int32_t *slot_ids,
                     int32_t *ids, int32_t *new_lengths, void *k_out, void *v_out, float *weights_out, int out_slots,
                     int B, int Hkv, int D, int R, int Smax, gqa_dtype kv_dtype, int n_keep, int n_first, int n_last,
                     int32_t *d_status, void *stream)
{
    EvictParams p = {};
    p.k_cache = k_cache;
    p.v_cache = v_cache;
    p.weights = weights;
    p.lengths = lengths;
    p.slot_ids = slot_ids;
    p.ids = ids;
    p.new_lengths = new_lengths;
    p.k_out = k_out;
    p.v_out = v_out;
    p.weights_out = weights_out;
    p.out_slots = out_slots;
    p.status = d_status;
    p.B = B;
    p.Hkv = Hkv;
    p.R = R;
    p.Smax = Smax;
    p.n_keep = n_keep;
    p.n_first = n_first;
    p.n_last = n_last;
    return run_evict(p, D, kv_dtype, stream);
}

gqa_status gqa_evict_paged(void *k_blocks, void *v_blocks, float *weights, const int32_t *block_table,
                           const int32_t *lengths, int32_t *ids, int32_t *new_lengths, void *k_out, void *v_out,
                           float *weights_out, int out_slots, int B, int Hkv, int D, int num_blocks, int block_size,
                           int max_blocks, gqa_dtype kv_dtype, int n_keep, int n_first, int n_last, int32_t *d_status,
                           void *stream)
{
    EvictParams p = {};
    p.k_cache = k_blocks;
    p.v_cache = v_blocks;
    p.weights = weights;
    p.block_table = block_table;
    p.lengths = lengths;
    p.ids = ids;
    p.new_lengths = new_lengths;
    p.k_out = k_out;
    p.v_out = v_out;
    p.weights_out = weights_out;
    p.out_slots = out_slots;
    p.status = d_status;
    p.B = B;
    p.Hkv = Hkv;
    p.paged = 1;
    p.num_blocks = num_blocks;
    p.block_size = block_size;
    p.max_blocks = max_blocks;
    p.n_keep = n_keep;
    p.n_first = n_first;
    p.n_last = n_last;
    return run_evict(p, D, kv_dtype, stream);
}

}  // extern "C"
