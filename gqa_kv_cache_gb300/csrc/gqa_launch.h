// Host-side entry points of the kernels, used by the C ABI layer.
#pragma once

#include <cuda.h>
#include <cuda_runtime.h>

#include "gqa_common.cuh"

namespace gqa {

// CUDA-core decode kernel (gqa_simt.cu).
bool simt_supports(int D, int G);
int simt_tile();
int simt_ctas_per_sm(bool bf16, int D, int G);  // occupancy of that instantiation
cudaError_t simt_launch(const DecodeParams &p, bool bf16, cudaStream_t st);

// TMA-ring + tensor-core decode kernel (gqa_tc.cu).
struct TcMaps {
    CUtensorMap k, v;      // tiled maps over the key / value cache, 128-byte swizzle
    CUtensorMap k16, v16;  // dense caches: the same with a box of kDenseBoxRows slots
};
// A dense cache's tile is one 64-slot box when every part of it is read; a
// tile that is only partly read (a unit's last tile, a window's first) is
// copied in boxes of kDenseBoxRows slots, those that hold a slot the step
// reads. A paged cache's box is its block (at most the tile).
constexpr int kDenseBoxRows = 16;
bool tc_supports(bool bf16, int D, int G, bool paged, int block_size);  // bf16: the cache
int tc_tile();
int tc_ctas_per_sm(bool kv8, int unit_rows);   // resident CTAs per SM of the instantiation
cudaError_t tc_launch(const DecodeParams &p, const TcMaps &maps, cudaStream_t st);
// The tcgen05 form of multi-token units of 17 to 32 query rows over a bf16
// cache (gqa_tc_multi.cu): whether it takes the step, and its launch.
bool tc5_takes(const DecodeParams &p);
cudaError_t tc5_launch_multi(const DecodeParams &p, const TcMaps &maps, cudaStream_t st);

// Small-cache kernel: one cluster of CTAs per unit, the unit staged in their
// shared memory (gqa_unit.cu). cap_rows: the row capacity in slots.
bool unit_supports(bool bf16, int D, int G, long long cap_rows);
size_t unit_smem_bytes(bool bf16, int D, int G, long long rows, int cl);
int unit_ctas_per_sm(bool bf16, int D, int G, long long cap_rows);
int unit_cluster(long long cap_rows, long long units, int sms);   // CTAs a unit
cudaError_t unit_launch(const DecodeParams &p, bool bf16, long long cap_rows, int sms, cudaStream_t st);

// Decode step and attend over an E2M1 cache (gqa_q4.cu): D = 64 or 128.
bool q4_supports(int D, int G);
int q4_tile();
bool q4_whole_units(long long capacity, long long units, int grid);   // one CTA a unit
int q4_ctas_per_sm(int D, bool q_bf16);   // resident CTAs per SM
cudaError_t q4_launch(const DecodeParams &p, cudaStream_t st);

// Packed tokens into a cache and slots back out (gqa_rows.cu).
struct RowsParams {
    const void *k_new, *v_new;       // append: (T, Hkv, D)
    void *k_out, *v_out;             // read: (T, Hkv, D)
    void *k_cache, *v_cache;         // dense (R, Hkv, Smax, row) or blocks (num_blocks, Hkv, block_size, row)
    void *k_group, *v_group;         // E2M1 caches: E4M3 scales, one per 16 dims
    const float *k_scale, *v_scale;  // E4M3 and E2M1 caches: (Hkv)
    void *bounds;                    // append: key bounds (block, head, 2, D) bfloat16, or null
    const int32_t *lengths, *cu_q, *slot_ids, *block_table;
    int32_t *status;
    int vec_bf16;                    // the vectors' type: 1 bfloat16, 0 float32
    int B, T, Hkv, D, R, Smax, paged, num_blocks, block_size, max_blocks;
    int bounds_block;                // slots a block of the bounds (paged: block_size)
    int chunk;                       // tokens a CTA (set by rows_launch)
    int wide;                        // vectors and caches lie on 32-byte boundaries (likewise)
};
__device__ __forceinline__ void rows_report(const RowsParams &p, int bits)
{
    if (p.status)
        atomicOr(p.status, bits);
}
cudaError_t rows_launch(RowsParams p, int kv_dtype, bool write, int sms, cudaStream_t st);

// Block selection from key bounds (gqa_select.cu).
struct SelectParams {
    const void *q;                   // (B, Hq, D)
    const void *bounds;              // dense (R, Hkv, NB, 2, D) or (num_blocks, Hkv, 2, D), bfloat16
    const int32_t *lengths, *slot_ids, *block_table;
    int32_t *ids;                    // (B, Hkv, n_select)
    int32_t *table;                  // (B * Hkv, n_select): blocks of the flattened pool
    int32_t *sel_lengths;            // (B * Hkv)
    int32_t *status;
    int q_bf16, B, Hq, Hkv, D, R, NB, paged, num_blocks, block_size;
    int n_select, n_first, n_last;
};
bool select_supports(int D, int NB);
cudaError_t select_launch(const SelectParams &p, int sms, cudaStream_t st);

// Content validation (gqa_validate.cu). *d_result must be zero on entry; the
// kernel sets it to 1 on any violation. attend = 1 checks the read-only
// attend's reading of lengths (the number of valid slots).
cudaError_t validate_launch(const int32_t *lengths, const int32_t *slot_ids,
                            const int32_t *block_table, int B, int R, int Smax,
                            int num_blocks, int block_size, int max_blocks, int attend,
                            const int32_t *cu_q, int T, int32_t *d_result, cudaStream_t st);

}  // namespace gqa
