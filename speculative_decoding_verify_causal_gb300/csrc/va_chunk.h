// What the chunk plan (va_chunk_plan.cpp) hands to the kernels of va_chunk.cu and va_weights.cu.
#pragma once

#include "va_internal.h"

namespace va {

// One CTA of chunk attention: `nt` new tokens from token t0 of a chunk on, with the query heads of kv head `kvh`,
// over the keys [k_begin, k_end).  q0: the row of q, out and lse of token t0.  vis0: the last key that token t0 sees.
// part: the first of its tiles' partial slots, -1 when the item covers all keys and writes the output itself.
struct ChunkItem {
    int b, kvh, q0, nt, vis0, k_begin, k_end, part;
};

// One tile of packed rows (tokens q0 .. q0 + nt - 1 of kv head kvh) whose n partials, `step` slots apart, are merged.
struct ChunkGroup {
    int kvh, q0, nt, first_part, n, step, pad0, pad1;
};

// One CTA cluster of the gathered weights: a block of keys of a kv head of sequence b, whose chunk of n tokens
// starts at row q0 of q; L keys are cached with them.
struct WeightItem {
    int b, kvh, key0, q0, n, L, pad0, pad1;
};

struct ChunkParams {
    const void *k_pages, *v_pages;
    const float *k_scale, *v_scale;
    const int32_t *block_table;
    const ChunkItem *items;
    uint16_t *out;
    float *lse;
    float *o_part;    // [parts][D][kMmaRows]: rows innermost, so that a warp's rows are one segment
    float *lse_part;  // [parts][kMmaRows]
    int *flags;
    int bt_stride, Hq, Hkv, G, tpt, num_pages;  // tpt: tokens per tile of packed rows
    float sm_scale_log2;
};

struct ChunkCombineParams {
    const ChunkGroup *groups;
    const float *o_part, *lse_part;
    uint16_t *out;
    float *lse;
    int Hq, G, D;
};

struct WeightParams {
    const void *k_pages;
    const float *k_scale, *lse;
    const int32_t *block_table;
    const WeightItem *items;
    float *weights;
    int32_t *slot_pos;         // or null
    const int32_t *positions;  // of the new tokens, with slot_pos
    int64_t stride_seq, stride_head;  // of weights and slot_pos, in elements
    int *flags;
    int bt_stride, Hq, Hkv, G, tpt, num_pages, accumulate, cluster;
    float sm_scale_log2;
};

constexpr int kChunkKeys = 80;  // keys of one tile of scores
constexpr int kWeightClusters = 8;  // most CTAs that share a block of keys
constexpr int weight_keys(int D) { return D == 256 ? 128 : 256; }  // keys of a block
constexpr int kFlagTimeoutBit = 4;
constexpr int chunk_tiles(int D) { return D == 256 ? 1 : 2; }  // tiles of packed rows that a CTA takes

cudaError_t launch_chunk(const ChunkParams &p, const va_heads &q, int N, int D, int dtype, int num_items, cudaStream_t s);
cudaError_t launch_weights(const WeightParams &p, const va_heads &q, int N, int D, int dtype, int num_blocks, cudaStream_t s);
cudaError_t launch_chunk_combine(const ChunkCombineParams &p, int num_groups, int num_sms, cudaStream_t s);

}  // namespace va
