// latent_absorbed.cuh -- arguments and launch of the absorbed latent attention
// (latent_absorbed.cu).
#pragma once

#include "latent_merge.cuh"
#include "pkv_common.cuh"

namespace pkv {

constexpr int kRopeDim = 64;      // rotary columns of a cached latent row
constexpr int kLatentRows = 64;   // query rows (token x head pairs) of a work item
constexpr int kLatentTile = 64;   // cached tokens of a tile

// Warp 0 loads, warp 1 issues QK, warps 2..5 are the softmax warpgroup, warp 6 issues PV.
constexpr int kAbsorbedThreads = 224;

struct AbsorbedArgs {
    __nv_bfloat16 *out;
    const int32_t *query_start_loc;  // null: one row per sequence
    const int32_t *block_tables;
    const int32_t *context_lens;
    int num_seqs;
    int total_q;
    int max_blocks_per_seq;
    int block_shift;                 // log2 of the block size (8 .. 64 tokens)
    int num_heads;
    int grid;
    bool causal;
    int64_t num_blocks;
    float scale_log2;
    LatentJob *ws_jobs;              // [grid]
    float2 *ws_ml;                   // [2 * grid][64]: a part's reference maxima and sums
    float *ws_o;                     // [2 * grid][64][latent_dim]: its unnormalised output
    int *err;
    uint64_t wait_ns;
};

struct AbsorbedPlan {
    int grid;
    size_t off_jobs, off_ml, off_o, ws_bytes;
};

void plan_absorbed(int latent_dim, int sms, AbsorbedPlan *p);

// q_map: q as (64 columns, row [total_q * num_heads], chunk) in boxes of 64 rows x all chunks;
// kv_map: the cache as (64 columns, token in group, chunk, group of 8 tokens, block) in boxes of
// min(block, 32 tokens) x all chunks.

cudaError_t launch_latent_absorbed(int latent_dim, const CUtensorMap &q_map, const CUtensorMap &kv_map,
                                   const AbsorbedArgs &a, cudaStream_t stream);

}  // namespace pkv
