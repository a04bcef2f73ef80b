// latent_expanded.cuh -- arguments and launches of the expanded latent attention: the
// expansion of cached latents into per-head keys and values (latent_expand.cu) and the
// attention over them (latent_expanded.cu).
#pragma once

#include "latent_merge.cuh"
#include "pkv_common.cuh"

namespace pkv {

constexpr int kExpHeadDim = 128;  // non-rotary key columns, and value columns, of a head
constexpr int kExpRope = 64;
constexpr int kExpTile = 128;     // cached tokens of an expansion tile, keys of an attention chunk
constexpr int kExpQTile = 256;    // query tokens of an attention tile (two MMA halves)

// The expanded keys and values of a call, for head h and padded token i (each sequence with query
// rows starts on the next multiple of 128): piece p (64 key columns, the next 64, 64 value columns,
// the next 64) is row (4 h + p) * padded + i of kv, so the 128 rows of a box are contiguous; rope
// row i is the token's rotary key part.  Rows past a context are zero.  Value column 16 j + 2 i + e of
// 64 (e < 2, i < 8) is stored as column 8 i + 2 j + e.  The values of each 32 padded tokens of a head
// have an exponent x in common: what is stored is 2^-x v.
struct ExpandedBuffers {
    __nv_bfloat16 *rope;  // [padded][64]
    uint16_t *kv;         // [num_heads][4][padded][64]: bf16 keys, fp16 values
    int8_t *value_exp;    // [num_heads][padded / 32]
    int64_t padded;       // tokens, a multiple of 128
};
constexpr int kValueExpMin = -64;  // value_exp is between this and 0

struct ExpandArgs {
    const int32_t *query_start_loc;
    const int32_t *block_tables;
    const int32_t *context_lens;
    const __nv_bfloat16 *cache;
    int num_seqs, total_q, max_blocks_per_seq, block_shift, num_heads;
    int grid;  // even: clusters of two CTAs
    int64_t num_blocks;
    ExpandedBuffers buf;
    int *err;
    uint64_t wait_ns;
};

struct ExpandedArgs {
    __nv_bfloat16 *out;  // [total_q][num_heads][128]
    const int32_t *query_start_loc;
    const int32_t *context_lens;
    int num_seqs, total_q, num_heads, grid;
    int64_t max_context;
    bool causal;
    float scale_log2;
    ExpandedBuffers buf;
    LatentJob *ws_jobs;  // [grid]
    float2 *ws_ml;       // [2 * grid][256]
    float *ws_o;         // [2 * grid][256][128]
    int *err;
    uint64_t wait_ns;
};

struct ExpandedPlan {
    int grid;
    int64_t padded;
    size_t off_rope, off_kv, off_exp, off_jobs, off_ml, off_o, ws_bytes;
};

void plan_expanded(int num_seqs, int64_t total_context, int num_heads, int sms, ExpandedPlan *p);

// kv_map: the latent cache in boxes of min(block, 32 tokens) x the latent chunks; wk_map, wv_map: 64
// columns of a head's 128 weight rows, in the order that the epilogues want.
cudaError_t launch_latent_expand(int latent_dim, const CUtensorMap &kv_map, const CUtensorMap &wk_map,
                                 const CUtensorMap &wv_map, const ExpandArgs &a, cudaStream_t stream);

// q_map: q as (64 columns, chunk, head, token) in boxes of 128 tokens x 64 columns; kv_map, rope_map:
// the expanded rows in boxes of 128 rows x 64 columns.
cudaError_t launch_latent_expanded(const CUtensorMap &q_map, const CUtensorMap &kv_map, const CUtensorMap &rope_map,
                                   const ExpandedArgs &a, cudaStream_t stream);

}  // namespace pkv
