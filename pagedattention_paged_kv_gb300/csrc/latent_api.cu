// latent_api.cu -- the extern "C" entry points of the latent-attention operators and of the
// step metadata (declared in include/pagedkv.h): argument checks, tensor maps, launches.
#include <cmath>
#include <cstdint>

#include "../../include/pagedkv.h"
#include "api_common.h"
#include "latent_absorbed.cuh"
#include "latent_expanded.cuh"
#include "step_metadata.cuh"

namespace pkv {
cudaError_t launch_latent_cache_write(void *cache, const void *latent, const void *rope,
                                      const int64_t *slot_mapping, int64_t num_tokens, int64_t num_slots,
                                      int latent_bytes, int rope_bytes, int num_sms, int *err,
                                      cudaStream_t stream);
}

using pkv::aligned_to;

namespace {

// log2 of a supported block size, or -1.
int block_shift(int block_size) {
    return block_size == 8 ? 3 : block_size == 16 ? 4 : block_size == 32 ? 5 : block_size == 64 ? 6 : -1;
}

// scale x log2(e), which the kernels take, or 0 for a scale that is not supported.
float log2_scale(float scale) {
    const float s = scale * 1.4426950408889634f;
    return scale > 0.f && s < INFINITY ? s : 0.f;
}

int check_latent(int num_seqs, int total_q, int max_blocks_per_seq, int num_heads, int latent_dim, int rope_dim,
                 int block_size, int64_t num_blocks, int dtype) {
    if (num_seqs < 0 || total_q < 0 || max_blocks_per_seq < 0 || num_heads <= 0 || latent_dim <= 0 ||
        rope_dim <= 0 || block_size <= 0 || num_blocks < 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_BF16) return PKV_ERR_UNSUPPORTED;
    if ((latent_dim != 256 && latent_dim != 512) || rope_dim != pkv::kRopeDim || block_shift(block_size) < 0)
        return PKV_ERR_UNSUPPORTED;
    if ((int64_t)total_q * num_heads > (int64_t)INT32_MAX - 128 || num_blocks > INT32_MAX ||
        (int64_t)max_blocks_per_seq * block_size > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    return PKV_OK;
}

// Whether the expanded rows of a batch can be addressed.
bool expanded_fits(int num_seqs, int64_t total_context, int num_heads) {
    return total_context <= INT32_MAX &&
           total_context + (int64_t)num_seqs * (pkv::kExpTile - 1) <= ((int64_t)INT32_MAX / 4 - 128) / num_heads;
}

// The cache as (64 columns, token in group, 64-column chunk, group of 8 tokens, block): a box of
// one block (at most 32 tokens of it) x box_chunks chunks lands as [group][chunk][8 tokens][64 columns].
int encode_latent_map(CUtensorMap *map, const void *cache, int64_t num_blocks, int block_size, int row_cols,
                      int box_chunks) {
    const uint64_t row = (uint64_t)row_cols * 2;
    const uint64_t dims[5] = {64, 8, (uint64_t)(row_cols / 64), (uint64_t)(block_size / 8), (uint64_t)num_blocks};
    const uint64_t strides[4] = {row, 128, row * 8, row * block_size};
    const uint32_t box[5] = {64, 8, (uint32_t)box_chunks, (uint32_t)(block_size < 32 ? block_size / 8 : 4), 1};
    return pkv::encode_tiled(map, 5, cache, dims, strides, box);
}

}  // namespace

extern "C" int pkv_step_metadata(int32_t *block_tables, int32_t *context_lens, int32_t *query_start_loc,
                                 int64_t *slot_mapping, int32_t *free_end, const int32_t *cached_lens,
                                 const int32_t *new_lens, const int32_t *free_blocks, const int32_t *free_begin,
                                 int num_seqs, int max_blocks_per_seq, int64_t num_slots, int64_t num_free,
                                 int64_t num_blocks, int block_size, void *stream) {
    if (num_seqs < 0 || max_blocks_per_seq < 0 || num_slots < 0 || num_free < 0 || num_blocks < 0 ||
        block_size <= 0)
        return PKV_ERR_INVALID_ARG;
    const int shift = block_shift(block_size);
    if (shift < 0 || num_seqs > pkv::kStepMaxSeqs || num_slots > INT32_MAX || num_free > INT32_MAX ||
        num_blocks > INT32_MAX || (int64_t)max_blocks_per_seq * block_size > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (!query_start_loc || !free_end || !free_begin || (num_seqs > 0 && (!context_lens || !cached_lens || !new_lens)) ||
        (num_seqs > 0 && max_blocks_per_seq > 0 && !block_tables) || (num_slots > 0 && !slot_mapping) ||
        (num_free > 0 && !free_blocks))
        return PKV_ERR_INVALID_ARG;
    if (!aligned_to(slot_mapping, 8)) return PKV_ERR_INVALID_ARG;
    pkv::DeviceFacts d;
    const int st = pkv::current_device(&d);
    if (st != PKV_OK) return st;
    pkv::StepArgs a;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.query_start_loc = query_start_loc;
    a.slot_mapping = slot_mapping;
    a.free_end = free_end;
    a.cached_lens = cached_lens;
    a.new_lens = new_lens;
    a.free_blocks = free_blocks;
    a.free_begin = free_begin;
    a.num_seqs = num_seqs;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.block_shift = shift;
    a.num_slots = num_slots;
    a.num_free = num_free;
    a.num_blocks = num_blocks;
    a.err = d.err;
    return pkv::launch_step_metadata(a, static_cast<cudaStream_t>(stream)) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}

extern "C" int pkv_latent_cache_write(void *latent_cache, const void *latent, const void *rope,
                                      const int64_t *slot_mapping, int64_t num_tokens, int64_t num_blocks,
                                      int block_size, int latent_dim, int rope_dim, int dtype, void *stream) {
    if (num_tokens < 0 || num_blocks < 0 || block_size <= 0 || latent_dim <= 0 || rope_dim <= 0)
        return PKV_ERR_INVALID_ARG;
    if (dtype != PKV_DTYPE_BF16 || latent_dim % 8 != 0 || rope_dim % 8 != 0 || latent_dim > 65536 ||
        rope_dim > 65536 || num_blocks > INT32_MAX)
        return PKV_ERR_UNSUPPORTED;
    if (num_tokens == 0) return PKV_OK;
    if (!latent_cache || !latent || !rope || !slot_mapping) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(latent_cache, 16) || !aligned_to(latent, 16) || !aligned_to(rope, 16) ||
        !aligned_to(slot_mapping, 8))
        return PKV_ERR_INVALID_ARG;
    pkv::DeviceFacts d;
    const int st = pkv::current_device(&d);
    if (st != PKV_OK) return st;
    return pkv::launch_latent_cache_write(latent_cache, latent, rope, slot_mapping, num_tokens,
                                          num_blocks * block_size, latent_dim * 2, rope_dim * 2, d.sms, d.err,
                                          static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

extern "C" size_t pkv_latent_workspace_size(int op, int num_seqs, int total_q_tokens, int64_t total_context,
                                            int num_heads, int latent_dim, int rope_dim) {
    if (check_latent(num_seqs, total_q_tokens, 0, num_heads, latent_dim, rope_dim, 16, 0, PKV_DTYPE_BF16) != PKV_OK ||
        total_context < 0)
        return 0;
    if (op == PKV_OP_LATENT_EXPANDED && !expanded_fits(num_seqs, total_context, num_heads)) return 0;
    pkv::DeviceFacts d;
    if (pkv::current_device(&d) != PKV_OK) return 0;
    if (op == PKV_OP_LATENT_ABSORBED) {
        pkv::AbsorbedPlan p;
        pkv::plan_absorbed(latent_dim, d.sms, &p);
        return p.ws_bytes;
    }
    if (op == PKV_OP_LATENT_EXPANDED) {
        pkv::ExpandedPlan p;
        pkv::plan_expanded(num_seqs, total_context, num_heads, d.sms, &p);
        return p.ws_bytes;
    }
    return 0;
}

extern "C" int pkv_latent_attention_absorbed(void *out, const void *q, const int32_t *query_start_loc,
                                             const void *latent_cache, const int32_t *block_tables,
                                             const int32_t *context_lens, int num_seqs, int total_q_tokens,
                                             int max_blocks_per_seq, int num_heads, int latent_dim, int rope_dim,
                                             int block_size, int64_t num_blocks, float scale, int causal,
                                             int dtype, void *workspace, size_t workspace_bytes, void *stream) {
    int st = check_latent(num_seqs, total_q_tokens, max_blocks_per_seq, num_heads, latent_dim, rope_dim, block_size,
                          num_blocks, dtype);
    if (st != PKV_OK) return st;
    const float scale_log2 = log2_scale(scale);
    if (scale_log2 == 0.f) return PKV_ERR_INVALID_ARG;
    if (!query_start_loc && total_q_tokens != num_seqs) return PKV_ERR_INVALID_ARG;
    if (num_seqs == 0 || total_q_tokens == 0) return PKV_OK;
    if (!out || !q || !latent_cache || !block_tables || !context_lens) return PKV_ERR_INVALID_ARG;
    if (!aligned_to(out, 16) || !aligned_to(q, 16) || !aligned_to(latent_cache, 16)) return PKV_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return PKV_ERR_INVALID_ARG;
    pkv::DeviceFacts d;
    st = pkv::current_device(&d);
    if (st != PKV_OK) return st;
    pkv::AbsorbedPlan p;
    pkv::plan_absorbed(latent_dim, d.sms, &p);
    if (!workspace || workspace_bytes < p.ws_bytes) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned_to(workspace, 256)) return PKV_ERR_INVALID_ARG;
    const int cols = latent_dim + rope_dim;
    CUtensorMap qmap, kvmap;
    const uint64_t qdims[3] = {64, (uint64_t)total_q_tokens * num_heads, (uint64_t)(cols / 64)};
    const uint64_t qstride[2] = {(uint64_t)cols * 2, 128};
    const uint32_t qbox[3] = {64, (uint32_t)pkv::kLatentRows, (uint32_t)(cols / 64)};
    st = pkv::encode_tiled(&qmap, 3, q, qdims, qstride, qbox);
    if (st == PKV_OK) st = encode_latent_map(&kvmap, latent_cache, num_blocks, block_size, cols,
                                                 cols / 64);
    if (st != PKV_OK) return st;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pkv::AbsorbedArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.query_start_loc = query_start_loc;
    a.block_tables = block_tables;
    a.context_lens = context_lens;
    a.num_seqs = num_seqs;
    a.total_q = total_q_tokens;
    a.max_blocks_per_seq = max_blocks_per_seq;
    a.block_shift = block_shift(block_size);
    a.num_heads = num_heads;
    a.grid = p.grid;
    a.causal = causal != 0;
    a.num_blocks = num_blocks;
    a.scale_log2 = scale_log2;
    a.ws_jobs = reinterpret_cast<pkv::LatentJob *>(ws + p.off_jobs);
    a.ws_ml = reinterpret_cast<float2 *>(ws + p.off_ml);
    a.ws_o = reinterpret_cast<float *>(ws + p.off_o);
    a.err = d.err;
    a.wait_ns = pkv::wait_limit_ns();
    return pkv::launch_latent_absorbed(latent_dim, qmap, kvmap, a, static_cast<cudaStream_t>(stream)) == cudaSuccess
               ? PKV_OK
               : PKV_ERR_CUDA;
}

extern "C" int pkv_latent_attention_expanded(void *out, const void *q, const int32_t *query_start_loc,
                                             const void *latent_cache, const int32_t *block_tables,
                                             const int32_t *context_lens, const void *w_k, const void *w_v,
                                             int num_seqs, int total_q_tokens, int64_t total_context,
                                             int max_blocks_per_seq, int num_heads, int latent_dim, int rope_dim,
                                             int nope_dim, int v_dim, int block_size, int64_t num_blocks,
                                             float scale, int causal, int dtype, void *workspace,
                                             size_t workspace_bytes, void *stream) {
    int st = check_latent(num_seqs, total_q_tokens, max_blocks_per_seq, num_heads, latent_dim, rope_dim, block_size,
                          num_blocks, dtype);
    if (st != PKV_OK) return st;
    const float scale_log2 = log2_scale(scale);
    if (total_context < 0 || nope_dim <= 0 || v_dim <= 0 || scale_log2 == 0.f) return PKV_ERR_INVALID_ARG;
    if (nope_dim != pkv::kExpHeadDim || v_dim != pkv::kExpHeadDim ||
        !expanded_fits(num_seqs, total_context, num_heads))
        return PKV_ERR_UNSUPPORTED;
    if (num_seqs == 0 || total_q_tokens == 0) return PKV_OK;
    if (!out || !q || !query_start_loc || !latent_cache || !block_tables || !context_lens || !w_k || !w_v)
        return PKV_ERR_INVALID_ARG;
    if (!aligned_to(out, 32) || !aligned_to(q, 16) || !aligned_to(latent_cache, 16) || !aligned_to(w_k, 16) ||
        !aligned_to(w_v, 16))
        return PKV_ERR_INVALID_ARG;
    if (num_blocks == 0 || max_blocks_per_seq == 0) return PKV_ERR_INVALID_ARG;
    pkv::DeviceFacts d;
    st = pkv::current_device(&d);
    if (st != PKV_OK) return st;
    pkv::ExpandedPlan p;
    pkv::plan_expanded(num_seqs, total_context, num_heads, d.sms, &p);
    if (!workspace || workspace_bytes < p.ws_bytes) return PKV_ERR_WORKSPACE_TOO_SMALL;
    if (!aligned_to(workspace, 256)) return PKV_ERR_INVALID_ARG;
    uint8_t *ws = static_cast<uint8_t *>(workspace);
    pkv::ExpandedBuffers buf;
    buf.rope = reinterpret_cast<__nv_bfloat16 *>(ws + p.off_rope);
    buf.kv = reinterpret_cast<uint16_t *>(ws + p.off_kv);
    buf.value_exp = reinterpret_cast<int8_t *>(ws + p.off_exp);
    buf.padded = p.padded;

    CUtensorMap latmap, wkmap, wvmap, qmap, kvmap, ropemap;
    st = encode_latent_map(&latmap, latent_cache, num_blocks, block_size, latent_dim + rope_dim, latent_dim / 64);
    // The weights' rows in the order in which the epilogues have the columns (tmem_ld_16x64 gives
    // thread j of four columns 8 i + 2 j + e, which it stores as its 16 j + 2 i + e): the keys' so that
    // they are stored in their own order, the values' so that the attention's output is.
    const uint64_t wrow = (uint64_t)latent_dim * 2, pieces = (uint64_t)num_heads * (pkv::kExpHeadDim / 64);
    const uint64_t kdims[5] = {(uint64_t)latent_dim, 2, 4, 8, pieces};
    const uint64_t kstride[4] = {wrow, 16 * wrow, 2 * wrow, 64 * wrow};
    const uint32_t kbox[5] = {64, 2, 4, 8, pkv::kExpHeadDim / 64};
    const uint64_t vdims[5] = {(uint64_t)latent_dim, 2, 16, 2, pieces};
    const uint64_t vstride[4] = {wrow, 4 * wrow, 2 * wrow, 64 * wrow};
    const uint32_t vbox[5] = {64, 2, 16, 2, pkv::kExpHeadDim / 64};
    if (st == PKV_OK) st = pkv::encode_tiled(&wkmap, 5, w_k, kdims, kstride, kbox);
    if (st == PKV_OK) st = pkv::encode_tiled(&wvmap, 5, w_v, vdims, vstride, vbox);
    const uint32_t rows128[2] = {64, 128};
    const uint64_t qcols = (uint64_t)nope_dim + rope_dim;
    const uint64_t qdims[4] = {64, qcols / 64, (uint64_t)num_heads, (uint64_t)total_q_tokens};
    const uint64_t qstride[3] = {128, qcols * 2, qcols * 2 * num_heads};
    const uint32_t qbox[4] = {64, 1, 1, 128};
    if (st == PKV_OK) st = pkv::encode_tiled(&qmap, 4, q, qdims, qstride, qbox);
    // a call whose sequences have no context at all has nothing to expand, but maps must be valid
    const int64_t padded = p.padded > 0 ? p.padded : pkv::kExpTile;
    const uint64_t kvdims[2] = {64, (uint64_t)padded * num_heads * 4};
    const uint64_t kvstride[1] = {128};
    if (st == PKV_OK) st = pkv::encode_tiled(&kvmap, 2, buf.kv, kvdims, kvstride, rows128);
    const uint64_t rdims[2] = {pkv::kExpRope, (uint64_t)padded};
    const uint64_t rstride[1] = {pkv::kExpRope * 2};
    if (st == PKV_OK) st = pkv::encode_tiled(&ropemap, 2, buf.rope, rdims, rstride, rows128);
    if (st != PKV_OK) return st;

    pkv::ExpandArgs e;
    e.query_start_loc = query_start_loc;
    e.block_tables = block_tables;
    e.context_lens = context_lens;
    e.cache = static_cast<const __nv_bfloat16 *>(latent_cache);
    e.num_seqs = num_seqs;
    e.total_q = total_q_tokens;
    e.max_blocks_per_seq = max_blocks_per_seq;
    e.block_shift = block_shift(block_size);
    e.num_heads = num_heads;
    e.grid = p.grid / 2 * 2;
    e.num_blocks = num_blocks;
    e.buf = buf;
    e.err = d.err;
    e.wait_ns = pkv::wait_limit_ns();
    cudaStream_t s = static_cast<cudaStream_t>(stream);
    if (pkv::launch_latent_expand(latent_dim, latmap, wkmap, wvmap, e, s) != cudaSuccess) return PKV_ERR_CUDA;

    pkv::ExpandedArgs a;
    a.out = static_cast<__nv_bfloat16 *>(out);
    a.query_start_loc = query_start_loc;
    a.context_lens = context_lens;
    a.num_seqs = num_seqs;
    a.total_q = total_q_tokens;
    a.num_heads = num_heads;
    a.grid = p.grid;
    a.max_context = (int64_t)max_blocks_per_seq * block_size;
    a.causal = causal != 0;
    a.scale_log2 = scale_log2;
    a.buf = buf;
    a.ws_jobs = reinterpret_cast<pkv::LatentJob *>(ws + p.off_jobs);
    a.ws_ml = reinterpret_cast<float2 *>(ws + p.off_ml);
    a.ws_o = reinterpret_cast<float *>(ws + p.off_o);
    a.err = d.err;
    a.wait_ns = e.wait_ns;
    return pkv::launch_latent_expanded(qmap, kvmap, ropemap, a, s) == cudaSuccess ? PKV_OK : PKV_ERR_CUDA;
}
