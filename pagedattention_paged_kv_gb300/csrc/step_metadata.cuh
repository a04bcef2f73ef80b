// step_metadata.cuh -- arguments and launch of the step-metadata kernel (step_metadata.cu).
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kStepMaxSeqs = 16384;  // 14 bytes a sequence in shared memory

struct StepArgs {
    int32_t *block_tables;     // [num_seqs][max_blocks_per_seq], new entries written
    int32_t *context_lens;     // [num_seqs]; may be cached_lens
    int32_t *query_start_loc;  // [num_seqs + 1]
    int64_t *slot_mapping;     // [num_slots]
    int32_t *free_end;         // [1]; may be free_begin
    const int32_t *cached_lens, *new_lens;
    const int32_t *free_blocks;  // [num_free]
    const int32_t *free_begin;   // [1]
    int num_seqs;
    int max_blocks_per_seq;
    int block_shift;
    int64_t num_slots, num_free, num_blocks;
    int *err;
};

cudaError_t launch_step_metadata(const StepArgs &a, cudaStream_t stream);

}  // namespace pkv
