// pages.cuh -- arguments and launches of the page kernels: fork, free and compact (pages.cu), copy
// (copy_pages.cu).
#pragma once

#include "pkv_common.cuh"

namespace pkv {

constexpr int kPageMaxSeqs = 16384;       // rows of a block table, forks or listed rows of a call
constexpr int64_t kPageMaxBlocks = 1 << 22;  // pages of a pool: free and compact keep two words for 32 of them in shared memory

// What the three kernels share: rows of block tables, their lengths, the counts of holders.  An
// array and the one that replaces it (cached_lens / context_lens, ref_counts / new_ref_counts,
// free_begin / free_end, block_tables / new_tables) may be the same.
struct PageArgs {
    const int32_t *cached_lens;   // [num_seqs]
    const int32_t *ref_counts;    // [num_blocks]
    int32_t *new_ref_counts;      // [num_blocks]
    int num_seqs, max_blocks_per_seq, block_shift;
    int64_t num_free, num_blocks;
    int *err;
};

struct ForkArgs : PageArgs {
    int32_t *block_tables;        // [num_seqs][max_blocks_per_seq], rows of the forks written
    int32_t *context_lens;        // [num_seqs]
    int32_t *block_pairs;         // [num_forks][2]
    int32_t *free_end;            // [1]
    const int32_t *free_blocks;   // [num_free]
    const int32_t *free_begin;    // [1]
    const int32_t *src, *dst;     // [num_forks]
    int num_forks;
};

struct FreeArgs : PageArgs {
    int32_t *context_lens;        // [num_seqs]
    int32_t *free_blocks;         // [num_free], entries before free_begin written
    int32_t *free_end;            // [1]
    const int32_t *block_tables;  // [num_seqs][max_blocks_per_seq]
    const int32_t *free_begin;    // [1]
    const int32_t *rows;          // [num_rows]
    int num_rows;
};

struct CompactArgs : PageArgs {
    int32_t *new_tables;          // [num_seqs][max_blocks_per_seq]
    int32_t *block_pairs;         // [max_pairs][2]
    int32_t *num_pairs;           // [1]
    int32_t *free_blocks;         // [num_free]
    int32_t *free_end;            // [1]
    const int32_t *block_tables;
    int64_t max_pairs;
};

cudaError_t launch_fork_pages(const ForkArgs &a, cudaStream_t stream);
cudaError_t launch_free_pages(const FreeArgs &a, cudaStream_t stream);
cudaError_t launch_compact_pages(const CompactArgs &a, cudaStream_t stream);

// Copies pages src -> dst (pairs) of `layers` layers; v may be null (one cache).  page_bytes is a
// multiple of 16, num_pairs (device) may be null.
cudaError_t launch_copy_pages(void *k, void *v, const int32_t *pairs, const int32_t *num_pairs, int64_t max_pairs,
                              int64_t num_layers, int64_t num_blocks, int64_t page_bytes, int num_sms, int *err,
                              cudaStream_t stream);

}  // namespace pkv
