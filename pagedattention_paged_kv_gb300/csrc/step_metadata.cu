// step_metadata.cu -- a step's context lengths, query offsets, block tables and slot map from
// the lengths of its requests, on the GPU (sm_103a).
//
//   context_lens[s]    = cached_lens[s] + new_lens[s]
//   query_start_loc    = exclusive prefix sum of new_lens
//   a sequence gains ceil(context / bs) - ceil(cached / bs) blocks, the next ones of the free
//   list in sequence order; new token t of sequence s at position p lands in slot
//   table[s][p / bs] * bs + p % bs
//
// Bound: latency.  128 sequences move under 4 KB and 1024 sequences with 64 chunks of 512
// tokens 0.3 MB, so one launch has to do it all and its chain of dependent loads is the time.
// Every CTA of one cluster reads all lengths and keeps the prefix sums in shared memory (no
// exchange through global memory); tokens, new blocks and sequences are then dealt out evenly
// and each finds its sequence by a binary search.  The cluster barrier between the last read
// and the first write lets outputs be the inputs' own buffers.
#include <cooperative_groups.h>

#include "attn_block.cuh"
#include "step_metadata.cuh"

namespace pkv {

namespace {

constexpr int kStepThreads = 1024;

struct StepSeq {
    int cached, fresh;  // tokens cached and (valid) new tokens
    int64_t need;       // blocks gained
};

__device__ __forceinline__ StepSeq step_seq(const StepArgs &a, int s, bool report) {
    StepSeq r;
    r.cached = a.cached_lens[s];
    r.fresh = a.new_lens[s];
    const int64_t room = (int64_t)a.max_blocks_per_seq << a.block_shift;
    if (r.cached < 0 || r.cached > room || r.fresh < 0 || (int64_t)r.cached + r.fresh > room) {
        if (report) flag_error(a.err, r.fresh < 0 ? PKV_DEVERR_QUERY_LEN : PKV_DEVERR_CONTEXT_LEN);
        r.fresh = 0;  // the sequence takes no part in this step
        r.need = 0;
        return r;
    }
    const int64_t m = (1 << a.block_shift) - 1;
    r.need = ((r.cached + (int64_t)r.fresh + m) >> a.block_shift) - ((r.cached + m) >> a.block_shift);
    return r;
}

// Last i in [0, n) with pre[i] <= x (pre ascending, pre[0] = 0 <= x).
__device__ __forceinline__ int last_at_most(const int32_t *pre, int n, int x) {
    int lo = 0, hi = n;
    while (hi - lo > 1) {
        const int mid = (lo + hi) >> 1;
        if (pre[mid] <= x) lo = mid; else hi = mid;
    }
    return lo;
}

// Inclusive sum over the block; *total gets the block's sum.
__device__ __forceinline__ int64_t block_scan(int64_t x, int64_t *tmp, int64_t *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t y = __shfl_up_sync(0xffffffffu, x, o);
        if (lane >= o) x += y;
    }
    if (lane == 31) tmp[warp] = x;
    __syncthreads();
    if (warp == 0) {
        int64_t w = lane < nw ? tmp[lane] : 0;
#pragma unroll
        for (int o = 1; o < 32; o <<= 1) {
            const int64_t y = __shfl_up_sync(0xffffffffu, w, o);
            if (lane >= o) w += y;
        }
        tmp[lane] = w;
    }
    __syncthreads();
    *total = tmp[31];
    const int64_t r = x + (warp > 0 ? tmp[warp - 1] : 0);
    __syncthreads();
    return r;
}

}  // namespace

__global__ void __launch_bounds__(kStepThreads, 1) step_metadata_kernel(const StepArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int64_t tmp[32];
    const int S = a.num_seqs, nt = blockDim.x, tid = threadIdx.x;
    int32_t *qsl = sm, *needed = sm + (S + 1), *cached = needed + (S + 1);
    pdl_wait();
    pdl_trigger();
    const int64_t begin = *a.free_begin;
    const int per = (S + nt - 1) / nt;
    const int first = min(S, tid * per), end = min(S, first + per);
    int64_t tokens = 0, blocks = 0;
    for (int s = first; s < end; ++s) {
        const StepSeq q = step_seq(a, s, blockIdx.x == 0);
        tokens += q.fresh;
        blocks += q.need;
    }
    int64_t total, need;
    int64_t t0 = block_scan(tokens, tmp, &total) - tokens;
    int64_t b0 = block_scan(blocks, tmp, &need) - blocks;
    // A step that does not fit is refused whole, as an allocation from the block manager is.
    const bool no_room = total > a.num_slots;
    const bool no_blocks = begin < 0 || begin > a.num_free || need > a.num_free - begin;
    const bool refused = no_room || no_blocks;
    if (refused && blockIdx.x == 0 && tid == 0)
        flag_error(a.err, (no_room ? PKV_DEVERR_QUERY_LEN : 0) | (no_blocks ? PKV_DEVERR_FREE_BLOCKS : 0));
    for (int s = first; s < end; ++s) {
        const StepSeq q = step_seq(a, s, false);
        qsl[s] = refused ? 0 : (int32_t)t0;
        needed[s] = refused ? 0 : (int32_t)b0;
        cached[s] = q.cached;
        t0 += q.fresh;
        b0 += q.need;
    }
    if (refused) total = need = 0;
    if (tid == 0) {
        qsl[S] = (int32_t)total;
        needed[S] = (int32_t)need;
    }
    // every read of the lengths and of free_begin, by any CTA, comes before any write
    if (gridDim.x > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();

    const int64_t g = (int64_t)blockIdx.x * nt + tid, gn = (int64_t)gridDim.x * nt;
    const int32_t mask = (1 << a.block_shift) - 1;
    for (int64_t s = g; s <= S; s += gn) {
        a.query_start_loc[s] = qsl[s];
        if (s < S) a.context_lens[s] = cached[s] + (qsl[s + 1] - qsl[s]);
    }
    if (g == 0) *a.free_end = (int32_t)(begin + need);
    // id of a fresh block, or -1 (flagged) if the free list names one outside the pool
    auto fresh_id = [&](int64_t i) -> int32_t {
        const int32_t id = a.free_blocks[begin + i];
        return id >= 0 && id < a.num_blocks ? id : -1;
    };
    for (int64_t i = g; i < need; i += gn) {
        const int s = last_at_most(needed, S, (int)i);
        const int32_t id = fresh_id(i);
        if (id < 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
        const int64_t held = ((int64_t)cached[s] + mask) >> a.block_shift;
        a.block_tables[(int64_t)s * a.max_blocks_per_seq + held + (i - needed[s])] = id;
    }
    for (int64_t t = g; t < a.num_slots; t += gn) {
        int64_t slot = -1;
        if (t < total) {
            const int s = last_at_most(qsl, S, (int)t);
            const int64_t p = (int64_t)cached[s] + (t - qsl[s]);
            const int64_t held = ((int64_t)cached[s] + mask) >> a.block_shift, j = p >> a.block_shift;
            int32_t id;
            if (j >= held) {
                id = fresh_id(needed[s] + (j - held));
            } else {
                id = a.block_tables[(int64_t)s * a.max_blocks_per_seq + j];
                if (id < 0 || id >= a.num_blocks) {
                    flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                    id = -1;
                }
            }
            if (id >= 0) slot = ((int64_t)id << a.block_shift) + (p & mask);
        }
        a.slot_mapping[t] = slot;
    }
}

cudaError_t launch_step_metadata(const StepArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const size_t smem = sizeof(int32_t) * (3 * (size_t)a.num_seqs + 2);
    cudaError_t e = allow_dynamic_smem(step_metadata_kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    // One CTA while a thread has at most a few items; beyond that a cluster of eight deals the
    // items out, at the price of a cluster launch and its barrier.
    const unsigned ctas = a.num_slots + a.num_seqs > 4 * kStepThreads ? 8 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(kStepThreads);
    cfg.dynamicSmemBytes = smem;
    cfg.stream = stream;
    cudaLaunchAttribute attr[2];
    attr[0].id = cudaLaunchAttributeProgrammaticStreamSerialization;
    attr[0].val.programmaticStreamSerializationAllowed = 1;
    attr[1].id = cudaLaunchAttributeClusterDimension;
    attr[1].val.clusterDim.x = ctas;
    attr[1].val.clusterDim.y = attr[1].val.clusterDim.z = 1;
    cfg.attrs = attr;
    cfg.numAttrs = ctas > 1 ? 2 : 1;
    return cudaLaunchKernelEx(&cfg, step_metadata_kernel, a);
}

}  // namespace pkv
