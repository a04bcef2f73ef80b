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
// tokens 0.3 MB, so one launch has to do it all and its chain of dependent steps is the time.
// Every CTA of one cluster reads all lengths and keeps the prefix sums in shared memory (no
// exchange through global memory).  The work is then dealt out by the block: a thread finds its
// block's sequence by a binary search, looks the block's id up once (writing the table entry of
// a fresh one) and writes the slots of the block's new tokens.  The cluster barrier between the
// last read and the first write lets outputs be the inputs' own buffers.
#include <cooperative_groups.h>

#include "attn_block.cuh"
#include "step_metadata.cuh"

namespace pkv {

namespace {

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

// Sums carried through a scan: new tokens, blocks gained, sequences whose first new token falls
// into a block they hold.
struct Sums {
    int64_t tokens, blocks;
    int partial;
};
__device__ __forceinline__ Sums warp_scan(Sums p) {
    const int lane = threadIdx.x & 31;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int64_t x = __shfl_up_sync(0xffffffffu, p.tokens, o), y = __shfl_up_sync(0xffffffffu, p.blocks, o);
        const int z = __shfl_up_sync(0xffffffffu, p.partial, o);
        if (lane >= o) {
            p.tokens += x;
            p.blocks += y;
            p.partial += z;
        }
    }
    return p;
}
// Sums over the threads before this one; *total over the block.  One barrier: every warp sums the
// warps' sums itself.
__device__ __forceinline__ Sums block_scan(const Sums &mine, Sums *tmp, Sums *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    Sums p = warp_scan(mine);
    if (lane == 31) tmp[warp] = p;
    __syncthreads();
    Sums w{0, 0, 0};
    if (lane < nw) w = tmp[lane];
    w = warp_scan(w);
    const int before = (warp + 31) & 31;
    total->tokens = __shfl_sync(0xffffffffu, w.tokens, 31);
    total->blocks = __shfl_sync(0xffffffffu, w.blocks, 31);
    total->partial = __shfl_sync(0xffffffffu, w.partial, 31);
    const int64_t bx = __shfl_sync(0xffffffffu, w.tokens, before), by = __shfl_sync(0xffffffffu, w.blocks, before);
    const int bz = __shfl_sync(0xffffffffu, w.partial, before);
    p.tokens += (warp > 0 ? bx : 0) - mine.tokens;
    p.blocks += (warp > 0 ? by : 0) - mine.blocks;
    p.partial += (warp > 0 ? bz : 0) - mine.partial;
    return p;
}

}  // namespace

__global__ void __launch_bounds__(1024, 1) step_metadata_kernel(const StepArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ Sums tmp[32];
    const int S = a.num_seqs, nt = blockDim.x, tid = threadIdx.x;
    // before each sequence: tokens, fresh blocks, sequences that go on in a block they hold; and
    // its cached tokens
    int32_t *qsl = sm, *fresh = sm + (S + 1), *cached = fresh + (S + 1);
    uint16_t *partial = reinterpret_cast<uint16_t *>(cached + S);
    pdl_wait();
    pdl_trigger();
    const int64_t begin = *a.free_begin;
    const int32_t mask = (1 << a.block_shift) - 1;
    const int per = (S + nt - 1) / nt;
    const int first = min(S, tid * per), end = min(S, first + per);
    Sums mine{0, 0, 0}, sum;
    for (int s = first; s < end; ++s) {
        const StepSeq q = step_seq(a, s, blockIdx.x == 0);
        mine.tokens += q.fresh;
        mine.blocks += q.need;
        mine.partial += q.fresh > 0 && (q.cached & mask) != 0;
    }
    Sums at = block_scan(mine, tmp, &sum);
    // A step that does not fit is refused whole, as an allocation from the block manager is.
    const bool no_room = sum.tokens > a.num_slots;
    const bool no_blocks = begin < 0 || begin > a.num_free || sum.blocks > a.num_free - begin;
    const bool refused = no_room || no_blocks;
    if (refused && blockIdx.x == 0 && tid == 0)
        flag_error(a.err, (no_room ? PKV_DEVERR_QUERY_LEN : 0) | (no_blocks ? PKV_DEVERR_FREE_BLOCKS : 0));
    if (refused) sum = Sums{0, 0, 0};
    for (int s = first; s < end; ++s) {
        const StepSeq q = step_seq(a, s, false);
        qsl[s] = refused ? 0 : (int32_t)at.tokens;
        fresh[s] = refused ? 0 : (int32_t)at.blocks;
        partial[s] = refused ? 0 : (uint16_t)at.partial;
        cached[s] = q.cached;
        at.tokens += q.fresh;
        at.blocks += q.need;
        at.partial += q.fresh > 0 && (q.cached & mask) != 0;
    }
    const int total = (int)sum.tokens, blocks = (int)sum.blocks + sum.partial;  // blocks that get tokens
    if (tid == 0) {
        qsl[S] = total;
        fresh[S] = (int)sum.blocks;
    }
    // every read of the lengths and of free_begin, by any CTA, comes before any write
    if (gridDim.x > 1) cooperative_groups::this_cluster().sync(); else __syncthreads();

    const int g = blockIdx.x * nt + tid, gn = gridDim.x * nt;
    for (int s = g; s <= S; s += gn) {
        a.query_start_loc[s] = qsl[s];
        if (s < S) a.context_lens[s] = cached[s] + (qsl[s + 1] - qsl[s]);
    }
    if (g == 0) *a.free_end = (int32_t)(begin + sum.blocks);
    for (int i = g; i < blocks; i += gn) {
        int s = 0, hi = S;  // the last sequence with no more than i blocks before it
        while (hi - s > 1) {
            const int mid = (s + hi) >> 1;
            if (fresh[mid] + partial[mid] <= i) s = mid; else hi = mid;
        }
        const int c = cached[s], held = (int)(((int64_t)c + mask) >> a.block_shift);
        const int j = (c >> a.block_shift) + (i - fresh[s] - partial[s]);
        int32_t *entry = a.block_tables + (int64_t)s * a.max_blocks_per_seq + j;
        int32_t id;
        if (j >= held) {
            id = a.free_blocks[begin + fresh[s] + (j - held)];
        } else {
            id = *entry;
        }
        if (id < 0 || id >= a.num_blocks) {
            flag_error(a.err, PKV_DEVERR_BLOCK_ID);
            id = -1;
        }
        if (j >= held) *entry = id;
        // the block's new tokens: positions p0 .. p1 - 1, two slots a store where they are aligned
        const int p0 = max(c, j << a.block_shift);
        const int n = (int)min64((int64_t)c + (qsl[s + 1] - qsl[s]), (int64_t)(j + 1) << a.block_shift) - p0;
        int64_t *out = a.slot_mapping + qsl[s] + (p0 - c);
        const int64_t slot0 = id < 0 ? -1 : ((int64_t)id << a.block_shift) + (p0 & mask), step = id < 0 ? 0 : 1;
        int k = 0;
        if (reinterpret_cast<uintptr_t>(out) & 8) out[k++] = slot0;
        for (; k + 1 < n; k += 2)
            *reinterpret_cast<longlong2 *>(out + k) = make_longlong2(slot0 + k * step, slot0 + (k + 1) * step);
        if (k < n) out[k] = slot0 + k * step;
    }
    for (int64_t t = total + (int64_t)g; t < a.num_slots; t += gn) a.slot_mapping[t] = -1;
}

cudaError_t launch_step_metadata(const StepArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const size_t smem = sizeof(int32_t) * (3 * (size_t)a.num_seqs + 2) + sizeof(uint16_t) * (size_t)a.num_seqs;
    cudaError_t e = allow_dynamic_smem(step_metadata_kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    // A few hundred items: one small CTA, as every further warp only adds to the time of the scan.
    // More: CTAs of 512, a cluster of eight of them beyond 1024 items (8.4 us with 1024 threads each,
    // 5.9 with 512, for 34,000 tokens).
    const int64_t items = a.num_seqs + (a.num_slots >> a.block_shift);
    const unsigned threads = a.num_seqs <= 512 && items <= 512 ? 256 : 512, ctas = items > 1024 ? 8 : 1;
    cudaLaunchConfig_t cfg = {};
    cfg.gridDim = dim3(ctas);
    cfg.blockDim = dim3(threads);
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
