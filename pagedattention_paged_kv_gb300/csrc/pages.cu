// pages.cu -- pages of a block-paged cache forked, freed and compacted on the GPU (sm_103a): block
// tables, counts of holders and the free list, so that a captured loop branches, ends and tidies
// its requests without the host.  Whole numbers only; the results do not depend on any order in
// which threads run.
//
//   fork     row d takes over row s: its full pages gain a holder, a page half full is replaced by
//            the next id of the free list (the pair tells copy_pages what to copy)
//   free     every page of the listed rows loses a holder; the pages left without one go in front
//            of the free list, in ascending order
//   compact  the highest live page moves into the lowest dead one for as long as that moves it
//            down; tables, counts and free list follow
//
// Bound: latency.  The arrays are a few MB at most, and each call is a chain of dependent steps
// (lengths, table entries, counts, sums over the whole pool): four branches of two requests take 3.9 us (in
// place as well), 1024 branches of 128 requests 9.8, one request of four freed 3.7 (in place 4.2), 900 of 1024
// freed 19.5 (19.8), 64 pages moved 7.4, a pool of 105,000 pages for 1024 requests squeezed 17.7.  One cluster of
// CTAs runs the chain in one launch: the hardware's cluster barrier stands between the steps, so no step costs a launch
// and no workspace is needed, and what the CTAs tell each other goes through their shared memory.
// The set of pages a call frees, or finds live, is a bitmap there: CTA c holds the bits of the c-th
// part of the pool, and ranks in ascending order come from counting bits.  Everything waits for
// memory, so lanes have several entries in flight, and half a warp takes a row of a table.
#include <climits>

#include <cooperative_groups.h>

#include "attn_block.cuh"
#include "pages.cuh"

namespace pkv {

namespace {

__device__ __forceinline__ void sync_all() {
    __syncwarp();
    if (gridDim.x > 1) cluster_barrier(); else __syncthreads();
}

// `p`'s place in the shared memory of CTA `rank` of the cluster.
template <typename T>
__device__ __forceinline__ T *of_cta(T *p, int rank) {
    return gridDim.x > 1 ? cooperative_groups::this_cluster().map_shared_rank(p, rank) : p;
}

// Exclusive sum of x over the threads of the CTA before this one; *total over all.  `tmp`: 32 ints,
// free again after the next barrier.
__device__ __forceinline__ int block_scan(int x, int *tmp, int *total) {
    const int lane = threadIdx.x & 31, warp = threadIdx.x >> 5, nw = blockDim.x >> 5;
    int p = x;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, p, o);
        if (lane >= o) p += y;
    }
    if (lane == 31) tmp[warp] = p;
    __syncthreads();
    int w = lane < nw ? tmp[lane] : 0;
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
        const int y = __shfl_up_sync(0xffffffffu, w, o);
        if (lane >= o) w += y;
    }
    *total = __shfl_sync(0xffffffffu, w, 31);
    const int before = __shfl_sync(0xffffffffu, w, (warp + 31) & 31);
    return p - x + (warp > 0 ? before : 0);
}

// Sum of the CTAs' totals before this one; *all over the cluster.  Between two sync_all; the whole warp.
__device__ __forceinline__ int cluster_scan(int *total, int *all) {
    const int lane = threadIdx.x & 31;
    const int t = lane < (int)gridDim.x ? *of_cta(total, lane) : 0;
    *all = __reduce_add_sync(0xffffffffu, t);
    return __reduce_add_sync(0xffffffffu, lane < (int)blockIdx.x ? t : 0);
}

__device__ __forceinline__ bool in_pool(const PageArgs &a, int32_t id) { return id >= 0 && id < a.num_blocks; }

__device__ __forceinline__ int64_t pages_of(const PageArgs &a, int32_t len) {
    return ((int64_t)len + (1 << a.block_shift) - 1) >> a.block_shift;
}

__device__ __forceinline__ bool good_len(const PageArgs &a, int32_t len) {
    return len >= 0 && (int64_t)len <= ((int64_t)a.max_blocks_per_seq << a.block_shift);
}

constexpr int kInFlight = 8;   // table entries, or counts, that a lane has in flight
constexpr int kRowLanes = 16;  // lanes that work on a row of a table (a request of 100 pages: one round)
// Behind its last holder a page's count is this much lower until the pages are gathered.
constexpr int kFreed = -(1 << 30);

}  // namespace

// ---------------------------------------------------------------------------------------------
// fork
// ---------------------------------------------------------------------------------------------

// Every CTA looks at all forks and lengths and keeps what it found in shared memory; behind the
// barrier, when all have read, the forks are dealt out to the warps of the cluster.
__global__ void __launch_bounds__(1024, 1) fork_pages_kernel(const ForkArgs a) {
    extern __shared__ int32_t sm[];
    __shared__ int tmp[32];
    const int S = a.num_seqs, n = a.num_forks, nt = blockDim.x, tid = threadIdx.x;
    int32_t *owner = sm;           // [S] the first fork into a row
    int32_t *rank = owner + S;     // [n] fresh pages before the fork, -1: no fork
    int32_t *length = rank + n;    // [n] tokens it takes over
    for (int s = tid; s < S; s += nt) owner[s] = INT_MAX;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const bool report = blockIdx.x == 0;
    const int32_t mask = (1 << a.block_shift) - 1;
    const int64_t begin = *a.free_begin;
    // a fork that can be made: between two rows, out of one with a good length, into an empty one
    for (int i = tid; i < n; i += nt) {
        const int32_t s = a.src[i], d = a.dst[i];
        int32_t len = -1;
        if (s >= 0) {  // a negative source is padding
            const bool rows = s < S && d >= 0 && d < S && d != s;
            if (rows) len = a.cached_lens[s];
            if (!rows || a.cached_lens[d] != 0) {
                if (report) flag_error(a.err, PKV_DEVERR_SEQ);
                len = -1;
            } else if (!good_len(a, len)) {
                if (report) flag_error(a.err, PKV_DEVERR_CONTEXT_LEN);
                len = -1;
            }
            if (len >= 0) atomicMin(owner + d, i);
        }
        length[i] = len;
    }
    __syncthreads();
    const int per = (n + nt - 1) / nt;
    const int first = min(n, tid * per), end = min(n, first + per);
    int need = 0, total;
    for (int i = first; i < end; ++i) {
        if (length[i] >= 0 && owner[a.dst[i]] != i) {  // a row takes one fork, the first listed
            if (report) flag_error(a.err, PKV_DEVERR_SEQ);
            length[i] = -1;
        }
        need += length[i] > 0 && (length[i] & mask) != 0;
    }
    int at = block_scan(need, tmp, &total);
    const bool refused = begin < 0 || begin > a.num_free || total > a.num_free - begin;
    if (refused && report && tid == 0) flag_error(a.err, PKV_DEVERR_FREE_BLOCKS);
    for (int i = first; i < end; ++i) {
        rank[i] = refused || length[i] < 0 ? -1 : at;
        at += length[i] > 0 && (length[i] & mask) != 0;
    }
    __syncthreads();
    const int64_t g = (int64_t)blockIdx.x * nt + tid, gn = (int64_t)gridDim.x * nt;
    if (a.new_ref_counts != a.ref_counts)
        for (int64_t b = g; b < a.num_blocks; b += gn) a.new_ref_counts[b] = a.ref_counts[b];
    if (a.context_lens != a.cached_lens)
        for (int64_t s = g; s < S; s += gn)
            if (owner[s] == INT_MAX || rank[owner[s]] < 0) a.context_lens[s] = a.cached_lens[s];
    sync_all();  // lengths and free_begin are read, the counts are in place

    if (g == 0) *a.free_end = (int32_t)(begin + (refused ? 0 : total));
    const int lane = tid % kRowLanes;
    for (int i = (int)(g / kRowLanes); i < n; i += (int)(gn / kRowLanes)) {
        int32_t pair0 = -1, pair1 = -1;
        if (rank[i] >= 0) {
            const int32_t len = length[i];
            const int full = len >> a.block_shift;
            const int32_t *from = a.block_tables + (int64_t)a.src[i] * a.max_blocks_per_seq;
            int32_t *to = a.block_tables + (int64_t)a.dst[i] * a.max_blocks_per_seq;
            for (int j0 = lane; j0 < full; j0 += kRowLanes * kInFlight) {
                int32_t id[kInFlight];
#pragma unroll
                for (int k = 0; k < kInFlight; ++k) id[k] = j0 + kRowLanes * k < full ? from[j0 + kRowLanes * k] : 0;
#pragma unroll
                for (int k = 0; k < kInFlight; ++k) {
                    if (j0 + kRowLanes * k >= full) break;
                    if (in_pool(a, id[k])) {
                        atomicAdd(a.new_ref_counts + id[k], 1);
                    } else {
                        flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                        id[k] = -1;
                    }
                    to[j0 + kRowLanes * k] = id[k];
                }
            }
            if (lane == 0) {
                if (len & mask) {
                    int32_t id = a.free_blocks[begin + rank[i]];
                    const int32_t old = from[full];
                    if (in_pool(a, id)) atomicAdd(a.new_ref_counts + id, 1); else id = -1;
                    if (id >= 0 && in_pool(a, old)) {
                        pair0 = old;
                        pair1 = id;
                    } else {
                        flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                    }
                    to[full] = id;
                }
                a.context_lens[a.dst[i]] = len;
            }
        }
        if (lane == 0) {
            a.block_pairs[2 * (int64_t)i] = pair0;
            a.block_pairs[2 * (int64_t)i + 1] = pair1;
        }
    }
}

// ---------------------------------------------------------------------------------------------
// free
// ---------------------------------------------------------------------------------------------

__global__ void __launch_bounds__(1024, 1) free_pages_kernel(const FreeArgs a, const int words_per_cta) {
    extern __shared__ uint32_t bits[];  // freed pages of this CTA's part, those before each word, the listed rows
    __shared__ int tmp[32], count;
    const int S = a.num_seqs, nt = blockDim.x, tid = threadIdx.x;
    uint32_t *before = bits + words_per_cta, *listed = before + words_per_cta;
    for (int w = tid; w < (S + 31) / 32; w += nt) listed[w] = 0;
    pdl_wait();
    pdl_trigger();
    __syncthreads();
    const bool report = blockIdx.x == 0;
    const int64_t begin = *a.free_begin;
    const bool refused = begin < 0 || begin > a.num_free;
    if (refused && report && tid == 0) flag_error(a.err, PKV_DEVERR_FREE_BLOCKS);
    for (int i = tid; i < a.num_rows; i += nt) {
        const int32_t s = a.rows[i];
        if (s < 0 || refused) continue;  // padding
        if (s < S) atomicOr(listed + (s >> 5), 1u << (s & 31));  // a row listed twice is freed once
        else if (report) flag_error(a.err, PKV_DEVERR_SEQ);
    }
    const int64_t g = (int64_t)blockIdx.x * nt + tid, gn = (int64_t)gridDim.x * nt;
    // A negative count is a damaged one: 0 from here on, so that only freed pages have one below.
    for (int64_t b0 = g; b0 < a.num_blocks; b0 += gn * kInFlight) {
        int32_t held[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) held[k] = b0 + gn * k < a.num_blocks ? a.ref_counts[b0 + gn * k] : 0;
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            if (b0 + gn * k >= a.num_blocks) break;
            const bool bad = held[k] < 0 && !refused;
            if (bad) flag_error(a.err, PKV_DEVERR_BLOCK_ID);
            if (bad || a.new_ref_counts != a.ref_counts) a.new_ref_counts[b0 + gn * k] = bad ? 0 : held[k];
        }
    }
    sync_all();  // the counts are in place, the rows known, free_begin read

    // A page that loses its last holder is marked by a count far below zero; nothing but a damaged table
    // takes from it again, and what that takes it puts back.
    const int lane = tid % kRowLanes;
    for (int s = (int)(g / kRowLanes); s < S; s += (int)(gn / kRowLanes)) {
        const int32_t len = a.cached_lens[s];
        const bool gone = listed[s >> 5] >> (s & 31) & 1, good = good_len(a, len);
        if (gone && !good && lane == 0) flag_error(a.err, PKV_DEVERR_CONTEXT_LEN);
        const int64_t held = gone && good ? pages_of(a, len) : 0;
        const int32_t *row = a.block_tables + (int64_t)s * a.max_blocks_per_seq;
        for (int64_t j0 = lane; j0 < held; j0 += kRowLanes * kInFlight) {
            int32_t id[kInFlight], old[kInFlight];
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) id[k] = j0 + kRowLanes * k < held ? row[j0 + kRowLanes * k] : 0;
#pragma unroll
            for (int k = 0; k < kInFlight; ++k)
                old[k] = j0 + kRowLanes * k < held && in_pool(a, id[k]) ? atomicSub(a.new_ref_counts + id[k], 1) : 0;
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                if (j0 + kRowLanes * k >= held) break;
                if (old[k] == 1) {  // its last holder
                    atomicAdd(a.new_ref_counts + id[k], kFreed);
                } else if (old[k] <= 0) {  // not in the pool, or held by nobody: nothing to give back
                    flag_error(a.err, PKV_DEVERR_BLOCK_ID);
                    if (in_pool(a, id[k])) atomicAdd(a.new_ref_counts + id[k], 1);
                }
            }
        }
        __syncwarp(0xffffu << (threadIdx.x & kRowLanes));  // the row's lanes have all read the length
        if (lane == 0 && (a.context_lens != a.cached_lens || (gone && good))) a.context_lens[s] = gone && good ? 0 : len;
    }
    sync_all();

    const int id0 = blockIdx.x * words_per_cta * 32;  // below 2^23
    const int wl = tid & 31, nw = nt >> 5;
    const int64_t gathered = refused ? 0 : a.num_blocks;  // refused: no page was freed, whatever the counts are
    for (int w0 = tid >> 5; w0 < words_per_cta; w0 += nw * kInFlight) {
        int32_t held[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int id = id0 + 32 * (w0 + nw * k) + wl;
            held[k] = w0 + nw * k < words_per_cta && id < gathered ? __ldcg(a.new_ref_counts + id) : 0;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const bool freed = held[k] < 0;
            const uint32_t word = __ballot_sync(0xffffffffu, freed);
            if (w0 + nw * k >= words_per_cta) continue;
            if (freed) a.new_ref_counts[id0 + 32 * (w0 + nw * k) + wl] = 0;
            if (wl == 0) bits[w0 + nw * k] = word;
        }
    }
    __syncthreads();
    const int per = (words_per_cta + nt - 1) / nt;
    const int first = min(words_per_cta, tid * per), end = min(words_per_cta, first + per);
    int mine = 0, total;
    for (int w = first; w < end; ++w) mine += __popc(bits[w]);
    int at = block_scan(mine, tmp, &total);
    for (int w = first; w < end; ++w) {
        before[w] = at;
        at += __popc(bits[w]);
    }
    if (tid == 0) count = total;
    sync_all();
    int freed;
    const int64_t pos = cluster_scan(&count, &freed) + begin - freed;
    if (g == 0) {
        *a.free_end = (int32_t)(refused ? begin : max64(0, begin - freed));
        if (!refused && freed > begin) flag_error(a.err, PKV_DEVERR_FREE_BLOCKS);
    }
    for (int w = tid >> 5; w < words_per_cta; w += nw) {
        const uint32_t word = bits[w];
        const int64_t to = pos + before[w] + __popc(word & ((1u << wl) - 1));
        if ((word >> wl & 1) && to >= 0) a.free_blocks[to] = (int32_t)(id0 + 32 * w + wl);
    }
    sync_all();  // no CTA leaves while another reads its count
}

// ---------------------------------------------------------------------------------------------
// compact
// ---------------------------------------------------------------------------------------------

// With L live pages, m = the live ids >= L (as many as dead ids < L), at most the room of the
// pairs: move k takes the k-th live id from the top into the k-th dead id from the bottom.  An id's
// part follows from the number of live ids below it.  While tables are renamed, the new count of a
// page that moved away holds where it went (-1 - id).
__global__ void __launch_bounds__(1024, 1) compact_pages_kernel(const CompactArgs a, const int words_per_cta) {
    extern __shared__ uint32_t bits[];  // live pages of this CTA's part, then live pages before each word
    __shared__ int tmp[32], count;
    const int nt = blockDim.x, tid = threadIdx.x, lane = tid & 31, nw = nt >> 5;
    uint32_t *before = bits + words_per_cta;
    const int NB = (int)a.num_blocks, id0 = blockIdx.x * words_per_cta * 32;  // below 2^23
    pdl_wait();
    pdl_trigger();
    for (int w0 = tid >> 5; w0 < words_per_cta; w0 += nw * kInFlight) {
        int32_t held[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int id = id0 + 32 * (w0 + nw * k) + lane;
            held[k] = w0 + nw * k < words_per_cta && id < NB ? a.ref_counts[id] : 0;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            if (held[k] < 0) flag_error(a.err, PKV_DEVERR_BLOCK_ID);  // counts as dead
            const uint32_t live = __ballot_sync(0xffffffffu, held[k] > 0);
            if (lane == 0 && w0 + nw * k < words_per_cta) bits[w0 + nw * k] = live;
        }
    }
    __syncthreads();
    const int per = (words_per_cta + nt - 1) / nt;
    const int first = min(words_per_cta, tid * per), end = min(words_per_cta, first + per);
    int mine = 0, total;
    for (int w = first; w < end; ++w) mine += __popc(bits[w]);
    int at = block_scan(mine, tmp, &total);
    for (int w = first; w < end; ++w) {
        before[w] = at;
        at += __popc(bits[w]);
    }
    if (tid == 0) count = total;
    sync_all();
    int L, m = 0;
    const int base = cluster_scan(&count, &L);
    if (L < NB) {  // live ids below L
        const int word = L >> 5, c = word / words_per_cta, w = word - c * words_per_cta;
        const int earlier = __reduce_add_sync(0xffffffffu, lane < c ? *of_cta(&count, lane) : 0);
        const int below = earlier + of_cta(before, c)[w] + __popc(of_cta(bits, c)[w] & ((1u << (L & 31)) - 1));
        m = (int)min64(L - below, a.max_pairs);
    }
    for (int w0 = tid >> 5; w0 < words_per_cta; w0 += nw * kInFlight) {
        int32_t held[kInFlight];
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int id = id0 + 32 * (w0 + nw * k) + lane;
            held[k] = w0 + nw * k < words_per_cta && id < NB ? a.ref_counts[id] : 0;
        }
#pragma unroll
        for (int k = 0; k < kInFlight; ++k) {
            const int w = w0 + nw * k;
            const int id = id0 + 32 * w + lane;
            if (w >= words_per_cta || id >= NB) continue;
            const uint32_t word = bits[w];
            const bool live = word >> lane & 1;
            const int lives = base + (int)before[w] + __popc(word & ((1u << lane) - 1));  // live ids below this one
            const int deads = id - lives, tops = L - 1 - lives;                          // dead ones; live ones above
            const bool leaves = live && tops < m, filled = !live && deads < m;
            if (leaves) a.block_pairs[2 * tops] = id;
            if (filled) a.block_pairs[2 * deads + 1] = id;
            if (leaves || (!live && !filled)) {  // free behind the call
                const int rank = max(deads - m, 0) + max(lives - (L - m), 0);
                a.free_blocks[a.num_free - (NB - L) + rank] = id;
            }
            if (!leaves && !filled && (a.new_ref_counts != a.ref_counts || held[k] < 0))
                a.new_ref_counts[id] = max(held[k], 0);
        }
    }
    const int64_t g = (int64_t)blockIdx.x * nt + tid, gn = (int64_t)gridDim.x * nt;
    for (int64_t k = m + g; k < a.max_pairs; k += gn) a.block_pairs[2 * k] = a.block_pairs[2 * k + 1] = -1;
    if (g == 0) {
        *a.num_pairs = m;
        *a.free_end = (int32_t)(a.num_free - (NB - L));
    }
    sync_all();
    constexpr int kMoves = 4;  // that a thread has in flight
    for (int64_t k0 = g; k0 < m; k0 += gn * kMoves) {
        int2 move[kMoves];
        int32_t held[kMoves];
#pragma unroll
        for (int k = 0; k < kMoves; ++k)
            if (k0 + gn * k < m) {
                move[k].x = __ldcg(a.block_pairs + 2 * (k0 + gn * k));
                move[k].y = __ldcg(a.block_pairs + 2 * (k0 + gn * k) + 1);
            }
#pragma unroll
        for (int k = 0; k < kMoves; ++k)
            if (k0 + gn * k < m) held[k] = a.ref_counts[move[k].x];
#pragma unroll
        for (int k = 0; k < kMoves; ++k)
            if (k0 + gn * k < m) {
                a.new_ref_counts[move[k].y] = held[k];
                a.new_ref_counts[move[k].x] = -1 - move[k].y;
            }
    }
    sync_all();
    const int rl = tid % kRowLanes;
    for (int64_t s = g / kRowLanes; s < a.num_seqs; s += gn / kRowLanes) {
        const int32_t len = a.cached_lens[s];
        if (!good_len(a, len)) {
            if (rl == 0) flag_error(a.err, PKV_DEVERR_CONTEXT_LEN);
            continue;
        }
        const int64_t held = pages_of(a, len);
        const int32_t *row = a.block_tables + s * a.max_blocks_per_seq;
        int32_t *to = a.new_tables + s * a.max_blocks_per_seq;
        for (int64_t j0 = rl; j0 < held; j0 += kRowLanes * kInFlight) {
            int32_t id[kInFlight], went[kInFlight];
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) id[k] = j0 + kRowLanes * k < held ? row[j0 + kRowLanes * k] : 0;
#pragma unroll
            for (int k = 0; k < kInFlight; ++k) {
                went[k] = 0;
                if (j0 + kRowLanes * k >= held) continue;
                if (in_pool(a, id[k])) went[k] = __ldcg(a.new_ref_counts + id[k]);
                else flag_error(a.err, PKV_DEVERR_BLOCK_ID);  // stays as it is
            }
#pragma unroll
            for (int k = 0; k < kInFlight; ++k)
                if (j0 + kRowLanes * k < held) to[j0 + kRowLanes * k] = went[k] < 0 ? -1 - went[k] : id[k];
        }
    }
    sync_all();
    for (int64_t k = g; k < m; k += gn) a.new_ref_counts[__ldcg(a.block_pairs + 2 * k)] = 0;
}

// ---------------------------------------------------------------------------------------------

namespace {

// CTAs for a pool of `blocks` pages and `rows` rows to walk through: one for what 1024 threads take in one
// or two rounds (a barrier of a cluster costs as much as a round), else a cluster of 4 or of 16, the most
// there may be (more than 8 have to be allowed).  us with 1 / 4 / 8 / 16 CTAs, the rows' pages of their own:
//     rows x pages   free                      compact, a quarter free   fork into `rows`, in place
//     16 x 16        4.7 / 6.8 / 6.7 / 7.5     4.8 / 7.4 / 7.3 / 8.6     4.0 / 5.0 / 5.0 / 4.8
//     64 x 64        9.7 / 11.1 / 11.1 / 12.1  10.0 / 11.2 / 10.8 / 12.4 6.4 / 7.0 / 7.1 / 6.9
//     64 x 120       14.9 / 15.2 / 15.1 / 16.0 15.2 / 13.6 / 13.4 / 14.8 8.1 / 8.5 / 8.6 / 9.1
//     128 x 120      26.2 / 15.9 / 15.8 / 16.5 27.0 / 14.7 / 14.2 / 15.8 12.6 / 8.9 / 9.1 / 9.1
//     512 x 60       48.1 / 18.0 / 12.5 / 13.3 50.3 / 19.4 / 12.8 / 14.1 22.5 / 13.0 / 9.0 / 8.9
//     1024 x 100     148 / 44.7 / 25.8 / 18.0  160 / 47.3 / 27.1 / 19.5  64.7 / 22.0 / 13.7 / 11.1
// The rule is within 1.4 us of the best of them, here and at seven sizes between.  (A fork that is not in
// place copies the pool's counts: 1.1 us more at most.)
int ctas_for(int64_t blocks, int64_t rows, int max_blocks_per_seq) {
    const int64_t rounds = rows * ((max_blocks_per_seq + kRowLanes * kInFlight - 1) / (kRowLanes * kInFlight));
    if (blocks <= 8192 && rounds <= 64) return 1;
    return blocks <= 32768 && rounds <= 256 ? 4 : 16;
}

template <typename... Params, typename... Args>
cudaError_t launch_cluster(void (*kernel)(Params...), int ctas, int threads, size_t smem, SmemAllowance &allowed,
                           cudaStream_t stream, const Args &...args) {
    cudaError_t e = allow_dynamic_smem(kernel, smem, allowed);
    if (e != cudaSuccess) return e;
    if (ctas == 1) return launch_pdl(kernel, dim3(1), dim3(threads), smem, stream, args...);
    if (ctas > 8) e = cudaFuncSetAttribute(kernel, cudaFuncAttributeNonPortableClusterSizeAllowed, 1);
    if (e != cudaSuccess) return e;
    return launch_pdl_cluster(kernel, dim3(ctas), dim3(1024), ctas, smem, stream, args...);
}

int threads_for(int64_t blocks, int64_t rows) { return blocks <= 2048 && rows <= 16 ? 256 : 1024; }

}  // namespace

cudaError_t launch_fork_pages(const ForkArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const size_t smem = 4 * ((size_t)a.num_seqs + 2 * (size_t)a.num_forks);
    const int64_t blocks = a.new_ref_counts == a.ref_counts ? 0 : a.num_blocks;  // in place: not walked through
    return launch_cluster(fork_pages_kernel, ctas_for(blocks, a.num_forks, a.max_blocks_per_seq),
                          threads_for(blocks, a.num_forks), smem, allowed, stream, a);
}

cudaError_t launch_free_pages(const FreeArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const int64_t rows = a.num_rows < a.num_seqs ? a.num_rows : a.num_seqs;
    const int ctas = ctas_for(a.num_blocks, rows, a.max_blocks_per_seq);
    const int words = (int)((a.num_blocks + 31) / 32), per = words > 0 ? (words + ctas - 1) / ctas : 1;
    const size_t smem = 4 * (2 * (size_t)per + (size_t)(a.num_seqs + 31) / 32);
    return launch_cluster(free_pages_kernel, ctas, threads_for(a.num_blocks, rows), smem, allowed, stream, a, per);
}

cudaError_t launch_compact_pages(const CompactArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    const int ctas = ctas_for(a.num_blocks, a.num_seqs, a.max_blocks_per_seq);
    const int words = (int)((a.num_blocks + 31) / 32), per = words > 0 ? (words + ctas - 1) / ctas : 1;
    return launch_cluster(compact_pages_kernel, ctas, threads_for(a.num_blocks, a.num_seqs), 8 * (size_t)per, allowed,
                          stream, a, per);
}

}  // namespace pkv
