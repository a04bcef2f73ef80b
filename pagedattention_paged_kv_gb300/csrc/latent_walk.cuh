// latent_walk.cuh -- how the latent-attention kernels read a ragged batch: one sequence's
// lengths with their checks, the block-wide sum of every sequence's work units, and a
// warp's walk over the sequences of its CTA's share.  No per-sequence table is kept in
// shared memory, which the tiles need.
#pragma once

#include "pkv_common.cuh"

namespace pkv {

struct SeqBatch {
    const int32_t *query_start_loc;  // null: sequence s has the one query row s
    const int32_t *context_lens;
    int num_seqs;
    int total_q;                     // rows of q and out
    int64_t max_context;             // positions a block-table row can hold
    int *err;
};

// A sequence's lengths.  q_len = 0: nothing to compute.  dead: its rows are inside the
// output but there is nothing valid to compute (idle, or bad metadata): zero rows.
struct SeqInfo {
    int ctx, q0, q_len;
    bool dead;
};

// What memory holds about sequence s; the three loads are independent and nothing waits for them here.
struct SeqRaw {
    int32_t q0, q1, ctx;
};
__device__ __forceinline__ SeqRaw fetch_seq(const SeqBatch &b, int s) {
    SeqRaw r;
    r.q0 = b.query_start_loc ? b.query_start_loc[s] : s;
    r.q1 = b.query_start_loc ? b.query_start_loc[s + 1] : s + 1;
    r.ctx = b.context_lens[s];
    return r;
}

__device__ __forceinline__ SeqInfo vet_seq(const SeqBatch &b, const SeqRaw &w, bool report) {
    SeqInfo r;
    r.q0 = w.q0;
    r.q_len = 0;
    r.ctx = 0;
    r.dead = false;
    if (w.q0 < 0 || w.q1 < w.q0 || w.q1 > b.total_q) {
        if (report) flag_error(b.err, PKV_DEVERR_QUERY_LEN);
        return r;
    }
    if (w.q1 == w.q0) return r;
    r.q_len = w.q1 - w.q0;
    r.ctx = w.ctx;
    if (r.ctx < 0 || r.ctx > b.max_context) {
        if (report) flag_error(b.err, PKV_DEVERR_CONTEXT_LEN);
        r.dead = true;
    } else if (r.q_len > r.ctx) {
        // an idle slot of a decode batch (context 0) is no error
        if (report && b.query_start_loc) flag_error(b.err, PKV_DEVERR_QUERY_LEN);
        r.dead = true;
    }
    return r;
}

__device__ __forceinline__ SeqInfo read_seq(const SeqBatch &b, int s, bool report) {
    return vet_seq(b, fetch_seq(b, s), report);
}

// Units(const SeqInfo &) -> int64_t gives the work units of a live sequence.
template <typename Units>
__device__ __forceinline__ int64_t units_of(const SeqInfo &q, const Units &units) {
    return q.q_len == 0 || q.dead ? 0 : units(q);
}

// The threads of a block take equal runs of consecutive sequences; for each of K counts of units
// run = units before this thread's first one.
template <int K>
struct BatchScan {
    int beg, end;
    SeqInfo first;  // of sequence beg, where there is one
    int64_t run[K], local[K], total[K];
};

// Whole block of NT threads; tmp holds NT / 32 entries a count and is not to be written again before
// the next __syncthreads.  (Every CTA of a launch starts with it, and what the block's size, the
// number of counts and the loads' independence leave to the compiler halved its time to 1,000 cycles.)
template <int NT, typename... Units>
__device__ __forceinline__ BatchScan<sizeof...(Units)> scan_batch(const SeqBatch &b, int64_t *tmp, bool report,
                                                                  const Units &...units) {
    constexpr int K = sizeof...(Units), NW = NT / 32;
    BatchScan<K> r;
    const int tid = threadIdx.x, lane = tid & 31, warp = tid >> 5;
    const int per = (b.num_seqs + NT - 1) / NT;
    r.beg = min(b.num_seqs, tid * per);
    r.end = min(b.num_seqs, r.beg + per);
    r.first.ctx = r.first.q0 = r.first.q_len = 0;
    r.first.dead = false;
    int64_t x[K];
#pragma unroll
    for (int k = 0; k < K; ++k) r.local[k] = 0;
    for (int s = r.beg; s < r.end; ++s) {
        const SeqInfo q = read_seq(b, s, report);
        if (s == r.beg) r.first = q;
        const int64_t u[K] = {units_of(q, units)...};
#pragma unroll
        for (int k = 0; k < K; ++k) r.local[k] += u[k];
    }
#pragma unroll
    for (int k = 0; k < K; ++k) x[k] = r.local[k];
#pragma unroll
    for (int o = 1; o < 32; o <<= 1) {
#pragma unroll
        for (int k = 0; k < K; ++k) {
            const int64_t y = __shfl_up_sync(0xffffffffu, x[k], o);
            if (lane >= o) x[k] += y;
        }
    }
    if (lane == 31)
#pragma unroll
        for (int k = 0; k < K; ++k) tmp[k * NW + warp] = x[k];
    __syncthreads();
#pragma unroll
    for (int k = 0; k < K; ++k) {
        int64_t before = 0, total = 0;
#pragma unroll
        for (int i = 0; i < NW; ++i) {
            const int64_t v = tmp[k * NW + i];
            if (i < warp) before += v;
            total += v;
        }
        r.run[k] = before + x[k] - r.local[k];
        r.total[k] = total;
    }
    return r;
}

// Where a CTA's share starts: the sequence that holds its first unit.
struct WalkStart {
    int64_t pre, units;  // units before the sequence, its units
    SeqInfo q;
    int s;
};

// The one thread whose run holds unit f (of count k) writes *start.  Callers synchronise afterwards.
template <int K, typename Units>
__device__ __forceinline__ bool find_unit(const SeqBatch &b, const Units &units, const BatchScan<K> &sc, int k,
                                          int64_t f, WalkStart *start) {
    if (f < sc.run[k] || f >= sc.run[k] + sc.local[k]) return false;
    int64_t run = sc.run[k];
    SeqInfo q = sc.first;
    for (int s = sc.beg;;) {
        const int64_t u = units_of(q, units);
        if (f < run + u) {
            start->pre = run;
            start->units = u;
            start->q = q;
            start->s = s;
            return true;
        }
        run += u;
        if (++s >= sc.end) return false;  // (not reached: the run's units are `local`)
        q = read_seq(b, s, false);
    }
}

// a / b for a >= 0, b > 0; the 64-bit division, many times slower, only where it is needed.
__device__ __forceinline__ int64_t quotient(int64_t a, int64_t b) {
    if (((a | b) >> 32) == 0) return (int64_t)((uint32_t)a / (uint32_t)b);
    return a / b;
}

// A warp's walk over the sequences from a starting one on, 32 sequences to a round of loads.
// Every call is warp-wide; the current sequence's data is uniform.
template <typename Units>
struct SeqWalk {
    int s;             // current sequence
    int64_t pre;       // units before it
    int64_t units;     // its units (> 0)
    SeqInfo q;
    int base;          // sequence of lane 0 (below 0: nothing fetched yet)
    SeqRaw raw;        // this lane's sequence, not looked at yet (fresh) ...
    bool fresh;
    SeqInfo mine;      // ... and once it has been
    int64_t my_units;

    __device__ __forceinline__ void fetch(const SeqBatch &b, int first) {
        base = first;
        raw.q0 = raw.q1 = raw.ctx = 0;
        const int i = first + (int)(threadIdx.x & 31);
        if (i < b.num_seqs) raw = fetch_seq(b, i);
        fresh = true;
    }
    __device__ __forceinline__ void look(const SeqBatch &b, const Units &u) {
        if (!fresh) return;
        fresh = false;
        mine = vet_seq(b, raw, false);
        my_units = mine.q_len > 0 && !mine.dead ? u(mine) : 0;
    }
    __device__ __forceinline__ void take(int l) {
        s = base + l;
        q.ctx = __shfl_sync(0xffffffffu, mine.ctx, l);
        q.q0 = __shfl_sync(0xffffffffu, mine.q0, l);
        q.q_len = __shfl_sync(0xffffffffu, mine.q_len, l);
        q.dead = false;
        units = __shfl_sync(0xffffffffu, my_units, l);
    }
    __device__ __forceinline__ void start(const WalkStart &st) {
        s = st.s;
        pre = st.pre;
        units = st.units;
        q = st.q;
        base = -1;
        fresh = false;
        my_units = 0;
    }
    // The loads of the sequences behind the first are under way from here on.  (Not from start on:
    // registers that a load fills are moved, and so waited for, before the first seek is over.)
    __device__ __forceinline__ void ahead(const SeqBatch &b) {
        if (base < 0) fetch(b, s);
    }
    // Moves on until the current sequence holds unit f (f >= pre, f below the batch's total).
    __device__ __forceinline__ void seek(const SeqBatch &b, const Units &u, int64_t f) {
        while (f >= pre + units) {
            pre += units;
            ahead(b);
            look(b, u);
            const int at = s - base;
            unsigned later = __ballot_sync(0xffffffffu, my_units > 0) & (at >= 31 ? 0u : 0xffffffffu << (at + 1));
            while (later == 0) {
                if (base + 32 >= b.num_seqs) return;  // past the last sequence (not reached for f < total)
                fetch(b, base + 32);
                look(b, u);
                later = __ballot_sync(0xffffffffu, my_units > 0);
            }
            take(__ffs(later) - 1);
        }
    }
};

// Zero rows of the dead sequences (of every one, with `all`) among cta, cta + grid, ..., by warp
// `w` of `nw`; one warp a sequence.
__device__ __forceinline__ void zero_dead_rows(const SeqBatch &b, int cta, int grid, __nv_bfloat16 *out,
                                               int64_t row_elems, int w, int nw, bool all = false) {
    const int lane = threadIdx.x & 31;
    for (int64_t s = cta + (int64_t)grid * w; s < b.num_seqs; s += (int64_t)grid * nw) {
        const SeqInfo q = read_seq(b, (int)s, false);
        if (q.q_len == 0 || !(q.dead || all)) continue;
        uint4 *o = reinterpret_cast<uint4 *>(out + q.q0 * row_elems);
        const int64_t n = q.q_len * row_elems / 8;
        for (int64_t i = lane; i < n; i += 32) o[i] = make_uint4(0u, 0u, 0u, 0u);
    }
}

}  // namespace pkv
