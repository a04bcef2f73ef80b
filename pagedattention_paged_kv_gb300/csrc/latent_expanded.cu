// latent_expanded.cu -- attention of prompt chunks over expanded per-head keys and values of
// a latent cache (sm_103a): scores over 128 + 64 columns (a head's key part, then the rotary
// part all heads share), values of 128 columns.
//
//   out[i][h] = softmax_j(scale * (q_nope . k[h][j] + q_rope . r_j)) v[h][j],  j <= position of i
//
// Bound: tensor, 2 * (192 + 128) operations a visible (query, key) pair and head.
//
// Layout
//  * A work tile is 256 query tokens of one head as two 128-row MMA halves; its units are
//    128-key chunks, causal tiles stop at their last query's position.  A persistent grid
//    takes equal contiguous shares of the flat unit list; split tiles are joined by a
//    second kernel (latent_merge.cuh).
//  * A chunk is 80 KiB: a pair of 64-column pieces of the head's keys, the rotary piece, and a
//    pair of its values.  Q takes 96 KiB, so two whole chunks do not fit; the pairs go through
//    three places and the rotary pieces through two; a place is reused by the pair three on in the
//    order keys, values, keys, .. .  (With one place for
//    values their latency was half of a chunk's time: 5,000 cycles for 2,560 of tensor work.)
//  * A causal tile's first half skips the chunks that only its second half sees.
//  * Per half TMEM holds S (128 columns, overwritten by the 16-bit weights P) and O (128).  The
//    issuer runs PV of one half and QK of its next chunk while the other half's warpgroup (one
//    thread a row) computes its weights, as in the paged prefill.
//  * Values and weights are fp16 (11 bits against bf16's 8; kind::f16 takes both operands of
//    one type, so they go together): with bf16 the rounding of each weighed as much as that
//    of the result and the error was 1.6 times the result's own rounding.  The weights are held
//    2^kWeightShift times larger, up to 2^15 by the rescale rule: each is off by 2^-11 of itself or
//    2^-32 of the largest, so that small ones count where the large one's value is near zero.
//  * The values of 32 keys are stored 2^-x times as large, so that small ones keep their bits
//    (latent_expand.cu): with s' = s + x,
//        out = sum_j 2^(s'_j - m) (2^-x v_j) / sum_j 2^-x 2^(s'_j - m)
//    where m is the running maximum of the s', so weights stay below 2^15 whatever the x.  Values past
//    fp16's range are clamped and flagged where they are made.  Keys stay bf16, the type of the
//    queries they meet.
//  * The kernel starts under the expansion's tail.  Every role waits for the expansion's end before its
//    first limited wait (the producer behind its first query load), so a limit counts this kernel's
//    own steps.  Waits are bounded in time; no CTA of the kernel waits on another.
//
// Measured with the expansion and the join, R = 512, 64 heads, in a graph of calls: a chunk of 512 queries
// behind 16,384 tokens 447 to 485 us (331 at the matrix products' peak rate), eight prompts of 500 to 2500
// tokens 475 to 499 (270).  With plain fp16 values, whose small ones were lost, these were 443 to 478 and
// 466 to 488.  Back to back the chunk runs at the board's power limit (1370 W, SM
// clock 1.65 GHz of 2.07): chunks of 96 keys in two whole stages with an issuer a half took 2,770 cycles
// for 96 keys against 4,500 for 128, and no less time.  At full clocks a chunk's 4,500 cycles are
// 2,550 of products, the issuer's steps between them, and waits for keys, which are asked for
// 1,270 cycles of products before they are needed.
#include "attn_block.cuh"
#include "fp32x2.cuh"
#include "latent_expanded.cuh"
#include "latent_walk.cuh"
#include "pkv_split.cuh"
#include "tcgen05.cuh"

namespace pkv {

namespace {

// A share that would begin this close to a tile's begin or end, in chunks, begins there instead
// (snap_start): a cut one chunk from an end would cost a part and its join for next to no balance.
constexpr int kSnap = 1;

// exp2(s - m + kWeightShift) <= 2^(kRescaleSlack + kWeightShift) = 2^15, half of fp16's range.  Sums and
// outputs of a row, and its parts', are all this much larger.
constexpr float kWeightShift = 7.0f;
static_assert(kRescaleSlack + kWeightShift <= 15.0f, "weights fit fp16");

constexpr int kExpandedThreads = 384;  // loads, MMAs, two idle warps, two softmax warpgroups

struct ExpandedSmem {
    static constexpr uint32_t PIECE = 128 * 128;             // 128 rows x 64 columns
    static constexpr uint32_t Q_BYTES = 2 * 3 * PIECE;       // [half][piece]
    static constexpr uint32_t PAIR = 2 * PIECE;
    static constexpr uint32_t OFF_PAIRS = Q_BYTES;           // three places
    static constexpr uint32_t OFF_ROPE = OFF_PAIRS + 3 * PAIR;  // two places
    static constexpr uint32_t OFF_MISC = OFF_ROPE + 2 * PIECE;
    static constexpr uint32_t BYTES = OFF_MISC + 1024 + 1024;
    static constexpr uint32_t HALF_COLS = 256, COL_O = 128;
    static_assert(BYTES <= 232448, "fits one CTA");
};

// Closed forms for the tiles of one (sequence, head).  Causal: full tile qt visits
// A + 2 (qt + 1) chunks, A = ceil((ctx - q_len) / 128); the last, partial one all of them.
struct ExpandedTiles {
    int A, nfull, rem, nk;
    bool causal;
    __device__ __forceinline__ ExpandedTiles(const SeqInfo &q, bool causal_) : causal(causal_) {
        A = (q.ctx - q.q_len + kExpTile - 1) / kExpTile;
        nfull = q.q_len / kExpQTile;
        rem = q.q_len % kExpQTile;
        nk = (q.ctx + kExpTile - 1) / kExpTile;
    }
    __device__ __forceinline__ int count() const { return nfull + (rem > 0); }
    __device__ __forceinline__ int64_t before(int qt) const {  // chunks before tile qt <= nfull
        return (int64_t)qt * (causal ? A + qt + 1 : nk);
    }
    __device__ __forceinline__ int chunks(int qt) const { return !causal || qt >= nfull ? nk : A + 2 * (qt + 1); }
    __device__ __forceinline__ int64_t per_head() const { return before(nfull) + (rem > 0 ? nk : 0); }
    __device__ __forceinline__ int tile_of(int64_t o) const {  // tile that holds chunk o
        if (o >= before(nfull)) return nfull;
        int lo = 0, hi = nfull;
        while (hi - lo > 1) {
            const int mid = (lo + hi) >> 1;
            if (before(mid) <= o) lo = mid; else hi = mid;
        }
        return lo;
    }
};

struct ExpandedUnits {
    int num_heads;
    bool causal;
    __device__ __forceinline__ int64_t operator()(const SeqInfo &q) const {
        return ExpandedTiles(q, causal).per_head() * num_heads;
    }
};

// Units of the expansion, whose sum tells whether the batch fits the workspace.
struct TokenTiles {
    __device__ __forceinline__ int64_t operator()(const SeqInfo &q) const { return (q.ctx + kExpTile - 1) / kExpTile; }
};

struct ExpandedSegment {
    int h, qt;           // head, tile
    int kb, chunks;      // first chunk of the segment, chunks in it
    int tokens;          // query tokens of the tile
    int first_half;      // chunks of the segment that the tile's first half sees
    bool whole;
};

// Where a share begins: tile qt of head h of the sequence in `seq`, chunk kb (kb = the tile's chunks:
// behind it).
struct ExpandedStart {
    WalkStart seq;
    int64_t tiles;  // expansion tiles before the sequence
    int64_t unit;
    int h, qt, kb;
};

// The start nearest unit f of the sequence in st->seq: where the tile that holds it begins or
// ends if that is at most kSnap chunks away, so that short tiles are not cut.
__device__ __forceinline__ void snap_start(ExpandedStart *st, bool causal, int64_t f) {
    const ExpandedTiles t(st->seq.q, causal);
    const int64_t ph = t.per_head(), o = f - st->seq.pre, h = quotient(o, ph), o1 = o - h * ph;
    const int qt = t.tile_of(o1), at = (int)(o1 - t.before(qt)), n = t.chunks(qt);
    const int kb = at <= kSnap ? 0 : n - at <= kSnap ? n : at;
    st->h = (int)h;
    st->qt = qt;
    st->kb = kb;
    st->unit = f + (kb - at);
}

// A warp's walk over the tiles of its CTA's share: steps, no division.  (The first pass through
// any code waits for its instructions, so what every role runs before its first tile is kept short:
// finding the tile of a unit anew for every segment put 9,000 cycles before the first load.)
struct TileWalk {
    SeqWalk<ExpandedUnits> w;
    ExpandedTiles t;
    int64_t left;   // units of the share from here on
    int64_t tiles;  // expansion tiles before the sequence
    int h, qt, kb;
    bool causal;
    int heads;
    __device__ __forceinline__ TileWalk(const SeqBatch &sb, const ExpandedUnits &u, const ExpandedStart &st, int64_t hi)
        : t(st.seq.q, u.causal), left(hi - st.unit), tiles(st.tiles), h(st.h), qt(st.qt), kb(st.kb),
          causal(u.causal), heads(u.num_heads) {
        w.start(st.seq);
        if (left > 0 && kb == t.chunks(qt)) next(sb, u);
    }
    __device__ __forceinline__ void next(const SeqBatch &sb, const ExpandedUnits &u) {
        kb = 0;
        if (++qt < t.count()) return;
        qt = 0;
        if (++h < heads) return;
        h = 0;
        tiles += t.nk;
        w.seek(sb, u, w.pre + w.units);
        t = ExpandedTiles(w.q, causal);
    }
    __device__ __forceinline__ ExpandedSegment segment() const {
        ExpandedSegment g;
        g.h = h;
        g.qt = qt;
        g.kb = kb;
        const int n = t.chunks(qt);
        g.chunks = (int)min64(n - kb, left);
        g.tokens = min(kExpQTile, w.q.q_len - qt * kExpQTile);
        g.whole = g.chunks == n;
        const int last0 = w.q.ctx - w.q.q_len + qt * kExpQTile + min(g.tokens, 128);  // keys its last token sees
        g.first_half = causal && g.tokens > 128
                           ? max(0, min(g.chunks, (last0 + kExpTile - 1) / kExpTile - kb)) : g.chunks;
        return g;
    }
    // past the segment
    __device__ __forceinline__ void advance(const SeqBatch &sb, const ExpandedUnits &u, const ExpandedSegment &g) {
        left -= g.chunks;
        if (left > 0) next(sb, u);
    }
};

struct ExpandedMisc {
    uint64_t q_full, q_empty, mma_done;
    uint64_t full[3], empty[3], rope_full[2], rope_empty[2];
    uint64_t s_full[2], p_full[2], pv_done[2], o_free[2];
    int64_t scan[2 * kExpandedThreads / 32];
    ExpandedStart start[2];  // of this share and the next
    uint32_t tmem_slot;
    int abort_flag;
};
static_assert(sizeof(ExpandedMisc) <= 1024, "fits its place");

// Chunks of a segment that half h has to do with.
__device__ __forceinline__ int half_chunks(const ExpandedSegment &g, int h) {
    return h == 0 ? g.first_half : g.tokens > 128 ? g.chunks : 0;
}

}  // namespace

__global__ void __launch_bounds__(kExpandedThreads, 1)
latent_expanded_kernel(const __grid_constant__ CUtensorMap q_map, const __grid_constant__ CUtensorMap kv_map,
                       const __grid_constant__ CUtensorMap rope_map, const ExpandedArgs a) {
    using L = ExpandedSmem;
    extern __shared__ uint8_t smem_raw[];
    uint8_t *smem = reinterpret_cast<uint8_t *>((reinterpret_cast<uintptr_t>(smem_raw) + 1023) & ~uintptr_t(1023));
    uint8_t *sQ = smem, *sPairs = smem + L::OFF_PAIRS, *sRope = smem + L::OFF_ROPE;
    ExpandedMisc &ms = *reinterpret_cast<ExpandedMisc *>(smem + L::OFF_MISC);
    volatile int *abort_flag = &ms.abort_flag;
    const int warp = threadIdx.x >> 5, lane = threadIdx.x & 31;
    const int c = blockIdx.x;

    if (threadIdx.x == 0) {
        mbar_init(&ms.q_full, 1);
        mbar_init(&ms.q_empty, 1);
        mbar_init(&ms.mma_done, 1);
        for (int i = 0; i < 3; ++i) {
            mbar_init(&ms.full[i], 1);
            mbar_init(&ms.empty[i], 1);
        }
        for (int i = 0; i < 2; ++i) {
            mbar_init(&ms.rope_full[i], 1);
            mbar_init(&ms.rope_empty[i], 1);
            mbar_init(&ms.s_full[i], 1);
            mbar_init(&ms.p_full[i], 4);  // one arrival per softmax warp of the half
            mbar_init(&ms.pv_done[i], 1);
            mbar_init(&ms.o_free[i], 4);
        }
        ms.abort_flag = 0;
        fence_barrier_init();
    }
    if (threadIdx.x == 32) {
        tma_prefetch_desc(&q_map);
        tma_prefetch_desc(&kv_map);
        tma_prefetch_desc(&rope_map);
    }
    // The expansion's CTAs let this kernel start once everything before them is complete, so all
    // inputs of the call may be read here; only what the expansion writes has to be waited for (CTAs
    // without work wait too, so that this grid ends behind the last).
    pdl_trigger();
    // A CTA of this kernel has the SM's shared memory, so no other holder of TMEM is there.
    if (warp == 1) tmem_alloc(&ms.tmem_slot, 512);
    const SeqBatch sb{a.query_start_loc, a.context_lens, a.num_seqs, a.total_q, a.max_context, a.err};
    const ExpandedUnits units{a.num_heads, a.causal};
    // (the expansion kernel has reported bad sequences already)
    const auto sc = scan_batch<kExpandedThreads>(sb, ms.scan, false, units, TokenTiles{});
    const bool fits = sc.total[1] <= a.buf.padded / kExpTile;
    const int64_t T = fits ? sc.total[0] : 0;
    const int ge = split_ctas(T, a.grid, 1);
    const bool works = T > 0 && c < ge;
    // This share's begin and the next one's, each found by the thread whose sequences hold it.
#pragma unroll 1
    for (int i = 0; i < 2 && works; ++i) {
        const int64_t f = quotient((c + i) * T, ge);
        ExpandedStart *st = &ms.start[i];
        if (f < T && find_unit(sb, units, sc, 0, f, &st->seq)) {
            snap_start(st, a.causal, f);
            st->tiles = sc.run[1];
            SeqInfo q = sc.first;
            for (int s = sc.beg; s < st->seq.s; q = read_seq(sb, ++s, false)) st->tiles += units_of(q, TokenTiles{});
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    const uint32_t tmem = ms.tmem_slot;
    const int64_t hi = !works ? 0 : c + 1 < ge ? ms.start[1].unit : T;

    if (warp == 2 || warp == 3) {  // (these have nothing else to do)
        // The merge job of the boundary before this CTA's share (see latent_absorbed.cu).
        if (threadIdx.x == 64) {
            LatentJob j{0, -1, -1, 0};
            if (works && c > 0) {
                const ExpandedStart st = ms.start[0];
                const int n = ExpandedTiles(st.seq.q, a.causal).chunks(st.qt);
                const int64_t begin = st.unit - st.kb;
                // a cut tile has more than 2 kSnap + 1 chunks; its first part is that of the last share
                // that begins before it or snapped to its begin
                if (st.kb > 0 && st.kb < n && share_owner(begin + kSnap, T, ge) == c - 1) {
                    j.out_off = ((int64_t)(st.seq.q.q0 + st.qt * kExpQTile) * a.num_heads + st.h) * kExpHeadDim;
                    j.c0 = c - 1;
                    j.c1 = share_owner(begin + n - kSnap - 1, T, ge);
                    j.rows = min(kExpQTile, st.seq.q.q_len - st.qt * kExpQTile);
                }
            }
            if (c > 0) a.ws_jobs[c - 1] = j;
            if (c == a.grid - 1) {
                j.c0 = -1;
                a.ws_jobs[c] = j;
            }
        }
        __syncwarp();
        zero_dead_rows(sb, c, a.grid, a.out, (int64_t)a.num_heads * kExpHeadDim, warp - 2, 2, !fits);
    }
    if (!works) {
        __syncwarp();
        if (warp == 1) tmem_dealloc(tmem, 512);
        pdl_wait();
        return;
    }

    TileWalk tw(sb, units, ms.start[0], hi);
    SeqWalk<ExpandedUnits> &w = tw.w;
    if (warp != 0) {  // the producer is on the critical path
        w.ahead(sb);
        pdl_wait();
    }
    auto wait_all = [&](uint64_t *bar, uint32_t parity) -> bool {
        return __all_sync(0xffffffffu, mbar_wait(bar, parity, abort_flag, a.wait_ns));
    };
    bool ok = true;

    if (warp == 0) {
        // ------------------------------ TMA producer ------------------------------
        // The warp runs it together on uniform values; one elected lane issues.
        const uint64_t policy = l2_policy_evict_normal(), once = l2_policy_evict_first();
        const uint32_t pairs0 = smem_u32(sPairs), rope0 = smem_u32(sRope);
        uint32_t n = 0, segs = 0;   // chunks and tiles issued
        uint32_t np = 0, nr = 0;    // pairs and rotary pieces issued
        // pair i = 2 chunk (keys) or 2 chunk + 1 (values) of the CTA
        const int pitch = (int)a.buf.padded;  // rows from a piece to the next
        auto load_pair = [&](uint32_t i, int row) -> bool {
            const uint32_t at = i % 3, times = i / 3;
            if (times > 0 && !wait_all(&ms.empty[at], (times - 1) & 1)) return false;
            mbar_arrive_expect_tx_warp(&ms.full[at], L::PAIR);
            tma_load_2d_warp(pairs0 + at * L::PAIR, &kv_map, &ms.full[at], 0, row, policy);
            tma_load_2d_warp(pairs0 + at * L::PAIR + L::PIECE, &kv_map, &ms.full[at], 0, row + pitch, policy);
            ++np;
            return true;
        };
        bool waited = false;
        while (tw.left > 0 && ok) {
            const ExpandedSegment g = tw.segment();
            int key = __shfl_sync(0xffffffffu, (int)(tw.tiles + g.kb) * kExpTile, 0);
            int row = __shfl_sync(0xffffffffu, (int)(4 * g.h * a.buf.padded) + key, 0);
            const int chunks = __shfl_sync(0xffffffffu, g.chunks, 0);
            if (segs > 0) ok = wait_all(&ms.q_empty, (segs - 1) & 1);
            if (!ok) break;
            const int nh = g.tokens > 128 ? 2 : 1;
            if (lane == 0) {
                mbar_arrive_expect_tx(&ms.q_full, nh * 3 * L::PIECE);
                for (int h = 0; h < nh; ++h)
                    for (int p = 0; p < 3; ++p)
                        tma_load_4d(sQ + (h * 3 + p) * L::PIECE, &q_map, &ms.q_full, 0, p, g.h,
                                    (int)(w.q.q0 + g.qt * kExpQTile) + h * 128, once);
            }
            __syncwarp();
            ++segs;
            if (!waited) pdl_wait();  // from here on the expansion's output is read
            waited = true;
            for (int ch = 0; ch < chunks; ++ch) {
                if (!load_pair(2 * n, row)) { ok = false; break; }
                if (n >= 2 && !wait_all(&ms.rope_empty[n & 1], ((n >> 1) - 1) & 1)) { ok = false; break; }
                mbar_arrive_expect_tx_warp(&ms.rope_full[n & 1], L::PIECE);
                tma_load_2d_warp(rope0 + (n & 1) * L::PIECE, &rope_map, &ms.rope_full[n & 1], 0, key, policy);
                ++nr;
                if (!load_pair(2 * n + 1, row + 2 * pitch)) { ok = false; break; }
                // The next chunk's pieces into L2, while their places are still in use.
                if (ch + 1 < chunks && lane < 4)
                    l2_prefetch(a.buf.kv + ((int64_t)row + kExpTile + (int64_t)lane * pitch) * 64, L::PIECE);
                __syncwarp();
                key += kExpTile;
                row += kExpTile;
                ++n;
                w.ahead(sb);
            }
            tw.advance(sb, units, g);
        }
        if (!waited) pdl_wait();
        if (lane == 0) {
            if (!ok) {
                flag_error(a.err, PKV_DEVERR_TIMEOUT);
                *abort_flag = 1;
            }
            // The copies land before this CTA ends, whoever else has given up waiting for them.
            for (uint32_t i = np > 3 ? np - 3 : 0; i < np; ++i) mbar_wait(&ms.full[i % 3], (i / 3) & 1, nullptr);
            for (uint32_t i = nr > 2 ? nr - 2 : 0; i < nr; ++i) mbar_wait(&ms.rope_full[i & 1], (i >> 1) & 1, nullptr);
            if (segs > 0) mbar_wait(&ms.q_full, (segs - 1) & 1, nullptr);
        }
    } else if (warp == 1) {
        // ------------------------------ MMA issuer ------------------------------
        // PV_h(c), then QK_h(c + 1) over the same S columns; the halves alternate.  The last half to
        // use a place gives it back.  (An issuer a half was slower: without turns the halves fall
        // into step, weights and MMAs of both at the same time; with turns a step waits for keys that
        // the other half's step makes room for.)
        constexpr uint32_t IDESC_QK = umma_idesc_bf16(128, kExpTile, 0, 0);
        constexpr uint32_t IDESC_PV = umma_idesc_f16(128, kExpHeadDim, 0, 1);
        const uint32_t tm = __shfl_sync(0xffffffffu, tmem, 0);
        const uint64_t dq0 = umma_desc_sw128(smem_u32(sQ), 16, 1024);
        const uint64_t dk0 = umma_desc_sw128(smem_u32(sPairs), 16, 1024);
        const uint64_t dr0 = umma_desc_sw128(smem_u32(sRope), 16, 1024);
        const uint64_t dv0 = umma_desc_sw128(smem_u32(sPairs), L::PIECE, 1024);
        uint32_t n = 0;             // chunks whose PV is behind
        uint32_t kp = 0, kq = 0;    // place and parity of the next chunk's keys
        uint32_t vp = 1, vq = 0;    // and of the current one's values
        uint32_t pq = 0;            // by half, a bit each: parity of its next weights,
        uint32_t oq = 0, used = 0;  // parity of its next accumulator's release, whether it had one
        uint32_t segs = 0;
        auto next2 = [&](uint32_t &place, uint32_t &parity) {  // two pairs on
            place += 2;
            if (place >= 3) {
                place -= 3;
                parity ^= 1;
            }
        };
        // QK of chunk `chunk` (its keys at kp, kq)
        auto issue_qk = [&](int h, uint32_t chunk, bool last) -> bool {
            if (!wait_all(&ms.full[kp], kq)) return false;
            tc_fence_after();
            const uint64_t dk = umma_desc_at(dk0, kp * L::PAIR), dr = umma_desc_at(dr0, (chunk & 1) * L::PIECE);
            const uint64_t dq = dq0 + h * (3 * L::PIECE >> 4);
            const uint32_t tS = tm + h * L::HALF_COLS;
#pragma unroll
            for (int ks = 0; ks < 8; ++ks) {
                const uint32_t off = ((ks / 4) * L::PIECE + (ks % 4) * 32) >> 4;
                umma_bf16_warp(tS, dq + off, dk + off, IDESC_QK, ks > 0);
            }
            if (last) umma_commit_warp(&ms.empty[kp]);
            if (!wait_all(&ms.rope_full[chunk & 1], (chunk >> 1) & 1)) return false;
            tc_fence_after();
#pragma unroll
            for (int ks = 0; ks < 4; ++ks)
                umma_bf16_warp(tS, dq + ((2 * L::PIECE + ks * 32) >> 4), dr + (ks * 32 >> 4), IDESC_QK, true);
            umma_commit_warp(&ms.s_full[h]);
            if (last) {
                umma_commit_warp(&ms.rope_empty[chunk & 1]);
                next2(kp, kq);
            }
            return true;
        };
        auto issue_pv = [&](int h, bool first, bool last) -> bool {
            if (!wait_all(&ms.full[vp], vq)) return false;
            tc_fence_after();
            const uint64_t dv = umma_desc_at(dv0, vp * L::PAIR);
            const uint32_t tP = tm + h * L::HALF_COLS;
#pragma unroll
            for (int ks = 0; ks < kExpTile / 16; ++ks)
                umma_bf16_tmem_a_warp(tP + L::COL_O, tP + ks * 8, dv + (ks * 2048 >> 4), IDESC_PV, !first || ks > 0);
            umma_commit_warp(&ms.pv_done[h]);
            if (last) {
                umma_commit_warp(&ms.empty[vp]);
                next2(vp, vq);
            }
            return true;
        };
        while (tw.left > 0 && ok) {
            const ExpandedSegment g = tw.segment();
            const int chunks = __shfl_sync(0xffffffffu, g.chunks, 0);
            const int cnt0 = __shfl_sync(0xffffffffu, half_chunks(g, 0), 0);
            const int cnt1 = __shfl_sync(0xffffffffu, half_chunks(g, 1), 0);
            const int last = cnt1 > 0 ? 1 : 0;  // the second half, where there is one, sees every chunk
            if (!wait_all(&ms.q_full, segs & 1)) { ok = false; break; }
            // One copy of the code for both halves and for the first scores: every line of it waits
            // for its instructions once, 2,000 cycles a copy.
#pragma unroll 1
            for (int step = -2; step < 2 * chunks && ok; ++step) {
                const int ch = step >> 1, h = step & 1, cnt = h ? cnt1 : cnt0;
                if (ch >= 0 && ch < cnt) {
                    if (ch == 0) {
                        if ((used >> h & 1) && !wait_all(&ms.o_free[h], oq >> h & 1)) { ok = false; break; }
                        oq ^= (used >> h & 1) << h;
                        used |= 1u << h;
                    }
                    if (!wait_all(&ms.p_full[h], pq >> h & 1)) { ok = false; break; }
                    pq ^= 1u << h;
                    if (!issue_pv(h, ch == 0, h == last)) { ok = false; break; }
                }
                if (ch + 1 < cnt) {
                    if (!issue_qk(h, n + ch + 1, h == last)) { ok = false; break; }
                    if (h == last && ch + 2 == chunks) umma_commit_warp(&ms.q_empty);
                }
            }
            if (!ok) break;
            n += chunks;
            tw.advance(sb, units, g);
            ++segs;
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
        umma_commit_warp(&ms.mma_done);  // every MMA is done before TMEM is released
        mbar_wait(&ms.mma_done, 0, nullptr);
        __syncwarp();
    } else if (warp >= 4) {
        // -------------- softmax: one warpgroup per half, one row per thread --------------
        const int h = (warp - 4) >> 2;
        const int quarter = warp & 3;
        const int row = quarter * 32 + lane;
        const uint32_t tS = tmem + ((uint32_t)(quarter * 32) << 16) + h * L::HALF_COLS;
        const uint32_t tO = tS + L::COL_O;
        const float sl2 = a.scale_log2;
        const uint64_t sc2 = f2_pack(sl2, sl2);
        uint32_t gh = 0;  // chunks this half has processed
        while (tw.left > 0 && ok) {
            const ExpandedSegment g = tw.segment();
            const int mine = half_chunks(g, h);
            if (mine == 0) {  // this half has no query rows here, or they see none of the segment's keys
                if (h == 0) {
                    const int slot = latent_slot(c, g.kb == 0);
                    a.ws_ml[(int64_t)slot * kExpQTile + row] = make_float2(-INFINITY, 0.f);
                }
                tw.advance(sb, units, g);
                continue;
            }
            const int ctx = w.q.ctx;
            const int tok = h * 128 + row;  // token inside the tile
            const int64_t pos = (int64_t)(ctx - w.q.q_len) + g.qt * kExpQTile + min(tok, g.tokens - 1);
            const int64_t lim = a.causal ? pos + 1 : ctx;
            float m_ref = -INFINITY, l = 0.f;
            // the exponents of the values of a chunk's four times 32 keys, a byte each, a chunk ahead
            const int32_t *exps = reinterpret_cast<const int32_t *>(a.buf.value_exp) +
                                  (int64_t)g.h * (a.buf.padded / kExpTile) + tw.tiles + g.kb;
            int32_t next_exps = __ldcg(exps);
            for (int ch = 0; ch < mine; ++ch, ++gh) {
                const int32_t chunk_exps = next_exps;
                if (ch + 1 < mine) next_exps = __ldcg(exps + ch + 1);
                if (!wait_all(&ms.s_full[h], gh & 1)) { ok = false; break; }
                tc_fence_after();
                const int vis = (int)max64(0, min64(lim - (int64_t)(g.kb + ch) * kExpTile, kExpTile));
                const bool full = __all_sync(0xffffffffu, vis >= kExpTile);
                // The row's 128 scores in two rounds of 64 columns, against a lazily moved
                // reference maximum; a move in the second round rescales the first round's
                // weights, already in TMEM, and any move rescales O.
                float a_o = 1.f, a_p0 = 1.f;
                bool any_o = false, any_p0 = false;
                uint64_t ps2[2] = {0, 0};
#pragma unroll 1
                for (int r = 0; r < 2; ++r) {
                    uint32_t v[64];
                    float red0, red1;
                    tmem_ld32_max(tS + r * 64, reinterpret_cast<uint32_t(&)[32]>(v[0]), red0);
                    tmem_ld32_max(tS + r * 64 + 32, reinterpret_cast<uint32_t(&)[32]>(v[32]), red1);
                    tmem_wait_ld();
                    reg_order32(reinterpret_cast<uint32_t(&)[32]>(v[0]));
                    reg_order32(reinterpret_cast<uint32_t(&)[32]>(v[32]));
                    if (!full) {
                        float m4[4] = {-INFINITY, -INFINITY, -INFINITY, -INFINITY};
#pragma unroll
                        for (int j = 0; j < 64; ++j)
                            if (r * 64 + j >= vis) v[j] = __float_as_uint(-INFINITY);
#pragma unroll
                        for (int j = 0; j < 64; j += 4)
#pragma unroll
                            for (int k = 0; k < 2; ++k) {
                                float &m = m4[2 * (j / 32) + k];
                                m = fmax3(m, __uint_as_float(v[j + 2 * k]), __uint_as_float(v[j + 2 * k + 1]));
                            }
                        red0 = fmaxf(m4[0], m4[1]);
                        red1 = fmaxf(m4[2], m4[3]);
                    }
                    const int xs[2] = {(int8_t)(chunk_exps >> (16 * r)), (int8_t)(chunk_exps >> (16 * r + 8))};
                    const float x0 = (float)xs[0], x1 = (float)xs[1];
                    const float mx = fmaxf(fmaf(red0, sl2, x0), fmaf(red1, sl2, x1));
                    const bool up = mx > m_ref + kRescaleSlack;
                    if (__any_sync(0xffffffffu, up)) {
                        const float alpha = up ? fast_exp2(m_ref - mx) : 1.f;
                        l *= alpha;
                        ps2[0] = f2_mul(ps2[0], f2_pack(alpha, alpha));
                        ps2[1] = f2_mul(ps2[1], f2_pack(alpha, alpha));
                        a_o *= alpha;
                        any_o = true;
                        if (r > 0) {
                            a_p0 = alpha;
                            any_p0 = true;
                        }
                        if (up) m_ref = mx;
                    }
                    const float base = m_ref == -INFINITY ? 0.f : m_ref - kWeightShift;
#pragma unroll
                    for (int q = 0; q < 2; ++q) {
                        const float b = (q ? x1 : x0) - base, grow = __int_as_float((127 - xs[q]) << 23);  // 2^-x
                        const uint64_t nb2 = f2_pack(b, b);
                        uint64_t gs2[2] = {0, 0};  // the 32 keys' weights
                        uint32_t pk[16];
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const uint64_t y2 = f2_fma(f2_pack(__uint_as_float(v[q * 32 + 2 * j]),
                                                               __uint_as_float(v[q * 32 + 2 * j + 1])),
                                                       sc2, nb2);
                            float y0, y1;
                            f2_unpack(y2, y0, y1);
                            const float e0 = fast_exp2(y0), e1 = fast_exp2(y1);
                            pk[j] = pack_f16x2(e0, e1);
                            gs2[j & 1] = f2_add(gs2[j & 1], f2_pack(e0, e1));
                        }
#pragma unroll
                        for (int k = 0; k < 2; ++k) ps2[k] = f2_fma(gs2[k], f2_pack(grow, grow), ps2[k]);
                        tmem_st16(tS + (2 * r + q) * 16, pk);
                    }
                }
                {
                    float a0, a1, b0, b1;
                    f2_unpack(ps2[0], a0, a1);
                    f2_unpack(ps2[1], b0, b1);
                    l += (a0 + a1) + (b0 + b1);
                }
                if (any_p0) {
                    tmem_wait_st();
#pragma unroll 1
                    for (int q = 0; q < 2; ++q) {
                        uint32_t x[16];
                        tmem_ld16(tS + q * 16, x);
                        tmem_wait_ld();
                        reg_order16(x);
#pragma unroll
                        for (int j = 0; j < 16; ++j) {
                            const float2 p = __half22float2(*reinterpret_cast<const __half2 *>(&x[j]));
                            x[j] = pack_f16x2(p.x * a_p0, p.y * a_p0);
                        }
                        tmem_st16(tS + q * 16, x);
                    }
                }
                if (any_o && ch > 0) {
                    if (!wait_all(&ms.pv_done[h], (gh - 1) & 1)) { ok = false; break; }
                    tc_fence_after();
#pragma unroll 1
                    for (int q = 0; q < kExpHeadDim / 32; ++q) {
                        uint32_t r[32];
                        tmem_ld32(tO + q * 32, r);
                        tmem_wait_ld();
                        reg_order32(r);
#pragma unroll
                        for (int j = 0; j < 32; ++j) r[j] = __float_as_uint(__uint_as_float(r[j]) * a_o);
                        tmem_st32(tO + q * 32, r);
                    }
                }
                tmem_wait_st();
                tc_fence_before();
                __syncwarp();
                if (lane == 0) mbar_arrive(&ms.p_full[h]);
            }
            if (!ok) break;
            // ---- epilogue: O / l of a whole tile, or the part for the merge ----
            if (!wait_all(&ms.pv_done[h], (gh - 1) & 1)) { ok = false; break; }
            tc_fence_after();
            const float inv = g.whole ? 1.f / l : 1.f;
            const int slot = g.whole ? 0 : latent_slot(c, g.kb == 0);
            // 16 rows x 64 columns at a time: four threads have a row's 64 columns, in the order in which
            // the values are stored 16 that belong together each, so a store writes whole lines (with a
            // row a thread the epilogue took twice as long).
            const int part = lane & 3;
#pragma unroll 1
            for (int i = 0; i < 4; ++i) {
                const int q = i >> 1, r0 = (i & 1) * 16 + (lane >> 2);  // rows r0, r0 + 8 of the warp's 32
                uint32_t r[32];
                tmem_ld_16x64(tO + ((uint32_t)((i & 1) * 16) << 16) + q * 64, r);
                tmem_wait_ld();
                reg_order32(r);
#pragma unroll
                for (int k = 0; k < 2; ++k) {
                    const float f = __shfl_sync(0xffffffffu, inv, r0 + 8 * k);
                    const int t = h * 128 + quarter * 32 + r0 + 8 * k;  // token inside the tile
                    if (t >= g.tokens) continue;
                    if (g.whole) {
                        uint32_t x[8];
#pragma unroll
                        for (int j = 0; j < 8; ++j)
                            x[j] = pack_bf16x2(__uint_as_float(r[4 * j + 2 * k]) * f,
                                               __uint_as_float(r[4 * j + 2 * k + 1]) * f);
                        st_global_32(a.out + ((int64_t)(w.q.q0 + g.qt * kExpQTile + t) * a.num_heads + g.h) * kExpHeadDim +
                                         q * 64 + part * 16, x);
                    } else {
                        float *o = a.ws_o + ((int64_t)slot * kExpQTile + t) * kExpHeadDim + q * 64 + part * 16;
#pragma unroll
                        for (int m = 0; m < 2; ++m) {
                            uint32_t x[8];
#pragma unroll
                            for (int j = 0; j < 8; ++j) x[j] = r[4 * (4 * m + j / 2) + 2 * k + j % 2];
                            st_global_32(o + 8 * m, x);
                        }
                    }
                }
                __syncwarp();
            }
            if (!g.whole && tok < g.tokens) a.ws_ml[(int64_t)slot * kExpQTile + tok] = make_float2(m_ref, l);
            tc_fence_before();
            __syncwarp();
            if (lane == 0) mbar_arrive(&ms.o_free[h]);
            tw.advance(sb, units, g);
        }
        if (!ok) {
            if (lane == 0) flag_error(a.err, PKV_DEVERR_TIMEOUT);
            *abort_flag = 1;
        }
    }
    tc_fence_before();
    __syncthreads();
    tc_fence_after();
    if (warp == 1) tmem_dealloc(tmem, 512);
}

void plan_expanded(int num_seqs, int64_t total_context, int num_heads, int sms, ExpandedPlan *p) {
    auto up = [](size_t x) { return (x + 255) / 256 * 256; };
    p->grid = sms;
    // each sequence is padded to whole tiles
    p->padded = (total_context + (int64_t)num_seqs * (kExpTile - 1)) / kExpTile * kExpTile;
    p->off_rope = 0;
    p->off_kv = p->off_rope + up((size_t)p->padded * kExpRope * 2);
    p->off_exp = p->off_kv + up((size_t)num_heads * p->padded * 2 * kExpHeadDim * 2);
    p->off_jobs = p->off_exp + up((size_t)num_heads * p->padded / 32);
    p->off_ml = p->off_jobs + up(sizeof(LatentJob) * (size_t)p->grid);
    p->off_o = p->off_ml + up(2 * (size_t)p->grid * kExpQTile * sizeof(float2));
    p->ws_bytes = p->off_o + up(2 * (size_t)p->grid * kExpQTile * kExpHeadDim * sizeof(float));
}

cudaError_t launch_latent_expanded(const CUtensorMap &q_map, const CUtensorMap &kv_map, const CUtensorMap &rope_map,
                                   const ExpandedArgs &a, cudaStream_t stream) {
    static SmemAllowance allowed;
    cudaError_t e = allow_dynamic_smem(latent_expanded_kernel, ExpandedSmem::BYTES, allowed);
    if (e != cudaSuccess) return e;
    e = launch_pdl(latent_expanded_kernel, dim3(a.grid), dim3(kExpandedThreads), ExpandedSmem::BYTES, stream, q_map,
                   kv_map, rope_map, a);
    if (e != cudaSuccess) return e;
    return launch_latent_merge<kExpHeadDim, kExpQTile, true>(a.ws_jobs, a.ws_ml, a.ws_o, a.out,
                                                       (int64_t)a.num_heads * kExpHeadDim, a.grid, stream);
}

}  // namespace pkv
